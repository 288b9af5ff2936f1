"""Linear attention with one fixed decay per head on the GPU: the chunked forward,
its gradients and the single-token step against the fp64 recurrence."""
import time

import pytest
import torch

import linear_plain as P
from gated_delta_rule_108_b200 import kda

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
ids = lambda x: str(x).replace("torch.", "")  # noqa: E731


def decays(kind, H):
    if kind == "none":
        return None
    l = -torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)])
    if kind == "strong":      # up to e^-20 a token, and one head that forgets everything
        l = 20 * l
        l[H - 1] = -float("inf")
    return l


def case(B, T, H, dk, dv, dtype, decay="slopes", lens=None, state=True, seed=0):
    g = torch.Generator().manual_seed(seed)

    def unit(*s):
        x = torch.randn(*s, generator=g)
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype)

    N = B if lens is None else len(lens)
    x = dict(q=unit(B, T, H, dk), k=unit(B, T, H, dk), v=torch.randn(B, T, H, dv, generator=g).to(dtype),
             log_decay=decays(decay, H), initial_state=None, cu_seqlens=None)
    if state:
        x["initial_state"] = 0.3 * torch.randn(N, H, dk, dv, generator=g)
    if lens is not None:
        x["cu_seqlens"] = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
    back = dict(d_o=torch.randn(B, T, H, dv, generator=g).to(dtype),
                d_final_state=0.3 * torch.randn(N, H, dk, dv, generator=g) if state else None)
    return x, back


def dev(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def plain(x):
    return P.forward(x["q"], x["k"], x["v"], x["log_decay"], x["initial_state"], x["cu_seqlens"])


def longest(x):
    B, T = x["q"].shape[:2]
    return max(P.lens_of(B, T, x["cu_seqlens"]) or [0])


def check_fwd(x, o, S):
    ref, Sf, om, Sm = plain(x)
    dt = x["q"].dtype
    P.assert_close(o, ref, om, dt, "o", longest(x))
    P.assert_close(S, Sf, Sm, dt, "final_state", longest(x), state=True)


def check_bwd(x, back, r):
    g, m = P.backward(x["q"], x["k"], x["v"], x["log_decay"], back["d_o"], x["initial_state"], back["d_final_state"],
                      x["cu_seqlens"])
    for n in ("dq", "dk", "dv", "dS0"):
        P.assert_close(r[n], g[n], m[n], x["q"].dtype, n, longest(x), state=n == "dS0")


SHAPES = [(1, 1), (2, 63), (1, 64), (2, 65), (1, 127), (1, 128), (2, 129), (1, 300)]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("dk,dv", [(128, 128), (128, 64), (64, 128), (64, 64)])
@pytest.mark.parametrize("B,T", SHAPES)
def test_forward(cuda_device, B, T, dk, dv, dtype):
    x, _ = case(B, T, 2, dk, dv, dtype, seed=T)
    o, S = kda.linear_chunk_fwd(**dev(x), check=True)
    check_fwd(x, o, S)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("decay", ["slopes", "strong", "none"])
def test_forward_decays(cuda_device, decay, dtype):
    x, _ = case(1, 413, 4, 128, 128, dtype, decay=decay, state=decay != "slopes", seed=5)
    o, S = kda.linear_chunk_fwd(**dev(x), check=True)
    check_fwd(x, o, S)


LENS = [(1, 0, 128, 200, 65), (0, 0, 5), (700, 1, 1, 0), (129,)]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_forward_packed(cuda_device, lens, dtype):
    x, _ = case(1, sum(lens), 3, 128, 64, dtype, lens=lens, seed=6)
    o, S = kda.linear_chunk_fwd(**dev(x), check=True)
    check_fwd(x, o, S)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("B,T,lens", [(1, 700, None), (2, 333, None), (1, 600, (600, 0)), (1, 3001, None), (2, 1500, None), (1, 3100, (2900, 0, 1, 199)), (1, 4000, (1300, 1350, 1350))],
                         ids=str)
def test_segments(cuda_device, B, T, lens, dtype):
    """Few heads and long sequences: cut into segments (a packed batch by its longest sequence)."""
    x, back = case(B, T, 1, 64, 64, dtype, lens=lens, seed=7)
    o, S = kda.linear_chunk_fwd(**dev(x), check=True)
    check_fwd(x, o, S)
    check_bwd(x, back, kda.linear_chunk_bwd(**dev(x), **dev(back), check=True))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("dk,dv", [(128, 128), (128, 64), (64, 128), (64, 64)])
@pytest.mark.parametrize("B,T", [(1, 1), (2, 65), (1, 128), (2, 300)])
def test_backward(cuda_device, B, T, dk, dv, dtype):
    x, back = case(B, T, 2, dk, dv, dtype, seed=20 + T)
    check_bwd(x, back, kda.linear_chunk_bwd(**dev(x), **dev(back), check=True))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("decay", ["strong", "none"])
def test_backward_packed(cuda_device, decay, dtype):
    lens = (1, 0, 128, 200, 65)
    x, back = case(1, sum(lens), 3, 64, 128, dtype, decay=decay, lens=lens, seed=8)
    check_bwd(x, back, kda.linear_chunk_bwd(**dev(x), **dev(back), check=True))
    x["initial_state"], back["d_final_state"] = None, None
    r = kda.linear_chunk_bwd(**dev(x), **dev(back), output_d_initial_state=False)
    assert r.pop("dS0") is None
    full = kda.linear_chunk_bwd(**dev(x), **dev(back))
    for n in r:
        if dtype == torch.float32 or n != "dv":     # dv's update has one part more where dS0 is asked for
            assert torch.equal(r[n], full[n]), n
    check_bwd(x, back, full)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
@pytest.mark.parametrize("T", [2000, 2048])
def test_more_chains_than_sms(cuda_device, T, dk, dv):
    """160 and 480 chains of 16 chunks: segments that follow one another, each from the state of the one before."""
    x, back = case(5, T, 32, dk, dv, torch.bfloat16, seed=T + dk)
    for _ in range(3):          # the flags of the last call do not count
        o, S = kda.linear_chunk_fwd(**dev(x), check=True)
        g = kda.linear_chunk_bwd(**dev(x), **dev(back), check=True)
    S0 = x["initial_state"].cuda()
    o2, S2 = kda.linear_chunk_fwd(**{**dev(x), "initial_state": S0}, final_state=S0)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    for b, h in ((0, 0), (2, 13), (4, 31)):
        one = {n: t[b:b + 1, :, h:h + 1] for n, t in x.items() if n in "qkv"}
        one.update(log_decay=x["log_decay"][h:h + 1], initial_state=x["initial_state"][b:b + 1, h:h + 1], cu_seqlens=None)
        ob = dict(d_o=back["d_o"][b:b + 1, :, h:h + 1], d_final_state=back["d_final_state"][b:b + 1, h:h + 1])
        check_fwd(one, o[b:b + 1, :, h:h + 1], S[b:b + 1, h:h + 1])
        check_bwd(one, ob, {n: (t[b:b + 1, h:h + 1] if n == "dS0" else t[b:b + 1, :, h:h + 1]) for n, t in g.items()})


def test_backward_against_differences(cuda_device):
    """L is linear in each input alone, so a step of any size changes it by <gradient, step>."""
    x, back = case(1, 200, 2, 64, 64, torch.float32, seed=9)
    x, back = dev(x), dev(back)
    g = kda.linear_chunk_bwd(**x, **back)

    def loss(**over):
        o, S = kda.linear_chunk_fwd(**{**x, **over})
        return float((o.double() * back["d_o"]).sum() + (S.double() * back["d_final_state"]).sum())

    gen = torch.Generator(device="cuda").manual_seed(1)
    for n, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("initial_state", "dS0")):
        step = torch.randn(x[n].shape, generator=gen, device="cuda")
        diff = (loss(**{n: x[n] + step}) - loss(**{n: x[n] - step})) / 2
        dot = float((g[gn].double() * step).sum())
        # both sides are sums of products in fp32: n 2^-24 of the products' 2-norm, n = 600 covers all sums here
        scale = float(g[gn].double().norm() * step.double().norm()) + abs(loss())
        assert abs(diff - dot) <= 600 * 2.0 ** -24 * scale, (n, diff, dot)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_other_sequences_do_not_leak(cuda_device, dtype):
    """NaN and infinities of one packed sequence, inside its neighbours' tiles, stay its own."""
    lens = (70, 40, 90)
    x, back = case(1, sum(lens), 2, 128, 128, dtype, lens=lens, seed=10)
    x, back = dev(x), dev(back)
    o, S = kda.linear_chunk_fwd(**x)
    g = kda.linear_chunk_bwd(**x, **back)
    bad = {n: t.clone() for n, t in x.items() if n in ("q", "k", "v")}
    for i, t in enumerate(bad.values()):
        t[:, 70:110] = [float("nan"), float("inf"), -float("inf")][i]
    d_o = back["d_o"].clone()
    d_o[:, 70:110] = float("nan")
    o2, S2 = kda.linear_chunk_fwd(**{**x, **bad})
    g2 = kda.linear_chunk_bwd(**{**x, **bad}, d_o=d_o, d_final_state=back["d_final_state"])
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    keep[70:110] = False
    assert torch.equal(o[:, keep], o2[:, keep]) and torch.equal(S[[0, 2]], S2[[0, 2]])
    for n in ("dq", "dk", "dv"):
        assert torch.equal(g[n][:, keep], g2[n][:, keep]), n
    assert torch.equal(g["dS0"][[0, 2]], g2["dS0"][[0, 2]])


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_state_in_place_and_repeat(cuda_device, dtype):
    """final_state may be initial_state itself; the same call gives the same bits."""
    for T in (200, 700, 3000):      # one segment, a few, many
        x, back = case(1, T, 1, 128, 128, dtype, seed=11)
        x, back = dev(x), dev(back)
        o, S = kda.linear_chunk_fwd(**x)
        S0 = x["initial_state"].clone()
        o2, S2 = kda.linear_chunk_fwd(**{**x, "initial_state": S0}, final_state=S0)
        assert S2.data_ptr() == S0.data_ptr() and torch.equal(o, o2) and torch.equal(S, S2)
        a, b = (kda.linear_chunk_bwd(**x, **back) for _ in range(2))
        assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_without_a_workspace(cuda_device, dtype):
    """Where the workspace holds nothing but the status, there may be none."""
    for T in (0, 100):
        x, back = case(2, T, 2, 128, 64, dtype, seed=19)
        assert kda.linear_chunk_fwd_workspace_size(2, T, 2, 128, 64, 2, False, dtype) == 256
        a, b = (kda.linear_chunk_fwd(**dev(x), check=c) for c in (False, True))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        a, b = (kda.linear_chunk_bwd(**dev(x), **dev(back), check=c) for c in (False, True))
        assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_no_tokens(cuda_device, dtype):
    x, back = case(2, 0, 2, 128, 64, dtype, seed=12)
    o, S = kda.linear_chunk_fwd(**dev(x), check=True)
    assert o.shape == (2, 0, 2, 64) and torch.equal(S.cpu(), x["initial_state"])
    r = kda.linear_chunk_bwd(**dev(x), **dev(back), check=True)
    assert torch.equal(r["dS0"].cpu(), back["d_final_state"])
    x, _ = case(0, 5, 2, 128, 64, dtype, seed=12)
    o, S = kda.linear_chunk_fwd(**dev(x), check=True)
    assert o.numel() == 0 and S.numel() == 0


@pytest.mark.parametrize("cu", [[0, 50, 40, 90], [1, 50, 60, 90], [0, 50, 60, 91], [0, -3, 60, 90], [0, 2 ** 31 - 1, 60, 90]],
                         ids=str)
def test_bad_cu_seqlens(cuda_device, cu):
    x, back = case(1, 90, 2, 128, 128, torch.bfloat16, lens=(30, 30, 30), seed=13)
    x, back = dev(x), dev(back)
    x["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, S = torch.full((1, 90, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((3, 2, 128, 128), 7.0, device="cuda")
    with pytest.raises(kda.KDAError, match="BAD_SEQLENS"):
        kda.linear_chunk_fwd(**x, o=o, final_state=S, check=True)
    assert bool((o == 7).all()) and bool((S == 7).all())
    with pytest.raises(kda.KDAError, match="BAD_SEQLENS"):
        kda.linear_chunk_bwd(**x, **back, check=True)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("dk,dv", [(128, 128), (128, 64), (64, 128), (64, 64)])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 5), (100, 8)])
def test_step(cuda_device, B, H, dk, dv, dtype):
    for kind in ("slopes", "strong", "none"):
        x, _ = case(B, 3, H, dk, dv, dtype, decay=kind, seed=14)
        d = dev(x)
        S = d["initial_state"].clone()
        o = torch.stack([kda.linear_recurrent_step(*(d[n][:, t].contiguous() for n in "qkv"), d["log_decay"], S)
                         for t in range(3)], 1)
        ref, Sf, om, Sm = plain(x)
        # each state element is one rounded product and sum a token, each output a sum of dk products
        assert ((S.cpu().double() - Sf).abs() <= 3 * 4 * 2.0 ** -24 * Sm + 1e-30).all()
        half = torch.finfo(dtype).eps / 2
        assert ((o.cpu().double() - ref).abs() <= half * ref.abs() + (dk + 16) * 2.0 ** -24 * om + 1e-30).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_prompt_then_steps(cuda_device, dtype):
    """A prompt by chunks, then tokens one by one, is the whole sequence at once."""
    x, _ = case(2, 140, 3, 128, 128, dtype, seed=15)
    d = dev(x)
    cut = {n: d[n][:, :133].contiguous() for n in "qkv"}
    _, S = kda.linear_chunk_fwd(**cut, log_decay=d["log_decay"], initial_state=d["initial_state"])
    o = [kda.linear_recurrent_step(*(d[n][:, t].contiguous() for n in "qkv"), d["log_decay"], S) for t in range(133, 140)]
    ref, Sf, om, Sm = plain(x)
    P.assert_close(torch.stack(o, 1), ref[:, 133:], om[:, 133:], dtype, "o", 140)
    P.assert_close(S, Sf, Sm, dtype, "state", 140, state=True)


@pytest.mark.parametrize("B,T,H,dtype", [(1, 2100, 2, torch.bfloat16), (1, 2100, 2, torch.float32), (1, 2300, 50, torch.bfloat16),
                                         (1, 100, 2, torch.bfloat16)], ids=str)
def test_side_stream_and_graph(cuda_device, B, T, H, dtype):
    x, back = case(B, T, H, 128, 128, dtype, seed=16)
    x, back = dev(x), dev(back)
    o, S = kda.linear_chunk_fwd(**x)
    g = kda.linear_chunk_bwd(**x, **back)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, S2 = kda.linear_chunk_fwd(**x, stream=side)
    g2 = kda.linear_chunk_bwd(**x, **back, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(S, S2) and all(torch.equal(g[n], g2[n]) for n in g)

    static = {n: t.clone() for n, t in x.items() if t is not None}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, Sg = kda.linear_chunk_fwd(**static)
        gg = kda.linear_chunk_bwd(**static, **back)
        step = kda.linear_recurrent_step(*(static[n][:, 0].contiguous() for n in "qkv"), static["log_decay"], Sg)
    for scale in (1.0, 2.0):
        static["v"].copy_(x["v"] * scale)
        graph.replay()
        torch.cuda.synchronize()
        oe, Se = kda.linear_chunk_fwd(**{**x, "v": x["v"] * scale})
        ge = kda.linear_chunk_bwd(**{**x, "v": x["v"] * scale}, **back)
        te = kda.linear_recurrent_step(*(static[n][:, 0].contiguous() for n in "qkv"), static["log_decay"], Se)
        assert torch.equal(og, oe) and torch.equal(Sg, Se) and torch.equal(step, te)
        assert all(torch.equal(gg[n], ge[n]) for n in gg)


def test_more_than_32_sequences(cuda_device):
    """A long one among 40 short: ordered, cut and checked by the whole block."""
    lens = [30 + i for i in range(20)] + [3000] + [0, 1] + [50 - i for i in range(18)]
    x, back = case(1, sum(lens), 1, 64, 64, torch.bfloat16, lens=lens, seed=27)
    o, S = kda.linear_chunk_fwd(**dev(x), check=True)
    check_fwd(x, o, S)
    check_bwd(x, back, kda.linear_chunk_bwd(**dev(x), **dev(back), check=True))
    d = dev(x)
    for at, value in ((0, 1), (41, sum(lens) + 1), (7, 2 ** 31 - 1), (9, -5), (30, 2000)):
        cu = x["cu_seqlens"].clone()
        cu[at] = value
        o, S = torch.full_like(o, 7.0), torch.full_like(S, 7.0)
        with pytest.raises(kda.KDAError, match="BAD_SEQLENS"):
            kda.linear_chunk_fwd(**{**d, "cu_seqlens": cu.cuda()}, o=o, final_state=S, check=True)
        assert bool((o == 7).all()) and bool((S == 7).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_two_streams_at_once(cuda_device, dtype):
    """Calls that overlap, each with its own workspace."""
    cases = [case(2, 900 + 100 * i, 3, 128, 128, dtype, seed=30 + i) for i in range(2)]
    ins = [(dev(x), dev(back)) for x, back in cases]
    ref = [(kda.linear_chunk_fwd(**x), kda.linear_chunk_bwd(**x, **b)) for x, b in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = []
    for _ in range(5):
        for s, (x, b) in zip(streams, ins):
            got.append((kda.linear_chunk_fwd(**x, stream=s), kda.linear_chunk_bwd(**x, **b, stream=s)))
    torch.cuda.synchronize()
    for i, ((o, S), g) in enumerate(got):
        (ro, rS), rg = ref[i % 2]
        assert torch.equal(o, ro) and torch.equal(S, rS) and all(torch.equal(g[n], rg[n]) for n in g)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_nan_decay_stays_with_its_head(cuda_device, dtype):
    """Nothing waits or skips on it: the call ends, and the other heads are as they were."""
    x, back = case(1, 3000, 3, 64, 64, dtype, seed=21)
    x, back = dev(x), dev(back)
    o, S = kda.linear_chunk_fwd(**x, check=True)
    g = kda.linear_chunk_bwd(**x, **back, check=True)
    x["log_decay"][1] = float("nan")
    o2, S2 = kda.linear_chunk_fwd(**x, check=True)
    g2 = kda.linear_chunk_bwd(**x, **back, check=True)
    keep = [0, 2]
    assert torch.equal(o[:, :, keep], o2[:, :, keep]) and torch.equal(S[:, keep], S2[:, keep])
    assert all(torch.equal(g[n][:, :, keep], g2[n][:, :, keep]) for n in ("dq", "dk", "dv"))


def test_many_short_sequences(cuda_device):
    """1500 packed sequences of 0 to 5 tokens."""
    lens = [int(n) for n in torch.randint(0, 6, (1500,), generator=torch.Generator().manual_seed(3))]
    for dtype in DTYPES:
        x, back = case(1, sum(lens), 1, 64, 64, dtype, lens=lens, seed=22)
        o, S = kda.linear_chunk_fwd(**dev(x), check=True)
        check_fwd(x, o, S)
        check_bwd(x, back, kda.linear_chunk_bwd(**dev(x), **dev(back), check=True))


@pytest.mark.parametrize("T,H,dk,dv,dtype,lens", [(1500, 60, 64, 64, torch.bfloat16, None), (1409, 60, 64, 64, torch.bfloat16, None),
                                                  (1500, 60, 64, 64, torch.float32, None), (1500, 30, 64, 128, torch.float32, None),
                                                  (1700, 60, 64, 64, torch.bfloat16, (1600, 0, 100))], ids=str)
@pytest.mark.parametrize("decay", ["slopes", "strong", "none"])
def test_segments_summed_in_pieces(cuda_device, T, H, dk, dv, dtype, lens, decay):
    """60 chains (20 heads for the gradients): two segments, the sum in two pieces; packed, one of the batch's three is cut."""
    N = 1 if lens is None else len(lens)
    slots = lambda size: (size - 256) / (H * dk * dv * 4)  # noqa: E731
    assert slots(kda.linear_chunk_fwd_workspace_size(1, T, H, dk, dv, N, lens is not None, dtype)) >= 4
    x, _ = case(1, T, H, dk, dv, dtype, decay=decay, lens=lens, seed=25)
    o, S = kda.linear_chunk_fwd(**dev(x), check=True)
    check_fwd(x, o, S)
    x, back = case(1, T, H // 3, dk, dv, dtype, decay=decay, lens=lens, seed=26)
    check_bwd(x, back, kda.linear_chunk_bwd(**dev(x), **dev(back), check=True))


def test_offsets_past_31_bits(cuda_device):
    """q, k, v and o of more than 2^31 elements each: the short sequence behind the long one, and the norm there."""
    lens, H, d = (524300, 200), 32, 128
    T = sum(lens)
    assert lens[0] * H * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(23)
    q, k, v, d_o = (torch.randn(1, T, H, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    cu = torch.tensor([0, lens[0], T], dtype=torch.int32, device="cuda")
    qn, kn = kda.qk_norm_rope(q, k, inv_freq=torch.ones(16, device="cuda"))
    pos = torch.arange(T - 200, T, dtype=torch.int32, device="cuda")[None]
    part = kda.qk_norm_rope(q[:, -200:], k[:, -200:], inv_freq=torch.ones(16, device="cuda"), positions=pos)
    assert torch.equal(qn[:, -200:], part[0]) and torch.equal(kn[:, -200:], part[1])
    del q, k, part
    log_decay = decays("slopes", H)
    o, S = kda.linear_chunk_fwd(qn, kn, v, log_decay.cuda(), cu_seqlens=cu, check=True)
    r = kda.linear_chunk_bwd(qn, kn, v, log_decay.cuda(), d_o, cu_seqlens=cu, check=True)
    for h in (0, H - 1):
        tail = lambda t: t[:, -200:, h:h + 1].cpu()  # noqa: E731
        x = dict(q=tail(qn), k=tail(kn), v=tail(v), log_decay=log_decay[h:h + 1], initial_state=None, cu_seqlens=None)
        check_fwd(x, tail(o), S[1:, h:h + 1].cpu())
        back = dict(d_o=tail(d_o), d_final_state=torch.zeros(1, 1, d, d))
        check_bwd(x, back, {**{n: tail(r[n]) for n in ("dq", "dk", "dv")}, "dS0": r["dS0"][1:, h:h + 1].cpu()})


@pytest.mark.parametrize("B,H", [(37, 16), (74, 8), (9, 32)])
def test_step_slices(cuda_device, B, H):
    """Around 592 pairs: states cut into slices of columns, and whole ones."""
    x, _ = case(B, 1, H, 128, 128, torch.bfloat16, seed=24)
    d = dev(x)
    S = d["initial_state"].clone()
    o = kda.linear_recurrent_step(*(d[n][:, 0] for n in "qkv"), d["log_decay"], S)
    few, Sf = [], []
    for b in range(B):      # every sequence by itself
        s = d["initial_state"][b:b + 1].clone()
        few.append(kda.linear_recurrent_step(*(d[n][b:b + 1, 0] for n in "qkv"), d["log_decay"], s))
        Sf.append(s)
    assert torch.equal(S, torch.cat(Sf))
    # sums over the same products in another order: dk roundings of the largest partial sum
    _, _, om, _ = plain(x)
    assert ((o - torch.cat(few)).abs().cpu().double() <= 2.0 ** -7 * o.abs().cpu().double() + 144 * 2.0 ** -24 * om[:, 0]).all()


def test_training_shape_sampled(cuda_device):
    """B=4, T=4096, H=16, bf16: two (sequence, head) pairs of the forward and the gradients."""
    x, back = case(4, 4096, 16, 128, 128, torch.bfloat16, seed=17)
    o, S = kda.linear_chunk_fwd(**dev(x), check=True)
    g = kda.linear_chunk_bwd(**dev(x), **dev(back), check=True)
    for b, h in ((0, 0), (3, 15)):
        one = {n: t[b:b + 1, :, h:h + 1] for n, t in x.items() if n in "qkv"}
        one.update(log_decay=x["log_decay"][h:h + 1], initial_state=x["initial_state"][b:b + 1, h:h + 1], cu_seqlens=None)
        ob = dict(d_o=back["d_o"][b:b + 1, :, h:h + 1], d_final_state=back["d_final_state"][b:b + 1, h:h + 1])
        check_fwd(one, o[b:b + 1, :, h:h + 1], S[b:b + 1, h:h + 1])
        check_bwd(one, ob, {n: (t[b:b + 1, h:h + 1] if n == "dS0" else t[b:b + 1, :, h:h + 1]) for n, t in g.items()})


@pytest.mark.parametrize("B,T,H", [(1, 100, 2), (3, 380, 50), (5, 2048, 32)])
def test_missing_copy_reports_timeout_then_recovers(cuda_device, B, T, H):
    """A wait that can never end gives up: one chunk, several, segments that wait for one another."""
    x, _ = case(B, T, H, 128, 64, torch.bfloat16, seed=18)
    d = dev(x)
    ws = torch.empty(kda.linear_chunk_fwd_workspace_size(B, T, H, 128, 64, B, False, torch.bfloat16), dtype=torch.uint8, device="cuda")
    o, S = kda.linear_chunk_fwd(**d, workspace=ws)
    assert kda.workspace_status(ws) == 0
    kda.linear_debug_drop_copy(4_000_000)     # about 2 ms
    t0 = time.perf_counter()
    kda.linear_chunk_fwd(**d, workspace=ws)
    assert kda.workspace_status(ws) == 4      # KDA_ERR_TIMEOUT
    assert time.perf_counter() - t0 < 1.0
    o2, S2 = kda.linear_chunk_fwd(**d, workspace=ws, check=True)
    assert torch.equal(o, o2) and torch.equal(S, S2)
