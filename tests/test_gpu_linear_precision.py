"""How exact the linear attention with one decay per head is, where the tests of its
results leave room: outputs that cancel against what they are summed from, states and
fp32 results in 2-norm, sums over a long sequence."""
import pytest
import torch

import linear_plain as P
from gated_delta_rule_108_b200 import kda
from linear_precision import assert_near
from test_gpu_linear import DTYPES, case, check_bwd, check_fwd, ids

pytestmark = pytest.mark.gpu


def dev(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def along(g, B, T, H, d, axis, c):
    """Unit rows around one channel pattern: `axis` (+1 or -1) names one of two orthogonal ones."""
    base = torch.ones(d)
    base[d // 2:] = axis
    x = base * d ** -0.5 + c * torch.randn(B, T, H, d, generator=g) * d ** -0.5
    return (x / x.norm(dim=-1, keepdim=True)).bfloat16()


def cancelling(B, T, H, dk, dv, c, decay, lens=None, seed=0):
    """Keys and queries around orthogonal directions, values and cotangents likewise: every
    output reads a state from a direction in which it holds little."""
    g = torch.Generator().manual_seed(seed)
    N = B if lens is None else len(lens)
    l = None if decay is None else torch.full((H,), decay)
    row = lambda d, axis: torch.cat((torch.ones(d // 2), axis * torch.ones(d - d // 2))) * d ** -0.5  # noqa: E731
    S0 = (8 * row(dk, 1)[:, None] * row(dv, 1)[None]).expand(N, H, dk, dv) + 0.01 * torch.randn(N, H, dk, dv, generator=g)
    dS = (8 * row(dk, -1)[:, None] * row(dv, -1)[None]).expand(N, H, dk, dv) + 0.01 * torch.randn(N, H, dk, dv, generator=g)
    x = dict(q=along(g, B, T, H, dk, -1, c), k=along(g, B, T, H, dk, 1, c), v=along(g, B, T, H, dv, 1, c), log_decay=l,
             initial_state=S0.contiguous(),
             cu_seqlens=None if lens is None else torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32))
    return x, dict(d_o=along(g, B, T, H, dv, -1, c), d_final_state=dS.contiguous())


def check_output(x, ref, mag, what, tokens):
    """bf16 outputs: their own rounding, and of the magnitudes summed what two bf16 parts of
    P, of the state and of the update's operand leave out, 2^-16 each, besides the fp32 sums'
    part (see linear_plain.assert_close)."""
    x, ref, mag = x.double().cpu(), ref.double(), mag.double()
    n = 2 * (300 + 24 * -(-tokens // 128)) * 2.0 ** -24 + 2.0 ** -22
    tol = (2.0 ** -8 + 2.0 ** -14) * ref.abs() + (3 * 2.0 ** -16 + n) * mag
    bad = ~((x - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, first at {bad.nonzero()[0].tolist()}, "
                           f"relative error {float((x - ref).norm() / ref.norm()):.2e}")


@pytest.mark.parametrize("c", [1.0, 0.3, 0.1])
@pytest.mark.parametrize("B,T,H,dk,dv,decay,lens", [
    (1, 300, 2, 128, 128, None, None), (2, 129, 1, 64, 64, -0.01, None), (1, 200, 2, 128, 64, None, None),
    (1, 260, 2, 64, 128, -0.001, None), (1, 1500, 1, 128, 128, None, None), (1, 3000, 1, 64, 64, -0.0005, None),
    (1, 700, 1, 128, 128, None, (1, 420, 0, 279))], ids=str)
def test_reads_that_cancel(cuda_device, B, T, H, dk, dv, decay, lens, c):
    x, back = cancelling(B, T, H, dk, dv, c, decay, lens, seed=T)
    longest = max(P.lens_of(B, T, x["cu_seqlens"]))
    ref, _, om, _ = P.forward(x["q"], x["k"], x["v"], x["log_decay"], x["initial_state"], x["cu_seqlens"])
    o, _ = kda.linear_chunk_fwd(**dev(x), check=True)
    check_output(o, ref, om, "o", longest)
    g, m = P.backward(x["q"], x["k"], x["v"], x["log_decay"], back["d_o"], x["initial_state"], back["d_final_state"],
                      x["cu_seqlens"])
    r = kda.linear_chunk_bwd(**dev(x), **dev(back), check=True)
    for n in ("dq", "dk", "dv"):
        check_output(r[n], g[n], m[n], n, longest)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("B,T,H,lens", [(2, 300, 2, None), (1, 3000, 1, None), (1, 1500, 60, None), (5, 2048, 32, None),
                                        (1, 700, 1, (1, 420, 0, 279))], ids=str)
def test_no_output_depends_on_another_being_asked_for(cuda_device, B, T, H, lens, dtype):
    """One segment, many, some summed in pieces, some that follow one another, packed."""
    g = torch.Generator(device="cuda").manual_seed(T)
    d = 64 if H > 2 else 128
    q, k, v, d_o = (torch.randn(B, T, H, d, generator=g, device="cuda").to(dtype) for _ in range(4))
    l = -torch.rand(H, generator=g, device="cuda")
    cu = None if lens is None else torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    o, S = kda.linear_chunk_fwd(q, k, v, l, cu_seqlens=cu)
    alone, none = kda.linear_chunk_fwd(q, k, v, l, cu_seqlens=cu, output_final_state=False)
    assert none is None and torch.equal(o, alone)
    full = kda.linear_chunk_bwd(q, k, v, l, d_o, cu_seqlens=cu)
    r = kda.linear_chunk_bwd(q, k, v, l, d_o, cu_seqlens=cu, output_d_initial_state=False)
    assert r["dS0"] is None and all(torch.equal(r[n], full[n]) for n in ("dq", "dk", "dv"))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("decay", ["slopes", "strong", "none"])
@pytest.mark.parametrize("T,dk,dv,lens", [(63, 128, 128, None), (128, 64, 128, None), (300, 128, 64, None), (413, 128, 128, None),
                                          (1500, 64, 64, None), (700, 64, 128, (1, 420, 0, 279))], ids=str)
def test_results_in_norm(cuda_device, T, dk, dv, lens, decay, dtype):
    x, back = case(1, T, 2, dk, dv, dtype, decay=decay, lens=lens, seed=40 + T)
    o, S = kda.linear_chunk_fwd(**dev(x), check=True)
    ref, Sf, _, _ = P.forward(x["q"], x["k"], x["v"], x["log_decay"], x["initial_state"], x["cu_seqlens"])
    assert_near(o, ref, "o", dtype)
    assert_near(S, Sf, "final_state")
    r = kda.linear_chunk_bwd(**dev(x), **dev(back), check=True)
    g, _ = P.backward(x["q"], x["k"], x["v"], x["log_decay"], back["d_o"], x["initial_state"], back["d_final_state"],
                      x["cu_seqlens"])
    for n in ("dq", "dk", "dv"):
        assert_near(r[n], g[n], n, dtype)
    assert_near(r["dS0"], g["dS0"], "dS0")


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("H,d", [(1, 128), (140, 64)])
def test_states_of_long_sequences(cuda_device, H, d, dtype):
    """16,384 tokens without a decay, one head (cut into segments) and as many as SMs (128 chunks
    in a row): the states are plain sums of products."""
    T = 16384
    g = torch.Generator(device="cuda").manual_seed(50)
    q, k, v, d_o = (torch.randn(1, T, H, d, generator=g, device="cuda").to(dtype) for _ in range(4))
    _, S = kda.linear_chunk_fwd(q, k, v, None, check=True)
    r = kda.linear_chunk_bwd(q, k, v, None, d_o, check=True)
    for h in sorted({0, H // 2, H - 1}):
        heads = [t[0, :, h].double() for t in (q, k, v, d_o)]
        assert_near(S[0, h], heads[1].T @ heads[2], "final_state")
        assert_near(r["dS0"][0, h], d ** -0.5 * heads[0].T @ heads[3], "dS0")


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("decay", ["slopes", "strong", "none"])
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 64)])
@pytest.mark.parametrize("lens", [None, (3000, 0, 1, 99)], ids=str)
def test_scanned_segments(cuda_device, lens, dk, dv, decay, dtype):
    """More than eight segments a sequence, forward and backward: several heads, unequal head sizes, initial states."""
    T, H, N = 3100, 2, 1 if lens is None else len(lens)
    for size, roles in ((kda.linear_chunk_fwd_workspace_size, 1), (kda.linear_chunk_bwd_workspace_size, 3)):
        slots = (size(1, T, H, dk, dv, N, lens is not None, dtype) - 256) // (H * dk * dv * 4 * roles)
        assert slots - (0 if lens is None else N) >= (9 if lens is None else 8)      # packed: one more than that per sequence
    x, back = case(1, T, H, dk, dv, dtype, decay=decay, lens=lens, seed=60)
    o, S = kda.linear_chunk_fwd(**dev(x), check=True)
    check_fwd(x, o, S)
    assert_near(S, P.forward(x["q"], x["k"], x["v"], x["log_decay"], x["initial_state"], x["cu_seqlens"])[1], "final_state")
    r = kda.linear_chunk_bwd(**dev(x), **dev(back), check=True)
    check_bwd(x, back, r)


@pytest.mark.parametrize("lens", [None, (1500, 1600)], ids=str)
def test_scanned_segments_of_many_heads(cuda_device, lens):
    """Seven heads that decay at seven rates."""
    x, back = case(1, 3100, 7, 64, 128, torch.bfloat16, decay="strong", lens=lens, seed=61)
    x["log_decay"][-1] = -0.3
    o, S = kda.linear_chunk_fwd(**dev(x), check=True)
    check_fwd(x, o, S)
    check_bwd(x, back, kda.linear_chunk_bwd(**dev(x), **dev(back), check=True))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("T,decay", [(100, "slopes"), (128, "none"), (300, "strong")])
def test_products_that_no_output_holds_may_overflow(cuda_device, T, decay, dtype):
    """A query against a later key, a cotangent against a later value: beyond fp32's range, and not part of any result."""
    x, back = case(1, T, 2, 64, 128, dtype, decay=decay, seed=90)
    x["initial_state"][:, :, 0], back["d_final_state"][:, :, 0] = 0, 0
    x["q"][..., 0], x["k"][..., 0] = 0, 0
    x["q"][:, 3, :, 0], x["k"][:, 20, :, 0] = 1e30, 1e30
    back["d_o"][:, 5, :, 0], x["v"][:, 25, :, 0] = 1e30, 1e30
    o, S = kda.linear_chunk_fwd(**dev(x), check=True)
    r = kda.linear_chunk_bwd(**dev(x), **dev(back), check=True)
    assert all(bool(t.isfinite().all()) for t in (o, S, *r.values()))
    # As linear_plain.assert_close, and what falls below fp32's normal numbers: a weight lambda^n or
    # an element of P below 2^-126 may be off by that much, so an output by 2^-126 of the products that
    # its weights would leave whole (the magnitudes without a decay) and of the row of c that P meets.
    q, k, v, d_o = (t.double().abs() for t in (x["q"], x["k"], x["v"], back["d_o"]))
    whole = lambda c: c.sum(1, keepdim=True).expand_as(c)  # noqa: E731
    args = x["q"], x["k"], x["v"]
    ref, Sf, om, Sm = P.forward(*args, x["log_decay"], x["initial_state"])
    _, _, ou, Su = P.forward(*args, None, x["initial_state"])
    g, m = P.backward(*args, x["log_decay"], back["d_o"], x["initial_state"], back["d_final_state"])
    _, u = P.backward(*args, None, back["d_o"], x["initial_state"], back["d_final_state"])
    n = 2 * (300 + 24 * -(-T // 128)) * 2.0 ** -24 + 2.0 ** -22
    for name, y, ref, mag, under, rounded in (
            ("o", o, ref, om, ou + whole(v), True), ("final_state", S, Sf, Sm, Su, False),
            ("dq", r["dq"], g["dq"], m["dq"], u["dq"] + whole(k), True), ("dk", r["dk"], g["dk"], m["dk"], u["dk"] + whole(q), True),
            ("dv", r["dv"], g["dv"], m["dv"], u["dv"] + whole(d_o), True), ("dS0", r["dS0"], g["dS0"], m["dS0"], u["dS0"], False)):
        tol = n * mag + 2.0 ** -126 * under + 1e-30
        if rounded and dtype == torch.bfloat16:
            tol = tol + (2.0 ** -8 + 2.0 ** -14) * ref.abs() + 3 * 2.0 ** -16 * mag
        bad = ~((y.double().cpu() - ref).abs() <= tol)
        assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} beyond the bound, first at {bad.nonzero()[0].tolist()}"


def unlucky(n, lo=1e-6, hi=3e-6):
    """A slow decay whose power e^(l n) lies as far as it can between two fp32 numbers."""
    l = -torch.linspace(lo, hi, 20001, dtype=torch.float64).float()
    e = (l.double() * n).exp()
    return float(l[((e.float().double() - e) / e).abs().argmax()])


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("T,H", [(65536, 4), (16384, 140)])
def test_slow_decays_over_long_sequences(cuda_device, T, H, dtype):
    """What a chunk leaves of a state is a power below one, taken hundreds of times: its rounding must not add up."""
    d, N = 64, torch.arange(T, device="cuda", dtype=torch.float64)
    g = torch.Generator(device="cuda").manual_seed(95)
    q, k, v, d_o = (torch.randn(1, T, H, d, generator=g, device="cuda").to(dtype) for _ in range(4))
    S0, dS = (T ** 0.5 * torch.randn(1, H, d, d, generator=g, device="cuda") for _ in range(2))
    slow = [unlucky(64), unlucky(128), unlucky(768), unlucky(1024)]
    l = torch.tensor([slow[h % 4] for h in range(H)], device="cuda")
    _, S = kda.linear_chunk_fwd(q, k, v, l, S0, check=True)
    r = kda.linear_chunk_bwd(q, k, v, l, d_o, S0, dS, check=True)
    for h in range(4):
        qh, kh, vh, oh = (t[0, :, h].double() for t in (q, k, v, d_o))
        power = lambda n: (l[h].double() * n).exp()  # noqa: E731
        assert_near(S[0, h], power(T) * S0[0, h].double() + (power(T - 1 - N)[:, None] * kh).T @ vh, f"final_state {h}")
        assert_near(r["dS0"][0, h], power(T) * dS[0, h].double() + d ** -0.5 * (power(N + 1)[:, None] * qh).T @ oh, f"dS0 {h}")


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
def test_slow_decays_over_many_steps(cuda_device, dk, dv):
    """20,000 tokens without input.  An element is rounded once a token, 2^-24 of it at most, and the
    same way for as long as its mantissa hardly moves, so an element may be off by n times that.  But
    elements round either way: what all of them lose alike, the decay's own error, is that divided by
    sqrt(3) and the root of their number, five times over, and 2^-23 of every |l| for the decay."""
    H, n = 4, 20000
    l = torch.tensor([unlucky(1), unlucky(1, 1e-5, 3e-5), unlucky(1, 1e-4, 3e-4), -2.0 ** -8], device="cuda")
    S = torch.randn(2, H, dk, dv, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    ref = (l.double() * n).exp()[:, None, None] * S.double()
    zero = torch.zeros(2, H, dk, device="cuda")
    v, o = torch.ones(2, H, dv, device="cuda"), torch.empty(2, H, dv, device="cuda")
    for _ in range(n):
        kda.linear_recurrent_step(zero, zero, v, l, S, o=o)
    for h in range(H):
        off, r, own = S[:, h].double() - ref[:, h], ref[:, h], n * abs(float(l[h])) * 2.0 ** -23
        assert bool((off.abs() <= (n * 2.0 ** -24 + own) * r.abs() + n * 2.0 ** -149).all()), h
        common = float((off * r).sum() / r.square().sum())
        assert abs(common) <= 5 * n * 2.0 ** -24 / (3 * r.numel()) ** 0.5 + own, (h, common)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
def test_slow_decays_over_steps_with_input(cuda_device, dk, dv):
    """5,000 tokens: every one moves each element by a random amount, so its roundings (two a token,
    2^-24 / sqrt(3) of the state each) are independent; twice what they add up to."""
    H, n = 2, 5000
    g = torch.Generator(device="cuda").manual_seed(2)
    l = torch.tensor([unlucky(1), unlucky(1, 1e-5, 3e-5)], device="cuda")
    S = 8 * torch.randn(2, H, dk, dv, generator=g, device="cuda")
    ref, e, o = S.double(), l.double().exp()[:, None, None], torch.empty(2, H, dv, device="cuda")
    for _ in range(n):
        k, v = (torch.randn(2, H, d, generator=g, device="cuda") for d in (dk, dv))
        kda.linear_recurrent_step(k, k, v, l, S, o=o)
        ref = e * ref + k.double()[..., :, None] * v.double()[..., None, :]
    for h in range(H):
        rel = float((S[:, h].double() - ref[:, h]).norm() / ref[:, h].norm())
        assert rel <= 2 * (2 * n) ** 0.5 * 2.0 ** -24 / 3 ** 0.5, (h, rel)
