"""Norm of queries and keys per head with the position rotation on the GPU, forward
and backward, against fp64; and a run of the operators together."""
import pytest
import torch

import linear_plain as P
from gated_delta_rule_108_b200 import kda
from oracle import oracle as orc

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
ids = lambda x: str(x).replace("torch.", "")  # noqa: E731


def case(B, T, Hq, Hk, d, rot, dtype, weights=True, far=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(B, T, Hq + 2 * Hk, d, generator=g) * (0.3 + torch.rand(d, generator=g))).to(dtype)
    x = dict(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hk], q_weight=None, k_weight=None, inv_freq=None, positions=None)
    if weights:
        x["q_weight"], x["k_weight"] = 1 + 0.2 * torch.randn(d, generator=g), 1 + 0.2 * torch.randn(d, generator=g)
    if rot:
        x["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()
        if far:
            x["positions"] = torch.randint(-5, 2 ** 31 - 1, (B, T), generator=g, dtype=torch.int32)
    dy = torch.randn(B, T, Hq, d, generator=g).to(dtype), torch.randn(B, T, Hk, d, generator=g).to(dtype)
    return x, dy, qkv


def dev(x, qkv):
    """On the GPU, queries and keys still slices of the joint projection."""
    Hq, Hk = x["q"].shape[2], x["k"].shape[2]
    joint = qkv.cuda()
    r = {n: None if t is None else t.cuda() for n, t in x.items()}
    return {**r, "q": joint[:, :, :Hq], "k": joint[:, :, Hq:Hq + Hk]}


def positions(x):
    B, T = x["q"].shape[:2]
    return x["positions"] if x["positions"] is not None else torch.arange(T).expand(B, T)


def reference(x, norm, eps, interleaved):
    return [P.norm_rope(x[n], x[n + "_weight"], x["inv_freq"], positions(x), norm, eps, interleaved) for n in "qk"]


def gradients(x, dy, norm, eps, interleaved):
    leaves = {n: None if t is None else t.double().requires_grad_() for n, t in x.items() if n not in ("inv_freq", "positions")}
    y = reference({**x, **leaves}, norm, eps, interleaved)
    sum((a * b.double()).sum() for a, b in zip(y, dy)).backward()
    return {"dq": leaves["q"].grad, "dk": leaves["k"].grad,
            "dq_weight": None if x["q_weight"] is None else leaves["q_weight"].grad,
            "dk_weight": None if x["k_weight"] is None else leaves["k_weight"].grad}


def close(y, ref, scale, dtype, what, n):
    """n fp32 roundings of magnitude `scale`, then one of the result to dtype."""
    y = y.double().cpu()
    half = 0.0 if dtype == torch.float32 else 2.0 ** -8
    bad = ~((y - ref).abs() <= half * ref.abs() + n * 2.0 ** -24 * scale + 1e-30)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}"


def row_max(t):
    return t.abs().amax(-1, keepdim=True)


def check(x, y, norm, eps, interleaved):
    # the sum of d squares is off by d / 8 + 5 roundings (halved by the root), root, products and rotation add 8, the
    # angle's own rounding pi 2^-24 of the pair, sincospi's 2 more: 48 covers d <= 256
    for n, a, b in zip("qk", y, reference(x, norm, eps, interleaved)):
        close(a, b, row_max(b), x[n].dtype, n, 48)


SIZES = [(1, 1, 1, 1, 128, 128), (2, 5, 4, 2, 64, 32), (1, 37, 3, 1, 80, 80), (1, 9, 2, 2, 96, 0), (2, 130, 8, 2, 128, 64),
         (1, 3, 5, 1, 256, 256), (1, 2, 1, 3, 8, 0), (1, 6, 2, 1, 16, 16), (1, 700, 16, 4, 128, 128), (1, 4, 2, 2, 192, 176)]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("norm,interleaved,weights", [("rms", False, True), ("l2", True, False), ("l2", False, True), ("rms", True, True)])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(cuda_device, size, norm, interleaved, weights, dtype):
    x, _, qkv = case(*size, dtype, weights=weights, seed=sum(size))
    y = kda.qk_norm_rope(**dev(x, qkv), norm=norm, eps=1e-5, interleaved=interleaved)
    check(x, y, norm, 1e-5, interleaved)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("norm,interleaved,weights", [("rms", False, True), ("l2", True, False), ("l2", False, True), ("rms", True, True)])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(cuda_device, size, norm, interleaved, weights, dtype):
    x, dy, qkv = case(*size, dtype, weights=weights, seed=sum(size) + 1)
    r = kda.qk_norm_rope_bwd(**{**dev(x, qkv)}, d_q_out=dy[0].cuda(), d_k_out=dy[1].cuda(), norm=norm, eps=1e-5,
                             interleaved=interleaved)
    ref = gradients(x, dy, norm, 1e-5, interleaved)
    for n, g in (("q", dy[0]), ("k", dy[1])):
        xx, w = x[n].double(), 1.0 if x[n + "_weight"] is None else x[n + "_weight"].double()
        m = xx.square().sum(-1, keepdim=True) / (xx.shape[-1] if norm == "rms" else 1) + 1e-5
        # both terms of dx scale with r |g w|; two row sums of d terms each
        h = (g.double().norm(dim=-1, keepdim=True) * (w.abs().max() if torch.is_tensor(w) else w)) / m.sqrt()
        close(r["d" + n], ref["d" + n], h, x[n].dtype, "d" + n, 96)
        if weights:
            # a sum over tokens and heads of products g r x: fp32 lanes of at most 64 terms, then trees and fp64
            scale = (g.double().norm(dim=-1, keepdim=True) * xx.abs() / m.sqrt()).flatten(0, 2).sum(0)
            close(r[f"d{n}_weight"], ref[f"d{n}_weight"], scale, torch.float32, f"d{n}_weight", 128)
        else:
            assert r[f"d{n}_weight"] is None


def test_backward_against_differences(cuda_device):
    x, dy, qkv = case(2, 9, 3, 2, 64, 32, torch.float32, far=False, seed=3)
    x = dev(x, qkv)
    dy = [t.cuda() for t in dy]
    g = kda.qk_norm_rope_bwd(**x, d_q_out=dy[0], d_k_out=dy[1], norm="rms")

    def loss(**over):
        y = kda.qk_norm_rope(**{**x, **over}, norm="rms")
        return float(sum((a.double() * b).sum() for a, b in zip(y, dy)))

    gen = torch.Generator(device="cuda").manual_seed(1)
    for n in ("q", "k", "q_weight", "k_weight"):
        step = torch.randn(x[n].shape, generator=gen, device="cuda")
        h = 2.0 ** -7
        diff = (loss(**{n: x[n] + h * step}) - loss(**{n: x[n] - h * step})) / (2 * h)
        dot = float((g["d" + n].double() * step).sum())
        # the difference's own error: h^2 / 6 of third derivatives (below 30 |g| |step|^3 a row here) and
        # 2^-24 of the loss's terms over h
        scale = float(g["d" + n].double().norm() * step.double().norm())
        assert abs(diff - dot) <= 5e-3 * scale + 1e-2, (n, diff, dot)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_single_tokens_in_place_and_zeros(cuda_device, dtype):
    x, _, qkv = case(6, 1, 4, 2, 128, 128, dtype, seed=4)
    x["q"][2] = 0                                   # a row of zeros gives zeros
    qkv[2, :, :4] = 0
    d = dev(x, qkv)
    y = kda.qk_norm_rope(**d, norm="l2")
    check(x, y, "l2", 1e-6, False)
    assert not y[0][2].any()
    one = {**d, "q": d["q"][:, 0], "k": d["k"][:, 0], "positions": d["positions"][:, 0].contiguous()}
    z = kda.qk_norm_rope(**one, norm="l2")
    assert torch.equal(z[0], y[0][:, 0]) and torch.equal(z[1], y[1][:, 0])
    q, k = one["q"].contiguous(), one["k"].contiguous()
    w = kda.qk_norm_rope(**{**one, "q": q, "k": k}, norm="l2", q_out=q, k_out=k)
    assert w[0] is q and torch.equal(q, z[0]) and torch.equal(k, z[1])


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_own_positions_and_no_tokens(cuda_device, dtype):
    x, dy, qkv = case(2, 33, 2, 1, 64, 64, dtype, far=False, seed=5)
    y = kda.qk_norm_rope(**dev(x, qkv))
    check(x, y, "l2", 1e-6, False)
    x, dy, qkv = case(2, 0, 2, 1, 64, 64, dtype, far=False, seed=5)
    assert kda.qk_norm_rope(**dev(x, qkv))[0].shape == (2, 0, 2, 64)
    r = kda.qk_norm_rope_bwd(**dev(x, qkv), d_q_out=dy[0].cuda(), d_k_out=dy[1].cuda())
    assert not r["dq_weight"].any() and not r["dk_weight"].any()


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_shared_heads_and_positions_below_zero(cuda_device, dtype):
    """Keys of one head, and queries of one batch row, seen by all (strides of zero)."""
    x, dy, qkv = case(3, 17, 4, 2, 64, 32, dtype, seed=8)
    x["positions"] = -torch.arange(3 * 17, dtype=torch.int32).view(3, 17) * 1000
    x["k"], x["q"] = x["k"][:, :, :1].expand(3, 17, 2, 64), x["q"][:1].expand(3, 17, 4, 64)
    d = {n: None if t is None else t.cuda() for n, t in x.items()}
    joint = qkv.cuda()
    d["k"], d["q"] = joint[:, :, 4:5].expand(3, 17, 2, 64), joint[:1, :, :4].expand(3, 17, 4, 64)
    assert d["k"].stride(2) == 0 and d["q"].stride(0) == 0
    check(x, kda.qk_norm_rope(**d), "l2", 1e-6, False)
    flat = {**d, "q": d["q"].contiguous(), "k": d["k"].contiguous()}
    r = kda.qk_norm_rope_bwd(**d, d_q_out=dy[0].cuda(), d_k_out=dy[1].cuda())
    f = kda.qk_norm_rope_bwd(**flat, d_q_out=dy[0].cuda(), d_k_out=dy[1].cuda())
    assert all(torch.equal(r[n], f[n]) for n in r)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("interleaved", [False, True])
def test_bad_rows_stay_their_own(cuda_device, dtype, interleaved):
    """NaN and infinities of one head of one token reach no other row."""
    x, dy, qkv = case(2, 40, 3, 2, 128, 64, dtype, seed=9)
    d, dy = dev(x, qkv), [t.cuda() for t in dy]
    kw = dict(d_q_out=dy[0], d_k_out=dy[1], interleaved=interleaved)
    y, r = kda.qk_norm_rope(**d, interleaved=interleaved), kda.qk_norm_rope_bwd(**d, **kw)
    bad = qkv.clone()
    bad[1, 7, 1] = float("nan")
    bad[0, 3, 4, 5] = float("inf")
    b = dev(x, bad)
    y2, r2 = kda.qk_norm_rope(**b, interleaved=interleaved), kda.qk_norm_rope_bwd(**b, **kw)
    keep_q, keep_k = (torch.ones(2, 40, n, dtype=torch.bool, device="cuda") for n in (3, 2))
    keep_q[1, 7, 1] = keep_k[0, 3, 1] = False
    for a, c in ((y, y2), ((r["dq"], r["dk"]), (r2["dq"], r2["dk"]))):
        assert torch.equal(a[0][keep_q], c[0][keep_q]) and torch.equal(a[1][keep_k], c[1][keep_k])


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_two_streams_and_two_graphs(cuda_device, dtype):
    """Calls that overlap, each with a workspace of its own, and two captured calls that share one, in turn."""
    cases = [case(1, 500 + 100 * i, 4, 2, 128, 128, dtype, seed=10 + i) for i in range(2)]
    ins = [({**dev(x, qkv)}, dict(d_q_out=dy[0].cuda(), d_k_out=dy[1].cuda())) for x, dy, qkv in cases]
    ref = [kda.qk_norm_rope_bwd(**d, **g) for d, g in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [kda.qk_norm_rope_bwd(**d, **g, stream=s) for _ in range(5) for s, (d, g) in zip(streams, ins)]
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(r[n], ref[i % 2][n]) for n in r)
    ws = torch.empty(kda.lib().kda_qk_norm_rope_bwd_workspace_size(128), dtype=torch.uint8, device="cuda")
    graphs, outs = [torch.cuda.CUDAGraph() for _ in ins], []
    for graph, (d, g) in zip(graphs, ins):
        with torch.cuda.graph(graph):
            outs.append(kda.qk_norm_rope_bwd(**d, **g, workspace=ws))
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for r, e in zip(outs, ref):
        assert all(torch.equal(r[n], e[n]) for n in r)


def test_only_one_weight(cuda_device):
    x, dy, qkv = case(1, 50, 2, 2, 64, 0, torch.float32, seed=6)
    x["q_weight"] = None
    r = kda.qk_norm_rope_bwd(**dev(x, qkv), d_q_out=dy[0].cuda(), d_k_out=dy[1].cuda())
    ref = gradients(x, dy, "l2", 1e-6, False)
    assert r["dq_weight"] is None
    assert float((r["dk_weight"].cpu() - ref["dk_weight"]).norm()) <= 1e-5 * float(ref["dk_weight"].norm())


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_side_stream_and_graph(cuda_device, dtype):
    x, dy, qkv = case(2, 300, 4, 2, 128, 64, dtype, seed=7)
    d, dy = dev(x, qkv), [t.cuda() for t in dy]
    y = kda.qk_norm_rope(**d)
    r = kda.qk_norm_rope_bwd(**d, d_q_out=dy[0], d_k_out=dy[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2 = kda.qk_norm_rope(**d, stream=side)
    r2 = kda.qk_norm_rope_bwd(**d, d_q_out=dy[0], d_k_out=dy[1], stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3 = kda.qk_norm_rope(**d)
        r3 = kda.qk_norm_rope_bwd(**d, d_q_out=dy[0], d_k_out=dy[1])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a in (y2, y3):
        assert torch.equal(a[0], y[0]) and torch.equal(a[1], y[1])
    for a in (r2, r3):
        assert all(torch.equal(a[n], r[n]) for n in r)


def test_norm_then_linear_attention(cuda_device):
    """A layer: joint projection -> norm and rotation -> chunked attention over a prompt -> single tokens,
    and the gradients of the prompt's part, against the same in fp64."""
    B, T, H, d, more = 2, 150, 3, 128, 3
    x, _, qkv = case(B, T + more, H, H, d, 64, torch.bfloat16, far=False, seed=8)
    joint = qkv.cuda()
    q, k, v = joint[:, :T, :H], joint[:, :T, H:2 * H], joint[:, :T, 2 * H:].contiguous()
    args = dict(q_weight=x["q_weight"].cuda(), k_weight=x["k_weight"].cuda(), inv_freq=x["inv_freq"].cuda(), norm="rms")
    l = torch.tensor([-0.5, -0.05, -0.005])
    qn, kn = kda.qk_norm_rope(q, k, **args)
    o, S = kda.linear_chunk_fwd(qn, kn, v, l.cuda(), check=True)
    outs = [o]
    for t in range(T, T + more):
        pos = torch.full((B,), t, dtype=torch.int32, device="cuda")
        qt, kt = kda.qk_norm_rope(joint[:, t, :H], joint[:, t, H:2 * H], positions=pos, **args)
        outs.append(kda.linear_recurrent_step(qt, kt, joint[:, t, 2 * H:].contiguous(), l.cuda(), S)[:, None])
    # the same from the kernels' own rounded queries and keys, and end to end
    xq, xk = (P.norm_rope(x[n], x[n + "_weight"], x["inv_freq"], positions(x), "rms", 1e-6, False) for n in "qk")
    ref, Sf, om, Sm = P.forward(xq, xk, qkv[:, :, 2 * H:], l)
    y = torch.cat(outs, 1).double().cpu()
    # queries and keys are rounded to bf16 once more: sqrt(2) of uniform errors of 2^-8 / sqrt(3) on top of o's two
    assert float((y - ref).norm() / ref.norm()) <= 2 * 2.0 ** -8 / 3 ** 0.5 * 1.2
    d_o = torch.randn(B, T, H, d, generator=torch.Generator().manual_seed(2)).bfloat16()
    g = kda.linear_chunk_bwd(qn, kn, v, l.cuda(), d_o.cuda())
    r = kda.qk_norm_rope_bwd(q, k, g["dq"], g["dk"], **args)
    leaves = {n: x[n][:, :T].double().requires_grad_() for n in "qk"}
    ws = {n: x[n + "_weight"].double().requires_grad_() for n in "qk"}
    yq, yk = (P.norm_rope(leaves[n], ws[n], x["inv_freq"], positions(x)[:, :T], "rms", 1e-6, False) for n in "qk")
    lag = torch.arange(T)[:, None] - torch.arange(T)[None]
    D = torch.exp(l.double()[:, None, None] * lag.clamp(min=0)) * (lag >= 0)
    A = torch.einsum("bthi,bshi->bhts", yq, yk) * D
    out = d ** -0.5 * torch.einsum("bhts,bshj->bthj", A, qkv[:, :T, 2 * H:].double())
    (out * d_o.double()).sum().backward()
    for n in "qk":
        for a, b in ((r["d" + n], leaves[n].grad), (r[f"d{n}_weight"], ws[n].grad)):
            # roundings to bf16 on the way: queries, keys, the gradients between the two calls and the result, and the
            # operands inside: six of 2^-8 / sqrt(3)
            assert float((a.double().cpu() - b).norm() / b.norm()) <= 6 ** 0.5 * 2.0 ** -8 / 3 ** 0.5 * 1.2, n


def test_norm_then_delta_rule(cuda_device):
    """Unit queries and keys straight into the delta rule's chunked forward."""
    B, T, H, d = 1, 100, 2, 128
    x, _, qkv = case(B, T, H, H, d, 0, torch.bfloat16, weights=False, seed=9)
    g = torch.Generator().manual_seed(10)
    la, beta = -torch.exp(torch.randn(B, T, H, d, generator=g)) / 16, torch.sigmoid(torch.randn(B, T, H, generator=g))
    dq = dev(x, qkv)
    qn, kn = kda.qk_norm_rope(dq["q"], dq["k"])
    v = qkv[:, :, 2 * H:].contiguous()
    o, S = kda.chunk_fwd(qn, kn, v.cuda(), la.cuda(), beta.cuda(), check=True)
    ref, Sf = orc.kda_forward(qn.cpu(), kn.cpu(), v, la, beta, None)
    ref = torch.as_tensor(ref)
    assert float((o.double().cpu() - ref).norm() / ref.norm()) <= 5e-3
