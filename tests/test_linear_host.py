"""Linear attention with one decay per head and the query/key norm, without a GPU:
the fp64 plain forms against closed forms and differences, the workspace sizes, and
every refusal of the C entry points and of the binding (nothing is launched)."""
import pytest
import torch

import linear_plain as P
from gated_delta_rule_108_b200 import kda

OK_PTR = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_108_b200 import build
    build.build()
    return kda.lib()


# ------------------------------------------------------------ the plain forms --
def draw(B=2, T=7, H=2, dk=3, dv=4, lens=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    N = B if lens is None else len(lens)
    cu = None if lens is None else torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist())
    return dict(q=r(B, T, H, dk), k=r(B, T, H, dk), v=r(B, T, H, dv), log_decay=-torch.rand(H, generator=g, dtype=torch.float64),
                S0=r(N, H, dk, dv), cu=cu), r(B, T, H, dv), r(N, H, dk, dv)


@pytest.mark.parametrize("lens", [None, (3, 0, 1, 3)], ids=str)
def test_plain_forward_is_the_quadratic_form(lens):
    x, _, _ = draw(B=1 if lens else 2, lens=lens)
    o, S, om, Sm = P.forward(**x)
    t0 = 0
    flat = {n: x[n].reshape(-1, *x[n].shape[2:]) for n in "qkv"}
    for n, L in enumerate(P.lens_of(*x["q"].shape[:2], x["cu"])):
        i = torch.arange(L, dtype=torch.float64)
        lag = i[:, None] - i[None]
        for h in range(2):
            l = x["log_decay"][h]
            q, k, v = (flat[m][t0:t0 + L, h] for m in "qkv")
            D = torch.exp(l * lag) * (lag >= 0)
            ref = 3 ** -0.5 * (((q @ k.T) * D) @ v + torch.exp(l * (i + 1))[:, None] * (q @ x["S0"][n, h]))
            assert torch.allclose(o.reshape(-1, 2, 4)[t0:t0 + L, h], ref, rtol=1e-12, atol=1e-12)
            end = (k * torch.exp(l * (L - 1 - i))[:, None]).T @ v + torch.exp(l * L) * x["S0"][n, h]
            assert torch.allclose(S[n, h], end, rtol=1e-12, atol=1e-12)
        t0 += L
    assert (om >= o.abs() - 1e-12).all() and (Sm >= S.abs() - 1e-12).all()


@pytest.mark.parametrize("lens", [None, (3, 0, 1, 3)], ids=str)
def test_plain_backward_against_differences(lens):
    """L is linear in each input alone: a step of any size changes it by <gradient, step>."""
    x, d_o, dS = draw(B=1 if lens else 2, lens=lens, seed=1)
    g, _ = P.backward(x["q"], x["k"], x["v"], x["log_decay"], d_o, x["S0"], dS, x["cu"])

    def loss(**over):
        o, S, _, _ = P.forward(**{**x, **over})
        return float((o * d_o).sum() + (S * dS).sum())

    gen = torch.Generator().manual_seed(2)
    for n, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("S0", "dS0")):
        for _ in range(3):
            step = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
            diff = (loss(**{n: x[n] + step}) - loss(**{n: x[n] - step})) / 2
            assert abs(diff - float((g[gn] * step).sum())) < 1e-10 * (1 + abs(diff))


@pytest.mark.parametrize("interleaved", [False, True])
def test_plain_rotation(interleaved):
    """A rotation keeps norms, is undone by its inverse, and moves inner products by the positions' difference only."""
    g = torch.Generator().manual_seed(3)
    f = torch.tensor([1.0, 0.3, 0.01, 0.001])
    x, y = (torch.randn(1, 1, 1, 10, generator=g, dtype=torch.float64) for _ in range(2))
    at = lambda t, p: P.rotate(t, torch.tensor([[p]]), f, interleaved)  # noqa: E731
    assert torch.allclose(at(x, 5).norm(), x.norm())
    assert torch.allclose(P.rotate(at(x, 5), torch.tensor([[5]]), f, interleaved, back=True), x)
    assert torch.allclose((at(x, 9) * at(y, 4)).sum(), (at(x, 105) * at(y, 100)).sum())
    assert torch.equal(at(x, 5)[..., 8:], x[..., 8:])


# -------------------------------------------------------------- the C entries --
def test_workspace_sizes(lib):
    f32, bf16 = 0, 1
    for fn in (lib.kda_linear_chunk_fwd_workspace_size, lib.kda_linear_chunk_bwd_workspace_size):
        assert fn(2, 100, 2, 96, 64, 2, 0, f32) == 0          # head size
        assert fn(2, 100, 2, 64, 64, 2, 1, f32) == 0          # packed needs B = 1
        assert fn(1, 1 << 30, 1, 64, 64, 1, 0, bf16) == 0     # too many tokens
        assert fn(1, 100, 2, 64, 64, -1, 1, bf16) == 0
        assert fn(1, 0, 2, 64, 64, 0, 1, bf16) >= 256         # a call without sequences still has a status
        assert fn(8, 128, 32, 128, 128, 8, 0, bf16) == 256    # nothing is cut: the header alone
    for fn in (lib.kda_linear_chunk_fwd_workspace_size, lib.kda_linear_chunk_bwd_workspace_size):
        assert fn(1, 65536, 8, 128, 128, 1, 0, bf16) > 2 * 8 * 128 * 128 * 4   # segments' states
    assert lib.kda_qk_norm_rope_bwd_workspace_size(128) > 0
    assert lib.kda_qk_norm_rope_bwd_workspace_size(12) == 0 and lib.kda_qk_norm_rope_bwd_workspace_size(264) == 0


def fwd(lib, **over):
    a = dict(q=OK_PTR, k=2 * OK_PTR, v=3 * OK_PTR, ld=OK_PTR, s0=None, cu=None, B=1, T=64, H=1, dk=64, dv=64, N=1, dtype=0,
             o=4 * OK_PTR, sf=None, ws=OK_PTR, wsb=1 << 30)
    a.update(over)
    return lib.kda_linear_chunk_fwd(a["q"], a["k"], a["v"], a["ld"], a["s0"], a["cu"], a["B"], a["T"], a["H"], a["dk"], a["dv"],
                                    a["N"], a["dtype"], a["o"], a["sf"], a["ws"], a["wsb"], None)


BAD = [(dict(dk=96), 2), (dict(dv=32), 2), (dict(dtype=7), 1), (dict(q=None), 1), (dict(k=OK_PTR + 4), 1), (dict(H=0), 1),
       (dict(B=-1), 1), (dict(B=2, cu=OK_PTR), 1), (dict(cu=OK_PTR, N=-1), 1), (dict(ws=None, T=6000, dtype=1), 5), (dict(ws=None, cu=OK_PTR), 5), (dict(ws=OK_PTR + 16), 5),
       (dict(wsb=16), 5), (dict(T=1 << 30), 2), (dict(H=70000), 2)]


@pytest.mark.parametrize("over,status", BAD + [
    (dict(o=None), 1), (dict(o=OK_PTR), 1),                            # o over q
    (dict(s0=OK_PTR, sf=OK_PTR + 64), 1), (dict(s0=OK_PTR + 4), 1),
    (dict(o=4 * OK_PTR, s0=4 * OK_PTR + 64), 1), (dict(sf=4 * OK_PTR + 16), 1), (dict(sf=2 * OK_PTR), 1)], ids=str)
def test_forward_refuses(lib, over, status):
    assert fwd(lib, **over) == status
    assert lib.kda_last_error()


@pytest.mark.parametrize("over,status", BAD + [
    (dict(dq=None), 1), (dict(dq=3 * OK_PTR), 1), (dict(dvo=OK_PTR + 8), 1), (dict(s0=OK_PTR, ds0=OK_PTR), 1),
    (dict(dsf=OK_PTR, ds0=OK_PTR + 1024), 1), (dict(dq=6 * OK_PTR + 64), 1), (dict(ds0=7 * OK_PTR), 1), (dict(ds0=OK_PTR), 1),
    (dict(s0=5 * OK_PTR), 1)], ids=str)
def test_backward_refuses(lib, over, status):
    a = dict(q=OK_PTR, k=2 * OK_PTR, v=3 * OK_PTR, ld=None, s0=None, cu=None, do=4 * OK_PTR, dsf=None, B=1, T=64, H=1, dk=64, dv=64,
             N=1, dtype=0, dq=5 * OK_PTR, dko=6 * OK_PTR, dvo=7 * OK_PTR, ds0=None, ws=OK_PTR, wsb=1 << 30)
    a.update(over)
    assert lib.kda_linear_chunk_bwd(a["q"], a["k"], a["v"], a["ld"], a["s0"], a["cu"], a["do"], a["dsf"], a["B"], a["T"], a["H"],
                                    a["dk"], a["dv"], a["N"], a["dtype"], a["dq"], a["dko"], a["dvo"], a["ds0"], a["ws"], a["wsb"],
                                    None) == status
    assert lib.kda_last_error()


@pytest.mark.parametrize("over,status", [(dict(dk=96), 2), (dict(dtype=3), 1), (dict(S=None), 1), (dict(v=OK_PTR + 2), 1),
                                         (dict(B=-1), 1), (dict(o=5 * OK_PTR + 16), 1), (dict(B=1 << 28), 2),
                                         (dict(o=OK_PTR), 1), (dict(o=3 * OK_PTR + 16), 1), (dict(S=2 * OK_PTR), 1)], ids=str)
def test_step_refuses(lib, over, status):
    a = dict(q=OK_PTR, k=2 * OK_PTR, v=3 * OK_PTR, ld=None, S=5 * OK_PTR, B=1, H=1, dk=64, dv=64, dtype=0, o=7 * OK_PTR)
    a.update(over)
    assert lib.kda_linear_recurrent_step(a["q"], a["k"], a["v"], a["ld"], a["S"], a["B"], a["H"], a["dk"], a["dv"], a["dtype"],
                                         a["o"], None) == status
    assert lib.kda_last_error()


def test_hook_arms_and_disarms(lib):
    assert lib.kda_linear_debug_drop_copy(-1) == 1
    assert lib.kda_linear_debug_drop_copy(1000) == 0 and lib.kda_linear_debug_drop_copy(0) == 0


NORM_BAD = [(dict(d=12), 2), (dict(d=264), 2), (dict(rot=24), 2), (dict(rot=80), 2), (dict(dtype=2), 1), (dict(norm=2), 1),
            (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(Hk=0), 1), (dict(q=None), 1),
            (dict(k=OK_PTR + 8), 1), (dict(qs=(64, 64, 62)), 1), (dict(freq=None), 1), (dict(wq=OK_PTR + 4), 1),
            (dict(B=1 << 16, T=1 << 15), 2)]


def norm_call(lib, bwd, **over):
    a = dict(q=OK_PTR, k=2 * OK_PTR, gq=8 * OK_PTR, gk=9 * OK_PTR, wq=None, wk=None, freq=OK_PTR, pos=None, B=1, T=3, Hq=1, Hk=1,
             d=64, rot=64, qs=(192, 64, 64), ks=(192, 64, 64), dtype=0, norm=0, eps=1e-6, oq=3 * OK_PTR, ok=4 * OK_PTR,
             dwq=None, dwk=None, ws=None, wsb=0)
    a.update(over)
    common = (a["wq"], a["wk"], a["freq"], a["pos"], a["B"], a["T"], a["Hq"], a["Hk"], a["d"], a["rot"], *a["qs"], *a["ks"],
              a["dtype"], a["norm"], a["eps"], 0, a["oq"], a["ok"])
    if not bwd:
        return lib.kda_qk_norm_rope(a["q"], a["k"], *common, None)
    return lib.kda_qk_norm_rope_bwd(a["q"], a["k"], a["gq"], a["gk"], *common, a["dwq"], a["dwk"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,status", NORM_BAD + [(dict(oq=OK_PTR + 256), 1), (dict(ok=OK_PTR), 1), (dict(oq=4 * OK_PTR), 1),
                                                    (dict(oq=OK_PTR, qs=(384, 128, 64)), 1)], ids=str)
def test_norm_refuses(lib, over, status):
    assert norm_call(lib, False, **over) == status
    assert lib.kda_last_error()


@pytest.mark.parametrize("over,status", NORM_BAD + [(dict(gq=None), 1), (dict(dwq=OK_PTR), 5), (dict(dwk=OK_PTR, ws=OK_PTR, wsb=64), 5),
                                                    (dict(dwk=OK_PTR, ws=OK_PTR + 16, wsb=1 << 30), 5), (dict(oq=OK_PTR), 1),
                                                    (dict(ok=8 * OK_PTR), 1)], ids=str)
def test_norm_backward_refuses(lib, over, status):
    assert norm_call(lib, True, **over) == status
    assert lib.kda_last_error()


# ---------------------------------------------------------------- the binding --
B, T, H, DK, DV = 2, 10, 3, 64, 32


def lin_args(**over):
    a = dict(q=torch.zeros(B, T, H, DK), k=torch.zeros(B, T, H, DK), v=torch.zeros(B, T, H, DV), log_decay=torch.zeros(H))
    a.update(over)
    return a


@pytest.mark.parametrize("name,bad", [("k", torch.zeros(B, T, H, DV)), ("v", torch.zeros(B, T + 1, H, DV)),
                                      ("log_decay", torch.zeros(H + 1)), ("log_decay", torch.zeros(B, T, H)),
                                      ("initial_state", torch.zeros(B + 1, H, DK, DV)), ("o", torch.zeros(B, T, H, DK)),
                                      ("final_state", torch.zeros(B, H, DV, DK))], ids=str)
def test_binding_refuses_shapes(name, bad):
    with pytest.raises(ValueError, match=name):
        kda.linear_chunk_fwd(**lin_args(**{name: bad}))
    if name not in ("o", "final_state"):
        with pytest.raises(ValueError, match=name):
            kda.linear_chunk_bwd(**lin_args(**{name: bad}), d_o=torch.zeros(B, T, H, DV))


def test_binding_refuses_the_rest():
    with pytest.raises(ValueError, match="d_o"):
        kda.linear_chunk_bwd(**lin_args(), d_o=torch.zeros(B, T, H, DK))
    with pytest.raises(ValueError, match="B == 1"):
        kda.linear_chunk_fwd(**lin_args(), cu_seqlens=torch.tensor([0, 4, 10], dtype=torch.int32))
    with pytest.raises(ValueError, match="q must have 4"):
        kda.linear_chunk_fwd(**lin_args(q=torch.zeros(T, H, DK)))
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.linear_chunk_fwd(**lin_args())
    with pytest.raises(ValueError, match="state"):
        kda.linear_recurrent_step(torch.zeros(B, H, DK), torch.zeros(B, H, DK), torch.zeros(B, H, DV), None, torch.zeros(B, H, DV, DK))
    q, k = torch.zeros(B, T, 4, DK), torch.zeros(B, T, 2, DK)
    for over, match in ((dict(q_weight=torch.zeros(DK + 1)), "q_weight"), (dict(positions=torch.zeros(B, T + 1, dtype=torch.int32)), "positions"),
                        (dict(norm="layer"), "norm"), (dict(q_out=torch.zeros(B, T, 2, DK)), "q_out"),
                        (dict(k=torch.zeros(B, T + 1, 2, DK)), "k must have"), (dict(inv_freq=torch.zeros(2, 2)), "inv_freq"), (dict(), "CUDA tensor")):
        with pytest.raises(ValueError, match=match):
            kda.qk_norm_rope(**{**dict(q=q, k=k), **over})
    with pytest.raises(ValueError, match="positions"):
        kda.qk_norm_rope(q[:, 0], k[:, 0], inv_freq=torch.zeros(32))
    with pytest.raises(ValueError, match="d_k_out"):
        kda.qk_norm_rope_bwd(q, k, q, q)
