"""Refusals of the linear attention and the norm that need no GPU: nothing is launched."""
import pytest

from gated_delta_rule_108_b200 import kda

P = 1 << 20
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_108_b200 import build
    build.build()
    return kda.lib()


def norm_call(lib, bwd, **over):
    a = dict(q=P, k=2 * P, gq=8 * P, gk=9 * P, wq=None, wk=None, freq=P, pos=None, B=2, T=3, Hq=4, Hk=4, d=64, rot=64,
             qs=(768, 256, 64), ks=(768, 256, 64), oq=3 * P, ok=4 * P, dwq=None, dwk=None, ws=None, wsb=0)
    a.update(over)
    common = (a["wq"], a["wk"], a["freq"], a["pos"], a["B"], a["T"], a["Hq"], a["Hk"], a["d"], a["rot"], *a["qs"], *a["ks"],
              0, 0, 1e-6, 0, a["oq"], a["ok"])
    if not bwd:
        return lib.kda_qk_norm_rope(a["q"], a["k"], *common, None)
    return lib.kda_qk_norm_rope_bwd(a["q"], a["k"], a["gq"], a["gk"], *common, a["dwq"], a["dwk"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("side", ["qs", "ks"])
@pytest.mark.parametrize("strides", [(768, 256, 1 << 62), (768, 256, -(1 << 62)), (768, 256, -(1 << 63)), (768, 1 << 62, 64),
                                     (1 << 62, 256, 64), (-(1 << 63), 256, 64), (768, 256, 1 << 29)], ids=str)
def test_strides_whose_products_wrap(lib, strides, side, bwd):
    """Refused, not cut down to what is left of them in fewer bits."""
    assert norm_call(lib, bwd, **{side: strides}) == UNSUPPORTED
    assert lib.kda_last_error()


@pytest.mark.parametrize("over", [dict(oq=P, wq=P + 256), dict(wk=3 * P + 512), dict(pos=4 * P + 4), dict(freq=3 * P),
                                  dict(ok=8 * P, oq=9 * P, wq=8 * P + 64)], ids=str)
def test_norm_refuses_outputs_over_what_is_shared(lib, over):
    assert norm_call(lib, False, **{**dict(q=P << 6, k=2 * P << 6), **over}) == INVALID
    assert b"overlaps a weight" in lib.kda_last_error()


SUMS = dict(wq=20 * P, wk=21 * P, dwq=22 * P, dwk=23 * P, ws=24 * P, wsb=P, freq=30 * P)


@pytest.mark.parametrize("over", [dict(dwk=22 * P + 128), dict(dwq=20 * P), dict(dwk=20 * P + 16), dict(dwq=24 * P + 256), dict(dwk=P),
                                  dict(dwq=3 * P), dict(dwk=8 * P + 64), dict(ws=9 * P), dict(ws=2 * P), dict(ws=21 * P), dict(dwq=30 * P),
                                  dict(pos=22 * P), dict(dwq=None, ws=23 * P)], ids=str)
def test_norm_refuses_weight_gradients_over_another_tensor(lib, over):
    assert norm_call(lib, True, **{**SUMS, **over}) == INVALID
    assert b"weight gradient or the workspace overlaps" in lib.kda_last_error()


@pytest.mark.parametrize("over", [dict(ld=4 * P + 64), dict(cu=4 * P, B=1), dict(ws=P), dict(ws=4 * P), dict(ws=5 * P), dict(ws=7 * P),
                                  dict(sf=9 * P), dict(cu=5 * P, B=1), dict(ws=9 * P + 256, ld=9 * P + 384)], ids=str)
def test_forward_refuses_outputs_over_the_rest(lib, over):
    a = dict(ld=9 * P, s0=7 * P, cu=None, B=2, T=64, N=2, dtype=0, sf=5 * P, ws=11 * P)
    a.update(over)
    status = lib.kda_linear_chunk_fwd(P, 2 * P, 3 * P, a["ld"], a["s0"], a["cu"], a["B"], a["T"], 1, 64, 64, a["N"], a["dtype"], 4 * P,
                                      a["sf"], a["ws"], P, None)
    assert status == INVALID and b"overlaps an input" in lib.kda_last_error()


@pytest.mark.parametrize("over", [dict(ld=6 * P), dict(cu=7 * P, B=1), dict(ws=P), dict(ws=4 * P), dict(ws=8 * P), dict(ds0=12 * P),
                                  dict(ds0=13 * P), dict(ws=13 * P)], ids=str)
def test_backward_refuses_gradients_over_the_rest(lib, over):
    a = dict(ld=13 * P, dsf=12 * P, cu=None, B=2, N=2, ds0=8 * P, ws=11 * P)
    a.update(over)
    status = lib.kda_linear_chunk_bwd(P, 2 * P, 3 * P, a["ld"], None, a["cu"], 4 * P, a["dsf"], a["B"], 64, 1, 64, 64, a["N"], 0, 5 * P,
                                      6 * P, 7 * P, a["ds0"], a["ws"], P, None)
    assert status == INVALID and b"overlaps an input" in lib.kda_last_error()


@pytest.mark.parametrize("over", [dict(ld=7 * P), dict(ld=5 * P + 1024)], ids=str)
def test_step_refuses_outputs_over_the_decays(lib, over):
    a = dict(ld=9 * P)
    a.update(over)
    assert lib.kda_linear_recurrent_step(P, 2 * P, 3 * P, a["ld"], 5 * P, 1, 1, 64, 64, 0, 7 * P, None) == INVALID
    assert b"overlaps" in lib.kda_last_error()
