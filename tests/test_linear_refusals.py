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
