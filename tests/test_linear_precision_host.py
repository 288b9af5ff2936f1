"""The bound on what is kept in fp32 sees a part left out: mistakes planted in the reference, on the CPU."""
import pytest
import torch

import linear_plain as P
from linear_precision import assert_near


def parts_of(x, parts):
    kept, rest = torch.zeros_like(x), x.clone()
    for _ in range(parts):
        p = rest.to(torch.bfloat16).double()
        kept, rest = kept + p, rest - p
    return kept


def draw(T, d=64, seed=0):
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(1, T, 1, d, generator=g).bfloat16() for _ in range(2))
    return k, v, torch.tensor([-0.01])


@pytest.mark.parametrize("T", [63, 128, 300])
def test_a_state_of_two_parts_is_seen(T):
    k, v, l = draw(T)
    _, ref, _, _ = P.forward(k, k, v, l)
    w = torch.exp(l.double() * torch.arange(T - 1, -1, -1)[:, None])
    for parts, seen in ((3, False), (2, True)):
        S = k[0, :, 0].double().T @ parts_of(w * v[0, :, 0].double(), parts)
        if seen:
            with pytest.raises(AssertionError, match="relative error"):
                assert_near(S[None, None], ref, "state")
        else:
            assert_near(S[None, None], ref, "state")


def test_sums_that_are_cut_off_are_seen():
    """16,384 tokens without a decay, added to one running fp32 sum that drops what does not fit."""
    k, v, _ = draw(16384, d=16)
    ref = k[0, :, 0].double().T @ v[0, :, 0].double()

    def cut(x):        # to fp32, towards zero
        y = x.float()
        return torch.where(y.double().abs() > x.abs(), torch.nextafter(y, torch.zeros_like(y)), y).double()

    S = torch.zeros(16, 16, dtype=torch.float64)
    for t in range(0, 16384, 16):       # 16 tokens a step, as the tensor core adds
        S = cut(S + k[0, t:t + 16, 0].double().T @ v[0, t:t + 16, 0].double())
    with pytest.raises(AssertionError, match="relative error"):
        assert_near(S, ref, "state")


@pytest.mark.parametrize("T", [1, 64, 413])
def test_inputs_of_14_bits_are_seen(T):
    g = torch.Generator().manual_seed(T)
    q, k, v = (torch.randn(1, T, 2, 64, generator=g) for _ in range(3))
    l = torch.tensor([-0.1, -0.001])
    o, S, _, _ = P.forward(q, k, v, l)
    cut = lambda x: (x.double() * (1 + 2.0 ** 39) - x.double() * 2.0 ** 39)  # noqa: E731  (keeps 14 bits)
    assert float((cut(q) - q).abs().max() / q.abs().max()) < 2.0 ** -12
    o2, S2, _, _ = P.forward(cut(q), cut(k), cut(v), l)
    for x, ref in ((o2, o), (S2, S)):
        with pytest.raises(AssertionError, match="relative error"):
            assert_near(x, ref, "result")
    assert_near(o.float(), o, "o")
