"""The norm's weight gradients over long batches."""
import pytest
import torch

from gated_delta_rule_108_b200 import kda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,d,dtype", [(400_000, 8, 256, torch.bfloat16), (100_000, 12, 64, torch.float32)], ids=str)
def test_weight_gradients_of_equal_rows(cuda_device, T, H, d, dtype):
    """Every row the same, so every sum adds one number over and over and rounds the same way:
    the error grows with the terms of a run, not with the batch.

    A run is cut after 64 terms and one token's heads: 64 + 2 H additions, 2^-24 of the sum each.
    A term itself: the sum of squares (8 products a lane, 5 joins), its root (half of that and two
    units in the last place), four products: 16 of 2^-24; the sum of each CTA is rounded once."""
    g = torch.Generator(device="cuda").manual_seed(d)
    rows = [torch.randn(d, generator=g, device="cuda").to(dtype) for _ in range(4)]
    q, k = (r.expand(1, T, H, d) for r in rows[:2])
    dq, dk = (r.expand(1, T, H, d).contiguous() for r in rows[2:])
    w = torch.ones(d, device="cuda")
    r = kda.qk_norm_rope_bwd(q, k, dq, dk, w, w, norm="rms")
    for x, y, n in ((rows[0], rows[2], "dq_weight"), (rows[1], rows[3], "dk_weight")):
        x, y = x.double(), y.double()
        ref = T * H * y * x * (x.square().mean() + 1e-6).rsqrt()
        off = ((r[n].double() - ref).abs() / ref.abs()).max()
        assert float(off) <= (64 + 2 * H + 18) * 2.0 ** -24, (n, float(off) * 2 ** 24)


def test_weight_gradients_of_a_long_batch(cuda_device):
    """Independent rows, 10^5 tokens, against the sums in fp64."""
    T, H, d = 100_000, 4, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, dq, dk = (torch.randn(1, T, H, d, generator=g, device="cuda") for _ in range(4))
    w = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    r = kda.qk_norm_rope_bwd(q, k, dq, dk, w, w, norm="l2")
    for x, y, n in ((q, dq, "dq_weight"), (k, dk, "dk_weight")):
        terms = y.double() * x.double() * (x.double().square().sum(-1, keepdim=True) + 1e-6).rsqrt()
        ref, mag = terms.sum((0, 1, 2)), terms.abs().sum((0, 1, 2))
        assert ((r[n].double() - ref).abs() <= (64 + 2 * H + 18) * 2.0 ** -24 * mag).all(), n
