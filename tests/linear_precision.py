"""How far results of the linear attention with one decay per head may be off in 2-norm,
where the reference does not cancel (independent random inputs)."""
import torch


def assert_near(x, ref, what, rounded=None):
    """Relative error in 2-norm: 1e-6 for what is kept in fp32, and for what is rounded to
    bf16 at the end (`rounded`) that rounding besides.

    fp32: a chunk's sum is built in 24 steps, each cut off below 2^-23 of the running sum:
    half of that on average, times 0.72 (the mean of 1 / mantissa) and 0.7 (the running sum
    against the whole): 7e-7, if all of it fell the same way.  Chunks add up independently,
    values and errors alike.  Each chunk's sum enters the state with one rounding, 2^-24 /
    sqrt(3), whose errors of n chunks grow to sqrt(n / 2) of that: 3e-7 after 128.  Sums of
    rounded products on CUDA cores, 48 in a row for each lane: sqrt(48) 2^-24 / sqrt(3), 2.4e-7;
    the decays' powers and the weights add 2^-24 each.  Together below 1e-6.
    A bf16 rounding is uniform within half a step: at most 2^-8 / sqrt(3) of the value, reached
    where every mantissa is 1; P, state and update's operand in two parts stay below 2^-14.
    """
    x, ref = x.double().cpu(), ref.double().cpu()
    assert x.shape == ref.shape, what
    rel = float((x - ref).norm() / ref.norm())
    tol = 1e-6 if rounded != torch.bfloat16 else 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -14
    assert rel <= tol, f"{what}: relative error {rel:.2e}, at most {tol:.2e}"
