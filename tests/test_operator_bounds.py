"""The error that the definition of differential attention allows its kernels: no more than their roundings make."""
import numpy as np

from oracle import ops


def test_lse_and_dlambda_are_held_to_32_bits():
    rng = np.random.default_rng(5)
    q, k, v, g = (rng.standard_normal((1, n, 3, 128)) for n in (300, 400, 400, 300))
    lam = np.array([0.5, 1e-30, 0.0])
    res = ops.diff_attn(q, k, v, lam, dout=g)
    assert (res["lse"][1] < 5e-5).all()  # a score's sum of 64 terms, and a sum of 400 probabilities
    value, bound = res["dlam"]
    sums = bound - ops.BF16 * np.abs(value)  # beside dlambda's own rounding
    # with lambda too small for dS_2 the rounding of O_2 to bf16 stays in
    assert sums[0] < sums[1] / 30 and sums[0] < sums[2] / 30
    # as a sum of 128 000 probabilities that adds one after the other: 2^-24 each
    assert ops.norm_error(128000) > 128000 / 16 * 2.0 ** -24
