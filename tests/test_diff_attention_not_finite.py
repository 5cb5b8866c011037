"""Differential attention where attended scores are not finite: a key whose score is -inf has no weight."""
import numpy as np
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from oracle import ops
from helpers import f64
from test_diff_attention import draw, on_gpu

pytestmark = pytest.mark.gpu

ROWS = [1, 2, 5, 300]  # one query, two (the few-row kernel), five, and tiles


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq", ROWS)
def test_every_other_key_without_weight(Sq, D):
    """Half of the keys score -inf in both maps: the results are those of the other half."""
    Sk = 280
    x = draw(1, Sq, Sk, 2, D, None, seed=72 + Sq)
    x["q"][..., 0] = x["q"][..., D // 2] = 1.0
    x["k"][:, ::2, :, 0] = x["k"][:, ::2, :, D // 2] = float("-inf")
    gx = on_gpu(x)
    out, out2, lse = uaa.diff_attn_fwd(gx["q"], gx["k"], gx["v"], gx["lam"])
    uaa.check_device_status()
    ref = ops.diff_attn(f64(x["q"]), f64(x["k"])[:, 1::2], f64(x["v"])[:, 1::2], f64(x["lam"]))
    for n, t in (("out", out), ("out2", out2), ("lse", lse)):
        value, bound = ref[n]
        assert (np.abs(t.cpu().double().numpy() - value) <= bound).all(), n
