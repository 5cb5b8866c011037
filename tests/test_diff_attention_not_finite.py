"""Differential attention where attended scores are not finite: a row with a NaN or +inf score shows it, in its results
and in every gradient that it enters; a key whose score is -inf has no weight."""
import numpy as np
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from oracle import ops
from helpers import f64
from test_diff_attention import draw, on_gpu, step

pytestmark = pytest.mark.gpu

ROWS = [1, 2, 5, 300]  # one query, two (the few-row kernel), five, and tiles


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq", ROWS)
@pytest.mark.parametrize("m", [0, 1])
def test_a_row_with_a_nan(Sq, D, m):
    """A NaN in query row i, in the columns of map m: that map of the row is NaN."""
    H, i = 2, Sq - 1
    x = draw(2, Sq, 400, H, D, "prefix", seed=70 + Sq)
    clean = step(on_gpu(x))
    y = {n: None if t is None else t.clone() for n, t in x.items()}
    y["q"][1, i, 0, m * (D // 2) + 3] = float("nan")
    got = step(on_gpu(y))
    for n in got:
        got[n], clean[n] = got[n].cpu().float(), clean[n].cpu().float()
    assert torch.isnan(got["lse"][1, 0, m, i]) and torch.isnan(got["out"][1, i, 0]).all()
    assert torch.isnan(got["out2"][1, i, 0]).all() == (m == 1)
    cols = slice(m * (D // 2), (m + 1) * (D // 2))
    keys = y["mask"][1]
    assert torch.isnan(got["dq"][1, i, 0, cols]).all()
    assert torch.isnan(got["dk"][1, keys, 0, cols]).all() and torch.isnan(got["dv"][1, keys, 0]).all()
    assert torch.isnan(got["dlam"][0]) == (m == 1)
    # masked keys, the other head, the other sequence and the other rows are what they were
    for n in ("dk", "dv"):
        assert not got[n][1, ~keys].any()
    got["lse"][1, 0, m, i], clean["lse"][1, 0, m, i] = 0, 0
    for n in ("out", "out2", "dq"):
        got[n][1, i, 0], clean[n][1, i, 0] = 0, 0
    for n in ("dk", "dv"):
        got[n][1, :, 0], clean[n][1, :, 0] = 0, 0
    got["dlam"][0], clean["dlam"][0] = 0, 0
    for n in got:
        assert torch.equal(got[n], clean[n]), n


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq", ROWS)
@pytest.mark.parametrize("mask", [None, "prefix"])
def test_rows_with_an_infinite_score(Sq, D, mask):
    """An infinity in a key's columns of map 2.  Queries of one sign there score +inf, lse = +inf and their maps are NaN;
    those of the other score -inf, and their results are those without the key."""
    Sk, at = 300, 17
    x = draw(1, Sq, Sk, 2, D, mask, seed=71 + Sq)
    x["q"][0, :, 0, D // 2] = torch.where(torch.arange(Sq) % 2 == 0, -1.0, 1.0).bfloat16()
    x["q"][0, :, 1, D // 2] = 1.0
    x["k"][0, at, :, D // 2] = float("inf")
    gx = on_gpu(x)
    out, out2, lse = uaa.diff_attn_fwd(gx["q"], gx["k"], gx["v"], gx["lam"], gx["mask"])
    grads = uaa.diff_attn_bwd(gx["q"], gx["k"], gx["v"], gx["lam"], out, out2, gx["do"], lse, gx["mask"])
    uaa.check_device_status()
    o, o2, l2 = (t.cpu().float() for t in (out, out2, lse))
    up = torch.arange(Sq) % 2 == 1
    for h, rows in ((0, up), (1, torch.ones(Sq, dtype=torch.bool))):
        assert torch.isposinf(l2[0, h, 1, rows]).all() and torch.isfinite(l2[0, h, 1, ~rows]).all()
        assert torch.isnan(o[0, rows, h]).all() and torch.isnan(o2[0, rows, h]).all()
        assert torch.isfinite(l2[0, h, 0]).all()
    # without that key in map 2: a column of 1000 there leaves it a weight below e^-100; the error of the 32-bit scores is
    # that of the other keys, whose terms are those of a column of 1 (in `out` it is small beside the rounding to bf16)
    down = (~up).numpy()
    ref, ordinary = ({}, {})
    for res, value in ((ref, 1000.0), (ordinary, 1.0)):
        k = f64(x["k"])[:, :, :1].copy()
        k[0, at, :, D // 2] = value
        res.update(ops.diff_attn(f64(x["q"])[:, down, :1], k, f64(x["v"])[:, :, :1], f64(x["lam"])[:1],
                                 None if mask is None else x["mask"].numpy()))
    for n, got in (("out", o[:, :, :1][:, ~up]), ("out2", o2[:, :, :1][:, ~up]), ("lse", l2[:, :1][..., ~up])):
        bound = ordinary[n][1] if n == "lse" else ref[n][1]
        assert (np.abs(got.double().numpy() - ref[n][0]) <= bound).all(), n
    # every gradient of head 1, all of whose rows are NaN in map 2
    keys = torch.ones(Sk, dtype=torch.bool) if mask is None else x["mask"][0]
    dq, dk, dv, dlam = (t.cpu().float() for t in grads)
    assert torch.isnan(dq[0, :, 1, D // 2:]).all() and torch.isnan(dlam[1])
    assert torch.isnan(dk[0, keys, 1, D // 2:]).all() and torch.isnan(dv[0, keys, 1]).all()


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
