"""Gradients of packed attention where queries read few keys: there Delta = rowsum(P dP) is as large as dP, and what it is
off by shows in dS = P (dP - Delta).

The tolerance, by mean squares.  A value rounded to bf16 is off by at most half a step, evenly spread: 2^-8 / sqrt(3) of its
binade's lowest value, so with mantissas x in [1, 2) of density 1 / (x ln 2) the mean square is (2^-8)^2 / 3 times the
integral of 1 / (x^3 ln 2), 3 / (8 ln 2), which is (0.4247 * 2^-8)^2 of the value's.  dQ and dK have two such roundings, of
dS and of the result: sqrt(2) * 0.4247 * 2^-8 = 0.00235.  A tenth more is for samples that are not spread like that.  (With
the roundings of P and of out within Delta = dout . out the kernels had 0.0037 for two tokens and 0.0027 for forty, causal.)
"""
import numpy as np
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from test_packed_attention import ALL, DEV, against, check, draw, step
from test_packed_gradients import mean_error

RMS = 1.1 * 2 ** 0.5 * 0.4247 * 2.0 ** -8


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hk,D", [(8, 4, 128), (6, 2, 64), (5, 1, 128)])
@pytest.mark.parametrize("n", [2, 3, 5, 9, 17, 40, 100, 128, 200])
def test_mean_error(n, Hq, Hk, D, causal):
    lens = [n] * max(4, 1200 // n)
    x = draw(lens, lens, Hq, Hk, D, seed=60 + n)
    got, want = step(x, causal), against(x, causal)
    check(got, want, ALL)
    for name in ("dq", "dk"):
        off = mean_error(got[name].cpu().double().numpy(), want[name][0])
        assert off <= RMS, (name, off)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,D", [(8, 4, 128), (6, 2, 64), (4, 4, 64)])
@pytest.mark.parametrize("cut", [(100, 60), (1, 90), (128, 128), (1, 1), (40, 300)])
def test_keys_in_pieces(cut, Hq, Hk, D):
    """The keys of a sequence in two calls, each with the out and lse of all of them: the gradients of the queries add up,
    those of the keys are the whole's."""
    n, m = 150, sum(cut)
    x = draw([n], [m], Hq, Hk, D, seed=70)
    want = against(x, False)
    y = {name: t.to(DEV) for name, t in x.items()}
    out, lse = uaa.attn_packed_fwd(y["q"], y["k"], y["v"], y["starts"], y["starts_k"], False)
    parts, at = [], 0
    for c in cut:
        k, v = (y[name][at: at + c] for name in ("k", "v"))
        parts.append(uaa.attn_packed_bwd(y["q"], k, v, out, y["do"], lse, y["starts"],
                                         torch.tensor([0, c], dtype=torch.int32, device=DEV), False))
        at += c
    uaa.check_device_status()
    dk, dv = (torch.cat([p[i] for p in parts]).cpu().double().numpy() for i in (1, 2))
    for name, t in (("dk", dk), ("dv", dv)):
        assert (np.abs(t - want[name][0]) <= want[name][1]).all(), name
    dq = sum(p[0].cpu().double().numpy() for p in parts)
    # each part is rounded by itself
    more = sum(np.abs(p[0].cpu().double().numpy()) for p in parts) * 2.0 ** -8
    assert (np.abs(dq - want["dq"][0]) <= want["dq"][1] + more).all()
