"""Gradients of packed attention over long sequences, whose items are cut several times, by their mean error.

The bounds of each element (oracle/seqs.py) add up every rounding at its worst, which for hundreds of keys is a good part of
the value.  Independent roundings add up by squares instead.  One to bf16 is uniform within half a step, 2^-8 of the binade's
lowest value; with mantissas x of density 1 / (x ln 2) its mean square is (2^-8)^2 / 3 times 3 / (8 ln 2), (0.425 * 2^-8)^2, of
the value's.  With normal inputs the terms of a sum are uncorrelated, and a sum of rounded terms is off by the same share of
its own mean square.  There are at most four on the way to a result: of dS, of P and of out where Delta = dout . out uses
them, and of the result.  Together: (2 * 0.425 * 2^-8)^2, below (2^-8)^2.
"""
import numpy as np
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from test_packed_attention import ALL, DEV, against, check, draw, step

RMS = 2.0 ** -8
GRADS = ("out", "dq", "dk", "dv")


def pieces(x, name):
    """The places of each sequence of 100 tokens or more in a result (fewer are no sample)."""
    st = x["starts_k" if name in ("dk", "dv") else "starts"].tolist()
    return [slice(a, b) for a, b in zip(st, st[1:]) if b - a >= 100]


def mean_error(got, want):
    return np.sqrt(((got - want) ** 2).sum() / (want ** 2).sum())


def check_mean(x, got, want, names=GRADS):
    for n in names:
        y = got[n].cpu().double().numpy()
        for at in pieces(x, n):
            assert mean_error(y[at], want[n][0][at]) <= RMS, (n, at, mean_error(y[at], want[n][0][at]))


def test_a_small_part_that_is_lost_shows():
    """What the mean has to see: 28 keys of 900 whose gradients are a tenth too small."""
    x = draw([900], [900], 3, 1, 64, seed=40)
    want = against(x, False)
    y = {n: torch.from_numpy(want[n][0].copy()) for n in GRADS}
    check_mean(x, y, want)
    y["dk"][-28:] *= 0.9
    with pytest.raises(AssertionError):
        check_mean(x, y, want)


CASES = [
    # (lens, lens_k, Hq, Hk): one long sequence, cut about twice and about five times an item; several; keys of their own
    ([4001], [4001], 6, 2),
    ([4001], [4001], 3, 1),
    ([3000, 130, 1, 0, 1111], [3000, 130, 1, 0, 1111], 12, 2),
    ([4099], [300], 6, 2),
    ([300, 200], [4099, 77], 10, 2),
]


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,lens_k,Hq,Hk", CASES, ids=lambda x: str(x))
def test_long_sequences(lens, lens_k, Hq, Hk, D, causal):
    if lens == [4099] and causal:
        lens = [450]  # (most queries would read no key)
    x = draw(lens, lens_k, Hq, Hk, D, seed=sum(lens) + Hq)
    got, want = step(x, causal), against(x, causal)
    check(got, want, ALL)
    check_mean(x, got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hk,D", [(10, 2, 64), (6, 2, 128), (4, 4, 64)])
def test_each_sequence_alone(Hq, Hk, D, causal):
    """A sequence in a pack and by itself: where its items have fewer than four inner tiles they are cut in neither, and the
    bits are the same; others are cut at other places, and each side is within its own mean error."""
    lens = [1, 40, 400, 130, 1500, 2, 33]
    x = draw(lens, lens, Hq, Hk, D, seed=41)
    got, at = step(x, causal), 0
    for n in lens:
        one = {name: x[name][at: at + n] for name in ("q", "k", "v", "do")}
        one["starts"] = one["starts_k"] = torch.tensor([0, n], dtype=torch.int32)
        alone = step(one, causal)
        forward_whole, backward_whole = n <= 3 * 128, n <= 3 * (128 // (Hq // Hk))
        for name in ALL:
            a, b = got[name][:, at: at + n] if name == "lse" else got[name][at: at + n], alone[name]
            if backward_whole or (forward_whole and name in ("out", "lse")):
                assert torch.equal(a, b), (n, name)
            elif name != "lse":
                a, b = (t.cpu().double().numpy() for t in (a, b))
                assert mean_error(a, b) <= 2 ** 0.5 * RMS, (n, name)
        at += n
