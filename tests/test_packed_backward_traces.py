"""Gradients of packed attention: what one sequence holds leaves no trace in another one, whatever a block has worked on
before.  Groups of query heads that do not fill a tile of 128 rows, and so many items that every block takes several."""
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from test_packed_attention import ALL, DEV, against, check, draw, step

HEADS = [(6, 2), (5, 1), (12, 1)]


def lengths(B, seed):
    """Mostly longer than a tile of keys and not a multiple of it, so that all lanes of a tile hold keys, of this sequence or
    of the next one; some of one token and of none."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(40, 300, (B,), generator=g).tolist()
    lens[3::17] = [1] * len(lens[3::17])
    lens[9::23] = [0] * len(lens[9::23])
    return lens


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", HEADS)
def test_values_that_are_not_finite(Hq, Hk, D, causal):
    """NaN in every other sequence: the others' results keep their bits."""
    lens = lengths(300, Hq)
    x = draw(lens, lens, Hq, Hk, D, seed=30 + Hq)
    odd = torch.repeat_interleave(torch.arange(len(lens)) % 2 == 1, torch.tensor(lens))
    clean = step(x, causal)
    for names in (("do",), ("v",), ("k", "q")):
        y = {n: t.clone() for n, t in x.items()}
        for n in names:
            y[n][odd] = float("nan")
        got = step(y, causal)
        for n in ALL:
            a, b = (t[n].T if n == "lse" else t[n] for t in (got, clean))
            assert torch.equal(a[~odd.to(DEV)], b[~odd.to(DEV)]), (names, n)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(600, 200), (1000, 200), (2400, 200)])
@pytest.mark.parametrize("causal", [True, False])
def test_tokens_behind_the_last_sequence(Hq, Hk, D, causal):
    """A buffer with room for more tokens than there are, NaN behind them: 200 items of one sequence, one after the other."""
    x = draw([70], [70], Hq, Hk, D, seed=33, tail=90)
    clean = step(x, causal)
    for n in ("q", "k", "v", "do"):
        x[n][70:] = float("nan")
    got = step(x, causal)
    for n in ALL:
        a, b = (t[n].T if n == "lse" else t[n] for t in (got, clean))
        assert torch.equal(a[:70], b[:70]), n


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", HEADS)
def test_a_neighbour_whose_keys_score_far_higher(Hq, Hk, D, causal):
    """Finite inputs: the keys of every other sequence score 200 above the others', exp(200) being past the 32-bit range."""
    lens = lengths(300, Hq)
    x = draw(lens, lens, Hq, Hk, D, seed=36 + Hq)
    odd = torch.repeat_interleave(torch.arange(len(lens)) % 2 == 1, torch.tensor(lens))
    x["q"][..., 0] = 8.0
    x["k"][..., 0] = torch.where(odd, 200.0 * D ** 0.5 / 8.0, 0.0)[:, None]
    got = step(x, causal)
    for n in ALL:
        assert torch.isfinite(got[n]).all(), n
    check(got, against(x, causal), ALL)
