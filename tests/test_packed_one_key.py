"""A softmax over one key is constant: queries that read one key have no gradient in q and k, not even a rounding's."""
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from test_packed_attention import ALL, DEV, against, check, draw, step


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hk,D", [(8, 4, 128), (6, 2, 64), (5, 1, 128), (128, 1, 64), (1, 1, 64)])
def test_sequences_of_one_token(Hq, Hk, D, causal):
    lens = [1] * 333
    x = draw(lens, lens, Hq, Hk, D, seed=80)
    got = step(x, causal)
    assert not got["dq"].any() and not got["dk"].any()
    check(got, against(x, causal), ALL)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,D", [(8, 4, 128), (6, 2, 64), (5, 1, 128), (65, 1, 64)])
@pytest.mark.parametrize("lens,lens_k", [([300, 2, 129, 1, 40], [300, 2, 129, 1, 40]), ([300, 200, 9], [40, 130, 1]), ([7] * 50, [3] * 50)])
def test_first_queries_of_causal_sequences(lens, lens_k, Hq, Hk, D):
    """The query at the first key, wherever it stands in its tile."""
    x = draw(lens, lens_k, Hq, Hk, D, seed=81)
    got, at = step(x), 0
    check(got, against(x), ALL)
    for n, m in zip(lens, lens_k):
        assert not got["dq"][at: at + n - m + 1].any()
        assert m == 1 or got["dq"][at + n - m + 1].any()
        at += n


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,D", [(8, 4, 128), (6, 2, 64), (24, 24, 64)])
def test_many_queries_over_one_key(Hq, Hk, D):
    x = draw([300, 5, 1], [1, 1, 200], Hq, Hk, D, seed=82)
    got = step(x, False)
    assert not got["dq"][:305].any() and not got["dk"][:2].any() and got["dq"][305:].any()
    check(got, against(x, False), ALL)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_one_key_of_several(D):
    """One key in a call of its own, with the out and lse of more keys: its gradients are there."""
    n, m = 40, 30
    x = draw([n], [m], 6, 2, D, seed=83)
    want = against(x, False)
    y = {name: t.to(DEV) for name, t in x.items()}
    out, lse = uaa.attn_packed_fwd(y["q"], y["k"], y["v"], y["starts"], y["starts_k"], False)
    one = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    _, dk, _ = uaa.attn_packed_bwd(y["q"], y["k"][:1], y["v"][:1], out, y["do"], lse, y["starts"], one, False)
    value, bound = (t[:1] for t in want["dk"])
    off = (dk.cpu().double() - torch.from_numpy(value)).abs()
    assert dk.any() and (off <= torch.from_numpy(bound)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["q", "k", "v", "do"])
def test_values_that_are_not_finite_show(name):
    x = draw([1, 1], [1, 1], 2, 2, 64, seed=84)
    x[name][0, 0, 3] = float("nan")
    got = step(x, True)
    assert torch.isnan(got["dq"][0, 0]).any() or torch.isnan(got["dk"][0, 0]).any()
    assert not got["dq"][1].any() and not got["dk"][1].any()
