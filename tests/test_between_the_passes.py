"""What happens to a pairing's inputs between its forward and its backward pass."""
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from ulysses_dit_attention_gb300 import synth

DEV = "cuda"
LENS, CAP = (40, 41, 30), 41


def _pairings(saved, mask):
    """Every pairing, as (leaves, call)."""
    B, S, H, D = 2, sum(LENS), 3, 64
    x = [torch.randn(B, S, H, D, device=DEV).bfloat16() for _ in range(3)]
    sh = [synth.pad_shards(t.cpu(), LENS, CAP).to(DEV) for t in x]
    lam = torch.rand(H, device=DEV)
    leaf = lambda ts: [t.clone().requires_grad_() for t in ts]  # noqa: E731
    return {
        "attention": (leaf(x), lambda q, k, v: uaa.attention(q, k, v, mask, saved=saved)),
        "ulysses": (leaf(sh), lambda q, k, v: uaa.ulysses_attention(q, k, v, LENS, mask, saved=saved)),
        "fused": (leaf(sh), lambda q, k, v: uaa.ulysses_attention_fused(q, k, v, LENS, mask, saved=saved)),
        "diff": (leaf(x + [lam]), lambda q, k, v, lm: uaa.diff_attention(q, k, v, lm, mask, saved=saved)),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("saved", [None, "int8"])
@pytest.mark.parametrize("which", ["attention", "ulysses", "fused", "diff"])
def test_a_mask_changed_between_the_passes_raises(which, saved):
    """As any other tensor that the backward pass reads: gradients of another mask would be wrong without a sign."""
    mask = torch.rand(2, sum(LENS), device=DEV) < 0.7
    mask[:, 0] = True
    leaves, call = _pairings(saved, mask)[which]
    out = call(*leaves)[0]
    mask[:, 1] = ~mask[:, 1]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.float().sum().backward()


@pytest.mark.gpu
@pytest.mark.parametrize("saved", [None, "int8"])
@pytest.mark.parametrize("which", ["attention", "ulysses", "fused", "diff"])
def test_a_mask_made_in_inference_mode(which, saved):
    """Autograd cannot keep such a tensor; the pairings take it all the same."""
    with torch.inference_mode():
        mask = torch.arange(sum(LENS), device=DEV)[None] < torch.tensor([[50], [90]], device=DEV)
    grads = []
    for m in (mask, mask.clone()):
        torch.manual_seed(3)
        leaves, call = _pairings(saved, m)[which]
        out = call(*leaves)[0]
        grads.append(torch.autograd.grad(out, leaves, torch.ones_like(out)))
    assert all(torch.equal(a, b) for a, b in zip(*grads))


def test_saved_is_checked_whether_a_gradient_is_wanted_or_not():
    q, lam = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16), torch.zeros(2)
    sh = torch.zeros(1, 1, 4, 2, 64, dtype=torch.bfloat16)
    for grad in (False, True):
        q.requires_grad_(grad)
        for call in (lambda: uaa.attention(q, q, q, saved="int4"), lambda: uaa.diff_attention(q, q, q, lam, saved="int4"),
                     lambda: uaa.ulysses_attention(sh, sh, sh, (4,), saved="int4"),
                     lambda: uaa.ulysses_attention_fused(sh, sh, sh, (4,), saved="int4")):
            with pytest.raises(ValueError, match="saved must be"):
                call()
