"""fp16 has no gradients; results without one are to be had of leaves that could have some."""
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from test_packed_attention import DEV, draw, step


def leaves(device="cpu"):
    x = draw([70, 3], [70, 3], 4, 2, 64, torch.float16, seed=24)
    return x, [x[n].to(device).requires_grad_() for n in ("q", "k", "v")], x["starts"].to(device)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_without_gradients_no_refusal_of_the_type(mode):
    _, qkv, starts = leaves()
    with mode(), pytest.raises(ValueError, match="CUDA"):
        uaa.packed_attention(*qkv, starts)


@pytest.mark.parametrize("which", range(3))
def test_gradients_are_refused(which):
    _, qkv, starts = leaves()
    for i, t in enumerate(qkv):
        t.requires_grad_(i == which)
    with pytest.raises(TypeError, match="gradients are built for bfloat16"):
        uaa.packed_attention(*qkv, starts)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("saved", [None, "int8"])
def test_results(mode, saved):
    x, qkv, starts = leaves(DEV)
    want = step(x, grads=False)
    with mode():
        out, lse = uaa.packed_attention(*qkv, starts, saved=saved)
    assert torch.equal(out, want["out"]) and torch.equal(lse, want["lse"]) and not out.requires_grad
    with pytest.raises(TypeError, match="gradients are built for bfloat16"):  # without the check of packed_attention
        uaa.PackedAttention.apply(*qkv, starts)[0].sum().backward()
