"""Rotation into memory that the same call still reads, or writes twice: refused before anything is launched."""
import itertools

import numpy as np
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa

B, S, D = 2, 3, 8
BASE = 1 << 20  # never read: every call here is refused, or has no GPU to run on


def _call(q, k=None):
    """q, k: (element offset of x, strides of x, offset of y, strides of y, heads), bf16."""
    def tensor(t):
        x, sx, y, sy, H = t
        return uaa._ROTARY_TENSOR.pack(BASE + 2 * x, BASE + 2 * y, *sx, *sy, H)

    plan = uaa.RotaryPlan([D])
    st = uaa.lib().uaa_rotary(plan._ref, tensor(q), None if k is None else tensor(k), None, 0, 0, 0, 0, B, S, D, 0, 0, None)
    return st == -1 and "overlap" in uaa.lib().uaa_last_error().decode()


def _cells(at, strides, H):
    i = np.indices((B, S, H, D)).reshape(4, -1)
    return set(at + i[0] * strides[0] + i[1] * strides[1] + i[2] * strides[2] + i[3])


def _rows(heads):
    """Strides of a (B, S, heads, D) tensor."""
    return S * heads * D, heads * D, D


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls that are not refused would run")
def test_against_the_elements_themselves():
    """Tensors of like strides, anywhere in one buffer: refused exactly where an element meets another's."""
    refused = 0
    for width, Hq, Hk in ((6, 2, 2), (6, 3, 1), (4, 1, 3), (2, 1, 1)):
        st = _rows(width)
        span = S * width * D
        for off in itertools.chain(range(-width * D - D, width * D + D + 1, 4), (span, -span, 2 * span, -2 * span, 4 * D + span)):
            # an output beside its input
            meets = off != 0 and bool(_cells(0, st, Hq) & _cells(off, st, Hq))
            assert _call((0, st, off, st, Hq)) == meets, (width, off)
            # k's output beside q, which is turned in place
            far = 10000
            meets = bool(_cells(0, st, Hq) & _cells(off, st, Hk))
            assert _call((0, st, 0, st, Hq), (far, st, off, st, Hk)) == meets, (width, off)
            # k's output beside q's output; q's input is elsewhere
            assert _call((far, st, 0, st, Hq), (2 * far, st, off, st, Hk)) == meets, (width, off)
            # q's output beside k's input
            assert _call((far, st, 0, st, Hq), (off, st, 2 * far, st, Hk)) == meets, (width, off)
            refused += meets
    assert refused > 50


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls that are not refused would run")
def test_other_strides():
    bshd, bhsd = _rows(2), (S * 2 * D, D, S * D)
    assert _call((0, bshd, 0, bhsd, 2))                               # in place, but rows in another order
    assert not _call((0, (0, 2 * D, D), 10000, bshd, 2))              # an input shared by the batch
    assert _call((0, (0, 2 * D, D), 0, bshd, 2))
    assert not _call((0, bshd, 0, bshd, 2), (10000, bhsd, 10000, bhsd, 2))


@pytest.mark.gpu
def test_packed_projections_and_refusals():
    plan = uaa.RotaryPlan([64])
    packed = torch.randn(2, 9, 24 + 2 * 8, 64, device="cuda").bfloat16()  # 24 heads of q, 8 of k, 8 of v
    q, k, v = packed.split((24, 8, 8), 2)
    want = uaa.rotary_fwd(q.contiguous(), k.contiguous(), plan)
    keep = v.clone()
    for bad in (dict(out_q=q, out_k=q[:, :, :8]), dict(out_k=q[:, :, 3:11]), dict(out_q=packed[:, :, 16:]),
                dict(out_q=packed[:, :, 1:25])):
        with pytest.raises(uaa.UAAError, match="overlap"):
            uaa.rotary_fwd(q, k, plan, **bad)
    uaa.rotary_fwd(q, k, plan, out_k=v)  # beside both
    assert torch.equal(v, want[1])
    v.copy_(keep)
    uaa.rotary_fwd(q, k, plan, out_q=q, out_k=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, keep)
    uaa.check_device_status()
