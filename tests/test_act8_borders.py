"""8-bit checkpoints: codes at the borders between two of them in fp16 and fp32, and the Ulysses steps' gradients against
those of the unpacked tensors, bit for bit."""
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from ulysses_dit_attention_gb300 import synth
from test_act8 import _check

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _borders(tops, dtype):
    """Rows that hold, under each top, the values of the type next to every border (2 k + 1) top / 254, and the top."""
    mid = tops.double()[:, None] * (2 * torch.arange(127).double() + 1) / 254
    near = mid.to(dtype)
    other = torch.where(near.double() > mid, torch.nextafter(near, torch.zeros_like(near)),
                        torch.nextafter(near, torch.full_like(near, torch.finfo(dtype).max)))
    sign = 1.0 - 2.0 * (torch.arange(127) % 2)
    x = torch.cat((near * sign.to(dtype), other * -sign.to(dtype), tops[:, None].to(dtype), -tops[:, None].to(dtype)), 1)
    assert (x.abs() <= tops[:, None]).all()
    return x


def test_every_fp16_top_at_every_border():
    """All significands, and ordinary, large and subnormal magnitudes."""
    for scale in (2.0 ** -10, 2.0 ** 5, 2.0 ** -23, 2.0 ** -15):
        tops = torch.arange(1024, 2048).double() * scale
        tops = tops[tops <= 65504].to(torch.float16)
        x = _borders(tops, torch.float16).to(DEV)
        _check(uaa.act8_pack([x]), [x])
    tops = torch.arange(1, 1024).double().mul(2.0 ** -24).to(torch.float16)  # below the normal numbers
    x = _borders(tops, torch.float16).to(DEV)
    _check(uaa.act8_pack([x]), [x])


@pytest.mark.parametrize("scale", [0, 100, -100, -118, 127])
def test_random_fp32_tops_at_every_border(scale):
    g = torch.Generator().manual_seed(7 + abs(scale))
    tops = ((1 + torch.rand(4096, generator=g, dtype=torch.float64)) * 2.0 ** scale).float()
    tops = torch.where(torch.isinf(tops), torch.full_like(tops, 3e38), tops)
    x = _borders(tops, torch.float32).to(DEV)
    _check(uaa.act8_pack([x]), [x])


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_ulysses_gradients_are_those_of_the_unpacked_tensors(fused, masked):
    lens, cap, B, H, D = (70, 71, 60), 71, 2, 5, 64
    inp = synth.draw(B, sum(lens), H, D, seed=9, masked=masked)
    mask = inp["mask"].to(DEV) if masked else None
    q, k, v = (synth.pad_shards(inp[n], lens, cap).to(DEV).requires_grad_() for n in ("q", "k", "v"))
    do = synth.pad_shards(inp["do"], lens, cap).to(DEV)
    call = uaa.ulysses_attention_fused if fused else uaa.ulysses_attention
    out, lse = call(q, k, v, lens, mask, saved="int8")
    got = torch.autograd.grad(out, (q, k, v), do)
    held = [t.detach() for t in (q, k, v)]
    if fused:
        kept = uaa.act8_unpack(uaa.act8_pack([*held, out.detach()]))
        want = uaa.ulysses_attn_bwd(*kept, do, lse, lens, mask)
    else:
        groups = [uaa.seq_to_head(t, lens) for t in held]
        o, lse = uaa.attn_fwd_groups(*groups, mask)
        kept = uaa.act8_unpack(uaa.act8_pack([*groups, o]))
        want = [uaa.head_to_seq(t, lens, cap, H)
                for t in uaa.attn_bwd_groups(*kept, uaa.seq_to_head(do, lens), lse, mask)]
    for a, w in zip(got, want):
        assert torch.equal(a, w)
    uaa.check_device_status()
