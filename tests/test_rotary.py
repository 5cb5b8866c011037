"""Rotary positions: the plan (host code, no GPU) and the kernel against the float64 definition."""
import numpy as np
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from oracle import ops
from helpers import bits

DEV = "cuda"


# --------------------------------------------------------------------------- the plan
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 4.0), ("parts", 8.0)])
@pytest.mark.parametrize("widths", [[2], [64], [128], [44, 42, 42], [0, 16], [256]])
def test_plan_frequencies(scaling, factor, widths):
    plan = uaa.RotaryPlan(widths, scaling=scaling, factor=factor, original=4096)
    rates, _ = ops.rotary_rates(widths, scaling=scaling, factor=factor, original=4096)
    # 64-bit fixed point: half a step of 2^-64, and the 53 bits that the frequency is computed with
    got, want = np.array(plan.turns), rates / (2 * np.pi)
    assert plan.rot == sum(widths) and plan.axes == len(widths)
    assert (np.abs(got - want) <= 2.0 ** -64 + 8 * 2.0 ** -53 * want).all()
    assert plan.magnitude == pytest.approx(0.1 * np.log(factor) + 1 if scaling == "parts" else 1.0, rel=2 ** -24)


def test_plan_refusals():
    for bad in (dict(widths=[3]), dict(widths=[-2]), dict(widths=[256, 2]), dict(widths=[]), dict(widths=[2] * 5),
                dict(widths=[64], base=0.5), dict(widths=[64], base=float("inf")),
                dict(widths=[64], scaling="linear", factor=0.5), dict(widths=[64], scaling="ntk", factor=float("nan")),
                dict(widths=[64], scaling="parts", factor=2.0, alpha=4.0, beta=4.0),
                dict(widths=[64], scaling="parts", factor=2.0, original=0)):
        with pytest.raises(uaa.UAAError):
            uaa.RotaryPlan(**bad)
    for bad in (dict(layout="other"), dict(scaling="other")):
        with pytest.raises(ValueError):
            uaa.RotaryPlan([64], **bad)


def test_refusals_without_gpu():
    plan = uaa.RotaryPlan([64])
    q = torch.zeros(2, 3, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        uaa.rotary_fwd(q, None, plan)
    with pytest.raises(TypeError, match="plan"):
        uaa.rotary_fwd(q, None, None)


def _raw(plan=None, q=None, k=None, pos=None, B=1, S=2, D=64, dtype=0):
    plan = plan or uaa.RotaryPlan([64])
    return uaa.lib().uaa_rotary(plan._ref, q, k, pos, 0, 0, 0, 0, B, S, D, dtype, 0, None)


def _tensor(x=4096, y=4096, strides=(512, 256, 64, 512, 256, 64), H=4):
    return uaa._ROTARY_TENSOR.pack(x or 0, y, *strides, H)


def test_refusals_of_the_call():
    L = uaa.lib()
    err = lambda: L.uaa_last_error().decode()  # noqa: E731
    assert _raw(q=_tensor(x=None)) == -1 and "NULL" in err()
    assert _raw(q=_tensor(x=4097)) == -1 and "aligned" in err()
    assert _raw(q=_tensor(), D=32) == -1 and "rotated" in err()
    assert _raw(q=_tensor(), dtype=7) == -1 and "dtype" in err()
    assert _raw(q=_tensor(), B=-1) == -1
    assert _raw(q=_tensor(strides=(512, 256, 64, 512, 128, 64))) == -1 and "overlap" in err()
    assert _raw(q=_tensor(strides=(512, 256, 64, 512, 256, 32))) == -1 and "overlap" in err()
    assert _raw(q=_tensor(strides=(-512, 256, 64, 512, 256, 64))) == -1 and "stride" in err()
    assert _raw(q=_tensor(), pos=4097) == -1 and "positions" in err()
    assert _raw(q=_tensor(), B=1 << 16, S=1 << 16) == -2
    # nothing to do: nothing launched
    assert _raw(q=_tensor(x=None), B=0) == 0
    assert _raw(q=_tensor(x=None, H=0)) == 0


# --------------------------------------------------------------------------- the kernel
def _eps(dtype):
    return torch.finfo(dtype).eps / 2


def _check(got, x, pos, plan_args, layout, dtype, inverse=False, name=""):
    rates, axis = ops.rotary_rates(**plan_args)
    mag = 0.1 * np.log(plan_args.get("factor", 1.0)) + 1 if plan_args.get("scaling") == "parts" else 1.0
    x64 = x.detach().cpu().double().numpy()
    ref, size = ops.rotary(x64, pos, rates, axis, layout, mag, inverse)
    # the angle: its 24 bits (pi 2^-24), sincospif (2^-22), 53-bit frequencies at far positions; three 32-bit
    # operations; one rounding to the type
    far = np.abs(pos).max() * 2.0 ** -50 if pos.size else 0.0
    bound = _eps(dtype) * np.abs(ref) + size * (2.0 ** -20 + far)
    err = np.abs(got.detach().cpu().double().numpy() - ref)
    assert (err <= bound).all(), f"{name}: {np.max(err - bound)}"


def _positions(kind, B, S, axes, g):
    if kind == "far":
        p = torch.randint(-(2 ** 31), 2 ** 31 - 1, (B, S, axes), generator=g)
        p[0, 0] = 2 ** 31 - 1
        return p
    return torch.randint(0, 30000, (B, S, axes), generator=g)


CASES = [
    # B, S, Hq, Hk, D, widths, layout, dtype, scaling
    (1, 1, 1, 1, 64, [64], "half", torch.bfloat16, "none"),
    (2, 1, 24, 24, 128, [128], "half", torch.bfloat16, "parts"),
    (2, 37, 3, 1, 128, [44, 42, 42], "interleaved", torch.bfloat16, "none"),
    (1, 300, 5, 5, 64, [40], "half", torch.float32, "ntk"),
    (3, 17, 2, 7, 64, [6, 2], "half", torch.float16, "linear"),
    (3, 17, 2, 7, 64, [34], "interleaved", torch.bfloat16, "linear"),
    (2, 9, 4, 2, 66, [66], "half", torch.bfloat16, "none"),   # pairs at an odd distance: one element an access
    (2, 9, 4, 2, 66, [66], "interleaved", torch.float32, "none"),
    (1, 50, 1, 3, 256, [256], "half", torch.bfloat16, "none"),
    (1, 5, 2, 2, 64, [0, 0], "half", torch.bfloat16, "none"),  # nothing is rotated: a copy
    (1, 3, 2, 2, 7, [6], "interleaved", torch.float32, "none"),
    # rows of whole 16-byte vectors whose runs of pairs are not
    (2, 40, 5, 3, 80, [50], "half", torch.bfloat16, "none"),
    (1, 33, 3, 2, 256, [250], "interleaved", torch.float16, "none"),
    (1, 21, 2, 9, 128, [100, 26], "half", torch.float32, "none"),
    (2, 19, 1, 2, 8, [6], "half", torch.bfloat16, "none"),
    (1, 19, 3, 0, 264, [250], "half", torch.bfloat16, "none"),  # more vectors than a warp has lanes
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("kind,wide", [("near", False), ("far", True)])
def test_rotary(case, kind, wide):
    B, S, Hq, Hk, D, widths, layout, dtype, scaling = case
    g = torch.Generator().manual_seed(hash((B, S, Hq, D)) % 1000)
    q, k, dq, dk = (torch.randn(B, S, h, D, generator=g).to(dtype).to(DEV) for h in (Hq, Hk, Hq, Hk))
    pos = _positions(kind, B, S, len(widths), g)
    args = dict(widths=widths, scaling=scaling, factor=4.0 if scaling != "none" else 1.0)
    plan = uaa.RotaryPlan(layout=layout, **args)
    given = (pos if len(widths) > 1 else pos[..., 0]).to(torch.int64 if wide else torch.int32).to(DEV)
    yq, yk = uaa.rotary_fwd(q, k, plan, given)
    gq, gk = uaa.rotary_bwd(dq, dk, plan, given)
    uaa.check_device_status()
    for got, x, inv, n in ((yq, q, False, "q"), (yk, k, False, "k"), (gq, dq, True, "dq"), (gk, dk, True, "dk")):
        _check(got, x, pos.numpy(), args, layout, dtype, inv, n)
    R = sum(widths)
    assert np.array_equal(bits(yq[..., R:]), bits(q[..., R:]))


@pytest.mark.gpu
def test_default_positions_one_tensor_and_in_place():
    plan, args = uaa.RotaryPlan([64]), dict(widths=[64])
    q = torch.randn(2, 33, 3, 64, device=DEV, dtype=torch.bfloat16)
    pos = np.broadcast_to((1000 + np.arange(33))[None, :, None], (2, 33, 1))
    y, none = uaa.rotary_fwd(q, None, plan, start=1000)
    assert none is None
    _check(y, q, pos, args, "half", torch.bfloat16)
    shared = torch.arange(1000, 1033, device=DEV)  # one row of positions for the batch
    assert torch.equal(uaa.rotary_fwd(q, None, plan, shared)[0], y)
    z = q.clone()
    assert uaa.rotary_fwd(z, None, plan, start=1000, out_q=z)[0] is z
    assert torch.equal(z, y)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(64, 50), (80, 78), (256, 130), (128, 20)])
def test_partial_rows_in_place_strided_and_off_the_grid(layout, D, rot):
    """Every access width gives the same bits; a row that lies between others is turned where it is."""
    plan = uaa.RotaryPlan([rot], layout=layout)
    B, S, H = 2, 45, 3
    x = torch.randn(B, S, H, D, device=DEV, dtype=torch.bfloat16)
    want = uaa.rotary_fwd(x, None, plan, start=9)[0]
    for off in (1, 2, 4, 8):
        flat = torch.zeros(x.numel() + 8, device=DEV, dtype=torch.bfloat16)
        y = flat[off:off + x.numel()].view(B, S, H, D).copy_(x)
        assert torch.equal(uaa.rotary_fwd(y, None, plan, start=9)[0], want), off
    packed = torch.randn(B, S, 3, H, D, device=DEV, dtype=torch.bfloat16)
    packed[:, :, 1] = x
    keep = packed.clone()
    uaa.rotary_fwd(packed[:, :, 1], None, plan, start=9, out_q=packed[:, :, 1])
    assert torch.equal(packed[:, :, 1], want)
    assert torch.equal(packed[:, :, 0], keep[:, :, 0]) and torch.equal(packed[:, :, 2], keep[:, :, 2])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strided_operands(layout):
    """Slices of a packed projection, heads before tokens, and bases off the 16-byte grid."""
    plan = uaa.RotaryPlan([32], layout=layout)
    B, S, H, D = 2, 21, 3, 64
    packed = torch.randn(B, S, 3, H, D, device=DEV, dtype=torch.bfloat16)
    q, k = packed[:, :, 0], packed[:, :, 1]
    want = uaa.rotary_fwd(q.contiguous(), k.contiguous(), plan, start=5)
    got = uaa.rotary_fwd(q, k, plan, start=5)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    before = packed[:, :, 2].clone()
    uaa.rotary_fwd(q, k, plan, start=5, out_q=q, out_k=k)  # into the packed tensor
    assert torch.equal(packed[:, :, 0], want[0]) and torch.equal(packed[:, :, 1], want[1])
    assert torch.equal(packed[:, :, 2], before)
    bhsd = want[0].transpose(1, 2).contiguous().transpose(1, 2)  # tokens innermost but for the columns
    a = uaa.rotary_fwd(bhsd, None, plan)[0]
    assert torch.equal(a, uaa.rotary_fwd(want[0], None, plan)[0])
    for off in (1, 2, 4):
        flat = torch.zeros(q.numel() + 8, device=DEV, dtype=torch.bfloat16)
        odd = flat[off:off + q.numel()].view(B, S, H, D).copy_(want[1])
        assert torch.equal(uaa.rotary_fwd(odd, None, plan)[0], uaa.rotary_fwd(want[1], None, plan)[0])
    wide = torch.zeros(B, S, H, D + 1, device=DEV, dtype=torch.bfloat16)  # an odd head stride
    wide[..., :D] = want[1]
    assert torch.equal(uaa.rotary_fwd(wide[..., :D], None, plan)[0], uaa.rotary_fwd(want[1], None, plan)[0])


@pytest.mark.gpu
def test_autograd_is_the_transpose():
    plan = uaa.RotaryPlan([24, 24], scaling="parts", factor=2.0)
    B, S, D = 2, 11, 64
    q = torch.randn(B, S, 4, D, device=DEV, requires_grad=True)
    k = torch.randn(1, S, 2, D, device=DEV, requires_grad=True)  # a key shared by the batch
    pos = torch.randint(0, 500, (B, S, 2), device=DEV)
    yq, yk = uaa.rotary(q, k.expand(B, S, 2, D), plan, pos)
    gq, gk = torch.randn_like(yq), torch.randn_like(yk)
    dq, dk = torch.autograd.grad((yq, yk), (q, k), (gq, gk))
    want_q, want_k = uaa.rotary_bwd(gq, gk, plan, pos)
    assert torch.equal(dq, want_q) and torch.allclose(dk, want_k.sum(0, keepdim=True), atol=1e-6)
    # <y, g> = <x, J^T g>: 2^-21 per term, 2 * 64 * 11 * 4 terms of about one
    assert abs(float(((yq.double() * gq).sum() - (q.double() * dq).sum()).detach())) < 2.0 ** -21 * q.numel()
    only_k = torch.autograd.grad(uaa.rotary(q, k.expand(B, S, 2, D), plan, pos)[1].sum(), k)[0]
    ones = torch.ones(B, S, 2, D, device=DEV)
    assert torch.allclose(only_k, uaa.rotary_bwd(ones, None, plan, pos)[0].sum(0, keepdim=True), atol=1e-6)


@pytest.mark.gpu
def test_shards_of_a_ulysses_step():
    """Shards rotated where they stand equal the shards of the rotated sequence."""
    lens, cap, B, H, D = (30, 31, 25), 31, 2, 3, 64
    N = sum(lens)
    plan = uaa.RotaryPlan([64])
    x = torch.randn(B, N, H, D, device=DEV, dtype=torch.bfloat16)
    whole = uaa.rotary_fwd(x, None, plan)[0]
    sh = torch.zeros(3, B, cap, H, D, device=DEV, dtype=torch.bfloat16)
    want = torch.zeros_like(sh)
    at = 0
    for p, n in enumerate(lens):
        sh[p, :, :n], want[p, :, :n] = x[:, at:at + n], whole[:, at:at + n]
        at += n
    pos = uaa.shard_positions(lens, cap, B, DEV)
    got = uaa.rotary_fwd(sh.view(3 * B, cap, H, D), None, plan, pos)[0].view_as(sh)
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    plan = uaa.RotaryPlan([128])
    q = torch.randn(4, 1, 24, 128, device=DEV, dtype=torch.bfloat16)
    pos = torch.zeros(4, 1, device=DEV, dtype=torch.int32)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        uaa.rotary_fwd(q, None, plan, pos, out_q=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        uaa.rotary_fwd(q, None, plan, pos, out_q=out)
    for step in (3, 70000):
        pos.fill_(step)
        graph.replay()
        assert torch.equal(out, uaa.rotary_fwd(q, None, plan, start=step)[0])


@pytest.mark.gpu
def test_refusals_on_the_gpu():
    plan = uaa.RotaryPlan([64])
    q = torch.zeros(2, 3, 4, 64, device=DEV, dtype=torch.bfloat16)
    pos = torch.zeros(2, 3, device=DEV, dtype=torch.int32)
    for args, kind in (((q.double(), None, plan), TypeError), ((q, q.float(), plan), TypeError),
                       ((q[0], None, plan), ValueError), ((q, q[:1], plan), ValueError),
                       ((q.transpose(2, 3), None, plan), ValueError), ((q, None, plan, pos[:1]), ValueError),
                       ((q, None, plan, pos.float()), TypeError), ((q, None, plan, pos.cpu()), ValueError),
                       ((q, None, plan, pos, 3), ValueError), ((q[..., :32], None, plan), uaa.UAAError)):
        with pytest.raises(kind):
            uaa.rotary_fwd(*args)
    with pytest.raises(ValueError):
        uaa.rotary_fwd(q, None, plan, out_q=torch.empty(1, device=DEV))
    with pytest.raises(uaa.UAAError, match="overlap"):
        uaa.rotary_fwd(q, None, plan, out_q=q[:, :1].expand_as(q))
    # empty batches and lengths
    for s in ((0, 3, 4, 64), (2, 0, 4, 64), (2, 3, 0, 64)):
        assert uaa.rotary_fwd(torch.empty(s, device=DEV), None, plan)[0].shape == s


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A view into a tensor of 2^32 + elements: the last rows are where they should be."""
    B, S, H, D = 2, 70000, 128, 128  # 2.3e9 elements
    free, _ = torch.cuda.mem_get_info()
    if free < 3 * B * S * H * D * 2:
        pytest.skip("not enough device memory")
    plan = uaa.RotaryPlan([128])
    q = torch.zeros(B, S, H, D, device=DEV, dtype=torch.bfloat16)
    q[-1, -3:] = torch.randn(3, H, D, device=DEV)
    y = uaa.rotary_fwd(q, None, plan)[0]
    tail = uaa.rotary_fwd(q[-1:, -3:].contiguous(), None, plan, start=S - 3)[0]
    assert torch.equal(y[-1:, -3:], tail) and not y[0, :5].any()
