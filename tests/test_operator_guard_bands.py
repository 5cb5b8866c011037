"""Out-of-bounds writes of rotary positions, 8-bit checkpoints and differential attention: every output and workspace lies
between canary bytes, which must be unchanged after the calls."""
import ctypes

import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from test_gpu_guard_bands import Guarded

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("Sq,Sk", [(1, 1), (1, 1000), (2, 129), (3, 700), (127, 81), (129, 257), (600, 79), (130, 640)])
@pytest.mark.parametrize("D,mask", [(64, None), (128, None), (64, "part"), (128, "part"), (128, "empty")])
def test_differential_attention(Sq, Sk, D, mask):
    B, H = 2, 3
    gen = torch.Generator(DEV).manual_seed(Sq * 1000 + Sk)
    q, do = (torch.randn(B, Sq, H, D, generator=gen, device=DEV).bfloat16() for _ in range(2))
    k, v = (torch.randn(B, Sk, H, D, generator=gen, device=DEV).bfloat16() for _ in range(2))
    m = None
    if mask:
        m = torch.rand(B, Sk, generator=gen, device=DEV) < 0.5
        m[0] = m[0] & (mask == "part")
    for dtype in (torch.bfloat16, torch.float32):
        g = Guarded()
        lam = torch.rand(H, generator=gen, device=DEV).to(dtype)
        out, out2, dq = (g.empty(q.shape, torch.bfloat16) for _ in range(3))
        dk, dv = (g.empty(k.shape, torch.bfloat16) for _ in range(2))
        lse, dlam = g.empty((B, H, 2, Sq), torch.float32), g.empty((H,), dtype)
        ws = g.empty((uaa.diff_attn_bwd_workspace_bytes(B, Sq, Sk, H, D),), torch.uint8)
        uaa.diff_attn_fwd(q, k, v, lam, m, out=out, out2=out2, lse=lse)
        uaa.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, m, dq=dq, dk=dk, dv=dv, dlam=dlam, workspace=ws)
        uaa.check_device_status()
        g.check()
        for t in (out, out2, dq, dk, dv, dlam):
            assert torch.isfinite(t.float()).all()


@pytest.mark.parametrize("D,rot,layout", [(64, 64, "half"), (64, 40, "interleaved"), (66, 66, "half"), (80, 50, "half"),
                                          (80, 78, "interleaved"), (7, 6, "half"), (256, 250, "half")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rotary(D, rot, layout, dtype):
    plan = uaa.RotaryPlan([rot], layout=layout)
    for B, S, Hq, Hk in ((1, 1, 1, 1), (2, 37, 3, 2), (1, 1000, 5, 1)):
        q, k = (torch.randn(B, S, h, D, device=DEV).to(dtype) for h in (Hq, Hk))
        g = Guarded()
        yq, yk = g.empty(q.shape, dtype), g.empty(k.shape, dtype)
        uaa.rotary_fwd(q, k, plan, out_q=yq, out_k=yk)
        g.check()
        # one column to the right of the guarded buffer's start, and heads apart: between the rows, nothing is written
        wide = torch.full((B, S, Hq, D + 3), 7.0, dtype=dtype, device=DEV)
        uaa.rotary_fwd(q, None, plan, out_q=wide[..., 1:1 + D])
        assert torch.equal(wide[..., 1:1 + D], yq) and (wide[..., 0] == 7).all() and (wide[..., 1 + D:] == 7).all()
    uaa.check_device_status()


@pytest.mark.parametrize("D", [16, 48, 64, 80, 128, 336, 512])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_checkpoints(D, dtype):
    rows = (1, 33, 0, 700)
    xs = [torch.randn(r, D, device=DEV).to(dtype) for r in rows]
    g = Guarded()
    codes, steps = [g.empty(x.shape, torch.int8) for x in xs], [g.empty((r,), torch.float32) for r in rows]
    ys = [g.empty(x.shape, dtype) for x in xs]
    arr = lambda ts: (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])  # noqa: E731
    n, kind, stream = (ctypes.c_longlong * len(rows))(*rows), uaa._DTYPES[dtype], torch.cuda.current_stream().cuda_stream
    L = uaa.lib()
    assert L.uaa_act8_pack(4, arr(xs), arr(codes), arr(steps), n, D, kind, stream) == 0
    assert L.uaa_act8_unpack(4, arr(codes), arr(steps), arr(ys), n, D, kind, stream) == 0
    uaa.check_device_status()
    g.check()
    for y, want in zip(ys, uaa.act8_unpack(uaa.act8_pack(xs))):
        assert torch.equal(y, want)


@pytest.mark.parametrize("Sq,Sk", [(1, 130), (200, 77)])
def test_backward_from_a_checkpoint(Sq, Sk):
    B, H, D = 2, 3, 64
    q, do = (torch.randn(B, Sq, H, D, device=DEV).bfloat16() for _ in range(2))
    k, v = (torch.randn(B, Sk, H, D, device=DEV).bfloat16() for _ in range(2))
    out, lse = uaa.attn_fwd(q, k, v)
    packed = uaa.act8_pack([q, k, v, out])
    g = Guarded()
    dq, dk, dv = (g.empty(t.shape, torch.bfloat16) for t in (q, k, v))
    ws = g.empty((int(uaa.lib().uaa_attn_bwd_act8_workspace_bytes(B, Sq, Sk, H, D)),), torch.uint8)
    uaa.attn_bwd_act8(packed, do, lse, dq=dq, dk=dk, dv=dv, workspace=ws)
    uaa.check_device_status()
    g.check()
