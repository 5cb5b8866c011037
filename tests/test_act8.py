"""Activation checkpoints in 8 bits: codes and steps against the definition, bit for bit, and their use by the
attention's backward pass."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import ulysses_dit_attention_gb300 as uaa
from oracle import ops
from ulysses_dit_attention_gb300 import synth
from helpers import bits, compare, f64

DEV = "cuda"


def test_refusals_of_the_call():
    L = uaa.lib()
    err = lambda: L.uaa_last_error().decode()  # noqa: E731
    arr, rows = (ctypes.c_void_p * 1), (ctypes.c_longlong * 1)

    def pack(x=4096, codes=4096, steps=4096, r=4, D=64, dtype=0, n=1):
        return L.uaa_act8_pack(n, arr(x), arr(codes), arr(steps), rows(r), D, dtype, None)

    assert pack(x=None) == -1 and "NULL" in err()
    assert pack(x=4104) == -1 and "16-byte" in err()
    assert pack(codes=4104) == -1 and "16-byte" in err()
    assert pack(steps=4098) == -1 and "4-byte" in err()
    assert pack(D=0) == -1 and pack(D=40) == -2 and pack(D=528) == -2 and pack(dtype=9) == -1
    assert pack(n=9) == -1 and pack(n=-1) == -1 and pack(r=-1) == -1
    assert pack(r=0, x=None) == 0 and pack(n=0) == 0
    # the backward from a checkpoint: its own workspace holds the four tensors and the backward's
    B, Sq, Sk, H, D = 1, 130, 300, 2, 64
    need = L.uaa_attn_bwd_act8_workspace_bytes(B, Sq, Sk, H, D)
    assert need == 4 * (Sq + Sk) * H * D + L.uaa_attn_bwd_workspace_bytes(B, Sq, H, D)
    f, four = ctypes.c_void_p(1 << 20), (ctypes.c_void_p * 4)(*[1 << 20] * 4)

    def bwd(codes=four, dout=f, lse=f, D=D, Sq=Sq, ws=f, n=need):
        return L.uaa_attn_bwd_act8(codes, four, dout, lse, None, f, f, f, B, Sq, Sk, H, D, ctypes.c_float(0.1), ws, n, None)

    assert bwd(n=need - 1) == -1 and "workspace" in err()
    assert bwd(ws=ctypes.c_void_p((1 << 20) + 64)) == -1 and "256-byte" in err()
    assert bwd(codes=None) == -1 and bwd(dout=None) == -1 and bwd(lse=None) == -1 and bwd(D=96) == -2 and bwd(Sq=0) == -1
    assert L.uaa_act8_unpack(1, arr(4096), arr(4096), arr(None), rows(4), 64, 0, None) == -1


def test_refusals_without_gpu():
    with pytest.raises(ValueError, match="CUDA"):
        uaa.act8_pack(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        uaa.act8_pack([])
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        uaa.attention(q, q, q, saved="int4")


def _expect(x):
    codes, top = ops.act8_codes(x.detach().cpu().double().numpy())
    t32 = torch.tensor(top, dtype=torch.float64).float()
    # the step: top / 127 rounded toward zero to 32 bits
    step = torch.tensor(top / 127.0, dtype=torch.float64)
    near = step.float()
    down = torch.where(near.double() > step, torch.nextafter(near, torch.zeros_like(near)), near)
    down = torch.where(t32.double() < 2.0 ** -119, torch.zeros_like(down), down)
    return codes, down


def _check(packed, xs):
    got = uaa.act8_unpack(packed)
    at = 0
    for x, y in zip(xs, got):
        codes, step = _expect(x)
        D, r = x.shape[-1], x.numel() // x.shape[-1]
        c = packed.codes[at * D:(at + r) * D].cpu().numpy().reshape(codes.shape)
        s = packed.steps[at:at + r].cpu().reshape(step.shape)
        assert np.array_equal(c, codes)
        assert torch.equal(s, step)
        want = (torch.tensor(codes, dtype=torch.float32) * step.unsqueeze(-1)).to(x.dtype)
        assert np.array_equal(bits(y), bits(want))
        at += r


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shapes", [[(1, 64)], [(3, 5, 7, 128)], [(33, 16)], [(9, 80), (4, 80), (1, 80)],
                                    [(17, 512), (0, 512), (2, 512)], [(129, 32)] * 8, [(5, 336)]])
def test_codes_and_values(shapes, dtype):
    g = torch.Generator().manual_seed(len(shapes) * 100 + shapes[0][-1])
    xs = [(torch.randn(s, generator=g) * torch.exp(torch.randn(s[-1], generator=g))).to(dtype).to(DEV) for s in shapes]
    packed = uaa.act8_pack(xs)
    uaa.check_device_status()
    _check(packed, xs)
    assert packed.nbytes == sum(x.numel() + 4 * (x.numel() // x.shape[-1]) for x in xs)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_borders_and_special_rows(dtype):
    D = 64
    rows = [torch.zeros(D)]
    for top in (1.0, 127.0, 2.54, 3.0e38, 1e-30, 2.0 ** -119, 2.0 ** -120, 1e-44):
        r = torch.full((D,), top)
        # every border between two codes, as near as the type allows, and a step to either side
        mid = ((torch.arange(D - 1) * 2 + 1).double() * top / 254.0).to(dtype).float()
        r[:D - 1] = torch.where(torch.arange(D - 1) % 2 == 0, mid, -mid)
        rows += [r, torch.nextafter(r, torch.zeros(D)), torch.nextafter(r, r.sign() * 3.3e38)]
        rows[-1][D - 1] = rows[-2][D - 1] = top
    x = torch.stack(rows).to(dtype).to(DEV)
    _check(uaa.act8_pack([x]), [x])
    half = torch.full((1, D), 3.0)
    half[0, 1:] = 1.5  # 63.5 steps: to the even code, 64
    packed = uaa.act8_pack(half.to(dtype).to(DEV))
    assert packed.codes.cpu().tolist()[:2] == [127, 64]


@pytest.mark.gpu
def test_every_bf16_pair():
    """Every significand under every top's, at every scale where it has a code."""
    X = torch.cat([torch.arange(128, 256).double() * 2.0 ** -s for s in range(11)])
    X = torch.cat((X, -X))
    rows = []
    for T in range(128, 256):
        x = X[X.abs() <= T]
        x = torch.cat((x, torch.zeros(-len(x) % 511))).view(-1, 511)
        rows.append(torch.cat((torch.full((len(x), 1), float(T)), x), 1))
    x = torch.cat(rows).bfloat16().to(DEV)
    assert torch.equal(x.cpu().double(), torch.cat(rows).double())
    _check(uaa.act8_pack([x]), [x])


@pytest.mark.gpu
def test_what_is_not_finite_shows():
    x = torch.randn(6, 128, device=DEV)
    x[1, 3], x[2, 127], x[4, 0] = math.inf, math.nan, -math.inf
    y = uaa.act8_unpack(uaa.act8_pack(x))
    bad = torch.tensor([False, True, True, False, True, False], device=DEV)
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


@pytest.mark.gpu
def test_empty_and_refused():
    assert uaa.act8_unpack(uaa.act8_pack(torch.empty(0, 64, device=DEV))).shape == (0, 64)
    x = torch.randn(4, 64, device=DEV)
    for bad, kind in (([x, x.bfloat16()], TypeError), ([x, torch.zeros(2, 32, device=DEV)], ValueError),
                      ([x.t()], ValueError), ([x] * 9, ValueError), ([x.double()], TypeError),
                      ([torch.zeros(2, 40, device=DEV)], uaa.UAAError), ([x, x.cpu()], ValueError)):
        with pytest.raises(kind):
            uaa.act8_pack(bad)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    rows, D = (1 << 23) + 70001, 512  # 4.3e9 elements
    free, _ = torch.cuda.mem_get_info()
    if free < 6 * rows * D:
        pytest.skip("not enough device memory")
    x = torch.zeros(rows, D, device=DEV, dtype=torch.bfloat16)
    x[-5:] = torch.randn(5, D, device=DEV)
    packed = uaa.act8_pack(x)
    _check(uaa.act8_pack([x[-5:].clone()]), [x[-5:]])
    assert torch.equal(packed.codes[-5 * D:], uaa.act8_pack(x[-5:].clone()).codes)
    y = uaa.act8_unpack(packed)
    assert torch.equal(y[-5:], uaa.act8_unpack(uaa.act8_pack(x[-5:].clone()))) and not y[:9].any()


def _values(x):
    return uaa.act8_unpack(uaa.act8_pack(x))


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,H,D,masked", [(2, 200, 3, 128, True), (1, 333, 2, 64, False)])
def test_attention_backward_from_the_checkpoint(B, S, H, D, masked):
    """The gradients are those of attn_bwd on the values of the codes, bit for bit; those are near the gradients
    of the unrounded step: a value is off by half a step of max/127, about 0.01 of the row's rms."""
    inp = synth.draw(B, S, H, D, seed=5, masked=masked)
    q, k, v, do = (inp[n].to(DEV) for n in ("q", "k", "v", "do"))
    mask = inp["mask"].to(DEV) if masked else None
    leaves = [t.requires_grad_() for t in (q, k, v)]
    out, lse = uaa.attention(*leaves, mask, saved="int8")
    grads = torch.autograd.grad(out, leaves, do)
    plain, _ = uaa.attention(*leaves, mask)
    assert torch.equal(out, plain)
    kept = [_values(t.detach()) for t in (q, k, v, out)]
    want = uaa.attn_bwd(*kept, do, lse, mask)
    for name, a, w in zip(("dq", "dk", "dv"), grads, want):
        assert np.array_equal(bits(a), bits(w)), name
    packed = uaa.act8_pack([t.detach() for t in (q, k, v, out)])
    for a, w in zip(uaa.attn_bwd_act8(packed, do, lse, mask), want):
        assert np.array_equal(bits(a), bits(w))
    with pytest.raises(ValueError):
        uaa.attn_bwd_act8(uaa.act8_pack([q.detach()] * 3), do, lse, mask)
    m = inp["mask"].numpy().astype(bool) if masked else None
    ref = oracle.attn_bwd(*(f64(t) for t in (q, k, v, do)), m, 1 / math.sqrt(D))
    for a, r in zip(grads, ref):
        # 0.6 % of rms in each of q, k, v, o; two of them meet in a product, and dS = P (dP - Delta)
        assert np.linalg.norm(f64(a) - r) <= 0.05 * np.linalg.norm(r)


@pytest.mark.gpu
def test_attention_across_lengths_from_the_checkpoint():
    q, do = (torch.randn(2, 70, 3, 64, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    k, v = (torch.randn(2, 200, 3, 64, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    mask = torch.rand(2, 200, device=DEV) < 0.5
    leaves = [t.requires_grad_() for t in (q, k, v)]
    out, lse = uaa.attention(*leaves, mask, 0.2, saved="int8")
    got = torch.autograd.grad(out, leaves, do)
    want = uaa.attn_bwd(*(_values(t.detach()) for t in (q, k, v, out)), do, lse, mask, 0.2)
    for a, w in zip(got, want):
        assert np.array_equal(bits(a), bits(w))
    assert torch.equal(uaa.attention(*(t.detach() for t in leaves), mask, 0.2, saved="int8")[0], out)  # nothing to keep


@pytest.mark.gpu
def test_memory_kept_between_the_passes():
    q, k, v = (torch.randn(1, 4096, 8, 128, device=DEV, dtype=torch.bfloat16, requires_grad=True) for _ in range(3))
    kept = {}
    for saved in (None, "int8"):
        seen = []
        with torch.autograd.graph.saved_tensors_hooks(lambda t: seen.append(t) or t, lambda t: t):
            uaa.attention(q, k, v, saved=saved)
        kept[saved] = sum(t.numel() * t.element_size() for t in seen)
    rows = 4096 * 8
    assert kept[None] == rows * (4 * 256 + 4) and kept["int8"] == rows * (4 * 132 + 4)


@pytest.mark.gpu
@pytest.mark.parametrize("fused", [False, True])
def test_ulysses_step_from_the_checkpoint(fused):
    lens, cap, B, H, D = (70, 71, 60), 71, 1, 5, 64
    call = uaa.ulysses_attention_fused if fused else uaa.ulysses_attention
    inp = synth.draw(B, sum(lens), H, D, seed=9, masked=False)
    sh = [synth.pad_shards(inp[n], lens, cap).to(DEV).requires_grad_() for n in ("q", "k", "v")]
    do = synth.pad_shards(inp["do"], lens, cap).to(DEV)
    out, _ = call(*sh, lens)
    ref = torch.autograd.grad(out, sh, do)
    out8, _ = call(*sh, lens, saved="int8")
    got = torch.autograd.grad(out8, sh, do)
    assert torch.equal(out, out8)
    for a, r in zip(got, ref):
        assert not torch.equal(a, r) and torch.linalg.norm((a - r).float()) <= 0.05 * torch.linalg.norm(r.float())


@pytest.mark.gpu
def test_captured_step():
    """Pack, unpack and the backward in one graph, replayed on new inputs."""
    q, k, v, do = (torch.randn(1, 300, 2, 128, device=DEV, dtype=torch.bfloat16) for _ in range(4))

    def step():
        out, lse = uaa.attn_fwd(q, k, v)
        kept = uaa.act8_unpack(uaa.act8_pack([q, k, v, out]))
        return uaa.attn_bwd(*kept, do, lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for t in (q, k, v, do):
        t.normal_()
    graph.replay()
    for a, w in zip(res, step()):
        assert torch.equal(a, w)
    uaa.check_device_status()
