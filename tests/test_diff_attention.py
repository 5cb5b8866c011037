"""Differential attention against the float64 definition, within the error that the operands' roundings allow."""
import ctypes
import math
import threading

import numpy as np
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from oracle import ops
from helpers import bits, f64

DEV = "cuda"


# --------------------------------------------------------------------------- the definition itself
def test_definition_against_differences():
    """The oracle's gradients against central differences of its outputs."""
    rng = np.random.default_rng(1)
    q, k, v, g = (rng.standard_normal((2, n, 2, 8)) for n in (3, 5, 5, 3))
    lam, mask = np.array([0.3, -0.7]), np.array([[1, 1, 0, 1, 1], [1, 0, 0, 0, 0]], bool)
    res = ops.diff_attn(q, k, v, lam, mask, 0.6, g)

    def loss(q, k, v, lam):
        return (ops.diff_attn(q, k, v, lam, mask, 0.6)["out"][0] * g).sum()

    args, h = [q, k, v, lam], 1e-5
    for n, name in enumerate(("dq", "dk", "dv", "dlam")):
        for at in list(np.ndindex(args[n].shape))[::3]:
            up, down = ([a.copy() for a in args] for _ in range(2))
            up[n][at] += h
            down[n][at] -= h
            assert abs((loss(*up) - loss(*down)) / (2 * h) - res[name][0][at]) < 1e-8, (name, at)


def test_definition_special_cases():
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((1, n, 1, 8)) for n in (4, 6, 6))
    zero = ops.diff_attn(q, k, v, np.array([0.0]))["out"][0]  # lambda = 0: the first map alone
    a = np.exp(q[0, :, 0, :4] @ k[0, :, 0, :4].T / 2.0)
    assert np.allclose(zero[0, :, 0], a / a.sum(-1, keepdims=True) @ v[0, :, 0], atol=1e-12)
    same = np.concatenate([q[..., :4]] * 2, -1), np.concatenate([k[..., :4]] * 2, -1)
    assert np.allclose(ops.diff_attn(*same, v, np.array([1.0]))["out"][0], 0, atol=1e-12)  # equal maps cancel
    none = ops.diff_attn(q, k, v, np.array([0.5]), np.zeros((1, 6), bool), dout=q)
    assert all(not none[n][0].any() for n in ("out", "out2", "dq", "dk", "dv", "dlam"))
    assert (none["lse"][0] == -np.inf).all()


# --------------------------------------------------------------------------- refusals
def test_refusals_of_the_call():
    L, P = uaa.lib(), ctypes.c_void_p
    err = lambda: L.uaa_last_error().decode()  # noqa: E731
    f = P(1 << 20)

    def fwd(q=f, lam=f, lt=0, out2=f, lse=f, B=1, Sq=4, Sk=4, D=64, scale=0.1):
        return L.uaa_diff_attn_fwd(q, f, f, lam, lt, None, f, out2, lse, B, Sq, Sk, 2, D, ctypes.c_float(scale), None)

    assert fwd(D=96) == -2 and "D=96" in err()
    assert fwd(scale=0.0) == -1 and "scale" in err()
    assert fwd(q=None) == -1 and "q is NULL" in err()
    assert fwd(q=P((1 << 20) + 8)) == -1 and "aligned" in err()
    assert fwd(out2=P((1 << 20) + 8)) == -1 and "out2" in err()
    assert fwd(lam=None) == -1 and "lambda" in err()
    assert fwd(lt=1) == -1 and "lambda" in err()
    assert fwd(lam=P((1 << 20) + 1)) == -1 and "lambda" in err()
    assert fwd(lse=None) == -1 and "lse" in err()
    assert fwd(Sk=0) == -1 and "keys" in err()
    assert fwd(q=None, Sq=0) == 0 and fwd(q=None, B=0) == 0

    def bwd(ws=P(1 << 24), n=1 << 30, Sq=4, out2=f, dlam=f):
        return L.uaa_diff_attn_bwd(f, f, f, f, 0, f, out2, f, f, None, f, f, f, dlam, 1, Sq, 4, 2, 64,
                                   ctypes.c_float(0.1), ws, n, None)

    assert bwd(n=16) == -1 and "workspace" in err()
    assert bwd(ws=P((1 << 24) + 16)) == -1 and "256-byte" in err()
    assert bwd(out2=None) == -1 and "out2" in err()
    assert bwd(dlam=None) == -1 and "lambda" in err()
    assert bwd(Sq=0) == -1 and "queries" in err()
    # per head Delta and -LSE*log2(e) of two maps, rows padded to 128, a sum per 64 rows and one per 128 keys
    assert L.uaa_diff_attn_bwd_workspace_bytes(2, 130, 300, 3, 128) == 2 * 3 * (256 * 4 + 4 + 3) * 4 // 256 * 256 + 256
    assert L.uaa_diff_attn_bwd_workspace_bytes(2, 130, 300, 3, 96) == 0


def test_refusals_without_gpu():
    q, lam = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        uaa.diff_attn_fwd(q, q, q, lam)
    with pytest.raises(ValueError, match="lam"):
        uaa.diff_attn_fwd(q, q, q, torch.zeros(3))
    with pytest.raises(TypeError, match="lam"):
        uaa.diff_attn_fwd(q, q, q, lam.double())
    with pytest.raises(ValueError, match="per-head"):
        uaa.diff_attn_fwd(q, q, q, lam, torch.ones(1, 2, 1, 4, dtype=torch.bool))
    with pytest.raises(ValueError, match="fit"):
        uaa.diff_attn_fwd(q, q[:, :, :1].contiguous(), q, lam)


# --------------------------------------------------------------------------- the kernels
def draw(B, Sq, Sk, H, D, mask=None, seed=0, peak=1.0):
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randn(B, n, H, D, generator=g).bfloat16() for n in (Sq, Sk, Sk, Sq))
    q = (q * peak).bfloat16()
    lam = (torch.rand(H, generator=g) * 1.2 - 0.2).bfloat16()
    m = None
    if mask == "prefix":
        m = torch.arange(Sk)[None] < torch.randint(max(1, Sk // 2), Sk + 1, (B, 1), generator=g)
    elif mask == "random":
        m = torch.rand(B, Sk, generator=g) < 0.5
    elif mask == "sparse":  # whole tiles without an attended key, between tiles with one
        m = torch.zeros(B, Sk, dtype=torch.bool)
        m[:, ::301] = True
    elif mask == "empty":
        m = torch.rand(B, Sk, generator=g) < 0.7
        m[0] = False
    elif mask == "none":
        m = torch.zeros(B, Sk, dtype=torch.bool)
    return dict(q=q, k=k, v=v, do=do, lam=lam, mask=m)


def on_gpu(x):
    return {n: None if t is None else t.to(DEV) for n, t in x.items()}


def step(x, scale=None):
    out, out2, lse = uaa.diff_attn_fwd(x["q"], x["k"], x["v"], x["lam"], x["mask"], scale)
    dq, dk, dv, dlam = uaa.diff_attn_bwd(x["q"], x["k"], x["v"], x["lam"], out, out2, x["do"], lse, x["mask"], scale)
    uaa.check_device_status()
    return dict(out=out, out2=out2, lse=lse, dq=dq, dk=dk, dv=dv, dlam=dlam)


def against_definition(x, got, scale=None, names=None):
    m = None if x["mask"] is None else x["mask"].numpy()
    lam = x["lam"].double().numpy()
    ref = ops.diff_attn(f64(x["q"]), f64(x["k"]), f64(x["v"]), lam, m, scale, f64(x["do"]))
    for n in names or got:
        if got[n] is None:
            continue
        value, bound = ref[n]
        g = got[n].detach().cpu().double().numpy()
        fin = np.isfinite(value)
        assert np.array_equal(g[~fin], value[~fin]), n
        over = np.abs(g[fin] - value[fin]) - bound[fin]
        assert (over <= 1e-30).all(), f"{n}: {over.max():.3e} over a bound of {bound[fin][over.argmax()]:.3e}"
    if m is not None:  # masked keys: exactly nothing
        for n in ("dk", "dv"):
            if n in got:
                assert not got[n].detach().cpu().float().numpy()[~m].any(), n


SHAPES = [
    # B, Sq, Sk, H, D, mask
    (1, 1, 1, 1, 64, None),
    (1, 1, 1, 2, 128, None),
    (2, 1, 300, 3, 128, "random"),
    (1, 3, 1000, 2, 64, "prefix"),
    (2, 5, 257, 2, 128, "empty"),
    (1, 16, 16, 16, 64, None),
    (2, 127, 127, 2, 128, None),
    (1, 128, 128, 3, 64, "random"),
    (2, 129, 129, 2, 128, "prefix"),
    (1, 255, 700, 2, 128, None),
    (1, 700, 77, 2, 64, "prefix"),
    (3, 200, 513, 2, 64, "empty"),
    (2, 130, 900, 1, 128, "sparse"),
    (1, 64, 130, 1, 128, "none"),
    (1, 600, 600, 2, 64, None),
    (1, 513, 640, 1, 128, None),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", SHAPES, ids=["-".join(map(str, c)) for c in SHAPES])
def test_step(case):
    B, Sq, Sk, H, D, mask = case
    x = draw(B, Sq, Sk, H, D, mask, seed=Sq + Sk)
    against_definition(x, step(on_gpu(x)))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale,peak", [(0.37, 1.0), (None, 6.0), (0.01, 1.0)])
def test_scales_and_peaked_rows(D, scale, peak):
    x = draw(1, 190, 270, 2, D, "prefix", seed=3, peak=peak)
    against_definition(x, step(on_gpu(x), scale), scale)


@pytest.mark.gpu
@pytest.mark.parametrize("lam", [0.0, 1.0, -0.5, 3.0])
def test_lambda_values_and_types(lam):
    x = draw(1, 140, 150, 2, 64, None, seed=4)
    x["lam"] = torch.tensor([lam, 0.25], dtype=torch.float32)
    got = step(on_gpu(x))
    assert got["dlam"].dtype == torch.float32
    against_definition(x, got)


@pytest.mark.gpu
@pytest.mark.parametrize("D,mask", [(64, None), (128, "random")])
def test_dlambda_does_not_hang_on_the_rounding_of_out2(D, mask):
    """dlambda is a sum of A_2 dA, whatever out2 holds: with the forward's, and with zeros in its place."""
    x = draw(2, 500, 400, 3, D, mask, seed=16)
    x["lam"] = torch.tensor([0.5, -0.3, 1e-3])
    g = on_gpu(x)
    out, out2, lse = uaa.diff_attn_fwd(g["q"], g["k"], g["v"], g["lam"], g["mask"])
    q2, k2 = (f64(x[n])[..., D // 2:].transpose(0, 2, 1, 3) for n in "qk")
    s = q2 @ k2.transpose(0, 1, 3, 2) / math.sqrt(D / 2)
    if mask:
        s = np.where(x["mask"].numpy()[:, None, None], s, -np.inf)
    a2 = np.exp(s - s.max(-1, keepdims=True))
    a2 /= a2.sum(-1, keepdims=True)
    da = f64(x["do"]).transpose(0, 2, 1, 3) @ f64(x["v"]).transpose(0, 2, 3, 1)
    want = -(a2 * da).sum((0, 2, 3))
    # a probability is off by 2^-18 (an exponent below 32 in 32 bits, ex2 2^-22), so A_2 sums to 1 within that and a row
    # sum is off by so much of its summands; adding up 400 keys and 1000 rows in 32 bits, in parts of at most 64: 2^-17
    bound = 2.0 ** -16 * (a2 * np.abs(da)).sum((0, 2, 3))
    for o2 in (out2, torch.zeros_like(out2)):
        dlam = uaa.diff_attn_bwd(g["q"], g["k"], g["v"], g["lam"], out, o2, g["do"], lse, g["mask"])[3]
        err = np.abs(dlam.cpu().double().numpy() - want)
        assert (err <= bound).all(), (err, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_forward_without_gradient(D):
    for Sq in (1, 2, 130):
        x = on_gpu(draw(2, Sq, 400, 2, D, "random", seed=6))
        a = uaa.diff_attn_fwd(x["q"], x["k"], x["v"], x["lam"], x["mask"])
        b = uaa.diff_attn_fwd(x["q"], x["k"], x["v"], x["lam"], x["mask"], need_out2=False)
        assert b[1] is None and torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq", [1, 4, 200, 600])
@pytest.mark.parametrize("value", [3e4, float("inf"), float("nan")])
def test_what_is_masked_does_not_matter(D, Sq, value):
    """Whatever a masked key's rows of K and V hold, infinities and NaN too: every result has the same bits."""
    x = draw(1, Sq, 333, 2, D, "random", seed=8)
    y = {n: None if t is None else t.clone() for n, t in x.items()}
    dead = ~x["mask"][0]
    y["k"][0, dead] = value
    y["v"][0, dead] = -value
    a, b = step(on_gpu(x)), step(on_gpu(y))
    for n in a:
        assert np.array_equal(bits(a[n]), bits(b[n])), n


@pytest.mark.gpu
@pytest.mark.parametrize("Sq", [1, 3, 130, 1030])
def test_keys_past_32_bits(Sq):
    """Offsets of K, V, dK and dV past 2^31 elements: only the last keys are attended, and the results are those of
    the short problem that has no others.  Its start is a border between tiles of both kernels (80 and 128 keys)."""
    Sk, start, H, D = 139008, 133120, 128, 128
    assert start * H * D > 2**31 and start % 640 == 0
    g = torch.Generator(DEV).manual_seed(41)
    new = lambda n: torch.randn(1, n, H, D, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    q, do, k, v = new(Sq), new(Sq), new(Sk), new(Sk)
    lam = torch.rand(H, generator=g, device=DEV)
    mask = torch.zeros(1, Sk, dtype=torch.bool, device=DEV)
    mask[:, start:] = True
    mask[:, -3] = False
    long = step(dict(q=q, k=k, v=v, do=do, lam=lam, mask=mask))
    cut = lambda t: t[:, start:].contiguous()  # noqa: E731
    short = step(dict(q=q, k=cut(k), v=cut(v), do=do, lam=lam, mask=cut(mask)))
    for n in ("dk", "dv"):
        assert not long[n][:, :start].any(), n
        long[n] = cut(long[n])
    if Sq <= 2:
        # The few-row kernel splits the keys by their number, so the forward's sums have another order.  A lane group
        # adds at most 400 of the products A v (5888 keys over 16 groups) and eight joins follow, so a sum is within
        # 408 * 2^-24 * sum A |v| < 2^-11, as |v| < 8 and the weights sum to 1 + lambda < 2; then a step of bf16.
        assert v.abs().max() < 8
        for n in ("out", "out2", "lse"):
            assert torch.allclose(long[n].float(), short[n].float(), rtol=2**-7, atol=2**-11), n
        short.update(zip(("dq", "dk", "dv", "dlam"),
                         uaa.diff_attn_bwd(q, cut(k), cut(v), lam, long["out"], long["out2"], do, long["lse"], cut(mask))))
    for n in ("out", "out2", "lse", "dq", "dk", "dv"):
        if Sq > 2 or n[0] == "d":
            assert torch.equal(long[n], short[n]), n
    # dlambda adds the same sums of key tiles in another order, at most eight of them that are not 0 on the way of one:
    # 2 * 8 * 2^-24 of their magnitudes, which come to 2 max_j |dA_ij| a row at most (A_2 sums to 1, Delta_2 is a mean of
    # dA), and |dA_ij| <= |do_i| |v_j|
    size = 2 * do.float().norm(dim=-1).sum((0, 1)) * v.float().norm(dim=-1).max()
    assert ((long["dlam"] - short["dlam"]).abs() <= 2**-20 * size).all()


@pytest.mark.gpu
def test_queries_past_32_bits():
    """Offsets of Q, O, dO and dQ past 2^31 elements: the last rows are those of the short problem."""
    Sq, start, H, D, Sk = 136000, 133120, 128, 128, 100
    assert start * H * D > 2**31 and start % 128 == 0
    g = torch.Generator(DEV).manual_seed(42)
    new = lambda n: torch.randn(1, n, H, D, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    q, do, k, v = new(Sq), new(Sq), new(Sk), new(Sk)
    lam = torch.rand(H, generator=g, device=DEV)
    long = step(dict(q=q, k=k, v=v, do=do, lam=lam, mask=None))
    cut = lambda t: t[:, start:].contiguous()  # noqa: E731
    short = step(dict(q=cut(q), k=k, v=v, do=cut(do), lam=lam, mask=None))
    for n in ("out", "out2", "dq"):
        assert torch.equal(cut(long[n]), short[n]), n
    assert torch.equal(long["lse"][..., start:], short["lse"])


@pytest.mark.gpu
@pytest.mark.parametrize("saved", [None, "int8"])
def test_captured_autograd_step(saved):
    """Forward and gradients by autograd, captured after a warm-up on another stream, replayed on new inputs."""
    x = on_gpu(draw(2, 200, 210, 2, 128, "prefix", seed=43))
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "lam")]

    def run():
        out, _ = uaa.diff_attention(*leaves, x["mask"], saved=saved)
        return (out.detach(),) + torch.autograd.grad(out, leaves, x["do"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    with torch.no_grad():
        for n in ("q", "k", "v", "do"):
            x[n].normal_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, w in zip(got, run()):
        assert np.array_equal(bits(a), bits(w))
    uaa.check_device_status()


@pytest.mark.gpu
def test_same_bits_every_time():
    x = on_gpu(draw(2, 500, 600, 3, 128, "prefix", seed=10))
    first = step(x)
    for _ in range(5):
        again = step(x)
        assert all(np.array_equal(bits(first[n]), bits(again[n])) for n in first)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [(4, 700, 300, 24, 64, None), (3, 300, 900, 30, 128, "prefix"),
                                  (2, 520, 130, 60, 128, None), (5, 130, 1100, 20, 64, "empty")],
                         ids=["queries", "masked", "few-keys", "empty"])
def test_many_items_a_block(case):
    """More tiles than the device has SMs, shared out in several ways: every sequence's results are those of a call of
    its own."""
    B, Sq, Sk, H, D, mask = case
    x = on_gpu(draw(B, Sq, Sk, H, D, mask, seed=50))
    whole = step(x)
    for b in range(B):
        one = step({n: t if t is None or n == "lam" else t[b:b + 1].contiguous() for n, t in x.items()})
        for n in ("out", "out2", "lse", "dq", "dk", "dv"):
            assert np.array_equal(bits(whole[n][b:b + 1]), bits(one[n])), (b, n)


@pytest.mark.gpu
def test_many_mask_rows():
    x = draw(300, 40, 140, 1, 64, "random", seed=11)
    x["mask"][7] = False
    against_definition(x, step(on_gpu(x)))


@pytest.mark.gpu
def test_autograd():
    x = draw(2, 150, 170, 2, 128, "prefix", seed=12)
    gx = on_gpu(x)
    leaves = [gx[n].requires_grad_() for n in ("q", "k", "v", "lam")]
    out, lse = uaa.diff_attention(*leaves, gx["mask"])
    assert not lse.requires_grad
    grads = torch.autograd.grad(out, leaves, gx["do"])
    against_definition(x, dict(zip(("dq", "dk", "dv", "dlam"), grads)))
    # a gradient without memory of its own
    out, _ = uaa.diff_attention(*leaves, gx["mask"])
    ones = torch.autograd.grad(out.sum(), leaves)
    out, _ = uaa.diff_attention(*leaves, gx["mask"])
    for a, b in zip(ones, torch.autograd.grad(out, leaves, torch.ones_like(out))):
        assert torch.equal(a, b)
    with torch.no_grad():
        assert torch.equal(uaa.diff_attention(*leaves, gx["mask"])[0], out)


@pytest.mark.gpu
def test_backward_from_the_checkpoint():
    x = on_gpu(draw(1, 260, 300, 2, 128, "random", seed=13))
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "lam")]
    out, lse = uaa.diff_attention(*leaves, x["mask"], saved="int8")
    grads = torch.autograd.grad(out, leaves, x["do"])
    o, o2, l2 = uaa.diff_attn_fwd(*(t.detach() for t in leaves), x["mask"])
    q, k, v, oo, oo2 = uaa.act8_unpack(uaa.act8_pack([x["q"].detach(), x["k"].detach(), x["v"].detach(), o, o2]))
    want = uaa.diff_attn_bwd(q, k, v, x["lam"].detach(), oo, oo2, x["do"], l2, x["mask"])
    for a, w in zip(grads, want):
        assert np.array_equal(bits(a), bits(w))


@pytest.mark.gpu
@pytest.mark.parametrize("saved", [None, "int8"])
def test_a_layer_of_all_three(saved):
    """Rotate, attend differentially, keep in 8 bits or not, and take the gradients back through the rotation."""
    B, S, H, D = 2, 300, 3, 128
    x = on_gpu(draw(B, S, S, H, D, "prefix", seed=14))
    plan = uaa.RotaryPlan([32, 16, 16], layout="interleaved")
    pos = torch.randint(0, 60, (B, S, 3), device=DEV, dtype=torch.int32)
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "lam")]
    rq, rk = uaa.rotary(leaves[0], leaves[1], plan, pos)
    out, _ = uaa.diff_attention(rq, rk, leaves[2], leaves[3], x["mask"], saved=saved)
    dq, dk, dv, dlam = torch.autograd.grad(out, leaves, x["do"])
    rot = uaa.rotary_fwd(x["q"].detach(), x["k"].detach(), plan, pos)
    o, o2, lse = uaa.diff_attn_fwd(*rot, x["v"].detach(), x["lam"].detach(), x["mask"])
    kept = [*rot, x["v"].detach(), o, o2]
    if saved:
        kept = uaa.act8_unpack(uaa.act8_pack(kept))
    g = uaa.diff_attn_bwd(*kept[:3], x["lam"].detach(), *kept[3:], x["do"], lse, x["mask"])
    wq, wk = uaa.rotary_bwd(g[0], g[1], plan, pos)
    for a, w in zip((out, dq, dk, dv, dlam), (o, wq, wk, g[2], g[3])):
        assert np.array_equal(bits(a), bits(w))
    uaa.check_device_status()


@pytest.mark.gpu
def test_captured_step_and_two_streams():
    xs = [on_gpu(draw(1, 300, 310, 2, 64, "prefix", seed=s)) for s in (20, 21)]
    want = [step(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    res = []
    for st, x in zip(streams, xs):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            out, out2, lse = uaa.diff_attn_fwd(x["q"], x["k"], x["v"], x["lam"], x["mask"])
            res.append((out,) + uaa.diff_attn_bwd(x["q"], x["k"], x["v"], x["lam"], out, out2, x["do"], lse, x["mask"]))
    torch.cuda.synchronize()
    for r, w in zip(res, want):
        for a, n in zip(r, ("out", "dq", "dk", "dv", "dlam")):
            assert np.array_equal(bits(a), bits(w[n])), n
    x = xs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, out2, lse = uaa.diff_attn_fwd(x["q"], x["k"], x["v"], x["lam"], x["mask"])
        grads = uaa.diff_attn_bwd(x["q"], x["k"], x["v"], x["lam"], out, out2, x["do"], lse, x["mask"])
    for n in ("q", "k", "v", "do"):
        x[n].normal_()
    graph.replay()
    torch.cuda.synchronize()
    again = step(x)
    for a, n in zip((out,) + grads, ("out", "dq", "dk", "dv", "dlam")):
        assert np.array_equal(bits(a), bits(again[n])), n


@pytest.mark.gpu
@pytest.mark.parametrize("Sq", [1, 2, 5])
def test_captured_decoding(Sq):
    """A captured call on a cache whose length, the mask's, grows between replays, on another stream."""
    x = on_gpu(draw(2, Sq, 900, 4, 128, "prefix", seed=22))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    uaa.diff_attn_fwd(x["q"], x["k"], x["v"], x["lam"], x["mask"], need_out2=False)
    with torch.cuda.graph(graph, stream=stream):
        out, _, lse = uaa.diff_attn_fwd(x["q"], x["k"], x["v"], x["lam"], x["mask"], need_out2=False)
    for n in (0, 1, 500, 899, 900):
        x["mask"][0] = torch.arange(900, device=DEV) < n
        x["q"].normal_()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.current_stream().wait_stream(stream)
        want = uaa.diff_attn_fwd(x["q"], x["k"], x["v"], x["lam"], x["mask"], need_out2=False)
        assert np.array_equal(bits(out), bits(want[0])) and np.array_equal(bits(lse), bits(want[2]))
        if n == 0:
            assert not out[0].any() and torch.isneginf(lse[0]).all()
    uaa.check_device_status()


@pytest.mark.gpu
def test_from_threads_that_made_no_cuda_call():
    """The library binds the device's context itself; two threads at once, each on its own stream."""
    xs = [on_gpu(draw(1, 150, 160, 2, 64, None, seed=s)) for s in (30, 31)]
    want = [step(x) for x in xs]
    got, streams = [None, None], [torch.cuda.Stream() for _ in xs]
    bufs = [{n: torch.empty_like(t) for n, t in w.items()} for w in want]  # so that the threads allocate nothing
    ws = [torch.empty(uaa.diff_attn_bwd_workspace_bytes(1, 150, 160, 2, 64), dtype=torch.uint8, device=DEV) for _ in xs]
    torch.cuda.synchronize()

    def work(i):
        x, b = xs[i], bufs[i]
        with torch.cuda.stream(streams[i]):
            out, out2, lse = uaa.diff_attn_fwd(x["q"], x["k"], x["v"], x["lam"], out=b["out"], out2=b["out2"],
                                               lse=b["lse"])
            uaa.diff_attn_bwd(x["q"], x["k"], x["v"], x["lam"], out, out2, x["do"], lse, dq=b["dq"], dk=b["dk"],
                              dv=b["dv"], dlam=b["dlam"], workspace=ws[i])
        got[i] = b

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert g is not None and all(np.array_equal(bits(g[n]), bits(w[n])) for n in w)


@pytest.mark.gpu
def test_empty_sizes_and_outputs_of_the_caller():
    lam = torch.full((2,), 0.5, device=DEV)
    new = lambda B, S: torch.zeros(B, S, 2, 64, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    for B, Sq, Sk in ((0, 3, 4), (2, 0, 4), (2, 0, 0)):
        q, k = new(B, Sq), new(B, Sk)
        out, out2, lse = uaa.diff_attn_fwd(q, k, k, lam)
        assert out.shape == q.shape and lse.shape == (B, 2, 2, Sq)
        if Sk and B:
            with pytest.raises(ValueError):
                uaa.diff_attn_bwd(q, k, k, lam, out, out2, q, lse)
        else:
            assert not uaa.diff_attn_bwd(q, k, k, lam, out, out2, q, lse)[3].any()
    with pytest.raises(uaa.UAAError, match="keys"):
        uaa.diff_attn_fwd(new(1, 3), new(1, 0), new(1, 0), lam)
    x = on_gpu(draw(1, 140, 140, 2, 64, None, seed=15))
    out = torch.empty_like(x["q"])
    assert uaa.diff_attn_fwd(x["q"], x["k"], x["v"], x["lam"], out=out)[0] is out
    with pytest.raises(ValueError):
        uaa.diff_attn_fwd(x["q"], x["k"], x["v"], x["lam"], out=out[:, 1:])


@pytest.mark.gpu
@pytest.mark.parametrize("D,mask", [(128, None), (64, "prefix"), (64, None), (128, "prefix")])
@pytest.mark.parametrize("n", [0, 1, 2, 5])
def test_a_load_that_never_comes(D, mask, n):
    """The n-th ring load of every CTA is not issued: the waits for it run out, every role meets the others to the end of
    its schedule, the status says so, and the next call, issued before it was read, is right."""
    x = on_gpu(draw(1, 300, 700, 2, D, mask, seed=40))
    want = step(x)
    uaa.set_wait_timeout_ms(20)
    uaa.debug_drop_load(n)
    try:
        uaa.diff_attn_fwd(x["q"], x["k"], x["v"], x["lam"], x["mask"])
        uaa.diff_attn_bwd(x["q"], x["k"], x["v"], x["lam"], want["out"], want["out2"], x["do"], want["lse"], x["mask"])
    finally:
        uaa.debug_drop_load(-1)
        uaa.set_wait_timeout_ms(0)
    out, out2, lse = uaa.diff_attn_fwd(x["q"], x["k"], x["v"], x["lam"], x["mask"])
    grads = uaa.diff_attn_bwd(x["q"], x["k"], x["v"], x["lam"], out, out2, x["do"], lse, x["mask"])
    torch.cuda.synchronize()
    with pytest.raises(uaa.UAAError) as e:
        uaa.check_device_status()
    assert e.value.status == -5
    uaa.check_device_status()
    for a, name in zip((out, out2, lse) + grads, ("out", "out2", "lse", "dq", "dk", "dv", "dlam")):
        assert np.array_equal(bits(a), bits(want[name])), name
