"""Attention over packed sequences against the float64 definition, within the error that the operands' roundings allow."""
import ctypes
import itertools
import weakref

import numpy as np
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from oracle import seqs as ref
from helpers import f64

DEV = "cuda"


# --------------------------------------------------------------------------- the definition itself
@pytest.mark.parametrize("causal", [True, False])
def test_definition_against_differences(causal):
    rng = np.random.default_rng(1)
    q, k, v, g = (rng.standard_normal((n, h, 8)) for n, h in ((5, 4), (7, 2), (7, 2), (5, 4)))
    starts, starts_k = [0, 3, 3, 5], [0, 2, 3, 7]
    res = ref.packed(q, k, v, starts, starts_k, causal, 0.6, g)

    def loss(q, k, v):
        return (ref.packed(q, k, v, starts, starts_k, causal, 0.6)["out"][0] * g).sum()

    args, h = [q, k, v], 1e-5
    for n, name in enumerate(("dq", "dk", "dv")):
        for at in list(np.ndindex(args[n].shape))[::3]:
            up, down = ([a.copy() for a in args] for _ in range(2))
            up[n][at] += h
            down[n][at] -= h
            assert abs((loss(*up) - loss(*down)) / (2 * h) - res[name][0][at]) < 1e-8, (name, at)


def test_definition_special_cases():
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((4, 1, 8)) for _ in range(3))
    one = ref.attention(q, k, v, True)
    assert np.allclose(one["out"][0][0], v[0])  # the first query reads the first key
    few = ref.attention(q, k[:2], v[:2], True, dout=q)  # more queries than keys: the first two read none
    assert not few["out"][0][:2].any() and (few["lse"][0][0, :2] == -np.inf).all() and not few["dq"][0][:2].any()
    assert np.allclose(few["out"][0][2], v[0])


# --------------------------------------------------------------------------- refusals
def args(**kw):
    f = 1 << 20
    x = dict(q=f, k=f, v=f, out=f, lse=f, starts=f, starts_k=0, table=0, lens=0, seqs=0, q_row=256, q_head=64, k_row=128,
             k_head=64, v_row=128, v_head=64, k_page=0, v_page=0, B=2, T=10, Tk=10, Hq=4, Hk=2, D=64, dtype=0, causal=1,
             pages=0, page=0, table_rows=0, width=0, rest=0, scale=0.1)
    x.update(kw)
    return uaa._SEQS.pack(*x.values())


def test_refusals_of_the_call():
    L, P = uaa.lib(), ctypes.c_void_p
    err = lambda: L.uaa_last_error().decode()  # noqa: E731
    ws, big = P(1 << 24), 1 << 40

    def fwd(ws=ws, n=big, **kw):
        return L.uaa_attn_packed_fwd(args(**kw), ws, n, None)

    assert L.uaa_attn_packed_fwd(None, ws, big, None) == -1 and "NULL" in err()
    assert fwd(D=96) == -2 and "D=96" in err()
    assert fwd(dtype=2) == -2 and "dtype" in err()
    assert fwd(Hq=5) == -1 and "query heads" in err()
    assert fwd(Hk=0) == -1 and "query heads" in err()
    assert fwd(Hq=258) == -2 and "128 at most" in err()
    assert fwd(B=-1) == -1 and "negative" in err()
    assert fwd(B=65536) == -2 and "65535" in err()
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert fwd(scale=scale) == -1 and "scale" in err()
    for name in ("q", "k", "v", "out"):
        assert fwd(**{name: 0}) == -1 and f"{name} is NULL" in err()
        assert fwd(**{name: (1 << 20) + 8}) == -1 and "aligned" in err()
    assert fwd(lse=0) == -1 and "lse" in err()
    assert fwd(lse=(1 << 20) + 2) == -1 and "lse" in err()
    assert fwd(starts=0) == -1 and "starts" in err()
    assert fwd(starts_k=6) == -1 and "starts" in err()
    for name in ("q_row", "q_head", "k_row", "k_head", "v_row", "v_head"):
        for x in (0, -64, 12, 1 << 40):
            assert fwd(**{name: x}) == -1 and "stride" in err()
    assert fwd(n=16) == -1 and "workspace" in err()
    assert fwd(ws=P((1 << 24) + 16)) == -1 and "256-byte" in err()
    assert fwd(ws=None) == -1 and "workspace" in err()
    assert fwd(q=0, T=0) == 0 and fwd(q=0, B=0) == 0

    def bwd(ws=ws, n=big, dout=P(1 << 20), dq=P(1 << 20), dk=P(1 << 20), dv=P(1 << 20), **kw):
        return L.uaa_attn_packed_bwd(args(**kw), dout, dq, dk, dv, ws, n, None)

    assert bwd(dtype=1) == -2 and "bf16" in err()
    assert bwd(dout=None) == -1 and "dout" in err()
    assert bwd(dq=P(8)) == -1 and "dq" in err()
    assert bwd(dk=None) == -1 and "dk" in err()
    assert bwd(dv=None) == -1 and "dv" in err()
    assert bwd(n=16) == -1 and "workspace" in err()
    assert bwd(ws=P((1 << 24) + 16)) == -1 and "256-byte" in err()
    assert bwd(B=0, q=0) == 0 and bwd(T=0, Tk=0, q=0) == 0
    assert uaa.attn_packed_bwd_workspace_bytes(-1, 4, 4, 2, 64) == 0 and uaa.attn_packed_bwd_workspace_bytes(1, 4, 4, 2, 96) == 0
    assert uaa.attn_seqs_workspace_bytes(1, -1, 4, 2, 64) == 0


def test_the_workspace_outlives_the_launch(monkeypatch):
    """Freed before the launch, another thread's tensor could take its place on the same stream."""
    made, seen, empty = [], [], torch.empty

    def make(*a, **kw):
        t = empty(*a, **kw)
        made.append((weakref.ref(t), t.data_ptr()))
        return t

    def call(dev, name, *a):
        live = [r() for r, _ in made]
        assert all(t is not None for t in live), name
        seen.append(name)
        assert any(t.data_ptr() in a for t in live), name

    q, kv = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    starts, lens = torch.tensor([0, 5], dtype=torch.int32), torch.tensor([5], dtype=torch.int32)
    pool = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    monkeypatch.setattr(uaa, "_same_device", lambda *ts: ts[0].device)
    monkeypatch.setattr(uaa, "_call", call)
    monkeypatch.setattr(torch, "empty", make)
    out, lse = uaa.attn_packed_fwd(q, kv, kv, starts)
    made.clear()
    uaa.attn_packed_bwd(q, kv, kv, out, q, lse, starts)
    made.clear()
    uaa.attn_paged_fwd(q, pool, pool, starts, torch.zeros(1, 2, dtype=torch.int32), lens)
    assert seen == ["uaa_attn_packed_fwd", "uaa_attn_packed_bwd", "uaa_attn_paged_fwd"]


@pytest.mark.parametrize("kw", [dict(T=2 ** 30 + 1, Hq=1, Hk=1), dict(Tk=2 ** 30 + 1, Hq=1, Hk=1)])
def test_refusal_of_too_many_tokens(kw):
    L, P = uaa.lib(), ctypes.c_void_p
    assert L.uaa_attn_packed_fwd(args(**kw), P(1 << 24), 1 << 40, None) == -2
    assert "2^30 tokens" in L.uaa_last_error().decode()
    f = P(1 << 20)
    assert L.uaa_attn_packed_bwd(args(**kw), f, f, f, f, P(1 << 24), 1 << 40, None) == -2
    assert "2^30 tokens" in L.uaa_last_error().decode()


def test_refusals_of_the_binding():
    x = torch.zeros(10, 4, 64, dtype=torch.bfloat16)
    kv = torch.zeros(10, 2, 64, dtype=torch.bfloat16)
    starts = torch.tensor([0, 10], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        uaa.attn_packed_fwd(x, kv, kv, starts)
    with pytest.raises(ValueError, match="dimensions"):
        uaa._packed_args(x[0], kv, kv, starts, None, True, None, None, None)
    with pytest.raises(ValueError, match="columns"):
        uaa._packed_args(x, torch.zeros(10, 2, 128, dtype=torch.bfloat16), kv, starts, None, True, None, None, None)
    with pytest.raises(ValueError, match="contiguous"):
        uaa._packed_args(x.transpose(1, 2), kv, kv, starts, None, True, None, None, None)
    with pytest.raises(ValueError, match="one shape"):
        uaa._packed_args(x, kv, kv[:5], starts, None, True, None, None, None)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        uaa._packed_args(x.float(), kv, kv, starts, None, True, None, None, None)
    with pytest.raises(TypeError, match="one type"):
        uaa._packed_args(x, kv.half(), kv, starts, None, True, None, None, None)
    with pytest.raises(TypeError, match="gradients"):
        uaa._packed_args(x.half(), kv.half(), kv.half(), starts, None, True, None, None, None, half=False)
    with pytest.raises(ValueError, match="starts"):
        uaa._packed_args(x, kv, kv, starts.long(), None, True, None, None, None)
    with pytest.raises(ValueError, match="one entry more"):
        uaa._packed_args(x, kv, kv, starts, starts[:1], True, None, None, None)
    with pytest.raises(ValueError, match="starts_k"):
        uaa._packed_args(x, kv[:5], kv[:5], starts, None, True, None, None, None)
    with pytest.raises(ValueError, match="out must"):
        uaa._packed_args(x, kv, kv, starts, None, True, None, x[:5], None)
    with pytest.raises(ValueError, match="saved"):
        uaa.packed_attention(x, kv, kv, starts, saved="int4")
    with pytest.raises(TypeError, match="gradients"):
        uaa.packed_attention(x.half().requires_grad_(), kv.half(), kv.half(), starts)


# --------------------------------------------------------------------------- on the GPU
def draw(lens, lens_k, Hq, Hk, D, dtype=torch.bfloat16, seed=0, tail=0):
    g = torch.Generator().manual_seed(1000 + seed)
    T, Tk = sum(lens) + tail, sum(lens_k) + tail
    x = {"q": torch.randn(T, Hq, D, generator=g), "k": torch.randn(Tk, Hk, D, generator=g),
         "v": torch.randn(Tk, Hk, D, generator=g), "do": torch.randn(T, Hq, D, generator=g)}
    x = {n: t.to(dtype) for n, t in x.items()}
    x["starts"], x["starts_k"] = (torch.tensor(list(itertools.accumulate(ls, initial=0)), dtype=torch.int32)
                                  for ls in (lens, lens_k))
    return x


def check(got, want, names, what=""):
    for n in names:
        value, bound = want[n]
        x = got[n].detach().cpu().double().numpy()
        own = np.isfinite(bound)
        gone = np.isinf(value) & own
        assert np.array_equal(x[gone], value[gone]), (n, what)
        own &= ~gone
        off = np.abs(x[own] - value[own]) - bound[own]
        assert (off <= 0).all(), (n, what, off.max(), int((~(off <= 0)).sum()))


def step(x, causal=True, scale=None, grads=True, **kw):
    y = {n: t.to(DEV) for n, t in x.items()}
    same = x["starts"].equal(x["starts_k"]) and x["q"].shape[0] == x["k"].shape[0]
    sk = None if same else y["starts_k"]
    out, lse = uaa.attn_packed_fwd(y["q"], y["k"], y["v"], y["starts"], sk, causal, scale, **kw)
    got = {"out": out, "lse": lse}
    if grads:
        got["dq"], got["dk"], got["dv"] = uaa.attn_packed_bwd(y["q"], y["k"], y["v"], out, y["do"], lse, y["starts"], sk,
                                                              causal, scale)
    uaa.check_device_status()
    return got


def against(x, causal=True, scale=None, grads=True):
    y = {n: f64(x[n]) for n in ("q", "k", "v", "do")}
    dtype = str(x["q"].dtype).split(".")[1]
    return ref.packed(y["q"], y["k"], y["v"], x["starts"].tolist(), x["starts_k"].tolist(), causal, scale,
                      y["do"] if grads else None, dtype)


ALL = ("out", "lse", "dq", "dk", "dv")
LENS = [[1], [2], [127], [128], [129], [255, 1], [257], [0, 5, 0, 0, 130, 1, 0], [300, 40, 1, 129], [700], [64, 64, 64, 64]]


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(lens, D, causal):
    x = draw(lens, lens, 4, 2, D, seed=sum(lens))
    check(step(x, causal), against(x, causal), ALL)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (3, 1), (5, 1), (14, 2), (6, 1), (16, 2), (24, 1), (48, 1), (65, 1), (128, 1)])
def test_heads(Hq, Hk, causal):
    lens = [70, 3, 150]
    x = draw(lens, lens, Hq, Hk, 64, seed=Hq)
    check(step(x, causal), against(x, causal), ALL)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,lens_k", [([1, 1, 1], [1, 300, 129]), ([130, 5], [77, 400]), ([200, 3], [1, 1]), ([4, 0, 7], [0, 9, 0]),
                                         ([0, 0], [5, 200]), ([33, 260], [1000, 256])], ids=str)
def test_other_keys_than_queries(lens, lens_k, D, causal):
    x = draw(lens, lens_k, 6, 2, D, seed=sum(lens_k))
    check(step(x, causal), against(x, causal), ALL)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[1], [129, 31], [600, 1, 50]], ids=str)
def test_fp16(lens, D):
    x = draw(lens, lens, 5, 1, D, torch.float16, seed=7)
    check(step(x, grads=False), against(x, grads=False), ("out", "lse"))


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.02, 0.5, 2.0])
def test_scales(scale):
    x = draw([260, 3], [260, 3], 4, 2, 64, seed=9)
    check(step(x, True, scale), against(x, True, scale), ALL)


@pytest.mark.gpu
def test_slices_of_a_packed_projection():
    lens, Hq, Hk, D = [130, 61], 4, 2, 64
    x = draw(lens, lens, Hq, Hk, D, seed=11)
    want = step(x)
    T = sum(lens)
    qkv = torch.cat([x[n].reshape(T, -1) for n in ("q", "k", "v")], 1).to(DEV)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hk * D, Hk * D], 1))
    s = x["starts"].to(DEV)
    out, lse = uaa.attn_packed_fwd(q, k, v, s)
    grads = uaa.attn_packed_bwd(q, k, v, out, x["do"].to(DEV), lse, s)
    for a, n in zip((out, lse) + grads, ALL):
        assert torch.equal(a, want[n]), n
    # heads first: (H, T, D) seen as (T, H, D)
    q, k, v = (x[n].to(DEV).transpose(0, 1).contiguous().transpose(0, 1) for n in ("q", "k", "v"))
    assert torch.equal(uaa.attn_packed_fwd(q, k, v, s)[0], want["out"])


@pytest.mark.gpu
def test_tokens_of_no_sequence():
    """Behind the last sequence: whatever the inputs hold there, results before it do not see it, and what the results
    held there stays."""
    lens = [100, 37]
    x = draw(lens, lens, 4, 2, 64, seed=12, tail=60)
    got = step(x)
    check(got, against(x), ALL)
    T = sum(lens)
    for n in ("q", "k", "v", "do"):
        x[n][T:] = float("nan")
    y = {n: t.to(DEV) for n, t in x.items()}
    keep = {n: torch.full(y[m].shape, 7.0, dtype=torch.bfloat16, device=DEV) for n, m in (("out", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v"))}
    lse = torch.full((4, T + 60), 7.0, device=DEV)
    uaa.attn_packed_fwd(y["q"], y["k"], y["v"], y["starts"], out=keep["out"], lse=lse)
    uaa.attn_packed_bwd(y["q"], y["k"], y["v"], keep["out"], y["do"], lse, y["starts"], dq=keep["dq"], dk=keep["dk"], dv=keep["dv"])
    uaa.check_device_status()
    for n, t in keep.items():
        assert (t[T:] == 7).all() and torch.equal(t[:T], got[n][:T]), n
    assert (lse[:, T:] == 7).all() and torch.equal(lse[:, :T], got["lse"][:, :T])


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e4])
@pytest.mark.parametrize("D", [64, 128])
def test_other_sequences_leave_no_trace(value, D):
    lens = [130, 60, 140]
    x = draw(lens, lens, 4, 2, D, seed=13)
    clean = step(x)
    y = {n: t.clone() for n, t in x.items()}
    for n in ("q", "k", "v", "do"):
        y[n][130:190] = value
    got = step(y)
    for n in ALL:
        a, b = got[n], clean[n]
        if n == "lse":
            a, b = a.T, b.T
        assert torch.equal(a[:130], b[:130]) and torch.equal(a[190:], b[190:]), n


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("Hq,Hk", [(2, 2), (8, 1), (3, 1)])
@pytest.mark.parametrize("at", [0, 5, 128, 200, 299])
def test_later_keys_leave_no_trace(value, Hq, Hk, at):
    """A value that is not finite at token `at`: queries before it do not see it, the others show it."""
    x = draw([300], [300], Hq, Hk, 64, seed=14)
    clean = step(x, grads=False)
    y = {n: t.clone() for n, t in x.items()}
    y["k"][at, 0, 3] = float("nan")
    got = step(y, grads=False)
    assert torch.equal(got["out"][:at], clean["out"][:at]) and torch.equal(got["lse"][:, :at], clean["lse"][:, :at])
    g = Hq // Hk
    assert torch.isnan(got["out"][at:, :g]).all() and torch.isnan(got["lse"][:g, at:]).all()
    assert torch.equal(got["out"][:, g:], clean["out"][:, g:])
    y = {n: t.clone() for n, t in x.items()}
    y["v"][at, 0, 3] = value
    got = step(y, grads=False)
    assert torch.equal(got["out"][:at], clean["out"][:at]) and torch.equal(got["lse"], clean["lse"])
    seen = got["out"][at:, :g, 3].float()
    assert (torch.isnan(seen) if value != value else seen == value).all()
    for c in (slice(0, 3), slice(4, None)):
        assert torch.equal(got["out"][..., c], clean["out"][..., c])


@pytest.mark.gpu
def test_scores_that_are_infinite():
    """A score of -inf is no weight; a row with one of +inf has lse = +inf and NaN."""
    x = draw([200], [200], 2, 1, 64, seed=15)
    x["q"][..., 0] = 1.0
    y = {n: t.clone() for n, t in x.items()}
    y["k"][:, :, 0] = torch.where(torch.arange(200)[:, None] % 2 == 0, float("-inf"), 0.0)
    got = step(y, grads=False)
    assert torch.isneginf(got["lse"][:, 0]).all() and not got["out"][0].any()
    q, k, v = (f64(x[n]) for n in ("q", "k", "v"))
    k[:, :, 0] = 0.0
    for i in (1, 2, 77, 199):  # the last query of its keys: the odd ones up to i
        want = ref.attention(q[i: i + 1], k[1: i + 1: 2], v[1: i + 1: 2], True)
        check({"out": got["out"][i: i + 1], "lse": got["lse"][:, i: i + 1]}, want, ("out", "lse"), i)
    y["k"][50, 0, 0] = float("inf")
    got = step(y, grads=False)
    assert torch.isposinf(got["lse"][:, 50:]).all() and torch.isnan(got["out"][50:]).all()
    assert torch.isfinite(got["lse"][:, 1:50]).all() and torch.isfinite(got["out"][:50]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("saved", [None, "int8"])
def test_autograd(saved):
    lens = [90, 1, 140]
    x = draw(lens, lens, 6, 2, 128, seed=16)
    y = {n: t.to(DEV) for n, t in x.items()}
    q, k, v = (y[n].requires_grad_() for n in ("q", "k", "v"))
    out, lse = uaa.packed_attention(q, k, v, y["starts"], saved=saved)
    assert not lse.requires_grad
    grads = torch.autograd.grad(out, (q, k, v), y["do"])
    want = step(x)
    assert torch.equal(out, want["out"]) and torch.equal(lse, want["lse"])
    if saved is None:
        for a, n in zip(grads, ("dq", "dk", "dv")):
            assert torch.equal(a, want[n]), n
    else:
        kept = [uaa.act8_unpack(uaa.act8_pack(y[n].detach())) for n in ("q", "k", "v")] + [uaa.act8_unpack(uaa.act8_pack(out.detach()))]
        for a, b in zip(grads, uaa.attn_packed_bwd(*kept, y["do"], lse, y["starts"])):
            assert torch.equal(a, b)
    # an expanded gradient, and results without one
    out, _ = uaa.packed_attention(q, k, v, y["starts"])
    out.sum().backward()
    assert torch.isfinite(q.grad.float()).all()
    with torch.no_grad():
        assert torch.equal(uaa.packed_attention(q, k, v, y["starts"])[0], want["out"])
    starts = y["starts"].clone()
    out, _ = uaa.packed_attention(q, k, v, starts)
    starts += 1
    with pytest.raises(RuntimeError, match="modified"):
        out.sum().backward()


@pytest.mark.gpu
@pytest.mark.parametrize("first,last", [(0, 50), (7, 50), (20, 64), (64, 64), (0, 0)])
def test_tokens_of_no_sequence_have_no_gradient(first, last):
    """Before the first sequence and behind the last one: zeros, where raw calls leave what was there."""
    x = draw([64], [64], 2, 1, 64, seed=17)
    x["starts"] = x["starts_k"] = torch.tensor([first, last], dtype=torch.int32)
    y = {n: t.to(DEV) for n, t in x.items()}
    for n in ("q", "k", "v", "do"):
        y[n][:first] = y[n][last:] = float("nan")
    q, k, v = (y[n].requires_grad_() for n in ("q", "k", "v"))
    for _ in range(2):  # the second time over memory that is not fresh
        out, lse = uaa.packed_attention(q, k, v, y["starts"])
        grads = torch.autograd.grad(out, (q, k, v), y["do"])
        got = dict(zip(ALL, (out, lse) + grads))
        want = against(x)
        check(got, want, ALL)
        for n, t in got.items():
            t = t.T if n == "lse" else t
            for rest in (t[:first], t[last:]):
                assert torch.isneginf(rest).all() if n == "lse" else not rest.any(), n
        del out, lse, grads, got, t
        torch.full((1 << 22,), float("nan"), device=DEV)
    uaa.check_device_status()


@pytest.mark.gpu
def test_same_bits_every_time_and_as_each_sequence_alone():
    lens = [1, 400, 130, 700, 2]
    x = draw(lens, lens, 10, 2, 64, seed=18)
    first = step(x)
    for _ in range(5):
        for n, t in step(x).items():
            assert torch.equal(t, first[n]), n


@pytest.mark.gpu
def test_captured():
    """A captured step, replayed with other lengths and other values."""
    x = draw([200, 56], [200, 56], 4, 2, 64, seed=19)
    y = {n: t.to(DEV) for n, t in x.items()}

    def go():
        out, lse = uaa.attn_packed_fwd(y["q"], y["k"], y["v"], y["starts"])
        return (out, lse) + uaa.attn_packed_bwd(y["q"], y["k"], y["v"], out, y["do"], lse, y["starts"])

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        go()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = go()
    for lens, seed in (([200, 56], 19), ([3, 253], 20), ([255, 1], 21)):
        z = draw(lens, lens, 4, 2, 64, seed=seed)
        for n in y:
            y[n].copy_(z[n])
        graph.replay()
        torch.cuda.synchronize()
        check(dict(zip(ALL, res)), against(z), ALL, lens)


@pytest.mark.gpu
def test_another_stream_and_thread():
    import threading

    x = draw([150, 20], [150, 20], 4, 2, 64, seed=22)
    want, got = step(x), {}

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            got.update(step(x))
            torch.cuda.current_stream().synchronize()

    t = threading.Thread(target=work)
    t.start()
    t.join()
    for n in ALL:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.gpu
def test_starts_that_are_wrong_stay_inside():
    """starts that decrease, or lie outside the tensors: nothing outside is touched; nothing hangs."""
    from test_gpu_guard_bands import Guarded

    x = draw([300], [300], 4, 2, 64, seed=23)
    y = {n: t.to(DEV) for n, t in x.items()}
    for s in ([0, 200, 100, 300], [-5, 50, 400, 10 ** 9], [300, 0, -(2 ** 31), 2 ** 31 - 1], [0, 0, 0, 0], [290, 295, 305, 310]):
        st = torch.tensor(s, dtype=torch.int32, device=DEV)
        g = Guarded()
        out, dq = (g.empty(y["q"].shape, torch.bfloat16) for _ in range(2))
        dk, dv = (g.empty(y["k"].shape, torch.bfloat16) for _ in range(2))
        lse = g.empty((4, 300), torch.float32)
        ws = g.empty((uaa.attn_packed_bwd_workspace_bytes(3, 300, 4, 2, 64),), torch.uint8)
        ws2 = g.empty((uaa.attn_seqs_workspace_bytes(3, 300, 4, 2, 64),), torch.uint8)
        for t in (out, dq, dk, dv, lse):
            t.zero_()
        uaa.attn_packed_fwd(y["q"], y["k"], y["v"], st, out=out, lse=lse, workspace=ws2)
        uaa.attn_packed_bwd(y["q"], y["k"], y["v"], out, y["do"], lse, st, dq=dq, dk=dk, dv=dv, workspace=ws)
        uaa.check_device_status()
        g.check()


@pytest.mark.gpu
@pytest.mark.parametrize("T,D", [(1, 64), (70, 128)])
def test_no_sequence_at_all(T, D):
    """No sequence: every token belongs to none, on memory that is not fresh."""
    q, k, v = (torch.randn(T, h, D, device=DEV, dtype=torch.bfloat16).requires_grad_() for h in (4, 2, 2))
    starts = torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(2):
        keep = [torch.full_like(t, float("nan")) for t in (q, q, k, v)] + [torch.full((4, T), float("nan"), device=DEV)]
        torch.cuda.synchronize()
        del keep
        out, lse = uaa.packed_attention(q, k, v, starts)
        grads = torch.autograd.grad(out, (q, k, v), torch.ones_like(out))
        assert torch.isneginf(lse).all() and not any(t.any() for t in (out,) + grads)
    uaa.check_device_status()
