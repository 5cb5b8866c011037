"""Attention of new tokens over the pages of a cache against the float64 definition."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from oracle import seqs as ref
from helpers import f64
from test_packed_attention import args, check

DEV = "cuda"


def test_refusals_of_the_call():
    L, P, f = uaa.lib(), ctypes.c_void_p, 1 << 20
    err = lambda: L.uaa_last_error().decode()  # noqa: E731

    def fwd(ws=P(1 << 24), n=1 << 40, **kw):
        return L.uaa_attn_paged_fwd(args(**{**dict(table=f, lens=f, k_page=2048, v_page=2048, pages=9, page=16, table_rows=2, width=4), **kw}),
                                    ws, n, None)

    for page in (0, -16, 8, 48, 96, 100, 200, 1 << 20):
        assert fwd(page=page) == -2 and "pages of" in err()
    for name in ("table", "lens"):
        assert fwd(**{name: 0}) == -1 and "table" in err()
        assert fwd(**{name: f + 2}) == -1 and "aligned" in err()
    assert fwd(seqs=f + 1) == -1 and "aligned" in err()
    for name in ("pages", "width", "table_rows"):
        assert fwd(**{name: -1}) == -1 and "negative" in err()
    assert fwd(B=3) == -1 and "table of 2 rows" in err()
    assert fwd(k_page=0) == -1 and "stride" in err()
    assert fwd(v_page=12) == -1 and "stride" in err()
    assert fwd(k=0) == -1 and "k is NULL" in err()
    assert fwd(n=16) == -1 and "workspace" in err()
    assert fwd(D=80) == -2 and fwd(Hq=3) == -1 and fwd(scale=0.0) == -1
    assert fwd(T=0, q=0) == 0 and fwd(B=0, q=0) == 0

    rows = dict(k=f, v=f, kp=f, vp=f, starts=f, seqs=0, table=f, lens=f, k0=128, k1=64, v0=128, v1=64, a0=2048, a1=128, a2=64,
                b0=2048, b1=128, b2=64, B=2, T=5, Hk=2, D=64, pages=9, page=16, table_rows=2, width=4)

    def write(**kw):
        return L.uaa_cache_write(uaa._CACHE_ROWS.pack(*{**rows, **kw}.values()), None)

    assert L.uaa_cache_write(None, None) == -1
    for name in ("k", "v", "kp", "vp"):
        assert write(**{name: 0}) == -1 and "NULL" in err()
        assert write(**{name: f + 8}) == -1 and "aligned" in err()
    for name in ("starts", "table", "lens"):
        assert write(**{name: 0}) == -1 and "NULL" in err()
    assert write(seqs=f + 2) == -1
    assert write(k0=-8) == -1 and "stride" in err()
    assert write(b2=4) == -1 and "stride" in err()
    assert write(D=12) == -2 and write(page=0) == -1 and write(B=3) == -1 and write(T=-1) == -1
    assert write(T=0, k=0) == 0 and write(B=0, k=0) == 0


def test_refusal_of_too_many_tokens():
    L, P, f = uaa.lib(), ctypes.c_void_p, 1 << 20
    x = dict(table=f, lens=f, k_page=2048, v_page=2048, pages=9, page=1024, table_rows=2, width=2 ** 20 + 1)
    assert L.uaa_attn_paged_fwd(args(**x), P(1 << 24), 1 << 40, None) == -2
    assert "2^30 tokens" in L.uaa_last_error().decode()


def test_refusals_of_the_binding():
    q, kv = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16)
    starts, lens = torch.tensor([0, 3], dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        uaa.attn_paged_fwd(q, kv, kv, starts, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        uaa.cache_write(q, q, kv, kv, starts, table, lens)
    for bad in (table.long(), table[0], table.T):
        with pytest.raises(ValueError, match="table"):
            uaa._table(bad, lens, None, 1)
    for bad in (lens.long(), lens[:1]):
        with pytest.raises(ValueError, match="lens"):
            uaa._table(table, bad, None, 1)
    for bad in (starts, starts.long()[:1]):
        with pytest.raises(ValueError, match="seqs"):
            uaa._table(table, lens, bad, 1)


# --------------------------------------------------------------------------- on the GPU
def draw(news, lens, Hq, Hk, D, page, dtype=torch.bfloat16, seed=0, spare=3, width=0):
    """A cache of shuffled pages that holds sequences of `lens` tokens, the last `news` of them new."""
    g = torch.Generator().manual_seed(2000 + seed)
    need = [-(-n // page) for n in lens]
    N, width = sum(need) + spare, max(need + [1]) + width
    order = torch.randperm(N, generator=g).tolist()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    x = {"q": torch.randn(sum(news), Hq, D, generator=g).to(dtype), "table": table,
         "k": torch.randn(N, page, Hk, D, generator=g).to(dtype), "v": torch.randn(N, page, Hk, D, generator=g).to(dtype),
         "lens": torch.tensor(lens, dtype=torch.int32),
         "starts": torch.tensor(list(itertools.accumulate(news, initial=0)), dtype=torch.int32)}
    return x


def step(x, seqs=None, causal=True, scale=None):
    y = {n: t.to(DEV) for n, t in x.items()}
    out, lse = uaa.attn_paged_fwd(y["q"], y["k"], y["v"], y["starts"], y["table"], y["lens"],
                                  None if seqs is None else torch.tensor(seqs, dtype=torch.int32, device=DEV), causal, scale)
    uaa.check_device_status()
    return {"out": out, "lse": lse}


def against(x, seqs=None, causal=True, scale=None):
    dtype = str(x["q"].dtype).split(".")[1]
    return ref.paged(f64(x["q"]), f64(x["k"]), f64(x["v"]), x["starts"].tolist(), x["table"].numpy(), x["lens"].tolist(), seqs,
                     causal, scale, dtype)


BOTH = ("out", "lse")


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("news,lens", [([1], [1]), ([1], [16]), ([1], [129]), ([1, 1, 1], [5, 700, 64]), ([3, 0, 40, 1], [3, 100, 300, 128]),
                                       ([130, 257], [131, 257]), ([1] * 9, [2000, 1, 17, 0, 31, 32, 33, 255, 640])], ids=str)
def test_lengths(news, lens, D, page):
    x = draw(news, lens, 4, 2, D, page, seed=sum(lens))
    check(step(x), against(x), BOTH)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (3, 1), (5, 1), (14, 2), (8, 1), (32, 2), (24, 1), (65, 1), (128, 1)])
@pytest.mark.parametrize("news", [[1, 1], [5, 2], [70, 1]])
def test_heads(Hq, Hk, news):
    x = draw(news, [700, 70], Hq, Hk, 64, 32, seed=Hq)
    check(step(x), against(x), BOTH)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[5000], [3001, 40], [12000, 7]], ids=str)
@pytest.mark.parametrize("g", [1, 5])
@pytest.mark.parametrize("new", [1, 4, 60])
def test_long_pasts(lens, g, new):
    """Few rows against many keys: the keys are split over the SMs."""
    news = [new] * len(lens)
    x = draw(news, lens, 2 * g, 2, 128, 64, seed=sum(lens) + g)
    check(step(x), against(x), BOTH)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("news,lens", [([1, 1], [300, 2500]), ([200], [900])], ids=str)
def test_fp16(news, lens, D):
    x = draw(news, lens, 10, 2, D, 16, torch.float16, seed=3)
    check(step(x), against(x), BOTH)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
def test_rows_of_the_table(causal):
    """Sequences in another order than the table's, one of them twice; without the causal border; a wider table."""
    seqs = [4, 0, 4, 2]
    x = draw([0] * 5, [300, 20, 129, 64, 500], 4, 2, 64, 32, seed=4, width=7)
    g = torch.Generator().manual_seed(5)
    news = [3, 2, 1, 60]
    x["q"] = torch.randn(sum(news), 4, 64, generator=g).bfloat16()
    x["starts"] = torch.tensor(list(itertools.accumulate(news, initial=0)), dtype=torch.int32)
    check(step(x, seqs, causal, 0.2), against(x, seqs, causal, 0.2), BOTH)


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e4])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("news", [[1, 1], [40, 7]])
def test_what_no_row_reads_leaves_no_trace(value, page, news):
    """Rows behind a sequence's end in its last page, pages of no sequence."""
    lens = [300, 45]
    x = draw(news, lens, 4, 2, 64, page, seed=6)
    clean = step(x)
    y = {n: t.clone() for n, t in x.items()}
    read = torch.zeros(x["k"].shape[:2], dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(n):
            read[x["table"][b, j // page], j % page] = True
    for n in ("k", "v"):
        y[n][~read] = value
    got = step(y)
    for n in BOTH:
        assert torch.equal(got[n], clean[n]), n


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 30])
def test_later_values_leave_no_trace(new):
    x = draw([new], [400], 8, 2, 64, 32, seed=7)
    clean = step(x)
    for at in (0, 100, 399):
        y = {n: t.clone() for n, t in x.items()}
        y["v"][x["table"][0, at // 32], at % 32, 0, 5] = float("inf")
        got = step(y)
        i = max(0, at - (400 - new))
        assert torch.equal(got["out"][:i], clean["out"][:i]) and torch.equal(got["lse"], clean["lse"])
        assert torch.isposinf(got["out"][i:, :4, 5]).all()
        assert torch.equal(got["out"][:, 4:], clean["out"][:, 4:])


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 50])
@pytest.mark.parametrize("page", [16, 128])
def test_bad_pages_are_skipped_and_reported(new, page):
    """Pages, table rows and lengths outside the cache: their keys have no weight, and the status says so."""
    lens = [1000, 300]
    x = draw([new, new], lens, 4, 2, 64, page, seed=8)
    y = {n: t.clone() for n, t in x.items()}
    bad = {0: -1, 2: x["k"].shape[0]} if page == 16 else {0: 2 ** 31 - 1, 2: -(2 ** 31)}
    for c, p in bad.items():
        y["table"][0, c] = p
    g = {n: t.to(DEV) for n, t in y.items()}
    out, lse = uaa.attn_paged_fwd(g["q"], g["k"], g["v"], g["starts"], g["table"], g["lens"])
    with pytest.raises(uaa.UAAError, match="UAA_ERR_BAD_PAGE"):
        uaa.check_device_status()
    want = against(x)
    keep = np.concatenate([np.arange(c * page, min((c + 1) * page, 1000)) for c in range(-(-1000 // page)) if c not in bad])
    kk, vv = (f64(x[n])[x["table"][0, : -(-1000 // page)].numpy()].reshape(-1, 2, 64)[keep] for n in ("k", "v"))
    one = ref.attention(f64(x["q"])[:new], kk, vv, True)
    for n in BOTH:
        for i in range(2):
            want[n][i][(slice(None), slice(0, new)) if n == "lse" else slice(0, new)] = one[n][i]
    check({"out": out, "lse": lse}, want, BOTH)
    # a table row and lengths outside
    seqs = torch.tensor([-1, 7], dtype=torch.int32, device=DEV)
    out, lse = uaa.attn_paged_fwd(g["q"], g["k"], g["v"], g["starts"], g["table"], g["lens"], seqs)
    with pytest.raises(uaa.UAAError, match="UAA_ERR_BAD_PAGE"):
        uaa.check_device_status()
    assert not out.any() and torch.isneginf(lse).all()
    g["lens"].copy_(torch.tensor([-3, 2 ** 31 - 1]))
    g["table"].fill_(1)
    out, lse = uaa.attn_paged_fwd(g["q"], g["k"], g["v"], g["starts"], g["table"], g["lens"])
    with pytest.raises(uaa.UAAError, match="UAA_ERR_BAD_PAGE"):
        uaa.check_device_status()
    assert not out[:new].any() and torch.isfinite(out[new:].float()).all()
    uaa.check_device_status()


@pytest.mark.gpu
def test_captured():
    """A captured call, replayed with other lengths, pages and chunks."""
    x = draw([1, 1, 1], [300, 20, 640], 6, 2, 64, 32, seed=9, spare=40, width=10)
    y = {n: t.to(DEV) for n, t in x.items()}

    def go():
        return uaa.attn_paged_fwd(y["q"], y["k"], y["v"], y["starts"], y["table"], y["lens"])

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        go()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = go()
    for seed, lens, news in ((9, [300, 20, 640], [1, 1, 1]), (10, [1, 700, 31], [1, 2, 0]), (11, [3, 2, 5], [3, 0, 0])):
        z = draw(news, lens, 6, 2, 64, 32, seed=seed)
        for n in ("q", "lens", "starts"):
            y[n].copy_(z[n])
        y["table"].fill_(-1)
        y["table"][:, : z["table"].shape[1]].copy_(z["table"])
        for n in ("k", "v"):
            y[n][: z[n].shape[0]].copy_(z[n])
        graph.replay()
        uaa.check_device_status()
        check({"out": out, "lse": lse}, against(z), BOTH, lens)


@pytest.mark.gpu
def test_other_strides_of_the_pools():
    """Pools kept heads first, and as one tensor of keys and values."""
    x = draw([3, 50], [200, 90], 4, 2, 64, 32, seed=12)
    want = step(x)
    y = {n: t.to(DEV) for n, t in x.items()}
    k, v = (y[n].transpose(1, 2).contiguous().transpose(1, 2) for n in ("k", "v"))
    assert torch.equal(uaa.attn_paged_fwd(y["q"], k, v, y["starts"], y["table"], y["lens"])[0], want["out"])
    both = torch.stack([y["k"], y["v"]], 3)  # (pages, page, Hk, 2, D)
    out, _ = uaa.attn_paged_fwd(y["q"], both[:, :, :, 0], both[:, :, :, 1], y["starts"], y["table"], y["lens"])
    assert torch.equal(out, want["out"])


@pytest.mark.gpu
def test_writes_stay_inside():
    from test_gpu_guard_bands import Guarded

    for news, lens in (([1], [1]), ([1, 1], [3000, 17]), ([129, 3], [500, 3])):
        x = draw(news, lens, 6, 2, 128, 16, seed=13)
        y = {n: t.to(DEV) for n, t in x.items()}
        g, T = Guarded(), sum(news)
        out, lse = g.empty((T, 6, 128), torch.bfloat16), g.empty((6, T), torch.float32)
        ws = g.empty((uaa.attn_seqs_workspace_bytes(len(lens), T, 6, 2, 128),), torch.uint8)
        uaa.attn_paged_fwd(y["q"], y["k"], y["v"], y["starts"], y["table"], y["lens"], out=out, lse=lse, workspace=ws)
        uaa.check_device_status()
        g.check()
        check({"out": out, "lse": lse}, against(x), BOTH)
