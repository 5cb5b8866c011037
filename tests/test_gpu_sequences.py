"""Attention over packed sequences and paged caches where it can go wrong beside the numbers: many sequences, tensors past
2^31 elements, stores past an output's end, a load that never comes, a warp that is far behind, the debug build's checks."""
import itertools
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from oracle import seqs as ref
from helpers import bits, f64
from test_gpu_abort_paths import _expect_timeout, dropped_load
from test_gpu_guard_bands import Guarded
from test_packed_attention import ALL, against, check, draw, step
import test_paged_attention as paged

pytestmark = pytest.mark.gpu

DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# --------------------------------------------------------------------------- many sequences
@pytest.mark.parametrize("B,longest", [(385, 9), (1500, 5), (5000, 2), (700, 140)])
@pytest.mark.parametrize("causal", [True, False])
def test_many_sequences(B, longest, causal):
    """More sequences than threads, and more in a share than shared memory keeps."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, longest + 1, (B,), generator=g).tolist()
    x = draw(lens, lens, 3, 1, 64, seed=B)
    check(step(x, causal), against(x, causal), ALL)


@pytest.mark.parametrize("page", [16, 128])
def test_many_sequences_of_a_cache(page):
    g = torch.Generator().manual_seed(5)
    B = 900
    lens = torch.randint(0, 400, (B,), generator=g).tolist()
    news = [min(n, 1 + (i % 7 == 0) * 30) for i, n in enumerate(lens)]
    x = paged.draw(news, lens, 2, 1, 64, page, seed=6)
    check(paged.step(x), paged.against(x), ("out", "lse"))


def test_the_most_sequences():
    B = 65535
    x = draw([1] * B, [1] * B, 1, 1, 64, seed=3)
    got = step(x)
    assert torch.equal(got["out"].cpu(), x["v"]) and torch.equal(got["dv"].cpu(), x["do"])  # one key each: P = 1
    # dS = P (dP - Delta) = 0: two 32-bit sums of the same products, in their own orders, each off by F32 of the magnitudes
    q, k, v, do = (f64(x[n]) for n in ("q", "k", "v", "do"))
    off = 64 ** -0.5 * 2 * ref.F32 * (np.abs(do) * np.abs(v)).sum(-1, keepdims=True)
    assert (np.abs(f64(got["dq"])) <= off * np.abs(k)).all() and (np.abs(f64(got["dk"])) <= off * np.abs(q)).all()


# --------------------------------------------------------------------------- tensors past 2^31 elements
@pytest.mark.parametrize("D", [128, 64])
def test_packed_past_2_31_elements(D):
    Hq, Hk = 128 * 128 // D, 64 * 128 // D
    lens = [150] * 930 + [77]
    T = sum(lens)
    assert T * Hq * D > 2 ** 31
    g = torch.Generator(DEV).manual_seed(8)
    q, do = (torch.randn(T, Hq, D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    k, v = (torch.randn(T, Hk, D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    starts = torch.tensor(list(itertools.accumulate(lens, initial=0)), dtype=torch.int32, device=DEV)
    out, lse = uaa.attn_packed_fwd(q, k, v, starts)
    grads = uaa.attn_packed_bwd(q, k, v, out, do, lse, starts)
    uaa.check_device_status()
    for b in (0, 500, 930):
        a, e = sum(lens[:b]), sum(lens[: b + 1])
        for j in (0, Hk - 1):
            hs, ks = slice(2 * j, 2 * j + 2), slice(j, j + 1)
            want = ref.attention(f64(q[a:e, hs]), f64(k[a:e, ks]), f64(v[a:e, ks]), True, None, f64(do[a:e, hs]))
            got = {"out": out[a:e, hs], "lse": lse[hs, a:e], "dq": grads[0][a:e, hs], "dk": grads[1][a:e, ks], "dv": grads[2][a:e, ks]}
            check(got, want, ALL, (b, j))
    del q, k, v, do, out, lse, grads, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("page", [64, 256])
def test_pools_past_2_31_elements(page):
    Hk, D, N = 8, 128, 2 ** 22 // page // 2 + 40
    assert N * page * Hk * D > 2 ** 31
    g = torch.Generator(DEV).manual_seed(9)
    k, v = (torch.randn(N, page, Hk, D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    lens, W = [3000, 700], -(-3000 // page)
    table = torch.full((2, W), -1, dtype=torch.int32)
    ids = [N - 1 - 3 * i for i in range(W)] + [5 * i for i in range(-(-700 // page))]
    table[0], table[1, : -(-700 // page)] = torch.tensor(ids[:W]), torch.tensor(ids[W:])
    starts, held = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0, 40, 41], lens))
    new = torch.randn(41, Hk, D, generator=g, device=DEV, dtype=torch.bfloat16)
    uaa.cache_write(new, -new, k, v, starts, table.to(DEV), held)
    q = torch.randn(41, 16, D, generator=g, device=DEV, dtype=torch.bfloat16)
    out, lse = uaa.attn_paged_fwd(q, k, v, starts, table.to(DEV), held)
    uaa.check_device_status()
    for b, (a, e) in enumerate(((0, 40), (40, 41))):
        p = table[b, : -(-lens[b] // page)].to(DEV).long()
        kk, vv = (t[p].flatten(0, 1)[: lens[b]] for t in (k, v))
        assert torch.equal(kk[lens[b] - (e - a):], new[a:e]) and torch.equal(vv[lens[b] - (e - a):], -new[a:e])
        want = ref.attention(f64(q[a:e]), f64(kk), f64(vv), True)
        check({"out": out[a:e], "lse": lse[:, a:e]}, want, ("out", "lse"), b)
    del k, v, kk, vv
    torch.cuda.empty_cache()


# --------------------------------------------------------------------------- bounds of every store
@pytest.mark.parametrize("lens,lens_k", [([1], [1]), ([127], [127]), ([129, 1], [129, 1]), ([257], [40]), ([3, 200], [300, 77]),
                                         ([700], [700]), ([0, 5], [130, 5])], ids=str)
@pytest.mark.parametrize("Hq,Hk,D", [(2, 2, 64), (6, 2, 128), (5, 1, 64)])
def test_stores_stay_inside(lens, lens_k, Hq, Hk, D):
    x = draw(lens, lens_k, Hq, Hk, D, seed=31)
    y = {n: t.to(DEV) for n, t in x.items()}
    T, Tk, B = sum(lens), sum(lens_k), len(lens)
    g = Guarded()
    out, dq = (g.empty((T, Hq, D), torch.bfloat16) for _ in range(2))
    dk, dv = (g.empty((Tk, Hk, D), torch.bfloat16) for _ in range(2))
    lse = g.empty((Hq, T), torch.float32)
    w1 = g.empty((uaa.attn_seqs_workspace_bytes(B, T, Hq, Hk, D),), torch.uint8)
    w2 = g.empty((uaa.attn_packed_bwd_workspace_bytes(B, T, Hq, Hk, D),), torch.uint8)
    uaa.attn_packed_fwd(y["q"], y["k"], y["v"], y["starts"], y["starts_k"], out=out, lse=lse, workspace=w1)
    uaa.attn_packed_bwd(y["q"], y["k"], y["v"], out, y["do"], lse, y["starts"], y["starts_k"], dq=dq, dk=dk, dv=dv, workspace=w2)
    uaa.check_device_status()
    g.check()
    check({"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}, against(x), ALL)


# --------------------------------------------------------------------------- a load that never comes
@pytest.mark.parametrize("n", [0, 1, 2, 3])
@pytest.mark.parametrize("lens,Hq,Hk,D", [([256], 1, 1, 128), ([700], 3, 1, 64), ([100, 90, 300], 2, 2, 64), ([64], 2, 1, 128)])
def test_forward_gives_up_and_the_next_call_is_correct(lens, Hq, Hk, D, n):
    """Some K or V tile of every block is never loaded: the call ends, says so, and the next one is right."""
    x = draw(lens, lens, Hq, Hk, D, seed=41)
    y = {m: t.to(DEV) for m, t in x.items()}
    go = lambda: uaa.attn_packed_fwd(y["q"], y["k"], y["v"], y["starts"])  # noqa: E731
    want = go()
    uaa.check_device_status()
    with dropped_load(n):
        go()
    again = go()
    torch.cuda.synchronize()
    if len(lens) == 1 and lens[0] <= 128 and n > 1:
        uaa.check_device_status()  # no block has so many loads
    else:
        _expect_timeout()
    for a, b in zip(again, want):
        assert np.array_equal(bits(a), bits(b))


@pytest.mark.parametrize("n", [0, 1, 3, 6])
@pytest.mark.parametrize("news,lens", [([1], [2000]), ([1] * 5, [600] * 5), ([300], [700])], ids=str)
def test_paged_gives_up_and_the_next_call_is_correct(news, lens, n):
    x = paged.draw(news, lens, 4, 1, 128, 32, seed=42)
    y = {m: t.to(DEV) for m, t in x.items()}
    go = lambda: uaa.attn_paged_fwd(y["q"], y["k"], y["v"], y["starts"], y["table"], y["lens"])  # noqa: E731
    want = go()
    uaa.check_device_status()
    with dropped_load(n):
        go()
    again = go()
    torch.cuda.synchronize()
    try:
        uaa.check_device_status()
        assert n == 6  # few blocks have so many loads
    except uaa.UAAError as e:
        assert e.status == -5
    uaa.check_device_status()
    for a, b in zip(again, want):
        assert np.array_equal(bits(a), bits(b))


@pytest.mark.parametrize("n", [0, 1, 2, 3])
@pytest.mark.parametrize("lens,Hq,Hk,D", [([256], 1, 1, 128), ([700], 3, 1, 64), ([130, 90, 300], 2, 2, 64)])
def test_backward_gives_up_and_the_next_call_is_correct(lens, Hq, Hk, D, n):
    x = draw(lens, lens, Hq, Hk, D, seed=43)
    y = {m: t.to(DEV) for m, t in x.items()}
    out, lse = uaa.attn_packed_fwd(y["q"], y["k"], y["v"], y["starts"])
    go = lambda: uaa.attn_packed_bwd(y["q"], y["k"], y["v"], out, y["do"], lse, y["starts"])  # noqa: E731
    want = go()
    uaa.check_device_status()
    with dropped_load(n):
        go()
    again = go()
    torch.cuda.synchronize()
    _expect_timeout()
    for a, b in zip(again, want):
        assert np.array_equal(bits(a), bits(b))


# --------------------------------------------------------------------------- a late warp
@pytest.mark.parametrize("lens,Hq,Hk,D,causal", [([700, 300, 1, 129, 260], 24, 8, 128, True), ([300] * 8, 24, 24, 64, False),
                                                 ([40] * 60, 16, 8, 128, True)])
def test_a_late_warp_changes_nothing(lens, Hq, Hk, D, causal):
    if not uaa.debug_build():
        pytest.skip("runs in the child process that loads the debug build")
    x = draw(lens, lens, Hq, Hk, D, seed=51)
    want = step(x, causal)
    for warp in range(12):
        uaa.debug_late_warp(warp, 20000)
        try:
            got = step(x, causal)
        finally:
            uaa.debug_late_warp()
        for n in ALL:
            assert np.array_equal(bits(got[n]), bits(want[n])), (warp, n)


@pytest.mark.parametrize("D", [64, 128])
def test_values_that_are_not_finite_in_every_item(D):
    """Items in a row with infinities and NaNs in the values that only some of their rows read, whichever warp comes late."""
    n, Hq, m = 256, 24, 128
    x = draw([n] * 40, [n] * 40, Hq, Hq, D, seed=53)
    bad = torch.arange(m - 1, n, m)  # the last key of each tile of keys
    v = x["v"].view(40, n, Hq, D)
    v[:, bad, :, 3] = float("inf")
    v[:, bad, :, 5] = float("nan")
    reads = torch.arange(n)[None, :, None] >= bad[0]
    late = range(8) if uaa.debug_build() else ()
    for warp in (-1, *late):
        if warp >= 0:
            uaa.debug_late_warp(warp, 1000000)  # longer than a way out with such values takes
        try:
            out = step(x, grads=False)["out"].cpu().float().view(40, n, Hq, D)
        finally:
            if warp >= 0:
                uaa.debug_late_warp()
        assert torch.equal(torch.isinf(out[..., 3]), reads.expand(40, n, Hq)), warp
        assert torch.equal(torch.isnan(out[..., 5]), reads.expand(40, n, Hq)), warp
        out[..., 3] = out[..., 5] = 0
        assert torch.isfinite(out).all(), warp


@pytest.mark.parametrize("D", [64, 128])
def test_a_late_warp_changes_nothing_with_fewer_keys_than_queries(D):
    """Items whose first tile reads no key behind items whose second tile has a step more than the first."""
    if not uaa.debug_build():
        pytest.skip("runs in the child process that loads the debug build")
    x = draw([256] * 800, [256, 128] * 400, 1, 1, D, seed=54)
    want = step(x)
    check(want, against(x), ALL)
    for warp in range(12):
        uaa.debug_late_warp(warp, 20000)
        try:
            got = step(x)
        finally:
            uaa.debug_late_warp()
        for n in ALL:
            assert np.array_equal(bits(got[n]), bits(want[n])), (warp, n)


@pytest.mark.parametrize("news,lens", [([1] * 30, [900] * 30), ([1, 200, 7, 1], [3000, 700, 129, 1])], ids=["tokens", "chunks"])
def test_a_late_warp_changes_nothing_over_pages(news, lens):
    if not uaa.debug_build():
        pytest.skip("runs in the child process that loads the debug build")
    x = paged.draw(news, lens, 24, 8, 128, 32, seed=52)
    want = paged.step(x)
    for warp in range(12):
        uaa.debug_late_warp(warp, 20000)
        try:
            got = paged.step(x)
        finally:
            uaa.debug_late_warp()
        for n in ("out", "lse"):
            assert np.array_equal(bits(got[n]), bits(want[n])), (warp, n)


# --------------------------------------------------------------------------- the debug build
@pytest.mark.parametrize("selection,least", [
    (["tests/test_packed_attention.py", "tests/test_paged_attention.py", "tests/test_cache_pages.py"], 300),
    (["tests/test_gpu_sequences.py", "-k", "late_warp or stores_stay or many or every_item"], 30)])
def test_under_the_debug_build(selection, least):
    """The operators' tests once more in a child process whose library checks every tensor-core operand and store."""
    if uaa.debug_build():
        pytest.skip("this is the child process")
    from ulysses_dit_attention_gb300 import build

    build.build(debug=True)
    cmd = [sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-m", "gpu", *selection]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, UAA_DEBUG="1"), capture_output=True, text=True, timeout=1800)
    tail = "\n".join((r.stdout + r.stderr).strip().splitlines()[-30:])
    assert r.returncode == 0, tail
    m = re.search(r"(\d+) passed", tail)
    assert m and int(m.group(1)) >= least and " skipped" not in tail, tail
