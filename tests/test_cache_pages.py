"""The pages of a cache: the host's bookkeeping against a plain model, and the device's pools, table and lengths."""
import ctypes
import random

import numpy as np
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from oracle import seqs as ref

DEV = "cuda"


class Host:
    """The C object without a device."""

    def __init__(self, pages, page, seqs, width):
        self.h = ctypes.c_void_p()
        self.status = uaa.lib().uaa_pages_create(ctypes.byref(self.h), pages, page, seqs, width)
        self.page, self.width = page, width

    def __del__(self):
        if self.h:
            uaa.lib().uaa_pages_destroy(self.h)

    def _two(self, a, b):
        n = len(a)
        return n, (ctypes.c_int * n)(*a), (ctypes.c_int * n)(*b)

    def append(self, seqs, counts):
        n, a, b = self._two(seqs, counts)
        return uaa.lib().uaa_pages_append(self.h, None, n, a, b, None, None, None)

    def fork(self, parents, children):
        n, a, b = self._two(parents, children)
        return uaa.lib().uaa_pages_fork(self.h, None, n, a, b, None)

    def truncate(self, seqs, lens):
        n, a, b = self._two(seqs, lens)
        return uaa.lib().uaa_pages_truncate(self.h, None, n, a, b, None)

    def compact(self):
        return uaa.lib().uaa_pages_compact(self.h, None, None)

    def row(self, seq):
        out = (ctypes.c_int * self.width)()
        n = uaa.lib().uaa_pages_row(self.h, seq, out, self.width)
        return n, list(out)[: -(-n // self.page)]

    def free(self):
        return uaa.lib().uaa_pages_free(self.h)


def err():
    return uaa.lib().uaa_last_error().decode()


def test_refusal_of_too_many_tokens():
    assert Host(4, 1024, 2, 2 ** 20).status == 0
    assert Host(4, 1024, 2, 2 ** 20 + 1).status == -2 and "table" in err()


def test_the_tensors_keep_their_places():
    """The calls hold the tensors' addresses: no other tensor takes their places."""
    c = uaa.PagedCache(1, 2, 16, 1, 64, 2, 2, device="cpu")
    for name in ("k", "v", "table", "lens", "page", "seqs"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name))


def test_refusals():
    L = uaa.lib()
    assert L.uaa_pages_create(None, 4, 16, 2, 2) == -1
    for bad in ((0, 16, 2, 2), (4, 16, 0, 2), (4, 16, 2, 0), (-1, 16, 2, 2)):
        assert Host(*bad).status == -1 and "positive" in err()
    for page in (0, 8, 48, 200):
        assert Host(4, page, 2, 2).status == -2 and "pages of" in err()
    assert Host(4, 16, 1 << 16, 1 << 16).status == -2 and "table" in err()
    h = Host(6, 16, 4, 3)
    assert h.status == 0 and h.free() == 6
    assert h.append([4], [1]) == -1 and "sequence 4" in err()
    assert h.append([-1], [1]) == -1
    assert h.append([1, 1], [1, 1]) == -1 and "twice" in err()
    assert h.append([1], [-1]) == -1 and "tokens" in err()
    assert h.append([1], [49]) == -1 and "49 tokens of 48" in err()
    assert h.append([0, 1, 2], [48, 48, 1]) == -7 and "7 pages wanted, 6 free" in err()
    assert h.free() == 6 and h.row(0) == (0, [])
    assert h.append([0, 1], [33, 5]) == 0 and h.free() == 2
    assert h.fork([0], [1]) == -1 and "not empty" in err()
    assert h.fork([0, 0], [2, 2]) == -1 and "twice" in err()
    assert h.fork([0, 2], [2, 3]) == -1 and "both" in err()
    assert h.fork([7], [2]) == -1
    assert h.truncate([0], [34]) == -1 and "33 tokens, not 34" in err()
    assert h.truncate([0], [-1]) == -1
    assert h.truncate([0, 0], [1, 1]) == -1 and "twice" in err()
    assert h.row(4)[0] == -1 and h.row(-1)[0] == -1
    assert h.row(0) == (33, [0, 1, 2]) and h.row(1) == (5, [3]) and h.free() == 2
    n, a, b = h._two([0], [1])
    assert L.uaa_pages_append(h.h, None, 5, a, b, None, None, None) == -1 and "5 sequences" in err()
    assert L.uaa_pages_append(h.h, None, -1, a, b, None, None, None) == -1
    assert L.uaa_pages_append(h.h, None, 1, None, b, None, None, None) == -1
    assert L.uaa_pages_append(None, None, 1, a, b, None, None, None) == -1
    assert L.uaa_pages_fork(None, None, 0, None, None, None) == -1 and L.uaa_pages_compact(None, None, None) == -1
    assert L.uaa_pages_row(None, 0, None, 0) == -1 and L.uaa_pages_free(None) == -1
    bad = [dict(k=0), dict(v=8), dict(table=0), dict(lens=2), dict(layers=0), dict(layers=40000), dict(row=8), dict(row=24)]
    for kw in bad:
        x = {**dict(k=1 << 20, v=1 << 20, table=1 << 20, lens=1 << 20, layers=1, row=256), **kw}
        assert L.uaa_pages_append(h.h, uaa._POOLS.pack(*x.values()), 1, a, b, None, None, None) == -1, kw
    assert h.row(0) == (33, [0, 1, 2])
    assert h.append([], []) == 0 and h.fork([], []) == 0 and h.truncate([], []) == 0 and h.compact() == 0
    with pytest.raises(TypeError):
        uaa.PagedCache(1, 4, 16, 2, 64, 2, 2, dtype=torch.float32)
    with pytest.raises(ValueError):
        uaa.PagedCache(1, 4, 16, 2, 80, 2, 2)
    with pytest.raises(uaa.UAAError, match="positive"):
        uaa.PagedCache(1, 0, 16, 2, 64, 2, 2)


def test_a_shared_last_page():
    h = Host(10, 16, 4, 4)
    assert h.append([0], [20]) == 0 and h.fork([0, 0], [1, 2]) == 0 and h.free() == 8
    assert h.append([0, 1, 2], [1, 1, 0]) == 0  # two of three holders get a page of their own
    assert [h.row(s)[1] for s in range(3)] == [[0, 2], [0, 3], [0, 1]]
    assert h.append([2], [1]) == 0 and h.row(2) == (21, [0, 1])  # the last one keeps it
    assert h.truncate([0, 1], [0, 16]) == 0 and h.free() == 8
    assert h.append([1], [1]) == 0 and h.row(1) == (17, [0, 2])
    # all holders at once: the last of them keeps the page
    h = Host(4, 16, 3, 2)
    assert h.append([0], [1]) == 0 and h.fork([0, 0], [1, 2]) == 0
    assert h.append([2, 0, 1], [1, 1, 1]) == 0 and [h.row(s)[1] for s in range(3)] == [[2], [0], [1]] and h.free() == 1
    # exactly as many pages as are wanted
    h = Host(3, 16, 3, 1)
    assert h.append([0], [1]) == 0 and h.fork([0, 0], [1, 2]) == 0 and h.append([0, 1, 2], [1, 1, 1]) == 0 and h.free() == 0
    h = Host(2, 16, 3, 1)
    assert h.append([0], [1]) == 0 and h.fork([0, 0], [1, 2]) == 0 and h.append([0, 1, 2], [1, 1, 1]) == -7 and h.free() == 1


def moves(rng, seqs, model, width, page):
    """A random operation that the model allows (or not for want of pages): its name and arguments."""
    op = rng.choice(("append",) * 4 + ("fork", "truncate", "truncate", "free", "compact"))
    some = rng.sample(range(seqs), rng.randint(0, seqs))
    if op == "append":
        return op, some, [rng.choice((0, 1, 1, rng.randint(0, 3 * page))) for _ in some]
    if op == "fork":
        empty = [s for s in some if not model.size[s]]
        full = [s for s in range(seqs) if model.size[s]]
        return (op, [rng.choice(full) for _ in empty], empty) if full else ("fork", [], [])
    if op == "truncate":
        return op, some, [rng.randint(0, model.size[s]) for s in some]
    return ("truncate", some, [0] * len(some)) if op == "free" else (op,)


@pytest.mark.parametrize("seed", range(30))
def test_random_operations_against_the_model(seed):
    rng = random.Random(seed)
    pages, page, seqs, width = rng.choice(((30, 16, 5, 9), (12, 32, 4, 6), (200, 16, 9, 30)))
    h, model = Host(pages, page, seqs, width), ref.Pages(pages, page, seqs)
    done = 0
    for _ in range(150):
        op, *a = moves(rng, seqs, model, width, page)
        before = [h.row(s) for s in range(seqs)]
        st = getattr(h, op)(*a)
        if st:
            assert op == "append" and [h.row(s) for s in range(seqs)] == before
            continue
        done += 1
        getattr(model, op)(*a)
        for s in range(seqs):
            assert h.row(s) == (model.size[s], model.held[s]), (op, a, s)
        assert h.free() == pages - len(model._used())
        if op == "compact":
            assert model._used() == set(range(len(model._used())))
    assert done > 60


# --------------------------------------------------------------------------- on the GPU
def same_as_model(c, model, shadow):
    """Table, lengths and every row that a sequence has filled."""
    table, lens = c.table.cpu().numpy(), c.lens.cpu().numpy()
    for s, row in model.held.items():
        assert lens[s] == model.size[s] and c.length(s) == model.size[s] and c.pages_of(s) == row
        assert table[s].tolist() == row + [-1] * (table.shape[1] - len(row)), s
    for pool, kept in ((c.k, shadow[0]), (c.v, shadow[1])):
        pool = pool.cpu()
        for s, row in model.held.items():
            for i, p in enumerate(row):
                n = min(c.page, model.size[s] - i * c.page)
                assert torch.equal(pool[:, p, :n], torch.stack([kept[s][layer][i * c.page: i * c.page + n] for layer in range(pool.shape[0])])), (s, i)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("seed,page,heads,dim,layers", [(0, 16, 1, 64, 2), (1, 32, 3, 64, 1), (2, 16, 8, 128, 3), (3, 128, 2, 64, 2)])
def test_random_operations_on_the_device(seed, page, heads, dim, layers, dtype):
    rng, g = random.Random(seed), torch.Generator().manual_seed(seed)
    pages, seqs, width = 40, 6, 8
    c, model = uaa.PagedCache(layers, pages, page, heads, dim, seqs, width, dtype=dtype), ref.Pages(pages, page, seqs)
    for pool in (c.k, c.v):
        pool.fill_(float("nan"))
    kept = [{s: [torch.empty(0, heads, dim, dtype=dtype)] * layers for s in range(seqs)} for _ in range(2)]
    done = 0
    for _ in range(80):
        op, *a = moves(rng, seqs, model, width, page)
        try:
            res = getattr(c, op)(*a)
        except uaa.UAAError:
            assert op == "append"
            continue
        done += 1
        getattr(model, op)(*a)
        if op == "append":
            starts, ids = res
            assert starts.tolist() == [sum(a[1][:i]) for i in range(len(a[1]) + 1)] and ids.tolist() == list(a[0])
            T = sum(a[1])
            for layer in range(layers):
                new = [torch.randn(T, heads, dim, generator=g).to(dtype) for _ in range(2)]
                c.write(layer, new[0].to(DEV), new[1].to(DEV), starts, ids)
                for x, t in zip(kept, new):
                    at = 0
                    for s, n in zip(*a):
                        x[s] = list(x[s])
                        x[s][layer] = torch.cat([x[s][layer], t[at: at + n]])
                        at += n
        elif op == "fork":
            for x in kept:
                for p, s in zip(*a):
                    x[s] = list(x[p])
        elif op == "truncate":
            for x in kept:
                for s, n in zip(*a):
                    x[s] = [t[:n] for t in x[s]]
        same_as_model(c, model, kept)
    uaa.check_device_status()
    assert done > 40


@pytest.mark.gpu
def test_many_changes_at_once():
    """More table changes and more moves than one launch takes."""
    page, seqs = 16, 2700
    c, model = uaa.PagedCache(1, 3 * seqs, page, 1, 64, seqs, 2), ref.Pages(3 * seqs, page, seqs)
    ids = list(range(seqs))
    starts, dev = c.append(ids, [17] * seqs)
    k = torch.randn(17 * seqs, 1, 64, device=DEV).bfloat16()
    c.write(0, k, -k, starts, dev)
    c.free(ids[::2])
    assert c.free_pages == 3 * seqs - 2 * (seqs // 2)
    c.compact()
    assert sorted(p for s in ids[1::2] for p in c.pages_of(s)) == list(range(2 * (seqs // 2)))
    for s in ids[1::300]:
        pages = torch.tensor(c.pages_of(s), device=DEV)
        assert torch.equal(c.table[s], pages.int()) and c.lens[s] == 17
        assert torch.equal(c.k[0][pages].flatten(0, 1)[:17], k[17 * s: 17 * s + 17])
        assert torch.equal(c.v[0][pages].flatten(0, 1)[:17], -k[17 * s: 17 * s + 17])
    assert (c.table[::2] == -1).all() and not c.lens[::2].any()
    # a fork of one sequence to many, each of which then gets a page of its own
    kids = ids[::2][:1300]
    c.fork([1] * len(kids), kids)
    c.append(kids, [3] * len(kids))
    assert len({c.pages_of(s)[1] for s in kids + [1]}) == len(kids) + 1 and {c.pages_of(s)[0] for s in kids} == {c.pages_of(1)[0]}
    last = torch.tensor([c.pages_of(s)[1] for s in kids], device=DEV)
    assert (c.k[0, last, 0] == k[17 + 16]).all() and (c.lens[torch.tensor(kids, device=DEV)] == 20).all()
    uaa.check_device_status()
    del model


@pytest.mark.gpu
def test_rows_that_no_one_filled_stay():
    """A copy takes the filled rows of a page and leaves the others."""
    c = uaa.PagedCache(2, 8, 32, 2, 64, 3, 2)
    c.k.fill_(1.0)
    c.v.fill_(2.0)
    c.append([0], [40])
    c.k[:, 1] = 5.0
    c.fork([0], [1])
    c.append([1], [1])
    assert c.pages_of(1) == [0, 2]
    assert (c.k[:, 2, :8] == 5).all() and (c.k[:, 2, 8:] == 1).all() and (c.v[:, 2] == 2).all() and (c.k[:, 3:] == 1).all()


@pytest.mark.gpu
def test_not_inside_a_capture():
    c = uaa.PagedCache(1, 8, 16, 1, 64, 2, 4)
    c.append([0], [5])
    x = torch.zeros(1, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x += 1
        for call in (lambda: c.append([0], [1]), lambda: c.fork([0], [1]), lambda: c.free([0]), c.compact):
            with pytest.raises(uaa.UAAError, match="capture"):
                call()
    graph.replay()
    assert c.length(0) == 5 and x.item() == 1


@pytest.mark.gpu
def test_bad_rows_are_skipped_and_reported():
    c = uaa.PagedCache(1, 4, 16, 2, 64, 3, 2)
    starts, seqs = c.append([0, 1], [3, 20])
    c.k.fill_(7.0)
    c.v.fill_(7.0)
    k = torch.ones(23, 2, 64, device=DEV).bfloat16()
    c.table[1, 1] = 4
    c.write(0, k, k, starts, seqs)
    with pytest.raises(uaa.UAAError, match="UAA_ERR_BAD_PAGE"):
        uaa.check_device_status()
    assert (c.k[0, 0, :3] == 1).all() and (c.k[0, 1] == 1).all() and (c.k[0, 2:] == 7).all() and (c.k[0, 0, 3:] == 7).all()
    c.k.fill_(7.0)
    for ids, lens in (([-1, 3], [3, 20]), ([0, 1], [-5, 2 ** 31 - 1]), ([0, 1], [2, 19])):
        c.lens[:2] = torch.tensor(lens, dtype=torch.int32)
        c.write(0, k, k, starts, torch.tensor(ids, dtype=torch.int32, device=DEV))
        with pytest.raises(uaa.UAAError, match="UAA_ERR_BAD_PAGE"):
            uaa.check_device_status()
    assert (c.k[0, 2:] == 7).all()
    # more tokens than sequences have: the rest goes nowhere
    c.lens[:2] = torch.tensor([3, 16], dtype=torch.int32)
    c.k.fill_(7.0)
    c.write(0, k, k, torch.tensor([0, 3], dtype=torch.int32, device=DEV), torch.tensor([0], dtype=torch.int32, device=DEV))
    uaa.check_device_status()
    assert (c.k[0, 0, :3] == 1).all() and (c.k[0, 0, 3:] == 7).all() and (c.k[0, 1:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("g", [1, 3])
def test_a_server_from_prompt_to_samples(g):
    """Prompts by packed attention, their continuation in chunks and token by token, samples that fork, sequences that end:
    every result equals packed attention over the whole sequence so far, within both sides' roundings."""
    layers, page, Hk, D, Hq = 2, 16, 2, 64, 2 * g
    c = uaa.PagedCache(layers, 200, page, Hk, D, 6, 30)
    gen = torch.Generator().manual_seed(g)
    past = {s: [[torch.empty(0, Hk, D).bfloat16()] * 2 for _ in range(layers)] for s in range(6)}

    def go(ids, counts):
        starts, seqs = c.append(ids, counts)
        T, worst = sum(counts), 0.0
        for layer in range(layers):
            q, k, v = (torch.randn(T, h, D, generator=gen).bfloat16() for h in (Hq, Hk, Hk))
            c.write(layer, k.to(DEV), v.to(DEV), starts, seqs)
            out, lse = c.attend(layer, q.to(DEV), starts, seqs)
            at = 0
            for s, n in zip(ids, counts):
                past[s][layer] = [torch.cat([a, b[at: at + n]]) for a, b in zip(past[s][layer], (k, v))]
                want = ref.attention(*(t.double().numpy() for t in (q[at: at + n], *past[s][layer])), True)
                for name, x in (("out", out[at: at + n]), ("lse", lse[:, at: at + n])):
                    assert (np.abs(x.cpu().double().numpy() - want[name][0]) <= want[name][1]).all(), (ids, s, name)
                at += n
            if all(past[s][layer][0].shape[0] == n for s, n in zip(ids, counts)):  # a prompt: packed attention is the same
                one, _ = uaa.attn_packed_fwd(q.to(DEV), k.to(DEV), v.to(DEV), starts)
                worst = max(worst, (one.float() - out.float()).abs().max().item())
        assert worst < 0.05

    go([0, 1, 2], [130, 1, 50])
    go([0, 1, 2], [1, 1, 1])
    go([1, 0], [70, 1])
    c.fork([0, 0], [3, 4])
    for a in (3, 4):
        past[a] = [list(x) for x in past[0]]
    for _ in range(3):
        go([0, 3, 4, 2], [1, 1, 1, 1])
    c.free([0, 2])
    past[0] = past[2] = [[torch.empty(0, Hk, D).bfloat16()] * 2 for _ in range(layers)]
    c.truncate([4], [131])
    past[4] = [[t[:131] for t in x] for x in past[4]]
    c.compact()
    go([4, 1, 3, 5], [2, 1, 40, 17])
    uaa.check_device_status()
