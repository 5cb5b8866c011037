"""What is measured of attention over sequences of their own lengths: packed sequences with grouped heads,
chunks of new tokens over a paged cache, and the cache's pages.

Each case is one pass as a program makes it; ``run`` computes it in elementary torch operations
(``own = False``) or through the library's calls (``own = True``), ``exact`` from the definition in
64 bits.
"""
import heapq
import math
import random

import torch

own = False

BF16, FP16 = "bfloat16", "float16"


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # Three short prompts at once, fewer key heads than query heads.  Latency counts.
        {"name": "prompt_short", "op": "packed", "n": 3, "shortest": 1, "longest": 150, "lens": 4, "Hq": 24, "Hk": 8,
         "D": 64, "causal": True, "dtype": BF16, "grad": False},
        # Prompts of very different lengths packed into one tensor, 16-bit floats with five queries a key head.
        {"name": "prompt_mixed", "op": "packed", "n": 11, "shortest": 60, "longest": 4500, "lens": 7, "Hq": 40, "Hk": 8,
         "D": 128, "causal": True, "dtype": FP16, "grad": False},
        # One long prompt of an odd length.
        {"name": "prompt_long", "op": "packed", "n": 1, "shortest": 16389, "longest": 16389, "lens": 1, "Hq": 40,
         "Hk": 8, "D": 128, "causal": True, "dtype": BF16, "grad": False},
        # Training step on images of several resolutions packed without padding: every token reads its own image.
        {"name": "pack_step_images", "op": "packed", "n": 12, "shortest": 256, "longest": 1100, "lens": 3, "Hq": 24,
         "Hk": 24, "D": 64, "causal": False, "dtype": BF16, "grad": True},
        # Training step on texts packed one behind the other, three queries a key head.
        {"name": "pack_step_texts", "op": "packed", "n": 6, "shortest": 300, "longest": 4100, "lens": 9, "Hq": 24,
         "Hk": 8, "D": 128, "causal": True, "dtype": BF16, "grad": True},
        # Training step on one long sequence.
        {"name": "pack_step_long", "op": "packed", "n": 1, "shortest": 8191, "longest": 8191, "lens": 1, "Hq": 24,
         "Hk": 8, "D": 128, "causal": True, "dtype": BF16, "grad": True},
        # One new token of one sequence with a short past, small pages.  Latency counts.
        {"name": "paged_token_short", "op": "paged", "n": 1, "new_least": 1, "new_most": 1, "shortest": 700,
         "longest": 700, "lens": 1, "Hq": 24, "Hk": 24, "D": 64, "page": 16, "dtype": BF16},
        # One new token of each of sixteen sequences with long pasts of different lengths.
        {"name": "paged_token_long", "op": "paged", "n": 16, "new_least": 1, "new_most": 1, "shortest": 6000,
         "longest": 24000, "lens": 5, "Hq": 40, "Hk": 8, "D": 128, "page": 64, "dtype": BF16},
        # Chunks of prompts beside sequences that go on token by token, in one batch.
        {"name": "paged_chunk_mixed", "op": "paged", "n": 24, "new_least": 1, "new_most": 700, "shortest": 100,
         "longest": 9000, "lens": 8, "Hq": 24, "Hk": 8, "D": 128, "page": 32, "dtype": FP16},
        # The last chunk of a long prompt.
        {"name": "paged_chunk_long", "op": "paged", "n": 1, "new_least": 2048, "new_most": 2048, "shortest": 27280,
         "longest": 27280, "lens": 1, "Hq": 40, "Hk": 8, "D": 128, "page": 128, "dtype": BF16},
        # Sampling several continuations of each prompt: the children share the parents' pages, and every one that
        # goes on gets a last page of its own.
        {"name": "pages_fork", "op": "fork", "n": 8, "children": 5, "shortest": 300, "longest": 2600, "lens": 2,
         "layers": 4, "Hk": 8, "D": 128, "page": 64, "pages": 448, "dtype": BF16},
        # A server's cache after half of the sequences have ended, closed up so that the others lie together.
        {"name": "pages_compact", "op": "compact", "n": 16, "children": 24, "shortest": 100, "longest": 2600,
         "lens": 6, "layers": 4, "Hk": 8, "D": 128, "page": 64, "pages": 1024, "dtype": BF16},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("packed", "packed", "packed", "paged", "paged", "paged", "fork", "compact"))
    D, dtype = rng.choice((64, 128)), rng.choice((BF16, BF16, FP16))
    lens = rng.randint(1, 1 << 20)
    if op in ("fork", "compact"):
        layers, Hk, page = rng.choice((1, 2, 4)), rng.choice((1, 4, 8)), rng.choice((16, 32, 64, 128))
        n, children = _log_int(rng, 1, 16), _log_int(rng, 1, 6) if op == "fork" else _log_int(rng, 2, 24)
        longest = _log_int(rng, 30, 2600)
        case = {"op": op, "n": n, "children": children, "shortest": rng.randint(1, longest), "longest": longest,
                "lens": lens, "layers": layers, "Hk": Hk, "D": D, "page": page, "pages": 0, "dtype": dtype}
        most = sum(-(-x // page) for x in _lengths(case) + (_lengths(case, 1) if op == "compact" else []))
        case["pages"] = most + (2 * n * children + n if op == "fork" else 0) + rng.randint(0, 40)
        return case
    Hk = rng.choice((1, 2, 4, 8, 16, 24))
    Hq = Hk * rng.choice([g for g in (1, 2, 3, 4, 5, 6, 7, 8, 12, 16) if Hk * g <= 40])
    n = _log_int(rng, 1, 32)
    if op == "packed":
        # pairs of a query and a key: below the largest listed case, a training step's counting for 3.5
        grad = dtype == BF16 and rng.random() < 0.6
        pairs = 24 * 8191 * 8191 // 2 if grad else 40 * 16389 * 16389 // 2
        top = max(2, int(math.sqrt(pairs / (n * Hq))))
        longest = _log_int(rng, 1, min(top, 8191 if grad else 16389))
        return {"op": op, "n": n, "shortest": rng.randint(1, longest), "longest": longest, "lens": lens, "Hq": Hq,
                "Hk": Hk, "D": D, "causal": rng.random() < 0.7, "dtype": dtype, "grad": grad}
    longest = _log_int(rng, 1, min(27280, 27280 * 40 * 8 // (n * Hk)))
    new_most = 1 if rng.random() < 0.5 else _log_int(rng, 1, max(1, min(longest, 27280 * 40 * 2048 // (n * Hq * longest))))
    return {"op": op, "n": n, "new_least": 1, "new_most": new_most, "shortest": rng.randint(min(new_most, longest), longest),
            "longest": longest, "lens": lens, "Hq": Hq, "Hk": Hk, "D": D, "page": rng.choice((16, 32, 64, 128, 256)),
            "dtype": dtype}


def _lengths(case, which=0):
    """The sequences' lengths, spread over the logarithm of their range; ``which`` = 1: those of the sequences that
    come and go in the cache."""
    rng = random.Random(1000 * case["lens"] + which)
    lens = [_log_int(rng, case["shortest"], case["longest"]) for _ in range(case["children"] if which else case["n"])]
    if not which and case["n"] > 1:
        lens[rng.randrange(case["n"])] = case["longest"]
    return lens


def _news(case):
    """New tokens of each sequence of a paged batch: chunks for a few of them, the least for the others."""
    rng = random.Random(1000 * case["lens"] + 2)
    lens = _lengths(case)
    news = [_log_int(rng, case["new_least"], case["new_most"]) if rng.random() < 0.3 else case["new_least"] for _ in lens]
    news[lens.index(max(lens))] = case["new_most"]
    return [min(n, x) for n, x in zip(news, lens)]


def work(case):
    D = case["D"]
    if case["op"] in ("fork", "compact"):
        row = 2 * 2 * case["layers"] * case["Hk"] * D  # one token's keys and values of all layers
        lens, page = _lengths(case), case["page"]
        if case["op"] == "fork":  # rows of the last pages that the children copy, and their new token
            rows = sum(case["children"] * (x % page + 1) for x in lens)
            return {"bytes": 2 * rows * row, "flops": 0}
        owner, moves = _compacted(case)
        rows = sum(r for _, _, r in moves) + sum(_lengths(case, 1))
        return {"bytes": 2 * rows * row, "flops": 0}
    Hq, Hk, lens = case["Hq"], case["Hk"], _lengths(case)
    if case["op"] == "packed":
        T = sum(lens)
        pairs = sum(x * (x + 1) // 2 if case["causal"] else x * x for x in lens)
        q, k = 2 * T * Hq * D, 2 * T * Hk * D
        if case["grad"]:
            return {"bytes": 4 * q + 4 * k, "flops": 14 * pairs * Hq * D}  # q, o, dout, dq; k, v, dk, dv
        return {"bytes": 2 * q + 2 * k + 4 * T * Hq, "flops": 4 * pairs * Hq * D}
    news = _news(case)
    pairs = sum(n * (x - n) + n * (n + 1) // 2 for n, x in zip(news, lens))
    q = 2 * sum(news) * Hq * D
    return {"bytes": 2 * q + 4 * sum(lens) * Hk * D + 4 * sum(news) * Hq, "flops": 4 * pairs * Hq * D}


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _starts(lens):
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    return _prepare(case, seed, own)


def _prepare(case, seed, library):
    g, dt, D = _gen(seed), getattr(torch, case["dtype"]), case["D"]
    lens = _lengths(case)
    if case["op"] == "packed":
        T = sum(lens)
        st = {"case": case, "lens": lens, "starts": _starts(lens), "q": _normal(g, T, case["Hq"], D, dtype=dt),
              "k": _normal(g, T, case["Hk"], D, dtype=dt), "v": _normal(g, T, case["Hk"], D, dtype=dt)}
        if case["grad"]:
            st["dout"] = _normal(g, T, case["Hq"], D, dtype=dt)
        return st
    if case["op"] == "paged":
        news, page = _news(case), case["page"]
        need = [-(-x // page) for x in lens]
        width, total = max(need) + 3, sum(need) + 5
        order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at: at + n]
            at += n
        return {"case": case, "lens": lens, "news": news, "starts": _starts(news), "table": table,
                "held": torch.tensor(lens, dtype=torch.int32, device="cuda"),
                "q": _normal(g, sum(news), case["Hq"], D, dtype=dt),
                "k": _normal(g, total, page, case["Hk"], D, dtype=dt),
                "v": _normal(g, total, page, case["Hk"], D, dtype=dt)}
    n, extra = case["n"], case["n"] * case["children"] if case["op"] == "fork" else case["children"]
    width = max(-(-(x + 1) // case["page"]) for x in lens + _lengths(case, 1)) + 1
    shape = (case["layers"], case["pages"], case["page"], case["Hk"], D)
    new = n + extra if case["op"] == "fork" else sum(_lengths(case, 1))
    st = {"case": case, "lens": lens, "newk": _normal(g, case["layers"], new, case["Hk"], D, dtype=dt),
          "newv": _normal(g, case["layers"], new, case["Hk"], D, dtype=dt)}
    if library:
        import ulysses_dit_attention_gb300 as uaa

        c = st["cache"] = uaa.PagedCache(case["layers"], case["pages"], case["page"], case["Hk"], D, n + extra, width,
                                         dtype=dt)
    else:
        c = st["cache"] = _Pages(case["pages"], case["page"], n + extra, width)
        c.k, c.v = (torch.empty(shape, dtype=dt, device="cuda") for _ in range(2))
    c.append(list(range(n)), lens)
    for pool in (c.k, c.v):
        for layer in range(case["layers"]):
            pool[layer].copy_(_normal(g, *shape[1:], dtype=dt))
    return st


# --------------------------------------------------------------------------- the library's calls
def _run_own(st):
    import ulysses_dit_attention_gb300 as uaa

    case = st["case"]
    if case["op"] == "packed":
        out, lse = uaa.attn_packed_fwd(st["q"], st["k"], st["v"], st["starts"], causal=case["causal"])
        if not case["grad"]:
            return out, lse
        return (out,) + tuple(uaa.attn_packed_bwd(st["q"], st["k"], st["v"], out, st["dout"], lse, st["starts"],
                                                  causal=case["causal"]))
    if case["op"] == "paged":
        return uaa.attn_paged_fwd(st["q"], st["k"], st["v"], st["starts"], st["table"], st["held"])
    return _turn(st)


def _turn(st):
    """One turn of a server's cache; ``st["cache"]`` is the library's or the plain one."""
    case, c, n = st["case"], st["cache"], st["case"]["n"]
    if case["op"] == "fork":
        kids = list(range(n, n + n * case["children"]))
        c.free(kids)
        c.truncate(list(range(n)), st["lens"])
        c.fork([(s - n) // case["children"] for s in kids], kids)
        going = kids + list(range(n))
        starts, seqs = c.append(going, [1] * len(going))
    else:
        going = list(range(n, n + case["children"]))
        c.free(going)
        starts, seqs = c.append(going, _lengths(case, 1))
    for layer in range(case["layers"]):
        c.write(layer, st["newk"][layer], st["newv"][layer], starts, seqs)
    if case["op"] == "compact":
        c.free(going[::2])
        c.compact()
    return c.k, c.v, c.table, c.lens


# --------------------------------------------------------------------------- plain forms, 32 bits
def _attend(q, k, v, causal):
    """q (n, Hq, D), k, v (m, Hk, D): the last query stands at the last key.  Out in 32 bits and the log-sum-exp."""
    n, Hq, D = q.shape
    m, Hk, _ = k.shape
    out = torch.empty((n, Hq, D), dtype=torch.float32, device=q.device)
    lse = torch.empty((Hq, n), dtype=torch.float32, device=q.device)
    hidden = None
    if causal and n > 1:
        hidden = torch.arange(m, device=q.device)[None, :] > torch.arange(m - n, m, device=q.device)[:, None]
    probs = []
    for h in range(Hk):
        heads = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
        s = torch.matmul(q[:, heads].float().transpose(0, 1), k[:, h].float().T) * (1.0 / math.sqrt(D))
        if hidden is not None:
            s.masked_fill_(hidden, -math.inf)
        top = s.amax(-1, keepdim=True)
        p = torch.exp(s - top)
        total = p.sum(-1, keepdim=True)
        lse[heads] = (top + torch.log(total)).squeeze(-1)
        p = p / total
        out[:, heads] = torch.matmul(p, v[:, h].float()).transpose(0, 1)
        probs.append(p)
    return out, lse, probs


def _plain_packed(st):
    case, dt = st["case"], st["q"].dtype
    outs, lses, dqs, dks, dvs, at = [], [], [], [], [], 0
    g = case["Hq"] // case["Hk"]
    scale = 1.0 / math.sqrt(case["D"])
    for n in st["lens"]:
        q, k, v = (st[x][at: at + n] for x in ("q", "k", "v"))
        out, lse, probs = _attend(q, k, v, case["causal"])
        outs.append(out.to(dt))
        lses.append(lse)
        if case["grad"]:
            do = st["dout"][at: at + n].float()
            dq, dk, dv = torch.empty_like(out), torch.empty_like(k, dtype=torch.float32), torch.empty_like(v, dtype=torch.float32)
            for h, p in enumerate(probs):
                heads = slice(h * g, h * g + g)
                d = do[:, heads].transpose(0, 1)
                dv[:, h] = torch.matmul(p.transpose(-1, -2), d).sum(0)
                ds = torch.matmul(d, v[:, h].float().T)
                ds = p * (ds - (p * ds).sum(-1, keepdim=True))
                dq[:, heads] = (torch.matmul(ds, k[:, h].float()) * scale).transpose(0, 1)
                dk[:, h] = (torch.matmul(ds.transpose(-1, -2), q[:, heads].float().transpose(0, 1)) * scale).sum(0)
            dqs.append(dq.to(dt))
            dks.append(dk.to(dt))
            dvs.append(dv.to(dt))
        del probs
        at += n
    if case["grad"]:
        return torch.cat(outs), torch.cat(dqs), torch.cat(dks), torch.cat(dvs)
    return torch.cat(outs), torch.cat(lses, 1)


def _plain_paged(st):
    outs, lses, at = [], [], 0
    page = st["case"]["page"]
    for b, (n, x) in enumerate(zip(st["news"], st["lens"])):
        ids = st["table"][b, : -(-x // page)].long()
        k, v = (st[t][ids].flatten(0, 1)[:x] for t in ("k", "v"))
        out, lse, _ = _attend(st["q"][at: at + n], k, v, True)
        outs.append(out.to(st["q"].dtype))
        lses.append(lse)
        at += n
    return torch.cat(outs), torch.cat(lses, 1)


class _Pages:
    """The cache's pages by lists and tensor indexing: the lowest free page is taken first; a page that several
    sequences share is copied before one of them writes into it; rows behind a sequence's end keep what they hold."""

    def __init__(self, pages, page, seqs, width):
        self.page, self.width = page, width
        self.unused, self.refs = list(range(pages)), [0] * pages
        self.held, self.size = [[] for _ in range(seqs)], [0] * seqs
        self.table = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.k = self.v = None

    def _take(self):
        p = heapq.heappop(self.unused)
        self.refs[p] = 1
        return p

    def _drop(self, p):
        self.refs[p] -= 1
        if not self.refs[p]:
            heapq.heappush(self.unused, p)

    def _tell(self, seqs):
        rows = torch.tensor([self.held[s] + [-1] * (self.width - len(self.held[s])) for s in seqs], dtype=torch.int32)
        at = torch.tensor(seqs, device="cuda")
        self.table[at] = rows.cuda()
        self.lens[at] = torch.tensor([self.size[s] for s in seqs], dtype=torch.int32).cuda()

    def _copy(self, moves):
        for src, dst, rows in moves:
            for pool in (self.k, self.v):
                pool[:, dst, :rows] = pool[:, src, :rows]

    def append(self, seqs, counts):
        moves = []
        for s, n in zip(seqs, counts):
            last = self.size[s] % self.page
            if n and last and self.refs[self.held[s][-1]] > 1:
                src, dst = self.held[s][-1], self._take()
                self._drop(src)
                self.held[s][-1] = dst
                moves.append((src, dst, last))
            self.size[s] += n
            while len(self.held[s]) * self.page < self.size[s]:
                self.held[s].append(self._take())
        self._copy(moves)
        self._tell(seqs)
        return [sum(counts[:i]) for i in range(len(counts) + 1)], seqs

    def fork(self, parents, children):
        for a, b in zip(parents, children):
            self.held[b], self.size[b] = list(self.held[a]), self.size[a]
            for p in self.held[b]:
                self.refs[p] += 1
        self._tell(children)

    def truncate(self, seqs, lens):
        for s, n in zip(seqs, lens):
            keep = -(-n // self.page)
            for p in self.held[s][keep:]:
                self._drop(p)
            del self.held[s][keep:]
            self.size[s] = n
        self._tell(seqs)

    def free(self, seqs):
        self.truncate(seqs, [0] * len(seqs))

    def write(self, layer, k, v, starts, seqs):
        at, slot = [], []
        for b, s in enumerate(seqs):
            for i in range(self.size[s] - (starts[b + 1] - starts[b]), self.size[s]):
                at.append(self.held[s][i // self.page])
                slot.append(i % self.page)
        at, slot = torch.tensor(at).cuda(), torch.tensor(slot).cuda()
        self.k[layer].index_put_((at, slot), k)
        self.v[layer].index_put_((at, slot), v)

    def compact(self):
        live = sum(1 for r in self.refs if r)
        holes = [p for p in range(live) if not self.refs[p]]
        far = [p for p in range(live, len(self.refs)) if self.refs[p]]
        to, fill = dict(zip(far, holes)), {}
        for s, pages in enumerate(self.held):
            for i, p in enumerate(pages):
                if p in to:
                    fill[p] = max(fill.get(p, 0), min(self.page, self.size[s] - i * self.page))
                    pages[i] = to[p]
        self._copy([(p, to[p], fill[p]) for p in far])
        for p in far:
            self.refs[to[p]], self.refs[p] = self.refs[p], 0
        self.unused = [p for p, r in enumerate(self.refs) if not r]
        self._tell(list(range(len(self.held))))


def run(st):
    if own:
        return _run_own(st)
    with torch.no_grad():
        if st["case"]["op"] == "packed":
            return _plain_packed(st)
        return _plain_paged(st) if st["case"]["op"] == "paged" else _turn(st)


# --------------------------------------------------------------------------- definitions, 64 bits
def _exact_rows(q, k, v, causal, out, lse):
    """One query head over one key head, in blocks of rows; returns nothing, writes out (n, D) and lse (n,)."""
    n, m = q.shape[0], k.shape[0]
    step = max(1, (1 << 27) // max(1, m))
    k, v = k.double(), v.double()
    for i in range(0, n, step):
        e = min(n, i + step)
        seen = m - n + e if causal else m
        s = (q[i:e].double() @ k[:seen].T) / math.sqrt(q.shape[1])
        if causal:
            s += torch.triu(torch.full_like(s, -math.inf), diagonal=m - n + i + 1)
        lse[i:e] = torch.logsumexp(s, -1)
        out[i:e] = torch.softmax(s, -1) @ v[:seen]


def _exact_grads(q, k, v, do, causal, dq, dk, dv):
    """Adds to dk, dv and writes dq: the softmax's Jacobian applied to dA = dO V^T, in blocks of rows."""
    n, m, scale = q.shape[0], k.shape[0], q.shape[1] ** -0.5
    step = max(1, (1 << 26) // max(1, m))
    k, v = k.double(), v.double()
    for i in range(0, n, step):
        e = min(n, i + step)
        seen = m - n + e if causal else m
        x, d = q[i:e].double(), do[i:e].double()
        s = scale * (x @ k[:seen].T)
        if causal:
            s += torch.triu(torch.full_like(s, -math.inf), diagonal=m - n + i + 1)
        a = torch.softmax(s, -1)
        da = d @ v[:seen].T
        ds = a * da - a * torch.einsum("ij,ij->i", a, da)[:, None]
        dq[i:e] = scale * (ds @ k[:seen])
        dk[:seen] += scale * (ds.T @ x)
        dv[:seen] += a.T @ d


def _exact_packed(st):
    case = st["case"]
    f = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros(st["q"].shape, **f), torch.zeros((case["Hq"], st["q"].shape[0]), **f)
    dq, dk, dv = (torch.zeros(st[x].shape, **f) for x in ("q", "k", "v"))
    at = 0
    for n in st["lens"]:
        rows = slice(at, at + n)
        for h in range(case["Hq"]):
            j = h * case["Hk"] // case["Hq"]
            args = st["q"][rows, h], st["k"][rows, j], st["v"][rows, j]
            _exact_rows(*args, case["causal"], out[rows, h], lse[h, rows])
            if case["grad"]:
                _exact_grads(*args, st["dout"][rows, h], case["causal"], dq[rows, h], dk[rows, j], dv[rows, j])
        at += n
    return [out, dq, dk, dv] if case["grad"] else [out, lse]


def _exact_paged(st):
    case, page = st["case"], st["case"]["page"]
    f = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros(st["q"].shape, **f), torch.zeros((case["Hq"], st["q"].shape[0]), **f)
    at = 0
    for b, (n, x) in enumerate(zip(st["news"], st["lens"])):
        where = torch.arange(x, device="cuda")
        ids, slot = st["table"][b][where // page].long(), where % page
        for j in range(case["Hk"]):
            k, v = st["k"][ids, slot, j], st["v"][ids, slot, j]
            for h in range(j * case["Hq"] // case["Hk"], (j + 1) * case["Hq"] // case["Hk"]):
                _exact_rows(st["q"][at: at + n, h], k, v, True, out[at: at + n, h], lse[h, at: at + n])
        at += n
    return [out, lse]


def _layout(case):
    """Pages of the sequences that stay (one behind the other), and how many they are."""
    at, pages = 0, []
    for x in _lengths(case):
        n = -(-x // case["page"])
        pages.append(list(range(at, at + n)))
        at += n
    return pages, at


def _compacted(case):
    """Pages of the sequences that came, before half of them left, and the moves (from, to, rows) that follow."""
    _, at = _layout(case)
    came, lens, page = [], _lengths(case, 1), case["page"]
    for x in lens:
        n = -(-x // page)
        came.append(list(range(at, at + n)))
        at += n
    left = sorted(p for pages in came[::2] for p in pages)
    stay = [(p, min(page, lens[s] - i * page)) for s in range(1, len(came), 2) for i, p in enumerate(came[s])]
    live = at - len(left)
    holes = [p for p in left if p < live]
    return came, [(p, to, rows) for (p, rows), to in zip([x for x in stay if x[0] >= live], holes)]


def _exact_pages(st, st0):
    """The state after a turn, put together page by page from the state before it (``st0``: its pools)."""
    case, page, lens, n = st["case"], st["case"]["page"], st["lens"], st["case"]["n"]
    k, v = st0
    table = torch.full(tuple(st["cache"].table.shape), -1, dtype=torch.int32)
    held, base = _layout(case)
    size = list(lens)
    if case["op"] == "fork":
        kids, at, i = n * case["children"], base, 0
        rows = [list(held[s // case["children"]]) for s in range(kids)]
        for s in range(kids):
            x = lens[s // case["children"]]
            if x % page:  # the last page is shared with the parent
                for pool in (k, v):
                    pool[:, at, : x % page] = pool[:, rows[s][-1], : x % page]
                rows[s][-1] = at
            else:
                rows[s].append(at)
            at += 1
        for s in range(n):
            if not lens[s] % page:
                held[s] = held[s] + [at]
                at += 1
        for i, (pages, x) in enumerate([(rows[s], lens[s // case["children"]]) for s in range(kids)] + list(zip(held, lens))):
            for pool, new in ((k, st["newk"]), (v, st["newv"])):
                pool[:, pages[x // page], x % page] = new[:, i].double()
        size = [x + 1 for x in lens] + [lens[s // case["children"]] + 1 for s in range(kids)]
        held = held + rows
    else:
        came, moves = _compacted(case)
        at = 0
        for pages, x in zip(came, _lengths(case, 1)):
            for i, p in enumerate(pages):
                r = min(page, x - i * page)
                for pool, new in ((k, st["newk"]), (v, st["newv"])):
                    pool[:, p, :r] = new[:, at: at + r].double()
                at += r
        for p, to, r in moves:
            for pool in (k, v):
                pool[:, to, :r] = pool[:, p, :r]
        moved = {p: to for p, to, _ in moves}
        for s, (pages, x) in enumerate(zip(came, _lengths(case, 1))):
            held.append([] if s % 2 == 0 else [moved.get(p, p) for p in pages])
            size.append(0 if s % 2 == 0 else x)
    for s, pages in enumerate(held):
        table[s, : len(pages)] = torch.tensor(pages, dtype=torch.int32)
    return [k, v, table, torch.tensor(size, dtype=torch.int32)]


def exact(case, seed):
    st = _prepare(case, seed, False)
    with torch.no_grad():
        if case["op"] in ("fork", "compact"):
            return _exact_pages(st, (st["cache"].k.double(), st["cache"].v.double()))
        return _exact_packed(st) if case["op"] == "packed" else _exact_paged(st)
