"""float64 definitions of attention over sequences of their own lengths and of a cache's pages, with the error that
each result may carry.

Plain NumPy, no code shared with the library.  A value rounded to bf16 is off by at most 2^-8 of itself, to fp16 by
2^-11 or, where it is small, by 2^-25; an exponential of the special-function unit by 2^-22, one of the FMA pipe by 2^-20
(``EXP`` covers both); 32-bit sums by ``F32`` times the sum of the terms' magnitudes.
"""
import numpy as np

ROUND = {"bfloat16": (2.0 ** -8, 0.0), "float16": (2.0 ** -11, 2.0 ** -25)}
EXP = 2.0 ** -20
F32 = 2.0 ** -20


def norm_error(m):
    """Relative error of a 32-bit sum of m probabilities, beside that of the probabilities: 128 of a tile in turn, then a
    product, an addition and an exponential (2^-22) a tile; parts of a split sequence are joined by as many again."""
    return (128 + 12 * (m / 128.0 + 2)) * 2.0 ** -24


def attention(q, k, v, causal, scale=None, dout=None, dtype="bfloat16"):
    """One sequence: q (n, Hq, D), k, v (m, Hk, D), the last query at the last key.  Returns name -> (value, bound)."""
    n, Hq, D = q.shape
    m, Hk, _ = k.shape
    g = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    rel, small = ROUND[dtype]
    res = {"out": (np.zeros(q.shape), np.zeros(q.shape)), "lse": (np.full((Hq, n), -np.inf), np.zeros((Hq, n)))}
    if dout is not None:
        res.update({x: (np.zeros(t.shape), np.zeros(t.shape)) for x, t in (("dq", q), ("dk", k), ("dv", v))})
    if n == 0 or m == 0:
        return res
    norm = norm_error(m)
    seen = np.arange(m)[None, :] <= np.arange(m - n, m)[:, None] if causal else np.ones((n, m), bool)
    for h in range(Hq):
        j = h // g
        x, kk, vv = q[:, h], k[:, j], v[:, j]
        s = np.where(seen, scale * (x @ kk.T), -np.inf)
        top = s.max(1, keepdims=True)
        e = np.exp(s - np.where(np.isinf(top), 0.0, top))
        total = e.sum(1, keepdims=True)
        p = e / np.where(total > 0, total, 1.0)
        some = total[:, 0] > 0
        lse = np.full(n, -np.inf)
        lse[some] = top[some, 0] + np.log(total[some, 0])
        es = F32 * scale * np.where(seen, np.abs(x) @ np.abs(kk).T, 0).max(1)  # error of a row's scores
        P = (rel + 2 * (EXP + es) + norm + F32)[:, None]
        o, size = p @ vv, p @ np.abs(vv)
        # the smallest probabilities of fp16: 2^-25 of the row's largest each
        eo = P * size + small * np.where(seen, 1.0, 0.0) @ np.abs(vv)
        res["out"][0][:, h], res["out"][1][:, h] = o, eo + rel * np.abs(o) + small
        elog = es + EXP + norm + F32 * np.where(some, np.abs(np.where(some, lse, 0)), 0)
        res["lse"][0][h], res["lse"][1][h] = lse, elog
        if dout is None:
            continue
        d = dout[:, h]
        da = d @ vv.T
        eda = F32 * (np.abs(d) @ np.abs(vv).T)
        rows = (p * da).sum(1, keepdims=True)
        erow = (np.abs(d) * (eo + rel * np.abs(o))).sum(1, keepdims=True) + F32 * (np.abs(d) * np.abs(o)).sum(1, keepdims=True)
        ds = p * (da - rows)
        ea = (es + elog + EXP)[:, None]
        eds = np.abs(ds) * (rel + ea + F32) + p * (eda + erow)
        dq, dk, dv = scale * ds @ kk, scale * ds.T @ x, p.T @ d
        res["dq"][0][:, h] = dq
        res["dq"][1][:, h] = scale * (eds + F32 * np.abs(ds)) @ np.abs(kk) + rel * np.abs(dq)
        # summed over the heads that share the key head; rounded once, at the end
        res["dk"][0][:, j] += dk
        res["dk"][1][:, j] += scale * (eds + F32 * np.abs(ds)).T @ np.abs(x)
        res["dv"][0][:, j] += dv
        res["dv"][1][:, j] += (p * (rel + ea + 2 * F32)).T @ np.abs(d)
    if dout is not None:
        for x in ("dk", "dv"):
            res[x][1][:] += rel * np.abs(res[x][0])
    return res


def packed(q, k, v, starts, starts_k=None, causal=True, scale=None, dout=None, dtype="bfloat16"):
    """Sequences packed one behind the other; tokens of none: 0, lse 0, with an infinite bound."""
    starts_k = starts if starts_k is None else starts_k
    out = {"out": q.shape, "lse": (q.shape[1], q.shape[0])}
    if dout is not None:
        out.update({"dq": q.shape, "dk": k.shape, "dv": v.shape})
    res = {x: (np.zeros(s), np.full(s, np.inf)) for x, s in out.items()}
    for b in range(len(starts) - 1):
        a, c = slice(starts[b], starts[b + 1]), slice(starts_k[b], starts_k[b + 1])
        one = attention(q[a], k[c], v[c], causal, scale, None if dout is None else dout[a], dtype)
        for x in out:
            at = (slice(None), a) if x == "lse" else c if x in ("dk", "dv") else a
            for i in range(2):
                res[x][i][at] = one[x][i]
    return res


def paged(q, k_pages, v_pages, starts, table, lens, seqs=None, causal=True, scale=None, dtype="bfloat16"):
    """New tokens over the pages of a cache."""
    page = k_pages.shape[1]
    res = {"out": (np.zeros(q.shape), np.full(q.shape, np.inf)),
           "lse": (np.zeros((q.shape[1], q.shape[0])), np.full((q.shape[1], q.shape[0]), np.inf))}
    for b in range(len(starts) - 1):
        r = b if seqs is None else seqs[b]
        ids = table[r, : -(-lens[r] // page)]
        k, v = (x[ids].reshape(-1, *x.shape[2:])[: lens[r]] for x in (k_pages, v_pages))
        a = slice(starts[b], starts[b + 1])
        one = attention(q[a], k, v, causal, scale, None, dtype)
        for i in range(2):
            res["out"][i][a], res["lse"][i][:, a] = one["out"][i], one["lse"][i]
    return res


class Pages:
    """A cache's pages by sets: the lowest free page first, a shared page copied before it is written into."""

    def __init__(self, pages, page, seqs):
        self.pages, self.page = pages, page
        self.held, self.size = {s: [] for s in range(seqs)}, {s: 0 for s in range(seqs)}
        self.moves = []

    def _used(self):
        return {p for row in self.held.values() for p in row}

    def _take(self):
        return min(set(range(self.pages)) - self._used())

    def append(self, seqs, counts):
        self.moves = []
        for s, n in zip(seqs, counts):
            row, last = self.held[s], self.size[s] % self.page
            if n and last and sum(r.count(row[-1]) for r in self.held.values()) > 1:
                p = self._take()
                self.moves.append((row[-1], p, last))
                row[-1] = p
            self.size[s] += n
            while len(row) * self.page < self.size[s]:
                row.append(self._take())

    def fork(self, parents, children):
        for a, b in zip(parents, children):
            self.held[b], self.size[b] = list(self.held[a]), self.size[a]

    def truncate(self, seqs, lens):
        for s, n in zip(seqs, lens):
            self.size[s] = n
            self.held[s] = self.held[s][: -(-n // self.page)]

    def compact(self):
        used = sorted(self._used())
        holes = sorted(set(range(len(used))) - set(used))
        to = dict(zip([p for p in used if p >= len(used)], holes))
        self.moves = [(p, q, max(min(self.page, self.size[s] - i * self.page) for s, row in self.held.items()
                                 for i, x in enumerate(row) if x == p)) for p, q in to.items()]
        self.held = {s: [to.get(p, p) for p in row] for s, row in self.held.items()}
