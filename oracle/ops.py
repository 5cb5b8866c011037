"""float64 definitions of the operators around attention: rotary positions, 8-bit activation
checkpoints and differential attention, with the error each result may carry.

Plain NumPy, no code shared with the library.  The error bounds count the roundings that the
kernels make: a value rounded to bf16 is off by at most 2^-8 of itself (``BF16``), an exponential of the
special-function unit by 2^-22 (``EXP``), to which the error of its argument comes; 32-bit sums and
products are covered by ``F32`` times the sum of the terms' magnitudes, a sum over all keys by ``norm_error``.
"""
import numpy as np

BF16 = 2.0 ** -8
EXP = 2.0 ** -22
F32 = 2.0 ** -20


# --------------------------------------------------------------------------- rotary positions
def rotary_rates(widths, base=10000.0, scaling="none", factor=1.0, original=8192, alpha=1.0, beta=32.0):
    """Radians per position of every pair, and the axis it follows."""
    rates, axis = [], []
    for a, w in enumerate(widths):
        for j in range(w // 2):
            b = base * factor ** (w / (w - 2.0)) if scaling == "ntk" and w > 2 else base
            f = b ** (-2.0 * j / w)
            if scaling == "linear":
                f /= factor
            elif scaling == "parts":
                keep = min(1.0, max(0.0, (original * f / (2 * np.pi) - alpha) / (beta - alpha)))
                f = keep * f + (1 - keep) * f / factor
            rates.append(f)
            axis.append(a)
    return np.array(rates), np.array(axis, dtype=int)


def rotary(x, positions, rates, axis, layout, magnitude=1.0, inverse=False):
    """x (B, S, H, D), positions (B, S, axes): returns the rotated x and the magnitude of each result's terms."""
    R = 2 * len(rates)
    angle = (positions[..., axis].astype(np.float64) * rates)[:, :, None, :]
    c, s = magnitude * np.cos(angle), magnitude * np.sin(angle) * (-1.0 if inverse else 1.0)
    lo, hi = (np.arange(R // 2), np.arange(R // 2) + R // 2) if layout == "half" else (np.arange(0, R, 2),
                                                                                      np.arange(1, R, 2))
    y, size = x.astype(np.float64).copy(), np.zeros(x.shape)
    y[..., lo], y[..., hi] = x[..., lo] * c - x[..., hi] * s, x[..., lo] * s + x[..., hi] * c
    size[..., lo] = size[..., hi] = magnitude * (np.abs(x[..., lo]) + np.abs(x[..., hi]))
    return y, size


# --------------------------------------------------------------------------- 8-bit checkpoints
def act8_codes(x):
    """Codes (whole numbers) of finite rows x (..., D), ties to even."""
    x = x.astype(np.float64)
    top = np.abs(x).max(-1, keepdims=True)
    codes = np.rint(127.0 * x / np.where(top > 0, top, 1.0))
    return np.where(top < 2.0 ** -119, 0.0, codes) + 0.0, top[..., 0]  # a code is an integer: no -0


# --------------------------------------------------------------------------- differential attention
def norm_error(Sk):
    """Relative error of a softmax's sum of Sk probabilities in 32 bits, beside that of the probabilities.

    In steps of 2^-24.  Tiles of 80 or 128 keys: 64 additions within one at most, then a product, an addition and an
    exponential (2^-22: four steps) to join it to the others: 64 + 6 (Sk / 80 + 1).  The few-row kernel adds every 16th key
    and joins after 6 of them at least, with a product and an exponential: Sk / 16 + 5 Sk / 96; then groups of lanes, warps
    and blocks, 16 + 3 additions and three times those five."""
    return (96 + Sk / 8.0) * 2.0 ** -24


def _maps(q, k, mask, scale):
    """Softmax maps and LSE of one batch element: q (Sq, H, D), k (Sk, H, D) -> (2, H, Sq, Sk), (2, H, Sq)."""
    w = q.shape[-1] // 2
    a, lse = [], []
    for m in range(2):
        s = scale * np.einsum("ihd,jhd->hij", q[..., m * w:m * w + w], k[..., m * w:m * w + w])
        if mask is not None:
            s = np.where(mask[None, None, :], s, -np.inf)
        top = s.max(-1, keepdims=True)
        e = np.exp(s - np.where(np.isinf(top), 0.0, top))
        total = e.sum(-1, keepdims=True)
        a.append(e / np.where(total > 0, total, 1.0))
        with np.errstate(divide="ignore"):
            lse.append((np.where(np.isinf(top), 0.0, top) + np.log(total))[..., 0])
    return np.stack(a), np.stack(lse)


def diff_attn(q, k, v, lam, mask=None, scale=None, dout=None):
    """Outputs and, with ``dout``, gradients; each as ``name: (value, error bound)``."""
    B, Sq, H, D = q.shape
    Sk, w = k.shape[1], D // 2
    scale = w ** -0.5 if scale is None else scale
    norm = norm_error(Sk)
    names = ["out", "out2", "lse"] + ([] if dout is None else ["dq", "dk", "dv", "dlam"])
    shapes = {"out": q.shape, "out2": q.shape, "lse": (B, H, 2, Sq), "dq": q.shape, "dk": k.shape, "dv": k.shape,
              "dlam": (H,)}
    res = {n: (np.zeros(shapes[n]), np.zeros(shapes[n])) for n in names}

    def put(n, at, value, bound):
        res[n][0][at], res[n][1][at] = value, bound

    L = lam[:, None, None]
    for b in range(B):
        a, lse = _maps(q[b], k[b], None if mask is None else mask[b], scale)
        vb = v[b]
        both = a[0] + np.abs(L) * a[1]
        o = np.einsum("hij,jhd->ihd", a[0] - L * a[1], vb)
        o2 = np.einsum("hij,jhd->ihd", a[1], vb)
        size = np.einsum("hij,jhd->ihd", both, np.abs(vb))
        size2 = np.einsum("hij,jhd->ihd", a[1], np.abs(vb))
        # 32-bit scores: their terms' magnitudes
        es = F32 * scale * np.stack([np.einsum("ihd,jhd->hij", np.abs(q[b][..., m * w:m * w + w]),
                                               np.abs(k[b][..., m * w:m * w + w])).max(-1) for m in range(2)])
        # a probability that a matrix product reads, and the sum that it is divided by
        P = (BF16 + 2 * (EXP + es.max(0)) + norm).T[..., None]
        eo, eo2 = (P + F32) * size + BF16 * np.abs(o), (P + F32) * size2 + BF16 * np.abs(o2)
        put("out", b, o, eo)
        put("out2", b, o2, eo2)
        elog = es + EXP + norm + F32 * np.where(np.isinf(lse), 0, np.abs(lse))
        put("lse", b, np.moveaxis(lse, 0, 1), np.moveaxis(elog, 0, 1))
        if dout is None:
            continue
        g = dout[b]
        da = np.einsum("ihd,jhd->hij", g, vb)
        eda = F32 * np.einsum("ihd,jhd->hij", np.abs(g), np.abs(vb))
        rows = np.einsum("mhij,hij->mhi", a, da)
        erow2 = np.einsum("ihd,ihd->hi", np.abs(g), eo2) + F32 * np.einsum("ihd,ihd->hi", np.abs(g), np.abs(o2))
        erow1 = (np.einsum("ihd,ihd->hi", np.abs(g), eo) + F32 * np.einsum("ihd,ihd->hi", np.abs(g), np.abs(o))
                 + np.abs(lam)[:, None] * erow2)
        weight = np.stack([np.ones_like(L), -L])
        ds = weight * a * (da - rows[..., None])
        # a probability formed again from the LSE: its score, the LSE and the exponential
        ea = (es + elog + EXP)[..., None]
        # an entry of dS: its probability, its rounding to bf16, and the row dots' error
        eds = (np.abs(ds) * (BF16 + ea + F32)
               + np.abs(weight) * a * (eda + np.stack([erow1, erow2])[..., None]))
        pv = a[0] - L * a[1]
        # each map's probability is rounded to bf16 by itself: |A1 2^-8| + |lambda A2 2^-8|
        epv = both * (BF16 + F32 + ea.max(0))
        dv = np.einsum("hij,ihd->jhd", pv, g)
        edv = np.einsum("hij,ihd->jhd", epv + F32 * np.abs(pv), np.abs(g))
        put("dv", b, dv, edv + BF16 * np.abs(dv))
        for m in range(2):
            c = slice(m * w, m * w + w)
            e = eds[m] + F32 * np.abs(ds[m])
            dq = scale * np.einsum("hij,jhd->ihd", ds[m], k[b][..., c])
            dk = scale * np.einsum("hij,ihd->jhd", ds[m], q[b][..., c])
            put("dq", (b, slice(None), slice(None), c), dq,
                scale * np.einsum("hij,jhd->ihd", e, np.abs(k[b][..., c])) + BF16 * np.abs(dq))
            put("dk", (b, slice(None), slice(None), c), dk,
                scale * np.einsum("hij,ihd->jhd", e, np.abs(q[b][..., c])) + BF16 * np.abs(dk))
        res["dlam"][0][:] -= rows[1].sum(-1)
        # Delta_2 of the rounded O_2, and what sum_j A_2 (dA - Delta_2) of 32 bits says is missing from it: with A_2 and dA
        # as they are computed, sum_j A_2 dA + (1 - sum_j A_2) Delta_2.  Where lambda is too small for dS_2, Delta_2 alone.
        size_da = np.einsum("hij,hij->hi", a[1], np.abs(da))
        near = ea[1, ..., 0] * (2 * size_da + erow2) + np.einsum("hij,hij->hi", a[1], eda)
        # added up in 32 bits: a key's rows one after the other, then tiles, keys and rows in parts of at most 64
        near = near + (Sq + 256) * 2.0 ** -24 * 2 * size_da
        erow = np.where(np.abs(lam)[:, None] >= 2.0 ** -60, near, erow2 + F32 * np.abs(rows[1]))
        res["dlam"][1][:] += erow.sum(-1)
    if dout is not None:
        res["dlam"][1][:] += BF16 * np.abs(res["dlam"][0])  # lambda in bf16
    return res
