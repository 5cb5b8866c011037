"""What is measured of the operators around attention: rotary positions, 8-bit activation
checkpoints and differential attention.

Each case is one pass as a program makes it; ``run`` computes it in elementary torch operations
(``own = False``) or through the library's calls (``own = True``), ``exact`` from the definition in
64 bits.
"""
import math

import torch

own = False

BF16, FP32 = "bfloat16", "float32"


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # One denoising step of a cached-context sampler: one new position per sequence, far along, with
        # frequencies interpolated by parts for an eight times longer context.  Latency counts.
        {"name": "rotary_token", "op": "rotary", "B": 16, "S": 1, "Hq": 24, "Hk": 24, "D": 128, "rot": 128,
         "layout": "half", "axes": 1, "scaling": "parts", "factor": 8.0, "far": 200000, "dtype": BF16, "grad": False},
        # Q and K of the long video sequence, rotated by frame, row and column, with the gradients.
        {"name": "rotary_video", "op": "rotary", "B": 1, "S": 27280, "Hq": 40, "Hk": 40, "D": 128, "rot": 128,
         "layout": "interleaved", "axes": 3, "scaling": "none", "factor": 1.0, "far": 0, "dtype": BF16, "grad": True},
        # Part of the head only, fewer key heads than query heads, an odd length, 32-bit tensors.
        {"name": "rotary_part", "op": "rotary", "B": 3, "S": 1537, "Hq": 24, "Hk": 8, "D": 64, "rot": 40,
         "layout": "half", "axes": 1, "scaling": "ntk", "factor": 4.0, "far": 0, "dtype": FP32, "grad": True},
        # Q and K of the image workload, put away in 8 bits and taken back.
        {"name": "act8_image", "op": "act8", "n": 2, "B": 2, "S": 1024, "H": 24, "D": 64, "dtype": BF16},
        # The four tensors that the attention of a long video sequence keeps for its backward pass.
        {"name": "act8_video", "op": "act8", "n": 4, "B": 1, "S": 27280, "H": 40, "D": 128, "dtype": BF16},
        # An attention training step whose Q, K, V and O wait for the backward pass in 8 bits.
        {"name": "act8_step_image", "op": "step8", "B": 2, "S": 1024, "H": 24, "D": 64, "mask": "none"},
        {"name": "act8_step_mask", "op": "step8", "B": 2, "S": 4096, "H": 24, "D": 128, "mask": "prefix"},
        # Differential attention: one query per sequence against a long context.
        {"name": "diff_token", "op": "diff", "B": 4, "Sq": 1, "Sk": 16389, "H": 24, "D": 128, "mask": "none",
         "grad": False},
        # Image tokens reading a short, padded text: few keys, many queries.
        {"name": "diff_text", "op": "diff", "B": 2, "Sq": 4096, "Sk": 777, "H": 24, "D": 128, "mask": "prefix",
         "grad": False},
        # Training steps: the image workload, the padded batch, and a long ragged sequence.
        {"name": "diff_step_image", "op": "diff", "B": 2, "Sq": 1024, "Sk": 1024, "H": 24, "D": 64, "mask": "none",
         "grad": True},
        {"name": "diff_step_mask", "op": "diff", "B": 2, "Sq": 4096, "Sk": 4096, "H": 24, "D": 128, "mask": "prefix",
         "grad": True},
        {"name": "diff_step_long", "op": "diff", "B": 1, "Sq": 8191, "Sk": 8191, "H": 24, "D": 128, "mask": "none",
         "grad": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rotary", "act8", "step8", "diff", "diff", "diff"))
    D = rng.choice((64, 128))
    if op == "rotary":
        B, axes = _log_int(rng, 1, 16), rng.choice((1, 1, 3))
        Hq = rng.choice((8, 16, 24, 40))
        rot = D if rng.random() < 0.5 else 2 * rng.randint(axes, D // 2)
        S = _log_int(rng, 1, max(1, min(27280, 27280 * 40 * 64 // (B * Hq * D))))
        return {"op": op, "B": B, "S": S, "Hq": Hq, "Hk": rng.choice((Hq, Hq, 8)), "D": D, "rot": rot,
                "layout": rng.choice(("half", "interleaved")), "axes": axes,
                "scaling": rng.choice(("none", "linear", "ntk", "parts")) if axes == 1 else "none",
                "factor": rng.choice((2.0, 4.0, 8.0)), "far": 0 if axes > 1 else rng.choice((0, 30000, 200000)),
                "dtype": rng.choice((BF16, BF16, FP32)), "grad": rng.random() < 0.6}
    if op == "act8":
        B, H = _log_int(rng, 1, 8), rng.choice((8, 16, 24, 40))
        return {"op": op, "n": rng.randint(1, 4), "B": B, "S": _log_int(rng, 1, 27280 * 40 // (B * H)), "H": H,
                "D": rng.choice((64, 80, 128)), "dtype": rng.choice((BF16, BF16, FP32))}
    B, H = _log_int(rng, 1, 4), rng.choice((4, 8, 16, 24))
    most = int(math.sqrt(24 * 5000 * 5000 / (B * H)))  # query x key pairs: below the largest listed case
    mask = rng.choice(("none", "prefix", "random", "empty") if B > 1 else ("none", "prefix", "random"))
    if op == "step8":
        return {"op": op, "B": B, "S": _log_int(rng, 16, min(most, 8191)), "H": H, "D": D, "mask": mask}
    if rng.random() < 0.35:
        return {"op": op, "B": B, "Sq": rng.randint(1, 4), "Sk": _log_int(rng, 1, 16389), "H": H, "D": D, "mask": mask,
                "grad": False}
    Sq = _log_int(rng, 16, min(most, 8191))
    Sk = Sq if rng.random() < 0.5 else _log_int(rng, 16, min(most, 8191))
    return {"op": op, "B": B, "Sq": Sq, "Sk": Sk, "H": H, "D": D, "mask": mask, "grad": rng.random() < 0.7}


def work(case):
    op = case["op"]
    if op == "rotary":
        size = 2 if case["dtype"] == BF16 else 4
        n = case["B"] * case["S"] * (case["Hq"] + case["Hk"])
        ways = 2 if case["grad"] else 1
        return {"bytes": ways * (2 * n * case["D"] * size + 4 * case["B"] * case["S"] * case["axes"]),
                "flops": ways * 3 * n * case["rot"]}
    if op == "act8":
        n = case["n"] * case["B"] * case["S"] * case["H"]
        size = 2 if case["dtype"] == BF16 else 4
        return {"bytes": 2 * n * (case["D"] * (size + 1) + 4), "flops": 4 * n * case["D"]}
    B, H, D = case["B"], case["H"], case["D"]
    Sq, Sk = (case["S"], case["S"]) if op == "step8" else (case["Sq"], case["Sk"])
    train = op == "step8" or case["grad"]
    q, k = 2 * B * Sq * H * D, 2 * B * Sk * H * D
    return {"bytes": 2 * q + 2 * k + (2 * q + 2 * k if train else 0),  # q, o, k, v; dout, dq, dk, dv
            "flops": (14 if train else 4) * B * H * Sq * Sk * D}


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _mask(g, case, B, Sk):
    kind = case["mask"]
    if kind == "none":
        return None
    at = torch.arange(Sk, device="cuda")
    if kind == "random":
        return (torch.rand((B, Sk), generator=g, device="cuda") < 0.6) | (at == 0)
    lens = torch.randint(max(1, Sk // 2), Sk + 1, (B,), generator=g, device="cuda")
    if kind == "empty":
        lens[0] = 0  # a sequence without an attended key
    return at[None, :] < lens[:, None]


def _axis_widths(case):
    """Rotated columns of each position axis: equal shares, what is left over to the first."""
    rot, axes = case["rot"], case["axes"]
    share = 2 * (rot // (2 * axes))
    return [rot - share * (axes - 1)] + [share] * (axes - 1)


# by-parts interpolation: the original context length and the limits, in turns over it
PARTS = {"original": 8192, "alpha": 1.0, "beta": 32.0}


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "rotary":
        dt = getattr(torch, case["dtype"])
        B, S, D, A = case["B"], case["S"], case["D"], case["axes"]
        st = {"case": case, "q": _normal(g, B, S, case["Hq"], D, dtype=dt), "k": _normal(g, B, S, case["Hk"], D, dtype=dt)}
        if case["grad"]:
            st["dq"], st["dk"] = (_normal(g, B, S, h, D, dtype=dt) for h in (case["Hq"], case["Hk"]))
        if A == 1:
            start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda")
            st["positions"] = (start + torch.arange(S, device="cuda")).to(torch.int32)
        else:  # frame, row and column of a video whose frames are 62 by 40 tokens
            at = torch.arange(S, device="cuda") + torch.randint(0, 16, (B, 1), generator=g, device="cuda") * 2480
            st["positions"] = torch.stack((at // 2480, at // 40 % 62, at % 40), -1).to(torch.int32)
        st["plan"] = _plan(case) if own else None
        return st
    if op == "act8":
        dt = getattr(torch, case["dtype"])
        shape = (case["B"], case["S"], case["H"], case["D"])
        # activations with a spread of magnitudes between channels
        spread = torch.exp(0.5 * torch.randn(case["D"], generator=g, device="cuda"))
        return {"case": case, "x": [(torch.randn(shape, generator=g, device="cuda") * spread).to(dt) for _ in range(case["n"])]}
    B, H, D = case["B"], case["H"], case["D"]
    Sq, Sk = (case["S"], case["S"]) if op == "step8" else (case["Sq"], case["Sk"])
    st = {"case": case, "q": _normal(g, B, Sq, H, D), "k": _normal(g, B, Sk, H, D), "v": _normal(g, B, Sk, H, D),
          "dout": _normal(g, B, Sq, H, D), "mask": _mask(g, case, B, Sk)}
    if op == "step8":
        for n in ("q", "k", "v"):
            st[n].requires_grad_()
    else:
        st["lam"] = (0.2 + 0.6 * torch.rand(H, generator=g, device="cuda")).to(torch.bfloat16)
    return st


# --------------------------------------------------------------------------- the library's calls
def _plan(case):
    import ulysses_dit_attention_gb300 as uaa

    return uaa.RotaryPlan(_axis_widths(case), layout=case["layout"], base=10000.0, scaling=case["scaling"],
                          factor=case["factor"], **PARTS)


def _run_own(st):
    import ulysses_dit_attention_gb300 as uaa

    case = st["case"]
    op = case["op"]
    if op == "rotary":
        out = uaa.rotary_fwd(st["q"], st["k"], st["plan"], st["positions"])
        if case["grad"]:
            out = out + uaa.rotary_bwd(st["dq"], st["dk"], st["plan"], st["positions"])
        return out
    if op == "act8":
        return uaa.act8_unpack(uaa.act8_pack(st["x"]))
    if op == "step8":
        out, _ = uaa.attention(st["q"], st["k"], st["v"], st["mask"], saved="int8")
        return (out,) + torch.autograd.grad(out, (st["q"], st["k"], st["v"]), st["dout"])
    if not case["grad"]:
        out, _, lse = uaa.diff_attn_fwd(st["q"], st["k"], st["v"], st["lam"], st["mask"], need_out2=False)
        return out, lse
    out, out2, lse = uaa.diff_attn_fwd(st["q"], st["k"], st["v"], st["lam"], st["mask"])
    return (out,) + uaa.diff_attn_bwd(st["q"], st["k"], st["v"], st["lam"], out, out2, st["dout"], lse, st["mask"])


# --------------------------------------------------------------------------- plain forms, 32 bits
def _turn_rates(case):
    """Angle per position of each pair, in 64 bits, and the axis that it follows."""
    rates, axis = [], []
    for a, width in enumerate(_axis_widths(case)):
        j = torch.arange(width // 2, dtype=torch.float64, device="cuda")
        s, base = case["factor"], 10000.0
        if case["scaling"] == "ntk" and width > 2:
            base *= s ** (width / (width - 2))
        f = base ** (-2.0 * j / max(width, 1))
        if case["scaling"] == "linear":
            f = f / s
        if case["scaling"] == "parts":
            p = PARTS
            keep = ((p["original"] * f / (2 * math.pi) - p["alpha"]) / (p["beta"] - p["alpha"])).clamp(0, 1)
            f = keep * f + (1 - keep) * f / s
        rates.append(f)
        axis.append(torch.full((width // 2,), a, dtype=torch.long, device="cuda"))
    return torch.cat(rates), torch.cat(axis)


def _magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "parts" else 1.0


def _plain_rotary(st):
    case = st["case"]
    rates, axis = _turn_rates(case)
    pos = st["positions"].unsqueeze(-1) if case["axes"] == 1 else st["positions"]
    angle = pos[..., axis].double() * rates  # 32 bits lose the angles of far positions
    cos, sin = (f(angle).float().unsqueeze(2) * _magnitude(case) for f in (torch.cos, torch.sin))
    R = case["rot"]

    def turn(x, sign):
        r, rest = x[..., :R].float(), x[..., R:]
        if case["layout"] == "half":
            a, b = r[..., : R // 2], r[..., R // 2:]
        else:
            a, b = r[..., 0::2], r[..., 1::2]
        u, w = a * cos - b * (sign * sin), a * (sign * sin) + b * cos
        y = torch.cat((u, w), -1) if case["layout"] == "half" else torch.stack((u, w), -1).flatten(-2)
        return torch.cat((y.to(x.dtype), rest), -1)

    out = (turn(st["q"], 1.0), turn(st["k"], 1.0))
    return out + (turn(st["dq"], -1.0), turn(st["dk"], -1.0)) if case["grad"] else out


def _plain_act8(x):
    r = x.double()  # 32 bits would round values next to a border between two codes to the wrong one
    top = r.abs().amax(-1, keepdim=True)
    codes = torch.where(top > 0, torch.round(r * 127.0 / top), torch.zeros_like(r))
    return (codes * (top / 127.0)).to(x.dtype)


def _heads(x):
    return x.float().transpose(1, 2)  # (B, H, S, D)


def _softmax_and_lse(s, mask):
    if mask is not None:
        s = s.masked_fill(~mask.reshape(mask.shape[0], *([1] * (s.dim() - 2)), -1), -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    return p / torch.where(total > 0, total, torch.ones_like(total)), lse


def _plain_step8(st):
    q, k, v, do = (_heads(st[n]) for n in ("q", "k", "v", "dout"))
    scale = 1.0 / math.sqrt(q.shape[-1])
    p, lse = _softmax_and_lse(torch.matmul(q, k.transpose(-1, -2)) * scale, st["mask"])
    out = torch.matmul(p, v).transpose(1, 2).to(torch.bfloat16)
    del p
    q, k, v, o = (_heads(_plain_act8(t)) for t in (st["q"], st["k"], st["v"], out))
    s = torch.matmul(q, k.transpose(-1, -2)) * scale
    if st["mask"] is not None:
        s = s.masked_fill(~st["mask"][:, None, None, :], -math.inf)
    lse = torch.where(torch.isinf(lse), torch.full_like(lse, math.inf), lse)  # no attended key: P = 0
    p = torch.exp(s - lse.unsqueeze(-1))
    dv = torch.matmul(p.transpose(-1, -2), do)
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True))
    dq, dk = torch.matmul(ds, k) * scale, torch.matmul(ds.transpose(-1, -2), q) * scale
    return (out,) + tuple(t.transpose(1, 2).to(torch.bfloat16) for t in (dq, dk, dv))


def _plain_diff(st):
    case = st["case"]
    q, k = (_heads(st[n]).unflatten(-1, (2, -1)).transpose(2, 3) for n in ("q", "k"))  # (B, H, 2, S, D/2)
    v, lam = _heads(st["v"]), st["lam"].float().reshape(1, -1, 1, 1)
    scale = 1.0 / math.sqrt(q.shape[-1])
    p, lse = _softmax_and_lse(torch.matmul(q, k.transpose(-1, -2)) * scale, st["mask"])
    a = p[:, :, 0] - lam * p[:, :, 1]
    out = torch.matmul(a, v).transpose(1, 2).to(torch.bfloat16)
    if not case["grad"]:
        return out, lse
    do = _heads(st["dout"])
    dv = torch.matmul(a.transpose(-1, -2), do)
    da = torch.matmul(do, v.transpose(-1, -2))
    del a
    rows = (p * da.unsqueeze(2)).sum(-1, keepdim=True)  # (B, H, 2, Sq, 1)
    dlam = -rows[:, :, 1].sum((0, 2, 3), dtype=torch.float64)
    ds = p * (da.unsqueeze(2) - rows)
    ds[:, :, 1] *= -lam
    del da, p
    dq, dk = torch.matmul(ds, k) * scale, torch.matmul(ds.transpose(-1, -2), q) * scale
    grads = tuple(t.transpose(2, 3).flatten(3).transpose(1, 2).to(torch.bfloat16) for t in (dq, dk))
    return (out,) + grads + (dv.transpose(1, 2).to(torch.bfloat16), dlam.to(st["lam"].dtype))


def run(st):
    if own:
        return _run_own(st)
    op = st["case"]["op"]
    with torch.no_grad():
        if op == "rotary":
            return _plain_rotary(st)
        if op == "act8":
            return [_plain_act8(x) for x in st["x"]]
        return _plain_step8(st) if op == "step8" else _plain_diff(st)


# --------------------------------------------------------------------------- definitions, 64 bits
def _exact_rotary(st):
    """Each pair as a complex number, multiplied by m * exp(i * angle)."""
    case = st["case"]
    R = case["rot"]
    pos = st["positions"].double().reshape(case["B"], case["S"], -1)
    parts = []
    for a, width in enumerate(_axis_widths(case)):
        n, s, inv = width // 2, case["factor"], []
        for j in range(n):
            f = 10000.0 ** (-2.0 * j / width)
            if case["scaling"] == "ntk" and width > 2:
                f = (10000.0 * s ** (width / (width - 2.0))) ** (-2.0 * j / width)
            elif case["scaling"] == "linear":
                f /= s
            elif case["scaling"] == "parts":
                p = PARTS
                turns = p["original"] * f / (2.0 * math.pi)
                g = min(1.0, max(0.0, (turns - p["alpha"]) / (p["beta"] - p["alpha"])))
                f = g * f + (1.0 - g) * f / s
            inv.append(f)
        parts.append(pos[..., a: a + 1] * torch.tensor(inv, dtype=torch.float64, device="cuda"))
    angle = torch.cat(parts, -1).unsqueeze(2)
    unit = torch.polar(torch.full_like(angle, _magnitude(case)), angle)

    def turn(x, w):
        r = x.double()
        y = r.clone()
        if case["layout"] == "half":
            z = torch.complex(r[..., : R // 2].contiguous(), r[..., R // 2: R].contiguous()) * w
            y[..., : R // 2], y[..., R // 2: R] = z.real, z.imag
        else:
            z = torch.complex(r[..., 0:R:2].contiguous(), r[..., 1:R:2].contiguous()) * w
            y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
        return y

    out = [turn(st["q"], unit), turn(st["k"], unit)]
    if case["grad"]:
        out += [turn(st["dq"], unit.conj()), turn(st["dk"], unit.conj())]
    return out


def _exact_act8(x, out_dtype=None):
    """The values that the codes stand for: whole multiples of the row's largest magnitude / 127."""
    r = x.double()
    top = r.abs().max(-1, keepdim=True).values
    safe = torch.where(top > 0, top, torch.ones_like(top))
    y = torch.round(127.0 * r / safe).mul(safe).div(127.0)
    return y if out_dtype is None else y.to(out_dtype).double()


def _exact_step8(st):
    """Per sequence and head: the softmax's Jacobian applied to dA = dO V^T, with the checkpoint's values."""
    case = st["case"]
    shape = st["q"].shape
    scale = shape[-1] ** -0.5
    out = torch.zeros(shape, dtype=torch.float64, device="cuda")
    lse = {}
    for b in range(case["B"]):
        keep = slice(None) if st["mask"] is None else st["mask"][b].nonzero().squeeze(-1)
        for h in range(case["H"]):
            s = scale * (st["q"][b, :, h].double() @ st["k"][b, keep, h].double().T)
            if s.shape[1]:
                lse[b, h] = torch.logsumexp(s, -1, keepdim=True)
                out[b, :, h] = torch.exp(s - lse[b, h]) @ st["v"][b, keep, h].double()
    q8, k8, v8, o8 = (_exact_act8(t, torch.bfloat16) for t in (st["q"], st["k"], st["v"], out.to(torch.bfloat16)))
    dq, dk, dv = (torch.zeros(shape, dtype=torch.float64, device="cuda") for _ in range(3))
    for (b, h), row in lse.items():
        keep = slice(None) if st["mask"] is None else st["mask"][b].nonzero().squeeze(-1)
        q, k, v, do = q8[b, :, h], k8[b, keep, h], v8[b, keep, h], st["dout"][b, :, h].double()
        a = torch.exp(scale * (q @ k.T) - row)
        ds = a * (do @ v.T - torch.einsum("id,id->i", do, o8[b, :, h])[:, None])
        dq[b, :, h] = scale * (ds @ k)
        dk[b, keep, h], dv[b, keep, h] = scale * (ds.T @ q), a.T @ do
    return [out, dq, dk, dv]


def _exact_diff(st):
    """Per sequence and head: two softmax maps over the attended keys only, and their Jacobians."""
    case = st["case"]
    B, H, D, Sq, Sk = case["B"], case["H"], case["D"], case["Sq"], case["Sk"]
    new = lambda *n: torch.zeros(n, dtype=torch.float64, device="cuda")  # noqa: E731
    out, lse = new(B, Sq, H, D), new(B, H, 2, Sq) - math.inf
    dq, dk, dv, dlam = new(B, Sq, H, D), new(B, Sk, H, D), new(B, Sk, H, D), new(H)
    w = D // 2
    for b in range(B):
        keep = slice(None) if st["mask"] is None else st["mask"][b].nonzero().squeeze(-1)
        for h in range(H):
            q, k, v = st["q"][b, :, h].double(), st["k"][b, keep, h].double(), st["v"][b, keep, h].double()
            if not k.shape[0]:
                continue
            lam = st["lam"][h].double()
            maps = []
            for m in range(2):
                s = (q[:, m * w: m * w + w] @ k[:, m * w: m * w + w].T) / math.sqrt(w)
                lse[b, h, m] = torch.logsumexp(s, -1)
                maps.append(torch.softmax(s, -1))
            out[b, :, h] = maps[0] @ v - lam * (maps[1] @ v)
            if case["grad"]:
                do = st["dout"][b, :, h].double()
                da = do @ v.T
                dv[b, keep, h] = maps[0].T @ do - lam * (maps[1].T @ do)
                dlam[h] -= torch.einsum("ij,ij->", maps[1], da)
                for m, weight in ((0, 1.0), (1, -lam)):
                    ds = weight * (maps[m] * da - maps[m] * torch.einsum("ij,ij->i", maps[m], da)[:, None]) / math.sqrt(w)
                    dq[b, :, h, m * w: m * w + w] = ds @ k[:, m * w: m * w + w]
                    dk[b, keep, h, m * w: m * w + w] = ds.T @ q[:, m * w: m * w + w]
    return [out, dq, dk, dv, dlam] if case["grad"] else [out, lse]


def exact(case, seed):
    st = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "rotary":
            return _exact_rotary(st)
        if case["op"] == "act8":
            return [_exact_act8(x) for x in st["x"]]
        return _exact_step8(st) if case["op"] == "step8" else _exact_diff(st)
