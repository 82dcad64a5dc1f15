"""The operators on integer 4-bit weights with group scales and the mixture-of-experts
layer for a few tokens: the cases they are measured on, their plain forms, and what
each gives in 64 bits.

int4_quantize    W [n, k] -> codes q in 0..15, a scale (and a zero point) per group of
                 consecutive weights of a row.  symmetric: s = max|w| / 7, q = rint(w / s) + 8;
                 asymmetric: s = (max(w, 0) - min(w, 0)) / 15, z = rint(-min(w, 0) / s),
                 q = rint(w / s) + z; both clamped to 0..15, every step in 32 bits.
                 (Measured with the restored weight, the values that the codes stand for.)
int4_dequantize  out[r][c] = (q[r][c] - z[c / g][r]) * s[c / g][r].
int4_linear      Y[t][r] = sum_c X[t][c] * (q[r][c] - z[c / g][r]) * s[c / g][r].
moe              the layer of E experts on m tokens: logits = X router^T, the top_k largest
                 of each row (ties to the lower index), weighted by their softmax
                 probability (renormalized over the chosen ones or not);
                 Y[t] = sum_e w[t][e] * D_e (silu(G_e x_t) * (U_e x_t)), with the experts'
                 weights in 4 bits: NF4 or FP4 levels with double-quantized block scales,
                 or integers with group scales.
"""
import random

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # one token through an attention projection of a 4096-wide model: latency counts
        {"name": "linear 1 4096x4096", "op": "linear", "m": 1, "n": 4096, "k": 4096, "group": 128, "zero": False,
         "scale": BF16, "out": BF16},
        # sixteen sequences through the widest projection of the benchmark's stress layer
        {"name": "linear 16 28672x8192", "op": "linear", "m": 16, "n": 28672, "k": 8192, "group": 64, "zero": True,
         "scale": BF16, "out": BF16},
        # a few sequences, ragged sizes, the finest groups, logits kept in 32 bits
        {"name": "linear 5 1003x1088", "op": "linear", "m": 5, "n": 1003, "k": 1088, "group": 32, "zero": True,
         "scale": F32, "out": F32},
        # a prompt through an up projection
        {"name": "linear 512 11008x4096", "op": "linear", "m": 512, "n": 11008, "k": 4096, "group": 128, "zero": False,
         "scale": BF16, "out": BF16},
        # one token, many small experts
        {"name": "moe 1 E64 top6 nf4", "op": "moe", "m": 1, "experts": 64, "top_k": 6, "h": 2048, "f": 1408,
         "format": "nf4", "renormalize": True},
        # sixteen tokens, eight large experts: every expert is read
        {"name": "moe 16 E8 top2 nf4", "op": "moe", "m": 16, "experts": 8, "top_k": 2, "h": 4096, "f": 14336,
         "format": "nf4", "renormalize": True},
        # seven tokens spread over many experts in integer weights
        {"name": "moe 7 E128 top8 int4", "op": "moe", "m": 7, "experts": 128, "top_k": 8, "h": 2048, "f": 768,
         "format": "int4", "group": 128, "zero": False, "scale": BF16, "renormalize": False},
        # a small layer, FP4 levels, one expert a token
        {"name": "moe 3 E4 top1 fp4", "op": "moe", "m": 3, "experts": 4, "top_k": 1, "h": 1024, "f": 704,
         "format": "fp4", "renormalize": False},
        # quantizing a checkpoint's layers at load time, and back in full to see what was kept
        {"name": "quantize 11008x4096", "op": "quantize", "n": 11008, "k": 4096, "group": 128, "zero": False,
         "scale": BF16, "dtype": BF16},
        {"name": "quantize 1003x1088", "op": "quantize", "n": 1003, "k": 1088, "group": 32, "zero": True,
         "scale": F32, "dtype": F32},
        # a weight back in full, for a product of one's own or an export
        {"name": "dequantize 11008x4096", "op": "dequantize", "n": 11008, "k": 4096, "group": 128, "zero": True,
         "scale": BF16, "out": BF16},
        {"name": "dequantize 1003x1088", "op": "dequantize", "n": 1003, "k": 1088, "group": 32, "zero": False,
         "scale": F32, "out": F32},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["linear", "linear", "moe", "moe", "quantize", "dequantize"])
    if op == "moe":
        while True:
            experts = rng.choice([4, 8, 10, 16, 32, 60, 64, 100, 128, 256])
            c = {"op": "moe", "m": _log(rng, 1, 16), "experts": experts, "top_k": rng.randint(1, min(8, experts)),
                 "format": rng.choice(["nf4", "nf4", "fp4", "int4"]), "renormalize": rng.random() < 0.5}
            if c["format"] == "int4":
                c.update(group=rng.choice([32, 64, 128]), zero=rng.random() < 0.5, scale=rng.choice([BF16, F32]))
            unit = max(64, c.get("group", 64))
            c.update(h=unit * _log(rng, 512 // unit, 5120 // unit), f=unit * _log(rng, 256 // unit, 14336 // unit))
            if experts * c["h"] * c["f"] <= 8 * 4096 * 14336 // 2:
                return c
    group = rng.choice([32, 64, 128, 256])
    while True:
        n = _log(rng, 16, 28672)
        k = max(group, 64) * _log(rng, 1, 16384 // max(group, 64))
        if 4096 <= n * k <= 28672 * 8192 // 2:
            break
    c = {"op": op, "n": n, "k": k, "group": group, "zero": rng.random() < 0.5, "scale": rng.choice([BF16, BF16, F32])}
    if op == "linear":
        c["m"] = _log(rng, 1, 16) if rng.random() < 0.75 else _log(rng, 17, 1024)
        if c["m"] * n * k > 512 * 11008 * 4096:
            c["m"] = max(1, 512 * 11008 * 4096 // (n * k))
        c["out"] = rng.choice([BF16, BF16, F32]) if c["m"] <= 16 else BF16
    elif op == "quantize":
        c["dtype"] = rng.choice([BF16, BF16, F32])
    else:
        c["out"] = rng.choice([BF16, BF16, F32])
    return c


def _int4_state(gen, n, k, group, zero, scale):
    """Codes as they come of normal weights (a group's largest is about 2.7 standard
    deviations), two to a byte with the even element in the high half; scales [k / g, n]."""
    dev = "cuda"
    wq = torch.empty(n * k // 2, dtype=torch.uint8, device=dev)
    step = 1 << 27
    for i in range(0, wq.numel(), step):
        e = min(wq.numel(), i + step)
        q = torch.randn(e - i, 2, device=dev, generator=gen).mul_(2.6).round_().add_(8).clamp_(0, 15).to(torch.uint8)
        wq[i:e] = q[:, 0] * 16 + q[:, 1]
    s = torch.rand(k // group, n, device=dev, generator=gen).mul_(0.004).add_(0.006).to(DTYPES[scale])
    z = torch.randint(5, 11, (k // group, n), device=dev, generator=gen, dtype=torch.uint8) if zero else None
    return {"wq": wq, "scale": s, "zero": z, "n": n, "k": k, "group": group}


def _nf4_state(gen, n, k, kind):
    """NF4 and FP4 codes are close to uniform by construction; absmax values spread around
    their mean as those of blocks of 64 normal weights do."""
    dev = "cuda"
    nb = n * k // 64
    return {"wq": torch.randint(0, 256, (n * k // 2,), device=dev, generator=gen, dtype=torch.uint8),
            "absmax_q": torch.randint(-100, 128, (nb,), device=dev, generator=gen, dtype=torch.int8),
            "absmax_scale": torch.rand((nb + 255) // 256, device=dev, generator=gen).mul_(0.004).add_(0.018),
            "absmax_offset": torch.full((1,), 0.047, device=dev), "n": n, "k": k, "kind": kind}


def _handle(w):
    """The framework's object for a weight, which a program keeps beside its tensors."""
    import quantized_linear_layers_nf4_b200 as nf4
    if "group" in w:
        return nf4.Int4Weight(w["n"], w["k"], w["group"], w["wq"], w["scale"], w["zero"])
    return nf4.NF4Weight(w["n"], w["k"], w["wq"], w["absmax_q"], w["absmax_scale"], w["absmax_offset"], w["kind"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    c, op = dict(case), case["op"]
    s = {"case": c}
    if op == "moe":
        m, e, h, f = c["m"], c["experts"], c["h"], c["f"]
        s["x"] = torch.randn(m, h, device="cuda", generator=gen).to(torch.bfloat16)
        s["router"] = torch.randn(e, h, device="cuda", generator=gen).mul_(1.5 * h ** -0.5).to(torch.bfloat16)
        if c["format"] == "int4":
            s["gate_up"] = _int4_state(gen, e * 2 * f, h, c["group"], c["zero"], c["scale"])
            s["down"] = _int4_state(gen, e * h, f, c["group"], c["zero"], c["scale"])
        else:
            s["gate_up"] = _nf4_state(gen, e * 2 * f, h, c["format"])
            s["down"] = _nf4_state(gen, e * h, f, c["format"])
        s["y"] = torch.empty(m, h, device="cuda", dtype=torch.bfloat16)
        if own:
            import quantized_linear_layers_nf4_b200 as nf4
            s["gate_up_h"], s["down_h"] = _handle(s["gate_up"]), _handle(s["down"])
            s["ws"] = nf4.moe_workspace(h, f, e, c["top_k"])
    elif op == "quantize":
        w = torch.randn(c["n"], c["k"], device="cuda", generator=gen).mul_(0.02)
        w[0, :c["group"]] = 0  # a group of zeros
        s["w"] = w.to(DTYPES[c["dtype"]])
    else:
        s["w"] = _int4_state(gen, c["n"], c["k"], c["group"], c["zero"], c["scale"])
        if op == "linear":
            s["x"] = torch.randn(c["m"], c["k"], device="cuda", generator=gen).to(torch.bfloat16)
            s["y"] = torch.empty(c["m"], c["n"], device="cuda", dtype=DTYPES[c["out"]])
        else:
            s["y"] = torch.empty(c["n"], c["k"], device="cuda", dtype=DTYPES[c["out"]])
        if own:
            s["w_h"] = _handle(s["w"])
    return s


# ------------------------------ plain forms ------------------------------
def _levels(kind):
    if kind == "fp4":
        v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
        return torch.tensor([x / 6 for x in v] + [-x / 6 for x in v], device="cuda", dtype=torch.float32)
    # quantiles of the normal distribution: eight above zero, seven below, zero itself
    d = ((1 - 1 / 30) + (1 - 1 / 32)) / 2
    p = [d - i * (d - 0.5) / 8 for i in range(8)] + [1 - (d - i * (d - 0.5) / 7) for i in range(7)] + [0.5]
    q = torch.special.ndtri(torch.tensor(p, dtype=torch.float64)).sort().values
    return (q / q.abs().max()).to(torch.float32).cuda()


def _codes(wq):
    return torch.stack((wq >> 4, wq & 15), -1)


def _dense(w, rows=None):
    """A weight in 32 bits, [n, k], or [len(rows), k] of the given rows."""
    n, k = w["n"], w["k"]
    q = w["wq"].view(n, k // 2)
    q = _codes(q if rows is None else q[rows]).flatten(1)
    if "group" in w:
        g = w["group"]
        s = (w["scale"] if rows is None else w["scale"][:, rows]).t().float()
        z = 8.0 if w["zero"] is None else (w["zero"] if rows is None else w["zero"][:, rows]).t().float().unsqueeze(-1)
        return ((q.float().view(-1, k // g, g) - z) * s.unsqueeze(-1)).view(-1, k)
    blocks = torch.arange(n * k // 64, device="cuda").view(n, k // 64)
    blocks = blocks if rows is None else blocks[rows]
    a = w["absmax_q"][blocks].float() / 127 * w["absmax_scale"][blocks >> 8] + w["absmax_offset"]
    return (_levels(w["kind"])[q.int()].view(-1, k // 64, 64) * a.unsqueeze(-1)).view(-1, k)


def _plain_moe(s):
    c = s["case"]
    e, h, f, top = c["experts"], c["h"], c["f"], c["top_k"]
    logits = s["x"].double() @ s["router"].double().t()
    value, ids = logits.sort(dim=1, descending=True, stable=True)
    value, ids = value[:, :top], ids[:, :top]
    weight = (value - value[:, :1]).exp()
    total = weight.sum(1, keepdim=True) if c["renormalize"] else (logits - value[:, :1]).exp().sum(1, keepdim=True)
    weight = (weight / total).float()
    x = s["x"].float()
    m = x.shape[0]
    if m * top <= e:  # the chosen experts alone, one for each (token, choice)
        pick = ids.flatten()
        gu = _dense(s["gate_up"], (pick[:, None] * (2 * f) + torch.arange(2 * f, device="cuda")).flatten())
        z = torch.matmul(gu.view(m, top * 2 * f, h), x.unsqueeze(-1)).view(m * top, 2 * f)
        a = z[:, :f] * torch.sigmoid(z[:, :f]) * z[:, f:] * weight.view(-1, 1)
        d = _dense(s["down"], (pick[:, None] * h + torch.arange(h, device="cuda")).flatten())
        y = torch.matmul(d.view(m * top, h, f), a.unsqueeze(-1)).view(m, top, h).sum(1)
    else:  # every expert on every token, weighted by zero where it was not chosen
        z = (x @ _dense(s["gate_up"]).t()).view(m, e, 2 * f)
        spread = torch.zeros(m, e, device="cuda").scatter_(1, ids, weight)
        a = z[:, :, :f] * torch.sigmoid(z[:, :, :f]) * z[:, :, f:] * spread.unsqueeze(-1)
        y = torch.matmul(_dense(s["down"]).view(e, h, f), a.permute(1, 2, 0)).sum(0).t()
    return y.to(torch.bfloat16), ids.int(), weight


def _plain_quantize(s):
    c = s["case"]
    w = s["w"].float().view(c["n"], c["k"] // c["group"], c["group"])
    if c["zero"]:
        lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
        # divided by a tensor: by a number it would be multiplied by a rounded reciprocal
        sc = ((hi - lo) / torch.full_like(lo, 15)).to(DTYPES[c["scale"]])
        d = torch.where(sc > 0, sc.float(), torch.ones_like(lo))
        z = (-lo / d).round().clamp(0, 15)
    else:
        top = w.abs().amax(-1)
        sc = (top / torch.full_like(top, 7)).to(DTYPES[c["scale"]])
        d = torch.where(sc > 0, sc.float(), torch.ones_like(top))
        z = torch.full_like(d, 8)
    q = ((w / d.unsqueeze(-1)).round() + z.unsqueeze(-1)).clamp(0, 15)
    back = ((q - z.unsqueeze(-1)) * sc.float().unsqueeze(-1)).view(c["n"], c["k"]).to(DTYPES[c["dtype"]])
    return (back, sc.t().contiguous()) + ((z.t().to(torch.uint8).contiguous(),) if c["zero"] else ())


def run(state):
    c, op = state["case"], state["case"]["op"]
    if own:
        import quantized_linear_layers_nf4_b200 as nf4
        if op == "moe":
            return nf4.nf4_moe(state["x"], state["router"], state["gate_up_h"], state["down_h"], c["top_k"],
                               renormalize=c["renormalize"], out=state["y"], workspace=state["ws"], return_routing=True)
        if op == "linear":
            return nf4.nf4_int4_linear(state["x"], state["w_h"], out=state["y"])
        if op == "dequantize":
            return nf4.nf4_int4_dequantize(state["w_h"], out=state["y"])
        w = nf4.int4_quantize_weight(state["w"], c["group"], symmetric=not c["zero"], scale_dtype=DTYPES[c["scale"]])
        return (nf4.nf4_int4_dequantize(w, DTYPES[c["dtype"]]), w.scale) + ((w.zero,) if c["zero"] else ())
    if op == "moe":
        return _plain_moe(state)
    if op == "linear":
        return (state["x"].float() @ _dense(state["w"]).t()).to(DTYPES[c["out"]])
    if op == "dequantize":
        return _dense(state["w"]).to(DTYPES[c["out"]])
    return _plain_quantize(state)


def _side(c, key="scale"):
    """Bytes of scale and zero point for each group."""
    return (2 if c[key] == BF16 else 4) + (1 if c["zero"] else 0)


def work(case):
    c, op = case, case["op"]
    if op == "moe":
        m, e, h, f, top = c["m"], c["experts"], c["h"], c["f"], c["top_k"]
        active = e * (1 - (1 - top / e) ** m)  # expected, each token's choice being even
        bit = 0.5 + (_side(c) / c["group"] if c["format"] == "int4" else 1 / 64 + 4 / 16384)
        return {"bytes": active * 3 * h * f * bit + e * h * 2 + m * h * 4 + m * top * 8,
                "flops": 2 * m * h * (e + 3 * top * f)}
    n, k = c["n"], c["k"]
    packed = n * k // 2 + n * (k // c["group"]) * _side(c)
    if op == "linear":
        return {"bytes": packed + c["m"] * k * 2 + c["m"] * n * (2 if c["out"] == BF16 else 4), "flops": 2 * c["m"] * n * k}
    if op == "quantize":  # the weight in and back, its codes between
        return {"bytes": packed + 2 * n * k * (2 if c["dtype"] == BF16 else 4), "flops": 6 * n * k}
    return {"bytes": packed + n * k * (2 if c["out"] == BF16 else 4), "flops": 2 * n * k}


# ------------------------------ in 64 bits ------------------------------
def _exact_levels(kind):
    if kind == "fp4":
        mag = np.array([0, 1, 2, 3, 4, 6, 8, 12], dtype=np.float64) / 12
        return torch.from_numpy(np.concatenate([mag, -mag]).astype(np.float32).astype(np.float64)).cuda()
    from statistics import NormalDist
    inv, delta = NormalDist().inv_cdf, 0.5 * (29 / 30 + 31 / 32)
    up = [inv(float(p)) for p in np.linspace(delta, 0.5, 9)[:-1]]
    down = [-inv(float(p)) for p in np.linspace(delta, 0.5, 8)[:-1]]
    v = np.array(sorted(up + down + [0.0])) / max(up)
    return torch.from_numpy(v.astype(np.float32).astype(np.float64)).cuda()


def _exact_rows(w, r0, r1):
    """Rows r0 .. r1 of a weight, element by element from its definition."""
    k = w["k"]
    at = torch.arange(r0 * k, r1 * k, device="cuda")
    byte = w["wq"][at // 2].long()
    code = torch.where(at % 2 == 0, byte // 16, byte % 16)
    if "group" in w:
        grp, row = (at % k) // w["group"], at // k
        z = w["zero"][grp, row].double() if w["zero"] is not None else 8.0
        return ((code.double() - z) * w["scale"][grp, row].double()).view(r1 - r0, k)
    b = at // 64
    a = w["absmax_q"][b].double() * w["absmax_scale"][b // 256].double() / 127 + w["absmax_offset"].double()
    return (_exact_levels(w["kind"])[code] * a).view(r1 - r0, k)


def _exact_product(w, r0, r1, x):
    """x [m, k] times rows r0 .. r1, a slab at a time."""
    step = max(1, (1 << 26) // w["k"])
    return torch.cat([x @ _exact_rows(w, i, min(r1, i + step)).t() for i in range(r0, r1, step)], 1)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], case["op"]
    if op == "linear":
        return _exact_product(s["w"], 0, c["n"], s["x"].double())
    if op == "dequantize":
        step = max(1, (1 << 26) // c["k"])
        return torch.cat([_exact_rows(s["w"], i, min(c["n"], i + step)) for i in range(0, c["n"], step)])
    if op == "quantize":  # every step is one in 32 bits, by definition, but for the last product
        g = c["group"]
        w = s["w"].float().cpu().numpy().reshape(c["n"], -1, g)
        if c["zero"]:
            lo, hi = np.minimum(w.min(-1), np.float32(0)), np.maximum(w.max(-1), np.float32(0))
            span = (hi - lo) / np.float32(15)
        else:
            span = np.abs(w).max(-1) / np.float32(7)
        sc = torch.from_numpy(span).to(DTYPES[c["scale"]]).float().numpy()
        d = np.where(sc > 0, sc, np.float32(1))
        z = np.clip(np.rint(-lo / d), 0, 15) if c["zero"] else np.full_like(d, 8)
        q = np.clip(np.rint(w / d[..., None]) + z[..., None], 0, 15)
        back = (q.astype(np.float64) - z[..., None]) * sc.astype(np.float64)[..., None]
        return (torch.from_numpy(back.reshape(c["n"], c["k"])), torch.from_numpy(span.astype(np.float64).T.copy())) + ((None,) if c["zero"] else ())
    x = s["x"].double()
    e, h, f, top = c["experts"], c["h"], c["f"], c["top_k"]
    logits = (x.unsqueeze(1) * s["router"].double()).sum(-1)
    y = torch.zeros_like(x)
    ids, ws = [], []
    for t in range(x.shape[0]):
        row = logits[t].tolist()
        best = sorted(range(e), key=lambda i: (-row[i], i))[:top]
        p = torch.tensor(row, dtype=torch.float64).softmax(0)[best]
        ids.append(best)
        ws.append((p / p.sum() if c["renormalize"] else p).tolist())
    for i in sorted({i for b in ids for i in b}):
        who = [(t, ids[t].index(i)) for t in range(len(ids)) if i in ids[t]]
        xe = x[[t for t, _ in who]]
        g = _exact_product(s["gate_up"], i * 2 * f, i * 2 * f + f, xe)
        u = _exact_product(s["gate_up"], i * 2 * f + f, (i + 1) * 2 * f, xe)
        o = _exact_product(s["down"], i * h, (i + 1) * h, g / (1 + torch.exp(-g)) * u)
        for j, (t, slot) in enumerate(who):
            y[t] += ws[t][slot] * o[j]
    return y, None, torch.tensor(ws, dtype=torch.float64)
