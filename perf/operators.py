"""The 4-bit tier and the mixture-of-experts layer: what is timed, and the
plain form of each operator.

fp4 recode   BF16 weights to 4-bit codes with one power-of-two scale per 32
             columns (wc.fp4_encode), and back to BF16 (wc.fp4_decode).
fp4 gemv     y = W x with W in that form (wc.fp4_gemv), batch 1..256.
moe          a whole mixture-of-experts layer for up to 64 tokens (wc.moe):
             router, top-k, the experts' gated products and their weighted
             sum, with experts in BF16 or in the 4-bit form.

Where `own` is false, run() computes with elementary torch operations.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 32  # columns that share a scale
MOST_TOKENS = 64
MOST_BATCH = 256


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # one head group's projection, coded once at load: the smallest recode
        {"name": "recode 1000x4100", "op": "recode", "rows": 1000, "cols": 4100},
        # a layer's up projection of the layer set
        {"name": "recode 24576x6144", "op": "recode", "rows": 24576, "cols": 6144},
        # a key/value projection for one token: latency counts
        {"name": "gemv 1024x4096 b1", "op": "gemv", "rows": 1024, "cols": 4096, "batch": 1},
        # a layer's large matrix for one token: bandwidth counts
        {"name": "gemv 24576x6144 b1", "op": "gemv", "rows": 24576, "cols": 6144, "batch": 1},
        # an MLP matrix for a few sequences
        {"name": "gemv 14336x4096 b4", "op": "gemv", "rows": 14336, "cols": 4096, "batch": 4},
        # rows that fill no row tile, columns that end inside a group
        {"name": "gemv 5003x4100 b16", "op": "gemv", "rows": 5003, "cols": 4100, "batch": 16},
        # long rows, a full decode batch
        {"name": "gemv 6144x24576 b32", "op": "gemv", "rows": 6144, "cols": 24576, "batch": 32},
        # the widest batch the entry point takes
        {"name": "gemv 4096x4096 b256", "op": "gemv", "rows": 4096, "cols": 4096, "batch": 256},
        # a small MoE layer for one token: latency counts
        {"name": "moe fp4 t1", "op": "moe", "kind": "fp4", "tokens": 1, "hidden": 2048, "inter": 1408,
         "experts": 64, "top_k": 6, "scoring": "softmax", "bias": False, "renorm": True},
        # few large experts kept in BF16, two sequences
        {"name": "moe bf16 t2", "op": "moe", "kind": "bf16", "tokens": 2, "hidden": 4096, "inter": 2048,
         "experts": 32, "top_k": 4, "scoring": "softmax", "bias": False, "renorm": False},
        # many experts, a decode batch, selection by biased sigmoid scores with two experts masked out
        {"name": "moe fp4 t16", "op": "moe", "kind": "fp4", "tokens": 16, "hidden": 4096, "inter": 1024,
         "experts": 128, "top_k": 8, "scoring": "sigmoid", "bias": True, "renorm": True},
        # the most tokens a call takes: nearly every expert is read
        {"name": "moe bf16 t64", "op": "moe", "kind": "bf16", "tokens": 64, "hidden": 2048, "inter": 1024,
         "experts": 64, "top_k": 8, "scoring": "softmax", "bias": False, "renorm": True},
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A matrix side: mostly a multiple of 128 or 32, sometimes any number."""
    n = _spread(rng, lo, hi)
    step = rng.choice((128, 128, 32, 8, 1))
    n = max(step, n // step * step)
    return n + step if 2 * n == 3072 or n == 3072 else n


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("recode", "gemv", "gemv", "moe", "moe"))
        if op == "recode":
            c = {"op": op, "rows": _size(rng, 64, 24576), "cols": _size(rng, 512, 24576)}
        elif op == "gemv":
            c = {"op": op, "rows": _size(rng, 512, 24576), "cols": _size(rng, 512, 24576),
                 "batch": _spread(rng, 1, MOST_BATCH)}
        else:
            experts = _spread(rng, 8, 128)
            c = {"op": op, "kind": rng.choice(("fp4", "bf16")), "tokens": _spread(rng, 1, MOST_TOKENS),
                 "hidden": _size(rng, 1024, 4096), "inter": _size(rng, 512, 2048), "experts": experts,
                 "top_k": rng.randint(1, 8), "scoring": rng.choice(("softmax", "sigmoid")),
                 "bias": rng.random() < 0.5, "renorm": rng.random() < 0.7}
        if _cost(c) <= most:
            return c


# ---- work --------------------------------------------------------------------

def _fp4_bytes(rows, cols):
    groups = -(-cols // GROUP)
    return rows * groups * (GROUP // 2 + 1)


def work(case):
    if case["op"] == "recode":
        n = case["rows"] * case["cols"]
        # encode reads the weights and writes the codes; decode the other way
        return {"bytes": 2 * (2 * n + _fp4_bytes(case["rows"], case["cols"])), "flops": 0}
    if case["op"] == "gemv":
        r, c, b = case["rows"], case["cols"], case["batch"]
        return {"bytes": _fp4_bytes(r, c) + 2 * b * c + 4 * b * r, "flops": 2 * b * r * c}
    t, h, i, e, k = (case[n] for n in ("tokens", "hidden", "inter", "experts", "top_k"))
    free = e - _masked(case)
    active = free * (1 - (1 - k / free) ** t)  # experts that some token is expected to reach
    per = (_fp4_bytes(2 * i, h) + _fp4_bytes(h, i)) if case["kind"] == "fp4" else 2 * 3 * h * i
    return {"bytes": active * per + 2 * e * h + 4 * t * h + 8 * t * k,
            "flops": 2 * t * e * h + 2 * t * k * 3 * h * i}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _masked(case):
    """Experts that the case's bias takes out of the selection."""
    return 2 if case["bias"] and case["experts"] >= case["top_k"] + 2 else 0


# ---- the plain forms ---------------------------------------------------------

VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # by the code's low three bits; bit 3 is the sign


def plain_encode(w):
    """codes [.., rows, 16 ceil(cols / 32)] and scales [.., rows, ceil(cols / 32)]
    of BF16 w [.., rows, cols].  A group's scale is 2^(e - 127), the smallest
    (e >= 1) that keeps every |w| within 7 of it, so that no weight moves by
    more than half of the largest step between two codes; weights round to the
    nearest of the 16 values that BF16 holds, ties to the even code.  A group
    that holds an infinity or a NaN gets e = 255."""
    cols = w.shape[-1]
    groups = -(-cols // GROUP)
    f = torch.nn.functional.pad(w.float(), (0, groups * GROUP - cols))
    f = f.reshape(*w.shape[:-1], groups, GROUP)
    bits = f.view(torch.int32) >> 16 & 0x7FFF
    top = bits.amax(-1)
    e = (top >> 7) - 2 + ((top & 0x7F) > 0x60).int()
    e = e.clamp(min=1)
    a = f.abs() * ((254 - e) << 23).view(torch.float32)[..., None]  # |w| / 2^(e - 127), exact
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
            + (a > 2.5).int() + (a >= 3.5).int() + (a > 5).int())
    code = torch.where(e[..., None] == 253, code.clamp(max=5), code)  # 4 * 2^126 is past BF16
    code = code | torch.signbit(f).int() << 3
    bad = top >= 0x7F80
    e = torch.where(bad, 255, e)
    code = torch.where(bad[..., None], 0, code)
    code = code.reshape(*w.shape[:-1], groups * GROUP)
    codes = (code[..., 0::2] | code[..., 1::2] << 4).to(torch.uint8)
    return codes.contiguous(), e.to(torch.uint8).contiguous()


def _two_to(e):
    """2^e in fp64 for whole e of -1022..1023, from its bits."""
    return (e.long() + 1023 << 52).view(torch.float64)


def plain_values(codes, scales, cols):
    """The fp32 values that codes and scales stand for, [.., rows, cols]."""
    dev = codes.device
    v = torch.tensor(VALUES + tuple(-x for x in VALUES), device=dev)
    s = _two_to(torch.arange(256, device=dev) - 127).float()
    s[255] = math.nan
    q = codes.to(torch.int32)
    w = v[torch.stack((q & 15, q >> 4), -1)].reshape(*scales.shape, GROUP)
    w = w * s[scales.to(torch.int32)][..., None]
    return w.reshape(*codes.shape[:-1], -1)[..., :cols]


def plain_route(x, router, k, scoring, bias, renorm):
    """ids [T, k] (int32, -1 where a token has fewer experts to choose from)
    and their weights [T, k]: the k largest logits, or score + bias where there
    is a bias; ties to the lowest index; a bias of -inf takes an expert out."""
    logits = x.double() @ router.double().T
    score = torch.sigmoid(logits) if scoring == "sigmoid" else torch.softmax(logits, -1)
    order = logits if bias is None else (score + bias.double())
    out = torch.zeros_like(order, dtype=torch.bool) if bias is None else torch.isneginf(bias).expand_as(order)
    # masked experts go behind every other one
    ids = torch.sort(torch.where(out, -math.inf, order), descending=True, stable=True).indices[:, :k]
    gone = out.gather(1, ids)
    weights = torch.where(gone, 0.0, score.gather(1, ids))
    if renorm:
        weights = weights / weights.sum(-1, keepdim=True)
    return torch.where(gone, -1, ids).int(), weights.float()


def plain_moe(s):
    case, x = s["case"], s["x"]
    t, h, i = case["tokens"], case["hidden"], case["inter"]
    ids, weights = plain_route(x, s["router"], case["top_k"], case["scoring"], s["bias"], case["renorm"])
    if t * case["top_k"] <= case["experts"]:
        # the chosen experts alone, one copy of each for each token that chose it
        at = ids.clamp(min=0).flatten().long()
        gate_up, down = _experts(s, "gate_up", h, at), _experts(s, "down", i, at)
        xs = x.float().repeat_interleave(case["top_k"], 0)
        gu = (gate_up @ xs[:, :, None])[..., 0]
        a = gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:] * weights.flatten()[:, None]
        y = (down @ a[:, :, None])[..., 0].reshape(t, -1, h).sum(1)
    else:
        gate_up, down = _experts(s, "gate_up", h), _experts(s, "down", i)
        share = torch.zeros(t, case["experts"], device=x.device)
        share.scatter_add_(1, ids.clamp(min=0).long(), weights)
        gu = (gate_up.reshape(-1, h) @ x.float().T).reshape(case["experts"], 2 * i, t)
        a = gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:] * share.T[:, None, :]
        y = (down @ a).sum(0).T
    return y.to(torch.bfloat16).contiguous(), ids, weights


def _experts(s, name, cols, at=None):
    """fp32 weights of all experts, or of those at `at`."""
    take = lambda v: v if at is None else v[at]  # noqa: E731
    if s["case"]["kind"] == "fp4":
        return plain_values(take(s[name][0]), take(s[name][1]), cols)
    return take(s[name]).float()


# ---- one pass ----------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, sigma=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * sigma).to(torch.bfloat16)

    def activations(n, cols):
        """N(0, 1) with a few strong channels, as hidden states have them."""
        x = torch.randn(n, cols, generator=g, device=DEV)
        x[:, torch.randint(cols, (max(1, cols // 512),), generator=g, device=DEV)] *= 8.0
        return x.to(torch.bfloat16)

    def matrix(*shape):
        """Rows of different spread, as trained matrices have them."""
        w = torch.randn(*shape, generator=g, device=DEV)
        w *= torch.exp(0.5 * torch.randn(*shape[:-1], 1, generator=g, device=DEV)) / math.sqrt(shape[-1])
        return w.to(torch.bfloat16)

    s = {"case": case}
    if case["op"] == "recode":
        s["w"] = matrix(case["rows"], case["cols"])
    elif case["op"] == "gemv":
        s["codes"], s["scales"] = plain_encode(matrix(case["rows"], case["cols"]))
        s["x"] = activations(case["batch"], case["cols"])
    else:
        e, h, i = case["experts"], case["hidden"], case["inter"]
        s["x"] = normal(case["tokens"], h)
        s["router"] = normal(e, h, sigma=1.0 / math.sqrt(h))
        s["bias"] = None
        if case["bias"]:
            s["bias"] = torch.randn(e, generator=g, device=DEV) * 0.05
            s["bias"][:_masked(case)] = -math.inf
        for name, shape in (("gate_up", (2 * i, h)), ("down", (h, i))):
            if case["kind"] == "bf16":
                s[name] = torch.stack([matrix(*shape) for _ in range(e)])
            else:
                parts = [plain_encode(matrix(*shape)) for _ in range(e)]
                s[name] = (torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]))
    return s


def run(s):
    case = s["case"]
    if own:
        import decode_gemv_sign_amd as wc
        if case["op"] == "recode":
            return wc.fp4_decode(wc.fp4_encode(s["w"]))
        if case["op"] == "gemv":
            return wc.fp4_gemv(wc.Fp4(s["codes"], s["scales"], case["cols"]), s["x"])
        gate_up, down = s["gate_up"], s["down"]
        if case["kind"] == "fp4":
            gate_up, down = wc.Fp4(*gate_up, case["hidden"]), wc.Fp4(*down, case["inter"])
        return wc.moe(s["x"], s["router"], gate_up, down, case["top_k"],
                      scoring=wc.SIGMOID if case["scoring"] == "sigmoid" else wc.SOFTMAX,
                      bias=s["bias"], renorm=case["renorm"])
    if case["op"] == "recode":
        return plain_values(*plain_encode(s["w"]), case["cols"]).to(torch.bfloat16)
    if case["op"] == "gemv":
        return s["x"].float() @ plain_values(s["codes"], s["scales"], case["cols"]).T
    return plain_moe(s)


# ---- the definitions in 64 bits ----------------------------------------------

def _power(e):
    """2^e in fp64, exact, for whole e of -130..130."""
    return torch.tensor([2.0 ** k for k in range(-130, 131)], dtype=torch.float64, device=e.device)[e + 130]


def _real(codes, scales, cols):
    """Values of one matrix by the codes' fields: sign, two exponent bits and
    one mantissa bit (exponent 0 is subnormal), times the group's scale."""
    c = torch.empty(*codes.shape, 2, dtype=torch.int64, device=codes.device)
    c[..., 0], c[..., 1] = codes % 16, codes // 16
    c = c.flatten(-2)
    sign, exp, man = 1.0 - 2.0 * (c // 8).double(), c // 2 % 4, (c % 2).double()
    mag = torch.where(exp == 0, man / 2, (1 + man / 2) * _power(exp - 1))
    scale = _power(scales.long() - 127)
    return (sign * mag * scale.repeat_interleave(GROUP, -1))[..., :cols]


def _exact_recode(w):
    """The nearest of the group's values, by distance to each of the eight
    magnitudes, in pieces of rows."""
    grid = torch.tensor(VALUES, dtype=torch.float64, device=w.device)
    prefer = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=w.device)  # even codes first: they win ties
    out = torch.empty(w.shape, dtype=torch.float64, device=w.device)
    cols = w.shape[1]
    for r in range(0, w.shape[0], 512):
        p = w[r:r + 512].double()
        a = torch.zeros(p.shape[0], -(-cols // GROUP) * GROUP, dtype=torch.float64, device=w.device)
        a[:, :cols] = p.abs()
        a = a.view(p.shape[0], -1, GROUP)
        top = a.amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(top / 7)).clamp(min=-126)  # smallest scale with top <= 7 * 2^e
        e = torch.where(7 * _power(e.long() - 1) >= top, e - 1, e)
        e = torch.where(7 * _power(e.long()) < top, e + 1, e).clamp(min=-126)
        step = _power(e.long())
        best, at = torch.full_like(a, math.inf), torch.zeros_like(a)
        for k in prefer.tolist():
            d = (a - grid[k] * step).abs()
            near = d < best
            best, at = torch.where(near, d, best), torch.where(near, grid[k] * step, at)
        out[r:r + 512] = at.view(p.shape[0], -1)[:, :cols] * torch.where(p < 0, -1.0, 1.0)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "recode":
        return _exact_recode(s["w"])
    if case["op"] == "gemv":
        parts = [s["x"].double() @ _real(c, z, case["cols"]).T
                 for c, z in zip(s["codes"].split(1024), s["scales"].split(1024))]
        return torch.cat(parts, 1)
    x, k, i = s["x"].double(), case["top_k"], case["inter"]
    logits = (x[:, None, :] * s["router"].double()[None]).sum(-1)
    top = logits.amax(-1, keepdim=True)
    p = 1 / (1 + torch.exp(-logits)) if case["scoring"] == "sigmoid" else torch.exp(logits - top)
    if case["scoring"] == "softmax":
        p = p / p.sum(-1, keepdim=True)
    value = (logits if s["bias"] is None else p + s["bias"].double()).tolist()
    ids = [sorted((j for j, v in enumerate(row) if v > -math.inf), key=lambda j: (-row[j], j))[:k] for row in value]
    y = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device=x.device)
    weights = torch.zeros(case["tokens"], k, dtype=torch.float64, device=x.device)
    for t, row in enumerate(ids):
        w = p[t, row]
        weights[t, :len(row)] = w / w.sum() if case["renorm"] else w
    for e in range(case["experts"]):
        at = [(t, row.index(e)) for t, row in enumerate(ids) if e in row]
        if not at:
            continue
        if case["kind"] == "fp4":
            gu = _real(s["gate_up"][0][e], s["gate_up"][1][e], case["hidden"])
            dn = _real(s["down"][0][e], s["down"][1][e], i)
        else:
            gu, dn = s["gate_up"][e].double(), s["down"][e].double()
        ts = torch.tensor([t for t, _ in at], device=x.device)
        r = x[ts] @ gu.T
        a = r[:, :i] / (1 + torch.exp(-r[:, :i])) * r[:, i:]
        y.index_add_(0, ts, (a * weights[ts, torch.tensor([j for _, j in at], device=x.device)][:, None]) @ dn.T)
    return y, None, weights
