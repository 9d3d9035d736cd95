"""Attention of a serving step with its 4-bit cache, and the scores of what the
output head gives: what is timed, and the plain form of each operator.

append    new keys and values into the 4-bit cache (wc.fp4_cache_append), and
          the values that it then holds (wc.fp4_cache_read).
cache     attention of 1..16 new tokens per sequence over a paged cache held in
          4 bits (wc.fp4_attention).
prompt    causal attention over whole prompts of different lengths, packed one
          after the other (wc.prompt_attention).
logprobs  log probabilities of given tokens, the entropy and the top
          alternatives of every row of logits (wc.token_logprobs).

Where `own` is false, run() computes with elementary torch operations.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 32  # columns that share a scale
TILE = 32   # tokens of a tile of the cache


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # one decode step of a batch: latency counts
        {"name": "append 32 tokens", "op": "append", "tokens": 32, "run": 1, "kv_heads": 8, "dim": 128,
         "page": 64},
        # the keys and values of a prompt, as slices of the fused projection's output
        {"name": "append 8192 tokens", "op": "append", "tokens": 8192, "run": 64, "kv_heads": 8, "dim": 128,
         "page": 64},
        # one sequence, one token: latency counts
        {"name": "cache b1 1500", "op": "cache", "batch": 1, "new": 1, "longest": 1500, "spread": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0},
        # a decode batch of sequences of very different lengths, one place of it unused
        {"name": "cache b32 to 8192", "op": "cache", "batch": 32, "new": 1, "longest": 8192, "spread": 64, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0},
        # few long sequences: bandwidth counts
        {"name": "cache b4 65536", "op": "cache", "batch": 4, "new": 1, "longest": 65536, "spread": 1, "heads": 64,
         "kv_heads": 8, "dim": 128, "page": 256, "window": 0},
        # several proposed tokens checked at once, a head of keys for each head, a sliding window
        {"name": "cache b16 new4 64", "op": "cache", "batch": 16, "new": 4, "longest": 4001, "spread": 16, "heads": 16,
         "kv_heads": 16, "dim": 64, "page": 32, "window": 1000},
        # a short prompt: latency counts
        {"name": "prompt 100", "op": "prompt", "batch": 1, "longest": 100, "spread": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "window": 0},
        # prompts of a serving batch
        {"name": "prompt b12 to 2048", "op": "prompt", "batch": 12, "longest": 2048, "spread": 16, "heads": 32,
         "kv_heads": 8, "dim": 128, "window": 0},
        # one long prompt: the matrix cores' rate counts
        {"name": "prompt 16384", "op": "prompt", "batch": 1, "longest": 16384, "spread": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "window": 0},
        # odd lengths, narrow heads, a sliding window
        {"name": "prompt b3 4001 64", "op": "prompt", "batch": 3, "longest": 4001, "spread": 3, "heads": 12,
         "kv_heads": 4, "dim": 64, "window": 1000},
        # the tokens of a decode step, logits as the 4-bit head gives them: latency counts
        {"name": "logprobs 4x32000", "op": "logprobs", "rows": 4, "vocab": 32000, "top": 5, "kind": "f32"},
        # scoring a text: a row for every token, of an odd length
        {"name": "logprobs 2048x100003", "op": "logprobs", "rows": 2048, "vocab": 100003, "top": 20, "kind": "bf16"},
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    kv = rng.choice((1, 2, 4, 8, 16))
    group = rng.choice((1, 2, 3, 4, 5, 8, 16))
    return kv * min(group, 64 // kv), kv


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    while True:
        op = rng.choice(("append", "cache", "cache", "prompt", "prompt", "logprobs"))
        heads, kv = _heads(rng)
        dim = rng.choice((128, 128, 64, 96, 192, 256, 32))
        if op == "append":
            c = {"op": op, "tokens": _spread(rng, 1, 8192), "kv_heads": kv, "dim": dim,
                 "page": rng.choice((32, 64, 128, 256))}
            c["run"] = rng.choice((1, rng.randint(1, c["page"]), c["page"]))
        elif op == "cache":
            c = {"op": op, "batch": _spread(rng, 1, 64), "new": rng.choice((1, 1, 1, 2, 5, 8, 16)),
                 "longest": _spread(rng, 1, 65536), "spread": _spread(rng, 1, 100), "heads": heads, "kv_heads": kv,
                 "dim": dim, "page": rng.choice((32, 64, 128, 256)), "window": 0}
        elif op == "prompt":
            c = {"op": op, "batch": _spread(rng, 1, 32), "longest": _spread(rng, 1, 16384),
                 "spread": _spread(rng, 1, 100), "heads": heads, "kv_heads": kv, "dim": dim, "window": 0}
        else:
            c = {"op": op, "rows": _spread(rng, 1, 4096), "vocab": _spread(rng, 1000, 260000),
                 "top": rng.choice((0, 1, 5, 20, 32)), "kind": rng.choice(("f32", "bf16"))}
        if op in ("cache", "prompt") and rng.random() < 0.3:
            c["window"] = _spread(rng, 1, c["longest"])
        # the plain form computes every pair of a padded batch
        if _cost(c) <= most[op] and _padded(c) <= 5e9:
            return c


def lengths(case):
    """The sequences' lengths: from `longest` down to `longest / spread`, evenly
    by their logarithm, the last of eight or more an empty one."""
    n = case["batch"]
    v = [max(1, int(case["longest"] * case["spread"] ** (-i / max(1, n - 1)))) for i in range(n)]
    if n >= 8:
        v[-1] = 0
    return v


def _pairs(case):
    """Pairs of a query and a position that it attends to, of one head."""
    total, w = 0, case["window"]
    for n in lengths(case):
        new = case["new"] if case["op"] == "cache" else n
        lo = max(0, n - new)  # the first query's position
        if w:
            short = max(lo, min(n, w))  # below it all earlier positions count
            total += (short * (short + 1) - lo * (lo + 1)) // 2 + (n - short) * w
        else:
            total += (n * (n + 1) - lo * (lo + 1)) // 2
    return total


def _read(case):
    """Cached positions of a head that some query attends to."""
    w, new = case["window"], case["new"]
    return sum(min(n, new + w - 1) if w else n for n in lengths(case))


def _padded(case):
    """Scores that the plain form holds."""
    if case["op"] == "cache":
        return case["batch"] * case["heads"] * case["new"] * case["longest"]
    if case["op"] == "prompt":
        return case["batch"] * case["heads"] * case["longest"] ** 2
    return 0


# ---- work --------------------------------------------------------------------

def work(case):
    if case["op"] == "append":
        n = case["tokens"] * case["kv_heads"] * case["dim"]
        # append reads both in 16 bits and writes them in 4.25, the read-back the other way
        return {"bytes": 2 * (2 * 2 * n + 2 * n * 17 // 32 + 8 * case["tokens"]), "flops": 0}
    if case["op"] == "logprobs":
        rows, vocab = case["rows"], case["vocab"]
        return {"bytes": rows * vocab * (4 if case["kind"] == "f32" else 2) + rows * (16 + 8 * case["top"]),
                "flops": 4 * rows * vocab}
    heads, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    flops = 4 * dim * heads * _pairs(case)
    if case["op"] == "cache":
        queries = case["batch"] * case["new"] * heads
        return {"bytes": _read(case) * kv * dim * 34 // 32 + queries * (4 * dim + 4), "flops": flops}
    return {"bytes": sum(lengths(case)) * (4 * dim * (heads + kv) + 4 * heads), "flops": flops}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 150)


# ---- the plain forms ---------------------------------------------------------

VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # by the code's low three bits; bit 3 is the sign


def plain_encode(w):
    """codes [.., cols / 2] and scales [.., cols / 32] of BF16 w [.., cols], cols
    a multiple of 32: a group's scale is 2^(e - 127), the smallest (e >= 1) that
    keeps every |w| within 7 of it; weights round to the nearest of the 16 values,
    ties to the even code.  (No group here holds an infinity, a NaN or the
    largest numbers of BF16.)"""
    f = w.float().reshape(*w.shape[:-1], -1, GROUP)
    top = (f.view(torch.int32) >> 16 & 0x7FFF).amax(-1)
    e = ((top >> 7) - 2 + ((top & 0x7F) > 0x60).int()).clamp(min=1)
    a = f.abs() * ((254 - e) << 23).view(torch.float32)[..., None]  # |w| / 2^(e - 127), exact
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
            + (a > 2.5).int() + (a >= 3.5).int() + (a > 5).int())
    code = (code | torch.signbit(f).int() << 3).reshape(w.shape)
    return (code[..., 0::2] | code[..., 1::2] << 4).to(torch.uint8), e.to(torch.uint8)


def plain_values(codes, scales):
    """The fp32 values that codes and scales stand for, [.., cols]."""
    v = torch.tensor(VALUES + tuple(-x for x in VALUES), device=codes.device)
    s = (torch.arange(256, device=codes.device, dtype=torch.int32) << 23).view(torch.float32)  # 2^(e - 127), e > 0
    q = codes.to(torch.int32)
    w = v[torch.stack((q & 15, q >> 4), -1)].reshape(*scales.shape, GROUP)
    return (w * s[scales.to(torch.int32)][..., None]).flatten(-2)


# A tile of the cache holds 32 tokens of one head, 34 bytes for each of the `dim`
# columns: the keys' codes, the values' codes, the keys' scales, the values'
# scales, each in the order in which a wave's lanes take them.  Token t of a tile
# is row r = 4 (t / 8) + t % 4 of half i = t / 4 % 2 for the keys, and element t % 8
# of quarter t / 8 for the values.  With G = dim / 32 groups of columns:
#   keys' codes     [half][quads of groups][part of 8 columns][row][group of the
#                   quad] dwords of 8 codes
#   values' codes   [pairs of groups][quarter][pair of columns][group of the
#                   pair][element] bytes of 2 codes
#   keys' scales    [row][half][group]
#   values' scales  [quarter][group][element]

def _split(groups, most):
    return [min(most, groups - g) for g in range(0, groups, most)]


def plain_pack(kc, ks, vc, vs):
    """Tiles [.., 34 dim] from codes [.., 32, dim / 2] and scales [.., 32, dim / 32]."""
    lead, g = kc.shape[:-2], ks.shape[-1]
    n = len(lead)
    axes = lambda *p: tuple(range(n)) + tuple(n + i for i in p)  # noqa: E731
    # tokens as [quarter, half, place of 4]; columns as [group, part, 4 bytes]
    k = kc.reshape(*lead, 4, 2, 4, g, 4, 4).permute(axes(1, 4, 0, 2, 3, 5))
    k = torch.cat([p.flatten(n + 1) for p in k.split(_split(g, 4), n + 4)], n + 1)
    v = vc.reshape(*lead, 4, 8, g, 16).permute(axes(0, 3, 2, 1))
    v = torch.cat([p.flatten(n) for p in v.split(_split(g, 2), n + 2)], n)
    a = ks.reshape(*lead, 4, 2, 4, g).permute(axes(0, 2, 1, 3))
    b = vs.reshape(*lead, 4, 8, g).permute(axes(0, 2, 1))
    return torch.cat([p.reshape(*lead, -1) for p in (k, v, a, b)], -1).contiguous()


def plain_unpack(tiles, dim):
    """The codes and scales that plain_pack takes, of tiles [.., 34 dim]."""
    lead, g = tiles.shape[:-1], dim // GROUP
    n = len(lead)
    axes = lambda *p: tuple(range(n)) + tuple(n + i for i in p)  # noqa: E731
    k, v, a, b = tiles.split((16 * dim, 16 * dim, 2 * dim // 2, 2 * dim // 2), -1)
    k = k.reshape(*lead, 2, -1).split([256 * w for w in _split(g, 4)], n + 1)
    k = torch.cat([p.reshape(*lead, 2, 4, 4, 4, -1, 4) for p in k], n + 4)
    v = v.split([1024 * w // 2 for w in _split(g, 2)], n)
    v = torch.cat([p.reshape(*lead, 4, 16, -1, 8) for p in v], n + 2)
    return (k.permute(axes(2, 0, 3, 4, 1, 5)).reshape(*lead, TILE, dim // 2),
            a.reshape(*lead, 4, 4, 2, g).permute(axes(0, 2, 1, 3)).reshape(*lead, TILE, g),
            v.permute(axes(0, 3, 2, 1)).reshape(*lead, TILE, dim // 2),
            b.reshape(*lead, 4, g, 8).permute(axes(0, 2, 1)).reshape(*lead, TILE, g))


def plain_append(s):
    """Codes of the new rows into their slots of the cache, and what those hold."""
    out = []
    for x in (s["k"], s["v"]):
        codes, scales = plain_encode(x)
        held_codes = codes.new_zeros(s["slot_count"], *codes.shape[1:])
        held_scales = scales.new_zeros(s["slot_count"], *scales.shape[1:])
        held_codes[s["slots"]], held_scales[s["slots"]] = codes, scales
        out.append(plain_values(held_codes[s["slots"]], held_scales[s["slots"]]).to(torch.bfloat16))
    return tuple(out)


def _attend(q, k, v, positions, ends, scale, window):
    """q [B, H, group, n, D], k and v [B, H, L, D] in fp32; positions [B, n] of
    the queries; ends [B]: positions that exist.  (o [B, H, group, n, D], lse)"""
    at = torch.arange(k.shape[2], device=q.device)
    ok = (at <= positions[..., None]) & (at < ends[:, None, None])
    if window:
        ok &= at > positions[..., None] - window
    b, h, g, n, d = q.shape
    s = (q.reshape(b * h, g * n, d) @ k.reshape(b * h, -1, d).transpose(1, 2)).view(b, h, g, n, -1)
    s.mul_(scale).masked_fill_(~ok[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    s.sub_(top.masked_fill(torch.isneginf(top), 0.0)).exp_()
    total = s.sum(-1, keepdim=True)
    o = (s.view(b * h, g * n, -1) @ v.reshape(b * h, -1, d)).view(q.shape)
    o = torch.where(total > 0, o / total, 0.0)
    return o, (top + torch.log(total))[..., 0]


def plain_cache(s):
    case = s["case"]
    b, n, d = case["batch"], case["new"], case["dim"]
    tiles = s["cache"][s["table"].clamp(min=0).long()].transpose(1, 2).flatten(2, 3)  # [B, H, tiles, 34 D]
    kc, ks, vc, vs = plain_unpack(tiles, d)
    k, v = (plain_values(c, e).flatten(2, 3) for c, e in ((kc, ks), (vc, vs)))
    at = s["lengths"].long()
    q = s["q"].float().view(b, n, case["kv_heads"], -1, d).permute(0, 2, 3, 1, 4)
    positions = at[:, None] - n + torch.arange(n, device=DEV)
    o, lse = _attend(q, k, v, positions, at, s["scale"], case["window"])
    return (o.permute(0, 3, 1, 2, 4).reshape(s["q"].shape).to(torch.bfloat16),
            lse.permute(0, 3, 1, 2).reshape(s["q"].shape[:-1]))


def plain_prompt(s):
    case = s["case"]
    d, kv, longest = case["dim"], case["kv_heads"], case["longest"]
    starts = s["starts"].long()
    ends = starts.diff()
    at = torch.arange(longest, device=DEV)
    real = at < ends[:, None]                                 # [B, longest]
    take = (starts[:-1, None] + at).clamp(max=s["q"].shape[0] - 1)
    q, k, v = (s[x].float()[take].view(case["batch"], longest, kv, -1, d) for x in "qkv")
    o, lse = _attend(q.permute(0, 2, 3, 1, 4), k[:, :, :, 0].transpose(1, 2), v[:, :, :, 0].transpose(1, 2),
                     at.expand(case["batch"], -1), ends, s["scale"], case["window"])
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[real]          # [tokens, heads, D]
    return o.to(torch.bfloat16), lse.permute(0, 3, 1, 2).flatten(2, 3)[real]


def plain_logprobs(s):
    x, tokens, top = s["logits"].float(), s["tokens"].long(), s["case"]["top"]
    m = x.amax(-1, keepdim=True)
    u = x - m
    p = torch.exp(u)
    total = p.sum(-1, keepdim=True)
    lp = u - torch.log(total)
    entropy = -torch.where(p > 0, p * lp, 0.0).sum(-1) / total[:, 0]
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :top]
    best = lp.gather(1, order)
    return (lp.gather(1, tokens[:, None])[:, 0], entropy,
            torch.where(torch.isneginf(best), -1, order).int(), best)


# ---- one pass ----------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def keys(*shape):
        """Rows of which a few channels are strong, as keys have them."""
        k = normal(*shape)
        k[..., :: max(1, shape[-1] // 4)] *= 4.0
        return k.to(torch.bfloat16)

    s = {"case": case}
    if case["op"] == "logprobs":
        rows, vocab = case["rows"], case["vocab"]
        x = normal(rows, vocab) * 2.5
        sure = torch.randint(vocab, (rows,), generator=g, device=DEV)  # the token that a model would rather take
        x[torch.arange(rows, device=DEV), sure] += 12.0 * torch.rand(rows, generator=g, device=DEV)
        x[:, : vocab // 50] = -math.inf                        # tokens that a grammar rules out
        s["logits"] = x.to(torch.float32 if case["kind"] == "f32" else torch.bfloat16)
        other = torch.randint(vocab // 50, vocab, (rows,), generator=g, device=DEV)
        s["tokens"] = torch.where(torch.rand(rows, generator=g, device=DEV) < 0.6, sure, other)
        return s
    h, d = case["kv_heads"], case["dim"]
    s["scale"] = d ** -0.5
    if case["op"] == "append":
        t, page = case["tokens"], case["page"]
        runs = -(-t // case["run"])  # of consecutive slots, each somewhere in a page of its own
        pages = runs + 8
        # slices of one projection's output, whose rows hold two query heads for a head of keys
        fused = keys(t, 4 * h, d)
        s["k"], s["v"] = fused[:, 2 * h:3 * h], fused[:, 3 * h:]
        s["slot_count"] = pages * page
        first = torch.randint(page - case["run"] + 1, (runs,), generator=g, device=DEV)
        first += torch.randperm(pages, generator=g, device=DEV)[:runs] * page
        s["slots"] = (first[:, None] + torch.arange(case["run"], device=DEV)).flatten()[:t]
        s["cache"] = torch.zeros(pages, h, page // TILE, 34 * d, dtype=torch.uint8, device=DEV)
        return s
    lens, hq = lengths(case), case["heads"]
    if case["op"] == "prompt":
        t = sum(lens)
        fused = keys(t, hq + 2 * h, d)
        s["q"], s["k"], s["v"] = fused[:, :hq], fused[:, hq:hq + h], fused[:, hq + h:]
        s["starts"] = torch.tensor([0] + lens, device=DEV).cumsum(0).int()
        return s
    b, page = case["batch"], case["page"]
    need = torch.tensor([-(-n // page) for n in lens])
    pages = int(need.sum()) + 3
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    width = -(-case["longest"] // page)
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((b, width), -1, dtype=torch.int32, device=DEV)
    used = torch.arange(width) < need[:, None]
    table[used.to(DEV)] = order[: int(need.sum())]
    s["table"] = table
    rows = (pages, h, page // TILE, TILE, d)
    s["cache"] = plain_pack(*plain_encode(keys(*rows)), *plain_encode(keys(*rows)))
    s["q"] = keys(b, case["new"], hq, d)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        import decode_gemv_sign_amd as wc
        if op == "append":
            wc.fp4_cache_append(s["cache"], s["k"], s["v"], s["slots"])
            return wc.fp4_cache_read(s["cache"], s["slots"])
        if op == "cache":
            return wc.fp4_attention(s["q"], s["cache"], s["table"], s["lengths"], scale=s["scale"],
                                    window=s["case"]["window"])
        if op == "prompt":
            return wc.prompt_attention(s["q"], s["k"], s["v"], s["starts"], scale=s["scale"],
                                       window=s["case"]["window"])
        return wc.token_logprobs(s["logits"], s["tokens"], s["case"]["top"])
    return {"append": plain_append, "cache": plain_cache, "prompt": plain_prompt, "logprobs": plain_logprobs}[op](s)


# ---- the definitions in 64 bits ----------------------------------------------

def _nearest(w):
    """The nearest of each group's values, by distance to each of the eight
    magnitudes, of w [tokens, heads, dim]."""
    p = w.double().reshape(*w.shape[:-1], -1, GROUP)
    a = p.abs()
    top = a.amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / 7)).clamp(min=-126)
    two = lambda n: torch.ldexp(torch.ones((), dtype=torch.float64, device=w.device), n)  # noqa: E731
    e = torch.where(7 * two(e - 1) >= top, e - 1, e)
    e = torch.where(7 * two(e) < top, e + 1, e).clamp(min=-126)
    step = two(e)
    best, at = torch.full_like(a, math.inf), torch.zeros_like(a)
    for k in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: they win ties
        dist = (a - VALUES[k] * step).abs()
        near = dist < best
        best, at = torch.where(near, dist, best), torch.where(near, VALUES[k] * step, at)
    return torch.where(p < 0, -at, at).reshape(w.shape)


def _held(cache, head, pages, n, d):
    """Keys and values [n, d] of one sequence's head: every byte looked up at its place."""
    dev, page = cache.device, cache.shape[2] * TILE
    at = torch.arange(n, device=dev)
    tiles = cache[pages.long()[at // page], head, at % page // TILE]  # [n, 34 d]
    t, c, groups = (at % TILE)[:, None], torch.arange(d, device=dev)[None], d // GROUP
    grp = c // 32
    quad, pair = grp // 4, grp // 2
    wide, both = (groups - 4 * quad).clamp(max=4), (groups - 2 * pair).clamp(max=2)
    row, half = t // 8 * 4 + t % 4, t // 4 % 2
    dword = half * 64 * groups + quad * 256 + ((c % 32 // 8) * 16 + row) * wide + grp % 4
    places = (dword * 4 + c % 8 // 2,
              16 * d + pair * 1024 + ((t // 8 * 16 + c % 32 // 2) * both + grp % 2) * 8 + t % 8)
    scales = (32 * d + (row * 2 + half) * groups + grp, 33 * d + (t // 8 * groups + grp) * 8 + t % 8)
    out = []
    for place, scale in zip(places, scales):
        byte = tiles.gather(1, place).long()
        code = torch.where(c % 2 == 0, byte % 16, byte // 16)
        exp, man = code // 2 % 4, (code % 2).double()
        mag = torch.where(exp == 0, man / 2, (1 + man / 2) * torch.ldexp(torch.ones_like(man), exp - 1))
        power = torch.ldexp(torch.ones_like(man), tiles.gather(1, scale).long() - 127)
        out.append(torch.where(code >= 8, -mag, mag) * power)
    return out


def _softmax_rows(q, k, v, first, scale, window):
    """o and lse of queries q [n, D] at positions first .. over k, v [L, D], in pieces of rows."""
    o, lse = torch.zeros_like(q), torch.full(q.shape[:1], -math.inf, dtype=q.dtype, device=q.device)
    for r in range(0, q.shape[0], 4096):
        e = min(q.shape[0], r + 4096)
        hi = max(0, min(k.shape[0], first + e))
        lo = max(0, first + r - window + 1) if window else 0
        if hi <= lo:
            continue
        p = (torch.arange(r, e, device=q.device) + first)[:, None]
        at = torch.arange(lo, hi, device=q.device)[None]
        s = q[r:e] @ k[lo:hi].T * scale
        s = torch.where((at <= p) & ((at > p - window) if window else True), s, -math.inf)
        lse[r:e] = torch.logsumexp(s, -1)
        o[r:e] = torch.nan_to_num(torch.exp(s - lse[r:e, None])) @ v[lo:hi]
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _nearest(s["k"]), _nearest(s["v"])
    if case["op"] == "logprobs":
        parts = []
        for x, tok in zip(s["logits"].split(256), s["tokens"].split(256)):
            x = x.double()
            lp = x - torch.logsumexp(x, -1, keepdim=True)
            ent = -(torch.exp(lp) * lp.clamp(min=-1e4)).sum(-1)
            parts.append((lp.gather(1, tok[:, None])[:, 0], ent,
                          torch.topk(lp, case["top"], -1).values))
        lp, ent, best = (torch.cat(p) for p in zip(*parts))
        return lp, ent, None, best
    group, lens = case["heads"] // case["kv_heads"], lengths(case)
    q = s["q"].double()
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:-1], dtype=torch.float64, device=DEV)
    start = 0
    for b, n in enumerate(lens):
        for h in range(case["kv_heads"]):
            if case["op"] == "cache":
                k, v = _held(s["cache"], h, s["table"][b], n, case["dim"])
            else:
                k, v = s["k"][start:start + n, h].double(), s["v"][start:start + n, h].double()
            for j in range(h * group, (h + 1) * group):
                if case["op"] == "cache":
                    o[b, :, j], lse[b, :, j] = _softmax_rows(q[b, :, j], k, v, n - case["new"], s["scale"], case["window"])
                else:
                    o[start:start + n, j], lse[start:start + n, j] = _softmax_rows(
                        q[start:start + n, j], k, v, 0, s["scale"], case["window"])
        start += n
    return o, lse
