"""Greedy decoding with 4-bit weights: every layer a mixture of experts, the
output head a 4-bit matrix-vector product, a whole step one HIP graph.

  python examples/moe_decode.py [--layers 4 --hidden 2048 --inter 768 ...]
  python examples/moe_decode.py --heads 16 --kv-heads 4 --prompt 200

Weights are seeded noise.  Without --heads attention is left out: what stands here
then is the part of a decode step that reads the weights.  With it every layer
has attention before its experts: the prompts (of different lengths) run through
wc.prompt_attention and leave their keys and values in a 4-bit cache, and the
decode steps append to it and attend over it (wc.fp4_attention); the log
probability of every decoded token is kept (wc.token_logprobs).  The first step's
logits are checked against the same layers in plain torch operations in fp32 on
the values that the codes stand for (wc.fp4_decode, wc.fp4_cache_read), then
`--steps` tokens per sequence are decoded and timed."""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import decode_gemv_sign_amd as wc  # noqa: E402


def noise(gen, *shape, sigma=1.0):
    return (torch.randn(shape, generator=gen, device=gen.device) * sigma).to(torch.bfloat16)


class Model:
    """Weights of the layers and the head, coded once to 4 bits."""

    def __init__(self, args, device):
        gen = torch.Generator(device).manual_seed(args.seed)
        H, I, E = args.hidden, args.inter, args.experts
        self.top_k = args.top_k
        self.embed = noise(gen, args.vocab, H)
        self.layers = []
        for _ in range(args.layers):
            router = noise(gen, E, H, sigma=H ** -0.5)
            gate_up = wc.fp4_encode(noise(gen, E, 2 * I, H, sigma=H ** -0.5))
            down = wc.fp4_encode(noise(gen, E, H, I, sigma=I ** -0.5))
            self.layers.append((router, gate_up, down))
        self.head = wc.fp4_encode(noise(gen, args.vocab, H, sigma=H ** -0.5))
        self.attention = Attention(args, gen, device) if getattr(args, "heads", 0) else None

    def coded_bytes(self):
        fp4 = [q for layer in self.layers for q in layer[1:]] + [self.head]
        if self.attention:
            fp4 += self.attention.qkv + self.attention.out
        return sum(q.codes.numel() + q.scales.numel() for q in fp4)

    def step(self, tokens):
        """Logits [batch, vocab] fp32 for the sequences' last tokens, and every
        layer's chosen experts."""
        h = self.embed[tokens].float()
        chosen = []
        if self.attention:
            self.attention.next_places()
        for i, (router, gate_up, down) in enumerate(self.layers):
            if self.attention:
                h = h + self.attention.step(i, normed(h))
            y, ids, _ = wc.moe(normed(h), router, gate_up, down, self.top_k)
            chosen.append(ids)
            h = h + y.float()
        return wc.fp4_gemv(self.head, normed(h)), chosen

    def plain_step(self, tokens, chosen):
        """step()'s logits in elementary operations, fp32, for the same experts
        (near ties may be chosen otherwise); y is rounded to BF16 as there."""
        h = self.embed[tokens].float()
        for i, ((router, gate_up, down), ids) in enumerate(zip(self.layers, chosen)):
            if self.attention:
                h = h + self.attention.plain_step(i, normed(h))
            x = normed(h).float()
            weights = (x @ router.float().T).gather(1, ids.long()).softmax(1)
            y = torch.zeros_like(h)
            gu, dn = wc.fp4_decode(gate_up), wc.fp4_decode(down)
            for t in range(len(tokens)):
                for w, e in zip(weights[t], ids[t].tolist()):
                    gate, up = (gu[e].float() @ x[t]).chunk(2)
                    y[t] += w * (dn[e].float() @ (torch.nn.functional.silu(gate) * up))
            h = h + y.to(torch.bfloat16).float()
        return normed(h).float() @ wc.fp4_decode(self.head).float().T


class Attention:
    """Every layer's projections, coded to 4 bits, its 4-bit cache and the place of
    each sequence in it."""
    PAGE = 64

    def __init__(self, args, gen, device):
        H, self.hq, self.hk, self.dim = args.hidden, args.heads, args.kv_heads, args.head_dim
        self.qkv = [wc.fp4_encode(noise(gen, (self.hq + 2 * self.hk) * self.dim, H, sigma=H ** -0.5))
                    for _ in range(args.layers)]
        self.out = [wc.fp4_encode(noise(gen, H, self.hq * self.dim, sigma=(self.hq * self.dim) ** -0.5))
                    for _ in range(args.layers)]
        # prompts of different lengths, and room for the steps behind them
        self.prompts = [max(1, args.prompt * (i + 1) // args.batch) for i in range(args.batch)]
        width = -(-(args.prompt + args.steps + 2) // self.PAGE)
        self.caches = [wc.fp4_cache(args.batch * width, self.PAGE, self.hk, self.dim, device)
                       for _ in range(args.layers)]
        self.table = torch.arange(args.batch * width, dtype=torch.int32, device=device).view(args.batch, width)
        self.lengths = torch.tensor(self.prompts, dtype=torch.int32, device=device)
        self.starts = torch.tensor([0] + self.prompts, device=device).cumsum(0).int()
        place = torch.cat([torch.arange(n) for n in self.prompts]).to(device)
        seq = torch.repeat_interleave(torch.arange(args.batch), torch.tensor(self.prompts)).to(device)
        self.prompt_slots = self.table[seq, place // self.PAGE].long() * self.PAGE + place % self.PAGE
        self.slots = None

    def split(self, x):
        """Queries, keys and values [tokens, heads, dim] of the projection's rows."""
        x = x.to(torch.bfloat16).unflatten(1, (-1, self.dim))
        return x[:, :self.hq], x[:, self.hq:self.hq + self.hk], x[:, self.hq + self.hk:]

    def project(self, q, x):
        """Rows x times a coded matrix, 256 of them at a time."""
        return torch.cat([wc.fp4_gemv(q, p.contiguous()) for p in x.split(256)])

    def prefill(self, i, x):
        """The prompts' rows through layer i, their keys and values into its cache."""
        q, k, v = self.split(self.project(self.qkv[i], x))
        wc.fp4_cache_append(self.caches[i], k, v, self.prompt_slots)
        o, _ = wc.prompt_attention(q, k, v, self.starts)
        return self.project(self.out[i], o.flatten(1))

    def next_places(self):
        """Each sequence grows by a token."""
        at = self.lengths.long()
        page = self.table.gather(1, (at // self.PAGE)[:, None])[:, 0].long()
        self.slots = page * self.PAGE + at % self.PAGE
        self.lengths += 1

    def step(self, i, x):
        q, k, v = self.split(wc.fp4_gemv(self.qkv[i], x))
        wc.fp4_cache_append(self.caches[i], k, v, self.slots)
        o, _ = wc.fp4_attention(q, self.caches[i], self.table, self.lengths)
        return wc.fp4_gemv(self.out[i], o.flatten(1))

    def plain_step(self, i, x):
        """step(), whose tokens are in the cache already, in elementary operations."""
        q, _, _ = self.split(x.float() @ wc.fp4_decode(self.qkv[i]).float().T)
        rows = []
        for b, n in enumerate(self.lengths.tolist()):
            p = torch.arange(n, device=x.device)
            k, v = wc.fp4_cache_read(self.caches[i], self.table[b, p // self.PAGE].long() * self.PAGE + p % self.PAGE)
            group = self.hq // self.hk
            k, v = (t.float().repeat_interleave(group, 1).transpose(0, 1) for t in (k, v))  # [heads, n, dim]
            s = (k @ q[b].float()[:, :, None])[..., 0] * self.dim ** -0.5
            rows.append((s.softmax(-1)[:, None] @ v).flatten())
        o = torch.stack(rows).to(torch.bfloat16).float()
        return o @ wc.fp4_decode(self.out[i]).float().T


def prefill(model, tokens):
    """The prompts' tokens through every layer (their experts 64 tokens at a time)."""
    h = model.embed[tokens].float()
    for i, (router, gate_up, down) in enumerate(model.layers):
        h = h + model.attention.prefill(i, normed(h))
        x = normed(h)
        h = h + torch.cat([wc.moe(p, router, gate_up, down, model.top_k)[0] for p in x.split(64)]).float()


def normed(h):
    return (h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6)).to(torch.bfloat16)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in [("batch", 4), ("layers", 4), ("hidden", 2048), ("inter", 768), ("experts", 64),
                        ("top-k", 8), ("vocab", 32000), ("steps", 64), ("seed", 1), ("heads", 0), ("kv-heads", 4),
                        ("head-dim", 128), ("prompt", 64)]:
        p.add_argument(f"--{name}", type=int, default=value)
    args = p.parse_args(argv)
    model = Model(args, torch.device("cuda:0"))
    tokens = torch.arange(args.batch, device="cuda:0") % args.vocab
    if model.attention:
        gen = torch.Generator("cuda:0").manual_seed(args.seed + 1)
        prefill(model, torch.randint(args.vocab, (sum(model.attention.prompts),), generator=gen, device="cuda:0"))

    logits, chosen = model.step(tokens)
    plain = model.plain_step(tokens, chosen)
    # a rounding to BF16 may fall the other way in either: 2^-8 of a value, a few times over the layers
    off = ((logits - plain).abs().amax() / plain.abs().amax()).item()
    print(f"first step: logits off by {off:.2e} of their largest", flush=True)
    if not off <= 4 * args.layers * 2.0 ** -8:
        raise SystemExit("the kernels' logits differ from the plain ones")

    # one step as a graph: the next tokens replace the last ones in place
    graph, out = torch.cuda.CUDAGraph(), torch.empty(args.steps, args.batch, dtype=torch.int64, device="cuda:0")
    score = torch.zeros(args.batch, device="cuda:0")  # log probability of what a sequence decoded
    if model.attention:
        model.attention.lengths -= 1  # the checked step's token is written again
    with torch.cuda.graph(graph):
        logits, _ = model.step(tokens)
        tokens.copy_(logits.argmax(1))
        if model.attention:
            score += wc.token_logprobs(logits, tokens)[0]
    torch.cuda.synchronize()
    start = time.perf_counter()
    for i in range(args.steps):
        graph.replay()
        out[i].copy_(tokens)
    torch.cuda.synchronize()
    us = (time.perf_counter() - start) / args.steps * 1e6
    print(f"{args.steps} steps of {args.batch} sequences: {us:.0f} us a step, "
          f"{args.batch * 1e6 / us:.0f} tokens/s, {model.coded_bytes() / 2**20:.0f} MiB of coded weights")
    if model.attention:
        held = model.attention.lengths.tolist()
        print(f"cache: {min(held)} to {max(held)} tokens a sequence; mean log probability of a decoded token "
              f"{score.mean().item() / args.steps:.3f}")
        return off, out, score
    return off, out


if __name__ == "__main__":
    main()
