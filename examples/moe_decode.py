"""Greedy decoding with 4-bit weights: every layer a mixture of experts, the
output head a 4-bit matrix-vector product, a whole step one HIP graph.

  python examples/moe_decode.py [--layers 4 --hidden 2048 --inter 768 ...]

Weights are seeded noise (attention is left out: what stands here is the part of
a decode step that reads the weights).  The first step's logits are checked
against the same layers in plain torch operations in fp32 on the values that the
codes stand for (wc.fp4_decode), then `--steps` tokens per sequence are decoded
and timed."""
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

    def coded_bytes(self):
        fp4 = [q for layer in self.layers for q in layer[1:]] + [self.head]
        return sum(q.codes.numel() + q.scales.numel() for q in fp4)

    def step(self, tokens):
        """Logits [batch, vocab] fp32 for the sequences' last tokens, and every
        layer's chosen experts."""
        h = self.embed[tokens].float()
        chosen = []
        for router, gate_up, down in self.layers:
            y, ids, _ = wc.moe(normed(h), router, gate_up, down, self.top_k)
            chosen.append(ids)
            h = h + y.float()
        return wc.fp4_gemv(self.head, normed(h)), chosen

    def plain_step(self, tokens, chosen):
        """step()'s logits in elementary operations, fp32, for the same experts
        (near ties may be chosen otherwise); y is rounded to BF16 as there."""
        h = self.embed[tokens].float()
        for (router, gate_up, down), ids in zip(self.layers, chosen):
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


def normed(h):
    return (h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6)).to(torch.bfloat16)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in [("batch", 4), ("layers", 4), ("hidden", 2048), ("inter", 768), ("experts", 64),
                        ("top-k", 8), ("vocab", 32000), ("steps", 64), ("seed", 1)]:
        p.add_argument(f"--{name}", type=int, default=value)
    args = p.parse_args(argv)
    model = Model(args, torch.device("cuda:0"))
    tokens = torch.arange(args.batch, device="cuda:0") % args.vocab

    logits, chosen = model.step(tokens)
    plain = model.plain_step(tokens, chosen)
    # a rounding to BF16 may fall the other way in either: 2^-8 of a value, a few times over the layers
    off = ((logits - plain).abs().amax() / plain.abs().amax()).item()
    print(f"first step: logits off by {off:.2e} of their largest", flush=True)
    if not off <= 4 * args.layers * 2.0 ** -8:
        raise SystemExit("the kernels' logits differ from the plain ones")

    # one step as a graph: the next tokens replace the last ones in place
    graph, out = torch.cuda.CUDAGraph(), torch.empty(args.steps, args.batch, dtype=torch.int64, device="cuda:0")
    with torch.cuda.graph(graph):
        tokens.copy_(model.step(tokens)[0].argmax(1))
    torch.cuda.synchronize()
    start = time.perf_counter()
    for i in range(args.steps):
        graph.replay()
        out[i].copy_(tokens)
    torch.cuda.synchronize()
    us = (time.perf_counter() - start) / args.steps * 1e6
    print(f"{args.steps} steps of {args.batch} sequences: {us:.0f} us a step, "
          f"{args.batch * 1e6 / us:.0f} tokens/s, {model.coded_bytes() / 2**20:.0f} MiB of coded weights")
    return off, out


if __name__ == "__main__":
    main()
