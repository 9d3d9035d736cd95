"""The decode example with attention: the operators of a serving step one after the
other (prompts into the 4-bit cache, steps over it, experts, head, log
probabilities), as one graph and step by step."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_sign_amd as wc  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("moe_decode", os.path.join(ROOT, "examples", "moe_decode.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


SIZE = ["--batch", "3", "--layers", "2", "--hidden", "256", "--inter", "96", "--experts", "8", "--top-k", "2",
        "--vocab", "500", "--steps", "6", "--seed", "5", "--heads", "6", "--kv-heads", "2", "--head-dim", "64",
        "--prompt", "70"]


def test_decode_with_attention():
    ex = load()
    _, tokens, score = ex.main(SIZE)  # checks the first step's logits itself
    args = {SIZE[i][2:].replace("-", "_"): int(SIZE[i + 1]) for i in range(0, len(SIZE), 2)}
    model = ex.Model(type("Args", (), args), torch.device("cuda:0"))
    gen = torch.Generator("cuda:0").manual_seed(args["seed"] + 1)
    ex.prefill(model, torch.randint(args["vocab"], (sum(model.attention.prompts),), generator=gen, device="cuda:0"))
    last, total = torch.arange(3, device="cuda:0"), torch.zeros(3, device="cuda:0")
    for row in tokens:
        logits, _ = model.step(last)
        last = logits.argmax(1)
        total += wc.token_logprobs(logits, last)[0]
        assert torch.equal(row, last)
    assert torch.equal(total, score)
    assert model.attention.lengths.tolist() == [n + 6 for n in model.attention.prompts]


def test_a_prompt_in_one_pass_or_token_by_token():
    """The last rows of prompt_attention on the values that the cache holds equal
    fp4_attention over the cache: 16 bits of a weight there and 8 here, each output
    rounded once (2^-8 of a value, twice, and 2^-8 of the terms that it is made of)."""
    torch.manual_seed(3)
    dev, heads, kv, dim, page = "cuda:0", 8, 2, 128, 64
    lengths = [200, 1, 65, 130]
    starts = torch.tensor([0] + lengths, device=dev).cumsum(0).int()
    n = sum(lengths)
    fused = torch.randn(n, heads + 2 * kv, dim, device=dev).bfloat16()
    cache = wc.fp4_cache(16, page, kv, dim, dev)
    table = torch.arange(16, dtype=torch.int32, device=dev).view(4, 4)
    place = torch.cat([torch.arange(m) for m in lengths]).to(dev)
    seq = torch.repeat_interleave(torch.arange(4), torch.tensor(lengths)).to(dev)
    slots = table[seq, place // page].long() * page + place % page
    wc.fp4_cache_append(cache, fused[:, heads:heads + kv], fused[:, heads + kv:], slots)
    k, v = wc.fp4_cache_read(cache, slots)
    out, lse = wc.prompt_attention(fused[:, :heads], k, v, starts)
    last = (starts[1:] - 1).long()
    got, got_lse = wc.fp4_attention(fused[last][:, :heads], cache, table,
                                    torch.tensor(lengths, dtype=torch.int32, device=dev))
    terms = v.abs().float().amax()
    assert bool(((got.float() - out[last].float()).abs() <= 2.0 ** -8 * (2.1 * got.float().abs() + 2.1 * terms)).all())
    # scores of 128 products, |s| below 20: far less than 1e-4
    assert bool(((got_lse - lse[last]).abs() <= 1e-4).all())
