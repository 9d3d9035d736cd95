"""The decode example at a small size: its own check of the logits, and the same
tokens from the graph as from eager steps."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_moe_decode_example():
    spec = importlib.util.spec_from_file_location("moe_decode", os.path.join(ROOT, "examples", "moe_decode.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    size = ["--batch", "3", "--layers", "2", "--hidden", "256", "--inter", "96", "--experts", "8",
            "--top-k", "2", "--vocab", "500", "--steps", "6", "--seed", "5"]
    _, tokens = ex.main(size)
    args = {size[i][2:].replace("-", "_"): int(size[i + 1]) for i in range(0, len(size), 2)}
    model = ex.Model(type("Args", (), args), torch.device("cuda:0"))
    last = torch.arange(3, device="cuda:0")
    for row in tokens:
        last = model.step(last)[0].argmax(1)
        assert torch.equal(row, last)
