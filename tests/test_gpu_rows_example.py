"""The example that runs the row operators together: it trains, and generating token by token gives
the logits of the whole sequence."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype,relative", [("f32", 1e-4), ("bf16", 0.1), ("f16", 0.02)])
def test_example_trains_and_generates(dtype, relative):
    """Logits of single tokens against those of the whole sequence: the states agree to FP32 rounding, so
    FP32 logits to about 1e-5 of their size; 16-bit rows may round to the neighbouring number
    (2^-8, 2^-11 of their size) at each of the blocks' five roundings."""
    spec = importlib.util.spec_from_file_location(
        "recurrent_block", os.path.join(ROOT, "examples", "recurrent_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    losses, far, size = module.main(["--dtype", dtype, "--steps", "40"])
    assert losses[-1] < 0.8 * losses[0], losses
    assert far <= relative * size, (far, size)
