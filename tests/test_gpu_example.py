"""The hybrid-layer example: a prompt continued token by token against the longer prompt at once (GPU)."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_prompts_continue_token_by_token():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hybrid_linear_attention_prefill_gb300 import build

    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_layer.py")
    spec = importlib.util.spec_from_file_location("hybrid_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # Two layers, each rounding its activations to bf16 (2^-9) and its norm's output to 8 bits (2^-4 of a
    # value, independent errors over the 512 columns of a projection: 2^-4 / sqrt(512) of the result's
    # size where they differ at all): a few per cent of the largest value bounds what the orders of the
    # same sums may do, and a wrong state or position is of its size.
    assert example.compare() < 0.05
