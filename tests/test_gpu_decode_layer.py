"""The decode-layer example end to end: projections, cache writes and attention
together, against the same layer in float32 from what the cache holds.

Each output of the last step is the bf16 rounding (2^-8) of a product whose
activations were rounded to bf16 (2^-8) after attention weights rounded to FP16
(2 x 2^-11); errors of a row's terms add at most in full, so the relative error of the
whole (in norm) stays below 2^-8 + 2^-8 + 2^-10 + binary32 sums (2^-12)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_decode_layer():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_layer.py")
    spec = importlib.util.spec_from_file_location("decode_layer", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    err = ex.main(tokens=3, hidden=320, q_heads=8, kv_heads=2, head_dim=64, prompts=(70, 1, 33))
    assert err < 2 * 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -12
    err = ex.main(tokens=2, hidden=2880, prompts=(500, 3))
    assert err < 2 * 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -12
