"""The experts of the mixture-of-experts layer example alone, within what their kernels' roundings leave: activations enter W2
with 2^-16 or less, y is rounded to bf16 (2^-8 is half a step), and sums are binary32 (2^-12)."""
import pytest

from test_gpu_moe_layer import ex  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [
    dict(steps=1, hidden=320, q_heads=8, kv_heads=2, experts=8, top_k=2, inter=96, prompts=(70, 1, 33)),
    dict(steps=1, hidden=320, q_heads=4, kv_heads=4, head_dim=128, experts=80, top_k=5, inter=160, prompts=(5,), chain=1, branches=()),
    dict(steps=1, hidden=2880, inter=736, prompts=(40, 3), chain=9, branches=(0, 1, 1, 4, 8, 13))])
def test_experts(ex, kw):  # noqa: F811
    assert ex.main(**kw)["y"] <= 2.0 ** -8 + 2.0 ** -16 + 2.0 ** -12
