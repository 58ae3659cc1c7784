"""The mixture-of-experts layer example end to end, part by part against float32 from what the part
before returned, and a training step's norm between two 4-bit products.

Bounds in norm, of terms whose errors add at most in full (2^-8 is half a step of bf16):
  residual, turned queries, cached rows  the same bits: the same binary32 operations in torch;
  a norm, a projection  its result's rounding, 2^-8, and binary32 sums, 2^-12;
  attention  the same, and weights rounded to FP16, 2 x 2^-11;
  the experts  their activations' rounding, 2^-8, their result's, 2^-8, and sums, 2^-12."""
import importlib.util
import os

import pytest
import torch

import block_scaled_fp4_amax_amd as fq

pytestmark = pytest.mark.gpu

HALF, SUMS = 2.0 ** -8, 2.0 ** -12
BOUNDS = dict(residual0=0, normed0=HALF + SUMS, qkv=HALF + SUMS, q=0, k=0, v=0, attn=HALF + 2 * 2.0 ** -11 + SUMS,
              projected=HALF + SUMS, residual=0, normed=HALF + SUMS, y=2 * HALF + SUMS)


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("kw", [
    dict(steps=2, hidden=320, q_heads=8, kv_heads=2, experts=8, top_k=2, inter=96, prompts=(70, 1, 33)),
    dict(steps=1, hidden=320, q_heads=4, kv_heads=4, head_dim=128, experts=80, top_k=5, inter=160, prompts=(5,), chain=1, branches=()),
    dict(steps=2, hidden=2880, inter=736, prompts=(1100, 3), chain=9, branches=(0, 1, 1, 4, 8, 13))])
def test_layer(ex, kw):
    err = ex.main(**kw)
    assert set(err) == set(BOUNDS)
    assert all(err[k] <= BOUNDS[k] for k in err), err


def test_norm_between_products():
    """y = (norm(x + r) w) W^T over W's rowwise buffers, and the gradient of its product with c over the columnwise
    ones, which quantise W along its columns, so they are a weight of their own: dy in bf16 (half a step, 2^-8), which enters dx = r (g - n mean(n g)) + dres and dw linearly; dx is rounded to bf16 (2^-8).  Two terms of dx
    cancel only for parts along n, a 1 / sqrt(hidden) of it here, which 2^-9 covers."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.manual_seed(5)
    rows, hidden, out = 300, 320, 192
    cfg = fq.make_cfg(format="nvfp4", two_level="outer_block", outer_block_size=64, outer_2d=True)
    b = fq.fp4_cast_transpose((torch.randn(out, hidden, device="cuda") * hidden ** -0.5).bfloat16(), cfg)
    x, r, dres = (torch.randn(rows, hidden, device="cuda").bfloat16() for _ in range(3))
    c = torch.randn(rows, out, device="cuda").bfloat16()
    w = 1 + 0.1 * torch.randn(hidden, device="cuda")
    n = fq.fp4_add_rms_norm(x, w, r, eps=1e-5)
    side = lambda s: {"codes": b[s + "_codes"], "scales": b[s + "_scales"], "outer": b["row_outer"]}  # noqa: E731
    y = fq.fp4_linear(n["y"], side("row"), cfg)
    dy = fq.fp4_linear(c, side("col"), cfg, outer_transposed=True)
    g = fq.fp4_add_rms_norm_backward(dy, n["residual"], w, n["rstd"], dresidual=dres)
    kw = dict(dtype=torch.float32)
    W = fq.fp4_dequantize(b["row_codes"], b["row_scales"], b["row_outer"], out, hidden, cfg, **kw).double()
    Wt = fq.fp4_dequantize(b["col_codes"], b["col_scales"], b["row_outer"], hidden, out, cfg, outer_transposed=True, **kw).double()
    h = n["residual"].double().requires_grad_()
    v = w.double().requires_grad_()
    normed = h * (h.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * v
    want = normed @ W.t()
    ((normed * (c.double() @ Wt.t())).sum() + (h * dres.double()).sum()).backward()
    off = lambda a, b: ((a.double() - b).norm() / b.norm()).item()  # noqa: E731
    assert off(y, want) <= 2 * HALF + SUMS
    assert off(g["dx"], h.grad) <= 2 * HALF + 2.0 ** -9 + SUMS
    assert off(g["dweight"], v.grad) <= HALF + 2.0 ** -9 + SUMS
