"""GPU tests of fp4_moe at the top of binary32's range: products whose weights bring values near 2^127 back are finite, row by row
as in groups.  Bounds as in tests/test_gpu_moe.py."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
import kv_reference as R
from test_gpu_moe import Layer, d, logits_of

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


@pytest.mark.parametrize("T", [1, 6, 40])
def test_the_largest_activations(T):
    """Activations of 3.395e38 weighed with 6 2^-6."""
    E, H, I = 2, 32, 32
    z = lambda *s: np.zeros(s, np.uint8)  # noqa: E731
    c1, c2, s = z(E, 2 * I, H // 2), z(E, H, I // 2), np.full((E, 2 * I, 1), 127, np.uint8)
    c2[:, :, 0] = 7                                      # the value 6 at place 0
    w1, w2 = dict(codes=d(c1), scales=d(s), outer=None), dict(codes=d(c2), scales=d(np.full((E, H, 1), 121, np.uint8)), outer=None)
    b1 = np.zeros((E, 2 * I), np.float32)
    b1[:, 0], b1[:, I] = 2.0 ** 64, np.float32(3.395e38) / 2.0 ** 64
    y = fq.fp4_moe(torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, E, device="cuda"), w1, w2,
                   fq.make_cfg(format="mxfp4"), top_k=1, b1=d(b1), out_dtype=torch.float32).cpu().numpy()
    want = np.float64(np.float32(3.395e38)) * 6 * 2.0 ** -6
    assert (np.abs(y - want) <= 2.0 ** -16 * want).all()


@pytest.mark.parametrize("T", [1, 6, 40])
def test_the_largest_inputs(T):
    """x up to 2^127 and rows of W1 of about 2^-125."""
    rng = np.random.default_rng(T)
    layer = Layer("mxfp4", "none", 3, 96, 64)
    scales = rng.integers(1, 4, tuple(layer.w1["scales"].shape)).astype(np.uint8)
    layer.v1 = R.decode(layer.w1["codes"].cpu().numpy(), scales, "mxfp4")
    layer.w1["scales"] = d(scales)
    x = torch.from_numpy(rng.normal(0, 1, (T, 96)).clip(-1, 1) * 2.0 ** 127).to(torch.bfloat16)
    layer.check(x, logits_of(rng, T, 3), 2, out_dtype=torch.float32)


@pytest.mark.parametrize("T", [1, 6, 40])
@pytest.mark.parametrize("byte,e", [(0, 46), (1, 46), (6, 44), (7, 44), (8, 44), (251, -60), (252, -60)])
def test_the_ends_of_mxfp4_scales(T, byte, e):
    """W2 of 2^-127 and of 2^125 by activations of about 2^(2 e) (biases alone), one block of NaN."""
    rng = np.random.default_rng(byte)
    layer = Layer("mxfp4", "none", 2, 64, 96, bias=True)
    layer.w1["codes"].zero_()
    layer.v1[:] = 0
    layer.b1 = (np.abs(layer.b1) * 2.0 ** e + 2.0 ** e).astype(np.float32)
    layer.b2[:] = 0
    scales = np.full(tuple(layer.w2["scales"].shape), byte, np.uint8)
    layer.v2 = R.decode(layer.w2["codes"].cpu().numpy(), scales, "mxfp4")
    layer.w2["scales"] = d(scales)
    x, l = torch.zeros(T, 64, dtype=torch.bfloat16), logits_of(rng, T, 2)
    layer.check(x, l, 2, out_dtype=torch.float32)
    scales[1, 5, 2] = 0xFF
    layer.w2["scales"] = d(scales)
    y = layer.run(x, l, 2)
    assert y[:, 5].isnan().all() and y.isnan().sum() == T
