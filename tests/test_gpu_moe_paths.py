"""GPU tests of fp4_moe's further paths against the same binary64 layer and bounds as tests/test_gpu_moe.py: rows of
more than one chunk of 4096 values, whose scale bytes are laid into LDS chunk by chunk, in groups of 16 and 32 pairs and row by
row; and tokens whose experts are excluded in calls of few pairs."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
from test_gpu_moe import Layer, logits_of, tokens

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


@pytest.mark.parametrize("fmt,kind,H,I", [
    ("mxfp4", "none", 4128, 64), ("mxfp4", "none", 64, 4128), ("mxfp4", "none", 8256, 64), ("nvfp4", "none", 4096, 32),
    ("nvfp4", "2d", 4160, 64), ("nvfp4", "2d", 64, 8256), ("nvfp4", "1d64", 4160, 128), ("nvfp4", "tensor", 96, 8224),
    ("amdfp4", "none", 8224, 96), ("amdfp4", "1d192", 8256, 192), ("amdfp4", "1d192", 192, 4224), ("amdfp4", "2d", 4160, 4160)])
@pytest.mark.parametrize("T,E", [(2, 2), (16, 2), (30, 2), (40, 4)])
def test_rows_of_several_chunks(fmt, kind, H, I, T, E):
    """4 pairs row by row, groups of 16 (one and more an expert), and of 32 (20 pairs an expert)."""
    rng = np.random.default_rng(H + I + T)
    layer = Layer(fmt, kind, E, H, I, bias=T == 30)
    x, l = tokens(rng, T, H), logits_of(rng, T, E)
    layer.check(x, l, 2, interleaved=T == 16, out_dtype=torch.float32)


@pytest.mark.parametrize("T,E,k", [(34, 4, 2), (35, 4, 2), (60, 4, 2), (61, 4, 2), (48, 4, 4), (49, 4, 4), (64, 7, 7), (18, 5, 5), (32, 6, 6),
                                   (64, 3, 2), (64, 10, 3)])
def test_groups_around_their_bounds(T, E, k):
    """Pairs an expert at and beside 17, 30 and 48, where groups are of 16 or 32, evenly and all of the same experts."""
    rng = np.random.default_rng(T + E)
    layer = Layer("nvfp4", "1d64", E, 192, 128, bias=True)
    x, l = tokens(rng, T, 192), logits_of(rng, T, E)
    y = layer.check(x, l, k)
    ws = fq.fp4_moe_workspace(64, E, k, 192, 128)        # of more tokens
    assert torch.equal(layer.run(x, l, k, workspace=ws), y)
    l[:, :k] += 50
    layer.check(x, l, k)


@pytest.mark.parametrize("k", [1, 2, 3])
def test_excluded_experts_and_rows_of_few_pairs(k):
    """Up to 24 pairs: -infinity and NaN are never taken, and a token of nothing else gives zeros."""
    rng = np.random.default_rng(2 + k)
    layer = Layer("nvfp4", "none", 9, 64, 64, bias=True)
    l = logits_of(rng, 8, 9)
    l[0] = -np.inf
    l[1] = np.nan
    l[2, 1:] = -np.inf
    l[3, ::2] = np.nan
    l[4] = np.finfo(np.float32).min
    l[5] = 0.0
    l[5, 3] = np.finfo(np.float32).min
    l[6, :7] = -np.inf
    x = tokens(rng, 8, 64)
    for renormalize in (True, False):
        y = layer.check(x, l, k, renormalize=renormalize)
        assert not y[:2].any()
        y = layer.check(x, l, k, renormalize=renormalize, out_dtype=torch.float32)
        assert not y[:2].any()
    l[7, 2] = np.inf
    y = layer.run(x, l, k)
    assert y[7].isnan().all() and not y[:7].isnan().any()
    # every row excluded: no pair at all
    assert not layer.run(x, np.full_like(l, -np.inf), k).any()
