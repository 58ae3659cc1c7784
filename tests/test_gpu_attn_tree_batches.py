"""GPU tests of fp4_attn_tree in batches of more sequences than a wave has lanes, of several tiles whose keys are not cut, and
in launches of more workgroups than one dimension takes, against the same binary64 reference and bounds as
tests/test_gpu_attn_tree.py."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
from test_gpu_attn import Setup
from test_gpu_attn_tree import check, trees

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


@pytest.mark.parametrize("fmt,D", [("mxfp4", 64), ("nvfp4", 128), ("amdfp4", 256)])
def test_several_tiles_of_keys_that_are_not_cut(fmt, D):
    """Up to 528 rows of a sequence and head, five tiles, and at most 256 keys, four rounds."""
    ql = [66, 40, 0, 66, 5, 17]
    s = Setup(fmt, D, 2, 8, 16, [250, 200, 30, 66, 256, 9], ql, outer=fmt == "nvfp4").device()
    assert fq.fp4_attn_workspace(s.cache, sum(ql), 16, len(ql), max_q=66, max_kv=256, trees=True) is None
    check(s, trees(np.random.default_rng(D), ql, 66), max_q=66, max_kv=256)


@pytest.mark.parametrize("fmt,D,batch,window", [("mxfp4", 64, 70, 0), ("nvfp4", 128, 130, 0), ("nvfp4", 64, 130, 700)])
def test_more_sequences_than_lanes(fmt, D, batch, window):
    """Ragged trees whose keys are cut, empty ones and ones without a context among them."""
    rng = np.random.default_rng(batch)
    ql = rng.integers(1, 7, batch)
    kv = rng.integers(1, 1700, batch)
    ql[[0, 63, 64, 69]], ql[[5, 40]] = 6, 0
    kv[[0, 63, 64, 65, batch - 1]], kv[[7, 66]], kv[68] = 1700, 3, 0
    s = Setup(fmt, D, 1, 7, 16, [int(n) for n in kv], [int(n) for n in ql], outer=fmt == "nvfp4").device()
    tree = trees(rng, [int(n) for n in ql], 6)
    assert fq.fp4_attn_workspace(s.cache, len(tree), 7, batch, max_q=6, max_kv=1700, window=window) is not None
    check(s, tree, window=window, max_q=6, max_kv=1700)


def test_more_workgroups_than_a_dimension_takes():
    """512 sequences of 8 heads with a bound of 2^18 nodes: 2^23 workgroups of 512 lanes."""
    rng = np.random.default_rng(2)
    ql = [int(n) for n in rng.integers(0, 4, 512)]
    s = Setup("mxfp4", 64, 8, 1, 16, [int(n) for n in rng.integers(1, 30, 512)], ql).device()
    check(s, trees(rng, ql, 3), max_q=1 << 18)
