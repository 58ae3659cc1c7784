"""GPU tests of fp4_attn_tree in batches of more sequences than a wave has lanes, and in launches of more workgroups than
one dimension takes, against the same binary64 reference and bounds as tests/test_gpu_attn_tree.py."""
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


def test_more_workgroups_than_a_dimension_takes():
    """512 sequences of 8 heads with a bound of 2^18 nodes: 2^23 workgroups of 512 lanes."""
    rng = np.random.default_rng(2)
    ql = [int(n) for n in rng.integers(0, 4, 512)]
    s = Setup("mxfp4", 64, 8, 1, 16, [int(n) for n in rng.integers(1, 30, 512)], ql).device()
    check(s, trees(rng, ql, 3), max_q=1 << 18)
