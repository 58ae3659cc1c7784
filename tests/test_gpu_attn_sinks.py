"""GPU tests of attention's sinks at the ends of binary32: the lowest finite value masks like -infinity, the
largest takes the whole weight, and neither makes a row NaN."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
from test_gpu_attn import Setup

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]

LOWEST = np.finfo(np.float32).min


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


# rows of few with one part and with several, tiles of rows, tiles whose keys are split; rows that see nothing
@pytest.mark.parametrize("kv,ql,wide", [([50, 0, 3], [1, 1, 1], 0), ([2000, 0, 70], [1, 2, 1], 300), ([90, 20], [40, 37], 0),
                                        ([2000], [40], 300)])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_sinks_at_the_ends(fmt, kv, ql, wide):
    s = Setup(fmt, 64, 2, 4, 16, kv, ql, extra_cols=wide).device()
    sinks = np.array([LOWEST, -LOWEST, -3e38, 3e38, -1e30, 1e30, -np.inf, 0.5], np.float32)
    out, lse = s.check(sinks=sinks, max_q=max(ql))
    assert torch.isfinite(out.float()).all()
    for h in (1, 3, 5):                                       # the sink takes the whole weight
        assert not out[:, h].any() and (lse[:, h] == float(sinks[h])).all()
    # masked sinks change nothing for rows that see a key
    plain, pl = s.run(max_q=max(ql))
    seen = torch.isfinite(pl[:, 0])
    for h in (0, 2, 4, 6):
        assert torch.equal(out[seen][:, h], plain[seen][:, h]) and torch.equal(lse[seen][:, h], pl[seen][:, h])
        assert (lse[~seen][:, h] == float(sinks[h])).all()
