"""GPU tests of the bits that attention keeps of its weights, against binary64 attention
over the same codes (bounds: kv_reference.py).

FP16 weights are rounded to half a step of 2^-11, or below 2^-14 to multiples of 2^-24 (off by 2^-25), in units that
put a row's largest weight at 2^7 or more: 2^-32 of it."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
import kv_reference as R

pytestmark = pytest.mark.gpu

ONE = {"nvfp4": 0x38, "amdfp4": 0x78, "mxfp4": 127}            # the scale byte of 1


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


def d(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def buffers(pages, H, page, D, fmt):
    buf = {}
    for c in "kv":
        buf[c + "_codes"] = np.zeros((pages, H, page, D // 2), np.uint8)
        buf[c + "_scales"] = np.full((pages, H, page, D // R.BLOCK[fmt]), ONE[fmt], np.uint8)
    return buf


def call(buf, fmt, q, lens, starts, scale, **kw):
    cache = fq.KVCache(*(d(buf[c + s]) for c in "kv" for s in ("_codes", "_scales")), fq.make_cfg(format=fmt))
    table = np.arange(buf["k_codes"].shape[0], dtype=np.int32)[None]
    out = fq.fp4_attn(q.cuda(), cache, d(table), d(lens), d(starts), scale=scale, out_dtype=torch.float32, **kw)
    return out.double().cpu().numpy(), table


@pytest.mark.parametrize("fmt", ["nvfp4", "amdfp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,max_kv", [(1, 512), (1, 1 << 15), (40, 512), (40, 1 << 15)])
def test_many_small_weights_under_a_large_one(fmt, D, n, max_kv):
    """Key 0 has the weight 1 and the value 0, every other one e^-18 (below 2^-25) and the value 1."""
    page, L = 16, min(max_kv, 3000)
    pages = -(-max_kv // page)
    buf = buffers(pages, 1, page, D, fmt)
    buf["k_codes"][..., 0] = 0x0F                             # -6 in the first place
    buf["v_codes"][:] = 0x22
    buf["k_codes"][0, 0, 0] = 0
    buf["v_codes"][0, 0, 0] = 0
    q = torch.zeros(n, 1, D, dtype=torch.bfloat16)
    q[:, :, 0] = 3.0
    lens, starts = np.array([L], np.int32), np.array([0, n], np.int32)
    got, table = call(buf, fmt, q, lens, starts, 1.0)
    o, _, tol, _ = R.attention(q.double().numpy(), buf, fmt, page, table, lens, starts, 1.0, u_p=2.0 ** -11, a_p=2.0 ** -32)
    assert np.all(tol < o / 4)                                # the bound is one that nothing but the small weights meets
    assert np.all(np.abs(got - o) <= tol + 2.0 ** -24 * np.abs(o))
