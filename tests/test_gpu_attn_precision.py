"""GPU tests of the bits that attention keeps of its weights, against binary64 attention
over the same codes (bounds: kv_reference.py).

FP16 weights are rounded to half a step of 2^-11, or below 2^-14 to multiples of 2^-24 (off by 2^-25), in units that
put a row's largest weight at 2^7 or more: 2^-32 of it."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
import kv_reference as R
from test_gpu_attn import Setup

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]

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


# two 16-bit terms of a weight: half a step of what the first has left
U_TWO = {"mxfp4": 2.0 ** -16, "nvfp4": 2.0 ** -22, "amdfp4": 2.0 ** -22}
A_TWO = {"mxfp4": 0.0, "nvfp4": 2.0 ** -32, "amdfp4": 2.0 ** -32}


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "amdfp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv,ql,G,window,wide", [([1, 70, 513], [1, 1, 1], 4, 0, 0), ([2000, 40], [3, 2], 8, 0, 200),
                                                 ([150, 60], [60, 2], 4, 0, 0), ([1500], [40], 2, 1100, 200)])
def test_binary32_results_keep_two_terms_of_a_weight(fmt, D, kv, ql, G, window, wide):
    """Few rows with one part and with several, tiles of rows, tiles with split keys."""
    s = Setup(fmt, D, 2, G, 16, kv, ql, outer=fmt == "amdfp4", extra_cols=wide).device()
    o, l, tol, ltol = R.attention(s.q.double().numpy(), s.buf, fmt, 16, s.table, s.kv_lens, s.q_starts,
                                  float(np.float32(D ** -0.5)), window=window, outer=s.outer, u_p=U_TWO[fmt], a_p=A_TWO[fmt])
    out, lse = (t.double().cpu().numpy() for t in s.run(window=window, max_q=max(ql), out_dtype=torch.float32))
    off = np.abs(out - o) / (tol + 2.0 ** -24 * np.abs(o) + 1e-37)
    assert np.all(off <= 1), "off by %.1f bounds" % off.max()
    assert np.all(np.abs(lse - l) <= ltol)


def test_poisoned_blocks_in_binary32_results():
    for n in (3, 80):
        s = Setup("mxfp4", 128, 1, 2, 16, [80, 80], [n, 1])
        s.buf["v_scales"][s.table[0, 4], 0, 14, 2] = 0xFF     # key 78, values 64 .. 95: the last two queries see it
        s.buf["v_scales"][s.table[1, 4], 0, 15, 0] = 0xFF
        out, _ = s.device().check(out_dtype=torch.float32)
        assert torch.isnan(out[n - 2:n, :, 64:96]).all() and not torch.isnan(out[:n - 2]).any()
