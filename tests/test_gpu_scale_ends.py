"""GPU tests of the outermost UE8M0 scale bytes in the products and in attention: byte 0 is
2^-127 (its smallest values are subnormal in bf16 and binary32) and byte 254 is 2^127.  Bounds as in
test_gpu_linear.py and kv_reference.py."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
import kv_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


def d(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def codes(rng, shape, top):
    """Two codes a byte of magnitudes below grid index `top`, either sign."""
    lo, hi = (rng.integers(0, top, shape) | rng.integers(0, 2, shape) << 3 for _ in "lh")
    return (lo | hi << 4).astype(np.uint8)


# magnitudes that keep byte 254's values finite: 2 x 2^127 is not
@pytest.mark.parametrize("byte,top,size", [(0, 8, 1.0), (0, 8, 2.0 ** 60), (1, 8, 2.0 ** 60), (253, 6, 2.0 ** -60), (254, 4, 2.0 ** -60)])
@pytest.mark.parametrize("M,N,K", [(1, 32, 128), (3, 33, 160), (20, 32, 256), (40, 64, 256), (100, 160, 288)])
def test_linear(byte, top, size, M, N, K):
    rng = np.random.default_rng(M + byte)
    c = codes(rng, (N, K // 2), top)
    s = np.full((N, K // 32), byte, np.uint8)
    w = R.decode(c, s, "mxfp4")
    x = torch.from_numpy(rng.normal(0, size, (M, K))).to(torch.bfloat16)
    y = fq.fp4_linear(x.cuda(), {"codes": d(c), "scales": d(s), "outer": None}, fq.make_cfg(format="mxfp4"),
                      out_dtype=torch.float32).double().cpu().numpy()
    x = x.double().numpy()
    want, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    # a sum below binary32's normal range is a multiple of 2^-149
    assert np.all(np.abs(y - want) <= (K + K / 64 + 2) * 2.0 ** -24 * mag + 2.0 ** -24 * np.abs(want) + 2.0 ** -149)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("k_byte,v_byte,top,size", [(0, 127, 8, 2.0 ** 120), (127, 0, 8, 1.0), (127, 1, 8, 1.0), (254, 127, 4, 2.0 ** -127)])
def test_attention(D, n, k_byte, v_byte, top, size):
    rng = np.random.default_rng(D + n + k_byte)
    H, G, page, L, pages = 1, 2, 16, 80, 5
    buf = {}
    for c, byte in (("k", k_byte), ("v", v_byte)):
        buf[c + "_codes"] = codes(rng, (pages, H, page, D // 2), top)
        buf[c + "_scales"] = np.full((pages, H, page, D // 32), byte, np.uint8)
    cache = fq.KVCache(*(d(buf[c + s]) for c in "kv" for s in ("_codes", "_scales")), fq.make_cfg(format="mxfp4"))
    table, lens, starts = np.arange(pages, dtype=np.int32)[None], np.array([L], np.int32), np.array([0, n], np.int32)
    # 2^-127 would be subnormal in q: byte 254 takes it from the scale
    scale = D ** -0.5
    if size < 2.0 ** -100:
        size, scale = 2.0 ** -27, scale * 2.0 ** -100
    q = torch.from_numpy(rng.normal(0, size, (n, H * G, D))).to(torch.bfloat16)
    out, lse = fq.fp4_attn(q.cuda(), cache, d(table), d(lens), d(starts), scale=scale, out_dtype=torch.float32, with_lse=True)
    o, l, tol, ltol = R.attention(q.double().numpy(), buf, "mxfp4", page, table, lens, starts, float(np.float32(scale)), u_p=2.0 ** -8)
    # products and sums below binary32's normal range are multiples of 2^-149
    assert np.all(np.abs(out.double().cpu().numpy() - o) <= tol + 2.0 ** -24 * np.abs(o) + (L + 1) * 2.0 ** -149)
    assert np.all(np.abs(lse.double().cpu().numpy() - l) <= ltol)
