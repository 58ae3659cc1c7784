"""GPU parity of the paged 4-bit cache's writer and reader (fp4_kv_append,
fp4_kv_read): every byte of the cache and every value read back against the
oracle's row quantiser and dequantiser, at a tolerance of 0."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
from oracle import ref

pytestmark = pytest.mark.gpu

SCALE = {"nvfp4": "e4m3", "amdfp4": "ue5m3"}
BLOCK = {"nvfp4": 16, "amdfp4": 16, "mxfp4": 32}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


def config(fmt, outer):
    return fq.make_cfg(format=fmt, two_level="tensorwise", outer_mode=1) if outer else fq.make_cfg(format=fmt)


def new_cache(fmt, pages, page, heads, dim, outer, rng, fill=0xA5):
    k_outer = v_outer = None
    if outer:
        k_outer, v_outer = (torch.from_numpy(np.exp(rng.normal(-4, 2, heads)).astype(np.float32)).cuda() for _ in "kv")
    c = fq.KVCache.empty(pages, page, heads, dim, config(fmt, outer), k_outer=k_outer, v_outer=v_outer)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.fill_(fill)
    return c


def oracle_rows(x, fmt, outer):
    """(codes, scales, bf16 bits, FP32 values) of [tokens, heads, dim] rows
    (uint16 bf16 bits or float32), outer: [heads] or None."""
    T, H, D = x.shape
    codes, scales = np.zeros((T, H, D // 2), np.uint8), np.zeros((T, H, D // BLOCK[fmt]), np.uint8)
    y, y32 = np.zeros((T, H, D), np.uint16), np.zeros((T, H, D), np.float32)
    for h in range(H):
        xh = np.ascontiguousarray(x[:, h])
        if fmt == "mxfp4":
            codes[:, h], scales[:, h], y[:, h] = ref.mx_qdq(xh)
            y32[:, h] = ref.mx_qdq(xh, y_dtype="fp32")[2]
        else:
            kw = dict(scale_fmt=SCALE[fmt])
            if outer is not None:
                kw.update(two_level="tensorwise", given_outer=(outer[h:h + 1], None))
            r = ref.nv_quantize(xh, **kw)
            codes[:, h], scales[:, h], y[:, h] = r["row_codes"], r["row_scales"], r["row_y"]
            y32[:, h] = ref.nv_quantize(xh, y_dtype="fp32", **kw)["row_y"]
    return codes, scales, y, y32


def rows(rng, T, H, D, dtype):
    """Rows of every size, with zeros, signed zeros, subnormals, infinities and NaN."""
    x = rng.normal(0, 1, (T, H, D)) * np.exp(rng.normal(0, 3, (T, H, 1)))
    x = x.astype(np.float32)
    flat = x.reshape(-1, 16)
    n = len(flat)
    for i, v in ((0, 0.0), (1, -0.0), (2, 1e-40), (3, np.inf), (4, -np.inf), (5, np.nan), (6, 3e38)):
        pick = np.arange(i, n, 37)
        flat[pick, rng.integers(0, 16, len(pick))] = v
    flat[7::37] = 0.0
    return x if dtype == "fp32" else ref.f32_to_bf16(x)


def dev(x):
    if x.dtype == np.uint16:
        return torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)
    return torch.from_numpy(x).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt,outer", [("mxfp4", False), ("nvfp4", False), ("nvfp4", True), ("amdfp4", False),
                                       ("amdfp4", True)])
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 64, 16), (37, 3, 64, 48), (129, 8, 128, 64), (70, 2, 256, 32)])
def test_append_and_read_match_the_oracle(fmt, outer, dtype, T, H, D, page):
    rng = np.random.default_rng(T * 1000 + H * 10 + D + page)
    pages = -(-T // page) + 2
    c = new_cache(fmt, pages, page, H, D, outer, rng)
    x = [rows(rng, T, H, D, dtype) for _ in "kv"]
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    # padding: slots outside the cache write nothing
    slots[T // 2:T // 2 + T // 9] = rng.choice([-1, -(1 << 62), pages * page, (1 << 62)], T // 9)
    sd = torch.from_numpy(slots).cuda()
    fq.fp4_kv_append(c, dev(x[0]), dev(x[1]), sd)
    got = fq.fp4_kv_read(c, sd)
    got32 = fq.fp4_kv_read(c, sd, dtype=torch.float32)
    torch.cuda.synchronize()
    inside = (slots >= 0) & (slots < pages * page)
    pg, at = slots[inside] // page, slots[inside] % page
    for i, kv in enumerate("kv"):
        o = getattr(c, kv + "_outer")
        codes, scales, y, y32 = oracle_rows(x[i], fmt, None if o is None else o.cpu().numpy())
        for name, want in ((kv + "_codes", codes), (kv + "_scales", scales)):
            full = np.full(tuple(getattr(c, name).shape), 0xA5, np.uint8)
            full[pg, :, at] = want[inside]
            np.testing.assert_array_equal(getattr(c, name).cpu().numpy(), full, err_msg=name)
        y[~inside], y32[~inside] = 0, 0.0
        np.testing.assert_array_equal(got[i].view(torch.int16).cpu().numpy().view(np.uint16), y)
        np.testing.assert_array_equal(got32[i].cpu().numpy().view(np.uint32), y32.view(np.uint32))


def test_views_of_a_fused_projection():
    rng = np.random.default_rng(3)
    T, H, D, page = 45, 2, 128, 16
    qkv = dev(rows(rng, T, 8 + 2 * H, D, "bf16"))
    k, v = qkv[:, 8:8 + H], qkv[:, 8 + H:]
    slots = torch.from_numpy(rng.permutation(64)[:T].astype(np.int64)).cuda()
    a, b = (new_cache("nvfp4", 4, page, H, D, False, rng) for _ in range(2))
    fq.fp4_kv_append(a, k, v, slots)
    fq.fp4_kv_append(b, k.contiguous(), v.contiguous(), slots)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n


def test_rows_equal_fp4_quantize():
    """A page's rows of one head are the buffers that fp4_quantize writes."""
    rng = np.random.default_rng(4)
    H, D, page = 2, 128, 32
    for fmt in BLOCK:
        c = new_cache(fmt, 1, page, H, D, False, rng)
        x = dev(rows(rng, page, H, D, "bf16"))
        fq.fp4_kv_append(c, x, x, torch.arange(page, device="cuda"))
        for h in range(H):
            q = fq.fp4_quantize(x[:, h], fq.make_cfg(format=fmt))
            assert torch.equal(c.k_codes[0, h], q["codes"]) and torch.equal(c.v_scales[0, h], q["scales"])


def test_slots_past_32_bits_of_bytes():
    """A cache whose code and scale offsets pass 2^32 bytes."""
    rng = np.random.default_rng(5)
    H, D, page = 8, 256, 64
    pages = (1 << 32) // (H * D // 2 * page) + 300
    c = fq.KVCache.empty(pages, page, H, D, config("nvfp4", False))
    assert c.k_codes.numel() > (1 << 32)
    x = [rows(rng, 40, H, D, "bf16") for _ in "kv"]
    slots = pages * page - 1 - np.arange(40, dtype=np.int64) * 7
    sd = torch.from_numpy(slots).cuda()
    fq.fp4_kv_append(c, dev(x[0]), dev(x[1]), sd)
    got = fq.fp4_kv_read(c, sd)
    for i in range(2):
        y = oracle_rows(x[i], "nvfp4", None)[2]
        np.testing.assert_array_equal(got[i].view(torch.int16).cpu().numpy().view(np.uint16), y)
    first = fq.fp4_kv_read(c, torch.arange(64, device="cuda"))
    assert not first[0].any() and not first[1].any()


def test_empty_calls():
    rng = np.random.default_rng(6)
    c = new_cache("mxfp4", 2, 16, 1, 64, False, rng)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    x = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    fq.fp4_kv_append(c, x, x, none)
    assert fq.fp4_kv_read(c, none)[0].shape == (0, 1, 64)
    e = fq.KVCache.empty(0, 16, 1, 64, config("mxfp4", False))
    x = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(3, dtype=torch.int64, device="cuda")
    fq.fp4_kv_append(e, x, x, s)
    assert not fq.fp4_kv_read(e, s)[1].any()


def test_side_stream_and_graph_replays():
    rng = np.random.default_rng(7)
    T, H, D, page = 33, 2, 64, 16
    c = new_cache("nvfp4", 6, page, H, D, True, rng)
    x = [dev(rows(rng, T, H, D, "bf16")) for _ in "kv"]
    slots = torch.from_numpy(rng.permutation(96)[:T].astype(np.int64)).cuda()
    fq.fp4_kv_append(c, *x, slots)
    want = [t.clone() for t in fq.fp4_kv_read(c, slots)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fq.fp4_kv_read(c, slots, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, want))
    out = tuple(torch.empty_like(t) for t in want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fq.fp4_kv_append(c, *x, slots)
        fq.fp4_kv_read(c, slots, out=out)
    for _ in range(3):
        c.k_codes.zero_()
        c.v_scales.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(out, want))
