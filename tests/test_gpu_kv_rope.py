"""GPU parity of fp4_kv_append_rope: the cache's bytes against the oracle's quantiser of
keys turned in numpy's binary32, one operation at a time, and the turned queries bit for
bit, at a tolerance of 0."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
from oracle import ref
from test_gpu_kv import dev, new_cache, oracle_rows, rows

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]

FORMATS = [("mxfp4", False), ("nvfp4", False), ("nvfp4", True), ("amdfp4", True)]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


def tables(n, half):
    angle = np.arange(n)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def f32(x):
    return x if x.dtype == np.float32 else (x.astype(np.uint32) << 16).view(np.float32)


def turned(x, positions, cos, sin, interleaved):
    """binary32 [tokens, heads, dim]: pairs (a, b) become (a c - b s, b c + a s)."""
    y, half = f32(x).copy(), cos.shape[1]
    c, s = cos[positions][:, None], sin[positions][:, None]
    i = np.arange(half)
    i, j = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    return y


def same_bits(got, want):
    """Equal bits, or NaN in both."""
    g, nan = got.float().cpu().numpy(), np.isnan(want)
    assert (np.isnan(g) == nan).all()
    want = torch.from_numpy(want).to(got.dtype).float().numpy()
    np.testing.assert_array_equal(g.view(np.uint32)[~nan], want.view(np.uint32)[~nan])


def check_cache(c, fmt, k, v, slots, written):
    pg, at = slots[written] // c.page_size, slots[written] % c.page_size
    for kv, x in (("k", k), ("v", v)):
        o = getattr(c, kv + "_outer")
        codes, scales, _, _ = oracle_rows(x, fmt, None if o is None else o.cpu().numpy())
        for name, want in ((kv + "_codes", codes), (kv + "_scales", scales)):
            full = np.full(tuple(getattr(c, name).shape), 0xA5, np.uint8)
            full[pg, :, at] = want[written]
            np.testing.assert_array_equal(getattr(c, name).cpu().numpy(), full, err_msg=name)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt,outer", FORMATS)
@pytest.mark.parametrize("T,Hq,H,D,rot,page", [(1, 1, 1, 64, 64, 16), (37, 6, 3, 64, 16, 48), (129, 8, 8, 128, 48, 64),
                                               (70, 10, 2, 256, 256, 32), (3, 5, 1, 128, 64, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_matches_the_oracle(fmt, outer, dtype, T, Hq, H, D, rot, page, interleaved):
    rng = np.random.default_rng(T * 1000 + H * 10 + D + rot)
    pages = -(-T // page) + 2
    c = new_cache(fmt, pages, page, H, D, outer, rng)
    q, k, v = (rows(rng, T, h, D, dtype) for h in (Hq, H, H))
    cos, sin = tables(500, rot // 2)
    positions = rng.integers(0, 500, T).astype(np.int32)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    # padding: by slot, and by position
    slots[T // 2:T // 2 + T // 9] = rng.choice([-1, -(1 << 62), pages * page, 1 << 62], T // 9)
    lost = np.arange(T) % 11 == 5
    positions[lost] = rng.choice([-1, 500, 1 << 30, -(1 << 31)], lost.sum())
    got = fq.fp4_kv_append_rope(c, dev(k), dev(v), dev(slots), dev(positions), dev(cos), dev(sin), q=dev(q),
                                interleaved=interleaved)
    torch.cuda.synchronize()
    at = np.where(lost, 0, positions)
    want = turned(q, at, cos, sin, interleaved)
    want[lost] = 0
    same_bits(got, want)
    check_cache(c, fmt, turned(k, at, cos, sin, interleaved), f32(v), slots,
                (slots >= 0) & (slots < pages * page) & ~lost)


@pytest.mark.parametrize("fmt,outer", FORMATS)
@pytest.mark.parametrize("tokens", [5, 3000])
def test_views_of_a_projection_turned_in_place(fmt, outer, tokens):
    """q, k and v as one projection gives them; the queries are turned where they are."""
    rng = np.random.default_rng(3)
    Hq, H, D = 12, 2, 64
    qkv = dev(rows(rng, tokens, Hq + 2 * H, D, "bf16"))
    q, k, v = qkv.split([Hq, H, H], 1)
    cos, sin = (dev(t) for t in tables(4096, 24))
    slots = torch.from_numpy(rng.permutation(4096)[:tokens].astype(np.int64)).cuda()
    positions = torch.from_numpy(rng.integers(0, 4096, tokens).astype(np.int32)).cuda()
    a, b, d = (new_cache(fmt, 64, 64, H, D, outer, np.random.default_rng(8)) for _ in range(3))
    want = fq.fp4_kv_append_rope(a, k.contiguous(), v.contiguous(), slots, positions, cos, sin, q=q.contiguous())
    assert fq.fp4_kv_append_rope(d, k, v, slots, positions, cos, sin) is None
    before = qkv[:, Hq:].clone()
    got = fq.fp4_kv_append_rope(b, k, v, slots, positions, cos, sin, q=q, q_out=q)
    torch.cuda.synchronize()
    assert got is q and torch.equal(q.view(torch.int16), want.view(torch.int16))
    assert torch.equal(qkv[:, Hq:].view(torch.int16), before.view(torch.int16))
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a, n), getattr(b, n)) and torch.equal(getattr(a, n), getattr(d, n)), n


def test_position_zero_is_the_plain_append():
    rng = np.random.default_rng(4)
    c, d = (new_cache("nvfp4", 4, 16, 2, 128, False, rng) for _ in range(2))
    k, v = (dev(rows(rng, 33, 2, 128, "bf16")) for _ in "kv")
    finite = ~(k.float().isnan() | k.float().isinf())
    k = torch.where(finite, k, torch.zeros_like(k))
    cos, sin = (dev(t) for t in tables(1, 64))
    slots = torch.arange(33, device="cuda")
    fq.fp4_kv_append(c, k, v, slots)
    fq.fp4_kv_append_rope(d, k, v, slots, torch.zeros(33, dtype=torch.int32, device="cuda"), cos, sin)
    for n in ("k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(c, n), getattr(d, n)), n
    # a zero may change its sign: a c - b s with b s = +0
    a, b = (getattr(x, "k_codes") for x in (c, d))
    for shift in (0, 4):
        x, y = (a >> shift) & 15, (b >> shift) & 15
        assert ((x == y) | (((x | y) & 7) == 0)).all()


def test_captured_and_replayed():
    rng = np.random.default_rng(5)
    c = new_cache("mxfp4", 8, 16, 2, 64, False, rng)
    q, k, v = (dev(rows(rng, 20, h, 64, "bf16")) for h in (4, 2, 2))
    cos, sin = (dev(t) for t in tables(64, 32))
    slots = torch.arange(20, device="cuda")
    positions = torch.arange(20, device="cuda", dtype=torch.int32)
    out = torch.zeros_like(q)
    call = lambda: fq.fp4_kv_append_rope(c, k, v, slots, positions, cos, sin, q=q, q_out=out)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for turn in range(3):
        positions.copy_(torch.arange(20, device="cuda", dtype=torch.int32) * (turn + 1))
        slots.copy_(torch.arange(20, device="cuda") + turn)
        c.k_codes.zero_()
        g.replay()
        torch.cuda.synchronize()
        got, codes = out.clone(), c.k_codes.clone()
        c.k_codes.zero_()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), out.view(torch.int16)) and torch.equal(codes, c.k_codes)


def test_another_stream_and_no_tokens():
    rng = np.random.default_rng(6)
    c = new_cache("nvfp4", 8, 16, 2, 64, False, rng)
    cos, sin = (dev(t) for t in tables(64, 32))
    q, k, v = (dev(rows(rng, 20, h, 64, "bf16")) for h in (4, 2, 2))
    slots = torch.arange(20, device="cuda")
    positions = torch.arange(20, device="cuda", dtype=torch.int32)
    want = fq.fp4_kv_append_rope(c, k, v, slots, positions, cos, sin, q=q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = fq.fp4_kv_append_rope(c, k, v, slots, positions, cos, sin, q=q, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    none = fq.fp4_kv_append_rope(c, k[:0], v[:0], slots[:0], positions[:0], cos, sin, q=q[:0])
    assert none.shape == (0, 4, 64)
