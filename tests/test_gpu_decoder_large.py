"""The decoder layer's operators where offsets pass 32 bits: rows of a norm and its gradient beyond 2^31 values, experts beyond
4 GiB of codes, and a cache beyond 4 GiB that is written with rotation and read by trees.  Each is compared with the
same call on the few rows, experts or pages that count, of which equal calls give equal bits, or (experts) with torch."""
import pytest
import torch

import block_scaled_fp4_amax_amd as fq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GiB of free device memory")
    fq.lib()
    yield
    torch.cuda.empty_cache()


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_rows_beyond_2_31_values():
    torch.manual_seed(1)
    rows, hidden = 140001, 16384
    pick = torch.tensor([0, 131071, 131072, rows - 2, rows - 1], device="cuda")
    x, r = (torch.empty(rows, hidden, dtype=torch.bfloat16, device="cuda").normal_() for _ in "xr")
    w = 1 + 0.1 * torch.randn(hidden, device="cuda")
    a = fq.fp4_add_rms_norm(x, w, r, fp8="mx", y=True)
    b = fq.fp4_add_rms_norm(x[pick], w, r[pick], fp8="mx", y=True)
    for k in ("residual", "rstd", "y", "fp8", "fp8_scales"):
        assert same(a[k][pick], b[k]), k
    dx = fq.fp4_add_rms_norm_backward(x, a["residual"], w, a["rstd"], dresidual=r, dx=r)["dx"]
    del a
    assert dx is r
    r2 = torch.empty_like(b["residual"]).copy_(b["residual"])
    torch.manual_seed(1)
    _, again = (torch.empty(rows, hidden, dtype=torch.bfloat16, device="cuda").normal_() for _ in "xr")
    want = fq.fp4_add_rms_norm_backward(x[pick], r2, w, b["rstd"], dresidual=again[pick])["dx"]
    assert same(dx[pick], want)


@pytest.mark.parametrize("T", [3, 20])
def test_experts_beyond_4_gib(T):
    """Bound in norm: y's rounding, 2^-8, the activations' 2^-16 and binary32 sums, 2^-12."""
    torch.manual_seed(2)
    E, H, I = 128, 8192, 8192
    cfg = fq.make_cfg(format="mxfp4")
    byte = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.uint8, device="cuda")  # noqa: E731
    w1 = {"codes": byte(0, 256, E, 2 * I, H // 2), "scales": byte(116, 120, E, 2 * I, H // 32)}
    w2 = {"codes": byte(0, 256, E, H, I // 2), "scales": byte(116, 120, E, H, I // 32)}
    x = torch.randn(T, H, device="cuda").bfloat16()
    logits = torch.full((T, E), -5.0, device="cuda")
    logits[:, 127], logits[:, 70] = 1.0, 0.5
    y = fq.fp4_moe(x, logits, w1, w2, cfg, top_k=2).double()
    share = torch.softmax(torch.tensor([1.0, 0.5], dtype=torch.float64), 0)
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e, a in zip((127, 70), share.tolist()):
        v1, v2 = (fq.fp4_dequantize(w["codes"][e], w["scales"][e], None, *n, cfg, dtype=torch.float32).double()
                  for w, n in ((w1, (2 * I, H)), (w2, (H, I))))
        g, u = (x.double() @ v1.t()).chunk(2, 1)
        want += a * ((g * torch.sigmoid(g) * u) @ v2.t())
        del v1, v2
    assert ((y - want).norm() / want.norm()).item() <= 2.0 ** -8 + 2.0 ** -16 + 2.0 ** -12


def test_pages_beyond_4_gib():
    """Rows written with rotation to the last and the first pages, and trees over them."""
    torch.manual_seed(3)
    H, G, D, page, pages, n, kv = 8, 2, 256, 64, 70000, 20, 190
    cfg = fq.make_cfg(format="nvfp4")
    big, small = (fq.KVCache.empty(p, page, H, D, cfg, device="cuda") for p in (pages, 6))
    assert big.k_codes.numel() > 1 << 32
    k, v, q = (torch.randn(2 * kv, h, D, device="cuda").bfloat16() for h in (H, H, H * G))
    angle = torch.arange(kv, device="cuda")[:, None] * 10000.0 ** (-torch.arange(64, device="cuda") / 64)
    positions = torch.arange(kv, dtype=torch.int32, device="cuda").repeat(2)
    tree = torch.tril(torch.rand(n, n, device="cuda") < 0.5).fill_diagonal_(True).repeat(2, 1)
    out = []
    for cache, table in ((big, [[pages - 1, 3, pages - 2], [0, pages - 3, 65536]]), (small, [[0, 1, 2], [3, 4, 5]])):
        t = torch.tensor(table, device="cuda")
        at = torch.arange(kv, device="cuda")
        slots = torch.cat([t[b][at // page] * page + at % page for b in range(2)])
        turned = fq.fp4_kv_append_rope(cache, k, v, slots, positions, angle.cos(), angle.sin(), q=q)
        drafted = torch.cat([turned[:n], turned[kv:kv + n]])
        lens, starts = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([kv, kv], [0, n, 2 * n]))
        o = fq.fp4_attn_tree(drafted, cache, t.int(), lens, starts, tree, max_q=n, max_kv=kv)
        out.append((turned, o, *fq.fp4_kv_read(cache, slots)))
    torch.cuda.synchronize()
    for a, b in zip(*out):
        assert same(a, b)
    # what was read is what was written: a block's largest value is 6, whose neighbour is 4, and its scale has 3 bits
    assert ((out[0][3].float() - v.float()).abs() <= v.float().abs().amax(-1, keepdim=True) / 4).all()
