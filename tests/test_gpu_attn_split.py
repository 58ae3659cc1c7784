"""GPU tests of attention whose rows see a window of keys that is split over
workgroups, at lengths of every residue of a round, against binary64 attention over
the same codes, scale bytes and queries.

Bounds as in tests/kv_reference.py: scores are off by (D + 4) 2^-24 scale sum |q k| and 2^-20 (1 + |s|)
in the exponential, weights are rounded to 16 bits before the product and the sum, sums of
n terms are binary32, and the result is rounded once to its type."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
import kv_reference as R

pytestmark = pytest.mark.gpu

U_P = {"mxfp4": 2.0 ** -8, "nvfp4": 2.0 ** -11, "amdfp4": 2.0 ** -11}
A_P = {"mxfp4": 0.0, "nvfp4": 2.0 ** -25, "amdfp4": 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


def expected(q, k, v, n, scale, window, fmt):
    """(out, lse, bound of out, bound of lse) of queries q [n, H, G, D] standing on the last n of the
    keys k, v [keys, H, D]; binary64 on the device."""
    m, D = k.shape[0], k.shape[2]
    q = q.permute(1, 0, 2, 3).reshape(q.shape[1], -1, D)                       # [H, n G, D]
    G = q.shape[1] // n
    k, v = k.permute(1, 2, 0).contiguous(), v.transpose(0, 1).contiguous()    # [H, D, keys], [H, keys, D]
    s, mag = q @ k * scale, q.abs() @ k.abs() * scale
    pos = torch.arange(m - n, m, device="cuda").repeat_interleave(G)[:, None]
    key = torch.arange(m, device="cuda")[None]
    hide = (key > pos) | (key <= pos - window)
    big, mag = s.masked_fill(hide, 0).abs().amax(-1), mag.masked_fill(hide, 0).amax(-1)
    s = s.masked_fill(hide, -float("inf"))
    lse = torch.logsumexp(s, -1)
    w = torch.softmax(s, -1)
    rel = 2 * (U_P[fmt] + (D + 4) * 2.0 ** -24 * mag + 2.0 ** -20 * (1 + big)) + window * 2.0 ** -23
    seen = (~hide).double().expand(q.shape[0], -1, -1).contiguous()
    tol = rel[..., None] * (w @ v.abs()) + A_P[fmt] * (seen @ v.abs())
    back = lambda t: t.reshape((t.shape[0], n, G) + t.shape[2:]).transpose(0, 1)  # noqa: E731
    return back(w @ v), back(lse), back(tol), back(rel + 2.0 ** -20 * (1 + lse.abs()))


@pytest.mark.parametrize("fmt,D,window,n,G,batch", [
    ("mxfp4", 64, 2000, 16, 4, 1), ("nvfp4", 64, 976, 16, 4, 2), ("nvfp4", 128, 984, 8, 8, 1),
    ("amdfp4", 128, 2000, 8, 8, 11), ("mxfp4", 128, 2000, 16, 4, 1), ("nvfp4", 64, 4096, 8, 8, 9),
    ("nvfp4", 256, 976, 5, 8, 2), ("mxfp4", 256, 960, 16, 4, 1), ("amdfp4", 64, 864, 129, 1, 1)])
def test_window_over_split_keys(fmt, D, window, n, G, batch):
    rng = np.random.default_rng(D + window)
    H, page, B = 8, 64, R.BLOCK[fmt]
    top = window + n + 300
    pages = -(-top // page)
    lo, hi = {"mxfp4": (124, 128), "nvfp4": (0x20, 0x38), "amdfp4": (0x60, 0x78)}[fmt]
    buf = {}
    for c in "kv":
        buf[c + "_codes"] = rng.integers(0, 256, (pages, H, page, D // 2)).astype(np.uint8)
        buf[c + "_scales"] = rng.integers(lo, hi, (pages, H, page, D // B)).astype(np.uint8)
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    cache = fq.KVCache(*(d(buf[c + s]) for c in "kv" for s in ("_codes", "_scales")), fq.make_cfg(format=fmt))
    order = rng.permutation(pages)
    # all sequences read the same pages, up to lengths of their own; far more could be named than is seen
    row = np.full(pages + 300, 2 ** 31 - 1, np.int32)
    row[:pages] = order
    table = d(np.repeat(row[None], batch, 0))
    k, v = (d(R.decode(buf[c + "_codes"], buf[c + "_scales"], fmt)[order].transpose(0, 2, 1, 3).reshape(-1, H, D)) for c in "kv")
    starts = torch.arange(0, (batch + 1) * n, n, dtype=torch.int32, device="cuda")
    q = torch.from_numpy(rng.normal(0, 2, (batch * n, H * G, D))).to(torch.bfloat16).cuda()
    ws = fq.fp4_attn_workspace(cache, batch * n, H * G, batch, max_q=n, table_cols=table.shape[1], window=window)
    assert ws is not None
    for first in range(0, 128, batch):
        lens = [top - min(first + b, 127) for b in range(batch)]
        out, lse = fq.fp4_attn(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), starts, max_q=n,
                               window=window, out_dtype=torch.float32, with_lse=True, workspace=ws)
        for b, m in enumerate(lens):
            if (first + b) % 3 and batch > 2:                # every third sequence of the larger batches
                continue
            at = slice(b * n, (b + 1) * n)
            o, l, tol, ltol = expected(q[at].double().view(n, H, G, D), k[:m], v[:m], n, float(np.float32(D ** -0.5)), window,
                                       fmt)
            off = (lse[at].double().view(n, H, G) - l).abs()
            assert bool((off <= ltol).all()), "lse at %d keys: off by %g" % (m, off.max().item())
            off = (out[at].double().view(n, H, G, D) - o).abs() - (tol * (1 + 2.0 ** -24) + 2.0 ** -24 * o.abs())
            assert bool((off <= 0).all()), "%d of %d off at %d keys" % (int((off > 0).sum()), off.numel(), m)
