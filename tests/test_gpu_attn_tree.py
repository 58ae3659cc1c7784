"""GPU tests of attention of drafted trees over the paged 4-bit cache (fp4_attn_tree) against a
plain binary64 reference on the same codes, scale bytes, queries and masks.  The bound of
each output follows from the kernels' stated roundings, as in tests/kv_reference.py (the
kernels are fp4_attn's), plus one rounding of the result to its type."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
import kv_reference as R
from test_gpu_attn import A_P, Setup, U_OUT, U_P

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


def seen_keys(mask, n, nq, i, there, window):
    """Which of a sequence's n keys query i of nq sees; mask: its row, by drafted key."""
    see = np.ones(n, bool)
    see[max(0, n - nq):] = False
    drafted = [n - nq + j for j in range(min(nq, len(mask))) if mask[j] and n - nq + j >= 0]
    if window:
        see[:max(0, n - nq + max(1, len(drafted)) - window)] = False
    see[drafted] = True
    return see & there


def reference(s, tree, scale, window, sinks):
    """(out, lse, their tolerances), binary64 (tests/kv_reference.py derives them)."""
    q, T, Hq, D = s.q.double().numpy(), len(s.q), s.H * s.G, s.D
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    tol, ltol = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    u_p, a_p = U_P[s.fmt], A_P[s.fmt]
    for b, n in enumerate(s.kv_lens):
        q0, q1 = s.q_starts[b], s.q_starts[b + 1]
        buf = {}
        for c in ("k", "v"):
            codes, there = R.sequence(s.buf[c + "_codes"], s.table[b], n, s.page)
            scales, _ = R.sequence(s.buf[c + "_scales"], s.table[b], n, s.page)
            buf[c] = R.decode(codes, scales, s.fmt)
        for i in range(q1 - q0):
            see = seen_keys(tree[q0 + i], n, q1 - q0, i, there, window)
            for qh in range(Hq):
                h = qh // s.G
                k, v = buf["k"][see, h], buf["v"][see, h]
                if s.outer is not None:
                    k, v = k * float(s.outer[0][h]), v * float(s.outer[1][h])
                at = q0 + i, qh
                sink = None if sinks is None else float(sinks[qh])
                if not len(k):
                    if sink is not None:
                        lse[at], ltol[at] = sink, 2.0 ** -20 * (1 + abs(sink))
                    continue
                x = k @ q[at] * scale
                mag = np.max(np.abs(k) @ np.abs(q[at])) * scale
                top = np.max(x) if sink is None else max(np.max(x), sink)
                p = np.exp(x - top)
                l = p.sum() + (0.0 if sink is None else np.exp(sink - top))
                out[at], lse[at] = (p / l) @ v, top + np.log(l)
                delta = (D + 4) * 2.0 ** -24 * mag + 2.0 ** -20 * (1 + np.max(np.abs(x)))
                rel = 2 * (u_p + delta) + len(x) * 2.0 ** -23
                tol[at] = rel * ((p / l) @ np.abs(v)) + a_p * np.abs(v).sum(0)
                ltol[at] = rel + 2.0 ** -20 * (1 + abs(lse[at]))
    return out, lse, tol, ltol


def trees(rng, q_lens, cols, empty=True):
    """Ancestors and itself of each node of random trees; some rows name nothing, some any set."""
    m = np.zeros((sum(q_lens), cols), bool)
    at = 0
    for n in q_lens:
        t = np.eye(max(n, 1), max(n, cols), dtype=bool)
        for i in range(1, n):
            t[i] |= t[rng.integers(max(0, i - 5), i)]
        m[at:at + n] = t[:n, :cols]
        at += n
    if empty and len(m) > 2:
        m[rng.integers(0, len(m), len(m) // 6 + 1)] = False
        m[len(m) // 2] = rng.random(cols) < 0.5
    return m


def run(s, tree, **kw):
    out, lse = fq.fp4_attn_tree(s.dq, s.cache, s.dt, s.dl, s.ds, torch.from_numpy(tree).cuda(), with_lse=True, **kw)
    torch.cuda.synchronize()
    return out, lse


def check(s, tree, window=0, sinks=None, out_dtype=torch.bfloat16, **kw):
    o, l, tol, ltol = reference(s, tree, float(np.float32(s.D ** -0.5)), window, sinks)
    out, lse = run(s, tree, window=window, sinks=None if sinks is None else torch.from_numpy(sinks).cuda(),
                   out_dtype=out_dtype, **kw)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    bound = tol * (1 + U_OUT[out_dtype]) + U_OUT[out_dtype] * np.abs(o) + 1e-37
    assert np.array_equal(np.isnan(got), np.isnan(o))
    bad = np.argwhere(~(np.abs(got - o) <= bound) & ~np.isnan(o))
    assert not len(bad), "%d of %d off; first %s: %r for %r +- %r" % (
        len(bad), o.size, bad[0], got[tuple(bad[0])], o[tuple(bad[0])], bound[tuple(bad[0])])
    assert np.array_equal(np.isinf(gl), np.isinf(l))
    ok = np.isfinite(l)
    assert np.all(np.abs(gl[ok] - l[ok]) <= ltol[ok])
    return out, lse


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "amdfp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 8])
@pytest.mark.parametrize("window", [0, 40])
def test_trees_behind_contexts(fmt, D, G, window):
    """Trees of few and many nodes behind contexts of every kind, none and shorter than the tree among them, in one call."""
    kv, ql = [100, 300, 77, 33, 13, 20, 0, 0, 515], [4, 31, 1, 32, 13, 37, 3, 0, 66]
    s = Setup(fmt, D, 2, G, 16, kv, ql, outer=fmt != "mxfp4").device()
    tree = trees(np.random.default_rng(D + G), ql, 66)
    out, lse = check(s, tree, window=window, max_q=66)
    assert not out[s.q_starts[6]:s.q_starts[7]].any() and torch.isinf(lse[s.q_starts[6]:s.q_starts[7]]).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "amdfp4"])
@pytest.mark.parametrize("n,G", [(1, 4), (7, 2), (8, 4), (16, 2), (5, 7), (3, 1)])
@pytest.mark.parametrize("window", [0, 1, 17, 200])
def test_few_rows(fmt, n, G, window):
    """At most 32 rows a head, whose keys are split over workgroups at the lengths that allow it."""
    kv = [n, n + 1, 31 + n, 32 + n, 33 + n, 95 + n, 1700, 5 * n + 640]
    s = Setup(fmt, 64, 2, G, 48, kv, [n] * len(kv), outer=fmt == "nvfp4").device()
    tree = trees(np.random.default_rng(n + G), [n] * len(kv), n)
    sinks = np.random.default_rng(n).normal(0, 1, 2 * G).astype(np.float32)
    check(s, tree, window=window, max_q=n, sinks=sinks)
    check(s, tree, window=window, max_q=n, out_dtype=torch.float32)


@pytest.mark.parametrize("fmt,D", [("mxfp4", 64), ("nvfp4", 128), ("amdfp4", 256)])
@pytest.mark.parametrize("n", [17, 64, 130])
@pytest.mark.parametrize("window", [0, 500])
def test_many_rows_with_split_keys(fmt, D, n, window):
    kv = [2100, 640 + n, n]
    s = Setup(fmt, D, 1, 8, 32, kv, [n, n, n]).device()
    tree = trees(np.random.default_rng(n), [n] * 3, n)
    check(s, tree, window=window, max_q=n)
    need = fq.fp4_attn_workspace(s.cache, 3 * n, 8, 3, max_q=n, max_kv=2100, window=window)
    assert need is not None
    need.fill_(0xFF)
    a, _ = run(s, tree, window=window, max_q=n, max_kv=2100, workspace=need)
    b, _ = run(s, tree, window=window, max_q=n, max_kv=2100)
    assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [0, 1, 5, 40])
def test_masks_of_other_widths(cols):
    """Drafted keys beyond the mask's columns are not seen; columns beyond the tree name nothing."""
    ql = [20, 3, 9]
    s = Setup("nvfp4", 64, 2, 2, 16, [200, 40, 9], ql).device()
    tree = np.random.default_rng(cols).random((sum(ql), cols)) < 0.6
    check(s, tree, max_q=20)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "amdfp4"])
@pytest.mark.parametrize("n", [4, 50])
def test_a_chain_is_a_causal_chunk(fmt, n):
    """The same keys, in the same steps (up to 256 keys of many rows are cut by neither call): equal bits."""
    s = Setup(fmt, 128, 2, 4, 16, [300, 1000, n] if n == 4 else [256, 131, n], [n, n, n]).device()
    chain = np.tile(np.tril(np.ones((n, n), bool)), (3, 1))
    a, al = run(s, chain, max_q=n)
    b, bl = s.run(max_q=n)
    assert torch.equal(a, b) and torch.equal(al, bl)


def test_any_value_but_zero_names_a_key():
    s = Setup("nvfp4", 64, 1, 4, 16, [90], [9]).device()
    tree = trees(np.random.default_rng(1), [9], 9)
    a, _ = run(s, tree)
    b, _ = run(s, tree.astype(np.uint8) * np.arange(1, 82, dtype=np.uint8).reshape(9, 9))
    assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "amdfp4"])
@pytest.mark.parametrize("n,G", [(6, 2), (40, 4)])
def test_bytes_of_keys_that_no_row_names(fmt, n, G):
    """A rejected draft's key may hold anything that the quantiser writes not: no result moves."""
    s = Setup(fmt, 64, 1, G, 16, [300], [n])
    tree = np.tril(np.ones((n, n), bool))
    tree[:, n // 2] = False
    want, wl = check(s.device(), tree, max_q=n)
    at = 300 - n + n // 2
    for c in "kv":
        s.buf[c + "_scales"][s.table[0, at // 16], 0, at % 16] = 0xFF
        s.buf[c + "_codes"][s.table[0, at // 16], 0, at % 16] = 0x7F
    o, l, tol, ltol = reference(s, tree, float(np.float32(64 ** -0.5)), 0, None)
    out, lse = (t.double().cpu().numpy() for t in run(s.device(), tree, max_q=n))
    assert np.all(np.abs(out - o) <= tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(o) + 1e-37) and np.all(np.abs(lse - l) <= ltol)


def test_a_poisoned_draft_reaches_the_rows_that_name_it_alone():
    for n, G in ((6, 2), (40, 4)):
        s = Setup("mxfp4", 64, 1, G, 16, [300], [n])
        at = 300 - n + 2
        s.buf["v_scales"][s.table[0, at // 16], 0, at % 16, 1] = 0xFF
        tree = trees(np.random.default_rng(2), [n], n, empty=False)
        tree[2, 2], tree[3, 2] = True, False
        out, _ = run(s.device(), tree, max_q=n)
        bad = out.isnan().cpu().numpy()
        assert np.array_equal(bad[..., 32:], np.broadcast_to(tree[:, 2, None, None], bad[..., 32:].shape))
        assert not bad[..., :32].any()


def test_missing_pages():
    s = Setup("nvfp4", 64, 2, 2, 16, [200, 48], [20, 10])
    s.table[0, 12], s.table[0, 3], s.table[1, 2] = -1, 1 << 30, -7
    check(s.device(), trees(np.random.default_rng(3), [20, 10], 20), max_q=20)


def test_replays_see_new_lengths_and_masks():
    """A captured call reads lengths, starts and masks anew."""
    rng = np.random.default_rng(4)
    s = Setup("mxfp4", 64, 2, 4, 16, [700, 650], [16, 16]).device()
    tree = torch.from_numpy(trees(rng, [16, 16], 16)).cuda()
    ws = fq.fp4_attn_workspace(s.cache, 32, 8, 2, max_q=16, max_kv=704)
    out = torch.empty(32, 8, 64, dtype=torch.bfloat16, device="cuda")
    call = lambda: fq.fp4_attn_tree(s.dq, s.cache, s.dt, s.dl, s.ds, tree, max_q=16, max_kv=704, out=out, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for turn in range(3):
        tree.copy_(torch.from_numpy(trees(rng, [16, 16], 16)))
        s.dl.copy_(torch.tensor([700 - 100 * turn, 650 - 300 * turn], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.zero_()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
    side = torch.cuda.Stream()
    y = fq.fp4_attn_tree(s.dq, s.cache, s.dt, s.dl, s.ds, tree, max_q=16, max_kv=704, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, out)
