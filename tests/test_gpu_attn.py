"""GPU tests of attention over the paged 4-bit cache (fp4_attn) against a plain
binary64 reference on the same codes, scale bytes and queries.  The bound of each
output follows from the kernel's stated roundings (tests/kv_reference.py), plus
one rounding of the result to its type."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
import kv_reference as R

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]

# half a step of the 16-bit type that weights are rounded to
U_P = {"mxfp4": 2.0 ** -8, "nvfp4": 2.0 ** -11, "amdfp4": 2.0 ** -11}
# half the smallest step of FP16; bf16 has binary32's range
A_P = {"mxfp4": 0.0, "nvfp4": 2.0 ** -25, "amdfp4": 2.0 ** -25}
U_OUT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


class Setup:
    """A cache of random codes and scale bytes with what lies beyond each
    sequence's keys set to poison, a shuffled page table, random queries."""

    def __init__(self, fmt, D, H, G, page, kv_lens, q_lens, seed=0, outer=False, extra_cols=0, k_size=1.0):
        rng = self.rng = np.random.default_rng(seed + D + 7 * H + page)
        self.fmt, self.page, self.D, self.H, self.G = fmt, page, D, H, G
        self.kv_lens = np.array(kv_lens, np.int32)
        self.q_starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        need = [-(-n // page) for n in kv_lens]
        pages = sum(need) + 2
        cols = max(max(need), 1) + extra_cols
        order = rng.permutation(pages)
        # entries beyond a sequence's pages are out of range
        self.table = np.full((len(kv_lens), cols), 2 ** 31 - 1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        B = R.BLOCK[fmt]
        self.buf = {}
        for c in "kv":
            codes = rng.integers(0, 256, (pages, H, page, D // 2)).astype(np.uint8)
            if fmt == "mxfp4":
                scales = rng.integers(124, 128, (pages, H, page, D // B))
            elif fmt == "nvfp4":
                scales = rng.integers(0x20, 0x38, (pages, H, page, D // B))
            else:
                scales = rng.integers(0x60, 0x78, (pages, H, page, D // B))
            scales[rng.random(scales.shape) < 0.02] = 1           # tiny blocks
            self.buf[c + "_codes"], self.buf[c + "_scales"] = codes, scales.astype(np.uint8)
            # what no sequence owns is poison
            owned = np.zeros((pages, page), bool)
            for b, n in enumerate(kv_lens):
                for t in range(n):
                    owned[self.table[b, t // page], t % page] = True
            self.buf[c + "_scales"].transpose(0, 2, 1, 3)[~owned] = 0xFF
            self.buf[c + "_codes"].transpose(0, 2, 1, 3)[~owned] = 0x77
        self.q = rng.normal(0, k_size, (self.q_starts[-1], H * G, D))
        self.q = torch.from_numpy(self.q).to(torch.bfloat16)
        self.outer = None
        if outer:
            self.outer = [np.exp(rng.normal(0, .5, H)).astype(np.float32) for _ in "kv"]

    def device(self):
        d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        cfg = fq.make_cfg(format=self.fmt, two_level="tensorwise", outer_mode=1) if self.outer else \
            fq.make_cfg(format=self.fmt)
        ko, vo = (d(x) for x in self.outer) if self.outer else (None, None)
        self.cache = fq.KVCache(*(d(self.buf[n]) for n in ("k_codes", "k_scales", "v_codes", "v_scales")), cfg,
                                k_outer=ko, v_outer=vo)
        self.dq, self.dt, self.dl, self.ds = self.q.cuda(), d(self.table), d(self.kv_lens), d(self.q_starts)
        return self

    def run(self, **kw):
        starts = kw.pop("q_starts", self.ds)
        out, lse = fq.fp4_attn(self.dq, self.cache, self.dt, self.dl, starts, with_lse=True, **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, scale=None, causal=True, window=0, sinks=None, out_dtype=torch.bfloat16, **kw):
        scale32 = float(np.float32(self.D ** -0.5 if scale is None else scale))
        o, l, tol, ltol = R.attention(self.q.double().numpy(), self.buf, self.fmt, self.page, self.table, self.kv_lens,
                                      self.q_starts, scale32, causal, window, sinks, self.outer, u_p=U_P[self.fmt], a_p=A_P[self.fmt])
        ds = None if sinks is None else torch.from_numpy(sinks).cuda()
        out, lse = self.run(scale=scale, causal=causal, window=window, sinks=ds, out_dtype=out_dtype, **kw)
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert out.dtype == out_dtype
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
def test_single_tokens(fmt, D):
    """Lengths from none to several steps, around every tile border."""
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 513]
    s = Setup(fmt, D, 2, 4, 16, lens, [1] * len(lens), outer=fmt != "mxfp4").device()
    s.check()
    out, lse = s.check(max_q=1)
    assert not out[0].any() and torch.isinf(lse[0]).all()
    again, _ = s.run(q_starts=None)
    assert torch.equal(out, again)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "amdfp4"])
@pytest.mark.parametrize("G", [1, 3, 8, 16, 20, 33])
def test_groups_of_heads(fmt, G):
    s = Setup(fmt, 64, 2, G, 32, [70, 5, 131], [1, 2, 3]).device()
    s.check()
    s.check(out_dtype=torch.float32)


@pytest.mark.parametrize("fmt,D,page,G", [("mxfp4", 128, 64, 4), ("nvfp4", 64, 48, 5), ("amdfp4", 256, 16, 2),
                                          ("mxfp4", 256, 32, 1), ("nvfp4", 128, 16, 8), ("amdfp4", 64, 128, 8)])
@pytest.mark.parametrize("window", [0, 1, 40])
def test_prompts_and_chunks(fmt, D, page, G, window):
    """Whole prompts, chunks behind a context, single tokens, more queries than
    keys (rows that see nothing), in one call."""
    kv, ql = [100, 300, 77, 1, 20, 0], [100, 45, 1, 1, 37, 3]
    s = Setup(fmt, D, 2, G, page, kv, ql, outer=fmt == "amdfp4").device()
    out, lse = s.check(window=window)
    first = int(s.q_starts[4])
    assert not out[first:first + 17].any() and torch.isinf(lse[first:first + 17]).all()
    assert not out[int(s.q_starts[5]):].any()


def test_not_causal():
    s = Setup("nvfp4", 64, 2, 4, 16, [90, 33, 0], [20, 40, 2]).device()
    s.check(causal=False)


def test_many_splits_and_bounds():
    """A wide page table splits the keys; tight bounds give another split of the
    same result; most splits of short sequences are empty."""
    for fmt in ("mxfp4", "nvfp4"):
        s = Setup(fmt, 64, 1, 8, 16, [2000, 1, 700, 0, 1300], [1] * 5, extra_cols=300).device()
        wide, _ = s.check()
        s.check(max_q=1, max_kv=2000)
        s.check(sinks=s.rng.normal(0, 2, 8).astype(np.float32), window=600)
        ws = fq.fp4_attn_workspace(s.cache, 5, 8, 5, max_q=5, table_cols=s.table.shape[1])
        assert ws is not None
        ws.fill_(0xFF)
        again, _ = s.run(workspace=ws)
        assert torch.equal(wide, again)
        s2 = Setup(fmt, 128, 2, 2, 16, [1100, 1500], [5, 30], extra_cols=200).device()
        s2.check()


@pytest.mark.parametrize("H", [1, 3])
def test_more_sequences_than_lanes(H):
    """Batches past 64 and 128 sequences, keys cut into parts in some of them, several without
    queries, and one of many rows."""
    rng = np.random.default_rng(11)
    lens = [int(n) for n in rng.integers(0, 40, 150)]
    for b, n in ((0, 900), (63, 700), (64, 2500), (127, 1), (128, 1300), (149, 3000)):
        lens[b] = n
    ql = [1] * 150
    for b in (5, 62, 65, 148):
        ql[b] = 0
    s = Setup("nvfp4", 64, H, 4, 16, lens, ql, extra_cols=3).device()
    s.check(max_q=1)
    ql[64], ql[149] = 9, 8
    s = Setup("mxfp4", 64, H, 4, 16, lens, ql, extra_cols=3).device()
    s.check(max_q=9)


def test_counts_beyond_the_bounds_are_cut():
    s = Setup("nvfp4", 64, 1, 2, 16, [64, 32], [1, 1]).device()
    full = s.kv_lens.copy()
    s.dl = torch.tensor([1 << 30, -5], dtype=torch.int32, device="cuda")     # the table names 64 keys
    s.kv_lens = np.array([64, 0], np.int32)
    s.check()
    s.dl = torch.from_numpy(full).cuda()
    s.kv_lens = np.array([40, 32], np.int32)
    s.check(max_kv=40)
    # q_starts outside the tensor are cut to it
    s.kv_lens = full
    out = torch.full((2, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    fq.fp4_attn(s.dq, s.cache, s.dt, s.dl, torch.tensor([-4, 1, 1 << 30], dtype=torch.int32, device="cuda"), out=out)
    want, _ = s.run()
    assert torch.equal(out, want)


def test_rows_of_no_sequence_are_not_written():
    for cols in (0, 400):                                     # without and with split keys
        s = Setup("nvfp4", 64, 1, 2, 16, [64], [3], extra_cols=cols).device()
        want, _ = s.run()
        starts = torch.tensor([1, 3], dtype=torch.int32, device="cuda")
        out = torch.full((3, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        fq.fp4_attn(s.dq, s.cache, s.dt, s.dl, starts, out=out)
        assert (out[0] == 7.0).all() and torch.equal(out[1:], want[1:])


def test_pages_outside_the_cache_are_absent():
    for bad in (-1, 2 ** 31 - 1, -2 ** 31, None):
        s = Setup("mxfp4", 128, 2, 4, 32, [200, 100, 64], [1, 9, 64])
        n = s.buf["k_codes"].shape[0]
        s.table[0, 2] = n if bad is None else bad
        s.table[1, 0] = n if bad is None else bad
        s.table[2, :] = n if bad is None else bad
        out, lse = s.device().check()
        assert not out[10:].any() and torch.isinf(lse[10:]).all()


def test_poisoned_blocks_reach_only_rows_that_see_them():
    """MXFP4 scale byte 0xFF in V makes that block's outputs NaN for the rows that
    see the key, in K the whole row; no other row changes."""
    for window in (0, 30):
        s = Setup("mxfp4", 128, 1, 2, 16, [80, 80], [80, 1])
        s.buf["v_scales"][s.table[0, 3], 0, 5, 2] = 0xFF      # key 53, values 64 .. 95
        s.buf["v_scales"][s.table[1, 4], 0, 15, 0] = 0xFF     # the last key
        out, _ = s.device().check(window=window)
        assert torch.isnan(out[53:80, :, 64:96]).any() and not torch.isnan(out[:53]).any()
        s.buf["k_scales"][s.table[0, 4], 0, 0, 1] = 0xFF      # key 64
        s.device()
        out, lse = s.run(window=window)
        assert not torch.isnan(out[:53]).any() and torch.isnan(out[64:80]).all()


def test_sinks_and_empty_rows():
    s = Setup("amdfp4", 64, 2, 4, 16, [50, 0, 3], [10, 2, 5]).device()
    sinks = s.rng.normal(0, 3, 8).astype(np.float32)
    sinks[3] = -np.inf
    sinks[5] = 40.0
    out, lse = s.check(sinks=sinks)
    assert not out[10:14].any()
    assert torch.allclose(lse[10], torch.from_numpy(sinks).cuda())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_large_scores(fmt):
    """Scores of hundreds, rising along the keys, so the running maximum moves."""
    s = Setup(fmt, 64, 1, 8, 16, [400, 90], [1, 60], k_size=30.0).device()
    s.check(scale=1.0)
    s.check(scale=2.0 ** -20)


def test_equal_values_are_returned_exactly():
    """The sum of weights is that of the rounded weights: equal rows of V come
    back without any rounding but the result's."""
    s = Setup("mxfp4", 64, 1, 4, 16, [333], [50])
    s.buf["v_codes"][:] = s.buf["v_codes"][0, :, :1]
    s.buf["v_scales"][:] = 126
    s.device()
    out, _ = s.run(out_dtype=torch.float32)
    v = R.decode(s.buf["v_codes"][0, 0, 0], s.buf["v_scales"][0, 0, 0], "mxfp4")
    np.testing.assert_allclose(out.cpu().numpy(), np.broadcast_to(v, (50, 4, 64)), rtol=2.0 ** -20)


def test_queries_with_a_token_pitch_side_stream_and_graph():
    s = Setup("nvfp4", 128, 2, 4, 16, [600, 70], [1, 3], extra_cols=100, outer=True).device()
    want, wl = s.check()
    wide = torch.zeros(4, 12, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = s.dq
    out = fq.fp4_attn(wide[:, 2:10], s.cache, s.dt, s.dl, s.ds)
    assert torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = fq.fp4_attn(s.dq, s.cache, s.dt, s.dl, s.ds, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    ws = fq.fp4_attn_workspace(s.cache, 4, 8, 2, table_cols=s.table.shape[1])
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fq.fp4_attn(s.dq, s.cache, s.dt, s.dl, s.ds, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_pages_past_32_bits_of_bytes():
    """The same sequences in low and in high pages of a cache beyond 4 GiB."""
    s = Setup("nvfp4", 256, 2, 4, 64, [300, 65], [1, 20]).device()
    want, _ = s.check()
    shift = (1 << 32) // (2 * 64 * 128) + 10
    big = fq.KVCache.empty(shift + s.buf["k_codes"].shape[0], 64, 2, 256, s.cache.cfg)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        getattr(big, n)[shift:] = getattr(s.cache, n)
    table = torch.from_numpy(np.where(s.table < 2 ** 30, s.table + shift, s.table).astype(np.int32)).cuda()
    assert torch.equal(fq.fp4_attn(s.dq, big, table, s.dl, s.ds), want)


def test_written_by_append():
    """Rows written by fp4_kv_append, attended over, against the values that
    fp4_kv_read returns."""
    torch.manual_seed(0)
    T, H, G, D, page = 90, 2, 4, 128, 16
    k, v = (torch.randn(T, H, D, device="cuda").bfloat16() for _ in "kv")
    q = torch.randn(T, H * G, D, device="cuda").bfloat16()
    cache = fq.KVCache.empty(8, page, H, D, fq.make_cfg(format="nvfp4"))
    table = torch.tensor([[5, 0, 7, 2, 1, 4]], dtype=torch.int32, device="cuda")
    t = torch.arange(T, device="cuda")
    slots = table[0].long()[t // page] * page + t % page
    fq.fp4_kv_append(cache, k, v, slots)
    out = fq.fp4_attn(q, cache, table, torch.tensor([T], dtype=torch.int32, device="cuda"),
                      torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    kr, vr = (x.double().cpu() for x in fq.fp4_kv_read(cache, slots, dtype=torch.float32))
    qd = q.double().cpu()
    for h in range(H * G):
        s = (qd[:, h] @ kr[:, h // G].T) * D ** -0.5
        s = s.masked_fill(torch.ones(T, T).triu(1).bool(), -np.inf)
        w = torch.softmax(s, -1)
        o = w @ vr[:, h // G]
        bound = (2 * 2.0 ** -11 + 2.0 ** -14) * (w @ vr[:, h // G].abs()) + 2.0 ** -8 * o.abs()
        assert ((out[:, h].double().cpu() - o).abs() <= bound).all()
