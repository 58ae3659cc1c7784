"""GPU tests of fp4_moe against a plain binary64 layer on the same codes, scale bytes,
activations and logits.

Bounds.  W is exact in the products.  With K = hidden, a sum of W1 is off by d = (K + K / 64 + 4) 2^-24 sum |x w|
(and its bias); g sigmoid(alpha g) has slope at most 1.1, so the activation is off by 1.1 d_g |u + shift| + |g sigmoid|
d_u + 1.1 d_g d_u and 16 binary32 roundings (the exponential two, and its argument's |alpha g| 2^-24); a share by
(|its logit - the largest| + top_k + 8) 2^-23 of itself.  Their product enters W2 as two bf16 terms (2^-16) or better,
and y is a binary32 sum of top_k inter products, in at most 64 parts more: (top_k inter + 64) 2^-24 of the
sum of magnitudes; then y's own rounding."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
import kv_reference as R

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]

U_OUT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U_MID = 2.0 ** -16
FORMATS = [("mxfp4", "none"), ("nvfp4", "none"), ("nvfp4", "2d"), ("nvfp4", "1d64"), ("nvfp4", "tensor"), ("amdfp4", "none"),
           ("amdfp4", "1d192"), ("amdfp4", "2d"), ("amdfp4", "tensor")]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


def d(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def config(fmt, kind):
    if kind == "tensor":
        return fq.make_cfg(format=fmt, two_level="tensorwise")
    if kind == "2d" or kind.startswith("1d"):
        return fq.make_cfg(format=fmt, two_level="outer_block", outer_block_size=64 if kind == "2d" else int(kind[2:]),
                           outer_2d=kind == "2d")
    return fq.make_cfg(format=fmt)


def experts(rng, fmt, kind, E, N, K):
    """Stacked random weights of about K^-1/2, and the values they stand for."""
    codes = rng.integers(0, 256, (E, N, K // 2)).astype(np.uint8)
    e = int(round(np.log2(K ** -0.5))) - 1
    bias, step = {"mxfp4": (127, 1), "nvfp4": (7, 8), "amdfp4": (15, 8)}[fmt]
    top = max(0, e + bias) * step
    scales = rng.integers(max(0, top - step), top + step, (E, N, K // R.BLOCK[fmt])).astype(np.uint8)
    v, outer = R.decode(codes, scales, fmt), None
    if kind == "tensor":
        outer = np.exp(rng.normal(0, .4, E)).astype(np.float32)
        v = v * outer[:, None, None].astype(np.float64)
    elif kind == "2d":
        outer = np.exp(rng.normal(0, .4, (E, N // 64, K // 64))).astype(np.float32)
        v = v * np.repeat(np.repeat(outer.astype(np.float64), 64, 1), 64, 2)
    elif kind != "none":
        obs = int(kind[2:])
        outer = np.exp(rng.normal(0, .4, (E, N, K // obs))).astype(np.float32)
        v = v * np.repeat(outer.astype(np.float64), obs, 2)
    return {"codes": d(codes), "scales": d(scales), "outer": None if outer is None else d(outer)}, v


class Layer:
    def __init__(self, fmt, kind, E, H, I, seed=0, bias=False):
        rng = np.random.default_rng(seed + E + H + I)
        self.E, self.H, self.I, self.cfg = E, H, I, config(fmt, kind)
        self.w1, self.v1 = experts(rng, fmt, kind, E, 2 * I, H)
        self.w2, self.v2 = experts(rng, fmt, kind, E, H, I)
        self.b1 = self.b2 = None
        if bias:
            self.b1, self.b2 = (rng.normal(0, 1, (E, n)).astype(np.float32) for n in (2 * I, H))

    def choices(self, logits, k, renormalize):
        """[(expert, share, relative bound of the share)] of a token."""
        l = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
        best = [e for e in sorted(range(self.E), key=lambda e: (-l[e], e))[:k] if l[e] > -np.inf]
        if not best:
            return []
        top = l[best[0]]
        total = np.exp(l[best if renormalize else l > -np.inf] - top).sum()
        return [(e, np.exp(l[e] - top) / total, (abs(l[e] - top) + len(l) + 8) * 2.0 ** -23) for e in best]

    def reference(self, x, logits, k, renormalize, interleaved, alpha, limit, shift, u_mid):
        y, tol = np.zeros((len(x), self.H)), np.zeros((len(x), self.H))
        for t in range(len(x)):
            mag, terms = np.zeros(self.H), 0
            for e, share, rs in self.choices(logits[t], k, renormalize):
                z, dz = self.v1[e] @ x[t], (self.H + self.H / 64 + 4) * 2.0 ** -24 * (np.abs(self.v1[e]) @ np.abs(x[t]))
                if self.b1 is not None:
                    z = z + self.b1[e]
                    dz = dz + 2.0 ** -24 * (np.abs(z) + np.abs(self.b1[e]))
                g, u = (z[0::2], z[1::2]) if interleaved else (z[:self.I], z[self.I:])
                dg, du = (dz[0::2], dz[1::2]) if interleaved else (dz[:self.I], dz[self.I:])
                if limit:
                    g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
                s = g / (1 + np.exp(-alpha * g))
                h = s * (u + shift)
                dh = 1.1 * dg * np.abs(u + shift) + np.abs(s) * du + 1.1 * dg * du
                dh = dh + (16 + np.abs(alpha * g)) * 2.0 ** -24 * np.abs(s) * (np.abs(u) + abs(shift))
                hs, dhs = h * share, dh * share * (1 + rs) + np.abs(h) * share * rs
                dhs = dhs + (u_mid + 2.0 ** -24) * (np.abs(hs) + dhs) + 2.0 ** -134
                a2 = np.abs(self.v2[e])
                y[t] += self.v2[e] @ hs
                tol[t] += a2 @ dhs
                mag += a2 @ (np.abs(hs) + dhs)
                if self.b2 is not None:
                    y[t] += share * self.b2[e]
                    tol[t] += rs * share * np.abs(self.b2[e])
                    mag += share * np.abs(self.b2[e])
                terms += self.I
            tol[t] += (terms + terms / 64 + 64) * 2.0 ** -24 * mag
        return y, tol

    def run(self, x, logits, k, out_dtype=torch.bfloat16, **kw):
        b1, b2 = (None if b is None else d(b) for b in (self.b1, self.b2))
        return fq.fp4_moe(x.cuda(), d(logits), self.w1, self.w2, self.cfg, top_k=k, b1=b1, b2=b2, out_dtype=out_dtype, **kw)

    def check(self, x, logits, k, renormalize=True, interleaved=False, alpha=1.0, limit=None, shift=0.0,
              out_dtype=torch.bfloat16):
        y = self.run(x, logits, k, out_dtype, renormalize=renormalize, interleaved=interleaved, alpha=alpha, limit=limit,
                     shift=shift)
        want, tol = self.reference(x.double().numpy(), logits, k, renormalize, interleaved, alpha, limit, shift,
                                   U_MID)
        bound = tol * (1 + U_OUT[out_dtype]) + U_OUT[out_dtype] * np.abs(want) + 1e-38
        got = y.double().cpu().numpy()
        bad = np.argwhere(~(np.abs(got - want) <= bound))
        assert not len(bad), "%d of %d off; first %s: %r for %r +- %r" % (
            len(bad), want.size, bad[0], got[tuple(bad[0])], want[tuple(bad[0])], bound[tuple(bad[0])])
        return y


def tokens(rng, T, H):
    return torch.from_numpy(rng.normal(0, 1, (T, H))).to(torch.bfloat16)


def logits_of(rng, T, E):
    return rng.normal(0, 2, (T, E)).astype(np.float32)


@pytest.mark.parametrize("fmt,kind", FORMATS)
@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 384, 192), (5, 3, 3, 192, 576), (16, 6, 1, 768, 192), (17, 20, 4, 192, 192),
                                       (40, 4, 2, 576, 384), (128, 5, 2, 192, 192)])
def test_every_format_and_outer_scale(fmt, kind, T, E, k, H, I):
    rng = np.random.default_rng(T + H)
    layer = Layer(fmt, kind, E, H, I, bias=T % 2 == 1)
    x, l = tokens(rng, T, H), logits_of(rng, T, E)
    layer.check(x, l, k)
    layer.check(x, l, k, interleaved=True, alpha=1.702, limit=0.9, shift=1.0, out_dtype=torch.float32)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "amdfp4"])
@pytest.mark.parametrize("H,I", [(32, 32), (64, 96), (160, 32), (96, 1056), (2080, 224), (32, 2016)])
@pytest.mark.parametrize("T", [1, 3, 31, 65])
def test_odd_sizes(fmt, H, I, T):
    rng = np.random.default_rng(H + I + T)
    layer = Layer(fmt, "none", 3, H, I, bias=H == 64)
    layer.check(tokens(rng, T, H), logits_of(rng, T, 3), 2)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (2, 64, 32), (3, 65, 8), (7, 511, 5), (128, 512, 2), (64, 128, 8), (128, 2, 2),
                                   (33, 7, 7), (15, 100, 1)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_counts_of_experts(T, E, k, renormalize):
    rng = np.random.default_rng(T + E)
    layer = Layer("mxfp4", "none", E, 64, 32)
    layer.check(tokens(rng, T, 64), logits_of(rng, T, E), k, renormalize=renormalize)


@pytest.mark.parametrize("T", [4, 50, 64, 100, 128])
def test_all_tokens_choose_the_same_experts(T):
    rng = np.random.default_rng(T)
    layer = Layer("nvfp4", "2d", 6, 128, 128, bias=True)
    l = logits_of(rng, T, 6)
    l[:, 4] += 100
    l[:, 1] += 90
    layer.check(tokens(rng, T, 128), l, 2)
    layer.check(tokens(rng, T, 128), l, 3, renormalize=False, out_dtype=torch.float32)


def test_ties_go_to_the_lower_expert():
    rng = np.random.default_rng(1)
    layer = Layer("mxfp4", "none", 70, 64, 32)
    l = np.zeros((6, 70), np.float32)
    l[1] = -0.0
    l[2, ::2] = -0.0
    l[3] = rng.integers(0, 2, 70)
    l[4] = -5.0
    l[5, 66:] = 1.0
    layer.check(tokens(rng, 6, 64), l, 3)


def test_logits_that_exclude_experts_and_rows():
    """-infinity and NaN are never taken; a token of nothing else gives zeros, the lowest finite logits count."""
    rng = np.random.default_rng(2)
    layer = Layer("nvfp4", "none", 9, 64, 64, bias=True)
    l = logits_of(rng, 8, 9)
    l[0] = -np.inf
    l[1] = np.nan
    l[2, 1:] = -np.inf
    l[3, ::2] = np.nan
    l[4] = np.finfo(np.float32).min
    l[5] = 0.0
    l[5, 3] = np.finfo(np.float32).min
    l[6, :7] = -np.inf
    for renormalize in (True, False):
        y = layer.check(tokens(rng, 8, 64), l, 4, renormalize=renormalize)
        assert not y[:2].any()
    l[7, 2] = np.inf
    y = layer.run(tokens(rng, 8, 64), l, 4)
    assert y[7].isnan().all() and not y[:7].isnan().any()


@pytest.mark.parametrize("T", [65, 129, 200, 1024])
def test_more_tokens_than_a_launch_takes(T):
    rng = np.random.default_rng(T)
    layer = Layer("amdfp4", "none", 5, 64, 64, bias=True)
    x, l = tokens(rng, T, 64), logits_of(rng, T, 5)
    y = layer.check(x, l, 2)
    for at in range(0, T, 64):
        assert torch.equal(y[at:at + 64], layer.run(x[at:at + 64], l[at:at + 64], 2))


@pytest.mark.parametrize("T", [12, 20])
def test_infinities_and_nan_stay_with_their_tokens(T):
    rng = np.random.default_rng(3)
    layer = Layer("mxfp4", "none", 4, 96, 64)
    x, l = tokens(rng, T, 96), logits_of(rng, T, 4)
    x[3, 5], x[11, 95] = float("inf"), float("nan")
    y = layer.run(x, l, 2).isnan().cpu().numpy()
    others = np.ones(T, bool)
    others[[3, 11]] = False
    assert y[11].all() and not y[others].any()


@pytest.mark.parametrize("T", [3, 30])
def test_an_infinite_activation_reaches_the_rows_that_weigh_it(T):
    """An infinite bias of a gate makes one activation of one expert infinite: y is infinite where its weight
    is not zero, with its sign, and NaN where it is."""
    rng = np.random.default_rng(9)
    layer = Layer("mxfp4", "none", 4, 96, 64, bias=True)
    layer.b1[1, 7] = np.inf
    x, l = tokens(rng, T, 96), logits_of(rng, T, 4)
    l[0, 1], l[-1, 1] = 50.0, -50.0                      # the first token takes that expert, the last does not
    y = layer.run(x, l, 2).double().cpu().numpy()
    took = 0
    for t in range(T):
        if 1 not in [e for e, _, _ in layer.choices(l[t], 2, True)]:
            assert np.isfinite(y[t]).all()
            continue
        took += 1
        u = layer.v1[1][64 + 7] @ x[t].double().numpy() + layer.b1[1, 64 + 7]
        want = layer.v2[1][:, 7] * u
        assert np.array_equal(np.isnan(y[t]), want == 0) and (y[t][want > 0] == np.inf).all() and (y[t][want < 0] == -np.inf).all()
    assert 0 < took < T


def test_activations_beyond_the_largest_bf16():
    """Activations of +-3.395e38, which round to infinity in bf16, weighed with 2^-6: y is finite."""
    z = lambda *s: np.zeros(s, np.uint8)  # noqa: E731
    E, H, I, T = 2, 32, 32, 40
    c1, c2, s = z(E, 2 * I, H // 2), z(E, H, I // 2), np.full((E, 2 * I, 1), 127, np.uint8)
    c2[:, :, 0] = 2                                      # the value 1 at place 0
    w1, w2 = dict(codes=d(c1), scales=d(s), outer=None), dict(codes=d(c2), scales=d(np.full((E, H, 1), 121, np.uint8)), outer=None)
    b1 = np.zeros((E, 2 * I), np.float32)
    b1[:, 0], b1[0, I], b1[1, I] = 2.0 ** 64, np.float32(3.395e38) / 2.0 ** 64, -np.float32(3.395e38) / 2.0 ** 64
    l = np.zeros((T, E), np.float32)
    l[::2, 0] = l[1::2, 1] = 1.0
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    cfg = fq.make_cfg(format="mxfp4")
    y = fq.fp4_moe(x, d(l), w1, w2, cfg, top_k=1, b1=d(b1), out_dtype=torch.float32).cpu().numpy()
    want = np.where(np.arange(T) % 2 == 0, 1, -1)[:, None] * np.float64(np.float32(3.395e38)) * 2.0 ** -6
    assert (np.abs(y - want) <= 2.0 ** -16 * np.abs(want)).all()


def test_sizes_of_a_real_layer():
    rng = np.random.default_rng(4)
    for fmt, kind, T in (("nvfp4", "2d", 1), ("mxfp4", "none", 48), ("amdfp4", "1d192", 6)):
        layer = Layer(fmt, kind, 6, 2880, 2880, bias=True)
        x, l = tokens(rng, T, 2880), logits_of(rng, T, 6)
        layer.check(x, l, 4, interleaved=True, alpha=1.702, limit=7.0, shift=1.0)
        layer.check(x, l, 2, out_dtype=torch.float32)


def test_views_given_outputs_and_workspace():
    rng = np.random.default_rng(5)
    layer = Layer("nvfp4", "none", 5, 96, 160)
    x, l = tokens(rng, 21, 96), logits_of(rng, 21, 5)
    want = layer.check(x, l, 2)
    wide = torch.full((21, 160), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 32:128] = x.cuda()
    out = torch.full((21, 111), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = fq.fp4_moe_workspace(21, 5, 2, 96, 160)
    ws.fill_(0xFF)
    y = fq.fp4_moe(wide[:, 32:128], d(l), layer.w1, layer.w2, layer.cfg, top_k=2, y=out[:, 5:101], workspace=ws)
    assert torch.equal(y, want) and (out[:, :5] == 7).all() and (out[:, 101:] == 7).all()
    flat = [{k: None if v is None else v.flatten() for k, v in w.items()} for w in (layer.w1, layer.w2)]
    assert torch.equal(fq.fp4_moe(x.cuda(), d(l), *flat, layer.cfg, top_k=2, workspace=ws), want)
    with pytest.raises(fq.Fp4Error) as e:
        fq.fp4_moe(x.cuda(), d(l), layer.w1, layer.w2, layer.cfg, top_k=2, workspace=ws[:-256])
    assert e.value.status == fq.ERR_WORKSPACE
    assert layer.run(x[:0], l[:0], 2).shape == (0, 96)


@pytest.mark.parametrize("T", [1, 8, 12])
def test_replays_and_other_streams(T):
    rng = np.random.default_rng(6)
    layer = Layer("nvfp4", "2d", 8, 256, 192)
    x, l = tokens(rng, T, 256).cuda(), d(logits_of(rng, T, 8))
    y = torch.empty(T, 256, dtype=torch.bfloat16, device="cuda")
    ws = fq.fp4_moe_workspace(T, 8, 3, 256, 192)
    call = lambda **kw: fq.fp4_moe(x, l, layer.w1, layer.w2, layer.cfg, top_k=3, **kw)  # noqa: E731
    call(y=y, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(y=y, workspace=ws)
    side = torch.cuda.Stream()
    for _ in range(4):
        l.copy_(d(logits_of(rng, T, 8)))
        x.mul_(0.75)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        again = call(stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, again) and torch.equal(call(), got)
