"""GPU tests of fp4_add_rms_norm and its gradient.

Forward: every step is a rounded binary32 operation but the sum of squares, which is
binary64, so h, r, y, the codes and the scales are compared bit for bit with numpy (r to one step:
numpy's own binary64 quotient and root may round the other way at a tie).
Gradient, binary32: with n = h r, g = dy w and N = hidden, each value of n g carries 3 roundings, its
sum over a row at most N / 64 + 7 + 3 additions in a row of a lane and across lanes,
and dx five more operations.  Let M = mean |n g|; then
  |dx - exact| <= 2^-24 r ((N / 64 + 16) |n| M + 6 |g| + 6 |n| |mean n g|) + 2^-24 (|dx| + |dres|), plus half a step of dx's type.
dweight sums at most rows terms of 3 roundings each in binary32: 2^-24 (rows + 4) sum |dy n|."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
HIDDEN = [8, 32, 40, 256, 488, 520, 1024, 1504, 2048, 2880, 3080, 4096, 4104, 5120, 8008, 8192, 8200, 12288, 16384]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


def inputs(rng, rows, hidden, dtype, spread=3.0):
    x = rng.normal(0, 1, (rows, hidden)) * np.exp(rng.normal(0, spread, (rows, 1)))
    return torch.from_numpy(x).to(TYPES[dtype])


def rounded(x, dtype):
    return torch.from_numpy(x).to(dtype).float().numpy()


E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)


def e4m3(q):
    """Codes of binary32 values, ties to even, at most 448; NaN stays NaN."""
    grid = E4M3[:127]
    mid = (grid[1:] + grid[:-1]) / 2
    a = np.minimum(np.abs(q.astype(np.float64)), 448.0)
    i = np.searchsorted(mid, a, side="left")
    tie = (i < 126) & (mid[np.minimum(i, 125)] == a) & (i % 2 == 1)
    c = (i + tie).astype(np.uint8) | (np.signbit(q).astype(np.uint8) << 7)
    return np.where(np.isnan(q), np.uint8(0x7F), c)


def forward(x, residual, w, eps, rstd=None):
    h = x.float().numpy()
    if residual is not None:
        h = rounded(h + residual.float().numpy(), residual.dtype)
    r64 = 1 / np.sqrt((h.astype(np.float64) ** 2).sum(1) / h.shape[1] + eps)
    r = r64.astype(np.float32) if rstd is None else rstd
    return h, r64, (h * r[:, None]) * w.float().numpy()


def finite_top(y):
    a = np.abs(y)
    return np.where(np.isfinite(a), a, np.float32(0)).max(-1)


def codes_of(y, mode):
    if mode == "row":
        s = finite_top(y) / np.float32(448)
        q = np.where(s[:, None] == 0, np.where(np.isfinite(y), np.copysign(np.float32(0), y), np.float32("nan")),
                     y / np.where(s == 0, np.float32(1), s)[:, None])
        return e4m3(q.astype(np.float32)), s
    b = y.reshape(y.shape[0], -1, 32)
    top = finite_top(b).astype(np.float64)
    e = np.where(top > 0, np.frexp(top)[1] - 9, -127).clip(-127, 127)
    q = (b.astype(np.float64) * 2.0 ** -e[..., None].astype(np.float64))
    return e4m3(q).reshape(y.shape), (e + 127).astype(np.uint8)


def same_codes(got, want):
    nan = (want & 0x7F) == 0x7F
    assert ((got & 0x7F) == 0x7F)[nan].all()
    np.testing.assert_array_equal(got[~nan], want[~nan])


def check_forward(o, x, residual, w, eps, mode, y_dtype):
    rstd = o["rstd"].cpu().numpy()
    h, r64, y = forward(x, residual, w, eps, rstd)
    ok = np.isfinite(r64)
    assert (np.abs(rstd[ok] - r64[ok]) <= r64[ok] * 2.0 ** -24 * (1 + 1e-6) + 2.0 ** -150).all()
    np.testing.assert_array_equal(o["residual"].float().cpu().numpy(), h)
    if o["y"] is not None:
        np.testing.assert_array_equal(o["y"].float().cpu().numpy(), rounded(y, y_dtype))
    if mode:
        codes, scales = codes_of(y, mode)
        np.testing.assert_array_equal(o["fp8_scales"].cpu().numpy(), scales)
        same_codes(o["fp8"].cpu().numpy(), codes)


@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16"), ("fp32", "fp32"), ("bf16", None),
                                   ("fp32", None)])
@pytest.mark.parametrize("hidden", HIDDEN)
@pytest.mark.parametrize("rows", [1, 5, 1030])
def test_forward(xt, rt, hidden, rows):
    rng = np.random.default_rng(hidden + rows)
    rows = min(rows, max(1, (1 << 22) // hidden))
    x = inputs(rng, rows, hidden, xt)
    residual = None if rt is None else inputs(rng, rows, hidden, rt)
    w = torch.from_numpy(rng.normal(1, 0.5, hidden)).to(TYPES[xt])
    mode = ["mx", "row"][rows % 2] if hidden % 32 == 0 else "row"
    for fp8, y, y_dtype in ((mode, False, None), (mode, True, torch.bfloat16), (None, True, torch.float32)):
        o = fq.fp4_add_rms_norm(x.cuda(), w.cuda(), None if residual is None else residual.cuda(), eps=1e-5, fp8=fp8, y=y,
                                y_dtype=y_dtype)
        assert (o["y"] is not None) == y and (o["fp8"] is not None) == (fp8 is not None)
        check_forward(o, x, residual, w, 1e-5, fp8, y_dtype)


@pytest.mark.parametrize("mode", ["mx", "row"])
def test_every_code(mode):
    """Values at, beside and between all E4M3 codes, at blocks and rows of every size: with eps so large that
    r is a power of two (but for the largest row), y is w's pattern itself."""
    grid = E4M3[:127]
    mids = (grid[1:] + grid[:-1]) / 2
    v = np.concatenate([grid, mids, np.nextafter(mids.astype(np.float32), np.float32(0)).astype(np.float64),
                        np.nextafter(mids.astype(np.float32), np.float32(1e9)).astype(np.float64), [460.0, 463.9, 464.0, 480.0, 511.9]])
    v = np.concatenate([v, -v])
    v = np.resize(v, -(-len(v) // 31) * 31).reshape(-1, 31)
    w = np.concatenate([np.full((len(v), 1), 448.0 if mode == "row" else 256.0), v], 1).astype(np.float32).ravel()
    if mode == "row":
        w = w.clip(-448, 448)
    w = np.resize(w, 2048)
    # h = 2^a with eps = 2^100: y = w 2^(a - 50).  r = 2^-50 (1 + 2^(2 a - 100))^-1/2 is within half a step (2^-25
    # below a power of two) of 2^-50 where 2^(2 a - 101) <= 2^-26, a <= 37; a = 39 gives 1 - 2^-23, two steps below.
    h = 2.0 ** np.arange(-60, 40, 9, dtype=np.float64)
    x = torch.from_numpy(np.repeat(h[:, None], 2048, 1)).float()
    o = fq.fp4_add_rms_norm(x.cuda(), torch.from_numpy(w).cuda(), eps=2.0 ** 100, fp8=mode, y=True, y_dtype=torch.float32)
    np.testing.assert_array_equal(o["rstd"].cpu().numpy(), np.where(h < 2.0 ** 38, 1, 1 - 2.0 ** -23) * 2.0 ** -50)
    check_forward(o, x, None, torch.from_numpy(w), 2.0 ** 100, mode, torch.float32)


def test_zeros_extremes_infinities_and_nan():
    x = torch.zeros(9, 64)
    x[1] = 3e38                                             # a sum that overflows binary32
    x[2], x[2, 3] = 1.0, float("inf")
    x[3], x[3, 9] = 1.0, float("nan")
    x[4] = 1e-40
    x[5, ::2] = -0.0
    x[6] = float("inf")
    x[7] = 1e-30
    x[8, 5] = 7.0
    w = torch.linspace(-2, 2, 64)
    w[10] = float("inf")
    for mode in ("mx", "row"):
        for eps in (0.0, 1e-6):
            o = fq.fp4_add_rms_norm(x.cuda(), w.cuda(), torch.zeros(9, 64).cuda(), eps=eps, fp8=mode, y=True,
                                    y_dtype=torch.float32)
            rstd = o["rstd"].cpu().numpy()
            h, r64, y = forward(x, torch.zeros(9, 64), w, eps, rstd)   # -0 + 0 is +0
            np.testing.assert_array_equal(rstd[[1, 7, 8]], r64.astype(np.float32)[[1, 7, 8]])
            got = o["y"].cpu().numpy()
            np.testing.assert_array_equal(np.isnan(got), np.isnan(y))
            np.testing.assert_array_equal(got[~np.isnan(y)], y[~np.isnan(y)])
            codes, scales = codes_of(y, mode)
            np.testing.assert_array_equal(o["fp8_scales"].cpu().numpy(), scales)
            same_codes(o["fp8"].cpu().numpy(), codes)


@pytest.mark.parametrize("rows", [4, 1100])
def test_pitched_views_in_place_and_given_outputs(rows):
    rng = np.random.default_rng(1)
    wide = inputs(rng, rows, 800, "bf16").cuda()
    x, r = wide[:, 8:328], inputs(rng, rows, 320, "bf16").cuda()
    w = torch.ones(320, dtype=torch.bfloat16, device="cuda")
    want = fq.fp4_add_rms_norm(x.contiguous(), w, r.clone(), fp8="row", y=True)
    pitched = torch.zeros(rows, 400, dtype=torch.bfloat16, device="cuda")
    pitched[:, :320] = r
    other = fq.fp4_add_rms_norm(x, w, pitched[:, :320], fp8="row", y=True)
    out = {"residual": r, "fp8": torch.empty(rows, 320, dtype=torch.uint8, device="cuda")}
    got = fq.fp4_add_rms_norm(x, w, r, fp8="row", y=True, out=out)
    assert got["residual"] is r and got["fp8"] is out["fp8"]
    for k in want:
        assert torch.equal(want[k], got[k]) and torch.equal(want[k], other[k]), k


def check_backward(got, dy, h, w, rstd, dres):
    rows, hidden = h.shape
    y, x, g = dy.double().numpy(), h.double().numpy(), dy.double().numpy() * w.double().numpy()
    r = rstd.double().numpy()[:, None]
    n = x * r
    mean, mag = (n * g).mean(1, keepdims=True), np.abs(n * g).mean(1, keepdims=True)
    d = 0.0 if dres is None else dres.double().numpy()
    dx = r * (g - n * mean) + d
    tol = 2.0 ** -24 * (r * ((hidden / 64 + 16) * np.abs(n) * mag + 6 * np.abs(g) + 6 * np.abs(n * mean)) + np.abs(dx) + np.abs(d))
    tol = tol * (1 + U[h.dtype]) + U[h.dtype] * np.abs(dx) + 1e-38
    err = np.abs(got["dx"].double().cpu().numpy() - dx)
    assert (err <= tol).all(), (err / tol).max()
    dw, wtol = (y * n).sum(0), 2.0 ** -24 * (rows + 4) * np.abs(y * n).sum(0) + 1e-38
    err = np.abs(got["dweight"].double().cpu().numpy() - dw)
    assert (err <= wtol).all(), (err / wtol).max()


@pytest.mark.parametrize("yt,ht", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("hidden", HIDDEN)
@pytest.mark.parametrize("rows", [1, 3, 1030, 2500])
def test_backward(yt, ht, hidden, rows):
    rng = np.random.default_rng(hidden + rows)
    rows = min(rows, max(1, (1 << 22) // hidden))
    dy, h, dres = inputs(rng, rows, hidden, yt, 1.0), inputs(rng, rows, hidden, ht, 1.0), inputs(rng, rows, hidden, ht, 1.0)
    w = torch.from_numpy(rng.normal(1, 0.5, hidden)).to(TYPES[ht])
    rstd = torch.from_numpy(1 / np.sqrt((h.double().numpy() ** 2).mean(1) + 1e-5)).float()
    for d in (dres, None):
        got = fq.fp4_add_rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dresidual=None if d is None else d.cuda())
        check_backward(got, dy, h, w, rstd, d)


def test_gradient_against_differences():
    """Central differences of the binary64 formula, at values of order 1: off by step^2 / 6 of a third derivative
    (below 50 here) and by 2^-52 / step; the gradient itself by its binary32 bound (below 2e-5)."""
    rng = np.random.default_rng(7)
    rows, hidden, step = 3, 40, 1e-4
    x, r, w = rng.normal(0, 1, (rows, hidden)), rng.normal(0, 1, (rows, hidden)), rng.normal(1, 0.3, hidden)
    x, r, w = (np.float32(t).astype(np.float64) for t in (x, r, w))
    cy, cr = rng.normal(0, 1, (rows, hidden)).astype(np.float32), rng.normal(0, 1, (rows, hidden)).astype(np.float32)

    def loss(x, r, w):
        h = x + r
        y = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-5) * w
        return (cy * y).sum() + (cr * h).sum()
    t = lambda v: torch.from_numpy(np.float32(v)).cuda()  # noqa: E731
    o = fq.fp4_add_rms_norm(t(x), t(w), t(r), eps=1e-5)
    g = fq.fp4_add_rms_norm_backward(t(cy), o["residual"], t(w), o["rstd"], dresidual=t(cr))
    for i, j in ((0, 0), (1, 7), (2, 39)):
        e = np.zeros((rows, hidden))
        e[i, j] = step
        for f in (lambda s: loss(x + s * e, r, w), lambda s: loss(x, r + s * e, w)):
            assert abs((f(1) - f(-1)) / (2 * step) - g["dx"][i, j].item()) < 3e-5
        e = e[i]
        assert abs((loss(x, r, w + e) - loss(x, r, w - e)) / (2 * step) - g["dweight"][j].item()) < 3e-5


def test_backward_views_in_place_no_rows_and_workspace():
    rng = np.random.default_rng(2)
    dy, h, d = (inputs(rng, 1300, 640, "bf16").cuda() for _ in range(3))
    w = torch.ones(320, device="cuda")
    rstd = torch.rand(1300, device="cuda") + 0.5
    v = [t[:, 16:336] for t in (dy, h, d)]
    want = fq.fp4_add_rms_norm_backward(v[0].contiguous(), v[1].contiguous(), w, rstd, dresidual=v[2].contiguous())
    got = fq.fp4_add_rms_norm_backward(v[0], v[1], w, rstd, dresidual=v[2])
    own = v[2].contiguous()
    need = fq.fp4q_add_rms_norm_backward_workspace_bytes(1300, 320)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    place = fq.fp4_add_rms_norm_backward(v[0], v[1], w, rstd, dresidual=own, dx=own, workspace=ws)
    for k in want:
        assert torch.equal(want[k], got[k]) and torch.equal(want[k], place[k])
    none = fq.fp4_add_rms_norm_backward(dy[:0, :320], h[:0, :320], w, rstd[:0],
                                        dweight=torch.full((320,), float("nan"), device="cuda"))
    assert none["dx"].shape == (0, 320) and (none["dweight"] == 0).all()
    with pytest.raises(fq.Fp4Error) as e:
        fq.fp4_add_rms_norm_backward(v[0], v[1], w, rstd, workspace=ws[:need - 16])
    assert e.value.status == fq.ERR_WORKSPACE
    assert fq.fp4_add_rms_norm(dy[:0, :320], w)["y"].shape == (0, 320)


def test_captured_replayed_and_on_another_stream():
    rng = np.random.default_rng(3)
    x, r, dy = (inputs(rng, 1200, 2880, "bf16").cuda() for _ in range(3))
    w = torch.rand(2880, device="cuda")
    out = {k: torch.empty_like(v) for k, v in fq.fp4_add_rms_norm(x, w, r, fp8="mx", y=True).items()}
    dx, dw = torch.empty_like(x), torch.empty(2880, device="cuda")
    ws = torch.empty(fq.fp4q_add_rms_norm_backward_workspace_bytes(1200, 2880), dtype=torch.uint8, device="cuda")

    def step():
        fq.fp4_add_rms_norm(x, w, r, fp8="mx", y=True, out=out)
        fq.fp4_add_rms_norm_backward(dy, out["residual"], w, out["rstd"], dx=dx, dweight=dw, workspace=ws)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    side = torch.cuda.Stream()
    for turn in range(3):
        x.mul_(0.5 + turn)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items()} | {"dx": dx.clone(), "dw": dw.clone()}
        for t in list(out.values()) + [dx, dw]:
            t.zero_()
        torch.cuda.synchronize()
        o = fq.fp4_add_rms_norm(x, w, r, fp8="mx", y=True, stream=side)
        b = fq.fp4_add_rms_norm_backward(dy, o["residual"], w, o["rstd"], stream=side)
        torch.cuda.synchronize()
        want = dict(o, dx=b["dx"], dw=b["dweight"])
        for k in got:
            assert torch.equal(got[k], want[k]), k
