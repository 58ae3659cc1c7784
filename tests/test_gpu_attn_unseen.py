"""GPU tests of attention with bytes that the quantiser never writes (they decode to
infinities and NaN): what unseen keys hold never reaches a result, bit for bit."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
import kv_reference as R
from test_gpu_attn import A_P, Setup, U_OUT, U_P

pytestmark = pytest.mark.gpu

# scale bytes beyond the largest that the quantiser writes
BYTES = {"mxfp4": (253, 254, 255), "nvfp4": (0x7F, 0xE8, 0xF8, 0xFF), "amdfp4": (0xFF,)}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "amdfp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_lens,window,wide", [([1, 1, 1], 40, 0), ([5, 2, 1], 77, 100), ([40, 33, 1], 50, 0), ([40], 1000, 400)])
def test_bytes_before_the_window(fmt, D, q_lens, window, wide):
    kv = [1717, 207, 95][:len(q_lens)]
    s = Setup(fmt, D, 2, 2, 16, kv, q_lens, extra_cols=wide)
    want, wl = s.device().check(window=window, max_q=max(q_lens))
    rng = np.random.default_rng(D)
    for c in "kv":
        for b, (n, q) in enumerate(zip(kv, q_lens)):
            for t in range(n - q + 1 - window):               # the first query sees keys from here on
                page, at = s.table[b, t // 16], t % 16
                scales = s.buf[c + "_scales"][page, :, at]
                scales[:] = rng.choice(BYTES[fmt], scales.shape)
                s.buf[c + "_codes"][page, :, at] = 0x7F
    out, lse = s.device().run(window=window, max_q=max(q_lens))
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("fmt", ["nvfp4", "amdfp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G", [(6, 2), (70, 2)])
def test_bytes_that_later_queries_see(fmt, D, n, G):
    """A key between a chunk's queries: those before it stay within their bounds (their last bits may
    follow the running maximum, which moves for all rows of a tile together)."""
    s = Setup(fmt, D, 1, G, 16, [300, 17], [n, 1])
    o, l, tol, ltol = R.attention(s.q.double().numpy(), s.buf, fmt, 16, s.table, s.kv_lens, s.q_starts,
                                  float(np.float32(D ** -0.5)), u_p=U_P[fmt], a_p=A_P[fmt])
    at = 300 - n // 2                                         # seen by the last n // 2 queries
    for c in "kv":
        s.buf[c + "_scales"][s.table[0, at // 16], 0, at % 16] = 0xFF
        s.buf[c + "_codes"][s.table[0, at // 16], 0, at % 16] = 0x7F
    out, lse = (t.double().cpu().numpy() for t in s.device().run())
    u = U_OUT[torch.bfloat16]
    bound = tol * (1 + u) + u * np.abs(o) + 1e-37
    for rows in (slice(0, n - n // 2), slice(n, None)):
        assert np.all(np.abs(out - o)[rows] <= bound[rows]) and np.all(np.abs(lse - l)[rows] <= ltol[rows])
