"""GPU parity of fp4_kv_append_rope where a workgroup takes 2, 4 or 8 heads one after another (prompts), with counts of
heads that these do not divide: the same comparisons, bit for bit, as tests/test_gpu_kv_rope.py."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_amax_amd as fq
from test_gpu_kv import dev, new_cache, rows
from test_gpu_kv_rope import check_cache, f32, same_bits, tables, turned

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]

HQ, H = 35, 5


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


def heads_of_a_workgroup(tokens, dim):
    """The launcher's choice: as many as leave 1024 workgroups, 256 lanes of 16 values each."""
    runs, per = -(-tokens // (256 // (dim // 16))), 1
    while per < 8 and runs * (2 * H + HQ) // (2 * per) >= 1024:
        per *= 2
    return per


@pytest.mark.parametrize("per,fmt,outer,dtype,D,rot,interleaved", [
    (2, "mxfp4", False, "bf16", 64, 64, False), (2, "nvfp4", True, "fp32", 128, 48, True), (4, "amdfp4", True, "bf16", 256, 256, True),
    (4, "nvfp4", False, "fp32", 64, 32, False), (8, "mxfp4", False, "fp32", 128, 128, False), (8, "nvfp4", True, "bf16", 256, 144, False),
    (8, "amdfp4", True, "bf16", 64, 16, True)])
def test_heads_one_after_another(per, fmt, outer, dtype, D, rot, interleaved):
    tokens_a_run = 256 // (D // 16)
    T = {2: 47, 4: 93, 8: 184}[per] * tokens_a_run - tokens_a_run // 2 - 1
    assert heads_of_a_workgroup(T, D) == per
    rng = np.random.default_rng(per + D)
    page = 48
    pages = -(-T // page) + 2
    c, d = (new_cache(fmt, pages, page, H, D, outer, np.random.default_rng(per)) for _ in "cd")
    qkv = rows(rng, T, HQ + 2 * H, D, dtype)
    q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + H], qkv[:, HQ + H:]
    cos, sin = tables(700, rot // 2)
    positions = rng.integers(0, 700, T).astype(np.int32)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[T // 2:T // 2 + 9] = [-1, -(1 << 62), pages * page, 1 << 62, -1, -1, -1, -1, -1]
    lost = np.arange(T) % 37 == 5
    positions[lost] = rng.choice([-1, 700, 1 << 30, -(1 << 31)], lost.sum())
    at = np.where(lost, 0, positions)
    want = turned(q, at, cos, sin, interleaved)
    want[lost] = 0
    tk, written = turned(k, at, cos, sin, interleaved), (slots >= 0) & (slots < pages * page) & ~lost
    rest = dev(slots), dev(positions), dev(cos), dev(sin)
    got = fq.fp4_kv_append_rope(c, dev(k), dev(v), *rest, q=dev(q), interleaved=interleaved)
    torch.cuda.synchronize()
    same_bits(got, want)
    check_cache(c, fmt, tk, f32(v), slots, written)
    # views of one projection, the queries where they are
    x = dev(qkv)
    dq, dk, dv = x.split([HQ, H, H], 1)
    before = x[:, HQ:].clone()
    fq.fp4_kv_append_rope(d, dk, dv, *rest, q=dq, q_out=dq, interleaved=interleaved)
    torch.cuda.synchronize()
    bits = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(dq.view(bits), got.view(bits)) and torch.equal(x[:, HQ:].view(bits), before.view(bits))
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(c, n), getattr(d, n)), n
