"""GPU tests of the serving calls on a stream that is not the current one: what they
allocate is neither memory that the current stream's queued work still writes, nor is it
handed out again while the current stream still reads it."""
import pytest
import torch

import block_scaled_fp4_amax_amd as fq

pytestmark = pytest.mark.gpu

TOKENS, H, D = 16384, 4, 64


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.lib()


def cache_of(value):
    c = fq.KVCache.empty(TOKENS // 64, 64, H, D, fq.make_cfg(format="mxfp4"))
    for codes, scales in ((c.k_codes, c.k_scales), (c.v_codes, c.v_scales)):
        codes.fill_(value * 0x11)
        scales.fill_(127)
    return c


def busy(a):
    """Queues some milliseconds of work on the current stream."""
    for _ in range(20):
        a = (a @ a).clamp_(-1, 1)
    return a


def test_results_are_not_memory_that_the_current_stream_still_writes():
    cache, a = cache_of(4), torch.randn(4096, 4096, device="cuda")      # code 4 is 2.0
    slots = torch.arange(TOKENS, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy(a)
    old = [torch.empty(TOKENS, H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    for t in old:
        t.fill_(7.0)                                                    # still queued when the memory is freed
    del t, old
    k, v = fq.fp4_kv_read(cache, slots, stream=side)
    torch.cuda.synchronize()
    assert (k == 2.0).all() and (v == 2.0).all()


def test_results_are_kept_until_the_current_stream_has_read_them():
    twos, fours, a = cache_of(4), cache_of(6), torch.randn(4096, 4096, device="cuda")
    slots = torch.arange(TOKENS, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = fq.fp4_kv_read(twos, slots, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    busy(a)
    kept = [t.clone() for t in out]                                     # reads out after the work before it
    del out
    again = fq.fp4_kv_read(fours, slots, stream=side)
    torch.cuda.synchronize()
    assert all((t == 2.0).all() for t in kept) and all((t == 4.0).all() for t in again)


@pytest.mark.parametrize("handle", [False, True])
def test_every_call_allocates_from_its_stream(handle):
    """Blocks that the current stream just freed are not handed to a call on another one."""
    cache = cache_of(4)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    s = side.cuda_stream if handle else side
    x, q = torch.ones(512, 4096, dtype=torch.bfloat16, device="cuda"), torch.ones(4096, 2 * H, D, dtype=torch.bfloat16, device="cuda")
    wt = {"codes": torch.zeros(4096, 2048, dtype=torch.uint8, device="cuda"),
          "scales": torch.full((4096, 128), 127, dtype=torch.uint8, device="cuda"), "outer": None}
    table = torch.arange(TOKENS // 64, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([TOKENS], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 4096], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for call in (lambda: fq.fp4_linear(x, wt, fq.make_cfg(format="mxfp4"), stream=s),
                 lambda: fq.fp4_attn(q, cache, table, lens, starts, stream=s)):
        call()
        torch.cuda.synchronize()
        freed = torch.empty(4096 * 2 * H * D * 2, dtype=torch.uint8, device="cuda")     # as large as either result
        at, end = freed.data_ptr(), freed.data_ptr() + freed.nbytes
        del freed
        y = call()
        torch.cuda.synchronize()
        assert not at <= y.data_ptr() < end
