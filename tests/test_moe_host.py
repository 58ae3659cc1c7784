"""Refusals of fp4_moe before anything is enqueued (no GPU): the C entry point's statuses, and the
binding's checks."""
import ctypes as ct

import pytest
import torch

import block_scaled_fp4_amax_amd as fq

FAKE, MIS = 0x10000, 0x10004
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="placeholder device pointers: host-only validation")


def moe(cfg=None, ws=FAKE, wsb=1 << 30, **kw):
    a = dict(x=FAKE, ld_x=128, logits=FAKE, w1_codes=FAKE, w1_scales=FAKE, w1_outer=None, w2_codes=FAKE, w2_scales=FAKE,
             w2_outer=None, b1=None, b2=None, y=FAKE, ld_y=128, tokens=4, experts=8, hidden=128, inter=64, top_k=2,
             renormalize=1, interleaved=0, reserved=0, alpha=1.0, limit=0.0, shift=0.0)
    a.update(kw)
    cfg = cfg if cfg is not None else fq.make_cfg()
    st = fq.lib().fp4_moe(ct.byref(cfg), ct.byref(fq._Moe(**a)), ws, wsb, None)
    assert st != fq.ERR_HIP, "a call reached a launch"
    return st


@no_gpu
@pytest.mark.parametrize("kw,st", [
    (dict(x=None), fq.ERR_NULL), (dict(logits=None), fq.ERR_NULL), (dict(w1_codes=None), fq.ERR_NULL), (dict(w2_scales=None), fq.ERR_NULL),
    (dict(y=None), fq.ERR_NULL), (dict(x=MIS), fq.ERR_ALIGN), (dict(w1_codes=MIS), fq.ERR_ALIGN), (dict(w2_codes=MIS), fq.ERR_ALIGN),
    (dict(logits=FAKE + 2), fq.ERR_ALIGN), (dict(y=FAKE + 1), fq.ERR_ALIGN), (dict(b1=FAKE + 2), fq.ERR_ALIGN), (dict(ld_x=132), fq.ERR_ALIGN),
    (dict(ld_x=120), fq.ERR_SHAPE), (dict(ld_x=(1 << 22) + 8), fq.ERR_UNSUPPORTED), (dict(ld_y=127), fq.ERR_SHAPE), (dict(hidden=48), fq.ERR_SHAPE), (dict(inter=16), fq.ERR_SHAPE),
    (dict(hidden=0), fq.ERR_SHAPE), (dict(inter=-32), fq.ERR_SHAPE), (dict(experts=0), fq.ERR_SHAPE), (dict(top_k=0), fq.ERR_SHAPE),
    (dict(top_k=9), fq.ERR_SHAPE), (dict(tokens=-1), fq.ERR_SHAPE), (dict(tokens=1025), fq.ERR_UNSUPPORTED),
    (dict(experts=513), fq.ERR_UNSUPPORTED), (dict(experts=64, top_k=33), fq.ERR_UNSUPPORTED), (dict(hidden=65568, ld_x=65568, ld_y=65568), fq.ERR_UNSUPPORTED),
    (dict(inter=65568), fq.ERR_UNSUPPORTED), (dict(renormalize=2), fq.ERR_MODE), (dict(interleaved=-1), fq.ERR_MODE),
    (dict(limit=-1.0), fq.ERR_MODE), (dict(limit=float("nan")), fq.ERR_MODE), (dict(alpha=float("nan")), fq.ERR_MODE),
    (dict(shift=float("nan")), fq.ERR_MODE), (dict(ws=None), fq.ERR_WORKSPACE), (dict(wsb=1024), fq.ERR_WORKSPACE),
    (dict(ws=MIS), fq.ERR_ALIGN), (dict(tokens=0, x=None, ws=None), fq.OK),
    (dict(w1_scales=FAKE + 1), fq.ERR_ALIGN), (dict(w2_scales=FAKE + 1), fq.ERR_ALIGN)])
def test_refusals(kw, st):
    assert moe(**kw) == st


@no_gpu
def test_configurations():
    outer = lambda **kw: fq.make_cfg(format="nvfp4", two_level="outer_block", **kw)  # noqa: E731
    assert moe(cfg=fq.make_cfg(input_dtype="fp32")) == fq.ERR_UNSUPPORTED
    assert moe(cfg=outer(outer_block_size=64, outer_2d=True)) == fq.ERR_NULL
    assert moe(cfg=outer(outer_block_size=128, outer_2d=True), inter=128, w1_outer=FAKE, w2_outer=FAKE) == fq.ERR_UNSUPPORTED
    assert moe(cfg=outer(outer_block_size=32), w1_outer=FAKE, w2_outer=FAKE) == fq.ERR_UNSUPPORTED
    assert moe(cfg=outer(outer_block_size=128), w1_outer=FAKE, w2_outer=FAKE) == fq.ERR_SHAPE      # inter 64
    assert moe(cfg=outer(outer_block_size=64, outer_2d=True), inter=96, w1_outer=FAKE, w2_outer=FAKE) == fq.ERR_SHAPE


def test_workspace_sizes():
    f = fq.fp4q_moe_workspace_bytes
    assert f(0, 8, 2, 128, 64) == 0 and f(1025, 8, 2, 128, 64) == 0 and f(4, 8, 9, 128, 64) == 0 and f(4, 8, 2, 100, 64) == 0
    assert f(4, 8, 2, 128, 64) >= 2 * 4 * 2 * 64 * 2


def test_binding_refusals():
    z = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype)  # noqa: E731
    good = dict(x=z(4, 128, dtype=torch.bfloat16), logits=z(4, 8, dtype=torch.float32), cfg=fq.make_cfg(), top_k=2,
                w1=dict(codes=z(8, 128, 64), scales=z(8, 128, 8)), w2=dict(codes=z(8, 128, 32), scales=z(8, 128, 4)))
    t = fq.make_cfg(two_level="tensorwise")
    for change, error in ((dict(), "device tensors"), (dict(x=good["x"].float()), "dtype"), (dict(logits=good["logits"].double()), "float32"),
                          (dict(logits=z(3, 8, dtype=torch.float32)), "logits"), (dict(w1=dict(codes=z(8, 64, 64), scales=z(8, 64, 8))), "w1"),
                          (dict(w1=dict(codes=z(8, 128, 64), scales=z(8, 128, 7))), "w1 scales"),
                          (dict(w2=dict(codes=z(8, 128, 32, dtype=torch.int16), scales=z(8, 128, 4))), "bytes"),
                          (dict(w2=dict(codes=z(7, 128, 32), scales=z(7, 128, 4))), "w1 codes"), (dict(cfg=t), "outer"),
                          (dict(b1=z(8, 64, dtype=torch.float32)), "b1"), (dict(b2=z(8, 128, dtype=torch.bfloat16)), "b2")):
        with pytest.raises((ValueError, fq.Fp4Error), match=error):
            fq.fp4_moe(**{**good, **change})


@pytest.mark.parametrize("experts,top_k", [(1, 1), (3, 1), (3, 3), (8, 2), (8, 4), (32, 4), (40, 5), (128, 8), (512, 32)])
def test_a_workspace_of_more_tokens_serves_fewer(experts, top_k):
    need = [fq.fp4q_moe_workspace_bytes(t, experts, top_k, 2880, 736) for t in range(0, 260)]
    assert need[0] == 0 and all(a <= b for a, b in zip(need, need[1:]))
