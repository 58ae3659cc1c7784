"""Refusals of fp4_kv_append_rope, fp4_add_rms_norm and its gradient before anything is
enqueued (no GPU): the C entry points' statuses, and the binding's checks."""
import ctypes as ct
import types

import pytest
import torch

import block_scaled_fp4_amax_amd as fq

FAKE, MIS = 0x10000, 0x10004
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="placeholder device pointers: host-only validation")


def status(st):
    assert st != fq.ERR_HIP, "a call reached a launch"
    return st


def rope(cfg=None, cache=None, **kw):
    d = dict(k=FAKE, v=FAKE, q=FAKE, q_out=FAKE + 4096, ld_k=128, ld_v=128, ld_q=256, ld_q_out=256, slots=FAKE, positions=FAKE,
             cos=FAKE, sin=FAKE, tokens=3, table_rows=9, rot_dim=64, q_heads=4, interleaved=0, reserved=0)
    d.update(kw)
    c = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, k_outer=None, v_outer=None, num_pages=4,
             page_size=16, kv_heads=2, head_dim=64, reserved=0)
    c.update(cache or {})
    cfg = cfg if cfg is not None else fq.make_cfg()
    return status(fq.lib().fp4_kv_append_rope(ct.byref(cfg), ct.byref(fq._KvCache(**c)), ct.byref(fq._KvRope(**d)), None))


@no_gpu
@pytest.mark.parametrize("kw,st", [
    (dict(k=None), fq.ERR_NULL), (dict(v=None), fq.ERR_NULL), (dict(slots=None), fq.ERR_NULL), (dict(positions=None), fq.ERR_NULL),
    (dict(cos=None), fq.ERR_NULL), (dict(sin=None), fq.ERR_NULL), (dict(q=None), fq.ERR_NULL), (dict(q_out=None), fq.ERR_NULL),
    (dict(k=MIS), fq.ERR_ALIGN), (dict(q=MIS), fq.ERR_ALIGN), (dict(q_out=MIS), fq.ERR_ALIGN), (dict(cos=MIS), fq.ERR_ALIGN),
    (dict(sin=MIS), fq.ERR_ALIGN), (dict(slots=MIS), fq.ERR_ALIGN), (dict(positions=FAKE + 2), fq.ERR_ALIGN),
    (dict(ld_k=129), fq.ERR_ALIGN), (dict(ld_q=260), fq.ERR_ALIGN), (dict(ld_q_out=257), fq.ERR_ALIGN),
    (dict(ld_k=120), fq.ERR_SHAPE), (dict(ld_v=64), fq.ERR_SHAPE), (dict(ld_q=248), fq.ERR_SHAPE), (dict(tokens=-1), fq.ERR_SHAPE),
    (dict(table_rows=-1), fq.ERR_SHAPE), (dict(rot_dim=0), fq.ERR_SHAPE), (dict(rot_dim=24), fq.ERR_SHAPE),
    (dict(rot_dim=80), fq.ERR_SHAPE), (dict(rot_dim=-16), fq.ERR_SHAPE), (dict(q_heads=0), fq.ERR_SHAPE),
    (dict(q_out=FAKE, ld_q_out=264), fq.ERR_SHAPE), (dict(interleaved=2), fq.ERR_MODE), (dict(tokens=1 << 28), fq.ERR_UNSUPPORTED),
    (dict(q_heads=65536, ld_q=1 << 23, ld_q_out=1 << 23), fq.ERR_UNSUPPORTED), (dict(table_rows=1 << 32), fq.ERR_UNSUPPORTED),
    (dict(q_heads=65532, ld_q=1 << 23, ld_q_out=1 << 23), fq.ERR_UNSUPPORTED),
    (dict(q_heads=32766, ld_q=1 << 23, ld_q_out=1 << 23), fq.ERR_UNSUPPORTED)])   # with kv_heads, 2^15
def test_rope_refusals(kw, st):
    assert rope(**kw) == st


@no_gpu
def test_rope_configurations_and_empty_calls():
    assert rope(cfg=fq.make_cfg(rounding="stochastic")) == fq.ERR_UNSUPPORTED
    assert rope(cfg=fq.make_cfg(input_dtype="fp16")) == fq.ERR_DTYPE
    assert rope(cache=dict(head_dim=96)) == fq.ERR_UNSUPPORTED
    assert rope(tokens=0) == fq.OK
    assert rope(cache=dict(num_pages=0), q=None, q_out=None) == fq.OK


def norm(**kw):
    d = dict(x=FAKE, residual=FAKE, ld_x=64, ld_residual=64, weight=FAKE, residual_out=FAKE, rstd=FAKE, y=FAKE, fp8=FAKE,
             fp8_scales=FAKE, rows=3, hidden=64, eps=1e-5, x_dtype=0, residual_dtype=2, weight_dtype=0, y_dtype=0, fp8_mode=1,
             reserved=0)
    d.update(kw)
    return status(fq.lib().fp4_add_rms_norm(ct.byref(fq._AddRmsNorm(**d)), None))


@no_gpu
@pytest.mark.parametrize("kw,st", [
    (dict(x=None), fq.ERR_NULL), (dict(weight=None), fq.ERR_NULL), (dict(residual_out=None), fq.ERR_NULL),
    (dict(residual=None), fq.ERR_NULL), (dict(fp8=None), fq.ERR_NULL), (dict(fp8_scales=None), fq.ERR_NULL),
    (dict(x=MIS), fq.ERR_ALIGN), (dict(residual=MIS), fq.ERR_ALIGN), (dict(weight=MIS), fq.ERR_ALIGN), (dict(y=MIS), fq.ERR_ALIGN),
    (dict(fp8=MIS), fq.ERR_ALIGN), (dict(rstd=FAKE + 2), fq.ERR_ALIGN), (dict(fp8_mode=2, fp8_scales=FAKE + 1), fq.ERR_ALIGN),
    (dict(ld_x=68), fq.ERR_ALIGN), (dict(ld_residual=66), fq.ERR_ALIGN), (dict(ld_x=56), fq.ERR_SHAPE),
    (dict(ld_residual=32), fq.ERR_SHAPE), (dict(rows=-1), fq.ERR_SHAPE), (dict(hidden=0), fq.ERR_SHAPE), (dict(hidden=-8), fq.ERR_SHAPE),
    (dict(hidden=60), fq.ERR_SHAPE), (dict(hidden=56), fq.ERR_SHAPE), (dict(hidden=16416, ld_x=16416, ld_residual=16416), fq.ERR_UNSUPPORTED),
    (dict(rows=1 << 28), fq.ERR_UNSUPPORTED), (dict(rows=1 << 40), fq.ERR_UNSUPPORTED), (dict(x_dtype=1), fq.ERR_DTYPE),
    (dict(residual_dtype=3), fq.ERR_DTYPE), (dict(weight_dtype=-1), fq.ERR_DTYPE), (dict(y_dtype=1), fq.ERR_DTYPE),
    (dict(fp8_mode=3), fq.ERR_MODE), (dict(fp8_mode=-1), fq.ERR_MODE), (dict(eps=-1e-5), fq.ERR_MODE), (dict(eps=float("nan")), fq.ERR_MODE),
    (dict(rows=1 << 26), fq.ERR_UNSUPPORTED), (dict(rows=1 << 26, hidden=32), fq.ERR_UNSUPPORTED), (dict(rows=0, x=None), fq.OK)])
def test_norm_refusals(kw, st):
    assert norm(**kw) == st


def grad(ws=FAKE, wsb=1 << 30, **kw):
    d = dict(dy=FAKE, h=FAKE, dresidual=FAKE, ld_dy=64, ld_h=64, ld_dresidual=64, weight=FAKE, rstd=FAKE, dx=FAKE, dweight=FAKE,
             rows=300, hidden=64, dy_dtype=0, h_dtype=0, weight_dtype=2, reserved=0)
    d.update(kw)
    return status(fq.lib().fp4_add_rms_norm_backward(ct.byref(fq._RmsNormGrad(**d)), ws, wsb, None))


@no_gpu
@pytest.mark.parametrize("kw,st", [
    (dict(dy=None), fq.ERR_NULL), (dict(h=None), fq.ERR_NULL), (dict(weight=None), fq.ERR_NULL), (dict(rstd=None), fq.ERR_NULL),
    (dict(dx=None), fq.ERR_NULL), (dict(rows=0, weight=None), fq.ERR_NULL), (dict(dy=MIS), fq.ERR_ALIGN), (dict(h=MIS), fq.ERR_ALIGN),
    (dict(dresidual=MIS), fq.ERR_ALIGN), (dict(dx=MIS), fq.ERR_ALIGN), (dict(dweight=MIS), fq.ERR_ALIGN),
    (dict(ld_dy=68), fq.ERR_ALIGN), (dict(ld_h=68), fq.ERR_ALIGN), (dict(ld_dresidual=68), fq.ERR_ALIGN),
    (dict(ld_dy=8), fq.ERR_SHAPE), (dict(ld_h=8), fq.ERR_SHAPE), (dict(ld_dresidual=8), fq.ERR_SHAPE), (dict(hidden=12), fq.ERR_SHAPE),
    (dict(rows=-2), fq.ERR_SHAPE), (dict(dy_dtype=1), fq.ERR_DTYPE), (dict(h_dtype=5), fq.ERR_DTYPE),
    (dict(ws=None), fq.ERR_WORKSPACE), (dict(wsb=16), fq.ERR_WORKSPACE), (dict(ws=MIS), fq.ERR_ALIGN),
    (dict(rows=1 << 26), fq.ERR_UNSUPPORTED), (dict(rows=0, dweight=None, weight=None), fq.OK)])
def test_norm_gradient_refusals(kw, st):
    assert grad(**kw) == st


def test_gradient_workspace():
    f = fq.fp4q_add_rms_norm_backward_workspace_bytes
    assert f(1, 64) == 0 and f(0, 64) == 0 and f(-1, 64) == 0 and f(5, 60) == 0
    assert f(1 << 20, 2880) == 256 * 2880 * 4


def cpu_cache():
    return types.SimpleNamespace(kv_heads=2, head_dim=64, page_size=16, num_pages=4, cfg=fq.make_cfg(), device=torch.device("cpu"),
                                 _by_dtype={torch.bfloat16: ct.byref(fq.make_cfg())}, _ref=None)


@pytest.mark.parametrize("change,error", [
    (dict(positions=torch.zeros(3, dtype=torch.int64)), "positions"), (dict(positions=torch.zeros(2, dtype=torch.int32)), "positions"),
    (dict(cos=torch.zeros(9, 32, dtype=torch.float64)), "cos"), (dict(sin=torch.zeros(9, 16)), "cos"),
    (dict(q_out=torch.zeros(3, 4, 64, dtype=torch.bfloat16), q=None), "q_out"), (dict(q=torch.zeros(2, 4, 64, dtype=torch.bfloat16)), "tokens"),
    (dict(q=torch.zeros(3, 4, 32, dtype=torch.bfloat16)), "q must"), (dict(v=torch.zeros(2, 2, 64, dtype=torch.bfloat16)), "agree"),
    (dict(q=torch.zeros(3, 4, 64)), "dtype"), (dict(slots=torch.zeros(3, dtype=torch.int32)), "slots")])
def test_rope_binding_refusals(change, error):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    a = dict(k=z(3, 2, 64), v=z(3, 2, 64), slots=torch.zeros(3, dtype=torch.int64), positions=torch.zeros(3, dtype=torch.int32),
             cos=torch.zeros(9, 32), sin=torch.zeros(9, 32), q=z(3, 4, 64))
    a.update(change)
    with pytest.raises((ValueError, fq.Fp4Error), match=error):
        fq.fp4_kv_append_rope(cpu_cache(), **a)


def test_norm_binding_refusals():
    x, w = torch.zeros(3, 64, dtype=torch.bfloat16), torch.ones(64)
    for bad, error in ((dict(x=x), "device tensors"), (dict(x=x.half()), "dtype"), (dict(x=x[0]), "2-D"), (dict(fp8="col"), "fp8"),
                       (dict(x=torch.zeros(64, 3).t()), "contiguous")):
        a = dict(x=x, weight=w)
        a.update(bad)
        with pytest.raises((ValueError, fq.Fp4Error), match=error):
            fq.fp4_add_rms_norm(**a)
    with pytest.raises(ValueError, match="device tensors"):
        fq.fp4_add_rms_norm_backward(x, x, w, torch.ones(3))
