"""The norm and its gradient in place, on the host: rows with a pitch, which their contiguous output would overwrite while they
are read, are refused before anything is enqueued."""
import ctypes as ct

import pytest
import torch

import block_scaled_fp4_amax_amd as fq

A, B = 0x10000, 0x80000
pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="placeholder device pointers: host-only validation")


def norm(**kw):
    d = dict(x=A, residual=B, ld_x=64, ld_residual=64, weight=A, residual_out=B, rstd=None, y=A, fp8=None, fp8_scales=None, rows=3,
             hidden=64, eps=1e-5, x_dtype=0, residual_dtype=0, weight_dtype=0, y_dtype=0, fp8_mode=0, reserved=0)
    d.update(kw)
    return fq.lib().fp4_add_rms_norm(ct.byref(fq._AddRmsNorm(**d)), None)


def grad(**kw):
    d = dict(dy=A, h=A, dresidual=B, ld_dy=64, ld_h=64, ld_dresidual=64, weight=A, rstd=A, dx=B, dweight=A, rows=300, hidden=64,
             dy_dtype=0, h_dtype=0, weight_dtype=2, reserved=0)
    d.update(kw)
    return fq.lib().fp4_add_rms_norm_backward(ct.byref(fq._RmsNormGrad(**d)), A, 1 << 30, None)


@pytest.mark.parametrize("dtype", [0, 2])
@pytest.mark.parametrize("pitch", [72, 128, 4096])
def test_pitched_rows_in_place(dtype, pitch):
    assert norm(ld_residual=pitch, residual_dtype=dtype) == fq.ERR_SHAPE
    assert grad(ld_dresidual=pitch, h_dtype=dtype) == fq.ERR_SHAPE


def test_others_reach_the_launch():
    """Contiguous rows in place, one row of any pitch, pitched rows with another output: without a GPU, a launch's error."""
    for kw in ({}, dict(rows=1, ld_residual=72), dict(ld_residual=72, residual_out=A), dict(residual=None, residual_out=None)):
        assert norm(**kw) == fq.ERR_HIP
    for kw in ({}, dict(rows=1, ld_dresidual=72), dict(ld_dresidual=72, dx=A), dict(dresidual=None)):
        assert grad(**kw) == fq.ERR_HIP
