"""Refusals of the serving calls' binding (no GPU): arguments that the C entry points
cannot see are wrong."""
import ctypes as ct
import types

import pytest
import torch

import block_scaled_fp4_amax_amd as fq


@pytest.mark.parametrize("codes,scales", [(torch.int32, torch.uint8), (torch.uint8, torch.int32),
                                          (torch.uint8, torch.float32), (torch.int16, torch.int16)])
def test_linear_refuses_wider_codes_and_scales(codes, scales):
    """A wider type of the same shape is large enough and would be read as bytes."""
    w = {"codes": torch.zeros(4, 16, dtype=codes), "scales": torch.zeros(4, 2, dtype=scales), "outer": None}
    with pytest.raises(ValueError, match="bytes"):
        fq.fp4_linear(torch.zeros(2, 32, dtype=torch.bfloat16), w, fq.make_cfg())


def cpu_cache():
    """What the binding reads of a KVCache, on the host."""
    return types.SimpleNamespace(kv_heads=2, head_dim=64, page_size=16, num_pages=4, cfg=fq.make_cfg(),
                                 device=torch.device("cpu"), _by_dtype={torch.bfloat16: ct.byref(fq.make_cfg())}, _ref=None)


@pytest.mark.parametrize("kw", [dict(max_kv=(1 << 32) + 16), dict(max_q=(1 << 32) + 1), dict(window=(1 << 32) + 8),
                                dict(max_kv=-(1 << 32) + 16), dict(window=1 << 31)])
def test_attention_refuses_bounds_beyond_32_bits(kw):
    """Taken modulo 2^32 they would be small valid bounds, and keys or queries would be cut."""
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(fq.Fp4Error) as e:
        fq.fp4_attn(q, cpu_cache(), z(2, 4), z(2), z(3), **kw)
    assert e.value.status == fq.ERR_UNSUPPORTED
    with pytest.raises(fq.Fp4Error) as e:
        fq.fp4_attn_workspace(cpu_cache(), 2, 4, 2, table_cols=4, **kw)
    assert e.value.status == fq.ERR_UNSUPPORTED
