"""Refusals of the serving calls' binding (no GPU): arguments that the C entry points
cannot see are wrong."""
import contextlib
import ctypes as ct
import os
import subprocess
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


def test_what_is_done_once_is_done_on_each_device(tmp_path):
    """The kernels' LDS limits are raised on every device that launches them."""
    exe = str(tmp_path / "per_device_check")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "pins", "per_device_check.cpp")
    subprocess.run(["g++", "-O1", "-std=c++17", "-o", exe, src], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_calls_run_with_the_device_of_their_tensors(monkeypatch):
    seen, current = [], [0]

    @contextlib.contextmanager
    def on(device):
        before, current[0] = current[0], device.index
        yield
        current[0] = before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", on)

    def entry(*args):
        seen.append((current[0], args))
        return 0 if args[0] else fq.ERR_SHAPE

    fq._launch("fp4_attn", entry, torch.device("cuda", 3), 1, 2)
    fq._launch("fp4_attn", entry, torch.device("cuda", 0), 5)
    assert seen == [(3, (1, 2)), (0, (5,))] and current == [0]
    with pytest.raises(fq.Fp4Error, match="fp4_attn"):
        fq._launch("fp4_attn", entry, torch.device("cuda", 1), 0)
