"""Host-side checks of fp4_attn_tree (no GPU): what a tree's queries see of the context against its
plain definition, and refusals before anything is enqueued."""
import ctypes as ct
import os
import subprocess
import types

import pytest
import torch

import block_scaled_fp4_amax_amd as fq

HERE = os.path.dirname(os.path.abspath(__file__))
FAKE = 0x10000
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="placeholder device pointers: host-only validation")


def test_context_ranges(tmp_path):
    exe = str(tmp_path / "tree_context_check")
    subprocess.run(["g++", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-std=c++17", "-o", exe,
                    os.path.join(HERE, "pins", "tree_context_check.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def tree(cache=None, cfg=None, mask=FAKE, cols=3, ws=None, wsb=0, **kw):
    c = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, k_outer=None, v_outer=None, num_pages=4,
             page_size=16, kv_heads=2, head_dim=64, reserved=0)
    c.update(cache or {})
    d = dict(q=FAKE, ld_q=256, page_table=FAKE, kv_lens=FAKE, q_starts=FAKE, sinks=None, out=FAKE, lse=None, scale=0.125,
             batch=2, total_q=5, q_heads=4, table_cols=4, max_q=3, max_kv=64, causal=1, window=0)
    d.update(kw)
    cfg = cfg if cfg is not None else fq.make_cfg()
    st = fq.lib().fp4_attn_tree(ct.byref(cfg), ct.byref(fq._KvCache(**c)), ct.byref(fq._Attn(**d)), mask, cols, ws, wsb, None)
    assert st != fq.ERR_HIP, "a call reached a launch"
    return st


@no_gpu
@pytest.mark.parametrize("kw,st", [
    (dict(mask=None), fq.ERR_NULL), (dict(cols=-1), fq.ERR_SHAPE), (dict(cols=1 << 30), fq.ERR_UNSUPPORTED), (dict(causal=0), fq.ERR_MODE), (dict(causal=0, window=3), fq.ERR_MODE),
    (dict(q=None), fq.ERR_NULL), (dict(kv_lens=None), fq.ERR_NULL), (dict(out=None), fq.ERR_NULL), (dict(q_heads=3), fq.ERR_SHAPE),
    (dict(window=-1), fq.ERR_SHAPE), (dict(scale=0.0), fq.ERR_MODE), (dict(cache=dict(head_dim=32)), fq.ERR_UNSUPPORTED),
    (dict(max_kv=1 << 28), fq.ERR_UNSUPPORTED), (dict(q=FAKE + 4), fq.ERR_ALIGN), (dict(batch=0), fq.OK), (dict(max_q=0), fq.OK),
    (dict(table_cols=512, max_kv=8192), fq.ERR_WORKSPACE)])
def test_refusals(kw, st):
    assert tree(**kw) == st


def cpu_cache():
    return types.SimpleNamespace(kv_heads=2, head_dim=64, page_size=16, num_pages=4, cfg=fq.make_cfg(), device=torch.device("cpu"),
                                 _by_dtype={torch.bfloat16: ct.byref(fq.make_cfg())}, _ref=None)


@pytest.mark.parametrize("mask", [torch.ones(4, 4, dtype=torch.bool), torch.ones(5, dtype=torch.bool), torch.ones(5, 5),
                                  torch.ones(5, 5, dtype=torch.int64), torch.ones(5, 9, dtype=torch.bool)[:, :5]])
def test_binding_refuses_masks(mask):
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="tree"):
        fq.fp4_attn_tree(q, cpu_cache(), z(2, 4), z(2), z(3), mask)
    with pytest.raises(TypeError):
        fq.fp4_attn_tree(q, cpu_cache(), z(2, 4), z(2), z(3), torch.ones(5, 5, dtype=torch.bool), causal=True)
