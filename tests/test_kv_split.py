"""How attention cuts the keys of many rows, on the host: the parts of every tile
of rows hold every key that a row sees."""
import ctypes as ct
import os
import subprocess

import pytest
import torch

import block_scaled_fp4_amax_amd as fq

HERE = os.path.dirname(os.path.abspath(__file__))


def test_parts_hold_every_key(tmp_path):
    exe = str(tmp_path / "kv_split_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-o", exe, os.path.join(HERE, "pins", "kv_split_check.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr
    assert int(r.stdout.split()[1]) > 100000               # the sweep reaches windows whose keys are cut


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="placeholder device pointers: host-only validation")
def test_splits_whose_join_does_not_fit_a_launch():
    """The join takes 64 lanes a row; a launch has fewer than 2^32.  Calls beyond do not split."""
    cache = fq._KvCache(*[0x10000] * 4, None, None, 4, 16, 2, 64, 0)

    def need(total_q):
        a = fq._Attn(q=0x10000, ld_q=128, page_table=0x10000, kv_lens=0x10000, q_starts=0x10000, out=0x10000, scale=0.125,
                     batch=1, total_q=total_q, q_heads=2, table_cols=1 << 16, max_q=64, max_kv=1 << 20, causal=1, window=0)
        return fq.lib().fp4q_attn_workspace_bytes(ct.byref(fq.make_cfg()), ct.byref(cache), ct.byref(a))

    rows = (1 << 26) - 4                                      # 2^24 - 1 workgroups of 256 lanes
    assert need(rows // 2) > 0
    assert need(rows // 2 + 1) == 0 and need(1 << 26) == 0
