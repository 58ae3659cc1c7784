"""Sizes of fp4_attn_workspace (no GPU): for fp4_attn alone, for fp4_attn_tree alone, and for both."""
import ctypes as ct

import pytest
import torch

import block_scaled_fp4_amax_amd as fq


class Cache:
    """What fp4_attn_workspace reads of a KVCache, on the host."""
    page_size, device = 64, torch.device("cpu")

    def __init__(self, kv_heads, head_dim):
        self.cfg, self.head_dim = fq.make_cfg(), head_dim
        self.args = fq._KvCache(*[0x10000] * 4, None, None, 4, 64, kv_heads, head_dim, 0)
        self._ref = ct.byref(self.args)


def sizes(D, batch, n, max_kv):
    c, L = Cache(8, D), fq.lib()
    a = fq._Attn(q=0x10000, ld_q=64 * D, page_table=0x10000, kv_lens=0x10000, q_starts=0x10000, out=0x10000, scale=1.0, batch=batch,
                 total_q=batch * n, q_heads=64, table_cols=-(-max_kv // 64), max_q=n, max_kv=max_kv, causal=1, window=0)
    of = lambda t: 0 if t is None else t.numel()  # noqa: E731
    got = [of(fq.fp4_attn_workspace(c, batch * n, 64, batch, max_q=n, max_kv=max_kv, **kw)) for kw in (dict(trees=False), dict(trees=True), {})]
    need = [f(ct.byref(c.cfg), c._ref, ct.byref(a)) for f in (L.fp4q_attn_workspace_bytes, L.fp4q_attn_tree_workspace_bytes)]
    return got, need


@pytest.mark.parametrize("D,batch,n,max_kv", [(128, 1, 1024, 1024), (64, 16, 64, 8192), (64, 4, 26, 131072), (64, 48, 1, 8192), (256, 2, 3, 100)])
def test_sizes(D, batch, n, max_kv):
    got, need = sizes(D, batch, n, max_kv)
    assert got == [*need, max(need)]


def test_a_prompt_needs_none():
    """The scratch of a tree as large as a prompt is not what the prompt's attention needs."""
    got, _ = sizes(128, 1, 1024, 1024)
    assert got[0] == 0 and got[1] > 1 << 26
