"""What the attention calls take (no GPU): a mask goes through fp4_attn_tree alone, which checks it."""
import inspect
import types

import pytest
import torch

import block_scaled_fp4_amax_amd as fq


def test_no_private_arguments():
    for f in (fq.fp4_attn, fq.fp4_attn_tree):
        assert not [n for n in inspect.signature(f).parameters if n.startswith("_")]
    tree, plain = (list(inspect.signature(f).parameters) for f in (fq.fp4_attn_tree, fq.fp4_attn))
    assert [n for n in tree if n != "tree"] == [n for n in plain if n != "causal"]


def test_fp4_attn_takes_no_mask():
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    cache = types.SimpleNamespace(device=torch.device("cpu"))
    with pytest.raises(TypeError):
        fq.fp4_attn(q, cache, z(2, 4), z(2), z(3), _tree=torch.zeros(1, 1))
    with pytest.raises(TypeError):
        fq.fp4_attn_tree(q, cache, z(2, 4), z(2), z(3), torch.ones(5, 5, dtype=torch.bool), causal=True)
