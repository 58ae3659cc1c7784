"""One decoder layer's attention served in 4 bits: NVFP4 projections, a paged
NVFP4 cache of keys and values, prompts and then single tokens.

    python examples/decode_layer.py [--tokens N]

Each step multiplies the hidden states with the quantised QKV weight
(fp4_linear), writes the new keys and values into the cache (fp4_kv_append),
attends over everything cached (fp4_attn) and multiplies with the quantised
output weight.  At the end the last step is compared with the same layer computed by
torch in float32 from the dequantised weights and the cached rows that fp4_kv_read
returns.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp4_amax_amd as fq  # noqa: E402


class AttentionLayer:
    """Weights in NVFP4 with 64 x 64 outer scales; the cache's pages are the caller's to assign."""

    def __init__(self, w_qkv, w_o, q_heads, kv_heads, head_dim, num_pages, page_size=64):
        self.cfg = fq.make_cfg(format="nvfp4", two_level="outer_block", outer_block_size=64, outer_2d=True)
        self.w_qkv, self.w_o = fq.fp4_quantize(w_qkv, self.cfg), fq.fp4_quantize(w_o, self.cfg)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.cache = fq.KVCache.empty(num_pages, page_size, kv_heads, head_dim, fq.make_cfg(format="nvfp4"),
                                      device=w_qkv.device)

    def step(self, x, slots, page_table, kv_lens, q_starts=None, *, max_q=1, max_kv=None):
        """x [tokens, hidden] of the sequences' new tokens, slots [tokens] where their keys and
        values go; kv_lens counts them."""
        qkv = fq.fp4_linear(x, self.w_qkv, self.cfg).view(x.shape[0], -1, self.head_dim)
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        fq.fp4_kv_append(self.cache, k, v, slots)
        o = fq.fp4_attn(q, self.cache, page_table, kv_lens, q_starts, max_q=max_q, max_kv=max_kv)
        return fq.fp4_linear(o.view(x.shape[0], -1), self.w_o, self.cfg), q


def slots_of(page_table, page_size, first, count):
    """Slots of tokens first .. first + count - 1 of the sequence with this page table row."""
    t = torch.arange(first, first + count, device=page_table.device)
    return page_table.long()[t // page_size] * page_size + t % page_size


def plain_last(layer, q, page_table, lens):
    """The single-token step in float32 torch, from what the cache holds."""
    wo = fq.fp4_dequantize(layer.w_o["codes"], layer.w_o["scales"], layer.w_o["outer"],
                           layer.w_o["codes"].shape[0], layer.q_heads * layer.head_dim, layer.cfg, dtype=torch.float32)
    group, out = layer.q_heads // layer.kv_heads, []
    for b, n in enumerate(lens):
        k, v = fq.fp4_kv_read(layer.cache, slots_of(page_table[b], layer.cache.page_size, 0, n), dtype=torch.float32)
        k, v = (t.repeat_interleave(group, 1) for t in (k, v))
        w = torch.softmax((q[b].float() * k).sum(-1) * layer.head_dim ** -0.5, 0)
        out.append((w[..., None] * v).sum(0).flatten())
    return torch.stack(out) @ wo.t()


def main(tokens=8, hidden=2880, q_heads=64, kv_heads=8, head_dim=64, prompts=(300, 1, 77, 1024), seed=0):
    torch.manual_seed(seed)
    page = 64
    lens = list(prompts)
    cols = -(-(max(lens) + tokens) // page)
    table = torch.randperm(len(lens) * cols, device="cuda").int().view(len(lens), cols)
    layer = AttentionLayer((torch.randn((q_heads + 2 * kv_heads) * head_dim, hidden, device="cuda") * hidden ** -0.5).bfloat16(),
                           (torch.randn(hidden, q_heads * head_dim, device="cuda") * 0.02).bfloat16(),
                           q_heads, kv_heads, head_dim, len(lens) * cols, page)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    # the prompts, in one ragged call
    x = torch.randn(starts[-1], hidden, device="cuda").bfloat16()
    slots = torch.cat([slots_of(table[b], page, 0, n) for b, n in enumerate(lens)])
    y, _ = layer.step(x, slots, table, ints(lens), ints(starts), max_q=max(lens), max_kv=max(lens))
    x = y[torch.tensor([s - 1 for s in starts[1:]], device="cuda")]
    # then token after token
    for _ in range(tokens):
        x = torch.nn.functional.rms_norm(x.float(), (hidden,)).bfloat16()
        slots = torch.cat([slots_of(table[b], page, n, 1) for b, n in enumerate(lens)])
        lens = [n + 1 for n in lens]
        x, q = layer.step(x, slots, table, ints(lens), max_kv=max(lens))
    want = plain_last(layer, q, table, lens)
    err = ((x.float() - want).norm() / want.norm()).item()
    print("%d sequences, %d cached tokens: last step within %.2g of the float32 layer" % (len(lens), sum(lens), err))
    return err


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=8)
    main(p.parse_args().tokens)
