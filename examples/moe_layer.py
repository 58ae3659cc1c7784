"""One mixture-of-experts decoder layer served in 4 bits: prompts, then trees of drafted
tokens, all of whose queries are answered at once.

    python examples/moe_layer.py [--steps N]

Each step takes the residual stream's norm (fp4_add_rms_norm), multiplies with the quantised QKV
weight (fp4_linear), turns queries and keys by their positions while it writes the new keys and values into the paged
cache (fp4_kv_append_rope), attends (fp4_attn for prompts, fp4_attn_tree for drafted trees),
multiplies with the output weight, adds and takes the norm again (fp4_add_rms_norm), and goes through the
experts that the router chooses (fp4_moe).  The last step's parts are compared, one by one, with torch
in float32 from what the part before returned.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp4_amax_amd as fq  # noqa: E402


class MoeLayer:
    """Projections in NVFP4 and experts in MXFP4; the cache's pages are the caller's to assign."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, experts, top_k, inter, num_pages, page_size, positions):
        rand = lambda n, k: (torch.randn(n, k, device="cuda") * k ** -0.5).bfloat16()  # noqa: E731
        self.cfg = fq.make_cfg(format="nvfp4", two_level="outer_block", outer_block_size=64, outer_2d=True)
        self.experts_cfg = fq.make_cfg(format="mxfp4")
        self.w_qkv = fq.fp4_quantize(rand((q_heads + 2 * kv_heads) * head_dim, hidden), self.cfg)
        self.w_o = fq.fp4_quantize(rand(hidden, q_heads * head_dim), self.cfg)
        self.w1 = fq.fp4_quantize(rand(experts * 2 * inter, hidden), self.experts_cfg)
        self.w2 = fq.fp4_quantize(rand(experts * hidden, inter), self.experts_cfg)
        self.b1, self.b2 = (0.1 * torch.randn(experts, n, device="cuda") for n in (2 * inter, hidden))
        self.router = torch.randn(experts, hidden, device="cuda") * hidden ** -0.5
        self.norms = [1 + 0.1 * torch.randn(hidden, device="cuda") for _ in range(2)]
        self.q_heads, self.kv_heads, self.head_dim, self.top_k, self.inter = q_heads, kv_heads, head_dim, top_k, inter
        self.cache = fq.KVCache.empty(num_pages, page_size, kv_heads, head_dim, fq.make_cfg(format="nvfp4"), device="cuda")
        angle = torch.arange(positions, device="cuda")[:, None] * 10000.0 ** (-torch.arange(head_dim // 2, device="cuda") * 2.0 / head_dim)
        self.cos, self.sin = angle.cos(), angle.sin()

    def experts(self, x, logits):
        return fq.fp4_moe(x, logits, self.w1, self.w2, self.experts_cfg, top_k=self.top_k, b1=self.b1, b2=self.b2, limit=7.0,
                          alpha=1.702, shift=1.0)

    def step(self, x, residual, positions, slots, page_table, kv_lens, q_starts, tree=None, **bounds):
        """x [tokens, hidden] is added to the residual stream (None: it starts with x); slots [tokens]
        is where the new keys and values go, and kv_lens counts them.  tree: which drafted tokens each one
        sees (None: those before it).  Returns every part's result by name; "y" and "residual" go to the next layer."""
        r = dict(zip(("residual0", "normed0"), self._norm(x, residual, 0)))
        r["qkv"] = fq.fp4_linear(r["normed0"], self.w_qkv, self.cfg).view(x.shape[0], -1, self.head_dim)
        q, k, v = r["qkv"].split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        r["q"] = fq.fp4_kv_append_rope(self.cache, k, v, slots, positions, self.cos, self.sin, q=q)
        if tree is None:
            r["attn"] = fq.fp4_attn(r["q"], self.cache, page_table, kv_lens, q_starts, **bounds)
        else:
            r["attn"] = fq.fp4_attn_tree(r["q"], self.cache, page_table, kv_lens, q_starts, tree, **bounds)
        r["projected"] = fq.fp4_linear(r["attn"].view(x.shape[0], -1), self.w_o, self.cfg)
        r["residual"], r["normed"] = self._norm(r["projected"], r["residual0"], 1)
        r["logits"] = r["normed"].float() @ self.router.t()
        # a call of the experts takes at most 1024 tokens
        r["y"] = torch.cat([self.experts(a, b) for a, b in zip(r["normed"].split(1024), r["logits"].split(1024))])
        return r

    def _norm(self, x, residual, which):
        n = fq.fp4_add_rms_norm(x, self.norms[which], residual, eps=1e-5)
        return n["residual"], n["y"]


def slots_of(page_table, page_size, first, count):
    """Slots of tokens first .. first + count - 1 of the sequence with this page table row."""
    t = torch.arange(first, first + count, device=page_table.device)
    return page_table.long()[t // page_size] * page_size + t % page_size


def draft(chain, branches):
    """A tree of `chain` tokens one after another, with a further child at each of `branches`: each node's depth
    and which nodes it sees."""
    parents = [i - 1 for i in range(chain)] + list(branches)
    sees, depth = torch.eye(len(parents), dtype=torch.bool), [0] * len(parents)
    for i, p in enumerate(parents):
        if p >= 0:
            sees[i] |= sees[p]
            depth[i] = depth[p] + 1
    return depth, sees


def turned(layer, x, positions):
    c, s = (t[positions.long()][:, None] for t in (layer.cos, layer.sin))
    a, b = x.float().chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def plain_parts(layer, r, x, residual, positions, slots, table, lens, nodes, sees):
    """The parts of a step in float32 from the parts before them, by name."""
    weight = lambda w, rows, cfg: fq.fp4_dequantize(w["codes"], w["scales"], w["outer"], rows, w["codes"].numel() * 2 // rows, cfg,  # noqa: E731
                                                    dtype=torch.float32)
    want = {"residual0": (x.float() + residual.float()).bfloat16()}
    norm = lambda h, w: h.float() * (h.float().square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w  # noqa: E731
    want["normed0"] = norm(r["residual0"], layer.norms[0])
    h, d, group = layer.q_heads, layer.head_dim, layer.q_heads // layer.kv_heads
    want["qkv"] = (r["normed0"].float() @ weight(layer.w_qkv, (h + 2 * layer.kv_heads) * d, layer.cfg).t()).view(len(slots), -1, d)
    q, k, v = r["qkv"].split([h, layer.kv_heads, layer.kv_heads], 1)
    want["q"] = turned(layer, q, positions).bfloat16()
    # the same rows turned by torch and written by the plain append
    other = fq.KVCache.empty(layer.cache.num_pages, layer.cache.page_size, layer.kv_heads, d, layer.cache.cfg, device="cuda")
    fq.fp4_kv_append(other, turned(layer, k, positions), v.float().contiguous(), slots)
    (r["k"], r["v"]), (want["k"], want["v"]) = (fq.fp4_kv_read(c, slots, dtype=torch.float32) for c in (layer.cache, other))
    out, at = [], 0
    for b, n in enumerate(lens):
        k, v = fq.fp4_kv_read(layer.cache, slots_of(table[b], layer.cache.page_size, 0, n), dtype=torch.float32)
        k, v = (t.repeat_interleave(group, 1).transpose(0, 1).contiguous() for t in (k, v))
        q = r["q"][at:at + nodes].float().transpose(0, 1).contiguous()
        score = torch.bmm(q, k.transpose(1, 2).contiguous()) * d ** -0.5
        score[:, :, n - nodes:].masked_fill_(~sees, float("-inf"))
        out.append(torch.bmm(torch.softmax(score, -1), v).transpose(0, 1))
        at += nodes
    want["attn"] = torch.cat(out)
    hidden = x.shape[1]
    want["projected"] = r["attn"].reshape(len(slots), -1).float() @ weight(layer.w_o, hidden, layer.cfg).t()
    want["residual"] = (r["projected"].float() + r["residual0"].float()).bfloat16()
    want["normed"] = norm(r["residual"], layer.norms[1])
    experts = layer.router.shape[0]
    w1 = weight(layer.w1, experts * 2 * layer.inter, layer.experts_cfg).view(experts, -1, hidden)
    w2 = weight(layer.w2, experts * hidden, layer.experts_cfg).view(experts, hidden, -1)
    y = torch.zeros_like(r["y"], dtype=torch.float32)
    top = torch.topk(r["logits"], layer.top_k)
    share = torch.softmax(top.values, -1)
    for t in range(len(slots)):
        for e, a in zip(top.indices[t].tolist(), share[t]):
            g, u = (w1[e] @ r["normed"][t].float() + layer.b1[e]).chunk(2)
            g, u = g.clamp(max=7.0), u.clamp(-7.0, 7.0)
            y[t] += a * (w2[e] @ (g * torch.sigmoid(1.702 * g) * (u + 1.0)) + layer.b2[e])
    want["y"] = y
    return want


def main(steps=4, hidden=2880, q_heads=64, kv_heads=8, head_dim=64, experts=32, top_k=4, inter=2880, prompts=(300, 1, 77, 1024),
         chain=5, branches=(0, 0, 2, 3), seed=0):
    torch.manual_seed(seed)
    page, lens, nodes = 64, list(prompts), chain + len(branches)
    depth, sees = draft(chain, branches)
    cols = -(-(max(lens) + steps * chain + nodes) // page)
    table = torch.randperm(len(lens) * cols, device="cuda").int().view(len(lens), cols)
    layer = MoeLayer(hidden, q_heads, kv_heads, head_dim, experts, top_k, inter, len(lens) * cols, page, cols * page)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    # the prompts, in one ragged call
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    x = torch.randn(starts[-1], hidden, device="cuda").bfloat16()
    slots = torch.cat([slots_of(table[b], page, 0, n) for b, n in enumerate(lens)])
    layer.step(x, None, torch.cat([ints(range(n)) for n in lens]), slots, table, ints(lens), ints(starts), max_q=max(lens), max_kv=max(lens))
    # then trees: the chain lies first, so what is accepted of it stays where it is
    tree = sees.repeat(len(lens), 1).cuda()
    starts = ints([nodes * b for b in range(len(lens) + 1)])
    for i in range(steps):
        x, residual = (torch.randn(nodes * len(lens), hidden, device="cuda").bfloat16() for _ in "xr")
        slots = torch.cat([slots_of(table[b], page, n, nodes) for b, n in enumerate(lens)])
        positions = ints([n + d for n in lens for d in depth])
        cached = [n + nodes for n in lens]
        r = layer.step(x, residual, positions, slots, table, ints(cached), starts, tree, max_q=nodes, max_kv=max(cached))
        lens = [n + 1 + (i + b) % chain for b, n in enumerate(lens)]
    want = plain_parts(layer, r, x, residual, positions, slots, table, cached, nodes, sees.cuda())
    err = {k: ((r[k].float() - want[k].float()).norm() / want[k].float().norm()).item() for k in want}
    print("%d trees of %d tokens, %d cached tokens: parts of the last step within %s of float32" % (
        len(lens), nodes, sum(cached), ", ".join("%s %.2g" % p for p in err.items())))
    return err


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=4)
    main(p.parse_args().steps)
