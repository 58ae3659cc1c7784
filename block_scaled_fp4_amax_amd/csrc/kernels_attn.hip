// kernels_attn.hip -- fp4_attn: how a call's keys are shared, and its launches (the kernels are
// attn_kernels.h's).
#include "attn_kernels.h"

namespace fp4q {

// Sequences of few rows.
static void plan_few(AttnPlan& p, const KvView& kv, int64_t batch, int64_t rows, int64_t keys)
{
    // Workgroups that the chip holds at once: 4 a compute unit (head_dim 64; 3 with two
    // tiles of rows), 2 (128) or 2 and 1 (256) by their LDS and registers.  Keys are not cut where
    // every sequence is short or the heads alone fill the chip twice.
    const bool one = rows <= 16;
    const int64_t slots = 256 * (kv.dim == 64 ? (one ? 4 : 3) : kv.dim == 128 || one ? 2 : 1);
    const int64_t heads = batch * kv.heads;
    p.groups = (int32_t)heads;
    if (keys <= kUnit * kMinShare || heads >= 2 * slots) return;
    if (heads * (keys / kUnit + 2) >= (int64_t)1 << 30) return;   // units are counted in 32 bits
    // no share makes more parts than these: a part is a share, or the last of its sequence
    const int64_t per_head = slots / kv.heads > 0 ? slots / kv.heads : 1;
    const int64_t parts = std::min(per_head + batch, batch * ((keys / kUnit + 2) / kMinShare + 1));
    p.slots = (int32_t)slots;
    p.groups = (int32_t)(parts * kv.heads);
    const size_t n = (size_t)p.groups * (one ? 16 : 32);
    p.few_ml = n * 2 * sizeof(float);
    p.few_o = n * kv.dim * sizeof(float);
}

AttnPlan plan_attn(const KvView& kv, int64_t batch, int64_t total_q, int64_t q_heads, int64_t max_q, int64_t max_kv,
                   int64_t table_cols, int64_t window)
{
    AttnPlan p{1, 1 << 30, 0, 0, 0, 0, 0, 0};
    const int64_t rows = max_q * (q_heads / kv.heads);
    if (rows == 0 || batch == 0) return p;
    const int64_t all = std::min(max_kv, table_cols * kv.page_size);
    // keys that the rows of few can see: their walk starts at the step of the first
    const int64_t keys = window ? std::min(all, window + max_q + kStep) : all;
    if (rows <= kFewRows || batch > 1) plan_few(p, kv, batch, std::min<int64_t>(rows, kFewRows), keys);
    if (rows <= kFewRows) return p;
    const TilePlan t = plan_tiles(batch, kv.heads, q_heads / kv.heads, max_q, all, window, kv.dim);
    // a launch of the join, four rows a workgroup of 256, has fewer than 2^32 lanes
    if (t.splits == 1 || (total_q * q_heads + 3) / 4 * 256 >= (int64_t)1 << 32) return p;
    p.splits = t.splits;
    p.chunk = t.chunk;
    const size_t n = (size_t)t.splits * total_q * q_heads;
    p.ml = n * 2 * sizeof(float);
    p.o = n * kv.dim * sizeof(float);
    return p;
}

// Trees of more rows than a wave's (k_attn_tiles with TREE).
static void plan_trees(AttnPlan& p, const KvView& kv, int64_t batch, int64_t rows, int64_t keys)
{
    const TreePlan t = plan_tree(batch, kv.heads, rows, keys, kv.dim);
    p.slots = t.slots;
    p.groups = t.parts * kv.heads;
    const size_t n = (size_t)p.groups * kTileRows;
    p.few_ml = n * 2 * sizeof(float);
    p.few_o = n * kv.dim * sizeof(float);
}

AttnPlan plan_attn_tree(const KvView& kv, int64_t batch, int64_t q_heads, int64_t max_q, int64_t max_kv,
                        int64_t table_cols, int64_t window)
{
    AttnPlan p{1, 1 << 30, 0, 0, 0, 0, 0, 0};
    const int64_t rows = max_q * (q_heads / kv.heads);
    if (rows == 0 || batch == 0) return p;
    const int64_t all = std::min(max_kv, table_cols * kv.page_size);
    const int64_t keys = window ? std::min(all, window + max_q + kv_round(kv.dim)) : all;
    if (rows <= kFewRows) plan_few(p, kv, batch, rows, keys);
    else plan_trees(p, kv, batch, rows, keys);
    return p;
}

hipError_t launch_attn(int bias, const AttnArgs& a, hipStream_t s)
{
    if (bias == 0) return launch_bias<0, false>(a, s);
    if (bias == 7) return launch_bias<7, false>(a, s);
    return launch_bias<15, false>(a, s);
}

}  // namespace fp4q
