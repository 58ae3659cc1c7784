// attn_kernels.h -- attention over the paged 4-bit cache for gfx950: the kernels of fp4_attn
// (kernels_attn.hip) and, with TREE, of fp4_attn_tree (kernels_attn_tree.hip).
//
//   o_i = sum_j p_ij v_j / l_i,  p_ij = exp(scale q_i . k_j - m_i),  l_i = sum_j p_ij
//
// over the keys that query i sees, in one pass over the keys with the running
// maximum m_i and sum l_i.
//
// Rows.  The queries of one sequence that read the same KV head (its queries
// times the q_heads / kv_heads heads of the group) are the rows of a tile, so a
// cached row is decoded once for all of them.  A wave takes QT tiles of 16 rows.
//
// Layout.  A step takes 32 keys.  S^T = K Q^T (A = K: lane l holds key l % 16,
// the quarter l / 16 of its row, which is one aligned load; Q's lanes hold the same
// quarter of their row, and a sum does not care about its order).  Its result has a
// row of Q in each column l % 16 and keys 4 (l / 16) .. + 3 in the lane, so P^T is
// already laid out as the B operand of O^T = V^T P^T when V's lanes hold those
// same keys: no value of P moves between lanes or through LDS.  For V, lane l
// holds the codes of head_dim / 16 neighbouring values (l % 16) of its 8 keys; decoding
// gives pairs along head_dim, one permute turns two keys' pairs into pairs along the
// keys.
//
// Rounding.  K and V decode exactly (mfma16.h).  P is rounded to the 16-bit
// operand type (half a step: 2^-8 of a term in bf16, 2^-11 in FP16), and l sums the rounded P
// (a product with ones), so a row of equal values of V is returned exactly; S, m, l
// and O are binary32.  Where the result is asked for in binary32 (FINE), P is two such terms, the
// second what the first has left (off by 2^-16 in bf16, 2^-22 in FP16), and each takes its
// products: 48 sequences up to 8192 keys (MXFP4, head_dim 64) 33 -> 36.5 us, two prompts of 4096 tokens
// (128) 285 -> 345 us.  FP16 holds q scaled by a power of two per row: its bits are
// kept down to 2^-28 of the row's largest value.
//
// Running maximum.  m moves only when some row's score exceeds it by 8 (powers of
// two), so O is seldom rescaled.  P stays below 2^8 in bf16.  In FP16 m is held 7 below the
// largest score when it moves: P's largest lies within [2^7, 2^15], and what FP16 rounds to multiples
// of 2^-24 is 2^7 further below it, at no cost.
//
// Few rows: the four waves of a workgroup take every fourth step of the same rows and
// join through LDS, and the keys are split over workgroups, whose partial (O, m, l) a
// second kernel joins (launch_attn).
//
// Trees (TREE).  A sequence's queries are drafted tokens, whose keys are the last of it.  A row sees
// the keys before them, the context, as far as its window goes, and of the drafted keys those
// that its row of a.tree names.  Only steps that reach beyond the context look at the mask, so a
// tree costs what a chunk of as many tokens does.
#pragma once

#include <algorithm>
#include <type_traits>

#include "fp4q_device.h"
#include "kv_index.h"
#include "launch.h"
#include "lds_load.h"
#include "mfma16.h"

namespace fp4q {

namespace {

constexpr int kWaves = 4;
constexpr int kUnit = 128;                               // keys that a workgroup of few rows takes at once
constexpr int kMinShare = 4;                             // units of a workgroup's share, at least
constexpr int kFewRows = 32;
constexpr int kStep = 32;                                // keys of a step
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3.4028235e38f;                 // m of a row that has seen no key
constexpr float kLazy = 8.0f;
// powers of two between m and the score that moves it
template <int BIAS>
constexpr float kRoom = BIAS == 0 ? 0.0f : 7.0f;

// A group's rows through a buffer descriptor in scalar registers: a lane's offsets are the
// same for every group, so a load takes no address arithmetic on lanes.
__device__ __forceinline__ rsrc_t rows_at(const uint8_t* base, int64_t row, int bytes)
{
    const uint64_t p = (uint64_t)base + (uint64_t)row * bytes;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)p), hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
    return make_rsrc((const void*)((uint64_t)hi << 32 | lo));
}

// The largest of a value over the four lanes of a column (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float column_max(float v)
{
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

// The codes and scale bytes of one step in a lane's registers.
template <int D, int BIAS>
struct Raw {
    static constexpr int kKW = D / 32;                   // dwords of a quarter row of K
    static constexpr int kVW = D / 16 < 8 ? 1 : D / 128; // dwords of D / 16 codes of V
    static constexpr int kSB = D / Dec<BIAS>::kBlock;    // scale bytes of a row
    // V's scale bytes of a lane's four neighbouring keys: whole rows together where
    // they fill up to 16 bytes, byte by byte where rows are longer
    static constexpr int kSW = kSB <= 4 ? kSB : 4;
    uint32_t k[2][kKW], ks[2], v[8][kVW], vs[2][kSW];

    // V's scale byte of key 4 s + t of the lane; bit: 8 times its block
    __device__ __forceinline__ uint32_t v_scale(int s, int t, uint32_t bit) const
    {
        if constexpr (kSB == 2) return __builtin_amdgcn_ubfe(vs[s][t >> 1], 16 * (t & 1) + bit, 8);
        else if constexpr (kSB == 4) return __builtin_amdgcn_ubfe(vs[s][t], bit, 8);
        else return vs[s][t];
    }
};

// A wave's steps on their way: kDepth stages of LDS, filled by loads that write LDS
// directly (16 bytes a lane to consecutive places), kDepth - 1 steps ahead of
// their use.  (The MXFP4 forms wait for them all at a step's first product: the compiler's wait
// for the loads of q, which nothing converts before the loop.)  A stage costs 3, 5 or 9 load
// instructions and no registers, where loading a lane's own words took 24 instructions and kept one step in flight
// (4 x 131072 keys, NVFP4, head_dim 128: 87 us, with this ring 79, and 71 with
// non-temporal loads).  Two stages and twice the workgroups take as long as four.
//   K codes   [32 keys][D / 2], D = 256 with a row's eight 16-byte chunks at
//             chunk ^ (key % 8), so that the lanes of a read spread over the banks;
//   V codes   [2][16 keys][D / 2], key 4 q + t of a group of 16 at place 4 t + q,
//             so that one read of the wave is contiguous;
//   K scales, V scales  [32 keys][D / block].
template <int D, int BIAS>
struct Ring {
    static constexpr int B = Dec<BIAS>::kBlock;
    static constexpr int kDepth = D == 256 ? 2 : 4;
    static constexpr int kCodes = 32 * D / 2, kScales = 32 * D / B;
    static constexpr int kStage = 2 * (kCodes + kScales);
    static constexpr int kWave = kDepth * kStage;
    static constexpr int kLoads = D == 64 ? 3 : D == 128 ? 5 : 9;

    lds_t* mem;                                          // the wave's stages
    const uint8_t *k_codes, *v_codes;
    uint64_t scales;                                     // the lane's place in the scales of row 0
    int lane;

    __device__ __forceinline__ Ring(unsigned char* lds, const KvView& kv, int lane)
        : mem((lds_t*)lds), k_codes(kv.k_codes), v_codes(kv.v_codes), lane(lane)
    {
        const uint64_t ks = (uint64_t)kv.k_scales, vs = (uint64_t)kv.v_scales;
        scales = ks + (lane / (D / B) & 2 ? vs - ks : 0) + (lane % (D / B)) * 16;
    }

    __device__ __forceinline__ void issue(int slot, const KvGroup (&g)[2])
    {
        const uint32_t to = lds_address(mem + slot * kStage);
        if constexpr (D == 64) {
            // a group of 16 keys is 512 bytes: lanes 0 .. 31 and 32 .. 63 take one each
            const int64_t row = g[0].row + (lane < 32 ? 0 : g[1].row - g[0].row);
            const uint32_t c = lane & 31, place = c >> 1;
            lds_load(k_codes + row * 32 + c * 16, to);
            lds_load(v_codes + row * 32 + (4 * (place & 3) + (place >> 2)) * 32 + (c & 1) * 16, to + kCodes);
        } else {
            constexpr int kPer = D / 32;                 // 16-byte chunks of a row
            constexpr int kHalves = D / 128;             // loads of a group
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const rsrc_t kc = rows_at(k_codes, g[s].row, D / 2), vc = rows_at(v_codes, g[s].row, D / 2);
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    const uint32_t place = h * (64 / kPer) + lane / kPer, c = lane % kPer;
                    const uint32_t at = to + (s * kHalves + h) * 1024;
                    lds_load(kc, place * (D / 2) + (D == 256 ? c ^ (place & 7) : c) * 16, at);
                    lds_load(vc, (4 * (place & 3) + (place >> 2)) * (D / 2) + c * 16, at + kCodes);
                }
            }
        }
        // scales: D / B chunks of 16 bytes for each of K's and V's two groups
        if (lane < 4 * (D / B)) {
            const int64_t row = g[0].row + (lane / (D / B) & 1 ? g[1].row - g[0].row : 0);
            lds_load((const void*)(scales + (uint64_t)row * (D / B)), to + 2 * kCodes);
        }
    }

    __device__ __forceinline__ void read(int slot, Raw<D, BIAS>& r) const
    {
        constexpr int KB = D / 4 / B > 0 ? D / 4 / B : 1;    // scale bytes of a quarter row of K
        const uint32_t m = lane & 15, q = (uint32_t)lane >> 4;
        const lds_t* k = mem + slot * kStage;
        const lds_t *v = k + kCodes, *ks = v + kCodes, *vs = ks + kScales;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const lds_t* kr = k + (16 * s + m) * (D / 2);
            if constexpr (D == 256) {
#pragma unroll
                for (int j = 0; j < 2; ++j) words<4>(kr + ((2 * q + j) ^ (m & 7)) * 16, r.k[s] + 4 * j);
            } else {
                words<D / 32>(kr + q * (D / 8), r.k[s]);
            }
            r.ks[s] = bytes<KB>(ks + (16 * s + m) * (D / B) + q * (D / 4) / B);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const lds_t* p = v + (16 * s + 4 * t + q) * (D / 2) + m * (D / 32);
                if constexpr (D == 64) r.v[4 * s + t][0] = bytes<2>(p);
                else words<D / 128>(p, r.v[4 * s + t]);
                if constexpr (D / B > 4) r.vs[s][t] = bytes<1>(vs + (16 * s + 4 * q + t) * (D / B) + m * (D / 16) / B);
            }
            if constexpr (D / B <= 4) words<D / B>(vs + (16 * s + 4 * q) * (D / B), r.vs[s]);
        }
    }

private:
    template <int N>
    static __device__ __forceinline__ void words(const lds_t* p, uint32_t* w)
    {
        if constexpr (N == 1) {
            w[0] = *(const __attribute__((address_space(3))) uint32_t*)p;
        } else if constexpr (N == 2) {
            const u32x2_t u = *(const __attribute__((address_space(3))) u32x2_t*)p;
            w[0] = u[0], w[1] = u[1];
        } else {
            const u32x4_t u = *(const __attribute__((address_space(3))) u32x4_t*)p;
            w[0] = u[0], w[1] = u[1], w[2] = u[2], w[3] = u[3];
        }
    }

    template <int N>
    static __device__ __forceinline__ uint32_t bytes(const lds_t* p)
    {
        if constexpr (N == 1) return *p;
        else if constexpr (N == 2) return *(const __attribute__((address_space(3))) uint16_t*)p;
        else return *(const __attribute__((address_space(3))) uint32_t*)p;
    }
};

// Rounds a row's head_dim / 4 values of q held by a lane to FP16 after scaling the row to
// [2^14, 2^15) by a power of two; returns what scores are multiplied by to undo it.
template <int N>
__device__ __forceinline__ float q_to_f16(uint4 (&q)[N])
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
        top = max(top, bf16_absmax_bits(w));
    }
    auto a = __builtin_amdgcn_permlane16_swap(top, top, false, false);
    top = max(a[0], a[1]);
    a = __builtin_amdgcn_permlane32_swap(top, top, false, false);
    top = max(a[0], a[1]);
    const uint32_t e = min(max(top >> 7, 20u), 254u);
    const float f = __uint_as_float((268u - e) << 23);   // 2^(14 - (e - 127))
#pragma unroll
    for (int i = 0; i < N; ++i) {
        uint32_t* w = (uint32_t*)&q[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = Dec<7>::round2(bf16_lo(w[j]) * f, bf16_hi(w[j]) * f);
    }
    return __uint_as_float((e - 14u) << 23);
}

// Sequence b's queries: query b alone without q_starts.
__device__ __forceinline__ QueryRange queries_of(const AttnArgs& a, int b)
{
    if (!a.q_starts) return QueryRange{b, 1};
    return query_range(a.q_starts[b], a.q_starts[b + 1], a.total_q, a.max_q);
}

// Keys that the rows of query i see, at least one of them or all.  With TREE, first_range ends
// with the keys that all rows see (from last_range's start), and last_range with the last key.
template <bool TREE>
__device__ __forceinline__ KeyRange first_range(const AttnArgs& a, int i, int n, int kv)
{
    if constexpr (TREE) return tree_context(kv, n, a.window, 0);
    return key_range(i, n, kv, a.causal, a.window);
}

template <bool TREE>
__device__ __forceinline__ KeyRange last_range(const AttnArgs& a, int i, int n, int kv)
{
    if constexpr (TREE) return KeyRange{tree_context(kv, n, a.window, n).lo, kv};
    return key_range(i, n, kv, a.causal, a.window);
}

// One row's result: o = O f, with lane l holding d = (D / 4) (l / 16) + 0 .. D / 4 - 1.
template <int D>
__device__ __forceinline__ void store_row(void* out, bool f32, int64_t row, int quarter, const float (&o)[D / 4])
{
    const int64_t at = row * D + quarter * (D / 4);
    if (f32) {
        float* p = (float*)out + at;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            *(float4*)(p + 4 * i) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    } else {
        uint16_t* p = (uint16_t*)out + at;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = Dec<0>::round2(o[8 * i + 2 * j], o[8 * i + 2 * j + 1]);
            *(uint4*)(p + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// The factor of a row's O and its log-sum-exp (natural) from (m, l) and the head's sink.
__device__ __forceinline__ float finish_row(float m, float l, const float* sinks, int head, float& lse)
{
    float f = 1.0f, sink = 0.0f;
    bool led = false;                                    // by the sink
    if (sinks) {
        sink = sinks[head];
        float s = sink * kLog2e;
        // a finite sink stays finite (its type's lowest value, or one above all scores)
        if (__builtin_isinf(s) && !__builtin_isinf(sink)) s = __builtin_copysignf(3.4028235e38f, s);
        const float top = fmaxf(m, s);
        f = __builtin_amdgcn_exp2f(m - top);
        l = l * f + __builtin_amdgcn_exp2f(s - top);
        m = top;
        led = s == top;
    }
    if (l == 0.0f) {                                     // a row that sees nothing
        lse = -__builtin_inff();
        return 0.0f;
    }
    lse = led ? sink + __builtin_log2f(l) * kLn2 : (m + __builtin_log2f(l)) * kLn2;
    return f / l;
}

// A joined row: lane l holds values (D / 64) l + 0 .. D / 64 - 1.
template <int D>
__device__ __forceinline__ void write_joined(const AttnArgs& a, int64_t row, int qh, float m, float l,
                                             const float (&acc)[D / 64], float unshift, int lane)
{
    constexpr int N = D / 64;
    float lse;
    const float f = finish_row(m, l, a.sinks, qh, lse) * unshift * (a.kv.v_outer ? a.kv.v_outer[qh / a.group] : 1.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float y = l == 0.0f ? 0.0f : acc[i] * f;
        if (a.out_f32) ((float*)a.out)[row * D + lane * N + i] = y;
        else ((uint16_t*)a.out)[row * D + lane * N + i] = (uint16_t)f32_to_bf16(y);
    }
    if (a.lse && lane == 0) a.lse[row] = lse;
}

// A scale byte of V that some rows see and others do not, as one whose products are finite (0 times it is then 0):
// E4M3 has no codes above 0x7F, which FP16 would read as infinity or NaN.
template <int BIAS>
__device__ __forceinline__ uint32_t finite_scale(uint32_t byte)
{
    return BIAS == 7 ? byte & 0x7Fu : byte;
}

// MXFP4 keys some rows see and others do not, with a poisoned block of V: 0 times
// its NaN would reach the rows that do not see the key.  Such blocks are cleared,
// and the product of (block is poisoned) with (row sees the key) says which
// outputs become NaN.  All of a lane's values of V lie in one block.
__device__ __forceinline__ bool poisoned_blocks(uint32_t (&vs)[8], uint4& bad)
{
    bool any = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) any |= vs[j] == 0xFFu;
    if (!__any(any)) return false;
    constexpr uint32_t one = Dec<0>::kOnes & 0xFFFFu;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = (vs[2 * j] == 0xFFu ? one : 0u) | (vs[2 * j + 1] == 0xFFu ? one << 16 : 0u);
#pragma unroll
    for (int j = 0; j < 8; ++j) vs[j] = vs[j] == 0xFFu ? 0u : vs[j];
    bad = make_uint4(w[0], w[1], w[2], w[3]);
    return true;
}

template <int ND, int QT>
__device__ __forceinline__ void mark_poisoned(uint4 bad, const f32x4_t (&sc)[QT][2], f32x4_t (&o)[QT][ND])
{
    constexpr uint32_t one = Dec<0>::kOnes & 0xFFFFu;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        uint32_t seen[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = sc[t][j >> 1][2 * (j & 1)], b = sc[t][j >> 1][2 * (j & 1) + 1];
            seen[j] = (a != -__builtin_inff() ? one : 0u) | (b != -__builtin_inff() ? one << 16 : 0u);
        }
        const f32x4_t n = Dec<0>::mfma(bad, make_uint4(seen[0], seen[1], seen[2], seen[3]), f32x4_t{0, 0, 0, 0});
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int d = 0; d < ND; ++d) o[t][d][r] = n[r] > 0.0f ? __builtin_nanf("") : o[t][d][r];
    }
}

// The rows of a wave: their queries, what scores are multiplied by, the keys that each
// sees (first / last: the tile's first and last rows'), and where results go.
template <int D, int BIAS, int QT, bool TREE>
struct Rows {
    uint4 q[QT][D / 32];
    float c[QT];
    KeyRange see[QT], first, last;
    int64_t out[QT];                                     // token * q_heads + head, -1: no row
    const uint8_t* mask;                                 // TREE: the sequence's rows of the mask,
    uint32_t tree[TREE ? QT : 1];                        // and a row's place there from its first drafted key's
    int drafted;                                         // (at see[].hi, the context's end) for so many keys

    // Which of the lane's eight keys of the step at `at` row t sees, a bit each.  Without branches: with the mask's
    // loads in branches of their own the compiler (clang of ROCm 7.2) lost the assignment of masked
    // scores where a wave has two tiles of rows.
    __device__ __forceinline__ uint32_t seen(int t, int at, int quarter) const
    {
        uint32_t bits = 0, named[8] = {};
        if constexpr (TREE) {
            const rsrc_t m = make_rsrc(mask);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t j = (uint32_t)(at + 16 * (k >> 2) + 4 * quarter + (k & 3) - see[t].hi);
                named[k] = __builtin_amdgcn_raw_buffer_load_b8(m, j < (uint32_t)drafted ? tree[t] + j : kOff, 0, 0);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int key = at + 16 * (k >> 2) + 4 * quarter + (k & 3);
            const uint32_t in = (uint32_t)(key >= see[t].lo) & (uint32_t)(key < see[t].hi);
            bits |= (in | (uint32_t)(named[k] != 0)) << k;
        }
        return bits;
    }

    __device__ __forceinline__ void load(const AttnArgs& a, const QueryRange& qr, int kv, int head, int row0, int lane)
    {
        using X = Dec<BIAS>;
        const int col = lane & 15, quarter = lane >> 4;
        const int rows = qr.count * a.group;
        first = first_range<TREE>(a, min(row0, rows - 1) / a.group, qr.count, kv);
        last = last_range<TREE>(a, (min(row0 + 16 * QT, rows) - 1) / a.group, qr.count, kv);
        // drafted tokens ahead of a sequence that is shorter than its tree have no key
        const int skip = TREE ? max(qr.count - kv, 0) : 0;
        drafted = TREE ? max(min(qr.count, a.tree_cols) - skip, 0) : 0;
        mask = TREE && a.tree ? a.tree + (int64_t)qr.first * a.tree_cols : nullptr;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int r = row0 + 16 * t + col;
            const bool live = r < rows;
            const int i = live ? r / a.group : 0, g = live ? r - i * a.group : 0;
            if constexpr (TREE) {
                tree[t] = (uint32_t)(i * a.tree_cols + skip);
                int named = 0;
                if (a.window > 0) {                      // a quarter of the row a lane
                    const rsrc_t m = make_rsrc(mask);
                    for (int j = 0; j < drafted; j += 4) {
                        const int k = j + quarter;
                        named += __builtin_amdgcn_raw_buffer_load_b8(m, k < drafted ? tree[t] + k : kOff, 0, 0) != 0;
                    }
                    named += __shfl_xor(named, 16, 64);
                    named += __shfl_xor(named, 32, 64);
                }
                see[t] = tree_context(kv, qr.count, a.window, named);
            } else {
                see[t] = key_range(i, qr.count, kv, a.causal, a.window);
            }
            out[t] = live ? (int64_t)(qr.first + i) * a.q_heads + head * a.group + g : -1;
            const uint16_t* p =
                a.q + (int64_t)(qr.first + i) * a.ld_q + (int64_t)(head * a.group + g) * D + quarter * (D / 4);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) q[t][k] = live ? ((const uint4*)p)[k] : make_uint4(0, 0, 0, 0);
            c[t] = a.scale * kLog2e * X::kUnshift;
            if constexpr (!X::kBf16) {
                c[t] *= q_to_f16<D / 32>(q[t]);
                if (a.kv.k_outer) c[t] *= a.kv.k_outer[head];
            }
            c[t] = fmaxf(c[t], 1.17549435e-38f);         // 0 would turn a masked score into NaN
        }
    }
};

// What a wave has summed.
template <int D, int QT>
struct Sums {
    f32x4_t o[QT][D / 16], l[QT];
    float m[QT];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            m[t] = kNoMax;
            l[t] = f32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int n = 0; n < D / 16; ++n) o[t][n] = f32x4_t{0, 0, 0, 0};
        }
    }

    // o[n][r] is the value d = (D / 4) quarter + (D / 16) r + n of the lane's row
};

// One step: 32 keys from `at`, whose operands `src` gives; bits 0 and 1 of `groups` say which of
// its two groups of 16 are there.
template <int D, int BIAS, int QT, bool FINE, bool TREE, class Src>
__device__ __forceinline__ void attend_step(Src& src, uint32_t groups, int at, int end, const Rows<D, BIAS, QT, TREE>& rows,
                                            int lane, Sums<D, QT>& sum)
{
    using X = Dec<BIAS>;
    constexpr int NK = D / 32;                           // products of a step's scores
    constexpr int ND = D / 16;                           // products of a step's outputs (values of V in a lane)
    const int quarter = lane >> 4;
    const uint4 ones = make_uint4(X::kOnes, X::kOnes, X::kOnes, X::kOnes);
    // scores: S^T[key, row], keys 16 s + 4 quarter + r
    f32x4_t sc[QT][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        uint4 kf[NK];
#pragma unroll
        for (int i = 0; i < NK; ++i) kf[i] = src.k(s, i);
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            sc[t][s] = f32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < NK; ++i) sc[t][s] = X::mfma(kf[i], rows.q[t][i], sc[t][s]);
        }
    }

    // A step whose keys are not all seen by all rows: scores of unseen keys are
    // -infinity.  V of keys that are not there, or that come before every row's window (their
    // bytes may be anything), is cleared, so that 0 times it is 0.
    const bool whole = (groups & 3) == 3 && at >= rows.last.lo && at + kStep <= rows.first.hi && at + kStep <= end;
    if (!whole) {
        uint32_t seen[QT];
#pragma unroll
        for (int t = 0; t < QT; ++t) seen[t] = rows.seen(t, at, quarter);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int key = at + 16 * s + 4 * quarter + r;
                const bool there = (groups >> s & 1) && key >= rows.first.lo && key < end;
#pragma unroll
                for (int t = 0; t < QT; ++t)
                    sc[t][s][r] = there && (seen[t] >> (4 * s + r) & 1) ? sc[t][s][r] : -__builtin_inff();
                src.keep(4 * s + r, there);
            }
    }
    if constexpr (BIAS == 0) src.poison(groups, whole, sc, sum.o);

    // running maximum, P
    uint4 p[QT], rest[FINE ? QT : 1];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        float top = fmaxf(fmaxf(fmaxf(sc[t][0][0], sc[t][0][1]), fmaxf(sc[t][0][2], sc[t][0][3])),
                          fmaxf(fmaxf(sc[t][1][0], sc[t][1][1]), fmaxf(sc[t][1][2], sc[t][1][3])));
        top *= rows.c[t];
        if (__any(top > sum.m[t] + (kLazy + kRoom<BIAS>))) {
            const float mn = fmaxf(sum.m[t], column_max(top) - kRoom<BIAS>);
            const float f = __builtin_amdgcn_exp2f(sum.m[t] - mn);
            sum.m[t] = mn;
            sum.l[t] *= f;
#pragma unroll
            for (int n = 0; n < ND; ++n) sum.o[t][n] *= f;
        }
        float e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            e[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][k >> 2][k & 3], rows.c[t], -sum.m[t]));
        p[t] = make_uint4(X::round2(e[0], e[1]), X::round2(e[2], e[3]), X::round2(e[4], e[5]), X::round2(e[6], e[7]));
        sum.l[t] = X::mfma(ones, p[t], sum.l[t]);
        if constexpr (FINE) {
            rest[t] = make_uint4(X::rest2(e[0], e[1], p[t].x), X::rest2(e[2], e[3], p[t].y), X::rest2(e[4], e[5], p[t].z),
                                 X::rest2(e[6], e[7], p[t].w));
            sum.l[t] = X::mfma(ones, rest[t], sum.l[t]);
        }
    }

    // O^T += V^T P^T, two values of head_dim (one byte of codes) at a time
    src.decode_scales();
    auto two = [&](auto byte_c) {
        constexpr int y = decltype(byte_c)::value;
        uint4 lo, hi;
        src.template v<y>(lo, hi);
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            sum.o[t][2 * y] = X::mfma(lo, p[t], sum.o[t][2 * y]);
            sum.o[t][2 * y + 1] = X::mfma(hi, p[t], sum.o[t][2 * y + 1]);
            if constexpr (FINE) {
                sum.o[t][2 * y] = X::mfma(lo, rest[t], sum.o[t][2 * y]);
                sum.o[t][2 * y + 1] = X::mfma(hi, rest[t], sum.o[t][2 * y + 1]);
            }
        }
    };
    two(std::integral_constant<int, 0>{});
    two(std::integral_constant<int, 1>{});
    if constexpr (ND > 4) {
        two(std::integral_constant<int, 2>{});
        two(std::integral_constant<int, 3>{});
    }
    if constexpr (ND > 8) {
        two(std::integral_constant<int, 4>{});
        two(std::integral_constant<int, 5>{});
        two(std::integral_constant<int, 6>{});
        two(std::integral_constant<int, 7>{});
    }
}

// V's operands of two neighbouring values of head_dim (the low and high codes of byte B of each
// key's word w[j]) for the lane's eight keys, with the keys' decoded scales.
template <int BIAS, int B>
__device__ __forceinline__ void decode_v(const uint32_t (&w)[8], const uint32_t (&scale)[8], uint4& lo, uint4& hi)
{
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = Dec<BIAS>::template pair<B>(w[j], scale[j]);
    lo = make_uint4(__builtin_amdgcn_perm(u[1], u[0], 0x05040100u), __builtin_amdgcn_perm(u[3], u[2], 0x05040100u),
                    __builtin_amdgcn_perm(u[5], u[4], 0x05040100u), __builtin_amdgcn_perm(u[7], u[6], 0x05040100u));
    hi = make_uint4(__builtin_amdgcn_perm(u[1], u[0], 0x07060302u), __builtin_amdgcn_perm(u[3], u[2], 0x07060302u),
                    __builtin_amdgcn_perm(u[5], u[4], 0x07060302u), __builtin_amdgcn_perm(u[7], u[6], 0x07060302u));
}

// Operands decoded by the wave that uses them, from the step's bytes.
template <int D, int BIAS, int QT>
struct FromRaw {
    const Raw<D, BIAS>& raw;
    uint32_t vs[8];

    __device__ __forceinline__ FromRaw(const Raw<D, BIAS>& raw, int lane) : raw(raw)
    {
        const uint32_t bit = 8 * ((lane & 15) * (D / 16) / Dec<BIAS>::kBlock);
#pragma unroll
        for (int j = 0; j < 8; ++j) vs[j] = raw.v_scale(j >> 2, j & 3, bit);
    }

    __device__ __forceinline__ uint4 k(int s, int i) const
    {
        constexpr int per = Dec<BIAS>::kBlock / 8;       // words of a block
        const uint32_t byte = D / 4 <= Dec<BIAS>::kBlock ? raw.ks[s] : (raw.ks[s] >> (8 * (i / per))) & 0xFFu;
        return Dec<BIAS>::octet(raw.k[s][i], Dec<BIAS>::scale(byte));
    }

    __device__ __forceinline__ void keep(int j, bool there) { vs[j] = there ? finite_scale<BIAS>(vs[j]) : 0; }

    __device__ __forceinline__ void poison(uint32_t, bool whole, const f32x4_t (&sc)[QT][2], f32x4_t (&o)[QT][D / 16])
    {
        uint4 bad;                                       // where all rows see the keys, the products do it
        if (!whole && poisoned_blocks(vs, bad)) mark_poisoned<D / 16, QT>(bad, sc, o);
    }

    __device__ __forceinline__ void decode_scales()
    {
#pragma unroll
        for (int j = 0; j < 8; ++j) vs[j] = Dec<BIAS>::scale(vs[j]);
    }

    template <int Y>
    __device__ __forceinline__ void v(uint4& lo, uint4& hi) const
    {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = raw.v[j][Y >> 2];
        decode_v<BIAS, (Y & 3)>(w, vs, lo, hi);
    }
};

// Steps at, at + stride, ... before end, through the wave's ring.  The rows of the next
// 64 steps are looked up together, a step a lane: a scalar look-up in each step would
// be waited for with the step's LDS reads, which count on the same counter.
template <int D, int BIAS, int QT, bool FINE, bool TREE>
__device__ __forceinline__ void attend(const AttnArgs& a, unsigned char* lds, const int32_t* table, int head, int at,
                                       int end, int stride, const Rows<D, BIAS, QT, TREE>& rows, int lane, Sums<D, QT>& sum)
{
    using R = Ring<D, BIAS>;
    if (at >= end) return;
    R ring(lds, a.kv, lane);
    uint32_t groups = 0;                                 // two bits for each step under way, the next one's lowest
    int next = at, slot = 0, known = 64;                 // the step to issue, its stage, its lane of `row`
    int64_t row[2];                                      // of a step's groups, -1: absent
    auto issue = [&](int behind) {
        if (known == 64) {
            known = 0;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const KvGroup g = kv_group(table, next + lane * stride + kKvGroup * s, end, a.per_page, a.kv.num_pages,
                                           a.kv.heads, head);
                row[s] = g.ok ? g.row : -1;
            }
        }
        KvGroup g[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)row[s], known);
            const int32_t hi = __builtin_amdgcn_readlane((int32_t)(row[s] >> 32), known);
            g[s].ok = hi >= 0;
            g[s].row = hi >= 0 ? (int64_t)hi << 32 | lo : 0;
        }
        ++known;
        wait_reads();                                    // of the step before, whose stage is filled now
        ring.issue(slot, g);
        groups |= (uint32_t)(g[0].ok | g[1].ok << 1) << (2 * behind);
        slot = (slot + 1) % R::kDepth;
        next += stride;
    };
#pragma unroll
    for (int i = 0; i < R::kDepth - 1; ++i)
        if (next < end) issue(i);
    for (int now = 0; at < end; at += stride, now = (now + 1) % R::kDepth, groups >>= 2) {
        if (next < end) {
            issue(R::kDepth - 1);
            wait_loads<(R::kDepth - 1) * R::kLoads>();
        } else {
            wait_loads<0>();
        }
        Raw<D, BIAS> raw;
        ring.read(now, raw);
        FromRaw<D, BIAS, QT> src(raw, lane);
        attend_step<D, BIAS, QT, FINE, TREE>(src, groups, at, end, rows, lane, sum);
    }
}

// Joins the four waves' sums of the same rows into wave 0's, in a fixed order: 2 and 3
// into 0 and 1, then 1 into 0.
template <int D, int QT>
struct JoinLds {
    float w[2][QT * (D / 4 + 2)][64];
};

// LDS of a workgroup: the waves' rings, and after them in time the join.
template <int D, int BIAS, int QT>
constexpr int lds_bytes()
{
    constexpr int ring = kWaves * Ring<D, BIAS>::kWave, join = (int)sizeof(JoinLds<D, QT>);
    return ring > join ? ring : join;
}

template <int D, int QT>
__device__ __forceinline__ void join_waves(JoinLds<D, QT>& lds, int wave, int lane, Sums<D, QT>& sum)
{
    __syncthreads();                                     // every wave is done with its ring
#pragma unroll
    for (int half = 2; half >= 1; half >>= 1) {
        if (wave >= half && wave < 2 * half) {
            float(*w)[64] = lds.w[wave - half];
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                w[t * (D / 4 + 2)][lane] = sum.m[t];
                w[t * (D / 4 + 2) + 1][lane] = sum.l[t][0];
#pragma unroll
                for (int n = 0; n < D / 16; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r) w[t * (D / 4 + 2) + 2 + 4 * n + r][lane] = sum.o[t][n][r];
            }
        }
        __syncthreads();
        if (wave < half) {
            float(*w)[64] = lds.w[wave];
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                const float mo = w[t * (D / 4 + 2)][lane], mn = fmaxf(sum.m[t], mo);
                const float f = __builtin_amdgcn_exp2f(sum.m[t] - mn), g = __builtin_amdgcn_exp2f(mo - mn);
                sum.m[t] = mn;
                sum.l[t][0] = sum.l[t][0] * f + w[t * (D / 4 + 2) + 1][lane] * g;
#pragma unroll
                for (int n = 0; n < D / 16; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        sum.o[t][n][r] = sum.o[t][n][r] * f + w[t * (D / 4 + 2) + 2 + 4 * n + r][lane] * g;
            }
        }
        __syncthreads();
    }
}

// Final results of a wave's rows.
template <int D, int BIAS, int QT, bool F32, bool TREE>
__device__ __forceinline__ void write_rows(const AttnArgs& a, const Rows<D, BIAS, QT, TREE>& rows, const Sums<D, QT>& sum,
                                           int head, int lane)
{
    const float unshift = Dec<BIAS>::kUnshift * (a.kv.v_outer ? a.kv.v_outer[head] : 1.0f);
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int64_t row = rows.out[t];
        if (row < 0) continue;
        float lse, y[D / 4];
        const float l = sum.l[t][0];
        const float f = finish_row(sum.m[t], l, a.sinks, (int)(row % a.q_heads), lse) * unshift;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int n = 0; n < D / 16; ++n) y[D / 16 * r + n] = l == 0.0f ? 0.0f : sum.o[t][n][r] * f;
        store_row<D>(a.out, F32, row, lane >> 4, y);
        if (a.lse && lane < 16) a.lse[row] = lse;
    }
}

// Partial results of a wave's rows: row t * 16 + column (or its place in the output) from
// `first` of the scratch.
template <int D, int BIAS, int QT, bool TREE>
__device__ __forceinline__ void write_parts(const AttnArgs& a, const Rows<D, BIAS, QT, TREE>& rows, const Sums<D, QT>& sum,
                                            int64_t first, bool by_output, int lane)
{
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        if (rows.out[t] < 0) continue;
        const int64_t row = first + (by_output ? rows.out[t] : 16 * t + (lane & 15));
        const float l = sum.l[t][0];
        if (lane < 16) *(float2*)(a.part_ml + row * 2) = make_float2(sum.m[t], l);
        if (l == 0.0f) continue;
        float y[D / 4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int n = 0; n < D / 16; ++n) y[D / 16 * r + n] = sum.o[t][n][r];
        store_row<D>(a.part_o, true, row, lane >> 4, y);
    }
}

// ---------------------------------------------------------------- few rows
// All rows of a sequence and KV head fit one wave, and the four waves of a workgroup take
// every fourth step of them.  A unit is 128 keys of one sequence and head; the keys of each are
// cut into parts of at most `share` units, one a workgroup, with the share chosen on the device
// (the lengths are there) so that the parts of all sequences fill the chip about once.  k_attn_few_join
// joins the parts.  48 sequences up to 8192 keys (MXFP4, head_dim 64): 32.4 us, against 35 to 38 with
// fixed parts of the longest sequence's keys and 44 with parts that run on from one
// head's keys to the next's (a second beginning and end costs more than it evens out).
// Bound: head_dim 128 memory, 71 us for 406 MB (5.7 TB/s; a plain non-temporal read of as much takes
// 70); head_dim 64 half arithmetic (about 150 vector instructions a step), half the
// look-up and first loads, about 6 us of the 32.
struct Seq {
    int first_q, queries, kv;
    int lo, hi;                                          // keys of all rows, from the step of the first
    int units;                                           // of one head, 0: none here
};

template <bool TREE>
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b)
{
    const QueryRange qr = queries_of(a, b);
    Seq s;
    s.first_q = qr.first;
    s.queries = qr.count;
    s.kv = kv_length(a.kv_lens[b], a.max_kv, a.table_cols, a.kv.page_size, a.kv.num_pages);
    s.lo = first_range<TREE>(a, 0, qr.count, s.kv).lo / kStep * kStep;
    s.hi = max(last_range<TREE>(a, qr.count - 1, qr.count, s.kv).hi, s.lo);
    // sequences of more rows are k_attn_tiles'
    s.units = qr.count == 0 || qr.count * a.group > kFewRows ? 0 : max(1, (s.hi - s.lo + kUnit - 1) / kUnit);
    return s;
}

__device__ __forceinline__ Seq seq_of_lane(const Seq& s, int lane)
{
    const auto r = [lane](int v) { return __builtin_amdgcn_readlane(v, lane); };
    return Seq{r(s.first_q), r(s.queries), r(s.kv), r(s.lo), r(s.hi), r(s.units)};
}

// Sequence b0 + lane, or none.
template <bool TREE>
__device__ __forceinline__ Seq seq_of_chunk(const AttnArgs& a, int b0, int lane)
{
    return b0 + lane < a.batch ? seq_of<TREE>(a, b0 + lane) : Seq{0, 0, 0, 0, 0, 0};
}

// Inclusive sums over the lanes of a wave.
__device__ __forceinline__ int lane_sums(int v)
{
    const auto add = [&v](int moved) { v += moved; };
    add(__builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));   // from 1, 2, 4, 8 lanes below in rows of 16
    add(__builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));
    add(__builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));
    add(__builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));
    add(__builtin_amdgcn_update_dpp(0, v, kDppBcast15, 0xA, 0xF, false));
    add(__builtin_amdgcn_update_dpp(0, v, kDppBcast31, 0xC, 0xF, false));
    return v;
}

// Units of a part: with `slots` workgroups at once and half a part lost a sequence.
__device__ __forceinline__ int share_of(int total, const AttnArgs& a)
{
    const int per_head = max(1, a.slots / a.kv.heads);
    const int parts = max(per_head - a.batch / 2, (per_head + 3) / 4);
    return max((total + parts - 1) / parts, kMinShare);
}

template <int D, int BIAS, int QT, bool FINE, bool TREE>
__global__ __launch_bounds__(64 * kWaves, QT == 1 && D == 64 ? 4 : D == 256 && QT == 2 ? 1 : 2) void k_attn_few(AttnArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int head = (int)blockIdx.x % a.kv.heads, place = (int)blockIdx.x / a.kv.heads;
    int seq = place, part = 0, parts = 1;
    Seq q;
    if (a.slots == 0) {                                  // one workgroup a sequence and head
        q = seq_of<TREE>(a, seq);
        if (q.units == 0) return;
    } else {
        // lane l holds sequence b0 + l of 64 at a time
        Seq mine = seq_of_chunk<TREE>(a, 0, lane);
        int total = __builtin_amdgcn_readlane(lane_sums(mine.units), 63);
        for (int b = 64; b < a.batch; b += 64)
            total += __builtin_amdgcn_readlane(lane_sums(seq_of_chunk<TREE>(a, b, lane).units), 63);
        const int share = share_of(total, a);
        int b0 = 0, before = 0;                          // parts of a head before chunk b0
        while (true) {
            const int n = parts_of(mine.units, share), upto = lane_sums(n);
            const uint64_t past = __ballot(before + upto > place);
            if (past) {
                const int j = __ffsll((unsigned long long)past) - 1;
                seq = b0 + j;
                parts = __builtin_amdgcn_readlane(n, j);
                part = place - before - (__builtin_amdgcn_readlane(upto, j) - parts);
                q = seq_of_lane(mine, j);
                break;
            }
            before += __builtin_amdgcn_readlane(upto, 63);
            b0 += 64;
            if (b0 >= a.batch) return;                   // more workgroups than parts
            mine = seq_of_chunk<TREE>(a, b0, lane);
        }
    }
    const int from = (int)((int64_t)q.units * part / parts), to = (int)((int64_t)q.units * (part + 1) / parts);
    Rows<D, BIAS, QT, TREE> rows;
    Sums<D, QT> sum;
    rows.load(a, QueryRange{q.first_q, q.queries}, q.kv, head, 0, lane);
    sum.clear();
    attend<D, BIAS, QT, FINE, TREE>(a, smem + wave * Ring<D, BIAS>::kWave, a.table + (int64_t)seq * a.table_cols, head,
                        q.lo + from * kUnit + wave * kStep, min(q.hi, q.lo + to * kUnit), kUnit, rows, lane, sum);
    join_waves<D, QT>(*reinterpret_cast<JoinLds<D, QT>*>(smem), wave, lane, sum);
    if (wave != 0) return;
    if (parts == 1) write_rows<D, BIAS, QT, FINE, TREE>(a, rows, sum, head, lane);
    else write_parts<D, BIAS, QT, TREE>(a, rows, sum, (int64_t)blockIdx.x * (16 * QT), false, lane);
}

// Joins the parts of one row (of a sequence and head) from their places in the scratch.
template <int D, class PartRow>
__device__ __forceinline__ void join_parts(const AttnArgs& a, int parts, PartRow part_row, const QueryRange& qr, int row,
                                           int head, float unshift, int lane)
{
    constexpr int N = D / 64;
    float acc[N] = {}, l = 0.0f, top = kNoMax;
    for (int p0 = 0; p0 < parts; p0 += 64) {
        const float2 ml = p0 + lane < parts ? *(const float2*)(a.part_ml + part_row(p0 + lane) * 2) : make_float2(0.0f, 0.0f);
        const float mn = fmaxf(top, group_max<64>(ml.y != 0.0f ? ml.x : kNoMax));
        const float f = __builtin_amdgcn_exp2f(top - mn), w = ml.y != 0.0f ? __builtin_amdgcn_exp2f(ml.x - mn) : 0.0f;
        top = mn;
        float part_l = ml.y * w;
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) part_l += __shfl_xor(part_l, i, 64);
        l = l * f + part_l;
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] *= f;
        const uint64_t used = __ballot(ml.y != 0.0f);    // parts without a key were not written
        const int here = min(64, parts - p0);
        for (int j0 = 0; j0 < here; j0 += 8) {
            float v[8][N];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool on = (used >> (j0 + j)) & 1;
                const float* p = a.part_o + part_row(p0 + j0 + j) * D + lane * N;
#pragma unroll
                for (int i = 0; i < N; ++i) v[j][i] = on ? p[i] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float g = __shfl(w, j0 + j, 64);
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] = __builtin_fmaf(v[j][i], g, acc[i]);
            }
        }
    }
    const int i = row / a.group, qh = head * a.group + row - i * a.group;
    write_joined<D>(a, (int64_t)(qr.first + i) * a.q_heads + qh, qh, top, l, acc, unshift, lane);
}

// Joins the parts of one row a wave.
template <int D, int QT, bool TREE>
__global__ __launch_bounds__(256) void k_attn_few_join(AttnArgs a, float unshift)
{
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int row = (int)blockIdx.x * 4 + wave;          // of a sequence and head
    const int head = (int)blockIdx.y, seq = (int)blockIdx.z;
    const QueryRange qr = queries_of(a, seq);
    if (row >= qr.count * a.group) return;
    int total = 0;
    Seq mine = seq_of_chunk<TREE>(a, 0, lane);
    total = __builtin_amdgcn_readlane(lane_sums(mine.units), 63);
    for (int b = 64; b < a.batch; b += 64)
        total += __builtin_amdgcn_readlane(lane_sums(seq_of_chunk<TREE>(a, b, lane).units), 63);
    const int share = share_of(total, a);
    int first = 0;                                       // parts of a head before this sequence's
    for (int b0 = 0; b0 + 64 <= seq; b0 += 64) {
        first += __builtin_amdgcn_readlane(lane_sums(parts_of(mine.units, share)), 63);
        mine = seq_of_chunk<TREE>(a, b0 + 64, lane);
    }
    const int n = parts_of(mine.units, share), upto = lane_sums(n);
    const int parts = __builtin_amdgcn_readlane(n, seq & 63);
    first += __builtin_amdgcn_readlane(upto, seq & 63) - parts;
    if (parts <= 1) return;
    const auto part_row = [&](int p) { return ((int64_t)(first + p) * a.kv.heads + head) * (16 * QT) + row; };
    join_parts<D>(a, parts, part_row, qr, row, head, unshift, lane);
}

// ---------------------------------------------------------------- many rows
// Eight waves take rows of their own and the same keys, 64 (head_dim 64: 128) at a time.  Each wave
// decodes a part of those keys' K and V once for all into LDS, as whole operands (64 lanes of 16
// bytes, written and read without bank conflicts), for the next keys while this one's are
// used; its bytes are loaded another round ahead.  Few workgroups split the keys `splits` ways.
// Two prompts of 4096 tokens (MXFP4, 32 / 8 heads of 128): 248 us a call among others, 266 to 280 under
// the profiler, about 0.7 PFLOP/s (305 with each wave decoding for itself).  Bound: of 507 thousand
// active cycles the vector unit takes 260 (softmax, decoding), LDS 225 (each operand that is read feeds one
// product) and the matrix unit 185, and they overlap little; 32 rows a wave
// (fewer vector instructions, half the waves), operands read ahead into
// registers and raised priority around the products all measured 270 to 300.
template <int D>
struct Tiles {
    static constexpr int kWaves = 8;
    static constexpr int kQT = 1;
    static constexpr int kKeys = kv_round(D);            // of a round
    static constexpr int kSteps = kKeys / kStep;
    static_assert(kWaves * 16 * kQT == kTileRows, "a workgroup's rows");
    static constexpr int kFrags = D / 16;                // operands of K, and of V, a step
    static constexpr int kStepBytes = (2 * kFrags + 1) * 1024;   // and which blocks of V are poisoned (MXFP4)
    static constexpr int kRound = kSteps * kStepBytes;
    static constexpr int kLds = 2 * kRound + 2 * kSteps * 16;
};

// Operands from a step's place in LDS.
template <int D, int BIAS, int QT>
struct FromLds {
    static constexpr int NF = D / 16;
    const lds_t* mem;                                    // the step's operands, at the lane's 16 bytes

    __device__ __forceinline__ uint4 frag(int n) const
    {
        const u32x4_t u = *(const __attribute__((address_space(3))) u32x4_t*)(mem + n * 1024);
        return make_uint4(u[0], u[1], u[2], u[3]);
    }

    __device__ __forceinline__ uint4 k(int s, int i) const { return frag(s * (D / 32) + i); }
    __device__ __forceinline__ void decode_scales() {}
    __device__ __forceinline__ void keep(int, bool) {}

    __device__ __forceinline__ void poison(uint32_t groups, bool, const f32x4_t (&sc)[QT][2], f32x4_t (&o)[QT][NF])
    {
        if (groups & 4) mark_poisoned<NF, QT>(frag(2 * NF), sc, o);
    }

    template <int Y>
    __device__ __forceinline__ void v(uint4& lo, uint4& hi) const
    {
        lo = frag(NF + 2 * Y);
        hi = frag(NF + 2 * Y + 1);
    }
};

// A wave's part of a round's decoding: K or V of one step (head_dim 256: half of it).
template <int D, int BIAS>
struct DecodePart {
    using T = Tiles<D>;
    static constexpr int B = Dec<BIAS>::kBlock;
    static constexpr int kHalves = 8 / (2 * T::kSteps);
    int step, half, lane;
    bool is_v;
    const uint8_t *codes, *scales;

    __device__ __forceinline__ DecodePart(const KvView& kv, int wave, int lane) : lane(lane)
    {
        step = wave % T::kSteps;
        is_v = wave / T::kSteps % 2;
        half = wave / (2 * T::kSteps);
        codes = is_v ? kv.v_codes : kv.k_codes;
        scales = is_v ? kv.v_scales : kv.k_scales;
    }

    struct Bytes {
        uint32_t w[8], s[8];
    };

    // row[2]: the rows of the step's groups, -1 where absent (then the cache's first rows)
    __device__ __forceinline__ void load(const int64_t (&row)[2], Bytes& b) const
    {
        const uint32_t m = lane & 15, q = (uint32_t)lane >> 4;
        if (!is_v) {
            constexpr int W = D / 32, KB = D / 4 / B > 0 ? D / 4 / B : 1;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (kHalves == 2 && s != half) continue; // uniform
                const int64_t r = row[s] < 0 ? 0 : row[s];
                const rsrc_t c = rows_at(codes, r, D / 2), f = rows_at(scales, r, D / B);
                uint32_t* w = b.w + (kHalves == 2 ? 0 : s * W);
                const uint32_t at = m * (D / 2) + q * (D / 8);
                if constexpr (W == 2) {
                    const u32x2_t u = __builtin_amdgcn_raw_buffer_load_b64(c, at, 0, 0);
                    w[0] = u[0], w[1] = u[1];
                } else {
#pragma unroll
                    for (int i = 0; i < W / 4; ++i) {
                        const uint4 u = buf_load16<0>(c, at + 16 * i);
                        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
                    }
                }
                const uint32_t fa = m * (D / B) + q * (D / 4) / B;
                uint32_t& o = b.s[kHalves == 2 ? 0 : s];
                if constexpr (KB == 1) o = __builtin_amdgcn_raw_buffer_load_b8(f, fa, 0, 0);
                else if constexpr (KB == 2) o = __builtin_amdgcn_raw_buffer_load_b16(f, fa, 0, 0);
                else o = __builtin_amdgcn_raw_buffer_load_b32(f, fa, 0, 0);
            }
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int64_t r = row[s] < 0 ? 0 : row[s];
                const rsrc_t c = rows_at(codes, r, D / 2), f = rows_at(scales, r, D / B);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t at = (4 * q + t) * (D / 2) + m * (D / 32);
                    if constexpr (D == 64) b.w[4 * s + t] = __builtin_amdgcn_raw_buffer_load_b16(c, at, 0, 0);
                    else b.w[4 * s + t] = __builtin_amdgcn_raw_buffer_load_b32(c, at + (D == 256 ? 4 * half : 0), 0, 0);
                    b.s[4 * s + t] = __builtin_amdgcn_raw_buffer_load_b8(f, (4 * q + t) * (D / B) + m * (D / 16) / B, 0, 0);
                }
            }
        }
    }

    // Writes the operands of the step at `at` to the round's LDS, and the step's flags: which groups are there,
    // and (bit 2) whether V has a poisoned block.  seen: the keys that some row of the workgroup sees; V of others
    // is cleared (attend_step).
    __device__ __forceinline__ void decode(const int64_t (&row)[2], int at, const KeyRange& seen, Bytes& b, lds_t* round,
                                           lds_t* flags) const
    {
        using X = Dec<BIAS>;
        lds_t* to = round + step * T::kStepBytes + lane * 16;
        const auto put = [&](int n, uint4 v) {
            *(__attribute__((address_space(3))) u32x4_t*)(to + n * 1024) = u32x4_t{v.x, v.y, v.z, v.w};
        };
        if (!is_v) {
            constexpr int W = D / 32, per = B / 8;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (kHalves == 2 && s != half) continue;
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const uint32_t sb = b.s[kHalves == 2 ? 0 : s];
                    const uint32_t byte = D / 4 <= B ? sb : (sb >> (8 * (i / per))) & 0xFFu;
                    put(s * W + i, X::octet(b.w[(kHalves == 2 ? 0 : s * W) + i], X::scale(byte)));
                }
            }
            return;
        }
        const uint32_t there = (row[0] >= 0 ? 1u : 0u) | (row[1] >= 0 ? 2u : 0u);
#pragma unroll
        for (int j = 0; j < 8; ++j) b.s[j] = finite_scale<BIAS>(b.s[j]);
        if (there != 3 || at < seen.lo || at + kStep > seen.hi) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int key = at + 16 * (j >> 2) + 4 * (lane >> 4) + (j & 3);
                if (!(there >> (j >> 2) & 1) || key < seen.lo || key >= seen.hi) b.s[j] = 0;
            }
        }
        uint32_t flag = there;
        if constexpr (BIAS == 0) {
            uint4 bad;
            if (poisoned_blocks(b.s, bad)) {
                flag |= 4;
                if (half == 0) put(2 * T::kFrags, bad);
            }
        }
        if (lane == 0 && half == 0) *(__attribute__((address_space(3))) uint32_t*)(flags + step * 16) = flag;
        uint32_t sc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sc[j] = X::scale(b.s[j]);
        // head_dim 128: a half's two bytes of the lane's word; 256: the lane's word of the half
        constexpr int kBytes = D / 32 / kHalves;
        if constexpr (D == 128 && kHalves == 2) {
#pragma unroll
            for (int j = 0; j < 8; ++j) b.w[j] >>= 16 * half;
        }
        const int n0 = T::kFrags + 2 * kBytes * half;
        uint4 lo, hi;
        decode_v<BIAS, 0>(b.w, sc, lo, hi);
        put(n0, lo), put(n0 + 1, hi);
        decode_v<BIAS, 1>(b.w, sc, lo, hi);
        put(n0 + 2, lo), put(n0 + 3, hi);
        if constexpr (kBytes == 4) {
            decode_v<BIAS, 2>(b.w, sc, lo, hi);
            put(n0 + 4, lo), put(n0 + 5, hi);
            decode_v<BIAS, 3>(b.w, sc, lo, hi);
            put(n0 + 6, lo), put(n0 + 7, hi);
        }
    }
};

// Trees: the rows of a sequence and head are its tiles, whose keys are cut, as those of few rows are, into
// parts of at most `share` rounds, chosen on the device so that all sequences' parts fill the
// chip about once; k_attn_tree_join joins them.  A part costs a first trip to memory and its share of the join, and
// whole sequences leave compute units idle behind the longest: 16 trees of up to 64 nodes after up to 8192
// keys (MXFP4, 64 / 8 heads of 64) 157 us a call uncut and 141 cut, 4 of 26 after up to 131072 (NVFP4, 32 / 8 of 128) 603
// with parts for one workgroup a compute unit and 271.  Bound as above, 0.45 PFLOP/s.
struct TreeSeq {
    int units, tiles;                                    // rounds of its keys, tiles of its rows
};

template <int D>
__device__ __forceinline__ TreeSeq tree_seq(const AttnArgs& a, int b)
{
    if (b >= a.batch) return TreeSeq{0, 0};
    const QueryRange qr = queries_of(a, b);
    const int kv = kv_length(a.kv_lens[b], a.max_kv, a.table_cols, a.kv.page_size, a.kv.num_pages);
    return TreeSeq{tree_rounds(kv, qr.count, a.window, kv_round(D)), tile_count(qr.count * a.group)};
}

// tree_share of all sequences (first: of the first 64).
template <int D>
__device__ __forceinline__ int share_of_trees(const AttnArgs& a, const TreeSeq& first, int lane)
{
    int rounds = __builtin_amdgcn_readlane(lane_sums(first.units * first.tiles), 63);
    int tiles = __builtin_amdgcn_readlane(lane_sums(first.tiles), 63);
    for (int b = 64; b < a.batch; b += 64) {
        const TreeSeq s = tree_seq<D>(a, b + lane);
        rounds += __builtin_amdgcn_readlane(lane_sums(s.units * s.tiles), 63);
        tiles += __builtin_amdgcn_readlane(lane_sums(s.tiles), 63);
    }
    return tree_share(rounds, tiles, a.slots, a.kv.heads);
}

struct TreePlace {
    int seq, tile, part, parts;                          // parts == 0: nothing here
    int first;                                           // place of the sequence's first part
    int tiles;
};

// Workgroup `place` of a head: the parts of sequence after sequence, tiles side by side in each.
// (Calls whose keys are not cut return here too: a branch around this in the kernel reloaded two more spilled registers a
// round at head_dim 128, and 4 trees of 26 after up to 131072 keys took 302 us for 271.)
template <int D>
__device__ __forceinline__ TreePlace tree_place(const AttnArgs& a, int place, int lane)
{
    if (a.slots == 0) return TreePlace{(int)blockIdx.z, (int)blockIdx.y, 0, 1, 0, 0};   // one workgroup a tile (tree_grid)
    TreeSeq mine = tree_seq<D>(a, lane);
    const int share = share_of_trees<D>(a, mine, lane);
    int before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        if (b0) mine = tree_seq<D>(a, b0 + lane);
        const int each = mine.tiles ? parts_of(mine.units, share) : 0, n = each * mine.tiles, upto = lane_sums(n);
        const uint64_t past = __ballot(before + upto > place);
        if (past) {
            const int j = __ffsll((unsigned long long)past) - 1;
            const int tiles = __builtin_amdgcn_readlane(mine.tiles, j), parts = __builtin_amdgcn_readlane(each, j);
            const int first = before + __builtin_amdgcn_readlane(upto, j) - tiles * parts, at = place - first;
            return TreePlace{b0 + j, at % tiles, at / tiles, parts, first, tiles};
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return TreePlace{0, 0, 0, 0, 0, 0};                  // more workgroups than parts
}

// Joins the parts of a row in sixteen lanes, D / 16 values each.  Three trips to memory one after another, so waves
// that take four rows each are done sooner than four times as many: 16 trees of up to 64 nodes (64 heads of 64, 33 MB of
// parts) 6 us, a row a wave 15.
template <int D>
__global__ __launch_bounds__(256) void k_attn_tree_join(AttnArgs a, float unshift)
{
    constexpr int N = D / 64, kAhead = 4;                // fours of a lane; parts that it loads together
    const int lane = (int)threadIdx.x & 63, in_row = lane & 15;
    const int row = (int)blockIdx.x * 16 + ((int)threadIdx.x >> 4);   // of a sequence and head
    const int head = (int)blockIdx.y, seq = (int)blockIdx.z;
    const QueryRange qr = queries_of(a, seq);
    const int rows = qr.count * a.group;
    if ((int)blockIdx.x * 16 >= rows) return;
    TreeSeq mine = tree_seq<D>(a, lane);
    const int share = share_of_trees<D>(a, mine, lane);
    int first = 0;                                       // parts of a head before this sequence's
    for (int b0 = 0; b0 + 64 <= seq; b0 += 64) {
        first += __builtin_amdgcn_readlane(lane_sums(mine.tiles ? parts_of(mine.units, share) * mine.tiles : 0), 63);
        mine = tree_seq<D>(a, b0 + 64 + lane);
    }
    const int each = mine.tiles ? parts_of(mine.units, share) : 0, upto = lane_sums(each * mine.tiles);
    const int parts = __builtin_amdgcn_readlane(each, seq & 63), tiles = __builtin_amdgcn_readlane(mine.tiles, seq & 63);
    first += __builtin_amdgcn_readlane(upto, seq & 63) - parts * tiles;
    if (parts <= 1) return;
    const bool live = row < rows;
    const int at = live ? row : rows - 1, tile = at / kTileRows, in_tile = at % kTileRows;
    const auto part_row = [&](int p) {
        return ((int64_t)(first + p * tiles + tile) * a.kv.heads + head) * kTileRows + in_tile;
    };
    f32x4_t acc[N] = {};
    float l = 0.0f, top = kNoMax;
    for (int p0 = 0; p0 < parts; p0 += 16) {
        const float2 ml = p0 + in_row < parts ? *(const float2*)(a.part_ml + part_row(p0 + in_row) * 2) : make_float2(0.0f, 0.0f);
        float mn = ml.y != 0.0f ? ml.x : kNoMax;
#pragma unroll
        for (int i = 1; i < 16; i <<= 1) mn = fmaxf(mn, __shfl_xor(mn, i, 16));
        mn = fmaxf(top, mn);
        const float f = __builtin_amdgcn_exp2f(top - mn), w = ml.y != 0.0f ? __builtin_amdgcn_exp2f(ml.x - mn) : 0.0f;
        top = mn;
        float part_l = ml.y * w;
#pragma unroll
        for (int i = 1; i < 16; i <<= 1) part_l += __shfl_xor(part_l, i, 16);
        l = l * f + part_l;
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] *= f;
        const int here = min(16, parts - p0);
        for (int j0 = 0; j0 < here; j0 += kAhead) {
            f32x4_t v[kAhead][N];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const float* const p = a.part_o + part_row(min(p0 + j0 + j, parts - 1)) * D + in_row * (4 * N);
#pragma unroll
                for (int i = 0; i < N; ++i) v[j][i] = ((const f32x4_t*)p)[i];
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const float g = j0 + j < here ? __shfl(w, j0 + j, 16) : 0.0f;
                if (g == 0.0f) continue;                 // a part without a key was not written
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][r] = __builtin_fmaf(v[j][i][r], g, acc[i][r]);
            }
        }
    }
    if (!live) return;
    const int i = row / a.group, qh = head * a.group + row - i * a.group;
    const int64_t out = (int64_t)(qr.first + i) * a.q_heads + qh;
    float lse;
    const float f = finish_row(top, l, a.sinks, qh, lse) * unshift * (a.kv.v_outer ? a.kv.v_outer[head] : 1.0f);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        float y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = l == 0.0f ? 0.0f : acc[n][r] * f;
        const int64_t to = out * D + in_row * (4 * N) + 4 * n;
        if (a.out_f32) *(float4*)((float*)a.out + to) = make_float4(y[0], y[1], y[2], y[3]);
        else *(uint2*)((uint16_t*)a.out + to) = make_uint2(Dec<0>::round2(y[0], y[1]), Dec<0>::round2(y[2], y[3]));
    }
    if (a.lse && in_row == 0) a.lse[out] = lse;
}

template <int D, int BIAS, bool FINE, bool TREE>
__global__ __launch_bounds__(512, D == 256 ? 2 : 4) void k_attn_tiles(AttnArgs a)
{
    using T = Tiles<D>;
    constexpr int QT = T::kQT;
    extern __shared__ __align__(16) unsigned char smem[];
    lds_t* const lds = (lds_t*)smem;
    lds_t* const flags = lds + 2 * T::kRound;
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    int head, b, split, block, parts = 1;
    if constexpr (TREE) {
        head = (int)blockIdx.x % a.kv.heads;
        const TreePlace p = tree_place<D>(a, (int)blockIdx.x / a.kv.heads, lane);
        if (p.parts == 0) return;
        b = p.seq, block = p.tile, split = p.part, parts = p.parts;
    } else {
        head = (int)blockIdx.x;
        b = (int)blockIdx.z % a.batch, split = (int)blockIdx.z / a.batch;
        // the last rows, which see the most keys, first
        block = (int)(gridDim.y - 1 - blockIdx.y);
    }
    const QueryRange qr = queries_of(a, b);
    const int kv = kv_length(a.kv_lens[b], a.max_kv, a.table_cols, a.kv.page_size, a.kv.num_pages);
    const int count = qr.count * a.group;
    if (!TREE && count <= kFewRows && a.batch > 1) return;   // k_attn_few's
    if (block * kTileRows >= count) return;
    const int row0 = block * kTileRows + wave * (16 * QT);
    Rows<D, BIAS, QT, TREE> rows;
    Sums<D, QT> sum;
    rows.load(a, qr, kv, head, row0, lane);
    sum.clear();
    // keys of the workgroup's rows (this split's part) and of the wave's
    const KeyRange kf = first_range<TREE>(a, block * kTileRows / a.group, qr.count, kv);
    const KeyRange kl = last_range<TREE>(a, (min((block + 1) * kTileRows, count) - 1) / a.group, qr.count, kv);
    const KeyRange seen{kf.lo, kl.hi};
    KeyRange mine;
    if constexpr (TREE) mine = tree_part(kf, kl, T::kKeys, split, parts);
    else mine = tile_part(kf, kl, T::kKeys, split, a.chunk);
    const int begin = mine.lo, end = mine.hi;
    const int my_end = row0 < count ? min(rows.last.hi, end) : 0;

    const DecodePart<D, BIAS> part(a.kv, wave, lane);
    const int32_t* table = a.table + (int64_t)b * a.table_cols;
    // rows of the part's step in the next 64 rounds, a round a lane
    int64_t row[2];
    int known = 64, looked = begin;                      // the next round to look up
    const auto next_rows = [&](int64_t (&g)[2]) {
        if (known == 64) {
            known = 0;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const KvGroup k = kv_group(table, looked + lane * T::kKeys + part.step * kStep + kKvGroup * s, kv, a.per_page,
                                           a.kv.num_pages, a.kv.heads, head);
                row[s] = k.ok ? k.row : -1;
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)row[s], known);
            const int32_t hi = __builtin_amdgcn_readlane((int32_t)(row[s] >> 32), known);
            g[s] = (int64_t)hi << 32 | lo;
        }
        ++known;
        looked += T::kKeys;
    };

    if (begin < end) {                                   // the same for all waves
        typename DecodePart<D, BIAS>::Bytes now, next;
        int64_t g0[2], g1[2];
        next_rows(g0);
        part.load(g0, now);
        next_rows(g1);
        part.load(g1, next);
        part.decode(g0, begin + part.step * kStep, seen, now, lds, flags);
        int buf = 0;
        for (int at = begin; at < end; at += T::kKeys, buf ^= 1) {
            lds_barrier();                               // this round is decoded, the other one's place is free
            now = next;
            g0[0] = g1[0], g0[1] = g1[1];
            if (at + T::kKeys < end) {
                next_rows(g1);
                part.load(g1, next);
                part.decode(g0, at + T::kKeys + part.step * kStep, seen, now, lds + (buf ^ 1) * T::kRound,
                            flags + (buf ^ 1) * (T::kSteps * 16));
            }
            if (my_end <= at || at + T::kKeys <= rows.first.lo) continue;   // nothing of this round is seen
#pragma unroll 1
            for (int s = 0; s < T::kSteps; ++s) {
                const int k = at + s * kStep;
                if (k >= my_end) break;
                FromLds<D, BIAS, QT> src{lds + buf * T::kRound + s * T::kStepBytes + lane * 16};
                const uint32_t groups = __builtin_amdgcn_readfirstlane(
                    *(const __attribute__((address_space(3))) uint32_t*)(flags + buf * (T::kSteps * 16) + s * 16));
                attend_step<D, BIAS, QT, FINE, TREE>(src, groups, k, my_end, rows, lane, sum);
            }
        }
    }
    if (row0 >= count) return;
    if (TREE && parts > 1)
        write_parts<D, BIAS, QT, TREE>(a, rows, sum, (int64_t)blockIdx.x * kTileRows + wave * (16 * QT), false, lane);
    else if (!TREE && a.splits > 1)
        write_parts<D, BIAS, QT, TREE>(a, rows, sum, (int64_t)split * a.total_q * a.q_heads, true, lane);
    else write_rows<D, BIAS, QT, FINE, TREE>(a, rows, sum, head, lane);
}

// Joins the splits of one row a wave: row r of sequence b's.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, float unshift)
{
    const int lane = (int)threadIdx.x & 63;
    const int64_t rows = (int64_t)a.total_q * a.q_heads;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= rows) return;
    // only rows that k_attn_tiles took have partial results
    const int token = (int)(row / a.q_heads), qh = (int)(row - (int64_t)token * a.q_heads);
    bool mine = false;
    for (int b = lane; b < a.batch; b += 64) {
        const QueryRange r = queries_of(a, b);
        mine |= token >= r.first && token < r.first + r.count && (a.batch == 1 || r.count * a.group > kFewRows);
    }
    if (!__any(mine)) return;
    // lane s holds split s's (m, l); a row's reference is the largest m of those that saw a key
    static_assert(kMaxSplits <= 64, "a lane for each split");
    const float2 ml = lane < a.splits ? *(const float2*)(a.part_ml + (lane * rows + row) * 2) : make_float2(0.0f, 0.0f);
    const float top = group_max<64>(ml.y != 0.0f ? ml.x : kNoMax);
    const float w = ml.y != 0.0f ? __builtin_amdgcn_exp2f(ml.x - top) : 0.0f;
    float l = ml.y * w;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) l += __shfl_xor(l, i, 64);
    constexpr int N = D / 64;
    float acc[N] = {};
    const uint64_t used = __ballot(ml.y != 0.0f);
    for (int s0 = 0; s0 < a.splits; s0 += 8) {
        float p[8][N];
#pragma unroll
        for (int j = 0; j < 8; ++j) {                    // parts without a key were not written
            const bool on = (used >> (s0 + j)) & 1;
            const float* q = a.part_o + ((s0 + j) * rows + row) * D + lane * N;
#pragma unroll
            for (int i = 0; i < N; ++i) p[j][i] = on ? q[i] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = __shfl(w, s0 + j, 64);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = __builtin_fmaf(p[j][i], f, acc[i]);
        }
    }
    write_joined<D>(a, row, qh, top, l, acc, unshift, lane);
}

template <int D, int BIAS, int QT, bool FINE, bool TREE>
hipError_t launch_few(AttnArgs a, hipStream_t s)
{
    constexpr int lds = lds_bytes<D, BIAS, QT>();
    static OncePerDevice once;
    const hipError_t st = allow_lds(once, reinterpret_cast<const void*>(k_attn_few<D, BIAS, QT, FINE, TREE>), lds);
    if (st != hipSuccess) return st;
    a.part_o = a.few_o;
    a.part_ml = a.few_ml;
    hipLaunchKernelGGL((k_attn_few<D, BIAS, QT, FINE, TREE>), dim3((uint32_t)a.groups), dim3(64 * kWaves), lds, s, a);
    if (a.slots) {
        const int64_t rows = std::min<int64_t>((int64_t)a.max_q * a.group, kFewRows);
        hipLaunchKernelGGL((k_attn_few_join<D, QT, TREE>), dim3((uint32_t)((rows + 3) / 4), (uint32_t)a.kv.heads, (uint32_t)a.batch),
                           dim3(256), 0, s, a, Dec<BIAS>::kUnshift);
    }
    return hipGetLastError();
}

template <int D, int BIAS, bool FINE, bool TREE>
hipError_t launch_dim(const AttnArgs& a, hipStream_t s)
{
    using T = Tiles<D>;
    const int64_t rows = (int64_t)a.max_q * a.group;
    if (rows <= 16) return launch_few<D, BIAS, 1, FINE, TREE>(a, s);
    if (rows <= kFewRows) return launch_few<D, BIAS, 2, FINE, TREE>(a, s);
    if (!TREE && a.groups) {                             // a batch may hold sequences of few rows too
        const hipError_t st = launch_few<D, BIAS, 2, FINE, TREE>(a, s);
        if (st != hipSuccess) return st;
    }
    static OncePerDevice once;
    const hipError_t st = allow_lds(once, reinterpret_cast<const void*>(k_attn_tiles<D, BIAS, FINE, TREE>), T::kLds);
    if (st != hipSuccess) return st;
    if constexpr (TREE) {
        AttnArgs t = a;
        t.part_o = a.few_o;
        t.part_ml = a.few_ml;
        const TreeGrid g = tree_grid(TreePlan{a.slots, a.slots ? a.groups / a.kv.heads : 0}, a.batch, a.kv.heads, rows);
        hipLaunchKernelGGL((k_attn_tiles<D, BIAS, FINE, TREE>), dim3(g.x, g.y, g.z), dim3(64 * T::kWaves), T::kLds, s, t);
        if (a.slots)
            hipLaunchKernelGGL((k_attn_tree_join<D>), dim3((uint32_t)((rows + 15) / 16), (uint32_t)a.kv.heads, (uint32_t)a.batch),
                               dim3(256), 0, s, t, Dec<BIAS>::kUnshift);
    } else {
        const dim3 grid((uint32_t)a.kv.heads, (uint32_t)((rows + kTileRows - 1) / kTileRows), (uint32_t)(a.batch * a.splits));
        hipLaunchKernelGGL((k_attn_tiles<D, BIAS, FINE, TREE>), grid, dim3(64 * T::kWaves), T::kLds, s, a);
        if (a.splits > 1) {
            const int64_t all = (int64_t)a.total_q * a.q_heads;
            hipLaunchKernelGGL((k_attn_join<D>), dim3((uint32_t)((all + 3) / 4)), dim3(256), 0, s, a, Dec<BIAS>::kUnshift);
        }
    }
    return hipGetLastError();
}

template <int BIAS, bool TREE>
hipError_t launch_bias(const AttnArgs& a, hipStream_t s)
{
    if (a.kv.dim == 64) return a.out_f32 ? launch_dim<64, BIAS, true, TREE>(a, s) : launch_dim<64, BIAS, false, TREE>(a, s);
    if (a.kv.dim == 128) return a.out_f32 ? launch_dim<128, BIAS, true, TREE>(a, s) : launch_dim<128, BIAS, false, TREE>(a, s);
    return a.out_f32 ? launch_dim<256, BIAS, true, TREE>(a, s) : launch_dim<256, BIAS, false, TREE>(a, s);
}

}  // namespace

}  // namespace fp4q
