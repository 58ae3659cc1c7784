// kernels_attn.hip -- attention over the paged 4-bit cache for gfx950.
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
// and O are binary32.  FP16 holds q scaled by a power of two per row: its bits are
// kept down to 2^-28 of the row's largest value.
//
// Running maximum.  m moves only when some row's score exceeds it by 8 (powers of
// two), so P stays below 2^8 and O is seldom rescaled.
//
// Few rows: the four waves of a workgroup take every fourth step of the same rows and
// join through LDS, and the keys are split over workgroups, whose partial (O, m, l) a
// second kernel joins (launch_attn).
#include <type_traits>

#include "fp4q_device.h"
#include "kv_index.h"
#include "launch.h"
#include "mfma16.h"

namespace fp4q {

namespace {

constexpr int kWaves = 4;
constexpr int kStep = 32;                                // keys of a step
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3.4028235e38f;                 // m of a row that has seen no key
constexpr float kLazy = 8.0f;

// The largest of a value over the four lanes of a column (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float column_max(float v)
{
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

// The codes and scale bytes of one step, as loaded.
template <int D, int BIAS>
struct Raw {
    static constexpr int kKW = D / 32;                   // dwords of a quarter row of K
    static constexpr int kVW = D / 16 < 8 ? 1 : D / 128; // dwords of D / 16 codes of V
    uint32_t k[2][kKW], ks[2], v[8][kVW], vs[8];
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w)
{
    if constexpr (N == 1) {
        w[0] = *(const uint32_t*)p;
    } else if constexpr (N == 2) {
        const uint2 u = *(const uint2*)p;
        w[0] = u.x, w[1] = u.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 u = ((const uint4*)p)[i];
            w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
    }
}

template <int N>
__device__ __forceinline__ uint32_t load_bytes(const uint8_t* p)
{
    if constexpr (N == 1) return *p;
    else if constexpr (N == 2) return *(const uint16_t*)p;
    else return *(const uint32_t*)p;
}

template <int D, int BIAS>
__device__ __forceinline__ void load_step(const KvView& kv, const KvGroup (&g)[2], int lane, Raw<D, BIAS>& r)
{
    constexpr int B = Dec<BIAS>::kBlock;
    constexpr int KB = D / 4 / B > 0 ? D / 4 / B : 1;    // scale bytes of a quarter row of K
    const int m = lane & 15, q = lane >> 4;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const uint8_t* kc = kv.k_codes + g[s].row * (D / 2);
        const uint8_t* ks = kv.k_scales + g[s].row * (D / B);
        const uint8_t* vc = kv.v_codes + g[s].row * (D / 2);
        const uint8_t* vs = kv.v_scales + g[s].row * (D / B);
        load_words<Raw<D, BIAS>::kKW>(kc + m * (D / 2) + q * (D / 8), r.k[s]);
        r.ks[s] = load_bytes<KB>(ks + m * (D / B) + q * (D / 4) / B);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint8_t* p = vc + (4 * q + t) * (D / 2) + m * (D / 32);
            if constexpr (D == 64) r.v[4 * s + t][0] = *(const uint16_t*)p;
            else load_words<Raw<D, BIAS>::kVW>(p, r.v[4 * s + t]);
            r.vs[4 * s + t] = vs[(4 * q + t) * (D / B) + m * (D / 16) / B];
        }
    }
}

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
    float f = 1.0f;
    if (sinks) {
        const float s = sinks[head] * kLog2e;
        const float top = fmaxf(m, s);
        f = __builtin_amdgcn_exp2f(m - top);
        l = l * f + __builtin_amdgcn_exp2f(s - top);
        m = top;
    }
    if (l == 0.0f) {                                     // a row that sees nothing
        lse = -__builtin_inff();
        return 0.0f;
    }
    lse = (m + __builtin_log2f(l)) * kLn2;
    return f / l;
}

// MXFP4 keys some rows see and others do not, with a poisoned block of V: 0 times
// its NaN would reach the rows that do not see the key.  Such blocks are cleared,
// and the product of (block is poisoned) with (row sees the key) says which
// outputs become NaN.  All of a lane's values of V lie in one block.
template <int ND, int QT, class R>
__device__ __forceinline__ void poison_seen(R& raw, const f32x4_t (&sc)[QT][2], f32x4_t (&o)[QT][ND], uint4 ones)
{
    bool any = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) any |= raw.vs[j] == 0xFFu;
    if (!__any(any)) return;
    uint32_t bad[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        bad[j] = (raw.vs[2 * j] == 0xFFu ? ones.x & 0xFFFFu : 0u) | (raw.vs[2 * j + 1] == 0xFFu ? ones.x & 0xFFFF0000u : 0u);
#pragma unroll
    for (int j = 0; j < 8; ++j) raw.vs[j] = raw.vs[j] == 0xFFu ? 0u : raw.vs[j];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        uint32_t seen[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = sc[t][j >> 1][2 * (j & 1)], b = sc[t][j >> 1][2 * (j & 1) + 1];
            seen[j] = (a != -__builtin_inff() ? ones.x & 0xFFFFu : 0u) | (b != -__builtin_inff() ? ones.x & 0xFFFF0000u : 0u);
        }
        const f32x4_t n = Dec<0>::mfma(make_uint4(bad[0], bad[1], bad[2], bad[3]),
                                       make_uint4(seen[0], seen[1], seen[2], seen[3]), f32x4_t{0, 0, 0, 0});
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int d = 0; d < ND; ++d) o[t][d][r] = n[r] > 0.0f ? __builtin_nanf("") : o[t][d][r];
    }
}

template <int D, int BIAS, int QT>
__global__ __launch_bounds__(64 * kWaves, D == 256 && QT == 2 ? 1 : 2) void k_attn(AttnArgs a)
{
    using X = Dec<BIAS>;
    constexpr int NK = D / 32;                           // products of a step's scores
    constexpr int ND = D / 16;                           // products of a step's outputs (values of V in a lane)
    constexpr int kRows = 16 * QT;
    constexpr int kLine = QT * (D / 4 + 2);              // floats of a lane's partial result
    __shared__ float join[2][kLine][64];

    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int head = (int)blockIdx.x;
    const int b = (int)blockIdx.z % a.batch, split = (int)blockIdx.z / a.batch;
    const QueryRange qr = queries_of(a, b);
    const int kv = kv_length(a.kv_lens[b], a.max_kv, a.table_cols, a.kv.page_size, a.kv.num_pages);
    const int rows = qr.count * a.group;
    if (rows == 0) return;
    // Rows that fit one wave are shared by the four (each takes every fourth step);
    // otherwise each wave has rows of its own and takes every step.
    const bool shared = rows <= kRows;
    const int row0 = shared ? 0 : ((int)blockIdx.y * kWaves + wave) * kRows;
    if (shared ? blockIdx.y > 0 : (int)blockIdx.y * kWaves * kRows >= rows) return;

    // keys of this wave's rows: those of its first and last query
    const bool idle = row0 >= rows;
    const int first_q = min(row0, rows - 1) / a.group, last_q = (min(row0 + kRows, rows) - 1) / a.group;
    const KeyRange kf = key_range(first_q, qr.count, kv, a.causal, a.window);
    const KeyRange kl = key_range(last_q, qr.count, kv, a.causal, a.window);
    const int base = kf.lo / kStep * kStep;
    const int begin = base + split * a.chunk;
    const int end = idle ? 0 : min(kl.hi, begin + a.chunk);

    uint4 q[QT][NK];
    float c[QT];
    KeyRange see[QT];
    int64_t out_row[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int r = row0 + 16 * t + col;
        const bool live = r < rows;
        const int i = live ? r / a.group : 0, g = live ? r - i * a.group : 0;
        see[t] = key_range(i, qr.count, kv, a.causal, a.window);
        out_row[t] = live ? (int64_t)(qr.first + i) * a.q_heads + head * a.group + g : -1;
        const uint16_t* p = a.q + (int64_t)(qr.first + i) * a.ld_q + (int64_t)(head * a.group + g) * D + quarter * (D / 4);
#pragma unroll
        for (int k = 0; k < NK; ++k) q[t][k] = live ? ((const uint4*)p)[k] : make_uint4(0, 0, 0, 0);
        c[t] = a.scale * kLog2e * X::kUnshift;
        if constexpr (!X::kBf16) {
            c[t] *= q_to_f16<NK>(q[t]);
            if (a.kv.k_outer) c[t] *= a.kv.k_outer[head];
        }
        c[t] = fmaxf(c[t], 1.17549435e-38f);             // 0 would turn a masked score into NaN
    }

    f32x4_t o[QT][ND], l[QT];
    float m[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        m[t] = kNoMax;
        l[t] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int n = 0; n < ND; ++n) o[t][n] = f32x4_t{0, 0, 0, 0};
    }

    const int32_t* table = a.table + (int64_t)b * a.table_cols;
    const int stride = shared ? kWaves * kStep : kStep;
    int at = begin + (shared ? wave * kStep : 0);
    KvGroup grp[2];
    Raw<D, BIAS> cur;
    const uint4 ones = make_uint4(X::kOnes, X::kOnes, X::kOnes, X::kOnes);
    auto fetch = [&](int t0, KvGroup (&g)[2], Raw<D, BIAS>& r) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
            g[s] = kv_group(table, t0 + 16 * s, end, a.per_page, a.kv.num_pages, a.kv.heads, head);
        load_step<D, BIAS>(a.kv, g, lane, r);
    };
    if (at < end) fetch(at, grp, cur);
    for (; at < end; at += stride) {
        Raw<D, BIAS> nxt;
        KvGroup grp_n[2];
        fetch(at + stride, grp_n, nxt);                  // past the end: the cache's first rows, unused

        // scores: S^T[key, row], keys 16 s + 4 quarter + r
        f32x4_t sc[QT][2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            uint4 kf8[NK];
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                constexpr int per = X::kBlock / 8;       // words of a block
                const uint32_t byte = D / 4 <= X::kBlock ? cur.ks[s] : (cur.ks[s] >> (8 * (i / per))) & 0xFFu;
                kf8[i] = X::octet(cur.k[s][i], X::scale(byte));
            }
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                sc[t][s] = f32x4_t{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < NK; ++i) sc[t][s] = X::mfma(kf8[i], q[t][i], sc[t][s]);
            }
        }

        // A step whose keys are not all seen by all rows: scores of unseen keys are
        // -infinity, and the scales of keys beyond the end (whose bytes may be
        // anything, NaN among them) are cleared so that 0 times V is 0.
        const bool whole = grp[0].ok && grp[1].ok && at >= kl.lo && at + kStep <= kf.hi && at + kStep <= end;
        if (!whole) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int key = at + 16 * s + 4 * quarter + r;
                    const bool there = grp[s].ok && key < end;
#pragma unroll
                    for (int t = 0; t < QT; ++t)
                        if (!there || key < see[t].lo || key >= see[t].hi) sc[t][s][r] = -__builtin_inff();
                    if (!there) cur.vs[4 * s + r] = 0;
                }
            if constexpr (BIAS == 0) poison_seen<ND, QT>(cur, sc, o, ones);
        }

        // running maximum, P
        uint4 p[QT];
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            float top = fmaxf(fmaxf(fmaxf(sc[t][0][0], sc[t][0][1]), fmaxf(sc[t][0][2], sc[t][0][3])),
                              fmaxf(fmaxf(sc[t][1][0], sc[t][1][1]), fmaxf(sc[t][1][2], sc[t][1][3])));
            top *= c[t];
            if (__any(top > m[t] + kLazy)) {
                const float mn = fmaxf(m[t], column_max(top));
                const float f = __builtin_amdgcn_exp2f(m[t] - mn);
                m[t] = mn;
                l[t] *= f;
#pragma unroll
                for (int n = 0; n < ND; ++n) o[t][n] *= f;
            }
            float e[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) e[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][k >> 2][k & 3], c[t], -m[t]));
            p[t] = make_uint4(X::round2(e[0], e[1]), X::round2(e[2], e[3]), X::round2(e[4], e[5]), X::round2(e[6], e[7]));
            l[t] = X::mfma(ones, p[t], l[t]);
        }

        // O^T += V^T P^T, two values of head_dim (one byte of codes) at a time
        uint32_t vs[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) vs[j] = X::scale(cur.vs[j]);
        auto two = [&](auto byte_c) {
            constexpr int y = decltype(byte_c)::value;
            uint32_t u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = X::template pair<(y & 3)>(cur.v[j][y >> 2], vs[j]);
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lo[j] = __builtin_amdgcn_perm(u[2 * j + 1], u[2 * j], 0x05040100u);
                hi[j] = __builtin_amdgcn_perm(u[2 * j + 1], u[2 * j], 0x07060302u);
            }
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                o[t][2 * y] = X::mfma(make_uint4(lo[0], lo[1], lo[2], lo[3]), p[t], o[t][2 * y]);
                o[t][2 * y + 1] = X::mfma(make_uint4(hi[0], hi[1], hi[2], hi[3]), p[t], o[t][2 * y + 1]);
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
        cur = nxt;
        grp[0] = grp_n[0];
        grp[1] = grp_n[1];
    }

    // This lane's part of a row: d = (D / 4) quarter + ND r + n from o[n][r].
    float res[QT][D / 4], lsum[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        lsum[t] = l[t][0];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int n = 0; n < ND; ++n) res[t][ND * r + n] = o[t][n][r];
    }

    if (shared) {
        // join the four waves: 2 and 3 into 0 and 1, then 1 into 0
#pragma unroll
        for (int half = 2; half >= 1; half >>= 1) {
            if (wave >= half && wave < 2 * half) {
                float(*w)[64] = join[wave - half];
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    w[t * (D / 4 + 2)][lane] = m[t];
                    w[t * (D / 4 + 2) + 1][lane] = lsum[t];
#pragma unroll
                    for (int i = 0; i < D / 4; ++i) w[t * (D / 4 + 2) + 2 + i][lane] = res[t][i];
                }
            }
            __syncthreads();
            if (wave < half) {
                float(*w)[64] = join[wave];
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    const float mo = w[t * (D / 4 + 2)][lane], mn = fmaxf(m[t], mo);
                    const float f = __builtin_amdgcn_exp2f(m[t] - mn), g = __builtin_amdgcn_exp2f(mo - mn);
                    m[t] = mn;
                    lsum[t] = lsum[t] * f + w[t * (D / 4 + 2) + 1][lane] * g;
#pragma unroll
                    for (int i = 0; i < D / 4; ++i) res[t][i] = res[t][i] * f + w[t * (D / 4 + 2) + 2 + i][lane] * g;
                }
            }
            __syncthreads();
        }
        if (wave != 0) return;
    }

    const float unshift = X::kUnshift * (a.kv.v_outer ? a.kv.v_outer[head] : 1.0f);
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        if (out_row[t] < 0) continue;
        if (a.splits > 1) {
            const int64_t row = (int64_t)split * a.total_q * a.q_heads + out_row[t];
            if (quarter == 0) *(float2*)(a.part_ml + row * 2) = make_float2(m[t], lsum[t]);
            if (lsum[t] != 0.0f) store_row<D>(a.part_o, true, row, quarter, res[t]);
        } else {
            const int qh = head * a.group + (int)((out_row[t] - (int64_t)head * a.group) % a.q_heads);
            float lse;
            const float f = finish_row(m[t], lsum[t], a.sinks, qh, lse) * unshift;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) res[t][i] = lsum[t] == 0.0f ? 0.0f : res[t][i] * f;
            store_row<D>(a.out, a.out_f32 != 0, out_row[t], quarter, res[t]);
            if (a.lse && quarter == 0) a.lse[out_row[t]] = lse;
        }
    }
}

// Joins the splits of one row a wave: row r of sequence b's.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, float unshift)
{
    const int lane = (int)threadIdx.x & 63;
    const int64_t rows = (int64_t)a.total_q * a.q_heads;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= rows) return;
    // only rows of some sequence have partial results
    const int token = (int)(row / a.q_heads), qh = (int)(row - (int64_t)token * a.q_heads);
    bool mine = false;
    for (int b = lane; b < a.batch; b += 64) {
        const QueryRange r = queries_of(a, b);
        mine |= token >= r.first && token < r.first + r.count;
    }
    if (!__any(mine)) return;
    float top = kNoMax;
    for (int s = lane; s < a.splits; s += 64) {
        const float2 ml = *(const float2*)(a.part_ml + (s * rows + row) * 2);
        if (ml.y != 0.0f) top = fmaxf(top, ml.x);
    }
    top = group_max<64>(top);
    constexpr int N = D / 64;
    float acc[N] = {}, l = 0.0f;
    for (int s = 0; s < a.splits; ++s) {
        const float2 ml = *(const float2*)(a.part_ml + (s * rows + row) * 2);
        if (ml.y == 0.0f) continue;
        const float f = __builtin_amdgcn_exp2f(ml.x - top);
        l += ml.y * f;
        const float* p = a.part_o + (s * rows + row) * D + lane * N;
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += p[i] * f;
    }
    float lse;
    const bool none = l == 0.0f;
    float f = finish_row(top, l, a.sinks, qh, lse) * unshift;
    if (a.kv.v_outer) f *= a.kv.v_outer[qh / a.group];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float y = none ? 0.0f : acc[i] * f;
        if (a.out_f32) ((float*)a.out)[row * D + lane * N + i] = y;
        else ((uint16_t*)a.out)[row * D + lane * N + i] = (uint16_t)f32_to_bf16(y);
    }
    if (a.lse && lane == 0) a.lse[row] = lse;
}

template <int D, int BIAS>
hipError_t launch_dim(const AttnArgs& a, hipStream_t s)
{
    const int64_t rows = (int64_t)a.max_q * a.group;
    const int block = attn_block_rows(rows);
    const dim3 grid((uint32_t)a.kv.heads, (uint32_t)((rows + block - 1) / block), (uint32_t)(a.batch * a.splits));
    if (rows <= 16) hipLaunchKernelGGL((k_attn<D, BIAS, 1>), grid, dim3(64 * kWaves), 0, s, a);
    else hipLaunchKernelGGL((k_attn<D, BIAS, 2>), grid, dim3(64 * kWaves), 0, s, a);
    hipError_t st = hipGetLastError();
    if (st != hipSuccess || a.splits == 1) return st;
    const int64_t all = (int64_t)a.total_q * a.q_heads;
    hipLaunchKernelGGL((k_attn_join<D>), dim3((uint32_t)((all + 3) / 4)), dim3(256), 0, s, a, Dec<BIAS>::kUnshift);
    return hipGetLastError();
}

template <int BIAS>
hipError_t launch_bias(const AttnArgs& a, hipStream_t s)
{
    if (a.kv.dim == 64) return launch_dim<64, BIAS>(a, s);
    if (a.kv.dim == 128) return launch_dim<128, BIAS>(a, s);
    return launch_dim<256, BIAS>(a, s);
}

}  // namespace

int attn_block_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 32 * kWaves; }

int attn_splits(int64_t batch, int32_t kv_heads, int64_t rows, int64_t max_kv)
{
    const int block = attn_block_rows(rows);
    const int64_t blocks = batch * kv_heads * ((rows + block - 1) / block);
    int64_t want = (1024 + blocks - 1) / blocks;
    const int64_t most = (max_kv + 511) / 512;           // at least four steps for each wave
    if (want > most) want = most;
    if (want > 64) want = 64;
    return want < 1 ? 1 : (int)want;
}

hipError_t launch_attn(int bias, const AttnArgs& a, hipStream_t s)
{
    if (bias == 0) return launch_bias<0>(a, s);
    if (bias == 7) return launch_bias<7>(a, s);
    return launch_bias<15>(a, s);
}

}  // namespace fp4q
