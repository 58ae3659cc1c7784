// kernels_moe.hip -- a mixture-of-experts layer with 4-bit experts for a few tokens.
//
//   y_t = sum over the k experts e with token t's largest logits of
//         a_te (W2_e act(W1_e x_t + b1_e) + b2_e),   a_te the softmax of the logits
//
// Every expert that a token reached is read once, which is what bounds the layer: 4 bits
// and a scale's share a weight, for few tokens each.  Three launches:
//   k_moe_route  one workgroup: each token's experts and their shares, then the (token, expert)
//                pairs in the order of the experts and their groups of up to kGroup
//                pairs of one expert;
//   k_moe_up     a workgroup takes 16 gate and 16 up rows of W1 for one group; its waves share K
//                and join through LDS; a times the activation goes to the scratch in bf16;
//   k_moe_down   a workgroup takes 16 rows of W2 for all groups: its waves share the
//                groups' K, each adding its sums to its own [tokens][16] of LDS, joined at the
//                end in order.  Where 16 rows a workgroup leave compute units idle the groups are
//                split over workgroups too, whose sums k_moe_join adds in order.
//
// Products as in kernels_linear.hip: v_mfma_f32_16x16x32_bf16 with rows of W decoded to bf16,
// exactly, as the A operand and tokens as the B operand; a step is two times 64 values of K, of
// which lane l holds 16 (l / 16) .. + 15 of row l % 16.  Sums are binary32.
//
// Rounding.  a act is rounded to bf16 before W2, as an activation between two products is;
// where the result is asked for in binary32 (FINE) it enters as two such terms, good to 2^-16.
#include "fp4q_device.h"
#include "launch.h"
#include "lds_load.h"
#include "mfma16.h"

namespace fp4q {

namespace {

enum { kInnerOnly = 0, kPerTile = 1, kPerRow = 2 };      // outer scales inside the sum: none (or one an expert), 2D, 1D

constexpr int kGroup = 64;                               // pairs of a group, at most
constexpr int kUpWaves = 4, kDownWaves = 16;
constexpr int kRouteThreads = 1024;

// ---------------------------------------------------------------- routing
// Order of logits: a key that compares as the numbers do, -0 as 0, NaN and -infinity 0 (not
// taken).
__device__ __forceinline__ uint32_t order_key(float v)
{
    v += 0.0f;
    const uint32_t u = __float_as_uint(v);
    if (!(v > -__builtin_inff())) return 0;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)v, m, 64);
        v = v > o ? v : o;
    }
    return v;
}

constexpr int kMaxPerLane = kMoeMaxExperts / 64;

__global__ __launch_bounds__(kRouteThreads) void k_moe_route(MoeArgs a)
{
    __shared__ uint32_t member[kMoeMaxExperts][kMoeMaxTokens / 32];
    __shared__ int first_pair[kMoeMaxExperts], first_group[kMoeMaxExperts];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    for (int i = (int)threadIdx.x; i < kMoeMaxExperts * (kMoeMaxTokens / 32); i += kRouteThreads) (&member[0][0])[i] = 0;
    __syncthreads();
    for (int t = wave; t < a.tokens; t += kRouteThreads / 64) {
        float l[kMaxPerLane];
        uint32_t key[kMaxPerLane];
#pragma unroll
        for (int j = 0; j < kMaxPerLane; ++j) {
            const int e = j * 64 + lane;
            l[j] = e < a.experts ? a.logits[(int64_t)t * a.experts + e] : -__builtin_inff();
            key[j] = order_key(l[j]);
        }
        float top = 0.0f, sum = 0.0f, mine = 0.0f;       // lane s keeps slot s's logit
        int chosen = -1;
        for (int s = 0; s < a.top_k; ++s) {
            uint64_t best = 0;
#pragma unroll
            for (int j = 0; j < kMaxPerLane; ++j) {
                const uint64_t c = (uint64_t)key[j] << 32 | (uint32_t)~(j * 64 + lane);
                best = key[j] != 0 && c > best ? c : best;
            }
            best = wave_max_u64(best);
            if (best == 0) break;                        // nothing left to take
            const int e = (int)~(uint32_t)best;
            float v = 0.0f;
#pragma unroll
            for (int j = 0; j < kMaxPerLane; ++j)
                if (j == e >> 6) {
                    v = l[j];
                    if ((e & 63) == lane) key[j] = 0;
                }
            v = __shfl(v, e & 63, 64);
            if (s == 0) top = v;
            sum += expf(v - top);
            if (lane == s) mine = v, chosen = e;
        }
        if (!a.renormalize) {                            // the softmax of all logits
            sum = 0.0f;
#pragma unroll
            for (int j = 0; j < kMaxPerLane; ++j) sum += l[j] > -__builtin_inff() ? expf(l[j] - top) : 0.0f;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m, 64);
        }
        if (lane < a.top_k) {
            a.expert[t * a.top_k + lane] = chosen;
            a.share[t * a.top_k + lane] = chosen >= 0 ? expf(mine - top) / sum : 0.0f;
            if (chosen >= 0) atomicOr(&member[chosen][t >> 5], 1u << (t & 31));
        }
    }
    __syncthreads();
    // pairs and groups before each expert's: wave 0, experts in runs of 64
    const auto count_of = [&](int e) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < kMoeMaxTokens / 32; ++w) n += __popc(member[e][w]);
        return n;
    };
    if (wave == 0) {
        int pairs = 0, groups = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 64) {
            const int e = e0 + lane, n = e < a.experts ? count_of(e) : 0, g = (n + kGroup - 1) / kGroup;
            int pn = n, gn = g;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const int p = __shfl_up(pn, m, 64), q = __shfl_up(gn, m, 64);
                pn += lane >= m ? p : 0;
                gn += lane >= m ? q : 0;
            }
            if (e < a.experts) {
                first_pair[e] = pairs + pn - n;
                first_group[e] = groups + gn - g;
            }
            pairs += __shfl(pn, 63, 64);
            groups += __shfl(gn, 63, 64);
        }
        if (lane == 0) a.counts[0] = groups, a.counts[1] = pairs;
    }
    __syncthreads();
    for (int e = (int)threadIdx.x; e < a.experts; e += kRouteThreads) {
        const int n = count_of(e);
        for (int g = 0; g * kGroup < n; ++g)
            a.groups[first_group[e] + g] = MoeGroup{e, first_pair[e] + g * kGroup, min(kGroup, n - g * kGroup), 0};
    }
    for (int p = (int)threadIdx.x; p < a.tokens * a.top_k; p += kRouteThreads) {
        const int e = a.expert[p], t = p / a.top_k;      // written by this workgroup before the barriers
        if (e < 0) continue;
        int at = first_pair[e];
        for (int w = 0; w < t >> 5; ++w) at += __popc(member[e][w]);
        at += __popc(member[e][t >> 5] & ((1u << (t & 31)) - 1));
        a.pair_token[at] = t;
        a.pair_share[at] = a.share[p];
    }
}

// ---------------------------------------------------------------- products
// Sixteen rows of one expert's weight, the lane's row among them, and their outer scales.
struct WRows {
    const uint8_t *codes, *scales;                       // at the lane's place of the row's first step
    const float* outer;                                  // 2D: the tile's first; 1D: of the first of the lane's four results
    int64_t outer_row;                                   // 1D: from one result's row to the next
};

// A lane's part of a step: 128 values of K in halves.
template <int OUTER>
struct WStep {
    uint2 c[2];
    uint32_t s[2];
    float o[OUTER == kInnerOnly ? 1 : 2][OUTER == kPerRow ? 4 : 1];
};

template <int BIAS, int OUTER>
__device__ __forceinline__ void load_step(const WRows& w, int k0, int K, int obs, int quarter, WStep<OUTER>& v)
{
    constexpr int B = Dec<BIAS>::kBlock;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int k = k0 + 64 * h;
        const bool in = k + 16 * quarter < K;            // values beyond K are zeros
        v.c[h] = in ? *(const uint2*)(w.codes + k / 2) : make_uint2(0, 0);
        v.s[h] = in ? w.scales[k / B] : 0;
        if constexpr (OUTER == kPerTile) v.o[h][0] = k < K ? w.outer[k >> 6] : 0.0f;
        if constexpr (OUTER == kPerRow) {
#pragma unroll
            for (int r = 0; r < 4; ++r) v.o[h][r] = k < K ? w.outer[r * w.outer_row + k / obs] : 0.0f;
        }
    }
}

template <int BIAS, int OUTER>
__device__ __forceinline__ void decode_half(const WStep<OUTER>& v, int h, uint4& w0, uint4& w1)
{
    const float sc = DecBf16<BIAS>::scale(v.s[h]);
    w0 = DecBf16<BIAS>::octet(v.c[h].x, sc);
    w1 = DecBf16<BIAS>::octet(v.c[h].y, sc);
}

template <int OUTER>
__device__ __forceinline__ void multiply_half(const WStep<OUTER>& v, int h, uint4 w0, uint4 w1, uint4 x0, uint4 x1, f32x4_t& acc)
{
    f32x4_t p = OUTER == kInnerOnly ? acc : f32x4_t{0, 0, 0, 0};
    p = Dec<0>::mfma(w0, x0, p);
    p = Dec<0>::mfma(w1, x1, p);
    if constexpr (OUTER == kInnerOnly) {
        acc = p;
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(p[r], v.o[h][OUTER == kPerRow ? r : 0], acc[r]);
    }
}

// Rows first + stride 0 .. 15 of expert e's weight of N rows (N is a multiple of 32).
template <int BIAS, int OUTER>
__device__ __forceinline__ WRows rows_of(const MoeWeight& w, int e, int first, int stride, int N, int K, int lane)
{
    constexpr int B = Dec<BIAS>::kBlock;
    const int row = lane & 15, quarter = lane >> 4;
    const int64_t r = (int64_t)e * N + first + stride * row;
    WRows v;
    v.codes = w.codes + r * (K / 2) + quarter * 8;
    v.scales = w.scales + r * (K / B) + (B == 16 ? quarter : quarter >> 1);
    v.outer = nullptr;
    v.outer_row = 0;
    if constexpr (OUTER == kPerTile) v.outer = w.outer + (((int64_t)e * N + first) >> 6) * (K >> 6);
    if constexpr (OUTER == kPerRow) {
        v.outer = w.outer + ((int64_t)e * N + first + stride * 4 * quarter) * (K / w.obs);   // results 4 quarter + 0 .. 3
        v.outer_row = (int64_t)stride * (K / w.obs);
    }
    return v;
}

__device__ __forceinline__ float gated(const MoeArgs& a, float g, float u)
{
    if (a.limit > 0.0f) {
        g = g > a.limit ? a.limit : g;
        u = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
    }
    return g / (1.0f + expf(-a.alpha * g)) * (u + a.shift);
}

template <int BIAS, int OUTER, int MT, bool FINE>
__global__ __launch_bounds__(64 * kUpWaves) void k_moe_up(MoeArgs a)
{
    __shared__ float join[kUpWaves][2 * MT * 4][64];
    if ((int)blockIdx.y >= a.counts[0]) return;
    const MoeGroup group = a.groups[blockIdx.y];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int i0 = (int)blockIdx.x * 16, K = a.hidden, N = 2 * a.inter;
    const int stride = a.interleaved ? 2 : 1;
    const WRows wg = rows_of<BIAS, OUTER>(a.w1, group.expert, i0 * stride, stride, N, K, lane);
    const WRows wu = rows_of<BIAS, OUTER>(a.w1, group.expert, a.interleaved ? 2 * i0 + 1 : a.inter + i0, stride, N, K, lane);
    const uint16_t* x[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        x[m] = 16 * m + col < group.count
                   ? a.x + (int64_t)a.pair_token[group.first + 16 * m + col] * a.ld_x + quarter * 16 : nullptr;

    f32x4_t acc[2][MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[0][m] = acc[1][m] = f32x4_t{0, 0, 0, 0};
    int k = wave * 128;
    WStep<OUTER> g, u;
    load_step<BIAS, OUTER>(wg, k, K, a.w1.obs, quarter, g);
    load_step<BIAS, OUTER>(wu, k, K, a.w1.obs, quarter, u);
    for (; k < K; k += kUpWaves * 128) {
        WStep<OUTER> gn, un;
        load_step<BIAS, OUTER>(wg, k + kUpWaves * 128, K, a.w1.obs, quarter, gn);
        load_step<BIAS, OUTER>(wu, k + kUpWaves * 128, K, a.w1.obs, quarter, un);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint4 g0, g1, u0, u1;
            decode_half<BIAS, OUTER>(g, h, g0, g1);
            decode_half<BIAS, OUTER>(u, h, u0, u1);
            const int at = k + 64 * h;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (16 * m >= group.count) break;        // uniform
                const bool in = x[m] != nullptr && at + 16 * quarter < K;
                const uint4* p = (const uint4*)(x[m] + at);
                const uint4 x0 = in ? p[0] : make_uint4(0, 0, 0, 0), x1 = in ? p[1] : make_uint4(0, 0, 0, 0);
                multiply_half<OUTER>(g, h, g0, g1, x0, x1, acc[0][m]);
                multiply_half<OUTER>(u, h, u0, u1, x0, x1, acc[1][m]);
            }
        }
        g = gn;
        u = un;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i) join[wave][m * 8 + i][lane] = acc[i >> 2][m][i & 3];
    __syncthreads();
    // wave m finishes token tile m
    if (wave >= MT || 16 * wave + col >= group.count) return;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = join[0][wave * 8 + i][lane];
#pragma unroll
        for (int w = 1; w < kUpWaves; ++w) v[i] += join[w][wave * 8 + i][lane];
    }
    const int pair = group.first + 16 * wave + col, i = i0 + 4 * quarter;
    const float whole = a.w1.outer_kind == kOuterTensor ? a.w1.outer[group.expert] : 1.0f, share = a.pair_share[pair];
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t b = (int64_t)group.expert * N + (a.interleaved ? 2 * (i + r) : i + r);
        const float gate = v[r] * whole + (a.b1 ? a.b1[b] : 0.0f);
        const float up = v[4 + r] * whole + (a.b1 ? a.b1[b + (a.interleaved ? 1 : a.inter)] : 0.0f);
        y[r] = share * gated(a, gate, up);
    }
    const uint2 hi = make_uint2(Dec<0>::round2(y[0], y[1]), Dec<0>::round2(y[2], y[3]));
    *(uint2*)(a.mid + (int64_t)pair * a.inter + i) = hi;
    if constexpr (FINE)
        *(uint2*)(a.mid_rest + (int64_t)pair * a.inter + i) =
            make_uint2(Dec<0>::rest2(y[0], y[1], hi.x), Dec<0>::rest2(y[2], y[3], hi.y));
}

// Four neighbouring values of y.
__device__ __forceinline__ void store_y4(const MoeArgs& a, int t, int n, f32x4_t v)
{
    const int64_t at = (int64_t)t * a.ld_y + n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (a.y_f32) ((float*)a.y)[at + i] = v[i];
        else ((uint16_t*)a.y)[at + i] = (uint16_t)Dec<0>::round2(v[i], 0.0f);
    }
}

// The token's shares of its experts' second biases, in the order of its choices.
__device__ __forceinline__ f32x4_t add_bias(const MoeArgs& a, int t, int n, f32x4_t v)
{
    if (!a.b2) return v;
    for (int s = 0; s < a.top_k; ++s) {
        const int e = a.expert[t * a.top_k + s];
        if (e < 0) break;
        const float share = a.share[t * a.top_k + s];
        const float* b = a.b2 + (int64_t)e * a.hidden;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(share, b[n + i], v[i]);
    }
    return v;
}

template <int BIAS, int OUTER, int MT, bool FINE>
__global__ __launch_bounds__(64 * kDownWaves) void k_moe_down(MoeArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int n0 = (int)blockIdx.x * 16, K = a.inter;
    const int groups = a.counts[0], steps = (K + 127) / 128;
    f32x4_t* const sums = (f32x4_t*)smem + wave * a.tokens * 4;   // [tokens][4 quarters of the 16 rows]
    for (int i = lane; i < a.tokens * 4; i += 64) sums[i] = f32x4_t{0, 0, 0, 0};

    const int parts = kDownWaves * (int)gridDim.y, part = (int)blockIdx.y * kDownWaves + wave;
    const int64_t total = (int64_t)groups * steps;
    const int from = (int)(total * part / parts), to = (int)(total * (part + 1) / parts);
    int at = from;
    while (at < to) {
        // the part's steps of one group
        const int gi = at / steps, s0 = at - gi * steps, s1 = min(steps, s0 + to - at);
        at += s1 - s0;
        const MoeGroup group = a.groups[gi];
        const WRows w = rows_of<BIAS, OUTER>(a.w2, group.expert, n0, 1, a.hidden, K, lane);
        const uint16_t* x[MT];
        int token[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int pair = group.first + 16 * m + col;
            const bool live = 16 * m + col < group.count;
            token[m] = live ? a.pair_token[pair] : -1;
            x[m] = live ? a.mid + (int64_t)pair * K + quarter * 16 : nullptr;
        }
        f32x4_t acc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m] = f32x4_t{0, 0, 0, 0};
        WStep<OUTER> v;
        load_step<BIAS, OUTER>(w, s0 * 128, K, a.w2.obs, quarter, v);
        for (int s = s0; s < s1; ++s) {
            WStep<OUTER> vn;
            load_step<BIAS, OUTER>(w, (s + 1 < s1 ? s + 1 : s) * 128, K, a.w2.obs, quarter, vn);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 w0, w1;
                decode_half<BIAS, OUTER>(v, h, w0, w1);
                const int k = s * 128 + 64 * h;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (16 * m >= group.count) break;
                    const bool in = x[m] != nullptr && k + 16 * quarter < K;
                    const uint4* p = (const uint4*)(x[m] + k);
                    uint4 x0 = in ? p[0] : make_uint4(0, 0, 0, 0), x1 = in ? p[1] : make_uint4(0, 0, 0, 0);
                    multiply_half<OUTER>(v, h, w0, w1, x0, x1, acc[m]);
                    if constexpr (FINE) {
                        const uint4* q = (const uint4*)(a.mid_rest + (x[m] - a.mid) + k);
                        x0 = in ? q[0] : make_uint4(0, 0, 0, 0), x1 = in ? q[1] : make_uint4(0, 0, 0, 0);
                        multiply_half<OUTER>(v, h, w0, w1, x0, x1, acc[m]);
                    }
                }
            }
            v = vn;
        }
        const float whole = a.w2.outer_kind == kOuterTensor ? a.w2.outer[group.expert] : 1.0f;
#pragma unroll
        for (int m = 0; m < MT; ++m)
            if (token[m] >= 0) sums[token[m] * 4 + quarter] += acc[m] * whole;   // a token is once in a group
    }
    __syncthreads();
    for (int i = (int)threadIdx.x; i < a.tokens * 4; i += 64 * kDownWaves) {
        const f32x4_t* p = (const f32x4_t*)smem + i;
        f32x4_t v = p[0];
        for (int w = 1; w < kDownWaves; ++w) v += p[w * a.tokens * 4];
        const int t = i >> 2, n = n0 + 4 * (i & 3);
        if (a.parts) *(f32x4_t*)(a.parts + ((int64_t)blockIdx.y * a.tokens + t) * a.parts_ld + n) = v;
        else store_y4(a, t, n, add_bias(a, t, n, v));
    }
}

// Adds the splits' sums in order: four values of a row a lane.
__global__ __launch_bounds__(256) void k_moe_join(MoeArgs a)
{
    const int quads = (int)(a.parts_ld / 4), at = (int)blockIdx.x * 256 + (int)threadIdx.x;
    if (at >= quads * a.tokens) return;
    const int t = at / quads, n = (at - t * quads) * 4;
    f32x4_t v = {0, 0, 0, 0};
    for (int s = 0; s < a.splits; ++s) v += *(const f32x4_t*)(a.parts + ((int64_t)s * a.tokens + t) * a.parts_ld + n);
    store_y4(a, t, n, add_bias(a, t, n, v));
}

template <int BIAS, int O1, int O2, int MT, bool FINE>
hipError_t launch_products(const MoeArgs& a, hipStream_t s)
{
    const int lds = kDownWaves * a.tokens * 64;
    static OncePerDevice once;
    const hipError_t st = allow_lds(once, reinterpret_cast<const void*>(k_moe_down<BIAS, O2, MT, FINE>),
                                    kDownWaves * kMoeMaxTokens * 64);
    if (st != hipSuccess) return st;
    hipLaunchKernelGGL((k_moe_up<BIAS, O1, MT, FINE>), dim3((uint32_t)(a.inter / 16), (uint32_t)a.max_groups),
                       dim3(64 * kUpWaves), 0, s, a);
    const int tiles = a.hidden / 16;
    hipLaunchKernelGGL((k_moe_down<BIAS, O2, MT, FINE>), dim3((uint32_t)tiles, (uint32_t)a.splits), dim3(64 * kDownWaves), lds, s, a);
    if (a.splits > 1)
        hipLaunchKernelGGL(k_moe_join, dim3((uint32_t)((a.parts_ld / 4 * a.tokens + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int BIAS, int OUTER, bool FINE>
hipError_t launch_tokens(const MoeArgs& a, hipStream_t s)
{
    if (a.tokens <= 16) return launch_products<BIAS, OUTER, OUTER, 1, FINE>(a, s);
    if (a.tokens <= 32) return launch_products<BIAS, OUTER, OUTER, 2, FINE>(a, s);
    return launch_products<BIAS, OUTER, OUTER, 4, FINE>(a, s);
}

template <int BIAS, int OUTER>
hipError_t launch_outer(const MoeArgs& a, hipStream_t s)
{
    return a.y_f32 ? launch_tokens<BIAS, OUTER, true>(a, s) : launch_tokens<BIAS, OUTER, false>(a, s);
}

template <int BIAS>
hipError_t launch_bias(const MoeArgs& a, hipStream_t s)
{
    if constexpr (BIAS != 0) {
        if (a.w1.outer_kind == kOuter2D) return launch_outer<BIAS, kPerTile>(a, s);
        if (a.w1.outer_kind == kOuter1D) return launch_outer<BIAS, kPerRow>(a, s);
    }
    return launch_outer<BIAS, kInnerOnly>(a, s);
}

size_t padded(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

MoePlan plan_moe(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inter)
{
    MoePlan p;
    const int64_t pairs = tokens * top_k;
    // an expert's pairs are at most the tokens
    const int64_t reached = experts < pairs ? experts : pairs, extra = pairs / kGroup;
    p.max_groups = (int32_t)(reached + (tokens > kGroup ? extra : 0));
    // Workgroups of k_moe_down: 16 rows of W2 each; few of them split the groups until they
    // fill the chip once, while each wave keeps four steps.
    const int64_t tiles = hidden / 16, steps = (inter + 127) / 128;
    int64_t splits = 256 / tiles;
    if (splits > p.max_groups * steps / (kDownWaves * 4)) splits = p.max_groups * steps / (kDownWaves * 4);
    p.splits = (int32_t)(splits < 1 ? 1 : splits);
    p.parts_ld = hidden;
    size_t at = 0;
    const auto take = [&at](size_t n) { const size_t here = at; at += padded(n); return here; };
    p.counts = take(16);
    p.groups = take(p.max_groups * sizeof(MoeGroup));
    p.expert = take(pairs * 4);
    p.share = take(pairs * 4);
    p.pair_token = take(pairs * 4);
    p.pair_share = take(pairs * 4);
    p.mid = take(pairs * inter * 2);
    p.mid_rest = take(pairs * inter * 2);
    p.parts = take(p.splits > 1 ? p.splits * tokens * p.parts_ld * 4 : 0);
    p.bytes = at;
    return p;
}

hipError_t launch_moe(int bias, const MoeArgs& a, hipStream_t s)
{
    hipLaunchKernelGGL(k_moe_route, dim3(1), dim3(kRouteThreads), 0, s, a);
    if (bias == 0) return launch_bias<0>(a, s);
    if (bias == 7) return launch_bias<7>(a, s);
    return launch_bias<15>(a, s);
}

}  // namespace fp4q
