// kernels_linear.hip -- y = x W^T with bf16 activations and a 4-bit weight.
//
// A wave computes 16 MT rows of y (columns of the product) by 16 NT of its columns, on
// v_mfma_f32_16x16x32_bf16 with W as the A operand (rows) and x as B (columns):
//   y^T[n, m] = sum_k W[n, k] x[m, k].
// A step covers 64 values of K in two products; lane l holds, of row l % 16 of either
// operand, the values 64 s + 16 (l / 16) .. + 15: eight bytes of codes under one
// inner scale, and 32 bytes of x.  W is decoded in registers to bf16, exactly
// (mfma16.h), so the products are exact and the sums binary32.  Where W has outer
// scales per 64 (or more) values of K, the two products of a step start from
// zero and the outer scale multiplies their sum into the accumulator.
//
// The waves of a workgroup share the tile and take every KS-th pair of steps; their sums
// are joined through LDS in a fixed order.
#include "fp4q_device.h"
#include "launch.h"
#include "mfma16.h"

namespace fp4q {

namespace {

// Outer scales inside the sum: none (or one for the tensor, applied to y), per
// 64 rows (2D) or per row (1D).
enum { kInnerOnly = 0, kPerTile = 1, kPerRow = 2 };

constexpr int kPair = 128;                               // values of K of a pair of steps

template <int BIAS, int NT>
struct WRaw {
    uint2 c[NT][2];
    uint32_t s[NT][2];
};

template <int BIAS, int MT, int NT, int OUTER, int KS>
__global__ __launch_bounds__(64 * KS) void k_linear(LinearArgs a)
{
    constexpr int B = Dec<BIAS>::kBlock;
    __shared__ float join[KS / 2][MT * NT * 4][64];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int row = lane & 15, quarter = lane >> 4;
    const int n0 = (int)blockIdx.x * (16 * NT), m0 = (int)blockIdx.y * (16 * MT);

    f32x4_t acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = f32x4_t{0, 0, 0, 0};

    // rows of W beyond N repeat the last one; their results are not stored
    const uint8_t *wc[NT], *ws[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int64_t r = min(n0 + 16 * n + row, a.N - 1);
        wc[n] = a.codes + r * (a.K / 2) + quarter * 8;
        ws[n] = a.scales + r * (a.K / B) + (B == 16 ? quarter : quarter >> 1);
    }
    const uint16_t* xr[MT];
    bool live[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        live[m] = m0 + 16 * m + row < a.M;
        xr[m] = a.x + (int64_t)(live[m] ? m0 + 16 * m + row : 0) * a.ld_x + quarter * 16;
    }

    // Lanes whose 16 values lie beyond K (K % 64 == 32: half a step; the second step of a last
    // pair) take zeros for both operands.
    auto load_w = [&](int k0, WRaw<BIAS, NT>& w) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k = k0 + 64 * s;
            const bool in = k + 16 * quarter < a.K;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                w.c[n][s] = in ? *(const uint2*)(wc[n] + k / 2) : make_uint2(0, 0);
                w.s[n][s] = in ? ws[n][k / B] : 0;
            }
        }
    };

    int k = wave * kPair;
    WRaw<BIAS, NT> cur;
    if (k < a.K) load_w(k, cur);
    for (; k < a.K; k += KS * kPair) {
        WRaw<BIAS, NT> nxt;
        load_w(k + KS * kPair, nxt);
        uint4 x[MT][2][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const bool in = live[m] && k + 64 * s + 16 * quarter < a.K;
                const uint4* p = (const uint4*)(xr[m] + k + 64 * s);
                x[m][s][0] = in ? p[0] : make_uint4(0, 0, 0, 0);
                x[m][s][1] = in ? p[1] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (OUTER != kInnerOnly && k + 64 * s >= a.K) break;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float sc = DecBf16<BIAS>::scale(cur.s[n][s]);
                const uint4 w0 = DecBf16<BIAS>::octet(cur.c[n][s].x, sc), w1 = DecBf16<BIAS>::octet(cur.c[n][s].y, sc);
                f32x4_t so;
                if constexpr (OUTER == kPerTile) {
                    const float v = a.outer[(min(n0 + 16 * n, a.N - 1) >> 6) * a.outer_n + ((k + 64 * s) >> 6) * a.outer_k];
                    so = f32x4_t{v, v, v, v};
                } else if constexpr (OUTER == kPerRow) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        so[r] = a.outer[min(n0 + 16 * n + 4 * quarter + r, a.N - 1) * a.outer_n + (k + 64 * s) / a.obs];
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    f32x4_t p = OUTER == kInnerOnly ? acc[m][n] : f32x4_t{0, 0, 0, 0};
                    p = Dec<0>::mfma(w0, x[m][s][0], p);
                    p = Dec<0>::mfma(w1, x[m][s][1], p);
                    if constexpr (OUTER == kInnerOnly) {
                        acc[m][n] = p;
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[m][n][r] = __builtin_fmaf(p[r], so[r], acc[m][n][r]);
                    }
                }
            }
        }
        cur = nxt;
    }

    // join the waves: the upper half of those left into the lower half
#pragma unroll
    for (int half = KS / 2; half >= 1; half >>= 1) {
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r) join[wave - half][(m * NT + n) * 4 + r][lane] = acc[m][n][r];
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[m][n][r] += join[wave][(m * NT + n) * 4 + r][lane];
        }
        __syncthreads();
    }
    if (wave != 0) return;
    const float whole = a.outer_kind == kOuterTensor ? a.outer[0] : 1.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (!live[m]) continue;
        const int64_t at = (int64_t)(m0 + 16 * m + row) * a.ld_y;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int c = n0 + 16 * n + 4 * quarter + r;
                const float v = acc[m][n][r] * whole;
                if (c >= a.N) continue;
                if (a.y_f32) ((float*)a.y)[at + c] = v;
                else ((uint16_t*)a.y)[at + c] = (uint16_t)f32_to_bf16(v);
            }
    }
}

template <int BIAS, int MT, int NT, int OUTER>
void launch_tile(const LinearArgs& a, hipStream_t s)
{
    constexpr int KS = MT * NT >= 8 ? 4 : 8;
    const dim3 grid((uint32_t)((a.N + 16 * NT - 1) / (16 * NT)), (uint32_t)((a.M + 16 * MT - 1) / (16 * MT)));
    hipLaunchKernelGGL((k_linear<BIAS, MT, NT, OUTER, KS>), grid, dim3(64 * KS), 0, s, a);
}

template <int BIAS, int OUTER>
hipError_t launch_outer(const LinearArgs& a, hipStream_t s)
{
    if (a.M <= 16) launch_tile<BIAS, 1, 1, OUTER>(a, s);
    else if (a.M <= 32) launch_tile<BIAS, 2, 2, OUTER>(a, s);
    else launch_tile<BIAS, 4, 2, OUTER>(a, s);
    return hipGetLastError();
}

template <int BIAS>
hipError_t launch_bias(const LinearArgs& a, hipStream_t s)
{
    if constexpr (BIAS != 0) {
        if (a.outer_kind == kOuter2D) return launch_outer<BIAS, kPerTile>(a, s);
        if (a.outer_kind == kOuter1D) return launch_outer<BIAS, kPerRow>(a, s);
    }
    return launch_outer<BIAS, kInnerOnly>(a, s);
}

}  // namespace

hipError_t launch_linear(int bias, const LinearArgs& a, hipStream_t s)
{
    if (bias == 0) return launch_bias<0>(a, s);
    if (bias == 7) return launch_bias<7>(a, s);
    return launch_bias<15>(a, s);
}

}  // namespace fp4q
