// kernels_linear.hip -- y = x W^T with bf16 activations and a 4-bit weight.
//
// Rows of W are the A operand and rows of x the B operand of v_mfma_f32_16x16x32_bf16,
//   y^T[n, m] = sum_k W[n, k] x[m, k],
// 16 of each a product.  A step covers 64 values of K in two products; lane l holds, of row
// l % 16 of either operand, the values 64 s + 16 (l / 16) .. + 15: eight bytes of codes under
// one inner scale, and 32 bytes of x.  W is decoded in registers to bf16, exactly
// (mfma16.h), so the products are exact and the sums binary32.  Where W has outer
// scales per 64 (or more) values of K, the two products of a step start from
// zero and the outer scale multiplies their sum into the accumulator.
//
// Small weights under at most 16 rows of x (k_linear): a workgroup takes 16 rows of W, its eight
// waves every eighth pair of steps, and joins them through LDS in a fixed order.  One row through
// 2880 x 2880 takes 5.2 us, of which a launch and one trip to memory are most.
#include "fp4q_device.h"
#include "launch.h"
#include "lds_load.h"
#include "mfma16.h"

namespace fp4q {

namespace {

#define LDS_PTR(t) __attribute__((address_space(3))) t*

// Outer scales inside the sum: none (or one for the tensor, applied to y), per
// 64 rows (2D) or per row (1D).
enum { kInnerOnly = 0, kPerTile = 1, kPerRow = 2 };

// Values c .. c + 3 of row r of y.
__device__ __forceinline__ void store4(const LinearArgs& a, int64_t r, int c, f32x4_t v)
{
    const int64_t at = r * a.ld_y + c;
    if (a.y_f32) {
        float* y = (float*)a.y + at;
        if (a.y_vec && c + 4 <= a.N) {
            *(f32x4_t*)y = v;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < a.N) y[i] = v[i];
    } else {
        uint16_t* y = (uint16_t*)a.y + at;
        if (a.y_vec && c + 4 <= a.N) {
            *(uint2*)y = make_uint2(Dec<0>::round2(v[0], v[1]), Dec<0>::round2(v[2], v[3]));
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < a.N) y[i] = (uint16_t)Dec<0>::round2(v[i], 0.0f);
    }
}

// Weights that k_linear takes.  Cold weights, 1 and 16 rows, MXFP4 (k_linear / tiles): 2880 x 2880 5.1, 6.2 /
// 9.1, 9.7 us; 4096 x 4096 7.6, 9.9 / 9.5, 10.1; 8192 x 4096 13.2, 17.4 / 10.9, 11.3; 8192 x
// 8192 22.9, 32.0 / 14.8, 14.9.
constexpr int64_t kSmallWeight = (int64_t)1 << 24;
constexpr int kPair = 128;                               // values of K of a pair of steps

// A lane's codes and scale bytes of a pair of steps.
struct WRaw {
    uint2 c[2];
    uint32_t s[2];
};

constexpr int kSmallWaves = 8;

template <int BIAS, int OUTER>
__global__ __launch_bounds__(64 * kSmallWaves) void k_linear(LinearArgs a)
{
    constexpr int B = Dec<BIAS>::kBlock;
    __shared__ float join[kSmallWaves / 2][4][64];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int row = lane & 15, quarter = lane >> 4;
    const int n0 = (int)blockIdx.x * 16;

    // rows of W beyond N repeat the last one; their results are not stored
    const int64_t r0 = min(n0 + row, a.N - 1);
    const uint8_t* const wc = a.codes + r0 * (a.K / 2) + quarter * 8;
    const uint8_t* const ws = a.scales + r0 * (a.K / B) + (B == 16 ? quarter : quarter >> 1);
    const bool live = row < a.M;
    const uint16_t* const xr = a.x + (int64_t)(live ? row : 0) * a.ld_x + quarter * 16;

    // Lanes whose 16 values lie beyond K (K % 64 == 32: half a step; the second step of a last
    // pair) take zeros for both operands.
    auto load_w = [&](int k0, WRaw& w) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k = k0 + 64 * s;
            const bool in = k + 16 * quarter < a.K;
            w.c[s] = in ? *(const uint2*)(wc + k / 2) : make_uint2(0, 0);
            w.s[s] = in ? ws[k / B] : 0;
        }
    };

    f32x4_t acc = {0, 0, 0, 0};
    int k = wave * kPair;
    WRaw cur;
    if (k < a.K) load_w(k, cur);
    for (; k < a.K; k += kSmallWaves * kPair) {
        WRaw nxt;
        load_w(k + kSmallWaves * kPair, nxt);
        uint4 x[2][2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const bool in = live && k + 64 * s + 16 * quarter < a.K;
            const uint4* p = (const uint4*)(xr + k + 64 * s);
            x[s][0] = in ? p[0] : make_uint4(0, 0, 0, 0);
            x[s][1] = in ? p[1] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (OUTER != kInnerOnly && k + 64 * s >= a.K) break;
            const float sc = DecBf16<BIAS>::scale(cur.s[s]);
            const uint4 w0 = DecBf16<BIAS>::octet(cur.c[s].x, sc), w1 = DecBf16<BIAS>::octet(cur.c[s].y, sc);
            f32x4_t so;
            if constexpr (OUTER == kPerTile) {
                const float v = a.outer[(min(n0, a.N - 1) >> 6) * a.outer_n + ((k + 64 * s) >> 6) * a.outer_k];
                so = f32x4_t{v, v, v, v};
            } else if constexpr (OUTER == kPerRow) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    so[r] = a.outer[min(n0 + 4 * quarter + r, a.N - 1) * a.outer_n + (k + 64 * s) / a.obs];
            }
            f32x4_t p = OUTER == kInnerOnly ? acc : f32x4_t{0, 0, 0, 0};
            p = Dec<0>::mfma(w0, x[s][0], p);
            p = Dec<0>::mfma(w1, x[s][1], p);
            if constexpr (OUTER == kInnerOnly) {
                acc = p;
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(p[r], so[r], acc[r]);
            }
        }
        cur = nxt;
    }

    // join the waves: the upper half of those left into the lower half
#pragma unroll
    for (int half = kSmallWaves / 2; half >= 1; half >>= 1) {
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int r = 0; r < 4; ++r) join[wave - half][r][lane] = acc[r];
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] += join[wave][r][lane];
        }
        __syncthreads();
    }
    if (wave != 0 || !live) return;
    store4(a, row, n0 + 4 * quarter, acc * (a.outer_kind == kOuterTensor ? a.outer[0] : 1.0f));
}

// ---------------------------------------------------------------- tiles
// Larger work: a workgroup of eight waves takes 16 MT rows of x and 32 kWN rows of W, S = 256
// values of K (128 with eight tiles of x rows, of whose stages LDS would not hold two) at a time
// through a ring of LDS stages filled by direct loads:
//   x       [16 MT][S] bf16, a row's S / 8 chunks of 16 bytes at chunk ^ (row % 16),
//   codes   [32 kWN][S / 2 bytes], a row's S / 32 chunks at chunk ^ (row & (S / 32 - 2)),
//   scales  [32 kWN][S / 32], a word for 32 values of K (one byte of MXFP4, two of the
//           others: rows of scale bytes have no better alignment, 90 bytes for
//           MXFP4 and K = 2880),
//   outer scales [S / 64][32 kWN] FP32, per 64 values of K.
// Wave w takes W's rows 32 (w % kWN) .. + 31 and the (w / kWN)-th part of the stage's K;
// the parts join through LDS.  Waves 0 to 3, one of each SIMD, issue the loads, and the SIMD's
// other wave computes meanwhile.  So a workgroup reads x from the caches once for
// 32 kWN rows of W, and a row of W is decoded once for 16 MT rows of x: with eight tiles the
// matrix instructions take as long as the decoding.  Few tiles: the stages are split over
// workgroups, whose binary32 sums k_linear_join adds in order.

template <int BIAS, int MT, bool OUTER>
struct Tile {
    static constexpr int B = Dec<BIAS>::kBlock;
    static constexpr int kStageK = MT == 8 ? 128 : 256;
    static constexpr int kWN = 4, kWK = 2;               // waves along W's rows and along K
    static constexpr int kN = 32 * kWN;
    static constexpr int kSteps = kStageK / kWK / 64;    // of 64 values of K, of a wave and stage
    static constexpr int kX = 16 * MT * kStageK * 2, kC = kN * kStageK / 2, kS = kN * kStageK / 8,
                         kO = OUTER ? kN * kStageK / 16 : 0;
    static constexpr int kStage = kX + kC + kS + kO;
    // 16-byte chunks of a row of x and of codes (scale words: half of the codes' chunks' values
    // each, as many), and the loads of a wave and stage
    static constexpr int kXC = kStageK / 8, kCC = kStageK / 32;
    static constexpr int kCX = kCC - 2;                  // the bits of a row that move its chunks
    static constexpr int kXL = 16 * MT * kXC / 256, kCL = kN * kCC / 256;
    // one workgroup fills a compute unit's LDS
    static constexpr int kDepth = 160 * 1024 / kStage < 4 ? 160 * 1024 / kStage : 4;
    static constexpr int kLds = kDepth * kStage;
    static constexpr int kOL = OUTER ? kN * kStageK / 64 / 256 : 0;
    static constexpr int kLoads = kXL + 2 * kCL + kOL;
    static_assert(kDepth >= 2 && kLds >= (kWK - 1) * kWN * MT * 8 * 64 * 4, "two stages; the parts join in their place");
};

template <int BIAS, int MT, bool OUTER>
__global__ __launch_bounds__(512) void k_linear_tile(LinearArgs a)
{
    using T = Tile<BIAS, MT, OUTER>;
    extern __shared__ __align__(16) unsigned char smem[];
    lds_t* const lds = (lds_t*)smem;
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wn = wave % T::kWN, wk = wave / T::kWN;
    const int row = lane & 15, quarter = lane >> 4;
    const int n0 = (int)blockIdx.x * T::kN, m0 = (int)blockIdx.y * (16 * MT);
    const int stages = (a.K + T::kStageK - 1) / T::kStageK;
    const int s0 = (int)((int64_t)stages * blockIdx.z / gridDim.z), s1 = (int)((int64_t)stages * (blockIdx.z + 1) / gridDim.z);

    // Descriptors from the tile's first rows; rows beyond M or N repeat the last one
    // (their results are not stored), values beyond K load as zeros.
    const rsrc_t xr = make_rsrc(a.x + (int64_t)m0 * a.ld_x), cr = make_rsrc(a.codes + (int64_t)n0 * (a.K / 2));
    const rsrc_t sr = make_rsrc(a.scales + (int64_t)n0 * (a.K / T::B));
    const rsrc_t outr = make_rsrc(a.outer);
    const int last_m = a.M - 1 - m0, last_n = a.N - 1 - n0;

    // A lane's offsets within the first stage.  A later stage adds the same to all lanes, so a
    // whole stage takes no lane arithmetic.
    const int xc = lane % T::kXC, cc = lane % T::kCC;
    uint32_t xo[T::kXL], co[T::kCL], ro[T::kCL];
    const auto x_row = [&](int j) { return (wave * T::kXL + j) * (64 / T::kXC) + lane / T::kXC; };
    const auto w_row = [&](int j) { return (wave * T::kCL + j) * (64 / T::kCC) + lane / T::kCC; };
#pragma unroll
    for (int j = 0; j < T::kXL; ++j)
        xo[j] = (uint32_t)(min(x_row(j), last_m) * (int)a.ld_x + 8 * (xc ^ (x_row(j) & 15))) * 2;
#pragma unroll
    for (int j = 0; j < T::kCL; ++j) {
        co[j] = (uint32_t)(min(w_row(j), last_n) * (a.K / 2) + 16 * (cc ^ (w_row(j) & T::kCX)));
        ro[j] = (uint32_t)(min(w_row(j), last_n) * (a.K / T::B) + cc * (32 / T::B));
    }
    auto issue = [&](int s, int slot) {
        const uint32_t to = lds_address(lds + slot * T::kStage);
        const int k0 = s * T::kStageK;
        const bool tail = k0 + T::kStageK > a.K;         // values beyond K load as zeros
#pragma unroll
        for (int j = 0; j < T::kXL; ++j) {
            uint32_t off = xo[j];
            if (tail) off = k0 + 8 * (xc ^ (x_row(j) & 15)) < a.K ? off : kOff;
            lds_load_kept(xr, off, to + (wave * T::kXL + j) * 1024, k0 * 2);
        }
#pragma unroll
        for (int j = 0; j < T::kCL; ++j) {
            const int piece = wave * T::kCL + j;
            uint32_t off = co[j], at = ro[j];
            if (tail) {
                off = k0 + 32 * (cc ^ (w_row(j) & T::kCX)) < a.K ? off : kOff;
                at = k0 + 32 * cc < a.K ? at : kOff;
            }
            lds_load_kept(cr, off, to + T::kX + piece * 1024, k0 / 2);
            if constexpr (T::B == 32) lds_load1(sr, at, to + T::kX + T::kC + piece * 256, k0 / T::B);
            else lds_load2(sr, at, to + T::kX + T::kC + piece * 256, k0 / T::B);
        }
#pragma unroll
        for (int j = 0; j < T::kOL; ++j) {               // outer scales
            const int i = (wave * T::kOL + j) * 64 + lane, r = i % T::kN, k = k0 + 64 * (i / T::kN);
            const int n = min(n0 + r, a.N - 1);
            const uint32_t at = (uint32_t)((a.outer_kind == kOuter2D ? n >> 6 : n) * (int)a.outer_n + k / a.obs * (int)a.outer_k) * 4;
            lds_load4(outr, k < a.K ? at : kOff, to + T::kX + T::kC + T::kS + (wave * T::kOL + j) * 256);
        }
    };

    f32x4_t acc[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = f32x4_t{0, 0, 0, 0};

#pragma unroll
    for (int i = 0; i < T::kDepth - 1; ++i)
        if (wave < 4 && s0 + i < s1) issue(s0 + i, i);
    int slot = 0;
    for (int s = s0; s < s1; ++s) {
        // a loading wave's part of the stage has landed; the barrier makes everybody's visible, and
        // says that the stage before, whose place is filled next, has been read
        if (s + T::kDepth - 2 < s1) wait_loads<(T::kDepth - 2) * T::kLoads>();
        else wait_loads<0>();
        wait_reads();
        lds_barrier();
        const int free = slot == 0 ? T::kDepth - 1 : slot - 1;
        if (wave < 4 && s + T::kDepth - 1 < s1) issue(s + T::kDepth - 1, free);
        const lds_t* const x = lds + slot * T::kStage;
        const lds_t* const c = x + T::kX;
        slot = slot + 1 == T::kDepth ? 0 : slot + 1;

#pragma unroll
        for (int step = 0; step < T::kSteps; ++step) {
            const int part = wk * T::kSteps + step;      // the stage's 64 values of K from 64 part
            // all of the step's reads are issued before its arithmetic: W's first, whose decoding
            // hides the wait for x
            u32x2_t code[2];
            uint32_t byte[2];
            f32x4_t so[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int r = 32 * wn + 16 * n + row;
                const int chunk = (2 * part + (quarter >> 1)) ^ (r & T::kCX);
                code[n] = *(const LDS_PTR(u32x2_t))(c + r * (T::kStageK / 2) + chunk * 16 + (quarter & 1) * 8);
                byte[n] = *(const LDS_PTR(uint32_t))(c + T::kC + (r * T::kCC + 2 * part + (quarter >> 1)) * 4);
                if constexpr (OUTER)
                    so[n] = *(const LDS_PTR(f32x4_t))(c + T::kC + T::kS + (part * T::kN + 32 * wn + 16 * n + 4 * quarter) * 4);
            }
            u32x4_t v[MT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int chunk = (8 * part + 2 * quarter + i) ^ row;
                    v[m][i] = *(const LDS_PTR(u32x4_t))(x + (16 * m + row) * (T::kStageK * 2) + chunk * 16);
                }
            __builtin_amdgcn_sched_barrier(0);
            uint4 w[2][2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                if constexpr (T::B == 16) byte[n] = __builtin_amdgcn_ubfe(byte[n], 8 * (quarter & 1), 8);
                const float sc = DecBf16<BIAS>::scale(byte[n]);
                w[n][0] = DecBf16<BIAS>::octet(code[n][0], sc);
                w[n][1] = DecBf16<BIAS>::octet(code[n][1], sc);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint4 v0 = make_uint4(v[m][0][0], v[m][0][1], v[m][0][2], v[m][0][3]);
                const uint4 v1 = make_uint4(v[m][1][0], v[m][1][1], v[m][1][2], v[m][1][3]);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    f32x4_t p = OUTER ? f32x4_t{0, 0, 0, 0} : acc[m][n];
                    p = Dec<0>::mfma(w[n][0], v0, p);
                    p = Dec<0>::mfma(w[n][1], v1, p);
                    if constexpr (OUTER) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[m][n][r] = __builtin_fmaf(p[r], so[n][r], acc[m][n][r]);
                    } else {
                        acc[m][n] = p;
                    }
                }
            }
        }
    }

    // the parts of K join the first in order
    __syncthreads();
    float* const join = reinterpret_cast<float*>(smem) + lane;
    if (wk > 0) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                join[(((wk - 1) * T::kWN + wn) * (MT * 8) + m * 8 + i) * 64] = acc[m][i >> 2][i & 3];
    }
    __syncthreads();
    if (wk > 0) return;
#pragma unroll 1
    for (int p = 0; p < T::kWK - 1; ++p)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[m][i >> 2][i & 3] += join[((p * T::kWN + wn) * (MT * 8) + m * 8 + i) * 64];

    const float whole = a.outer_kind == kOuterTensor && a.parts == nullptr ? a.outer[0] : 1.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int64_t r = m0 + 16 * m + row;
        if (r >= a.M) continue;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int c = n0 + 32 * wn + 16 * n + 4 * quarter;
            if (a.parts) {
                *(float4*)(a.parts + (blockIdx.z * (int64_t)a.M + r) * a.parts_ld + c) =
                    make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
                continue;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] *= whole;
            store4(a, r, c, acc[m][n]);
        }
    }
}

// Adds the splits' sums in order: four values of a row a lane.
__global__ __launch_bounds__(256) void k_linear_join(LinearArgs a)
{
    const int64_t quads = a.parts_ld / 4;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= quads * a.M) return;
    const int64_t r = at / quads;
    const int c = (int)(at - r * quads) * 4;
    const float* p = a.parts + r * a.parts_ld + c;
    f32x4_t sum = {0, 0, 0, 0};
    for (int s = 0; s < a.splits; ++s) sum += *(const f32x4_t*)(p + s * (int64_t)a.M * a.parts_ld);
    if (a.outer_kind == kOuterTensor) sum *= a.outer[0];
    store4(a, r, c, sum);
}

template <int BIAS, int MT, bool OUTER>
hipError_t launch_tile(const LinearArgs& a, hipStream_t s)
{
    using T = Tile<BIAS, MT, OUTER>;
    static OncePerDevice once;
    const hipError_t st = allow_lds(once, reinterpret_cast<const void*>(k_linear_tile<BIAS, MT, OUTER>), T::kLds);
    if (st != hipSuccess) return st;
    const dim3 grid((uint32_t)((a.N + T::kN - 1) / T::kN), (uint32_t)((a.M + 16 * MT - 1) / (16 * MT)), (uint32_t)a.splits);
    hipLaunchKernelGGL((k_linear_tile<BIAS, MT, OUTER>), grid, dim3(512), T::kLds, s, a);
    if (a.parts) {
        const int64_t quads = a.parts_ld / 4 * a.M;
        hipLaunchKernelGGL(k_linear_join, dim3((uint32_t)((quads + 255) / 256)), dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

template <int BIAS, int OUTER>
hipError_t launch_outer(const LinearArgs& a, hipStream_t s)
{
    if (a.splits == 0) {
        hipLaunchKernelGGL((k_linear<BIAS, OUTER>), dim3((uint32_t)((a.N + 15) / 16)), dim3(64 * kSmallWaves), 0, s, a);
        return hipGetLastError();
    }
    if (a.M <= 16) return launch_tile<BIAS, 1, OUTER != kInnerOnly>(a, s);
    if (a.M <= 32) return launch_tile<BIAS, 2, OUTER != kInnerOnly>(a, s);
    if (a.M <= 48) return launch_tile<BIAS, 3, OUTER != kInnerOnly>(a, s);
    if (a.M <= 64) return launch_tile<BIAS, 4, OUTER != kInnerOnly>(a, s);
    return launch_tile<BIAS, 8, OUTER != kInnerOnly>(a, s);
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

LinearPlan plan_linear(int64_t M, int64_t N, int64_t K)
{
    LinearPlan p{0, 0, 0};
    // small weights under few rows: one launch without parts
    if (M <= 16 && N * K <= kSmallWeight) return p;
    const int64_t rows = M <= 16 ? 16 : M <= 32 ? 32 : M <= 48 ? 48 : M <= 64 ? 64 : 128, cols = 128;
    const int64_t blocks = (N + cols - 1) / cols * ((M + rows - 1) / rows);
    const int64_t stages = (K + 255) / 256;
    int64_t want = 256 / blocks;                         // one workgroup a compute unit
    if (want > stages / 4) want = stages / 4;
    p.splits = want < 1 ? 1 : (int32_t)want;
    if (p.splits > 1) {
        p.ld = (N + cols - 1) / cols * cols;
        p.bytes = (size_t)p.splits * M * p.ld * sizeof(float);
    }
    return p;
}

hipError_t launch_linear(int bias, const LinearArgs& a, hipStream_t s)
{
    if (bias == 0) return launch_bias<0>(a, s);
    if (bias == 7) return launch_bias<7>(a, s);
    return launch_bias<15>(a, s);
}

}  // namespace fp4q
