// kernels_norm.hip -- the residual's addition, the root-mean-square norm, its
// output in 8 bits with scales, and the norm's gradient.
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = (h r) w
//   n = h r,  g = dy w,  dx = r (g - n mean(n g)) + dresidual,  dw = sum over rows of dy n
//
// Rounding.  h is rounded to the residual's type, and the norm is of what is stored, so
// that the gradient, which reads it, is the gradient of what was computed.  The sum of
// squares is binary64 (its terms are exact there), so r is the rounded value
// whatever the order of the sum, and y = RN(RN(h r) w) and its codes do not depend on how a
// row is shared among lanes.  Two vector instructions a value, about 2 of the 40 us of 8192 rows of
// 2880.
//
// Both kernels move bytes.  A row's values stay in the registers of its lanes
// between the sums and the outputs: 8 neighbouring values a chunk, C chunks a
// lane, W waves a row.  Four neighbouring lanes hold a block of 32 values.
#include "fp4q_device.h"
#include "launch.h"
#include "mfma16.h"

namespace fp4q {

namespace {

template <int W>
constexpr int kRowThreads = W < 4 ? 256 : 64 * W;
template <int W>
constexpr int kGradThreads = W < 16 ? 512 : 64 * W;

// Eight values from memory, bf16 or FP32 (16-byte aligned).
template <bool F32>
struct Chunk {
    uint4 w[F32 ? 2 : 1];

    __device__ __forceinline__ void load(const void* p, int64_t at)
    {
        const char* q = (const char*)p + at * (F32 ? 4 : 2);
        w[0] = ld_nt16(q);
        if constexpr (F32) w[1] = ld_nt16(q + 16);
    }

    __device__ __forceinline__ void clear()
    {
        w[0] = make_uint4(0, 0, 0, 0);
        if constexpr (F32) w[1] = w[0];
    }

    __device__ __forceinline__ void values(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (F32) {
                    v[4 * i + j] = __uint_as_float(u[j]);
                } else {
                    v[2 * j] = bf16_lo(u[j]);
                    v[2 * j + 1] = bf16_hi(u[j]);
                }
            }
        }
    }
};

__device__ __forceinline__ void store8(void* p, bool f32, int64_t at, const float (&v)[8])
{
    if (f32) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            st_nt16((float*)p + at + 4 * i, make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                                       __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])));
    } else {
        st_nt16((uint16_t*)p + at, make_uint4(Dec<0>::round2(v[0], v[1]), Dec<0>::round2(v[2], v[3]),
                                              Dec<0>::round2(v[4], v[5]), Dec<0>::round2(v[6], v[7])));
    }
}

// The weight's eight values from column `at` (read again by every row, so through the caches).
__device__ __forceinline__ void load_weight(const void* w, bool f32, int at, float (&v)[8])
{
    if (f32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 u = ((const float4*)((const float*)w + at))[i];
            v[4 * i] = u.x, v[4 * i + 1] = u.y, v[4 * i + 2] = u.z, v[4 * i + 3] = u.w;
        }
    } else {
        const uint4 u = *(const uint4*)((const uint16_t*)w + at);
        const uint32_t b[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[2 * j] = bf16_lo(b[j]), v[2 * j + 1] = bf16_hi(b[j]);
    }
}

// The sum over the lanes of a row's W waves, in all of them.  slots: W places of the row in LDS
// that no other sum of the row uses before the next barrier.
template <int W, class T>
__device__ __forceinline__ T row_sum(T v, T* slots, int wave)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) slots[wave] = v;
        __syncthreads();
        v = slots[0];
#pragma unroll
        for (int i = 1; i < W; ++i) v += slots[i];
    }
    return v;
}

template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* slots, int wave)
{
    v = wave_max_u32(v);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) slots[wave] = v;
        __syncthreads();
        v = slots[0];
#pragma unroll
        for (int i = 1; i < W; ++i) v = max(v, slots[i]);
    }
    return v;
}

// Bits of the largest finite magnitude.
__device__ __forceinline__ uint32_t finite_bits(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        m = max(m, b < 0x7F800000u ? b : 0u);
    }
    return m;
}

typedef short s16x2_t __attribute__((ext_vector_type(2)));

// E4M3 codes of v / s (s a power of two), RNE, at most 448 in magnitude; NaN stays NaN.
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float s)
{
    const float top = 448.0f * s;
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = v[i] > top ? top : v[i] < -top ? -top : v[i];
    s16x2_t a = {0, 0}, b = {0, 0};
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, c[0], c[1], s, false);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, c[2], c[3], s, true);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, c[4], c[5], s, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, c[6], c[7], s, true);
    return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
}

template <int W, int C, bool XF32, bool RF32>
__global__ __launch_bounds__(kRowThreads<W>) void k_add_rms_norm(NormArgs a)
{
    constexpr int kRows = kRowThreads<W> / (64 * W);     // of a workgroup
    __shared__ double sums[kRowThreads<W> / 64];
    __shared__ uint32_t tops[kRowThreads<W> / 64];
    const int wave = (int)threadIdx.x >> 6, in_row = wave % W, first = wave - in_row;
    const int t = in_row * 64 + ((int)threadIdx.x & 63);
    const int64_t row = (int64_t)blockIdx.x * kRows + wave / W;
    if (row >= a.rows) return;                           // whole waves; with W > 1 the whole workgroup
    const int n = (int)(a.hidden >> 3);
    const char* const x = (const char*)a.x + row * a.ld_x * (XF32 ? 4 : 2);
    const char* const r = (const char*)a.residual + row * a.ld_r * (RF32 ? 4 : 2);

    Chunk<XF32> xc[C];
    Chunk<RF32> rc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = c * 64 * W + t;
        if (at < n) xc[c].load(x, 8 * at);
        else xc[c].clear();
        if (a.residual && at < n) rc[c].load(r, 8 * at);
        else rc[c].clear();
    }
    float h[C][8];
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = c * 64 * W + t;
        float rv[8];
        xc[c].values(h[c]);
        if (a.residual) {
            rc[c].values(rv);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] += rv[i];
            if constexpr (!RF32) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const uint32_t u = Dec<0>::round2(h[c][i], h[c][i + 1]);
                    h[c][i] = bf16_lo(u), h[c][i + 1] = bf16_hi(u);
                }
            }
            if (at < n) store8(a.residual_out, RF32, row * a.hidden + 8 * at, h[c]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)h[c][i], (double)h[c][i], sum);
    }
    sum = row_sum<W>(sum, sums + first, in_row);
    const float rstd = (float)(1.0 / sqrt(sum / (double)a.hidden + a.eps));
    if (t == 0 && a.rstd) a.rstd[row] = rstd;

    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = c * 64 * W + t;
        float w[8];
        if (at < n) load_weight(a.weight, a.w_f32, 8 * at, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] = at < n ? h[c][i] * rstd * w[i] : 0.0f;
        if (a.y && at < n) store8(a.y, a.y_f32, row * a.hidden + 8 * at, h[c]);
        if (a.fp8_mode == kFp8Mx) {
            // 2^E, E = floor(log2 amax) - 8 within [-127, 127]
            const uint32_t e = quad_max_u32(finite_bits(h[c]), 4) >> 23;
            const uint32_t byte = e > 8 ? e - 8 : 0;
            if (at < n) {
                st_nt64(a.fp8 + row * a.hidden + 8 * at, e4m3x8(h[c], byte ? __uint_as_float(byte << 23) : 0x1p-127f));
                if ((t & 3) == 0) ((uint8_t*)a.fp8_scales)[row * (a.hidden >> 5) + (at >> 2)] = (uint8_t)byte;
            }
        } else if (a.fp8_mode == kFp8Row) {
            top = max(top, finite_bits(h[c]));
        }
    }
    if (a.fp8_mode != kFp8Row) return;
    const float scale = __uint_as_float(row_max<W>(top, tops + first, in_row)) / 448.0f;
    if (t == 0) ((float*)a.fp8_scales)[row] = scale;
    // the rounded quotients (a subnormal one is 0 as a code either way)
    const double inv = scale == 0.0f ? 0.0 : 1.0 / (double)scale;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = c * 64 * W + t;
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = div_inv64(h[c][i], inv);
        if (at < n) st_nt64(a.fp8 + row * a.hidden + 8 * at, e4m3x8(q, 1.0f));
    }
}

// A lane's part of a row on its way.
template <int C, bool YF32, bool HF32>
struct GradRow {
    Chunk<YF32> y[C];
    Chunk<HF32> h[C], r[C];
    float rstd;

    // A row beyond the last is zeros.
    __device__ __forceinline__ void load(const NormGradArgs& a, int64_t row, int t, int stride)
    {
        const int n = row < a.rows ? (int)(a.hidden >> 3) : 0;
        const char* const dyr = (const char*)a.dy + row * a.ld_dy * (YF32 ? 4 : 2);
        const char* const hr = (const char*)a.h + row * a.ld_h * (HF32 ? 4 : 2);
        const char* const dr = (const char*)a.dres + row * a.ld_dres * (HF32 ? 4 : 2);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = c * stride + t;
            if (at < n) y[c].load(dyr, 8 * at), h[c].load(hr, 8 * at);
            else y[c].clear(), h[c].clear();
            if (a.dres && at < n) r[c].load(dr, 8 * at);
            else r[c].clear();
        }
        rstd = row < a.rows ? a.rstd[row] : 0.0f;
    }
};

// Every workgroup takes rows blockIdx.x, + gridDim.x, ... (times the rows it holds at
// once), the next one on its way while one is used, and keeps the sums of dy n of its lanes'
// columns in registers; they join through LDS, then over the workgroups in k_norm_join.  The weight lies in LDS: its
// registers hold the next row.  8192 rows of 2880 in bf16 (189 MB): 35 us and k_norm_join 4; a wave a row
// with the weight in registers and nothing ahead 45, the weight in LDS 39, and the next row's registers spill (76).
template <int W, int C, bool YF32, bool HF32>
__global__ __launch_bounds__(kGradThreads<W>) void k_rms_norm_backward(NormGradArgs a)
{
    constexpr int kRows = kGradThreads<W> / (64 * W);
    constexpr bool kAhead = W < 16;                      // with 16 waves there are no registers for it
    __shared__ float sums[2][kGradThreads<W> / 64];
    // the weight, then the sums' join (W < 16)
    constexpr bool kShared = W < 16;
    __shared__ __align__(16) float lds[kShared ? 8 * C * 64 * W : 1];
    const int wave = (int)threadIdx.x >> 6, in_row = wave % W, first = wave - in_row;
    const int t = in_row * 64 + ((int)threadIdx.x & 63);
    const int n = (int)(a.hidden >> 3);
    const float inv_n = 1.0f / (float)a.hidden;
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + wave / W;
    using Row = GradRow<C, YF32, HF32>;
    Row now;
    if constexpr (kAhead) now.load(a, row, t, 64 * W);
    float w[kShared ? 1 : C][8], dw[C][8];
    const auto weight = [&](int c, float (&v)[8]) {
        if constexpr (kShared) {                         // two reads of 16 bytes: lanes side by side
            const float4 lo = *(const float4*)(lds + 2 * c * 256 * W + t * 4), hi = *(const float4*)(lds + (2 * c + 1) * 256 * W + t * 4);
            v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = w[c][i];
        }
    };
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = c * 64 * W + t;
        float v[8] = {};
        if (at < n) load_weight(a.weight, a.w_f32, 8 * at, v);
        if constexpr (kShared) {
            if (wave / W == c % kRows) {
                *(float4*)(lds + 2 * c * 256 * W + t * 4) = make_float4(v[0], v[1], v[2], v[3]);
                *(float4*)(lds + (2 * c + 1) * 256 * W + t * 4) = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dw[c][i] = 0.0f;
            if constexpr (!kShared) w[c][i] = v[i];
        }
    }
    if constexpr (kShared) __syncthreads();
    int turn = 0;
    // all of a workgroup's waves take as many turns, for their barriers
    for (int64_t head = (int64_t)blockIdx.x * kRows; head < a.rows; head += step, row += step, turn ^= 1) {
        Row next;
        if constexpr (kAhead) next.load(a, row + step, t, 64 * W);
        else now.load(a, row, t, 64 * W);
        const float rstd = now.rstd;
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float dy[8], h[8], wc[8];
            now.y[c].values(dy);
            now.h[c].values(h);
            weight(c, wc);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float nv = h[i] * rstd;
                dw[c][i] = __builtin_fmaf(dy[i], nv, dw[c][i]);
                s = __builtin_fmaf(dy[i] * wc[i], nv, s);
            }
        }
        // two turns' sums have places of their own: a wave that is a row ahead writes others
        s = row_sum<W>(s, sums[turn] + first, in_row) * inv_n;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = c * 64 * W + t;
            float dy[8], h[8], d[8], wc[8];
            now.y[c].values(dy);
            now.h[c].values(h);
            now.r[c].values(d);
            weight(c, wc);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] += rstd * (dy[i] * wc[i] - h[i] * rstd * s);
            if (row < a.rows && at < n) store8(a.dx, HF32, row * a.hidden + 8 * at, d);
        }
        if constexpr (kAhead) now = next;
    }
    if (!a.dw) return;
    float* const out = a.parts ? a.parts + (int64_t)blockIdx.x * a.hidden : a.dw;
    if constexpr (kRows > 1) {                           // wave after wave adds its sums, in order
        for (int p = 1; p < kRows; ++p) {
            __syncthreads();                             // every wave is done with its rows, or with the wave before
            if (wave / W == p) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    *(float4*)(lds + 2 * c * 256 * W + t * 4) = make_float4(dw[c][0], dw[c][1], dw[c][2], dw[c][3]);
                    *(float4*)(lds + (2 * c + 1) * 256 * W + t * 4) = make_float4(dw[c][4], dw[c][5], dw[c][6], dw[c][7]);
                }
            }
            __syncthreads();
            if (wave < W) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float v[8];
                    weight(c, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dw[c][i] += v[i];
                }
            }
        }
        if (wave >= W) return;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = c * 64 * W + t;
        if (at >= n) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *(float4*)(out + 8 * at + 4 * i) = make_float4(dw[c][4 * i], dw[c][4 * i + 1], dw[c][4 * i + 2], dw[c][4 * i + 3]);
    }
}

// The weight's gradient from the workgroups' sums: 16 columns a workgroup, whose 64 groups of
// lanes take every 64th part, in binary64 and in a fixed order.
__global__ __launch_bounds__(1024) void k_norm_join(const float* parts, int count, int64_t hidden, float* dw)
{
    __shared__ double part[64][16];
    const int lane = (int)threadIdx.x & 15, group = (int)threadIdx.x >> 4;
    const int64_t col = (int64_t)blockIdx.x * 16 + lane;
    double s = 0.0;
    if (col < hidden)
        for (int p = group; p < count; p += 256) {       // four loads on their way
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = p + 64 * i < count ? parts[(p + 64 * i) * hidden + col] : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) s += (double)v[i];
        }
    part[group][lane] = s;
    __syncthreads();
    if (group >= 4) return;
    s = part[group][lane];                               // one wave: groups 4 apart, then its four rows of lanes
#pragma unroll
    for (int p = 1; p < 16; ++p) s += part[4 * p + group][lane];
    s += __shfl_xor(s, 16, 64);
    s += __shfl_xor(s, 32, 64);
    if (group == 0 && col < hidden) dw[col] = (float)s;
}

// Waves of a row.  Forward one while rows are many and a lane can hold its chunks (8); backward two while rows are
// many and a lane can hold three chunks of this row and three of the next; more where few rows
// would leave lanes idle.
int fwd_waves(int64_t rows, int64_t hidden) { return rows >= 1024 && hidden / 8 <= 64 * 8 ? 1 : 4; }
int bwd_waves(int64_t rows, int64_t hidden) { return hidden / 8 > 512 * 2 ? 16 : rows >= 1024 && hidden / 8 <= 128 * 3 ? 2 : 8; }

int chunks_of(int64_t hidden, int waves) { return (int)((hidden / 8 + 64 * waves - 1) / (64 * waves)); }

template <int W, int C>
void launch_fwd(const NormArgs& a, hipStream_t s)
{
    constexpr int rows = kRowThreads<W> / (64 * W);
    const dim3 grid((uint32_t)((a.rows + rows - 1) / rows)), block(kRowThreads<W>);
    if (a.x_f32 && a.r_f32) hipLaunchKernelGGL((k_add_rms_norm<W, C, true, true>), grid, block, 0, s, a);
    else if (a.x_f32) hipLaunchKernelGGL((k_add_rms_norm<W, C, true, false>), grid, block, 0, s, a);
    else if (a.r_f32) hipLaunchKernelGGL((k_add_rms_norm<W, C, false, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_add_rms_norm<W, C, false, false>), grid, block, 0, s, a);
}

template <int W, int C>
void launch_bwd(const NormGradArgs& a, hipStream_t s)
{
    const dim3 grid((uint32_t)a.groups), block(kGradThreads<W>);
    if (a.dy_f32 && a.h_f32) hipLaunchKernelGGL((k_rms_norm_backward<W, C, true, true>), grid, block, 0, s, a);
    else if (a.dy_f32) hipLaunchKernelGGL((k_rms_norm_backward<W, C, true, false>), grid, block, 0, s, a);
    else if (a.h_f32) hipLaunchKernelGGL((k_rms_norm_backward<W, C, false, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_rms_norm_backward<W, C, false, false>), grid, block, 0, s, a);
}

}  // namespace

hipError_t launch_add_rms_norm(const NormArgs& a, hipStream_t s)
{
    const int waves = fwd_waves(a.rows, a.hidden), chunks = chunks_of(a.hidden, waves);
    if (waves == 1) {
        if (chunks <= 2) launch_fwd<1, 2>(a, s);
        else if (chunks <= 4) launch_fwd<1, 4>(a, s);
        else if (chunks <= 6) launch_fwd<1, 6>(a, s);
        else launch_fwd<1, 8>(a, s);
    } else {
        if (chunks <= 1) launch_fwd<4, 1>(a, s);
        else if (chunks <= 2) launch_fwd<4, 2>(a, s);
        else if (chunks <= 4) launch_fwd<4, 4>(a, s);
        else launch_fwd<4, 8>(a, s);
    }
    return hipGetLastError();
}

NormGradPlan plan_rms_norm_backward(int64_t rows, int64_t hidden)
{
    const int waves = bwd_waves(rows, hidden);
    const int64_t at_once = waves == 2 ? 4 : 1, need = (rows + at_once - 1) / at_once;
    // one workgroup a compute unit: two leave twice the sums to join, and are not faster (4096 rows of 8192, both
    // kernels: 52.5 us, with two 56)
    const int64_t most = 256;
    NormGradPlan p;
    p.groups = (int32_t)(need < 1 ? 1 : need < most ? need : most);
    p.bytes = p.groups > 1 ? (size_t)p.groups * hidden * sizeof(float) : 0;
    return p;
}

hipError_t launch_rms_norm_backward(const NormGradArgs& a, hipStream_t s)
{
    const int waves = bwd_waves(a.rows, a.hidden), chunks = chunks_of(a.hidden, waves);
    if (waves == 2) {
        if (chunks <= 2) launch_bwd<2, 2>(a, s);
        else launch_bwd<2, 3>(a, s);
    } else if (waves == 8) {
        if (chunks <= 1) launch_bwd<8, 1>(a, s);
        else launch_bwd<8, 2>(a, s);
    } else {
        launch_bwd<16, 2>(a, s);
    }
    if (a.parts && a.dw)
        hipLaunchKernelGGL(k_norm_join, dim3((uint32_t)((a.hidden + 15) / 16)), dim3(1024), 0, s, a.parts, a.groups,
                           a.hidden, a.dw);
    return hipGetLastError();
}

}  // namespace fp4q
