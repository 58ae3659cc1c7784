// kernels_kv.hip -- writing rows of keys and values into the paged 4-bit cache
// and reading them back.
//
// Write: each row of head_dim values of one token and head is quantised as a
// row of fp4_quantize is (NVFP4 / AMD-FP4 with or without a given FP32 scale
// per head, MXFP4), RNE, and its codes and scale bytes go to the row of the
// token's slot.  Read: w = RN(+-G[m] d [s_h]), rounded once more to bf16 where
// that is the target.
//
// Both move bytes: 2 per value on the 16-bit side and 1/2 + 1/block on the
// cache's.  A workgroup of the writer takes one head and a run of tokens, so what it
// writes is contiguous while the tokens' slots are (a page's rows of a head are):
// 32768 tokens of 8 x 128 (170 MB, MXFP4) 36 us, 4.7 TB/s; all heads of the same
// tokens side by side took 39.
#include "fp4q_device.h"
#include "kv_index.h"
#include "launch.h"
#include "mfma16.h"
#include "nv_block.h"

namespace fp4q {

namespace {

constexpr int kThreads = 256;
constexpr int kReadHeads = 4;                            // neighbouring heads of a token that a lane of the reader takes

// Scale exponent of an MXFP4 block from the binary32 bits of its largest
// magnitude: the least k with amax <= 6 2^k, within [-126, 125].
__device__ __forceinline__ int mx_block_exponent(uint32_t abits)
{
    const int e = (int)(abits >> 23);
    int k = e - 129 + (int)((abits & 0x7FFFFFu) > 0x400000u);
    k = e == 0 ? -126 : k;
    return min(max(k, -126), 125);
}

// 16 values of a lane, from bf16 or FP32 (16-byte aligned).
template <bool XF32>
__device__ __forceinline__ void load16(const void* p, float (&v)[16])
{
    constexpr int N = XF32 ? 4 : 2;
    uint4 w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = ld_nt16((const char*)p + 16 * i);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (XF32) {
                v[4 * i + j] = __uint_as_float(u[j]);
            } else {
                v[8 * i + 2 * j] = bf16_lo(u[j]);
                v[8 * i + 2 * j + 1] = bf16_hi(u[j]);
            }
        }
    }
}

// One lane quantises 16 values: a whole NVFP4 / AMD-FP4 block, or half of an
// MXFP4 block whose other half is its neighbour's.  BIAS 0 is MXFP4.
template <int BIAS, bool XF32>
__global__ __launch_bounds__(kThreads) void k_kv_append(KvAppendArgs a)
{
    __shared__ double recip[kRecipTableSize];
    __shared__ float2 rne[BIAS == 0 ? 1 : kRneTableSize];
    if constexpr (BIAS != 0) {
        fill_recip_table(recip, (int)threadIdx.x);
        fill_rne_table<BIAS>(rne, (int)threadIdx.x);
        __syncthreads();
    }
    const int lanes = a.kv.dim >> 4;                       // lanes of a row: 4, 8 or 16
    const int head = (int)blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const int64_t token = (int64_t)blockIdx.x * (kThreads / lanes) + (int)threadIdx.x / lanes;
    const int part = (int)threadIdx.x % lanes;
    if (token >= a.tokens) return;                         // whole rows leave together
    const int64_t row = kv_row_of_slot(a.slots[token], a.num_slots, a.per_page, a.kv.heads, head);
    if (row < 0) return;
    const char* x = (const char*)(is_v ? a.v : a.k);
    const int64_t ld = is_v ? a.ld_v : a.ld_k;
    float v[16];
    load16<XF32>(x + (token * ld + (int64_t)head * a.kv.dim + part * 16) * (XF32 ? 4 : 2), v);
    uint2 code;
    uint32_t scale;
    if constexpr (BIAS == 0) {
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        am = quad_max_u32(am, 2);
        const bool poisoned = am >= 0x7F800000u;           // an infinity or a NaN poisons its block
        const int k = mx_block_exponent(am);
        const float s = __uint_as_float((uint32_t)(127 + k) << 23);
        code.x = code.y = 0;
        code.x = fp4x2_rne_scaled<0>(code.x, v[0], v[1], s);
        code.x = fp4x2_rne_scaled<1>(code.x, v[2], v[3], s);
        code.x = fp4x2_rne_scaled<2>(code.x, v[4], v[5], s);
        code.x = fp4x2_rne_scaled<3>(code.x, v[6], v[7], s);
        code.y = fp4x2_rne_scaled<0>(code.y, v[8], v[9], s);
        code.y = fp4x2_rne_scaled<1>(code.y, v[10], v[11], s);
        code.y = fp4x2_rne_scaled<2>(code.y, v[12], v[13], s);
        code.y = fp4x2_rne_scaled<3>(code.y, v[14], v[15], s);
        scale = (uint32_t)(k + 127);
        if (poisoned) {
            code = make_uint2(0, 0);
            scale = 0xFFu;
        }
    } else {
        const float* outer = is_v ? a.kv.v_outer : a.kv.k_outer;
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = sanitize(v[i]);
        if (outer) {
            const float s_o = outer[head];
            const double inv = s_o == 0.0f ? 0.0 : 1.0 / (double)s_o;
            float vn[16];
            normalize16<false, true>(v, s_o, inv, vn);     // RNE codes need no subnormal quotients
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = vn[i];
        }
        const BlockScale<BIAS> s = block_scale<BIAS>(max_abs16(v), recip);
        code = codes16_rne(v, rne[s.code]);
        scale = s.code;
    }
    uint8_t* codes = is_v ? a.kv.v_codes : a.kv.k_codes;
    uint8_t* scales = is_v ? a.kv.v_scales : a.kv.k_scales;
    *(uint2*)(codes + row * (a.kv.dim / 2) + part * 8) = code;
    if constexpr (BIAS == 0) {
        if ((part & 1) == 0) scales[row * (a.kv.dim / 32) + part / 2] = (uint8_t)scale;
    } else {
        scales[row * (a.kv.dim / 16) + part] = (uint8_t)scale;
    }
}

// Eight values a lane, so that a store of the wave writes whole rows of bf16, of four heads of a
// token.  Measured: 131072 rows of 8 x 128 (689 MB, AMD-FP4) 140 us, 4.9 TB/s; the rows that 32768
// tokens just wrote (MXFP4) 26 us.  Sixteen values a lane write half lines with each store: 133
// and 43 us (non-temporal), 141 and 28 us (ordinary stores).
template <int BIAS, bool YF32>
__global__ __launch_bounds__(kThreads) void k_kv_read(KvReadArgs a)
{
    const int lanes = a.kv.dim >> 3;
    // neighbouring workgroups take all heads of the same tokens
    const uint32_t groups = (uint32_t)(a.kv.heads + kReadHeads - 1) / kReadHeads;
    const uint32_t run = blockIdx.x / groups;
    const int head0 = (int)(blockIdx.x - run * groups) * kReadHeads;
    const bool is_v = blockIdx.y != 0;
    const int64_t token = (int64_t)run * (kThreads / lanes) + (int)threadIdx.x / lanes;
    const int part = (int)threadIdx.x % lanes;
    if (token >= a.tokens) return;
    const uint8_t* codes = is_v ? a.kv.v_codes : a.kv.k_codes;
    const uint8_t* scales = is_v ? a.kv.v_scales : a.kv.k_scales;
    const float* outer = is_v ? a.kv.v_outer : a.kv.k_outer;
    constexpr int kBlock = BIAS == 0 ? 32 : 16;
    const int64_t row = kv_row_of_slot(a.slots[token], a.num_slots, a.per_page, a.kv.heads, head0);
    uint32_t c[kReadHeads], sb[kReadHeads];
#pragma unroll
    for (int u = 0; u < kReadHeads; ++u) {               // rows that are not there read as zeros
        const bool in = row >= 0 && head0 + u < a.kv.heads;
        const int64_t r = row + (int64_t)u * a.kv.page_size;
        c[u] = in ? *(const uint32_t*)(codes + r * (a.kv.dim / 2) + part * 4) : 0;
        sb[u] = in ? scales[r * (a.kv.dim / kBlock) + part * 8 / kBlock] : 0;
    }
#pragma unroll
    for (int u = 0; u < kReadHeads; ++u) {
        const int head = head0 + u;
        if (head >= a.kv.heads) return;
        float d, y[8];
        if constexpr (BIAS == 0) d = sb[u] == 0 ? 0x1p-127f : __uint_as_float(sb[u] << 23);
        else d = DecBf16<BIAS>::scale(sb[u]);
        decode_byte<0>(c[u], d, y[0], y[1]);
        decode_byte<1>(c[u], d, y[2], y[3]);
        decode_byte<2>(c[u], d, y[4], y[5]);
        decode_byte<3>(c[u], d, y[6], y[7]);
        if (BIAS != 0 && outer) {
            const float s_o = outer[head];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] *= s_o;
        }
        if (BIAS == 0 && sb[u] == 0xFFu) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(0x7FC00000u);
        }
        const int64_t at = (token * a.kv.heads + head) * a.kv.dim + part * 8;
        if (YF32) {
            float* o = (float*)(is_v ? a.v : a.k) + at;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                st_nt16(o + 4 * i, make_uint4(__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]),
                                              __float_as_uint(y[4 * i + 2]), __float_as_uint(y[4 * i + 3])));
        } else {
            st_nt16((uint16_t*)(is_v ? a.v : a.k) + at,
                    make_uint4(Dec<0>::round2(y[0], y[1]), Dec<0>::round2(y[2], y[3]), Dec<0>::round2(y[4], y[5]),
                               Dec<0>::round2(y[6], y[7])));
        }
    }
}

}  // namespace

hipError_t launch_kv_append(int bias, bool x_f32, const KvAppendArgs& a, hipStream_t s)
{
    const int rows = kThreads / (a.kv.dim / 16);
    const dim3 grid((uint32_t)((a.tokens + rows - 1) / rows), (uint32_t)a.kv.heads, 2);
#define FP4Q_APPEND(B)                                                                                  \
    do {                                                                                                \
        if (x_f32) hipLaunchKernelGGL((k_kv_append<B, true>), grid, dim3(kThreads), 0, s, a);           \
        else hipLaunchKernelGGL((k_kv_append<B, false>), grid, dim3(kThreads), 0, s, a);                \
    } while (0)
    if (bias == 0) FP4Q_APPEND(0);
    else if (bias == 7) FP4Q_APPEND(7);
    else FP4Q_APPEND(15);
#undef FP4Q_APPEND
    return hipGetLastError();
}

hipError_t launch_kv_read(int bias, bool y_f32, const KvReadArgs& a, hipStream_t s)
{
    const int rows = kThreads / (a.kv.dim / 8), groups = (a.kv.heads + kReadHeads - 1) / kReadHeads;
    const dim3 grid((uint32_t)((a.tokens + rows - 1) / rows * groups), 2);
#define FP4Q_READ(B)                                                                                    \
    do {                                                                                                \
        if (y_f32) hipLaunchKernelGGL((k_kv_read<B, true>), grid, dim3(kThreads), 0, s, a);             \
        else hipLaunchKernelGGL((k_kv_read<B, false>), grid, dim3(kThreads), 0, s, a);                  \
    } while (0)
    if (bias == 0) FP4Q_READ(0);
    else if (bias == 7) FP4Q_READ(7);
    else FP4Q_READ(15);
#undef FP4Q_READ
    return hipGetLastError();
}

}  // namespace fp4q
