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

// Quantises a lane's 16 values of a row of K or V and writes their codes and scale bytes: a
// whole NVFP4 / AMD-FP4 block, or half of an MXFP4 block whose other half is its
// neighbour's.
template <int BIAS>
__device__ __forceinline__ void quantise_row16(const KvView& kv, bool is_v, int head, int part, int64_t row,
                                               float (&v)[16], const double* recip, const float2* rne)
{
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
        const float* outer = is_v ? kv.v_outer : kv.k_outer;
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
    uint8_t* codes = is_v ? kv.v_codes : kv.k_codes;
    uint8_t* scales = is_v ? kv.v_scales : kv.k_scales;
    *(uint2*)(codes + row * (kv.dim / 2) + part * 8) = code;
    if constexpr (BIAS == 0) {
        if ((part & 1) == 0) scales[row * (kv.dim / 32) + part / 2] = (uint8_t)scale;
    } else {
        scales[row * (kv.dim / 16) + part] = (uint8_t)scale;
    }
}

// BIAS 0 is MXFP4.
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
    quantise_row16<BIAS>(a.kv, is_v, head, part, row, v, recip, rne);
}

// Rotation of a lane's 16 values of a row by its token's angles, then as above.
//
// A pair (a, b) of the first rot_dim values turns into (a c - b s, b c + a s), each product,
// sum and difference rounded to binary32: value j and j + rot_dim / 2, or 2 j and 2 j + 1
// (interleaved), with c and s at place j of the token's row of the tables.  rot_dim is a multiple
// of 16, so a chunk of eight values lies in one half, or beyond; where its partners are
// another chunk, the lane of q gets them from the lane that holds them, and a lane of K, whose two chunks
// need not have theirs in one lane, loads that one too (from the caches, where its own lane's load
// brings it).
template <bool XF32>
struct Chunk {
    uint4 w[XF32 ? 2 : 1];

    __device__ __forceinline__ void load(const void* p, int64_t at)
    {
        const uint4* const q = (const uint4*)((const char*)p + at * (XF32 ? 4 : 2));
        w[0] = q[0];
        if constexpr (XF32) w[1] = q[1];
    }

    __device__ __forceinline__ void load_nt(const void* p, int64_t at)
    {
        const uint4* const q = (const uint4*)((const char*)p + at * (XF32 ? 4 : 2));
        w[0] = ld_nt16(q);
        if constexpr (XF32) w[1] = ld_nt16(q + 1);
    }

    // The chunk that `lane` of the wave holds.
    __device__ __forceinline__ Chunk of_lane(int lane) const
    {
        Chunk c;
#pragma unroll
        for (int i = 0; i < (XF32 ? 2 : 1); ++i)
            c.w[i] = make_uint4(__shfl(w[i].x, lane, 64), __shfl(w[i].y, lane, 64), __shfl(w[i].z, lane, 64), __shfl(w[i].w, lane, 64));
        return c;
    }

    __device__ __forceinline__ void values(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < (XF32 ? 2 : 1); ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (XF32) v[4 * i + j] = __uint_as_float(u[j]);
                else v[2 * j] = bf16_lo(u[j]), v[2 * j + 1] = bf16_hi(u[j]);
            }
        }
    }
};

// The angles of a chunk of eight values from `at`: eight of each (halves), or four (interleaved).
struct Angles {
    float c[8], s[8];
    int partner;                                         // distance to the pair's other chunk; 0: no rotation

    __device__ __forceinline__ void load(const KvRopeArgs& a, int64_t position, int at)
    {
        const int half = a.rot >> 1;
        partner = at >= a.rot ? 0 : a.interleaved ? 1 : at < half ? half : -half;
        if (partner == 0) return;
        const int64_t from = position * half + (a.interleaved ? at >> 1 : at < half ? at : at - half);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i == 1 && a.interleaved) break;
            const float4 u = ((const float4*)(a.cos + from))[i], w = ((const float4*)(a.sin + from))[i];
            c[4 * i] = u.x, c[4 * i + 1] = u.y, c[4 * i + 2] = u.z, c[4 * i + 3] = u.w;
            s[4 * i] = w.x, s[4 * i + 1] = w.y, s[4 * i + 2] = w.z, s[4 * i + 3] = w.w;
        }
    }

    // x: the chunk's values; p: their partners' (halves)
    __device__ __forceinline__ void turn(bool interleaved, const float (&x)[8], const float (&p)[8], float (&y)[8]) const
    {
        if (interleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[2 * j] = x[2 * j] * c[j] - x[2 * j + 1] * s[j];
                y[2 * j + 1] = x[2 * j + 1] * c[j] + x[2 * j] * s[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float other = p[j] * s[j];
                y[j] = partner > 0 ? x[j] * c[j] - other : x[j] * c[j] + other;
            }
        }
    }
};

// A chunk of one head on its way, with its partners' where they are another one.
template <bool XF32>
struct Turned {
    Chunk<XF32> own, other;

    __device__ __forceinline__ void load(const void* x, int64_t at, const Angles& turn, bool interleaved)
    {
        own.load(x, at);
        if (turn.partner != 0 && !interleaved) other.load(x, at + turn.partner);
    }

    __device__ __forceinline__ void values(const Angles& turn, bool interleaved, float (&y)[8]) const
    {
        float x[8], p[8];
        own.values(x);
        if (turn.partner != 0) {
            if (!interleaved) other.values(p);
            turn.turn(interleaved, x, p, y);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = x[j];
        }
    }
};

constexpr int kRopeAhead = 4;                            // heads of q, and chunks of K or V, that a lane loads together

// Queries: eight values a lane, so that a store of the wave writes whole rows.
template <bool XF32>
__device__ __forceinline__ void turn_queries(const KvRopeArgs& a, int64_t token, int part, int h0, int h1)
{
    const int64_t position = a.positions[token];
    const bool known = position >= 0 && position < a.table_rows, interleaved = a.interleaved != 0;
    Angles turn;
    turn.partner = 0;
    if (known) turn.load(a, position, part * 8);
    for (int h = h0; h < h1; h += kRopeAhead) {
        Turned<XF32> x[kRopeAhead];
#pragma unroll
        for (int u = 0; u < kRopeAhead; ++u)
            x[u].own.load_nt(a.q, token * a.ld_q + (int64_t)min(h + u, h1 - 1) * a.kv.dim + part * 8);
        // q_out may be q: every lane of the rows has its values before one of them stores
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int u = 0; u < kRopeAhead; ++u) {
            if (h + u >= h1) break;
            float v[8];
            if (!interleaved) x[u].other = x[u].own.of_lane(((int)threadIdx.x & 63) + turn.partner / 8);   // of the same row
            x[u].values(turn, interleaved, v);
            if (!known) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = 0.0f;
            }
            const int64_t to = token * a.ld_out + (int64_t)(h + u) * a.kv.dim + part * 8;
            if (XF32) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *(float4*)((float*)a.q_out + to + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            } else {
                *(uint4*)((uint16_t*)a.q_out + to) = make_uint4(Dec<0>::round2(v[0], v[1]), Dec<0>::round2(v[2], v[3]),
                                                                Dec<0>::round2(v[4], v[5]), Dec<0>::round2(v[6], v[7]));
            }
        }
    }
}

// A workgroup takes `per` heads of K, of V or of q (blockIdx.y; q in two halves of its tokens) for a run of tokens: a
// lane keeps its angles for all of them.
// 16001 tokens of 32 heads of q and 8 of K and V, head_dim 128 (MXFP4, half of a head turned, 345 MB): 61 us, 5.7 TB/s.  A head
// at a time with sixteen values a lane took 92, four heads of q together 77; q read past the caches, which its
// output then fills, gave the rest.
template <int BIAS, bool XF32>
__global__ __launch_bounds__(kThreads) void k_kv_append_rope(KvRopeArgs a)
{
    __shared__ double recip[kRecipTableSize];
    __shared__ float2 rne[BIAS == 0 ? 1 : kRneTableSize];
    int unit = (int)blockIdx.y;
    const int lanes = a.kv.dim >> 4, run = kThreads / lanes;   // of 16 values; tokens
    const int64_t token0 = (int64_t)blockIdx.x * run;
    const int kv_units = (a.kv.heads + a.per - 1) / a.per;
    if (unit >= 2 * kv_units) {
        unit -= 2 * kv_units;
        const int h0 = (unit >> 1) * a.per;
        const int64_t token = token0 + (unit & 1) * (run >> 1) + (int)threadIdx.x / (2 * lanes);
        if (token < a.tokens) turn_queries<XF32>(a, token, (int)threadIdx.x % (2 * lanes), h0, min(a.q_heads, h0 + a.per));
        return;
    }
    const bool is_v = unit >= kv_units;
    unit -= is_v ? kv_units : 0;
    if constexpr (BIAS != 0) {
        fill_recip_table(recip, (int)threadIdx.x);
        fill_rne_table<BIAS>(rne, (int)threadIdx.x);
        __syncthreads();
    }
    const int64_t token = token0 + (int)threadIdx.x / lanes;
    const int part = (int)threadIdx.x % lanes;
    if (token >= a.tokens) return;
    const int64_t position = a.positions[token];
    const int h0 = unit * a.per, h1 = min(a.kv.heads, h0 + a.per);
    int64_t row = -1;
    if (position >= 0 && position < a.table_rows) row = kv_row_of_slot(a.slots[token], a.num_slots, a.per_page, a.kv.heads, h0);
    if (row < 0) return;                                 // a row's lanes leave together
    const void* const x = is_v ? a.v : a.k;
    const int64_t from = token * (is_v ? a.ld_v : a.ld_k) + part * 16;
    const bool interleaved = a.interleaved != 0;
    Angles turn[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        turn[i].partner = 0;
        if (!is_v) turn[i].load(a, position, part * 16 + 8 * i);
    }
    for (int h = h0; h < h1; h += kRopeAhead / 2) {
        Turned<XF32> c[kRopeAhead / 2][2];
#pragma unroll
        for (int u = 0; u < kRopeAhead / 2; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) c[u][i].load(x, from + (int64_t)min(h + u, h1 - 1) * a.kv.dim + 8 * i, turn[i], interleaved);
#pragma unroll
        for (int u = 0; u < kRopeAhead / 2; ++u) {
            if (h + u >= h1) break;
            float v[16];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float y[8];
                c[u][i].values(turn[i], interleaved, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[8 * i + j] = y[j];
            }
            quantise_row16<BIAS>(a.kv, is_v, h + u, part, row, v, recip, rne);
            row += a.kv.page_size;
        }
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

hipError_t launch_kv_append_rope(int bias, bool x_f32, const KvRopeArgs& given, hipStream_t s)
{
    KvRopeArgs a = given;
    const int rows = kThreads / (a.kv.dim / 16);
    const int64_t runs = (a.tokens + rows - 1) / rows;
    // heads of a workgroup: as many as leave four workgroups a compute unit
    a.per = 1;
    while (a.per < 8 && runs * (2 * a.kv.heads + a.q_heads) / (2 * a.per) >= 1024) a.per *= 2;
    const int units = 2 * ((a.kv.heads + a.per - 1) / a.per) + 2 * ((a.q_heads + a.per - 1) / a.per);
    const dim3 grid((uint32_t)runs, (uint32_t)units);
#define FP4Q_ROPE(B)                                                                                    \
    do {                                                                                                \
        if (x_f32) hipLaunchKernelGGL((k_kv_append_rope<B, true>), grid, dim3(kThreads), 0, s, a);      \
        else hipLaunchKernelGGL((k_kv_append_rope<B, false>), grid, dim3(kThreads), 0, s, a);           \
    } while (0)
    if (bias == 0) FP4Q_ROPE(0);
    else if (bias == 7) FP4Q_ROPE(7);
    else FP4Q_ROPE(15);
#undef FP4Q_ROPE
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
