// kernels_moe.hip -- a mixture-of-experts layer with 4-bit experts for a few tokens.
//
//   y_t = sum over the k experts e with token t's largest logits of
//         a_te (W2_e act(W1_e x_t + b1_e) + b2_e),   a_te the softmax of the logits
//
// Reading every expert that a token reached is what bounds the layer: 4 bits and a scale's share a
// weight, for few tokens each.  Four launches:
//   k_moe_route  one workgroup: each token's experts and their shares, then the (token, expert)
//                pairs in the order of the experts and their groups of up to 16 MT (MT 1 or 2)
//                pairs of one expert, for each of which the expert is read (plan_moe);
//   k_moe_up     a workgroup takes 32 gate and 32 up rows of W1 for one group; its waves share K
//                and join through LDS; a times the activation goes to the scratch;
//   k_moe_down   the same for 64 rows of W2; each pair's products go to the scratch in binary32;
//   k_moe_join   adds a token's pairs in the order of its choices, so its result does not depend on
//                which other tokens are there.  (W2's sums kept in LDS for all tokens, a workgroup
//                going through all groups with no scratch, took 58 us for 48 tokens of 32 experts of
//                2880 x 2880 where k_moe_down and k_moe_join took 44, with activations of one bf16
//                term: parts of K a wave end at every group.)
// 48 tokens, 4 of 32 experts of 2880 x 2880 each (MXFP4, 423 MB of weights): 7 + 73 + 45 + 5 us, k_moe_up 3.9 TB/s; NVFP4 with
// 2D outer scales (448 MB) 7 + 85 + 53 + 5; 64 tokens, 8 of those, 11 + 116 + 76 + 6.  Bound: loads in flight.  A wave holds a unit
// of 64 bytes of 64 rows and the next one, in registers.  Waves a SIMD by those: three in k_moe_up for all formats and in k_moe_down for MXFP4;
// two in k_moe_down for NVFP4 and AMD-FP4 (172 registers with 2D outer scales, 230 without), and with MT = 2.  Tried with MXFP4, k_moe_up:
// four waves spill the second unit (81 us), loads past the caches fetch lines twice (85: two waves share each line), two units
// of a line by one wave 76, 128 rows a workgroup 75.  Not tried: units that wait in LDS, which loads straight to it
// (lds_load.h) would hold without registers.
// Up to kMoeFewPairs pairs take two launches instead, rows of W as they lie (below).
//
// Products as in kernels_linear.hip: v_mfma_f32_16x16x32_bf16 with rows of W decoded to bf16,
// exactly, as the A operand and tokens as the B operand; a unit is 128 values of K, of which
// lane l loads 32 (l / 16) .. + 31 of row l % 16.  Sums are binary32.
//
// Rounding.  a act enters W2 as two bf16 terms (good to 2^-16); one term would add its 2^-8 to that of y.  With MT = 1 the terms lie
// side by side in the registers while a unit of W2 is decoded once for both; with MT = 2 there is no room for that
// (rows64), and each 4096 values of W2 are loaded (again from the caches) and decoded for one term, then for the other.  A few
// tokens' a act stays binary32.
#include <algorithm>

#include "fp4q_device.h"
#include "launch.h"
#include "lds_load.h"
#include "mfma16.h"

namespace fp4q {

namespace {

enum { kInnerOnly = 0, kPerTile = 1, kPerRow = 2 };      // outer scales inside the sum: none (or one an expert), 2D, 1D

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

// The sum over a wave's lanes, in all of them.
__device__ __forceinline__ float wave_sum(float v)
{
    const auto add = [&v](auto moved) { v += __int_as_float(moved(__float_as_int(v))); };
    add([](int x) { return __builtin_amdgcn_update_dpp(0, x, kDppXor1, 0xF, 0xF, false); });
    add([](int x) { return __builtin_amdgcn_update_dpp(0, x, kDppXor2, 0xF, 0xF, false); });
    add([](int x) { return __builtin_amdgcn_update_dpp(0, x, kDppHalfMirror, 0xF, 0xF, false); });
    add([](int x) { return __builtin_amdgcn_update_dpp(0, x, kDppMirror, 0xF, 0xF, false); });
    const float a = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0)), b = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16));
    const float c = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32)), d = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48));
    return (a + b) + (c + d);
}

struct Choice {
    int expert;                                          // of slot `lane`, -1: none
    float share;
};

// A token's logits.  PER: experts of a lane, expert j 64 + lane in place j.
template <int PER>
__device__ __forceinline__ void load_logits(const MoeArgs& a, int t, int lane, float (&l)[PER])
{
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = j * 64 + lane;
        l[j] = e < a.experts && t < a.tokens ? a.logits[(int64_t)t * a.experts + e] : -__builtin_inff();
    }
}

// The experts of a token and their shares, slot s in lane s.
template <int PER>
__device__ __forceinline__ Choice choose(const MoeArgs& a, const float (&l)[PER])
{
    const int lane = (int)threadIdx.x & 63;
    uint32_t key[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) key[j] = order_key(l[j]);
    float top = 0.0f, mine = 0.0f;
    int chosen = -1;
#pragma unroll 1
    for (int s = 0; s < a.top_k; ++s) {
        uint32_t most = key[0];
#pragma unroll
        for (int j = 1; j < PER; ++j) most = max(most, key[j]);
        most = wave_max_u32(most);
        if (most == 0) break;                            // nothing left to take
        // the lowest expert that has it
        int e = -1;
        float v = 0.0f;
#pragma unroll
        for (int j = PER - 1; j >= 0; --j) {
            const uint64_t has = __ballot(key[j] == most);
            const int at = has ? __ffsll((unsigned long long)has) - 1 : 0;
            e = has ? j * 64 + at : e;
            v = has ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(l[j]), at)) : v;
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) key[j] = j * 64 + lane == e ? 0u : key[j];
        if (s == 0) top = v;
        mine = lane == s ? v : mine;
        chosen = lane == s ? e : chosen;
    }
    const float weight = chosen >= 0 ? expf(mine - top) : 0.0f;
    float sum = weight;
    if (!a.renormalize) {                                // the softmax of all logits
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j) sum += l[j] > -__builtin_inff() ? expf(l[j] - top) : 0.0f;
    }
    sum = wave_sum(sum);
    return Choice{chosen, chosen >= 0 ? weight / sum : 0.0f};
}

// One workgroup.
template <int PER>
__global__ __launch_bounds__(kRouteThreads) void k_moe_route(MoeArgs a)
{
    __shared__ uint32_t member[PER * 64][kMoeMaxTokens / 32];
    __shared__ int first_group[PER * 64];
    __shared__ Choice chosen[kMoeMaxTokens * kMoeMaxTopK];
    constexpr int kTurns = kMoeMaxTokens * 64 / kRouteThreads;   // tokens of a wave
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    float l[kTurns][PER];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) load_logits<PER>(a, wave + i * (kRouteThreads / 64), lane, l[i]);
    for (int i = (int)threadIdx.x; i < PER * 64 * (kMoeMaxTokens / 32); i += kRouteThreads) (&member[0][0])[i] = 0;
    // places of the groups that no pair takes
    for (int i = (int)threadIdx.x; i < a.max_groups * a.group; i += kRouteThreads) a.pair_token[i] = -1;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int t = wave + i * (kRouteThreads / 64);
        if (t >= a.tokens) break;
        const Choice c = choose<PER>(a, l[i]);
        if (lane < a.top_k) {
            chosen[t * a.top_k + lane] = c;
            a.expert[t * a.top_k + lane] = c.expert;
            a.share[t * a.top_k + lane] = c.share;
            if (c.expert >= 0) atomicOr(&member[c.expert][t >> 5], 1u << (t & 31));
        }
    }
    __syncthreads();
    // groups before each expert's: wave 0, experts in runs of 64
    const auto count_of = [&](int e) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < kMoeMaxTokens / 32; ++w) n += __popc(member[e][w]);
        return n;
    };
    if (wave == 0) {
        int groups = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = j * 64 + lane, n = count_of(e), g = (n + a.group - 1) / a.group;
            int before = g;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const int q = __shfl_up(before, m, 64);
                before += lane >= m ? q : 0;
            }
            const int first = groups + before - g;
            first_group[e] = first;
            for (int i = 0; i < g; ++i) a.groups[first + i] = MoeGroup{e, min(a.group, n - i * a.group)};
            groups += __builtin_amdgcn_readlane(before, 63);
        }
        for (int i = groups + lane; i < a.max_groups; i += 64) a.groups[i] = MoeGroup{0, 0};
    }
    __syncthreads();
    for (int p = (int)threadIdx.x; p < a.tokens * a.top_k; p += kRouteThreads) {
        const Choice c = chosen[p];
        const int e = c.expert, t = p / a.top_k;
        if (e < 0) {
            a.place[p] = -1;
            continue;
        }
        int rank = __popc(member[e][t >> 5] & ((1u << (t & 31)) - 1));
        for (int w = 0; w < t >> 5; ++w) rank += __popc(member[e][w]);
        const int at = first_group[e] * a.group + rank;  // an expert's groups follow one another
        a.pair_token[at] = t;
        a.pair_share[at] = c.share;
        a.place[p] = at;
    }
}

// ---------------------------------------------------------------- products
// NT tiles of sixteen rows of one expert's weight, through buffer descriptors at their first
// rows: a lane's offsets are the same for every unit (128 values of K), what moves is a scalar, and
// lanes beyond K load zeros without a branch, so the compiler's waits count exactly and units
// stay in flight while earlier ones are used.
template <int BIAS, int OUTER, int NT>
struct Weights {
    static constexpr int B = Dec<BIAS>::kBlock;
    rsrc_t codes[NT], row_outer[OUTER == kPerRow ? NT : 1];
    const float* tile_outer[OUTER == kPerTile ? NT / 2 : 1];   // of two neighbouring tiles, which lie in one of 64 rows
    uint32_t code_off, outer_off;                        // of the lane
    int obs, last;

    // One unit of a lane: 32 values of K of its row in each tile, and outer scales.
    struct Unit {
        uint4 c[NT];
        float o[OUTER == kPerTile ? NT / 2 : OUTER == kPerRow ? NT : 1][2];
    };

    // Tile n: rows first[n] + stride 0 .. 15 of expert e's N (a multiple of 32).
    __device__ __forceinline__ Weights(const MoeWeight& w, int e, const int (&first)[NT], int stride, int N, int K, int lane)
    {
        const int row = lane & 15, quarter = lane >> 4;
        code_off = (uint32_t)(stride * row) * (uint32_t)(K / 2) + quarter * 16;
        outer_off = 0;
        obs = w.obs;
        last = (K >> 6) - 1;
        // of the lane's results, 4 quarter + 0 .. 3, each lane of a quad loads one
        if constexpr (OUTER == kPerRow) outer_off = (uint32_t)(stride * (4 * quarter + (lane & 3))) * (uint32_t)(K / obs) * 4;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int64_t r = (int64_t)e * N + first[n];
            codes[n] = make_rsrc(w.codes + r * (K / 2));
            if constexpr (OUTER == kPerTile) tile_outer[n >> 1] = w.outer + (r >> 6) * (K >> 6);
            if constexpr (OUTER == kPerRow) row_outer[n] = make_rsrc(w.outer + r * (K / obs));
        }
    }

    // Values k .. k + 127 of K, zeros from `end` on (a multiple of 32).
    __device__ __forceinline__ void load(int k, int end, int quarter, Unit& u) const
    {
        const bool in = k + 32 * quarter < end;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const u32x4_t c = __builtin_amdgcn_raw_buffer_load_b128(codes[n], in ? code_off : kOff, k / 2, 0);
            u.c[n] = make_uint4(c[0], c[1], c[2], c[3]);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if constexpr (OUTER == kPerTile)
                    if (n % 2 == 0) u.o[n >> 1][b] = tile_outer[n >> 1][min((k >> 6) + b, last)];
                if constexpr (OUTER == kPerRow)
                    u.o[n][b] = buf_load_f32(row_outer[n], k + 64 * b < end ? outer_off + (k + 64 * b) / obs * 4 : kOff);
            }
        }
    }
};

// Inner scale bytes in LDS.  Loaded a unit at a time they cost the cache a line's access for
// each row and two bytes, more than the codes do (48 tokens through 32 experts of 2880 x 2880, MXFP4: 97 us in k_moe_up,
// as many accesses as cycles); so a row's bytes of a whole chunk of K are loaded side by side, a row
// an instruction, and stay in LDS while the chunk is multiplied.
template <int BIAS, int CHUNK>
struct Scales {
    static constexpr int B = Dec<BIAS>::kBlock;
    static constexpr int kPiece = B == 32 ? 1 : 2;       // bytes of a load: rows have no better alignment
    static constexpr int kPieces = CHUNK / B / kPiece;   // of a row
    static constexpr int kStride = CHUNK / B + 4;        // of a row in LDS; rows lie in different banks
    static_assert((kPieces & (kPieces - 1)) == 0, "rows in whole loads of a wave, or loads of whole rows");

    // ROWS rows from descriptor r's place, `pitch` bytes apart, bytes at .. of a row, to LDS rows `to`; `bytes` of
    // the chunk are there.
    template <int ROWS>
    static __device__ __forceinline__ void stage(rsrc_t r, uint32_t pitch, int at, int bytes, lds_t* to, int lane)
    {
        constexpr int kLoads = ROWS * kPieces / 64;
        uint32_t v[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t row = (i * 64 + lane) / kPieces, o = (i * 64 + lane) % kPieces * kPiece;
            const uint32_t from = o < (uint32_t)bytes ? row * pitch + o : kOff;
            if constexpr (kPiece == 1) v[i] = __builtin_amdgcn_raw_buffer_load_b8(r, from, at, 0);
            else v[i] = __builtin_amdgcn_raw_buffer_load_b16(r, from, at, 0);
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            lds_t* const p = to + (i * 64 + lane) / kPieces * kStride + (i * 64 + lane) % kPieces * kPiece;
            if constexpr (kPiece == 1) *p = (unsigned char)v[i];
            else *(__attribute__((address_space(3))) uint16_t*)p = (uint16_t)v[i];
        }
    }

    // Of the lane's row at `row`, unit u of the chunk: the scales of 64 b .. + 63 that the lane multiplies
    // (place_of), for NVFP4 and AMD-FP4 one byte for each h.
    static __device__ __forceinline__ uint32_t read(const lds_t* row, int u, int b, int quarter)
    {
        const lds_t* const p = row + u * (128 / B) + b * (64 / B) + (quarter & 1) * (32 / B);
        if constexpr (kPiece == 1) return *p;
        else return *(const __attribute__((address_space(3))) uint16_t*)p;
    }
};

// A lane's part of a unit of the tokens, for each tile of them: of its column's token the eight values of
// each 64 that its place in the products takes (multiply), as one or two bf16 terms.
template <int MT, int TERMS>
struct Tokens {
    uint4 x[TERMS][MT][2][2];

    // term i through descriptor r[i]
    __device__ __forceinline__ void load(const rsrc_t (&r)[TERMS], const uint32_t (&off)[MT], int k, int end, int place)
    {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = k + 64 * b + 16 * h + place < end;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < TERMS; ++i) {
                        const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r[i], in ? off[m] : kOff, (k + 64 * b + 16 * h) * 2, 0);
                        x[i][m][b][h] = make_uint4(v[0], v[1], v[2], v[3]);
                    }
            }
    }
};

// A lane's place among 64 values of K: 16 h + 32 (quarter % 2) + 8 (quarter / 2), h = 0 and 1.
__device__ __forceinline__ int place_of(int quarter) { return 32 * (quarter & 1) + 8 * (quarter >> 1); }

// The two halves of a wave hold different 64 values of K (16-byte loads, whole 64-byte runs of a row),
// and swap words so that a product's lanes hold the same 64, under one outer scale.
template <int BIAS, int OUTER, int NT, int MT, int TERMS>
__device__ __forceinline__ void multiply(const typename Weights<BIAS, OUTER, NT>::Unit& u, const uint32_t (&scale)[NT][2],
                                         const Tokens<MT, TERMS>& x, f32x4_t (&acc)[NT][MT])
{
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const auto a = __builtin_amdgcn_permlane32_swap(u.c[n].x, u.c[n].y, false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(u.c[n].z, u.c[n].w, false, false);
        const uint32_t code[2][2] = {{a[0], b[0]}, {a[1], b[1]}};
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            float o[4];
            if constexpr (OUTER == kPerTile) o[0] = o[1] = o[2] = o[3] = u.o[n >> 1][d];
            if constexpr (OUTER == kPerRow) {            // from the quad's lanes
                const int v = __float_as_int(u.o[n][d]);
                o[0] = __int_as_float(__builtin_amdgcn_mov_dpp(v, 0x00, 0xF, 0xF, true));
                o[1] = __int_as_float(__builtin_amdgcn_mov_dpp(v, 0x55, 0xF, 0xF, true));
                o[2] = __int_as_float(__builtin_amdgcn_mov_dpp(v, 0xAA, 0xF, 0xF, true));
                o[3] = __int_as_float(__builtin_amdgcn_mov_dpp(v, 0xFF, 0xF, 0xF, true));
            }
            uint4 w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t byte = Dec<BIAS>::kBlock == 32 ? scale[n][d] : __builtin_amdgcn_ubfe(scale[n][d], 8 * h, 8);
                w[h] = DecBf16<BIAS>::octet(code[d][h], DecBf16<BIAS>::scale(byte));
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                f32x4_t p = OUTER == kInnerOnly ? acc[n][m] : f32x4_t{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < TERMS; ++i) {
                    p = Dec<0>::mfma(w[0], x.x[i][m][d][0], p);
                    p = Dec<0>::mfma(w[1], x.x[i][m][d][1], p);
                }
                if constexpr (OUTER == kInnerOnly) {
                    acc[n][m] = p;
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[n][m][r] = __builtin_fmaf(p[r], o[r], acc[n][m][r]);
                }
            }
        }
    }
}

// Units k, k + stride, ... before end, the next one on its way while one is used.  `ready` is called when the first of
// them is; then scale rows are in LDS, those of tile n at rows + n * apart, from value k0 on.  The loop stays rolled: a
// kernel of ten thousand bytes of code takes longer to fetch than a token's weights (W2 of one
// token, 4 experts of 2880 x 2880, unrolled four times 16.6 us, rolled 9.9).
template <int CHUNK, int BIAS, int OUTER, int NT, int MT, int TERMS, class Ready>
__device__ __forceinline__ void stream(const Weights<BIAS, OUTER, NT>& w, const rsrc_t (&x)[TERMS], const uint32_t (&off)[MT], int k, int end,
                                       int stride, const lds_t* rows, int apart, int k0, int quarter, f32x4_t (&acc)[NT][MT],
                                       Ready ready)
{
    using S = Scales<BIAS, CHUNK>;
    const int place = place_of(quarter);
    typename Weights<BIAS, OUTER, NT>::Unit u;
    Tokens<MT, TERMS> t;
    w.load(k, end, quarter, u);
    t.load(x, off, k, end, place);
    ready();
#pragma unroll 1
    for (; k < end; k += stride) {
        typename Weights<BIAS, OUTER, NT>::Unit next;
        Tokens<MT, TERMS> then;
        w.load(k + stride, end, quarter, next);          // zeros beyond the end
        then.load(x, off, k + stride, end, place);
        uint32_t scale[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int b = 0; b < 2; ++b) scale[n][b] = S::read(rows + n * apart, (k - k0) >> 7, b, quarter);
        multiply<BIAS, OUTER, NT, MT, TERMS>(u, scale, t, acc);
        u = next;
        t = then;
    }
}

__device__ __forceinline__ float gated(const MoeArgs& a, float g, float u)
{
    if (a.limit > 0.0f) {
        g = g > a.limit ? a.limit : g;
        u = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
    }
    return g / (1.0f + expf(-a.alpha * g)) * (u + a.shift);
}

// 64 rows of W times a group's tokens: the waves of a workgroup share K, and join through LDS in order.  `finish(n, m,
// v)` gets the sums of tiles n and n + 2 for tile m of the tokens.
constexpr int kWaves = 4, kChunk = 4096;                 // values of K whose scale bytes LDS holds

template <int BIAS, int OUTER, int MT, int TERMS, class Finish>
__device__ __forceinline__ void rows64(const MoeWeight& weight, int expert, const int (&first)[4], int stride, int N, int K,
                                       const uint16_t* const (&x)[TERMS], const uint32_t (&off)[MT], Finish finish)
{
    using S = Scales<BIAS, kChunk>;
    constexpr int kJoin = kWaves * 16 * MT * 64 * 4, kScales = 64 * S::kStride;
    __shared__ __align__(16) unsigned char smem[kJoin > kScales ? kJoin : kScales];
    float(*const join)[16 * MT][64] = reinterpret_cast<float(*)[16 * MT][64]>(smem);
    lds_t* const lds = (lds_t*)smem;
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const Weights<BIAS, OUTER, 4> w(weight, expert, first, stride, N, K, lane);
    f32x4_t acc[4][MT];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[n][m] = f32x4_t{0, 0, 0, 0};
    // a wave stages the scale bytes of a tile
    static_assert(kWaves == 4, "a tile's scale rows for each wave");
    const int first_row = wave == 0 ? first[0] : wave == 1 ? first[1] : wave == 2 ? first[2] : first[3];
    const rsrc_t sr = make_rsrc(weight.scales + ((int64_t)expert * N + first_row) * (K / S::B));
    for (int k0 = 0; k0 < K; k0 += kChunk) {
        const int end = min(K, k0 + kChunk);
        if (k0) __syncthreads();                         // everybody is done with the chunk before
        S::template stage<16>(sr, stride * (K / S::B), k0 / S::B, (end - k0) / S::B, lds + 16 * wave * S::kStride, lane);
        const lds_t* const rows = lds + col * S::kStride;
        const auto go = [&](const auto& terms, auto ready) {
            stream<kChunk, BIAS, OUTER, 4, MT>(w, terms, off, k0 + wave * 128, end, kWaves * 128, rows, 16 * S::kStride, k0, quarter,
                                               acc, ready);
        };
        const auto scales_in = [] { lds_barrier(); };
        if constexpr (TERMS == 2 && MT > 1) {
            // two terms of more than one tile of tokens have no room in the registers beside the next unit's
            const rsrc_t first_term[1] = {make_rsrc(x[0])}, second[1] = {make_rsrc(x[1])};
            go(first_term, scales_in);
            go(second, [] {});
        } else {
            rsrc_t terms[TERMS];
#pragma unroll
            for (int i = 0; i < TERMS; ++i) terms[i] = make_rsrc(x[i]);
            go(terms, scales_in);
        }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) join[wave][(n * MT + m) * 4 + r][lane] = acc[n][m][r];
    __syncthreads();
    const float whole = weight.outer_kind == kOuterTensor ? weight.outer[expert] : 1.0f;
    // a wave finishes every fourth of the pairs of two tiles of rows and 16 tokens
    for (int p = wave; p < 2 * MT; p += kWaves) {
        const int n = p & 1, m = p >> 1;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = ((n + (i & 4 ? 2 : 0)) * MT + m) * 4 + (i & 3);
            v[i] = join[0][at][lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v[i] += join[w][at][lane];
            v[i] *= whole;
        }
        finish(n, m, v);
    }
}

// y as a bf16 value and what it leaves: an infinity leaves nothing, and a number that would round to one is the
// largest bf16 and the rest.
__device__ __forceinline__ void two_terms(float y, float& hi, float& rest)
{
    constexpr float kMost = 3.38953139e38f;              // (2 - 2^-7) 2^127
    const float near = bf16_lo(Dec<0>::round2(y, 0.0f)), size = fabsf(y);
    hi = size > kMost && size < __builtin_inff() ? copysignf(kMost, y) : near;
    rest = size == __builtin_inff() ? 0.0f : y - hi;
}

// 32 gate rows and the same 32 up rows of W1.
template <int BIAS, int OUTER, int MT>
__global__ __launch_bounds__(64 * kWaves) void k_moe_up(MoeArgs a)
{
    const MoeGroup group = a.groups[blockIdx.y];
    if (group.count == 0) return;
    const int first_pair = (int)blockIdx.y * a.group, lane = (int)threadIdx.x & 63, col = lane & 15, quarter = lane >> 4;
    const int i0 = (int)blockIdx.x * 32, N = 2 * a.inter;
    // tiles: gate rows i0 .. + 15 and + 16 .. + 31, the same up rows
    const int s = a.interleaved ? 2 : 1, up = a.interleaved ? 1 : a.inter;
    const int first[4] = {s * i0, s * (i0 + 16), s * i0 + up, s * (i0 + 16) + up};
    uint32_t off[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int token = a.pair_token[first_pair + 16 * m + col];   // -1: none
        off[m] = token >= 0 ? (uint32_t)token * (uint32_t)(a.ld_x * 2) + place_of(quarter) * 2 : kOff;
    }
    rows64<BIAS, OUTER, MT, 1>(a.w1, group.expert, first, s, N, a.hidden, {a.x}, off, [&](int n, int m, const float (&v)[8]) {
        if (16 * m + col >= group.count) return;
        const int pair = first_pair + 16 * m + col, i = i0 + 16 * n + 4 * quarter;
        const float share = a.pair_share[pair];
        float y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t b = (int64_t)group.expert * N + s * (i + r);
            const float gate = v[r] + (a.b1 ? a.b1[b] : 0.0f);
            const float upper = v[4 + r] + (a.b1 ? a.b1[b + up] : 0.0f);
            y[r] = share * gated(a, gate, upper);
        }
        float hi[4], rest[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) two_terms(y[r], hi[r], rest[r]);
        *(uint2*)(a.mid + (int64_t)pair * a.inter + i) = make_uint2(Dec<0>::round2(hi[0], hi[1]), Dec<0>::round2(hi[2], hi[3]));
        *(uint2*)(a.mid_rest + (int64_t)pair * a.inter + i) =
            make_uint2(Dec<0>::round2(rest[0], rest[1]), Dec<0>::round2(rest[2], rest[3]));
    });
}

// 64 rows of W2, as many as there are in the last workgroup.
template <int BIAS, int OUTER, int MT>
__global__ __launch_bounds__(64 * kWaves) void k_moe_down(MoeArgs a)
{
    const MoeGroup group = a.groups[blockIdx.y];
    if (group.count == 0) return;
    const int first_pair = (int)blockIdx.y * a.group, lane = (int)threadIdx.x & 63, col = lane & 15, quarter = lane >> 4;
    const int n0 = (int)blockIdx.x * 64, further = min(n0 + 32, a.hidden - 32);   // a multiple of 32
    const int first[4] = {n0, n0 + 16, further, further + 16};
    uint32_t off[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        off[m] = 16 * m + col < group.count ? (uint32_t)(first_pair + 16 * m + col) * (uint32_t)(a.inter * 2) + place_of(quarter) * 2 : kOff;
    rows64<BIAS, OUTER, MT, 2>(a.w2, group.expert, first, 1, a.hidden, a.inter, {a.mid, a.mid_rest}, off,
                            [&](int n, int m, const float (&v)[8]) {
        if (16 * m + col >= group.count) return;
        float* const to = a.parts + (int64_t)(first_pair + 16 * m + col) * a.hidden + n0 + 16 * n + 4 * quarter;
        *(f32x4_t*)to = f32x4_t{v[0], v[1], v[2], v[3]};
        if (n0 + 32 < a.hidden) *(f32x4_t*)(to + 32) = f32x4_t{v[4], v[5], v[6], v[7]};
    });
}

// A token's sums over its experts in the order of its choices: four values of a row a lane, four experts' on their
// way together.
__global__ __launch_bounds__(256) void k_moe_join(MoeArgs a)
{
    const int n = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 4, t = (int)blockIdx.y;
    if (n >= a.hidden) return;
    f32x4_t v = {0, 0, 0, 0};
    for (int s = 0; s < a.top_k; s += 4) {
        int place[4];
        f32x4_t part[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) place[i] = s + i < a.top_k ? a.place[t * a.top_k + s + i] : -1;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            part[i] = place[i] >= 0 ? *(const f32x4_t*)(a.parts + (int64_t)place[i] * a.hidden + n) : f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (place[i] < 0) break;                     // none from here on
            v += part[i];
            if (!a.b2) continue;
            const float share = a.share[t * a.top_k + s + i];
            const float* b = a.b2 + (int64_t)a.expert[t * a.top_k + s + i] * a.hidden + n;
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(share, b[r], v[r]);
        }
    }
    const int64_t to = (int64_t)t * a.ld_y + n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (a.y_f32) ((float*)a.y)[to + i] = v[i];
        else ((uint16_t*)a.y)[to + i] = (uint16_t)Dec<0>::round2(v[i], 0.0f);
    }
}

// ---------------------------------------------------------------- a few tokens
// A wave takes rows of W as they lie, 16 values a lane and 1024 a pass, and multiplies them with its token's
// values in binary32: each 16 products are summed and their scales (inner times outer) multiply the sum.  No product is wasted on tokens that are not there, a row is read in whole lines, and waves need neither
// LDS nor a launch to join.  Each wave finds its token's experts itself.
// One token, 4 of 32 experts of 2880 x 2880 (NVFP4, 2D outer scales, 56 MB): 14 + 11 us, where groups take 35 in all.
// Bound: the trips one after another (logits, weights, the second launch, its logits, weights), about 7 us of each
// launch, then memory.
constexpr int kFewUpRows = 4, kFewDownRows = 8;          // of a wave: gate and up rows each, rows of W2
constexpr int kFewWaves = 4;

// One pass of a lane over R rows: codes, scale bytes, outer scales; and the token's values.  Each RUN of
// the rows lies in one tile of 64.
template <int BIAS, int OUTER, int R, int RUN, bool X32>
struct Pass {
    static constexpr int B = Dec<BIAS>::kBlock;
    // Codes enter as 2^-7 of their values (MXFP4: of their scaled values), since sixteen products of up to 6 x may pass binary32
    // where a scale brings them back; NVFP4's and AMD-FP4's sums of rows are multiplied by kBack.
    static constexpr float kBack = BIAS == 0 ? 1.0f : 0x1p7f;
    uint2 c[R];
    uint32_t s[R];
    float o[OUTER == kPerTile ? R / RUN : OUTER == kPerRow ? R : 1];
    uint4 x[X32 ? 4 : 2];

    // rows: the rows' numbers in W; x: the token's values; k: the lane's first value, from `K` on zeros
    __device__ __forceinline__ void load(const MoeWeight& w, const int64_t (&rows)[R], const void* token, int k, int K)
    {
        const bool in = k < K;
        const uint4* const from = (const uint4*)((const char*)token + k * (X32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (X32 ? 4 : 2); ++i) x[i] = in ? from[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            c[r] = in ? *(const uint2*)(w.codes + rows[r] * (K / 2) + k / 2) : make_uint2(0, 0);
            s[r] = in ? w.scales[rows[r] * (K / B) + k / B] : 0;
            if constexpr (OUTER == kPerTile)
                if (r % RUN == 0) o[r / RUN] = in ? w.outer[(rows[r] >> 6) * (K >> 6) + (k >> 6)] : 0.0f;
            if constexpr (OUTER == kPerRow) o[r] = in ? w.outer[rows[r] * (K / w.obs) + div_by((uint32_t)k >> 6, w.per_outer)] : 0.0f;
        }
    }

    __device__ __forceinline__ void add(float whole, float (&acc)[R]) const
    {
        float v[16];
#pragma unroll
        for (int i = 0; i < (X32 ? 4 : 2); ++i) {
            const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (X32) v[4 * i + j] = __uint_as_float(u[j]);
                else v[8 * i + 2 * j] = bf16_lo(u[j]), v[8 * i + 2 * j + 1] = bf16_hi(u[j]);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            // MXFP4's 2^k enters with the codes as 2^(k - 7) and with the sum as the rest (the conversion reads the
            // exponent alone: byte 0 is 2^-127, 0xFF NaN); others' scales multiply the sum
            const uint32_t part = s[r] == 0xFFu ? 0xFFu : s[r] > 7 ? s[r] - 7 : 0;
            const float with_codes = BIAS == 0 ? __uint_as_float(part << 23) : 1.0f / kBack;
            float d;
            if constexpr (BIAS == 0) d = __uint_as_float((min(s[r], 7u) + 127) << 23);
            else d = DecBf16<BIAS>::scale(s[r]) * (OUTER == kInnerOnly ? whole : o[OUTER == kPerTile ? r / RUN : r]);
            float sum = 0.0f;
            const auto eight = [&](uint32_t code, const float* p) {
                const auto two = [&](auto g, const float* q) { sum = __builtin_fmaf(g[1], q[1], __builtin_fmaf(g[0], q[0], sum)); };
                two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, with_codes, 0), p);
                two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, with_codes, 1), p + 2);
                two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, with_codes, 2), p + 4);
                two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, with_codes, 3), p + 6);
            };
            eight(c[r].x, v);
            eight(c[r].y, v + 8);
            acc[r] = __builtin_fmaf(sum, d, acc[r]);
        }
    }
};

// Steps 0 .. steps - 1 (`load` fetches one), two on their way while one is added.
template <class P, class Load, class Add>
__device__ __forceinline__ void passes(int steps, Load load, Add add)
{
    P p, next, then;
    load(0, p);
    load(1, next);
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
        load(i + 2, then);
        add(i, p);
        p = next;
        next = then;
    }
}

template <int BIAS, int OUTER, int PER>
__global__ __launch_bounds__(64 * kFewWaves) void k_moe_few_up(MoeArgs a)
{
    constexpr int R = 2 * kFewUpRows;
    using P = Pass<BIAS, OUTER, R, kFewUpRows, false>;
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int pair = (int)blockIdx.y, t = pair / a.top_k, slot = pair - t * a.top_k;
    const int i0 = ((int)blockIdx.x * kFewWaves + wave) * kFewUpRows, K = a.hidden, N = 2 * a.inter;
    if (i0 >= a.inter) return;
    float logits[PER];
    load_logits<PER>(a, t, lane, logits);
    const Choice mine = choose<PER>(a, logits);
    const int e = __builtin_amdgcn_readlane(mine.expert, slot);
    if (e < 0) return;
    int64_t rows[R];
    const int s = a.interleaved ? 2 : 1, up = a.interleaved ? 1 : a.inter;
#pragma unroll
    for (int r = 0; r < kFewUpRows; ++r) {
        rows[r] = (int64_t)e * N + s * (i0 + r);         // the intermediate size is a multiple of four
        rows[kFewUpRows + r] = rows[r] + up;
    }
    const float whole = a.w1.outer_kind == kOuterTensor ? a.w1.outer[e] : 1.0f;
    const uint16_t* const x = a.x + (int64_t)t * a.ld_x;
    // results r and r + kFewUpRows are finished by lane r
    const int i = i0 + (lane & (kFewUpRows - 1));
    const float* const b1 = a.b1 ? a.b1 + (int64_t)e * N + s * i : nullptr;
    const float bg = b1 ? b1[0] : 0.0f, bu = b1 ? b1[up] : 0.0f;
    float acc[R] = {};
    passes<P>((K + 1023) / 1024, [&](int j, P& p) { p.load(a.w1, rows, x, j * 1024 + lane * 16, K); },
              [&](int, const P& p) { p.add(whole, acc); });
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int r = 0; r < kFewUpRows; ++r) {
        const float gr = wave_sum(acc[r]) * P::kBack, ur = wave_sum(acc[kFewUpRows + r]) * P::kBack;
        g = lane == r ? gr : g;
        u = lane == r ? ur : u;
    }
    if (lane >= kFewUpRows) return;
    const float y = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine.share), slot)) * gated(a, g + bg, u + bu);
    a.mid32[(int64_t)pair * a.inter + i] = y;
}

// The waves of a workgroup take the passes of all of its token's experts over the same rows in turn, and join through
// LDS in order.
template <int BIAS, int OUTER, int PER>
__global__ __launch_bounds__(64 * kFewWaves) void k_moe_few_down(MoeArgs a)
{
    constexpr int R = kFewDownRows;
    using P = Pass<BIAS, OUTER, R, R, true>;
    __shared__ float join[kFewWaves][R];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int t = (int)blockIdx.y, n0 = (int)blockIdx.x * R, K = a.inter;
    float logits[PER];
    load_logits<PER>(a, t, lane, logits);
    const Choice mine = choose<PER>(a, logits);
    const int taken = __popcll(__ballot(mine.expert >= 0));   // slots 0 .. taken - 1
    const int of_slot = (K + 1023) / 1024, all = taken * of_slot;
    const int steps = wave < all ? (all - wave + kFewWaves - 1) / kFewWaves : 0;
    float acc[R] = {};
    if (steps > 0) {
        // the slot and the first value of the wave's step j (K, where nothing is loaded, for a step beyond the last)
        const auto place = [&](int j, int& s, int& k) {
            const int at = wave + kFewWaves * min(j, steps - 1);
            s = at / of_slot;
            k = j < steps ? (at - s * of_slot) * 1024 + lane * 16 : K;
        };
        passes<P>(steps, [&](int j, P& p) {
            int s, k;
            place(j, s, k);
            const int64_t first = (int64_t)__builtin_amdgcn_readlane(mine.expert, s) * a.hidden + n0;
            int64_t rows[R];
#pragma unroll
            for (int r = 0; r < R; ++r) rows[r] = first + r;
            p.load(a.w2, rows, a.mid32 + (int64_t)(t * a.top_k + s) * K, k, K);
        }, [&](int j, const P& p) {
            int s, k;
            place(j, s, k);
            const float whole = a.w2.outer_kind == kOuterTensor ? a.w2.outer[__builtin_amdgcn_readlane(mine.expert, s)] : 1.0f;
            p.add(whole, acc);
        });
    }
    float y = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float v = wave_sum(acc[r]) * P::kBack;
        y = lane == r ? v : y;
    }
    if (lane < R) join[wave][lane] = y;
    __syncthreads();
    if (wave != 0 || lane >= R) return;
    const int n = n0 + lane;
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) y += join[w][lane];
    if (a.b2)                                            // in the order of the token's choices
        for (int s = 0; s < taken; ++s) {
            const int e = __builtin_amdgcn_readlane(mine.expert, s);
            y = __builtin_fmaf(__int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine.share), s)), a.b2[(int64_t)e * a.hidden + n], y);
        }
    const int64_t out = (int64_t)t * a.ld_y + n;
    if (a.y_f32) ((float*)a.y)[out] = y;
    else ((uint16_t*)a.y)[out] = (uint16_t)Dec<0>::round2(y, 0.0f);
}

template <int BIAS, int OUTER, int MT>
hipError_t launch_products(const MoeArgs& a, hipStream_t s)
{
    hipLaunchKernelGGL((k_moe_up<BIAS, OUTER, MT>), dim3((uint32_t)(a.inter / 32), (uint32_t)a.max_groups),
                       dim3(64 * kWaves), 0, s, a);
    hipLaunchKernelGGL((k_moe_down<BIAS, OUTER, MT>), dim3((uint32_t)((a.hidden + 63) / 64), (uint32_t)a.max_groups),
                       dim3(64 * kWaves), 0, s, a);
    hipLaunchKernelGGL(k_moe_join, dim3((uint32_t)((a.hidden / 4 + 255) / 256), (uint32_t)a.tokens), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int BIAS, int OUTER, int PER>
hipError_t launch_few(const MoeArgs& a, hipStream_t s)
{
    const int i = kFewWaves * kFewUpRows;
    hipLaunchKernelGGL((k_moe_few_up<BIAS, OUTER, PER>), dim3((uint32_t)((a.inter + i - 1) / i), (uint32_t)(a.tokens * a.top_k)),
                       dim3(64 * kFewWaves), 0, s, a);
    hipLaunchKernelGGL((k_moe_few_down<BIAS, OUTER, PER>), dim3((uint32_t)(a.hidden / kFewDownRows), (uint32_t)a.tokens),
                       dim3(64 * kFewWaves), 0, s, a);
    return hipGetLastError();
}

template <int BIAS, int OUTER>
hipError_t launch_outer(const MoeArgs& a, hipStream_t s)
{
    if (a.few) return a.experts <= 64 ? launch_few<BIAS, OUTER, 1>(a, s) : launch_few<BIAS, OUTER, 8>(a, s);
    if (a.experts <= 64) hipLaunchKernelGGL((k_moe_route<1>), dim3(1), dim3(kRouteThreads), 0, s, a);
    else if (a.experts <= 128) hipLaunchKernelGGL((k_moe_route<2>), dim3(1), dim3(kRouteThreads), 0, s, a);
    else hipLaunchKernelGGL((k_moe_route<8>), dim3(1), dim3(kRouteThreads), 0, s, a);
    if (a.group == 16) return launch_products<BIAS, OUTER, 1>(a, s);
    return launch_products<BIAS, OUTER, 2>(a, s);
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
    // Row by row an expert is read for each of its pairs.  Against groups, us: 4 pairs of 32 experts of 2880 x 2880
    // (NVFP4) 24 : 35, 16 65 : 70, 24 91 : 87, 48 156 : 115; 9 pairs of 20 experts of 2048 x 736
    // (AMD-FP4) 15 : 21, 21 22 : 27, 30 30 : 28.
    p.few = pairs <= kMoeFewPairs ? 1 : 0;
    // Pairs of a group: an expert of more is read again for each further group (from the caches), one of fewer pays for
    // tiles of tokens that it has not, and with few experts more groups fill the chip better.  Groups of 16 against
    // 32, us, by pairs an expert: 8 experts of 2880 x 2880, 4 a token (NVFP4) 16 65 : 74, 17 65 : 68, 19 74 : 69, 24 78 : 72, 28
    // 83 : 77, 32 88 : 89; all 8 a token (MXFP4) 20 67 : 63, 32 71 : 73, 33 91 : 103, 48 101 : 107, 49 113 : 107, 64 124 : 115; 16 of
    // 2048 x 1024, 8 a token (AMD-FP4, 1D) 18 60 : 51, 26 64 : 57, 32 77 : 78; 2 of 2880 x 2880 (NVFP4, 2D) 20
    // 40 : 46, 40 51 : 55, 64 56 : 58.  Groups of 64 (one wave a SIMD but for MXFP4) gain at most 5 % on the better of
    // these (49 of each of the 8, MXFP4, 102) and lose up to 70 % (24 of each of 8, 4 a token, NVFP4, 2D, 136 for 79).
    const bool most = experts >= 4 && pairs > 17 * experts;
    p.group = most && (pairs <= 30 * experts || pairs > 48 * experts) ? 32 : 16;
    const int64_t reached = experts < pairs ? experts : pairs;
    const auto groups_of = [&](int64_t group) { return reached + (tokens > group ? pairs / group : 0); };
    p.max_groups = (int32_t)groups_of(p.group);
    // room for either, so that scratch of more tokens serves fewer
    const int64_t places = std::max(groups_of(16) * 16, most ? groups_of(32) * 32 : 0);
    size_t at = 0;
    const auto take = [&at](size_t n) { const size_t here = at; at += padded(n); return here; };
    p.groups = take(places / 16 * sizeof(MoeGroup));
    p.expert = take(pairs * 4);
    p.share = take(pairs * 4);
    p.place = take(pairs * 4);
    p.pair_token = take(places * 4);
    p.pair_share = take(places * 4);
    p.mid = take(places * inter * 4);
    p.parts = take(p.few ? 0 : places * hidden * 4);
    p.bytes = at;
    return p;
}

hipError_t launch_moe(int bias, const MoeArgs& a, hipStream_t s)
{
    if (bias == 0) return launch_bias<0>(a, s);
    if (bias == 7) return launch_bias<7>(a, s);
    return launch_bias<15>(a, s);
}

}  // namespace fp4q
