// fp4q_api.cpp -- the C ABI of libfp4q.so: configuration and shape validation
// on the host, then kernel launches on the caller's stream.  Nothing is
// enqueued unless every check passes; no device memory is allocated.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/fp4q.h"
#include "launch.h"

using namespace fp4q;

namespace {

struct Resolved {
    int fmt;          // FP4Q_NVFP4 / FP4Q_AMDFP4 / FP4Q_MXFP4
    int bias;         // 7 (E4M3) or 15 (UE5M3) for NV/AMD
    int outer_kind;   // kOuterNone / kOuterTensor / kOuter1D / kOuter2D
    int obs;
    bool sr;
    bool given;       // outer scales supplied by the caller
    bool inner2d;     // 16 x 16 inner tiles
    bool x_f32;       // FP32 source (else bf16)
    bool y_f32;       // FP32 dequantised output (else bf16)
};

bool misaligned(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) != 0; }

// Configuration rules: ALTO page, Technical design (two_level_scaling is one of
// none / tensorwise / outer_block; outer_block_size a multiple of 16) and
// Implementation (outer knobs rejected outside outer-block mode; AMD-FP4
// pinned to UE5M3); "MXFP4 weight QAT recipes", Guards (fp16 rejected).
int resolve(const fp4q_cfg* c, Resolved& r)
{
    if (!c) return FP4Q_ERR_NULL;
    if (c->abi_version != FP4Q_ABI_VERSION) return FP4Q_ERR_ABI;
    if (c->inner_2d != 0 && c->inner_2d != 1) return FP4Q_ERR_MODE;
    if (c->input_dtype != FP4Q_DTYPE_BF16 && c->input_dtype != FP4Q_DTYPE_FP32) return FP4Q_ERR_DTYPE;
    if (c->output_dtype != FP4Q_DTYPE_BF16 && c->output_dtype != FP4Q_DTYPE_FP32) return FP4Q_ERR_DTYPE;
    if (c->rounding != FP4Q_RNE && c->rounding != FP4Q_STOCHASTIC) return FP4Q_ERR_MODE;
    if (c->outer_mode != 0 && c->outer_mode != 1) return FP4Q_ERR_MODE;
    if (c->outer_2d != 0 && c->outer_2d != 1) return FP4Q_ERR_MODE;
    r.fmt = c->format;
    r.sr = c->rounding == FP4Q_STOCHASTIC;
    r.given = c->outer_mode == 1;
    r.inner2d = c->inner_2d == 1;
    r.x_f32 = c->input_dtype == FP4Q_DTYPE_FP32;
    r.y_f32 = c->output_dtype == FP4Q_DTYPE_FP32;
    r.obs = 0;
    r.bias = 0;
    r.outer_kind = kOuterNone;
    switch (c->format) {
    case FP4Q_NVFP4:
        if (c->scale_format == FP4Q_SCALE_DEFAULT || c->scale_format == FP4Q_SCALE_E4M3) r.bias = 7;
        else if (c->scale_format == FP4Q_SCALE_UE5M3) r.bias = 15;
        else return FP4Q_ERR_MODE;
        break;
    case FP4Q_AMDFP4:
        if (c->scale_format == FP4Q_SCALE_DEFAULT || c->scale_format == FP4Q_SCALE_UE5M3) r.bias = 15;
        else return FP4Q_ERR_MODE;
        break;
    case FP4Q_MXFP4:
        if (c->scale_format != FP4Q_SCALE_DEFAULT && c->scale_format != FP4Q_SCALE_UE8M0) return FP4Q_ERR_MODE;
        if (c->two_level != FP4Q_TWO_LEVEL_NONE || c->outer_block_size != 0 || c->outer_2d != 0 || r.given ||
            r.inner2d)
            return FP4Q_ERR_MODE;
        if (r.sr) return FP4Q_ERR_UNSUPPORTED;
        return FP4Q_OK;
    default:
        return FP4Q_ERR_MODE;
    }
    switch (c->two_level) {
    case FP4Q_TWO_LEVEL_NONE:
    case FP4Q_TENSORWISE:
        if (c->outer_block_size != 0 || c->outer_2d != 0) return FP4Q_ERR_MODE;
        if (c->two_level == FP4Q_TWO_LEVEL_NONE && r.given) return FP4Q_ERR_MODE;
        r.outer_kind = c->two_level == FP4Q_TENSORWISE ? kOuterTensor : kOuterNone;
        break;
    case FP4Q_OUTER_BLOCK:
        if (c->outer_block_size <= 0 || c->outer_block_size % 16 != 0) return FP4Q_ERR_SHAPE;
        r.obs = c->outer_block_size;
        r.outer_kind = c->outer_2d ? kOuter2D : kOuter1D;
        // 16 x 16 inner tiles make one decision per element for both
        // directions; 1D outer groups normalise each direction differently
        if (r.inner2d && r.outer_kind == kOuter1D) return FP4Q_ERR_MODE;
        break;
    default:
        return FP4Q_ERR_MODE;
    }
    return FP4Q_OK;
}

// Shape rules common to the quantising entry points.
int check_shape(const Resolved& r, int64_t rows, int64_t cols, int64_t ld, bool columnwise)
{
    if (rows < 0 || cols < 0) return FP4Q_ERR_SHAPE;
    const int inner = r.fmt == FP4Q_MXFP4 ? 32 : 16;
    if (cols % inner) return FP4Q_ERR_SHAPE;
    if (rows > 0 && ld < cols) return FP4Q_ERR_SHAPE;
    if ((columnwise || r.inner2d) && rows % 16) return FP4Q_ERR_SHAPE;
    if (r.outer_kind == kOuter1D || r.outer_kind == kOuter2D) {
        if (cols % r.obs) return FP4Q_ERR_SHAPE;
        if ((r.outer_kind == kOuter2D || columnwise) && rows % r.obs) return FP4Q_ERR_SHAPE;
    }
    // 32-bit block indexing inside the kernels, and 32-bit byte offsets within
    // a 64-row tile (x rows of ld_x bf16, residual rows of cols FP32)
    if (rows * (cols / 8) >= (int64_t)1 << 31) return FP4Q_ERR_UNSUPPORTED;
    if (ld > ((int64_t)1 << 24) || cols > ((int64_t)1 << 23)) return FP4Q_ERR_UNSUPPORTED;
    return FP4Q_OK;
}

// Sources read in 16-byte row chunks (the 64 x 64 tile kernels and the FP8
// re-encode): bf16 only, every row start 16-byte aligned.
int check_vector_source(const Resolved& r, int64_t ld)
{
    if (r.x_f32) return FP4Q_ERR_UNSUPPORTED;
    if (ld % 8) return FP4Q_ERR_ALIGN;
    return FP4Q_OK;
}

size_t outer_count(const Resolved& r, int64_t rows, int64_t cols, bool columnwise)
{
    switch (r.outer_kind) {
    case kOuterTensor: return columnwise ? 0 : 1;
    case kOuter2D: return columnwise ? 0 : (size_t)((rows / r.obs) * (cols / r.obs));
    case kOuter1D: return columnwise ? (size_t)(cols * (rows / r.obs)) : (size_t)(rows * (cols / r.obs));
    default: return 0;
    }
}

size_t ws_bytes_for(const Resolved& r)
{
    if (r.fmt != FP4Q_MXFP4 && r.outer_kind == kOuterTensor && !r.given) return sizeof(float) * (1 + kAmaxPartials);
    return 0;
}

int hip_status(hipError_t e) { return e == hipSuccess ? FP4Q_OK : FP4Q_ERR_HIP; }

// Cast-transpose workspace: [0, partial) the tensorwise partial maxima (when
// the scale is computed), then, 128-byte aligned, the staged tile blocks of
// the largest launch (groups go 64 to a launch; launches run in stream order
// and reuse the region).
constexpr size_t kPartialRegion = 4096;
constexpr size_t kStageAlign = 128;

size_t partial_bytes_for(const Resolved& r)
{
    return (r.outer_kind == kOuterTensor && !r.given) ? kPartialRegion : 0;
}

size_t stage_bytes_for(const Resolved& r, int32_t ngroups, const int64_t* rows, int64_t cols)
{
    const int64_t tc = (cols + 63) / 64;
    const int64_t blk = stage_block_bytes(r.outer_kind, r.obs);
    size_t most = 0;
    for (int32_t g0 = 0; g0 < ngroups; g0 += kMaxGroupsPerLaunch) {
        size_t sum = 0;
        for (int32_t g = g0; g < ngroups && g < g0 + kMaxGroupsPerLaunch; ++g)
            sum += (size_t)(((rows[g] + 63) / 64) * tc * blk);
        most = std::max(most, sum);
    }
    return most;
}

size_t ct_workspace_bytes(const Resolved& r, bool ef, int32_t ngroups, const int64_t* rows, int64_t cols)
{
    size_t n = partial_bytes_for(r);
    if (stage_applies(r.sr, ef, r.outer_kind, r.inner2d)) {
        const size_t st = stage_bytes_for(r, ngroups, rows, cols);
        if (st) n += st + kStageAlign;
    }
    return n;
}

// The staged region of a workspace large enough for staging, else null.
uint8_t* stage_region(const Resolved& r, bool ef, int32_t ngroups, const int64_t* rows, int64_t cols, void* ws,
                      size_t ws_bytes)
{
    if (!ws || !stage_applies(r.sr, ef, r.outer_kind, r.inner2d)) return nullptr;
    const size_t st = stage_bytes_for(r, ngroups, rows, cols);
    if (st == 0 || ws_bytes < partial_bytes_for(r) + st + kStageAlign) return nullptr;
    const uintptr_t p = reinterpret_cast<uintptr_t>(ws) + partial_bytes_for(r);
    return reinterpret_cast<uint8_t*>((p + kStageAlign - 1) & ~(uintptr_t)(kStageAlign - 1));
}

// Switch a tile launch to the staged walk (one tile per unit) over its groups.
void use_stage(TileArgs& a, const Resolved& r, uint8_t* stage)
{
    a.stage = stage;
    a.stage_block = stage_block_bytes(r.outer_kind, r.obs);
    a.tiles_c = (int32_t)((a.cols + 63) / 64);
    for (int g = 0; g < a.ngroups; ++g) {
        const int32_t R = a.row0[g + 1] - a.row0[g];
        a.tile0[g + 1] = a.tile0[g] + ((R + 63) / 64) * a.tiles_c;
    }
    a.total_tiles = a.tile0[a.ngroups];
    set_tile_grid(a.total_tiles, a.per_xcd, a.wgs_per_xcd);
}

// The gather pass for a staged tile launch.
hipError_t gather_staged(const TileArgs& a, const Resolved& r, hipStream_t s)
{
    GatherArgs gth;
    std::memset(&gth, 0, sizeof(gth));
    gth.stage = a.stage;
    gth.stage_block = a.stage_block;
    gth.ngroups = a.ngroups;
    gth.cols = a.cols;
    gth.tiles_c = a.tiles_c;
    gth.obs = (r.outer_kind == kOuter1D && !r.given) ? r.obs : 0;
    bool s4 = a.cols % 64 == 0 && !misaligned(a.row_scales, 4) && !misaligned(a.col_scales, 4);
    for (int g = 0; g <= a.ngroups; ++g) {
        gth.row0[g] = a.row0[g];
        gth.tile0[g] = a.tile0[g];
        if (g < a.ngroups && (a.row0[g + 1] - a.row0[g]) % 64) s4 = false;
    }
    gth.scales4 = s4 ? 1 : 0;
    gth.row_codes = a.row_codes;
    gth.row_scales = a.row_scales;
    gth.row_outer = gth.obs ? a.row_outer : nullptr;
    gth.col_codes = a.col_codes;
    gth.col_scales = a.col_scales;
    gth.col_outer = gth.obs ? a.col_outer : nullptr;
    return launch_gather(gth, s);
}

TileArgs tile_args_single(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld)
{
    TileArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.ld = ld;
    a.cols = cols;
    a.ngroups = 1;
    a.tiles_c = (int32_t)((cols + 127) / 128);
    a.row0[0] = 0;
    a.row0[1] = (int32_t)rows;
    a.tile0[0] = 0;
    a.tile0[1] = (int32_t)(((rows + 127) / 128) * a.tiles_c);
    a.total_tiles = a.tile0[1];
    set_tile_grid(a.total_tiles, a.per_xcd, a.wgs_per_xcd);
    return a;
}

// Rowwise quantisation shared by fp4_quantize and fp4_qdq.
int rowwise(const fp4q_cfg* cfg, const void* x, int64_t rows, int64_t cols, int64_t ld, void* y,
            uint8_t* codes, uint8_t* scales, float* outer, float* residual, void* ws, size_t ws_bytes, void* stream,
            bool is_qdq)
{
    Resolved r;
    int st = resolve(cfg, r);
    if (st) return st;
    st = check_shape(r, rows, cols, ld, false);
    if (st) return st;
    if (r.outer_kind == kOuter2D && r.obs != 64) return FP4Q_ERR_UNSUPPORTED;
    if (r.outer_kind == kOuter1D && r.obs != 16 && r.obs != 32 && r.obs != 64 && r.obs != 128)
        return FP4Q_ERR_UNSUPPORTED;
    if (r.fmt == FP4Q_MXFP4 && residual) return FP4Q_ERR_UNSUPPORTED;
    // the 64 x 64 tile modes read bf16 in 16-byte row chunks and write bf16
    const bool tile_mode = r.fmt != FP4Q_MXFP4 && (r.outer_kind == kOuter2D || r.inner2d);
    if (tile_mode) {
        if (r.y_f32 && is_qdq) return FP4Q_ERR_UNSUPPORTED;
        st = check_vector_source(r, ld);
        if (st) return st;
    }
    const uintptr_t esize = r.x_f32 ? 4 : 2;
    const bool empty = rows == 0 || cols == 0;
    const size_t need_ws = ws_bytes_for(r);
    if (!empty) {
        if (!x) return FP4Q_ERR_NULL;
        if (is_qdq) {
            if (!y) return FP4Q_ERR_NULL;
            if (r.given && r.outer_kind != kOuterNone && !outer) return FP4Q_ERR_NULL;
        } else {
            if (!codes || !scales) return FP4Q_ERR_NULL;
            if (r.outer_kind != kOuterNone && !outer) return FP4Q_ERR_NULL;
        }
        if (need_ws && !ws) return FP4Q_ERR_NULL;
        if ((codes == nullptr) != (scales == nullptr)) return FP4Q_ERR_NULL;
        // a misaligned view: x aligned to its element size only (not in the tile modes)
        if (misaligned(x, tile_mode ? 16 : esize) || misaligned(y, 16) || misaligned(codes, 16) ||
            misaligned(residual, 16) || misaligned(outer, 4) || misaligned(ws, 16))
            return FP4Q_ERR_ALIGN;
    }
    if (ws_bytes < need_ws) return FP4Q_ERR_WORKSPACE;
    if (empty) return FP4Q_OK;
    hipStream_t s = (hipStream_t)stream;
    // 16-byte vector loads when x and every row start are 16-byte aligned
    const bool x_vec = !misaligned(x, 16) && ((uint64_t)ld * esize) % 16 == 0;

    if (r.fmt == FP4Q_MXFP4)
        return hip_status(launch_mx_qdq(x, r.x_f32, x_vec, rows, cols, ld, y, r.y_f32, codes, scales, s));

    if (tile_mode) {
        // 64 x 64 tiles: the 2D outer tile, and the 16 x 16 inner tiles
        TileArgs a = tile_args_single(static_cast<const uint16_t*>(x), rows, cols, ld);
        a.row_codes = codes;
        a.row_scales = scales;
        a.row_outer = outer;
        a.residual = residual;
        a.y = static_cast<uint16_t*>(y);
        a.seed = cfg->seed;
        a.step = cfg->step;
        a.index_base = cfg->index_base;
        a.obs16 = 4;
        a.outer_given = r.given;
        a.inner_2d = r.inner2d ? 1 : 0;
        if (r.outer_kind == kOuterTensor) {
            if (r.given) {
                a.tensor_scale = outer;
            } else {
                float* wsf = (float*)ws;
                hipError_t e = launch_amax(r.bias, x, false, true, rows, cols, ld, residual, wsf + 1, kAmaxPartials, wsf,
                                           outer, s);
                if (e != hipSuccess) return FP4Q_ERR_HIP;
                a.tensor_scale = wsf;
            }
        }
        return hip_status(launch_tiles(r.bias, r.outer_kind, r.sr, a, s));
    }
    RowArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.rows = rows;
    a.cols = cols;
    a.ld = ld;
    a.codes = codes;
    a.scales = scales;
    a.outer = outer;
    a.residual = residual;
    a.y = y;
    a.seed = cfg->seed;
    a.step = cfg->step;
    a.index_base = cfg->index_base;
    a.obs16 = r.obs / 16;
    a.outer_given = r.given;
    a.x_vec = x_vec ? 1 : 0;
    a.y_f32 = r.y_f32 ? 1 : 0;
    if (r.outer_kind == kOuterTensor) {
        if (r.given) {
            a.tensor_scale = outer;
        } else if (rows * cols > kSmallTensorElems || residual != nullptr) {
            float* wsf = (float*)ws;
            hipError_t e = launch_amax(r.bias, x, r.x_f32, x_vec, rows, cols, ld, residual, wsf + 1, kAmaxPartials, wsf,
                                       outer, s);
            if (e != hipSuccess) return FP4Q_ERR_HIP;
            a.tensor_scale = wsf;
        }
        // else: a small tensor without a residual -- one launch, each workgroup
        // takes the amax itself (tensor_scale stays null; the kernel writes
        // outer when given).  With error feedback the amax is over x + r while
        // other workgroups rewrite r in place, so those calls keep the passes.
    }
    return hip_status(launch_rows(r.bias, r.outer_kind, r.sr, r.x_f32, a, s));
}

}  // namespace

extern "C" {

uint32_t fp4q_abi_version(void) { return FP4Q_ABI_VERSION; }

const char* fp4q_status_str(int status)
{
    switch (status) {
    case FP4Q_OK: return "ok";
    case FP4Q_ERR_NULL: return "a required pointer is NULL";
    case FP4Q_ERR_DTYPE: return "dtype not accepted (bf16 or fp32; fp16 is rejected)";
    case FP4Q_ERR_SHAPE: return "shape violates the block or outer-block divisibility rules";
    case FP4Q_ERR_MODE: return "illegal combination of format, scale format and two-level mode";
    case FP4Q_ERR_UNSUPPORTED: return "configuration valid but not implemented";
    case FP4Q_ERR_ALIGN: return "pointer or leading dimension misaligned";
    case FP4Q_ERR_WORKSPACE: return "workspace too small";
    case FP4Q_ERR_HIP: return "HIP launch error";
    case FP4Q_ERR_ABI: return "ABI version mismatch";
    default: return "unknown status";
    }
}

size_t fp4q_workspace_bytes(const fp4q_cfg* cfg, int64_t rows, int64_t cols)
{
    (void)rows;
    (void)cols;
    Resolved r;
    if (resolve(cfg, r)) return 0;
    return ws_bytes_for(r);
}

int fp4q_buffer_sizes(const fp4q_cfg* cfg, int64_t rows, int64_t cols, fp4q_sizes* out)
{
    if (!out) return FP4Q_ERR_NULL;
    Resolved r;
    int st = resolve(cfg, r);
    if (st) return st;
    std::memset(out, 0, sizeof(*out));
    const bool colwise_ok = (r.fmt != FP4Q_MXFP4) && rows % 16 == 0;
    st = check_shape(r, rows, cols, cols, false);
    if (st) return st;
    const size_t n = (size_t)rows * (size_t)cols;
    const int inner = r.fmt == FP4Q_MXFP4 ? 32 : 16;
    out->row_codes = n / 2;
    out->row_scales = n / inner;
    out->row_outer = outer_count(r, rows, cols, false) * sizeof(float);
    if (colwise_ok) {
        out->col_codes = n / 2;
        out->col_scales = n / 16;
        out->col_outer = (r.outer_kind == kOuter1D && rows % r.obs == 0) ? outer_count(r, rows, cols, true) * sizeof(float) : 0;
    }
    out->y = n * (r.y_f32 ? 4 : 2);
    out->residual = r.fmt == FP4Q_MXFP4 ? 0 : n * 4;
    out->workspace = ws_bytes_for(r);
    return FP4Q_OK;
}

int fp4_quantize(const fp4q_cfg* cfg, const void* x, int64_t rows, int64_t cols, int64_t ld_x, uint8_t* codes,
                 uint8_t* scales, float* outer, float* residual, void* workspace, size_t workspace_bytes, void* stream)
{
    return rowwise(cfg, x, rows, cols, ld_x, nullptr, codes, scales, outer, residual, workspace, workspace_bytes,
                   stream, false);
}

int fp4_qdq(const fp4q_cfg* cfg, const void* x, int64_t rows, int64_t cols, int64_t ld_x, void* y,
            uint8_t* codes, uint8_t* scales, float* outer, float* residual, void* workspace, size_t workspace_bytes,
            void* stream)
{
    return rowwise(cfg, x, rows, cols, ld_x, y, codes, scales, outer, residual, workspace, workspace_bytes, stream,
                   true);
}

int fp4_dequantize(const fp4q_cfg* cfg, const uint8_t* codes, const uint8_t* scales, const float* outer, int64_t rows,
                   int64_t cols, int32_t outer_transposed, void* y, void* stream)
{
    Resolved r;
    int st = resolve(cfg, r);
    if (st) return st;
    if (outer_transposed != 0 && outer_transposed != 1) return FP4Q_ERR_MODE;
    if (outer_transposed && r.outer_kind != kOuter2D) return FP4Q_ERR_MODE;
    if (rows < 0 || cols < 0) return FP4Q_ERR_SHAPE;
    const int inner = r.fmt == FP4Q_MXFP4 ? 32 : 16;
    if (cols % inner) return FP4Q_ERR_SHAPE;
    if (r.outer_kind == kOuter1D && cols % r.obs) return FP4Q_ERR_SHAPE;
    if (r.outer_kind == kOuter2D && (rows % r.obs || cols % r.obs)) return FP4Q_ERR_SHAPE;
    if (rows * (cols / 8) >= (int64_t)1 << 31) return FP4Q_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return FP4Q_OK;
    if (!codes || !scales || !y) return FP4Q_ERR_NULL;
    if (r.outer_kind != kOuterNone && !outer) return FP4Q_ERR_NULL;
    if (misaligned(codes, 16) || misaligned(y, 16) || misaligned(outer, 4)) return FP4Q_ERR_ALIGN;
    hipStream_t s = (hipStream_t)stream;
    if (r.fmt == FP4Q_MXFP4) return hip_status(launch_dequant_mx(codes, scales, rows, cols, y, r.y_f32, s));
    return hip_status(launch_dequant_nv(r.bias, r.outer_kind, outer_transposed, r.obs, codes, scales, outer, rows, cols,
                                        y, r.y_f32, s));
}

int fp4_cast_transpose(const fp4q_cfg* cfg, const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x,
                       uint8_t* row_codes, uint8_t* row_scales, float* row_outer, uint8_t* col_codes,
                       uint8_t* col_scales, float* col_outer, float* residual, void* workspace,
                       size_t workspace_bytes, void* stream)
{
    Resolved r;
    int st = resolve(cfg, r);
    if (st) return st;
    if (r.fmt == FP4Q_MXFP4) return FP4Q_ERR_UNSUPPORTED;
    st = check_shape(r, rows, cols, ld_x, true);
    if (st) return st;
    st = check_vector_source(r, ld_x);
    if (st) return st;
    if (r.outer_kind == kOuter2D && r.obs != 64) return FP4Q_ERR_UNSUPPORTED;
    if (r.outer_kind == kOuter1D && r.obs != 16 && r.obs != 32 && r.obs != 64 && r.obs != 128)
        return FP4Q_ERR_UNSUPPORTED;
    if ((r.outer_kind == kOuter2D || r.outer_kind == kOuterTensor) && col_outer && col_outer != row_outer)
        return FP4Q_ERR_MODE;
    const size_t need_ws = partial_bytes_for(r) ? ws_bytes_for(r) : 0;
    const bool empty = rows == 0 || cols == 0;
    if (!empty) {
        if (!x || !row_codes || !row_scales || !col_codes || !col_scales) return FP4Q_ERR_NULL;
        if (r.outer_kind != kOuterNone && !row_outer) return FP4Q_ERR_NULL;
        if (r.outer_kind == kOuter1D && !col_outer) return FP4Q_ERR_NULL;
        if (need_ws && !workspace) return FP4Q_ERR_NULL;
        if (misaligned(x, 16) || misaligned(row_codes, 16) || misaligned(col_codes, 16) || misaligned(residual, 16) ||
            misaligned(row_outer, 4) || misaligned(col_outer, 4) || misaligned(workspace, 16))
            return FP4Q_ERR_ALIGN;
    }
    if (workspace_bytes < need_ws) return FP4Q_ERR_WORKSPACE;
    if (empty) return FP4Q_OK;
    hipStream_t s = (hipStream_t)stream;
    TileArgs a = tile_args_single(x, rows, cols, ld_x);
    a.row_codes = row_codes;
    a.row_scales = row_scales;
    a.row_outer = row_outer;
    a.col_codes = col_codes;
    a.col_scales = col_scales;
    a.col_outer = col_outer;
    a.residual = residual;
    a.seed = cfg->seed;
    a.step = cfg->step;
    a.index_base = cfg->index_base;
    a.obs16 = r.obs ? r.obs / 16 : 1;
    a.outer_given = r.given;
    a.inner_2d = r.inner2d ? 1 : 0;
    // 1D groups of 128 span two tiles: their scales are computed first and
    // the tile kernel reads them as precomputed ones
    Resolved rt = r;
    if (r.outer_kind == kOuter1D && r.obs == 128 && !r.given) {
        st = hip_status(launch_outer128(r.bias, a, s));
        if (st) return st;
        a.outer_given = 1;
        rt.given = true;
    }
    uint8_t* stage = stage_region(rt, residual != nullptr, 1, &rows, cols, workspace, workspace_bytes);
    if (stage) use_stage(a, rt, stage);
    if (r.outer_kind == kOuterTensor) {
        if (r.given) {
            a.tensor_scale = row_outer;
        } else {
            float* wsf = (float*)workspace;
            hipError_t e = launch_amax(r.bias, x, false, true, rows, cols, ld_x, residual, wsf + 1, kAmaxPartials, wsf,
                                       row_outer, s);
            if (e != hipSuccess) return FP4Q_ERR_HIP;
            a.tensor_scale = wsf;
        }
    }
    st = hip_status(launch_tiles(r.bias, r.outer_kind, r.sr, a, s));
    if (st || !stage) return st;
    return hip_status(gather_staged(a, rt, s));
}

int fp4_mx_project_fp8(const fp4q_cfg* cfg, const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x,
                       uint16_t* y, uint8_t* mx8_row, uint8_t* mx8_row_scales, uint8_t* mx8_col,
                       uint8_t* mx8_col_scales, uint8_t* blk, uint8_t* blk_t, float* blk_scales, void* stream)
{
    Resolved r;
    int st = resolve(cfg, r);
    if (st) return st;
    if (r.fmt != FP4Q_MXFP4) return FP4Q_ERR_MODE;
    st = check_shape(r, rows, cols, ld_x, false);
    if (st) return st;
    if (r.y_f32) return FP4Q_ERR_UNSUPPORTED;
    st = check_vector_source(r, ld_x);
    if (st) return st;
    if ((mx8_row == nullptr) != (mx8_row_scales == nullptr)) return FP4Q_ERR_NULL;
    if ((mx8_col == nullptr) != (mx8_col_scales == nullptr)) return FP4Q_ERR_NULL;
    const bool want_blk = blk || blk_t || blk_scales;
    if (mx8_col && rows % 32) return FP4Q_ERR_SHAPE;
    if (want_blk && (rows % 128 || cols % 128)) return FP4Q_ERR_SHAPE;
    // 32-bit byte offsets inside a 128-row tile
    if (rows > ((int64_t)1 << 22) || ld_x > ((int64_t)1 << 22)) return FP4Q_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return FP4Q_OK;
    if (!x) return FP4Q_ERR_NULL;
    if (misaligned(x, 16) || misaligned(y, 16) || misaligned(mx8_row, 16) || misaligned(mx8_col, 16) ||
        misaligned(blk, 16) || misaligned(blk_t, 16) || misaligned(blk_scales, 4))
        return FP4Q_ERR_ALIGN;
    if (!y && !mx8_row && !mx8_col && !want_blk) return FP4Q_OK;   // nothing asked
    Mx8Args a;
    a.x = x;
    a.rows = rows;
    a.cols = cols;
    a.ld = ld_x;
    a.y = y;
    a.mx8_row = mx8_row;
    a.mx8_row_sc = mx8_row_scales;
    a.mx8_col = mx8_col;
    a.mx8_col_sc = mx8_col_scales;
    a.blk = blk;
    a.blk_t = blk_t;
    a.blk_sc = blk_scales;
    return hip_status(launch_mx_fp8(a, (hipStream_t)stream));
}

size_t fp4q_mx_scales_tiled_bytes(int64_t rows, int64_t K)
{
    if (rows <= 0 || K <= 0) return 0;
    return (size_t)((rows + 255) / 256) * (size_t)((K + 255) / 256) * 256 * 8;
}

int fp4_mx_scales_tiled(const uint8_t* scales, int64_t rows, int64_t K, uint8_t* out, void* stream)
{
    if (rows < 0 || K < 0 || K % 32) return FP4Q_ERR_SHAPE;
    if (K > ((int64_t)1 << 22) || rows > ((int64_t)1 << 24)) return FP4Q_ERR_UNSUPPORTED;
    if (rows == 0 || K == 0) return FP4Q_OK;
    if (!scales || !out) return FP4Q_ERR_NULL;
    if (misaligned(out, 8)) return FP4Q_ERR_ALIGN;
    return hip_status(launch_mx_scales_tiled(scales, rows, K, out, (hipStream_t)stream));
}

int fp4_mm(const fp4q_cfg* cfg, const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
           const uint8_t* b_scales, int64_t M, int64_t N, int64_t K, int32_t scale_layout, void* c, int64_t ldc,
           void* stream)
{
    Resolved r;
    int st = resolve(cfg, r);
    if (st) return st;
    if (r.fmt != FP4Q_MXFP4) return FP4Q_ERR_MODE;
    if (scale_layout != 0 && scale_layout != 1) return FP4Q_ERR_MODE;
    if (M < 0 || N < 0 || K < 0 || K % 64) return FP4Q_ERR_SHAPE;
    if (M > 0 && N > 0 && ldc < N) return FP4Q_ERR_SHAPE;
    if (K > ((int64_t)1 << 22) || M > ((int64_t)1 << 24) || N > ((int64_t)1 << 24)) return FP4Q_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return FP4Q_OK;
    if (!c || (K > 0 && (!a_codes || !a_scales || !b_codes || !b_scales))) return FP4Q_ERR_NULL;
    if (misaligned(a_codes, 16) || misaligned(b_codes, 16) || misaligned(c, r.y_f32 ? 4 : 2)) return FP4Q_ERR_ALIGN;
    if (scale_layout == 1 && (misaligned(a_scales, 8) || misaligned(b_scales, 8))) return FP4Q_ERR_ALIGN;
    GemmArgs g;
    g.a = a_codes;
    g.as = a_scales;
    g.b = b_codes;
    g.bs = b_scales;
    g.M = (int32_t)M;
    g.N = (int32_t)N;
    g.K = (int32_t)K;
    g.tiles_m = (int32_t)((M + 255) / 256);
    g.tiles_n = (int32_t)((N + 255) / 256);
    g.c_f32 = r.y_f32 ? 1 : 0;
    // rowwise scales with whole 256-value K-tiles and 8-byte aligned bases take
    // one 8-byte load per row and K-tile, otherwise one load per byte
    if (scale_layout == 1) g.scale_layout = 2;
    else g.scale_layout = (K % 256 == 0 && !misaligned(a_scales, 8) && !misaligned(b_scales, 8)) ? 1 : 0;
    g.c = c;
    g.ldc = ldc;
    return hip_status(launch_mx_gemm(g, (hipStream_t)stream));
}

int fp4_cast_transpose_grouped(const fp4q_cfg* cfg, int32_t groups, const int64_t* rows_per_group, int64_t cols,
                               const uint16_t* x, int64_t ld_x, uint8_t* row_codes, uint8_t* row_scales,
                               float* row_outer, uint8_t* col_codes, uint8_t* col_scales, float* col_outer,
                               float* residual, void* workspace, size_t workspace_bytes, void* stream)
{
    Resolved r;
    int st = resolve(cfg, r);
    if (st) return st;
    if (r.fmt == FP4Q_MXFP4 || r.outer_kind == kOuterTensor) return FP4Q_ERR_UNSUPPORTED;
    st = check_vector_source(r, ld_x);
    if (st) return st;
    if (groups < 0) return FP4Q_ERR_SHAPE;
    if (groups > 0 && !rows_per_group) return FP4Q_ERR_NULL;
    int64_t total = 0;
    for (int32_t g = 0; g < groups; ++g) {
        const int64_t R = rows_per_group[g];
        st = check_shape(r, R, cols, ld_x, true);
        if (st) return st;
        total += R;
    }
    st = check_shape(r, total, cols, ld_x, true);
    if (st) return st;
    if (total >= ((int64_t)1 << 31)) return FP4Q_ERR_UNSUPPORTED;
    if (r.outer_kind == kOuter2D && r.obs != 64) return FP4Q_ERR_UNSUPPORTED;
    if (r.outer_kind == kOuter1D && r.obs != 16 && r.obs != 32 && r.obs != 64 && r.obs != 128)
        return FP4Q_ERR_UNSUPPORTED;
    if (r.outer_kind == kOuter2D && col_outer && col_outer != row_outer) return FP4Q_ERR_MODE;
    if (total == 0 || cols == 0) return FP4Q_OK;
    if (!x || !row_codes || !row_scales || !col_codes || !col_scales) return FP4Q_ERR_NULL;
    if (r.outer_kind != kOuterNone && !row_outer) return FP4Q_ERR_NULL;
    if (r.outer_kind == kOuter1D && !col_outer) return FP4Q_ERR_NULL;
    if (misaligned(x, 16) || misaligned(row_codes, 16) || misaligned(col_codes, 16) || misaligned(residual, 16) ||
        misaligned(row_outer, 4) || misaligned(col_outer, 4))
        return FP4Q_ERR_ALIGN;
    hipStream_t s = (hipStream_t)stream;
    const int32_t tiles_c = (int32_t)((cols + 127) / 128);
    const bool outer128 = r.outer_kind == kOuter1D && r.obs == 128 && !r.given;
    Resolved rt = r;
    if (outer128) rt.given = true;
    uint8_t* stage = stage_region(rt, residual != nullptr, groups, rows_per_group, cols, workspace, workspace_bytes);
    int64_t row_before = 0;
    for (int32_t g0 = 0; g0 < groups; g0 += kMaxGroupsPerLaunch) {
        const int32_t ng = std::min<int32_t>(kMaxGroupsPerLaunch, groups - g0);
        TileArgs a;
        std::memset(&a, 0, sizeof(a));
        a.x = x;
        a.ld = ld_x;
        a.cols = cols;
        a.row_codes = row_codes;
        a.row_scales = row_scales;
        a.row_outer = row_outer;
        a.col_codes = col_codes;
        a.col_scales = col_scales;
        a.col_outer = col_outer;
        a.residual = residual;
        a.seed = cfg->seed;
        a.step = cfg->step;
        a.index_base = cfg->index_base;
        a.obs16 = r.obs ? r.obs / 16 : 1;
        a.outer_given = r.given;
        a.inner_2d = r.inner2d ? 1 : 0;
        a.ngroups = ng;
        a.tiles_c = tiles_c;
        int64_t rr = row_before;
        int32_t tt = 0;
        for (int32_t k = 0; k < ng; ++k) {
            a.row0[k] = (int32_t)rr;
            a.tile0[k] = tt;
            const int64_t R = rows_per_group[g0 + k];
            rr += R;
            tt += (int32_t)(((R + 127) / 128) * tiles_c);
        }
        a.row0[ng] = (int32_t)rr;
        a.tile0[ng] = tt;
        a.total_tiles = tt;
        set_tile_grid(tt, a.per_xcd, a.wgs_per_xcd);
        row_before = rr;
        if (tt == 0) continue;
        if (outer128) {
            st = hip_status(launch_outer128(r.bias, a, s));
            if (st) return st;
            a.outer_given = 1;
        }
        if (stage) use_stage(a, rt, stage);
        st = hip_status(launch_tiles(r.bias, r.outer_kind, r.sr, a, s));
        if (st) return st;
        if (stage) {
            st = hip_status(gather_staged(a, rt, s));
            if (st) return st;
        }
    }
    return FP4Q_OK;
}

size_t fp4q_cast_transpose_workspace_bytes(const fp4q_cfg* cfg, int32_t groups, const int64_t* rows_per_group,
                                           int64_t cols, int32_t with_residual)
{
    Resolved r;
    if (resolve(cfg, r) || r.fmt == FP4Q_MXFP4 || groups < 0 || cols < 0 || (groups > 0 && !rows_per_group))
        return 0;
    for (int32_t g = 0; g < groups; ++g)
        if (rows_per_group[g] < 0) return 0;
    return ct_workspace_bytes(r, with_residual != 0, groups, rows_per_group, cols);
}

namespace {

// Configuration of a 4-bit cache: RNE rows of one tensor per head, whose FP32
// scale, if any, is given.
int resolve_cache(const fp4q_cfg* cfg, const fp4q_kv_cache* c, Resolved& r, KvView& v)
{
    const int st = resolve(cfg, r);
    if (st) return st;
    if (!c) return FP4Q_ERR_NULL;
    if (r.sr || r.outer_kind == kOuter1D || r.outer_kind == kOuter2D) return FP4Q_ERR_UNSUPPORTED;
    if (r.inner2d || (r.outer_kind == kOuterTensor && !r.given)) return FP4Q_ERR_MODE;
    if (c->num_pages < 0 || c->kv_heads < 1 || c->page_size < kKvGroup || c->page_size % kKvGroup)
        return FP4Q_ERR_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return FP4Q_ERR_UNSUPPORTED;
    if (c->page_size > kKvMaxPage || c->kv_heads > 65535 || c->num_pages > ((int64_t)1 << 31) - 1)
        return FP4Q_ERR_UNSUPPORTED;
    if (c->num_pages > 0 && (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)) return FP4Q_ERR_NULL;
    if (r.outer_kind == kOuterTensor && (!c->k_outer || !c->v_outer)) return FP4Q_ERR_NULL;
    if (misaligned(c->k_codes, 16) || misaligned(c->k_scales, 16) || misaligned(c->v_codes, 16) ||
        misaligned(c->v_scales, 16) || misaligned(c->k_outer, 4) || misaligned(c->v_outer, 4))
        return FP4Q_ERR_ALIGN;
    const bool outer = r.outer_kind == kOuterTensor;
    v = KvView{c->k_codes, c->k_scales, c->v_codes, c->v_scales, outer ? c->k_outer : nullptr,
               outer ? c->v_outer : nullptr, c->num_pages, c->page_size, c->kv_heads, c->head_dim};
    return FP4Q_OK;
}

constexpr int64_t kMaxKvRows = (int64_t)1 << 27;     // tokens of one append or read

int check_attn(const KvView& kv, const fp4q_attn* a)
{
    if (!a) return FP4Q_ERR_NULL;
    if (a->batch < 0 || a->total_q < 0 || a->table_cols < 0 || a->max_q < 0 || a->max_kv < 0 || a->window < 0)
        return FP4Q_ERR_SHAPE;
    if (a->q_heads < 1 || a->q_heads % kv.heads) return FP4Q_ERR_SHAPE;
    if (!a->q_starts && a->total_q != a->batch) return FP4Q_ERR_SHAPE;
    if (a->total_q > 1 && a->ld_q < (int64_t)a->q_heads * kv.dim) return FP4Q_ERR_SHAPE;
    if ((a->causal != 0 && a->causal != 1) || (a->window > 0 && !a->causal)) return FP4Q_ERR_MODE;
    if (!(a->scale > 0.0f) || a->scale > 3.4028235e38f) return FP4Q_ERR_MODE;
    if (a->max_kv > kKvMaxTokens || (int64_t)a->table_cols * kv.page_size >= (int64_t)1 << 31) return FP4Q_ERR_UNSUPPORTED;
    const int64_t rows = (int64_t)a->max_q * (a->q_heads / kv.heads);
    if (rows > ((int64_t)1 << 22) || a->batch > 65535 || (int64_t)a->batch * kv.heads >= (int64_t)1 << 24 ||
        (int64_t)a->total_q * a->q_heads >= (int64_t)1 << 31)
        return FP4Q_ERR_UNSUPPORTED;
    return FP4Q_OK;
}

size_t attn_bytes(const AttnPlan& p) { return p.o + p.few_o + p.ml + p.few_ml; }

AttnPlan plan_of(const KvView& kv, const fp4q_attn* a)
{
    return plan_attn(kv, a->batch, a->total_q, a->q_heads, a->max_q, a->max_kv, a->table_cols, a->window);
}

}  // namespace

int fp4_kv_append(const fp4q_cfg* cfg, const fp4q_kv_cache* cache, const void* k, int64_t ld_k, const void* v,
                  int64_t ld_v, const int64_t* slots, int64_t tokens, void* stream)
{
    Resolved r;
    KvAppendArgs a;
    const int st = resolve_cache(cfg, cache, r, a.kv);
    if (st) return st;
    const int64_t row = (int64_t)a.kv.heads * a.kv.dim;
    if (tokens < 0 || (tokens > 1 && (ld_k < row || ld_v < row))) return FP4Q_ERR_SHAPE;
    if (tokens > kMaxKvRows || ld_k > ((int64_t)1 << 31) || ld_v > ((int64_t)1 << 31)) return FP4Q_ERR_UNSUPPORTED;
    if (tokens == 0 || a.kv.num_pages == 0) return FP4Q_OK;
    if (!k || !v || !slots) return FP4Q_ERR_NULL;
    const int64_t per16 = r.x_f32 ? 4 : 8;
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(slots, 8) ||
        (tokens > 1 && (ld_k % per16 || ld_v % per16)))
        return FP4Q_ERR_ALIGN;
    a.k = k;
    a.v = v;
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.slots = slots;
    a.tokens = tokens;
    a.num_slots = a.kv.num_pages * a.kv.page_size;
    a.per_page = make_div64((uint32_t)(a.kv.page_size / kKvGroup));
    return hip_status(launch_kv_append(r.bias, r.x_f32, a, (hipStream_t)stream));
}

int fp4_kv_read(const fp4q_cfg* cfg, const fp4q_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k, void* v,
                void* stream)
{
    Resolved r;
    KvReadArgs a;
    const int st = resolve_cache(cfg, cache, r, a.kv);
    if (st) return st;
    if (tokens < 0) return FP4Q_ERR_SHAPE;
    // the reader's lanes (eight values of four heads of a token each) are counted in 32 bits
    if (tokens > kMaxKvRows || tokens * ((a.kv.heads + 3) / 4) * (a.kv.dim / 8) >= (int64_t)1 << 31)
        return FP4Q_ERR_UNSUPPORTED;
    if (tokens == 0) return FP4Q_OK;
    if (!k || !v || !slots) return FP4Q_ERR_NULL;
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(slots, 8)) return FP4Q_ERR_ALIGN;
    a.k = k;
    a.v = v;
    a.slots = slots;
    a.tokens = tokens;
    a.num_slots = a.kv.num_pages * a.kv.page_size;
    a.per_page = make_div64((uint32_t)(a.kv.page_size / kKvGroup));
    return hip_status(launch_kv_read(r.bias, r.y_f32, a, (hipStream_t)stream));
}

size_t fp4q_attn_workspace_bytes(const fp4q_cfg* cfg, const fp4q_kv_cache* cache, const fp4q_attn* attn)
{
    Resolved r;
    KvView kv;
    if (resolve_cache(cfg, cache, r, kv) || check_attn(kv, attn)) return 0;
    const AttnPlan p = plan_of(kv, attn);
    return attn_bytes(p);
}

int fp4_attn(const fp4q_cfg* cfg, const fp4q_kv_cache* cache, const fp4q_attn* attn, void* workspace,
             size_t workspace_bytes, void* stream)
{
    Resolved r;
    AttnArgs a;
    int st = resolve_cache(cfg, cache, r, a.kv);
    if (st) return st;
    st = check_attn(a.kv, attn);
    if (st) return st;
    if (attn->batch == 0 || attn->total_q == 0 || attn->max_q == 0) return FP4Q_OK;
    if (!attn->q || !attn->kv_lens || !attn->out || (attn->table_cols > 0 && !attn->page_table))
        return FP4Q_ERR_NULL;
    if (misaligned(attn->q, 16) || misaligned(attn->out, 16) || misaligned(attn->page_table, 4) ||
        misaligned(attn->kv_lens, 4) || misaligned(attn->q_starts, 4) || misaligned(attn->sinks, 4) ||
        misaligned(attn->lse, 4) || (attn->total_q > 1 && attn->ld_q % 8))
        return FP4Q_ERR_ALIGN;
    const AttnPlan p = plan_of(a.kv, attn);
    const size_t need = attn_bytes(p);
    if (need > 0 && (!workspace || workspace_bytes < need)) return FP4Q_ERR_WORKSPACE;
    if (need > 0 && misaligned(workspace, 16)) return FP4Q_ERR_ALIGN;
    a.q = attn->q;
    a.ld_q = attn->ld_q;
    a.table = attn->page_table;
    a.kv_lens = attn->kv_lens;
    a.q_starts = attn->q_starts;
    a.sinks = attn->sinks;
    a.out = attn->out;
    a.lse = attn->lse;
    char* ws = (char*)workspace;
    a.part_o = (float*)ws;
    a.few_o = (float*)(ws + p.o);
    a.part_ml = (float*)(ws + p.o + p.few_o);
    a.few_ml = (float*)(ws + p.o + p.few_o + p.ml);
    a.scale = attn->scale;
    a.batch = attn->batch;
    a.total_q = attn->total_q;
    a.q_heads = attn->q_heads;
    a.group = attn->q_heads / a.kv.heads;
    a.table_cols = attn->table_cols;
    a.max_q = attn->max_q;
    a.max_kv = attn->max_kv;
    a.causal = attn->causal;
    a.window = attn->window;
    a.slots = p.slots;
    a.groups = p.groups;
    a.splits = p.splits;
    a.chunk = p.chunk;
    a.out_f32 = r.y_f32 ? 1 : 0;
    a.per_page = make_div((uint32_t)(a.kv.page_size / kKvGroup));
    return hip_status(launch_attn(r.bias, a, (hipStream_t)stream));
}

size_t fp4q_linear_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M <= 0 || N <= 0 || K <= 0 || M > ((int64_t)1 << 20) || N > ((int64_t)1 << 24) || K > ((int64_t)1 << 22)) return 0;
    return plan_linear(M, N, K).bytes;
}

int fp4_linear(const fp4q_cfg* cfg, const uint16_t* x, int64_t M, int64_t ld_x, const uint8_t* codes,
               const uint8_t* scales, const float* outer, int32_t outer_transposed, int64_t N, int64_t K, void* y,
               int64_t ld_y, void* workspace, size_t workspace_bytes, void* stream)
{
    Resolved r;
    int st = resolve(cfg, r);
    if (st) return st;
    if (r.x_f32) return FP4Q_ERR_UNSUPPORTED;
    if (outer_transposed != 0 && outer_transposed != 1) return FP4Q_ERR_MODE;
    if (outer_transposed && r.outer_kind == kOuter1D) return FP4Q_ERR_MODE;
    if (M < 0 || N < 0 || K < 0 || K % 32) return FP4Q_ERR_SHAPE;
    if (M > 1 && (ld_x < K || ld_y < N)) return FP4Q_ERR_SHAPE;
    if (r.obs && (K % r.obs || (r.outer_kind == kOuter2D && N % r.obs))) return FP4Q_ERR_SHAPE;
    if ((r.outer_kind == kOuter2D && r.obs != 64) || (r.outer_kind == kOuter1D && r.obs % 64)) return FP4Q_ERR_UNSUPPORTED;
    if (K > ((int64_t)1 << 22) || M > ((int64_t)1 << 20) || N > ((int64_t)1 << 24)) return FP4Q_ERR_UNSUPPORTED;
    // byte offsets below 2^31 within a tile of x (128 rows: 127 of 2^24 bytes and K's 2^23) and within
    // the outer scales
    if (M > 1 && ld_x > ((int64_t)1 << 23)) return FP4Q_ERR_UNSUPPORTED;
    if ((r.outer_kind == kOuter1D ? N * (K / r.obs) : r.outer_kind == kOuter2D ? (N / 64) * (K / 64) : 0) >= (int64_t)1 << 29)
        return FP4Q_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return FP4Q_OK;
    if (!y || (K > 0 && (!x || !codes || !scales))) return FP4Q_ERR_NULL;
    if (K > 0 && r.outer_kind != kOuterNone && !outer) return FP4Q_ERR_NULL;
    if (misaligned(x, 16) || misaligned(codes, 16) || misaligned(outer, 4) ||
        (r.fmt != FP4Q_MXFP4 && misaligned(scales, 2)) || misaligned(y, r.y_f32 ? 4 : 2) || (M > 1 && K > 0 && ld_x % 8))
        return FP4Q_ERR_ALIGN;
    const LinearPlan p = plan_linear(M, N, K);
    if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes)) return FP4Q_ERR_WORKSPACE;
    if (p.bytes > 0 && misaligned(workspace, 16)) return FP4Q_ERR_ALIGN;
    LinearArgs a;
    a.x = x;
    a.ld_x = M > 1 ? ld_x : 0;
    a.codes = codes;
    a.scales = scales;
    a.outer_kind = K > 0 ? r.outer_kind : kOuterNone;
    a.outer = r.outer_kind == kOuterNone ? nullptr : outer;
    a.obs = r.obs;
    a.outer_n = a.outer_k = 0;
    if (r.outer_kind == kOuter1D) {
        a.outer_n = K / r.obs;
        a.outer_k = 1;
    } else if (r.outer_kind == kOuter2D) {
        a.outer_n = outer_transposed ? 1 : K / 64;
        a.outer_k = outer_transposed ? N / 64 : 1;
    }
    a.M = (int32_t)M;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.y_f32 = r.y_f32 ? 1 : 0;
    a.y = y;
    a.ld_y = ld_y;
    a.y_vec = !misaligned(y, r.y_f32 ? 16 : 8) && (M == 1 || ld_y % 4 == 0) ? 1 : 0;
    a.splits = p.splits;
    a.parts = p.bytes > 0 ? (float*)workspace : nullptr;
    a.parts_ld = p.ld;
    return hip_status(launch_linear(r.bias, a, (hipStream_t)stream));
}

}  // extern "C"
