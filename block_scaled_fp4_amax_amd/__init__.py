"""block_scaled_fp4_amax_amd -- Python binding of libfp4q.so, the gfx950
block-scaled FP4 quantisation library.

The functions carry the C-ABI names (fp4_quantize, fp4_dequantize, fp4_qdq,
fp4_cast_transpose, fp4_cast_transpose_grouped, fp4_mm, fp4_linear,
fp4_kv_append, fp4_kv_append_rope, fp4_kv_read, fp4_attn, fp4_attn_tree, fp4_moe, fp4_add_rms_norm,
fp4_add_rms_norm_backward and the fp4q_* helpers).  They
only marshal arguments: torch supplies device memory and the current HIP
stream, every step of the computation runs in the library's HIP kernels.  If
the library is not built, importing the binding raises; there is no fallback.

Layouts, numerics and error rules are those documented in include/fp4q.h.
"""
import ctypes as ct
import os

__all__ = [
    "Fp4Error", "Cfg", "Sizes", "make_cfg", "lib", "fp4q_abi_version", "fp4q_status_str", "fp4q_buffer_sizes",
    "fp4q_workspace_bytes", "fp4q_cast_transpose_workspace_bytes", "fp4_quantize", "fp4_dequantize", "fp4_qdq", "fp4_cast_transpose",
    "fp4_cast_transpose_grouped", "fp4_mx_project_fp8", "fp4_mm", "fp4_mx_scales_tiled",
    "fp4q_mx_scales_tiled_bytes", "fp4_qdq_noalloc", "ErrorFeedback", "fp4_linear", "fp4q_linear_workspace_bytes", "KVCache", "fp4_kv_append",
    "fp4_kv_append_rope", "fp4_kv_read", "fp4_attn", "fp4_attn_tree", "fp4_attn_workspace", "fp4_moe", "fp4_moe_workspace", "fp4q_moe_workspace_bytes", "fp4_add_rms_norm", "fp4_add_rms_norm_backward",
    "fp4q_add_rms_norm_backward_workspace_bytes", "LIB_PATH",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                        "libfp4q_ubsan.so" if os.environ.get("FP4Q_SANITIZE") == "1" else "libfp4q.so")

OK, ERR_NULL, ERR_DTYPE, ERR_SHAPE, ERR_MODE, ERR_UNSUPPORTED, ERR_ALIGN, ERR_WORKSPACE, ERR_HIP, ERR_ABI = range(10)
ABI_VERSION = 2

FORMATS = {"nvfp4": 0, "amdfp4": 1, "mxfp4": 2}
SCALE_FORMATS = {None: 0, "default": 0, "e4m3": 1, "ue5m3": 2, "ue8m0": 3}
TWO_LEVEL = {"none": 0, "tensorwise": 1, "outer_block": 2}
ROUNDING = {"rne": 0, "stochastic": 1}
DTYPES = {"bf16": 0, "fp16": 1, "fp32": 2}


class Fp4Error(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, fp4q_status_str(status), status))


class Cfg(ct.Structure):
    _fields_ = [("abi_version", ct.c_uint32), ("format", ct.c_int32), ("scale_format", ct.c_int32),
                ("two_level", ct.c_int32), ("outer_block_size", ct.c_int32), ("outer_2d", ct.c_int32),
                ("rounding", ct.c_int32), ("outer_mode", ct.c_int32), ("input_dtype", ct.c_int32),
                ("inner_2d", ct.c_int32), ("output_dtype", ct.c_int32), ("seed", ct.c_uint64),
                ("step", ct.c_uint64), ("index_base", ct.c_uint64)]


class Sizes(ct.Structure):
    _fields_ = [(n, ct.c_size_t) for n in ("row_codes", "row_scales", "row_outer", "col_codes", "col_scales",
                                           "col_outer", "y", "residual", "workspace")]


class _KvCache(ct.Structure):
    _fields_ = [(n, ct.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales", "k_outer", "v_outer")] + [
        ("num_pages", ct.c_int64), ("page_size", ct.c_int32), ("kv_heads", ct.c_int32), ("head_dim", ct.c_int32),
        ("reserved", ct.c_int32)]


class _Attn(ct.Structure):
    _fields_ = [("q", ct.c_void_p), ("ld_q", ct.c_int64)] + [
        (n, ct.c_void_p) for n in ("page_table", "kv_lens", "q_starts", "sinks", "out", "lse")] + [
        ("scale", ct.c_float)] + [(n, ct.c_int32) for n in ("batch", "total_q", "q_heads", "table_cols", "max_q",
                                                            "max_kv", "causal", "window")]


class _KvRope(ct.Structure):
    _fields_ = [(n, ct.c_void_p) for n in ("k", "v", "q", "q_out")] + [
        (n, ct.c_int64) for n in ("ld_k", "ld_v", "ld_q", "ld_q_out")] + [
        (n, ct.c_void_p) for n in ("slots", "positions", "cos", "sin")] + [
        ("tokens", ct.c_int64), ("table_rows", ct.c_int64)] + [
        (n, ct.c_int32) for n in ("rot_dim", "q_heads", "interleaved", "reserved")]


class _Moe(ct.Structure):
    _fields_ = [("x", ct.c_void_p), ("ld_x", ct.c_int64)] + [
        (n, ct.c_void_p) for n in ("logits", "w1_codes", "w1_scales", "w1_outer", "w2_codes", "w2_scales", "w2_outer", "b1", "b2",
                                   "y")] + [
        (n, ct.c_int64) for n in ("ld_y", "tokens", "experts", "hidden", "inter")] + [
        (n, ct.c_int32) for n in ("top_k", "renormalize", "interleaved", "reserved")] + [
        (n, ct.c_float) for n in ("alpha", "limit", "shift")]


class _AddRmsNorm(ct.Structure):
    _fields_ = [("x", ct.c_void_p), ("residual", ct.c_void_p), ("ld_x", ct.c_int64), ("ld_residual", ct.c_int64)] + [
        (n, ct.c_void_p) for n in ("weight", "residual_out", "rstd", "y", "fp8", "fp8_scales")] + [
        ("rows", ct.c_int64), ("hidden", ct.c_int64), ("eps", ct.c_double)] + [
        (n, ct.c_int32) for n in ("x_dtype", "residual_dtype", "weight_dtype", "y_dtype", "fp8_mode", "reserved")]


class _RmsNormGrad(ct.Structure):
    _fields_ = [(n, ct.c_void_p) for n in ("dy", "h", "dresidual")] + [
        (n, ct.c_int64) for n in ("ld_dy", "ld_h", "ld_dresidual")] + [
        (n, ct.c_void_p) for n in ("weight", "rstd", "dx", "dweight")] + [
        ("rows", ct.c_int64), ("hidden", ct.c_int64)] + [
        (n, ct.c_int32) for n in ("dy_dtype", "h_dtype", "weight_dtype", "reserved")]


def make_cfg(format="nvfp4", scale_format=None, two_level="none", outer_block_size=0, outer_2d=False,
             rounding="rne", outer_mode=0, seed=0, step=0, index_base=0, input_dtype="bf16", inner_2d=False,
             output_dtype="bf16"):
    """Build an fp4q_cfg (string names or the raw integers of include/fp4q.h).

    inner_2d: one inner scale per 16 x 16 tile instead of per 1 x 16 block.
    input_dtype / output_dtype: "bf16" or "fp32" (the entry points below set
    them from the tensors they are given)."""
    def pick(table, v):
        return v if isinstance(v, int) and not isinstance(v, bool) else table[v]
    return Cfg(ABI_VERSION, pick(FORMATS, format), pick(SCALE_FORMATS, scale_format), pick(TWO_LEVEL, two_level),
               int(outer_block_size), int(bool(outer_2d)), pick(ROUNDING, rounding), int(outer_mode),
               pick(DTYPES, input_dtype), int(inner_2d), pick(DTYPES, output_dtype), int(seed), int(step),
               int(index_base))


def _with_dtypes(cfg, input_dtype=None, output_dtype=None):
    """A copy of cfg with its dtype fields set from the tensors of a call."""
    c = Cfg.from_buffer_copy(cfg)
    if input_dtype is not None:
        c.input_dtype = DTYPES[input_dtype]
    if output_dtype is not None:
        c.output_dtype = DTYPES[output_dtype]
    return c


_lib = None


def lib():
    """The loaded libfp4q.so (ctypes), with argument types declared."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libfp4q.so is not built (run __graft_entry__.build() or "
                              "python block_scaled_fp4_amax_amd/build.py)")
        L = ct.CDLL(LIB_PATH)
        P, I64, SZ = ct.c_void_p, ct.c_int64, ct.c_size_t
        C = ct.POINTER(Cfg)
        L.fp4q_abi_version.restype = ct.c_uint32
        L.fp4q_abi_version.argtypes = []
        L.fp4q_status_str.restype = ct.c_char_p
        L.fp4q_status_str.argtypes = [ct.c_int]
        L.fp4q_buffer_sizes.restype = ct.c_int
        L.fp4q_buffer_sizes.argtypes = [C, I64, I64, ct.POINTER(Sizes)]
        L.fp4q_workspace_bytes.restype = SZ
        L.fp4q_workspace_bytes.argtypes = [C, I64, I64]
        L.fp4q_cast_transpose_workspace_bytes.restype = SZ
        L.fp4q_cast_transpose_workspace_bytes.argtypes = [C, ct.c_int32, P, I64, ct.c_int32]
        L.fp4_quantize.restype = ct.c_int
        L.fp4_quantize.argtypes = [C, P, I64, I64, I64, P, P, P, P, P, SZ, P]
        L.fp4_dequantize.restype = ct.c_int
        L.fp4_dequantize.argtypes = [C, P, P, P, I64, I64, ct.c_int32, P, P]
        L.fp4_qdq.restype = ct.c_int
        L.fp4_qdq.argtypes = [C, P, I64, I64, I64, P, P, P, P, P, P, SZ, P]
        L.fp4_qdq_noalloc.restype = ct.c_int
        L.fp4_qdq_noalloc.argtypes = [C, P, I64, I64, I64, P, P, P, P, P, P]
        L.fp4_cast_transpose.restype = ct.c_int
        L.fp4_cast_transpose.argtypes = [C, P, I64, I64, I64, P, P, P, P, P, P, P, P, SZ, P]
        L.fp4_cast_transpose_grouped.restype = ct.c_int
        L.fp4_cast_transpose_grouped.argtypes = [C, ct.c_int32, P, I64, P, I64, P, P, P, P, P, P, P, P, SZ, P]
        L.fp4_mm.restype = ct.c_int
        L.fp4_mm.argtypes = [C, P, P, P, P, I64, I64, I64, ct.c_int32, P, I64, P]
        L.fp4q_mx_scales_tiled_bytes.restype = SZ
        L.fp4q_mx_scales_tiled_bytes.argtypes = [I64, I64]
        L.fp4_mx_scales_tiled.restype = ct.c_int
        L.fp4_mx_scales_tiled.argtypes = [P, I64, I64, P, P]
        L.fp4_mx_project_fp8.restype = ct.c_int
        L.fp4_mx_project_fp8.argtypes = [C, P, I64, I64, I64, P, P, P, P, P, P, P, P, P]
        KV, AT = ct.POINTER(_KvCache), ct.POINTER(_Attn)
        L.fp4_kv_append.restype = ct.c_int
        L.fp4_kv_append.argtypes = [C, KV, P, I64, P, I64, P, I64, P]
        L.fp4_kv_append_rope.restype = ct.c_int
        L.fp4_kv_append_rope.argtypes = [C, KV, ct.POINTER(_KvRope), P]
        L.fp4_moe.restype = ct.c_int
        L.fp4_moe.argtypes = [C, ct.POINTER(_Moe), P, SZ, P]
        L.fp4q_moe_workspace_bytes.restype = SZ
        L.fp4q_moe_workspace_bytes.argtypes = [I64] * 5
        L.fp4_add_rms_norm.restype = ct.c_int
        L.fp4_add_rms_norm.argtypes = [ct.POINTER(_AddRmsNorm), P]
        L.fp4_add_rms_norm_backward.restype = ct.c_int
        L.fp4_add_rms_norm_backward.argtypes = [ct.POINTER(_RmsNormGrad), P, SZ, P]
        L.fp4q_add_rms_norm_backward_workspace_bytes.restype = SZ
        L.fp4q_add_rms_norm_backward_workspace_bytes.argtypes = [I64, I64]
        L.fp4_kv_read.restype = ct.c_int
        L.fp4_kv_read.argtypes = [C, KV, P, I64, P, P, P]
        L.fp4q_attn_workspace_bytes.restype = SZ
        L.fp4q_attn_workspace_bytes.argtypes = [C, KV, AT]
        L.fp4_attn.restype = ct.c_int
        L.fp4_attn.argtypes = [C, KV, AT, P, SZ, P]
        L.fp4q_attn_tree_workspace_bytes.restype = SZ
        L.fp4q_attn_tree_workspace_bytes.argtypes = [C, KV, AT]
        L.fp4_attn_tree.restype = ct.c_int
        L.fp4_attn_tree.argtypes = [C, KV, AT, P, ct.c_int32, P, SZ, P]
        L.fp4_linear.restype = ct.c_int
        L.fp4_linear.argtypes = [C, P, I64, I64, P, P, P, ct.c_int32, I64, I64, P, I64, P, SZ, P]
        L.fp4q_linear_workspace_bytes.restype = SZ
        L.fp4q_linear_workspace_bytes.argtypes = [I64, I64, I64]
        if L.fp4q_abi_version() != ABI_VERSION:
            raise ImportError("libfp4q.so ABI %d, binding expects %d" % (L.fp4q_abi_version(), ABI_VERSION))
        _lib = L
    return _lib


def fp4q_abi_version():
    return lib().fp4q_abi_version()


def fp4q_status_str(status):
    return lib().fp4q_status_str(int(status)).decode()


def fp4q_buffer_sizes(cfg, rows, cols):
    s = Sizes()
    st = lib().fp4q_buffer_sizes(ct.byref(cfg), int(rows), int(cols), ct.byref(s))
    if st:
        raise Fp4Error(st, "fp4q_buffer_sizes")
    return {n: getattr(s, n) for n, _ in Sizes._fields_}


def fp4q_workspace_bytes(cfg, rows, cols):
    return lib().fp4q_workspace_bytes(ct.byref(cfg), int(rows), int(cols))


def fp4q_cast_transpose_workspace_bytes(cfg, rows_per_group, cols, with_residual=False):
    """Workspace that lets the cast-transpose stage its outputs (see
    include/fp4q.h); rows_per_group is a list of row counts (one entry for a
    single tensor)."""
    rows = [int(r) for r in rows_per_group]
    arr = (ct.c_int64 * max(len(rows), 1))(*rows)
    return lib().fp4q_cast_transpose_workspace_bytes(ct.byref(cfg), len(rows), arr, int(cols), int(bool(with_residual)))


def _ct_workspace(cfg, rows, cols, residual, device, workspace, staged):
    """(workspace, bytes) for a cast-transpose call: the caller's, or one
    sized for staged outputs (staged=True) or for the tensorwise scratch only."""
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    nb = fp4q_cast_transpose_workspace_bytes(cfg, rows, cols, residual is not None) if staged else \
        fp4q_workspace_bytes(cfg, sum(rows), cols)
    if nb == 0:
        return None, 0
    return _empty(nb, _torch().uint8, device), nb


# ------------------------------------------------------------------ marshalling helpers
_torch_module = None


def _torch():
    """torch, imported by the first call that needs it (an import statement costs every call)."""
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t):
    """Device address of a tensor (None for None).  Host tensors are refused:
    every pointer the library takes is a device pointer."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("fp4q takes device tensors; got one on %s" % t.device)
    return ct.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    if stream is None:
        return ct.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ct.c_void_p(stream)
    return ct.c_void_p(stream.cuda_stream)


def _check(st, where):
    if st:
        raise Fp4Error(st, where)


def _src(x, allow_f32=False):
    """(tensor, rows, cols, ld) for a 2-D bf16 (or 16-bit integer) source, or
    a float32 one where the entry point takes FP32."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    ok = (torch.bfloat16, torch.int16, torch.uint16) + ((torch.float32,) if allow_f32 else ())
    if x.dtype not in ok:
        raise Fp4Error(ERR_DTYPE, "source dtype %s" % x.dtype)
    if x.shape[1] > 1 and x.stride(1) != 1:
        raise ValueError("source rows must be contiguous (stride(1) == 1)")
    ld = x.stride(0) if x.shape[0] > 1 else x.shape[1]
    return x, x.shape[0], x.shape[1], ld


def _need(t, nbytes, what):
    """A caller-supplied buffer must be contiguous and hold at least nbytes
    (the library trusts its buffer sizes, so this is checked before any call)."""
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError("%s holds %d bytes, needs %d" % (what, have, nbytes))


def _need_residual(residual, R, C):
    if residual is None:
        return
    if residual.dtype != _torch().float32 or tuple(residual.shape) != (R, C):
        raise ValueError("residual must be a float32 [%d, %d] tensor" % (R, C))
    _need(residual, R * C * 4, "residual")


def _dtype_name(t):
    return "fp32" if t.dtype == _torch().float32 else "bf16"


def _empty(n, dtype, device):
    torch = _torch()
    return torch.empty(int(n), dtype=dtype, device=device)


def _inner(cfg):
    return 32 if cfg.format == FORMATS["mxfp4"] else 16


def _workspace(cfg, rows, cols, device, workspace):
    nb = fp4q_workspace_bytes(cfg, rows, cols)
    if nb == 0:
        return None, 0
    if workspace is None:
        workspace = _empty(nb, _torch().uint8, device)
    return workspace, workspace.numel() * workspace.element_size()


# ------------------------------------------------------------------ entry points
def fp4_quantize(x, cfg, *, residual=None, outer=None, workspace=None, stream=None, out=None):
    """Rowwise quantisation of a bf16 or float32 x (views with any storage
    offset and row pitch are accepted).  Returns {"codes", "scales", "outer"}
    (outer None without a two-level mode).  `outer` is read when
    cfg.outer_mode == 1.  `out` may supply preallocated "codes" / "scales"."""
    torch = _torch()
    x, R, C, ld = _src(x, allow_f32=True)
    cfg = _with_dtypes(cfg, _dtype_name(x))
    dev = x.device
    sizes = fp4q_buffer_sizes(cfg, R, C)
    out = out or {}
    codes = out.get("codes")
    if codes is None:
        codes = _empty(sizes["row_codes"], torch.uint8, dev).view(R, C // 2)
    scales = out.get("scales")
    if scales is None:
        scales = _empty(sizes["row_scales"], torch.uint8, dev).view(R, C // _inner(cfg))
    if outer is None and sizes["row_outer"]:
        outer = _empty(sizes["row_outer"] // 4, torch.float32, dev)
    _need(codes, sizes["row_codes"], "codes")
    _need(scales, sizes["row_scales"], "scales")
    _need(outer, sizes["row_outer"], "outer")
    _need_residual(residual, R, C)
    ws, wsb = _workspace(cfg, R, C, dev, workspace)
    _check(lib().fp4_quantize(ct.byref(cfg), _ptr(x), R, C, ld, _ptr(codes), _ptr(scales), _ptr(outer),
                              _ptr(residual), _ptr(ws), wsb, _stream(stream)), "fp4_quantize")
    return {"codes": codes, "scales": scales, "outer": outer}


def fp4_qdq(x, cfg, *, residual=None, outer=None, with_codes=False, workspace=None, stream=None, y=None,
            y_dtype=None):
    """Quantise-dequantise rowwise (bf16 or float32 x; y in y_dtype, default
    x's dtype, or the dtype of a given y).  Returns {"y", "codes", "scales", "outer"}."""
    torch = _torch()
    x, R, C, ld = _src(x, allow_f32=True)
    dev = x.device
    if y is not None:
        y_dtype = y.dtype
    ydt = torch.float32 if (y_dtype if y_dtype is not None else x.dtype) == torch.float32 else torch.bfloat16
    cfg = _with_dtypes(cfg, _dtype_name(x), "fp32" if ydt == torch.float32 else "bf16")
    sizes = fp4q_buffer_sizes(cfg, R, C)
    if y is None:
        y = torch.empty((R, C), dtype=ydt, device=dev)
    codes = scales = None
    if with_codes:
        codes = _empty(sizes["row_codes"], torch.uint8, dev).view(R, C // 2)
        scales = _empty(sizes["row_scales"], torch.uint8, dev).view(R, C // _inner(cfg))
    if outer is None and sizes["row_outer"] and (with_codes or cfg.outer_mode == 0):
        outer = _empty(sizes["row_outer"] // 4, torch.float32, dev)
    _need(y, sizes["y"], "y")
    _need(outer, sizes["row_outer"], "outer")
    _need_residual(residual, R, C)
    ws, wsb = _workspace(cfg, R, C, dev, workspace)
    _check(lib().fp4_qdq(ct.byref(cfg), _ptr(x), R, C, ld, _ptr(y), _ptr(codes), _ptr(scales), _ptr(outer),
                         _ptr(residual), _ptr(ws), wsb, _stream(stream)), "fp4_qdq")
    return {"y": y, "codes": codes, "scales": scales, "outer": outer}


def fp4_qdq_noalloc(x, cfg, *, y, codes=None, scales=None, outer=None, residual=None, stream=None):
    """fp4_qdq without a workspace (the library's own per-GPU scratch), for
    callers that cannot allocate: every output tensor is passed in (y, and
    optionally codes, scales and outer), nothing is allocated here.  Calls that
    overlap on one GPU race.  Returns {"y", "codes", "scales", "outer"}."""
    x, R, C, ld = _src(x, allow_f32=True)
    cfg = _with_dtypes(cfg, _dtype_name(x), _dtype_name(y))
    sizes = fp4q_buffer_sizes(cfg, R, C)
    _need(y, sizes["y"], "y")
    _need(codes, sizes["row_codes"], "codes")
    _need(scales, sizes["row_scales"], "scales")
    _need(outer, sizes["row_outer"], "outer")
    _need_residual(residual, R, C)
    _check(lib().fp4_qdq_noalloc(ct.byref(cfg), _ptr(x), R, C, ld, _ptr(y), _ptr(codes), _ptr(scales), _ptr(outer),
                                 _ptr(residual), _stream(stream)), "fp4_qdq_noalloc")
    return {"y": y, "codes": codes, "scales": scales, "outer": outer}


def fp4_dequantize(codes, scales, outer, rows, cols, cfg, *, outer_transposed=False, stream=None, y=None,
                   dtype=None):
    """bf16 (or float32: dtype=torch.float32, or a float32 y) [rows, cols]
    from stored codes, scales and outer scales."""
    torch = _torch()
    if y is None:
        y = torch.empty((rows, cols), dtype=dtype if dtype is not None else torch.bfloat16, device=codes.device)
    cfg = _with_dtypes(cfg, output_dtype=_dtype_name(y))
    if rows and cols:
        sizes = fp4q_buffer_sizes(cfg, rows, cols)
        _need(codes, sizes["row_codes"], "codes")
        _need(scales, sizes["row_scales"], "scales")
        _need(outer, sizes["row_outer"], "outer")
        _need(y, sizes["y"], "y")
    _check(lib().fp4_dequantize(ct.byref(cfg), _ptr(codes), _ptr(scales), _ptr(outer), int(rows), int(cols),
                                int(bool(outer_transposed)), _ptr(y), _stream(stream)), "fp4_dequantize")
    return y


def fp4_cast_transpose(x, cfg, *, residual=None, row_outer=None, col_outer=None, workspace=None, stream=None,
                       out=None, staged=True):
    """Rowwise and columnwise buffers from one read of x.  Returns
    {"row_codes", "row_scales", "row_outer", "col_codes", "col_scales", "col_outer"}.
    `out` may supply any of the four code / scale tensors preallocated.
    Without a `workspace`, one is allocated: large enough to stage the outputs
    (staged=True) or only for the tensorwise scratch (staged=False)."""
    torch = _torch()
    x, R, C, ld = _src(x)
    dev = x.device
    sizes = fp4q_buffer_sizes(cfg, R, C)
    given = out or {}
    out = {
        "row_codes": given.get("row_codes"), "row_scales": given.get("row_scales"),
        "col_codes": given.get("col_codes"), "col_scales": given.get("col_scales"),
    }
    shapes = {"row_codes": (R, C // 2), "row_scales": (R, C // 16), "col_codes": (C, R // 2),
              "col_scales": (C, R // 16)}
    for k, shp in shapes.items():
        if out[k] is None:
            out[k] = _empty(shp[0] * shp[1], torch.uint8, dev).view(*shp)
    if row_outer is None and sizes["row_outer"]:
        row_outer = _empty(sizes["row_outer"] // 4, torch.float32, dev)
    if col_outer is None and sizes["col_outer"]:
        col_outer = _empty(sizes["col_outer"] // 4, torch.float32, dev)
    out["row_outer"], out["col_outer"] = row_outer, col_outer
    for k, shp in shapes.items():
        _need(out[k], shp[0] * shp[1], k)
    _need(row_outer, sizes["row_outer"], "row_outer")
    _need(col_outer, sizes["col_outer"], "col_outer")
    _need_residual(residual, R, C)
    ws, wsb = _ct_workspace(cfg, [R], C, residual, dev, workspace, staged)
    _check(lib().fp4_cast_transpose(ct.byref(cfg), _ptr(x), R, C, ld, _ptr(out["row_codes"]), _ptr(out["row_scales"]),
                                    _ptr(row_outer), _ptr(out["col_codes"]), _ptr(out["col_scales"]), _ptr(col_outer),
                                    _ptr(residual), _ptr(ws), wsb, _stream(stream)), "fp4_cast_transpose")
    return out


def fp4_cast_transpose_grouped(x, rows_per_group, cfg, *, residual=None, stream=None, out=None, workspace=None,
                               staged=True):
    """Per-group cast-transpose of groups stacked along rows (one launch per 64
    groups).  Returns flat stacked buffers (see include/fp4q.h).  `workspace`
    and `staged` as for fp4_cast_transpose."""
    torch = _torch()
    x, total, C, ld = _src(x)
    dev = x.device
    rows = [int(r) for r in rows_per_group]
    if sum(rows) != total:
        raise ValueError("rows_per_group does not sum to x.shape[0]")
    n_ro = n_co = 0
    for R in rows:
        s = fp4q_buffer_sizes(cfg, R, C)
        n_ro += s["row_outer"] // 4
        n_co += s["col_outer"] // 4
    if out is None:
        out = {
            "row_codes": _empty(total * C // 2, torch.uint8, dev).view(total, C // 2),
            "row_scales": _empty(total * C // 16, torch.uint8, dev).view(total, C // 16),
            "col_codes": _empty(total * C // 2, torch.uint8, dev),
            "col_scales": _empty(total * C // 16, torch.uint8, dev),
            "row_outer": _empty(n_ro, torch.float32, dev) if n_ro else None,
            "col_outer": _empty(n_co, torch.float32, dev) if n_co else None,
        }
    for k, n in (("row_codes", total * C // 2), ("row_scales", total * C // 16), ("col_codes", total * C // 2),
                 ("col_scales", total * C // 16), ("row_outer", 4 * n_ro), ("col_outer", 4 * n_co)):
        _need(out.get(k), n, k)
    _need_residual(residual, total, C)
    arr = (ct.c_int64 * max(len(rows), 1))(*rows)
    ws, wsb = _ct_workspace(cfg, rows, C, residual, dev, workspace, staged)
    _check(lib().fp4_cast_transpose_grouped(ct.byref(cfg), len(rows), arr, C, _ptr(x), ld, _ptr(out["row_codes"]),
                                            _ptr(out["row_scales"]), _ptr(out["row_outer"]), _ptr(out["col_codes"]),
                                            _ptr(out["col_scales"]), _ptr(out["col_outer"]), _ptr(residual), _ptr(ws),
                                            wsb, _stream(stream)), "fp4_cast_transpose_grouped")
    return out


def fp4_mx_project_fp8(x, cfg=None, *, y=True, mx8_row=True, mx8_col=True, blk=True, stream=None, out=None):
    """MXFP4 projection of x and its FP8 re-encodings in one pass.  Returns a
    dict with the requested outputs: "y" (bf16 [R, C]); "mx8_row" (uint8 E4M3
    [R, C]) and "mx8_row_scales" (uint8 UE8M0 [R, C/32]); "mx8_col" ([C, R]) and
    "mx8_col_scales" ([C, R/32]); "blk" ([R, C]), "blk_t" ([C, R]) and
    "blk_scales" (float32 [R/128, C/128]).  `out` may supply any of them."""
    torch = _torch()
    x, R, C, ld = _src(x)
    dev = x.device
    cfg = cfg if cfg is not None else make_cfg(format="mxfp4")
    out = dict(out or {})
    want = {"y": (y, (R, C), torch.bfloat16), "mx8_row": (mx8_row, (R, C), torch.uint8),
            "mx8_row_scales": (mx8_row, (R, C // 32), torch.uint8), "mx8_col": (mx8_col, (C, R), torch.uint8),
            "mx8_col_scales": (mx8_col, (C, R // 32), torch.uint8), "blk": (blk, (R, C), torch.uint8),
            "blk_t": (blk, (C, R), torch.uint8), "blk_scales": (blk, (R // 128, C // 128), torch.float32)}
    for k, (on, shp, dt) in want.items():
        if on and out.get(k) is None:
            out[k] = torch.empty(shp, dtype=dt, device=dev)
        if not on:
            out[k] = None
        else:
            _need(out[k], shp[0] * shp[1] * torch.empty((), dtype=dt).element_size(), k)
    g = out.get
    _check(lib().fp4_mx_project_fp8(ct.byref(cfg), _ptr(x), R, C, ld, _ptr(g("y")), _ptr(g("mx8_row")),
                                    _ptr(g("mx8_row_scales")), _ptr(g("mx8_col")), _ptr(g("mx8_col_scales")),
                                    _ptr(g("blk")), _ptr(g("blk_t")), _ptr(g("blk_scales")), _stream(stream)),
           "fp4_mx_project_fp8")
    return {k: v for k, v in out.items() if v is not None}


def fp4q_mx_scales_tiled_bytes(rows, K):
    return lib().fp4q_mx_scales_tiled_bytes(int(rows), int(K))


def fp4_mx_scales_tiled(scales, K, stream=None, out=None):
    """GEMM-ready layout of rowwise MXFP4 scales [rows, K/32] (uint8, flat)."""
    torch = _torch()
    rows = scales.shape[0]
    _need(scales, rows * (K // 32), "scales")
    if out is None:
        out = torch.empty(fp4q_mx_scales_tiled_bytes(rows, K), dtype=torch.uint8, device=scales.device)
    _need(out, fp4q_mx_scales_tiled_bytes(rows, K), "tiled scales")
    _check(lib().fp4_mx_scales_tiled(_ptr(scales), int(rows), int(K), _ptr(out), _stream(stream)),
           "fp4_mx_scales_tiled")
    return out


def fp4_mm(a, b, cfg=None, *, out_dtype=None, c=None, stream=None):
    """C = a @ b^T on the FP4 matrix cores with MXFP4 operands.  a ([M, K]) and
    b ([N, K]) are dicts {"codes", "scales"} as fp4_quantize returns them for
    MXFP4 (rowwise scales), or {"codes", "scales_tiled"} with GEMM-ready
    scales (fp4_mx_scales_tiled), or bf16 / float32 tensors, which are
    quantised and their scales tiled first.  C is bf16 unless out_dtype (or a
    given c) is float32."""
    torch = _torch()
    cfg = cfg if cfg is not None else make_cfg(format="mxfp4")

    def operand(x):
        if isinstance(x, dict):
            if "scales_tiled" in x:
                return x["codes"], x["scales_tiled"], 1
            return x["codes"], x["scales"], 0
        q = fp4_quantize(x, cfg, stream=stream)
        return q["codes"], fp4_mx_scales_tiled(q["scales"], x.shape[1], stream=stream), 1
    ac, asc, la = operand(a)
    bc, bsc, lb = operand(b)
    if la != lb:
        raise ValueError("both operands need the same scale layout")
    M, N, K = ac.shape[0], bc.shape[0], ac.shape[1] * 2
    if bc.shape[1] * 2 != K:
        raise ValueError("operands disagree on K (%d vs %d)" % (K, bc.shape[1] * 2))
    for nm, codes, sc, rows in (("a", ac, asc, M), ("b", bc, bsc, N)):
        _need(codes, rows * K // 2, nm + " codes")
        _need(sc, fp4q_mx_scales_tiled_bytes(rows, K) if la else rows * (K // 32), nm + " scales")
    if c is None:
        c = torch.empty((M, N), dtype=out_dtype if out_dtype is not None else torch.bfloat16, device=ac.device)
    if tuple(c.shape) != (M, N) or (N > 1 and c.stride(1) != 1) or c.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("c must be a bf16 or float32 [%d, %d] view with contiguous rows" % (M, N))
    ccfg = _with_dtypes(cfg, output_dtype=_dtype_name(c))
    _check(lib().fp4_mm(ct.byref(ccfg), _ptr(ac), _ptr(asc), _ptr(bc), _ptr(bsc), M, N, K, la, _ptr(c),
                        c.stride(0) if M > 1 else N, _stream(stream)), "fp4_mm")
    return c


def fp4q_linear_workspace_bytes(M, N, K):
    return lib().fp4q_linear_workspace_bytes(int(M), int(N), int(K))


def fp4_linear(x, w, cfg, *, outer_transposed=False, out_dtype=None, y=None, workspace=None, stream=None):
    """y = x @ W^T with bf16 x [M, K] (a view with a row pitch is accepted) and a
    4-bit W [N, K] given as {"codes", "scales", "outer"} in cfg's format, as fp4_quantize
    returns it (or the row_* buffers of fp4_cast_transpose under those names).  Outer scales: none,
    one for the tensor, 64 x 64 tiles, or row segments of a multiple of 64.

    The gradient of x is the same product over the columnwise buffers: with
    w = {"codes": col_codes [K, N / 2], "scales": col_scales, "outer": ...} and dy [M, N] in
    x's place it returns dy @ W [M, K]; a 2D outer array is passed as it is, with
    outer_transposed=True.  y is bf16 unless out_dtype (or a given y) is float32.
    workspace: a tensor of at least fp4q_linear_workspace_bytes(M, N, K) bytes, else one is
    allocated where it is needed."""
    torch = _torch()
    codes, scales, outer = w["codes"], w["scales"], w.get("outer")
    if x.dtype != torch.bfloat16:
        raise Fp4Error(ERR_DTYPE, "x dtype %s" % x.dtype)
    if x.dim() != 2 or codes.dim() != 2:
        raise ValueError("x and the weight's codes must be 2-D")
    (M, K), N = x.shape, codes.shape[0]
    if codes.element_size() != 1 or scales.element_size() != 1:
        raise ValueError("codes and scales must hold bytes, got %s and %s" % (codes.dtype, scales.dtype))
    if codes.shape[1] * 2 != K:
        raise ValueError("x and the weight disagree on K (%d vs %d)" % (K, codes.shape[1] * 2))
    if K > 1 and x.stride(1) != 1:
        raise ValueError("x rows must be contiguous (stride(1) == 1)")
    _need(codes, N * K // 2, "codes")
    _need(scales, N * (K // _inner(cfg)), "scales")
    if cfg.two_level == TWO_LEVEL["tensorwise"]:
        _need(outer, 4, "outer")
    elif cfg.two_level == TWO_LEVEL["outer_block"] and cfg.outer_block_size > 0:
        _need(outer, 4 * (N // (cfg.outer_block_size if cfg.outer_2d else 1)) * (K // cfg.outer_block_size), "outer")
    if outer is not None and outer.dtype != torch.float32:
        raise ValueError("outer must be float32")
    dev = x.device
    if not x.is_cuda:
        raise ValueError("fp4q takes device tensors; got one on %s" % dev)
    if codes.device != dev or scales.device != dev or (outer is not None and outer.device != dev):
        raise ValueError("x and the weight must be on one device")
    if y is None:
        y = _new((M, N), out_dtype if out_dtype is not None else torch.bfloat16, dev, stream)
    elif tuple(y.shape) != (M, N) or (N > 1 and y.stride(1) != 1) or y.device != dev:
        raise ValueError("y must be a [%d, %d] view with contiguous rows on %s" % (M, N, dev))
    if y.dtype not in (torch.bfloat16, torch.float32):
        raise Fp4Error(ERR_DTYPE, "y dtype %s" % y.dtype)
    if workspace is None:
        need = lib().fp4q_linear_workspace_bytes(M, N, K)
        if need:
            workspace = _new(need, torch.uint8, dev, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on %s" % dev)
    size, scratch = (0, None) if workspace is None else (workspace.nbytes, workspace.data_ptr())
    ycfg = _with_dtypes(cfg, "bf16", _dtype_name(y))
    _launch("fp4_linear", lib().fp4_linear, dev, ct.byref(ycfg), x.data_ptr(), M, x.stride(0) if M > 1 else K,
            codes.data_ptr(), scales.data_ptr(), None if outer is None else outer.data_ptr(), 1 if outer_transposed else 0, N,
            K, y.data_ptr(), y.stride(0) if M > 1 else N, scratch, size, _raw_stream(stream, dev))
    return y


# ------------------------------------------------------------------ the paged 4-bit cache
# Single tokens make these calls every few microseconds, so they are marshalled with what costs
# least: plain addresses (checked to be on the cache's device), configurations and structures
# built once for a cache, and the stream's raw handle.
def _new(shape, dtype, device, stream):
    """A tensor that work on `stream` writes.  It is that stream's own memory (what the current
    stream has freed may still be written by its queued work), and once it is freed it stays
    reserved until what the current stream has queued by then is done."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _raw_stream(stream, device):
    if stream is None:
        return _torch()._C._cuda_getCurrentRawStream(device.index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _heads_rows(t, heads, dim, what, dtypes):
    """Token pitch of a [tokens, heads, dim] tensor whose tokens are whole runs."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError("%s must be [tokens, %d, %d], got %s" % (what, heads, dim, tuple(shape)))
    if t.dtype not in dtypes:
        raise Fp4Error(ERR_DTYPE, "%s dtype %s" % (what, t.dtype))
    s0, s1, s2 = t.stride()
    if shape[0] and (s2 != 1 or (heads > 1 and s1 != dim)):
        raise ValueError("%s: a token's heads must be contiguous" % what)
    return s0 if shape[0] > 1 else heads * dim


def _ints(t, dtype, rows, cols, what, device):
    """t: [rows] (cols None) or [rows, any], rows None: any."""
    shape = t.shape
    if t.dtype != dtype or len(shape) != (1 if cols is None else 2) or (rows is not None and shape[0] != rows):
        raise ValueError("%s must be %s [%s%s], got %s %s" % (what, dtype, "n" if rows is None else rows,
                                                              "" if cols is None else ", cols", t.dtype, list(shape)))
    if not t.is_contiguous() or t.device != device:
        raise ValueError("%s must be contiguous and on %s" % (what, device))


def _ints32(where, *values):
    """The structures' 32-bit fields would take larger integers modulo 2^32."""
    if max(values) > 0x7FFFFFFF or min(values) < -0x80000000:
        raise Fp4Error(ERR_UNSUPPORTED, "%s: %s" % (where, values))


def _launch(where, entry, device, *args):
    """Calls a C entry point with the tensors' device current: its kernels start there."""
    torch = _torch()
    if torch._C._cuda_getDevice() == device.index:
        st = entry(*args)
    else:
        with torch.cuda.device(device):
            st = entry(*args)
    _check(st, where)


class KVCache:
    """The paged 4-bit cache of one layer's keys and values (layout and rules
    in include/fp4q.h): uint8 codes [pages, kv_heads, page_size, head_dim / 2]
    and scales [pages, kv_heads, page_size, head_dim / 16] (/ 32 for MXFP4), and with
    cfg two_level "tensorwise", outer_mode 1, the calibrated float32 scales k_outer and v_outer
    [kv_heads].  The tensors are the caller's; KVCache.empty() allocates them."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, cfg, *, k_outer=None, v_outer=None):
        torch = _torch()
        if k_codes.dim() != 4:
            raise ValueError("codes must be [pages, kv_heads, page_size, head_dim / 2]")
        pages, heads, page, half = k_codes.shape
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, half * 2
        self.cfg = Cfg.from_buffer_copy(cfg)
        self.device = k_codes.device
        self._by_dtype = {torch.bfloat16: ct.byref(_with_dtypes(cfg, "bf16", "bf16")),
                          torch.float32: ct.byref(_with_dtypes(cfg, "fp32", "fp32"))}
        shapes = {"k_codes": half, "v_codes": half, "k_scales": half * 2 // _inner(cfg),
                  "v_scales": half * 2 // _inner(cfg)}
        for n, t in (("k_codes", k_codes), ("k_scales", k_scales), ("v_codes", v_codes), ("v_scales", v_scales)):
            want = (pages, heads, page, shapes[n])
            if tuple(t.shape) != want or t.dtype != torch.uint8 or not t.is_contiguous() or t.device != self.device:
                raise ValueError("%s must be a contiguous uint8 %s on %s" % (n, list(want), self.device))
        for n, t in (("k_outer", k_outer), ("v_outer", v_outer)):
            if t is not None and (tuple(t.shape) != (heads,) or t.dtype != torch.float32 or not t.is_contiguous()
                                  or t.device != self.device):
                raise ValueError("%s must be a contiguous float32 [%d] on %s" % (n, heads, self.device))
        if (k_outer is None) != (v_outer is None) or (k_outer is not None) != (cfg.two_level == TWO_LEVEL["tensorwise"]):
            raise ValueError("k_outer and v_outer go with cfg two_level 'tensorwise' (outer_mode 1), and only with it")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.k_outer, self.v_outer = k_outer, v_outer
        self._c = _KvCache(_ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), _ptr(k_outer), _ptr(v_outer),
                           pages, page, heads, half * 2, 0)
        self._ref = ct.byref(self._c)

    @classmethod
    def empty(cls, num_pages, page_size, kv_heads, head_dim, cfg, *, device="cuda", k_outer=None, v_outer=None):
        """A cache of zeros."""
        torch = _torch()
        codes, scales = ((num_pages, kv_heads, page_size, n) for n in (head_dim // 2, head_dim // _inner(cfg)))
        z = [torch.zeros(s, dtype=torch.uint8, device=device) for s in (codes, scales, codes, scales)]
        return cls(*z, cfg, k_outer=k_outer, v_outer=v_outer)


def fp4_kv_append(cache, k, v, slots, *, stream=None):
    """Quantises k and v (bf16 or float32 [tokens, kv_heads, head_dim]; views with a
    token pitch are accepted) into the cache's slots (int64 [tokens], page *
    page_size + place; a slot outside the cache writes nothing)."""
    torch, dev = _torch(), cache.device
    types = (torch.bfloat16, torch.float32)
    ld_k = _heads_rows(k, cache.kv_heads, cache.head_dim, "k", types)
    ld_v = _heads_rows(v, cache.kv_heads, cache.head_dim, "v", types)
    n = k.shape[0]
    if k.dtype != v.dtype or v.shape[0] != n or k.device != dev or v.device != dev:
        raise ValueError("k and v must agree in shape and dtype and lie on the cache's device")
    _ints(slots, torch.int64, n, None, "slots", dev)
    _launch("fp4_kv_append", lib().fp4_kv_append, dev, cache._by_dtype[k.dtype], cache._ref, k.data_ptr(), ld_k, v.data_ptr(),
            ld_v, slots.data_ptr(), n, _raw_stream(stream, dev))


def _same_device(device, **tensors):
    for n, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError("%s must be on %s, got %s" % (n, device, t.device))


def fp4_kv_append_rope(cache, k, v, slots, positions, cos, sin, *, q=None, q_out=None, interleaved=False, stream=None):
    """fp4_kv_append of keys that are turned by their positions on the way; returns the
    queries of the same tokens turned too, or None without q (see include/fp4q.h).

    k, v, slots  as in fp4_kv_append; q: their dtype, [tokens, q_heads, head_dim], a view with a token
                 pitch is accepted.
    positions    int32 [tokens]: a token's row of the tables.  A token whose position lies outside them
                 is padding: nothing is cached for it, and its queries come back as zeros.
    cos, sin     float32 [rows, rot_dim / 2]; the first rot_dim values of a head (a multiple of 16) turn.
    interleaved  pairs are values 2 j and 2 j + 1 of a head; else j and j + rot_dim / 2.
    q_out        where the queries go; q itself turns them in place."""
    torch, dev = _torch(), cache.device
    types = (torch.bfloat16, torch.float32)
    ld_k = _heads_rows(k, cache.kv_heads, cache.head_dim, "k", types)
    ld_v = _heads_rows(v, cache.kv_heads, cache.head_dim, "v", types)
    n = k.shape[0]
    if k.dtype != v.dtype or v.shape[0] != n or k.device != dev or v.device != dev:
        raise ValueError("k and v must agree in shape and dtype and lie on the cache's device")
    _ints(slots, torch.int64, n, None, "slots", dev)
    _ints(positions, torch.int32, n, None, "positions", dev)
    if (cos.dim() != 2 or cos.shape != sin.shape or cos.dtype != torch.float32 or sin.dtype != torch.float32
            or not cos.is_contiguous() or not sin.is_contiguous()):
        raise ValueError("cos and sin must be contiguous float32 [rows, rot_dim / 2]")
    _same_device(dev, cos=cos, sin=sin, q=q, q_out=q_out)
    ld_q = ld_out = q_heads = 0
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
    else:
        if q.dim() != 3:
            raise ValueError("q must be [tokens, q_heads, head_dim]")
        q_heads = q.shape[1]
        ld_q = _heads_rows(q, q_heads, cache.head_dim, "q", (k.dtype,))
        if q_out is None:
            q_out = _new((n, q_heads, cache.head_dim), q.dtype, dev, stream)
        ld_out = _heads_rows(q_out, q_heads, cache.head_dim, "q_out", (k.dtype,))
        if q.shape[0] != n or q_out.shape[0] != n:
            raise ValueError("q and q_out must hold the %d tokens of k" % n)
    _ints32("fp4_kv_append_rope", q_heads, 2 * cos.shape[1])
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    a = _KvRope(k.data_ptr(), v.data_ptr(), p(q), p(q_out), ld_k, ld_v, ld_q, ld_out, slots.data_ptr(), positions.data_ptr(),
                cos.data_ptr(), sin.data_ptr(), n, cos.shape[0], 2 * cos.shape[1], q_heads, 1 if interleaved else 0, 0)
    _launch("fp4_kv_append_rope", lib().fp4_kv_append_rope, dev, cache._by_dtype[k.dtype], cache._ref, ct.byref(a),
            _raw_stream(stream, dev))
    return q_out


def fp4_kv_read(cache, slots, *, dtype=None, stream=None, out=None):
    """(k, v): bf16 (or float32: dtype) [tokens, kv_heads, head_dim] that the
    cache holds at slots (int64 [tokens]; zeros for one outside the cache).  `out` may supply
    the pair."""
    torch, dev = _torch(), cache.device
    n = slots.shape[0] if slots.dim() else 0
    _ints(slots, torch.int64, None, None, "slots", dev)
    shape = (n, cache.kv_heads, cache.head_dim)
    if out is None:
        dtype = dtype if dtype is not None else torch.bfloat16
        k, v = (_new(shape, dtype, dev, stream) for _ in "kv")
    else:
        k, v = out
        for t in (k, v):
            if tuple(t.shape) != shape or t.dtype != k.dtype or not t.is_contiguous() or t.device != dev:
                raise ValueError("out must be two contiguous %s tensors of one dtype" % list(shape))
    cfg = cache._by_dtype.get(k.dtype)
    if cfg is None:
        raise Fp4Error(ERR_DTYPE, "k dtype %s" % k.dtype)
    _launch("fp4_kv_read", lib().fp4_kv_read, dev, cfg, cache._ref, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(),
            _raw_stream(stream, dev))
    return k, v


def fp4_attn_workspace(cache, total_q, q_heads, batch, *, max_q=None, max_kv=None, table_cols=None, window=0, trees=None):
    """Scratch for fp4_attn and fp4_attn_tree calls of this size (None if they need none), to keep
    between calls.  max_q, max_kv, window and table_cols as in the call; without
    table_cols, the columns that max_kv needs.  trees: False sizes it for fp4_attn alone and True for
    fp4_attn_tree alone, which cuts keys that fp4_attn does not (a prompt of 1024 tokens, 64 / 8 heads of 128: None
    and 68 MB); None for both."""
    torch = _torch()
    if max_kv is None and table_cols is None:
        raise ValueError("give max_kv or table_cols")
    if table_cols is None:
        table_cols = -(-int(max_kv) // cache.page_size)
    n = [int(v) for v in (batch, total_q, q_heads, table_cols, total_q if max_q is None else max_q,
                          table_cols * cache.page_size if max_kv is None else max_kv, window)]
    _ints32("fp4_attn_workspace", *n)
    a = _Attn(batch=n[0], total_q=n[1], q_heads=n[2], table_cols=n[3], max_q=n[4], max_kv=n[5], causal=1, window=n[6],
              scale=1.0, ld_q=n[2] * cache.head_dim, q_starts=16)
    sizes = {False: lib().fp4q_attn_workspace_bytes, True: lib().fp4q_attn_tree_workspace_bytes}
    n = max(f(ct.byref(cache.cfg), cache._ref, ct.byref(a)) for t, f in sizes.items() if trees is None or t == bool(trees))
    return torch.empty(n, dtype=torch.uint8, device=cache.device) if n else None


def _attention(tree, q, cache, page_table, kv_lens, q_starts, max_q, max_kv, scale, causal, window, sinks, out, out_dtype, with_lse,
               workspace, stream):
    """fp4_attn, or fp4_attn_tree with its (checked) mask."""
    torch = _torch()
    if q.dim() != 3:
        raise ValueError("q must be [tokens, q_heads, head_dim]")
    T, Hq, D = q.shape
    ld = _heads_rows(q, Hq, cache.head_dim, "q", (torch.bfloat16,))
    dev = cache.device
    if q.device != dev:
        raise ValueError("q must be on the cache's device")
    _ints(kv_lens, torch.int32, None, None, "kv_lens", dev)
    batch = kv_lens.shape[0]
    _ints(page_table, torch.int32, batch, True, "page_table", dev)
    if q_starts is not None:
        _ints(q_starts, torch.int32, batch + 1, None, "q_starts", dev)
    elif T != batch:
        raise ValueError("without q_starts, q holds one query for each of the %d sequences, got %d" % (batch, T))
    if sinks is not None and (sinks.dtype != torch.float32 or tuple(sinks.shape) != (Hq,) or not sinks.is_contiguous()
                              or sinks.device != dev):
        raise ValueError("sinks must be a contiguous float32 [%d] on %s" % (Hq, dev))
    if out is None:
        out = _new((T, Hq, D), out_dtype if out_dtype is not None else torch.bfloat16, dev, stream)
    elif tuple(out.shape) != (T, Hq, D) or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must be a contiguous %s on %s" % ([T, Hq, D], dev))
    cfg = cache._by_dtype.get(out.dtype)
    if cfg is None:
        raise Fp4Error(ERR_DTYPE, "out dtype %s" % out.dtype)
    lse = _new((T, Hq), torch.float32, dev, stream) if with_lse else None
    cols = page_table.shape[1]
    if max_q is None:
        max_q = 1 if q_starts is None else T
    if max_kv is None:
        max_kv = cols * cache.page_size
    _ints32("fp4_attn", max_q, max_kv, window)
    a = ct.byref(_Attn(q.data_ptr(), ld, page_table.data_ptr(), kv_lens.data_ptr(),
                       None if q_starts is None else q_starts.data_ptr(), None if sinks is None else sinks.data_ptr(),
                       out.data_ptr(), None if lse is None else lse.data_ptr(),
                       D ** -0.5 if scale is None else scale, batch, T, Hq, cols, max_q, max_kv, 1 if causal else 0,
                       window))
    if workspace is None:
        need = (lib().fp4q_attn_workspace_bytes if tree is None else lib().fp4q_attn_tree_workspace_bytes)(cfg, cache._ref, a)
        if need:
            workspace = _new(need, torch.uint8, dev, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on %s" % dev)
    size, scratch = (0, None) if workspace is None else (workspace.nbytes, workspace.data_ptr())
    if tree is None:
        _launch("fp4_attn", lib().fp4_attn, dev, cfg, cache._ref, a, scratch, size, _raw_stream(stream, dev))
    else:
        _launch("fp4_attn_tree", lib().fp4_attn_tree, dev, cfg, cache._ref, a, tree.data_ptr(), tree.shape[1], scratch,
                size, _raw_stream(stream, dev))
    return (out, lse) if with_lse else out


def fp4_attn(q, cache, page_table, kv_lens, q_starts=None, *, max_q=None, max_kv=None, scale=None, causal=True, window=0,
             sinks=None, out=None, out_dtype=None, with_lse=False, workspace=None, stream=None):
    """Attention of q (bf16 [tokens, q_heads, head_dim]) over the cache (see
    include/fp4q.h for masks, limits and rounding).

    page_table   int32 [batch, cols], kv_lens int32 [batch] on the device.
    q_starts     int32 [batch + 1]: sequence b's queries are q[q_starts[b]:
                 q_starts[b + 1]]; None: one query each.
    max_q, max_kv  bounds of the sequences' query and key counts (default: all of q,
                 all that the page table can name); tight ones make better launches.
    scale        of q . k, default head_dim ** -0.5.
    window       > 0: each query sees at most that many keys, up to its own.
    sinks        float32 [q_heads]: a logit that joins each row's softmax.
    Returns out (bf16, or out_dtype float32, which also keeps twice the bits of the
    weights), or (out, lse) with with_lse."""
    return _attention(None, q, cache, page_table, kv_lens, q_starts, max_q, max_kv, scale, causal, window, sinks, out, out_dtype,
                      with_lse, workspace, stream)


def fp4_attn_tree(q, cache, page_table, kv_lens, q_starts, tree, *, max_q=None, max_kv=None, scale=None, window=0, sinks=None,
                  out=None, out_dtype=None, with_lse=False, workspace=None, stream=None):
    """fp4_attn of trees of drafted tokens: each sequence's queries are the nodes of its tree, and
    their keys are the last of its kv_lens.

    tree   bool (or uint8) [tokens, cols]: row i names the drafted keys of its sequence that query i sees,
           by their place in the tree (its ancestors and itself); all see the whole context before them, or
           with a window as much of it as makes the window full.
    Other arguments (but causal) and results as in fp4_attn; fp4_attn_workspace sizes these calls too."""
    torch = _torch()
    if tree.dim() != 2 or tree.shape[0] != q.shape[0] or tree.dtype not in (torch.bool, torch.uint8):
        raise ValueError("tree must be bool or uint8 [%d, cols], got %s %s" % (q.shape[0], tree.dtype, list(tree.shape)))
    if not tree.is_contiguous() or tree.device != cache.device:
        raise ValueError("tree must be contiguous and on %s" % cache.device)
    _ints32("fp4_attn_tree", tree.shape[1])
    return _attention(tree, q, cache, page_table, kv_lens, q_starts, max_q, max_kv, scale, True, window, sinks, out, out_dtype,
                      with_lse, workspace, stream)


# ------------------------------------------------------------------ mixture of experts
def fp4q_moe_workspace_bytes(tokens, experts, top_k, hidden, inter):
    return lib().fp4q_moe_workspace_bytes(int(tokens), int(experts), int(top_k), int(hidden), int(inter))


def fp4_moe_workspace(tokens, experts, top_k, hidden, inter, *, device="cuda"):
    """Scratch for fp4_moe calls of this size, to keep between calls (one call at a time)."""
    torch = _torch()
    return torch.empty(fp4q_moe_workspace_bytes(tokens, experts, top_k, hidden, inter), dtype=torch.uint8, device=device)


def _expert_weight(w, what, experts, rows, cols, cfg, device):
    """Addresses of stacked experts' codes, scale bytes and outer scales."""
    codes, scales, outer = w["codes"], w["scales"], w.get("outer")
    if codes.element_size() != 1 or scales.element_size() != 1:
        raise ValueError("%s codes and scales must hold bytes, got %s and %s" % (what, codes.dtype, scales.dtype))
    if codes.numel() != experts * rows * cols // 2:
        raise ValueError("%s codes must be [%d, %d, %d], got %s" % (what, experts, rows, cols // 2, list(codes.shape)))
    _need(codes, experts * rows * cols // 2, what + " codes")
    _need(scales, experts * rows * (cols // _inner(cfg)), what + " scales")
    n = 0
    if cfg.two_level == TWO_LEVEL["tensorwise"]:
        n = experts
    elif cfg.two_level == TWO_LEVEL["outer_block"] and cfg.outer_block_size > 0:
        n = experts * rows * (cols // cfg.outer_block_size) // (cfg.outer_block_size if cfg.outer_2d else 1)
    if n:
        if outer is None:
            raise ValueError("%s needs outer scales" % what)
        if outer.dtype != _torch().float32:
            raise ValueError("%s outer must be float32" % what)
        _need(outer, 4 * n, what + " outer")
    for t in (codes, scales, outer):
        if t is not None and t.device != device:
            raise ValueError("%s must be on %s" % (what, device))
    return codes.data_ptr(), scales.data_ptr(), None if outer is None else outer.data_ptr()


def fp4_moe(x, logits, w1, w2, cfg, *, top_k, renormalize=True, b1=None, b2=None, interleaved=False, alpha=1.0, limit=None,
            shift=0.0, out_dtype=None, y=None, workspace=None, stream=None):
    """A mixture-of-experts layer with 4-bit experts for a few tokens (64 at a time, at most 1024), from the
    router's logits (see include/fp4q.h for ties, empty rows, rounding and limits).

    x            bf16 [tokens, hidden], a view with a row pitch is accepted; logits float32 [tokens, experts].
    w1, w2       {"codes", "scales", "outer"} of the stacked experts in cfg's format: gate and up rows [experts * 2 inter,
                 hidden] and [experts * hidden, inter], in these shapes or any others of the same memory.
                 Outer scales as in fp4_linear, but one for each expert where cfg is "tensorwise".
    top_k        experts of a token, by the largest logits; renormalize: shares are the softmax of those,
                 else of all logits.
    b1, b2       float32 [experts, 2 inter] and [experts, hidden], or None.
    interleaved  gate and up rows alternate; else each expert's gate rows come first.
    alpha, limit, shift  g sigmoid(alpha g) (u + shift), with g at most limit and u within +-limit first.
    Returns y [tokens, hidden], bf16 unless out_dtype (or a given y) is float32.  workspace: from
    fp4_moe_workspace, else one is allocated."""
    torch = _torch()
    if x.dtype != torch.bfloat16:
        raise Fp4Error(ERR_DTYPE, "x dtype %s" % x.dtype)
    if x.dim() != 2 or logits.dim() != 2 or logits.shape[0] != x.shape[0]:
        raise ValueError("x must be [tokens, hidden] and logits [tokens, experts]")
    (T, H), E, dev = x.shape, logits.shape[1], x.device
    if H > 1 and x.stride(1) != 1:
        raise ValueError("x rows must be contiguous (stride(1) == 1)")
    if logits.dtype != torch.float32 or not logits.is_contiguous():
        raise ValueError("logits must be contiguous float32")
    if not E or not H or (w2["codes"].numel() * 2) % (E * H):
        raise ValueError("w2 codes do not hold %d experts of %d rows" % (E, H))
    inter = w2["codes"].numel() * 2 // (E * H)
    p1 = _expert_weight(w1, "w1", E, 2 * inter, H, cfg, dev)
    p2 = _expert_weight(w2, "w2", E, H, inter, cfg, dev)
    for n, t, shape in (("b1", b1, (E, 2 * inter)), ("b2", b2, (E, H))):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shape or not t.is_contiguous()):
            raise ValueError("%s must be a contiguous float32 %s" % (n, list(shape)))
    if not x.is_cuda:
        raise ValueError("fp4q takes device tensors; got one on %s" % dev)
    _same_device(dev, logits=logits, b1=b1, b2=b2, y=y, workspace=workspace)
    if y is None:
        y = _new((T, H), out_dtype if out_dtype is not None else torch.bfloat16, dev, stream)
    elif tuple(y.shape) != (T, H) or (H > 1 and y.stride(1) != 1):
        raise ValueError("y must be a [%d, %d] view with contiguous rows" % (T, H))
    if y.dtype not in (torch.bfloat16, torch.float32):
        raise Fp4Error(ERR_DTYPE, "y dtype %s" % y.dtype)
    if workspace is None:
        workspace = _new(lib().fp4q_moe_workspace_bytes(T, E, top_k, H, inter), torch.uint8, dev, stream)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _ints32("fp4_moe", top_k)
    a = _Moe(x.data_ptr(), x.stride(0) if T > 1 else H, logits.data_ptr(), *p1, *p2, None if b1 is None else b1.data_ptr(),
             None if b2 is None else b2.data_ptr(), y.data_ptr(), y.stride(0) if T > 1 else H, T, E, H, inter, top_k,
             1 if renormalize else 0, 1 if interleaved else 0, 0, alpha, 0.0 if limit is None else limit, shift)
    ycfg = _with_dtypes(cfg, "bf16", _dtype_name(y))
    _launch("fp4_moe", lib().fp4_moe, dev, ct.byref(ycfg), ct.byref(a), workspace.data_ptr(), workspace.nbytes,
            _raw_stream(stream, dev))
    return y


# ------------------------------------------------------------------ residual and norm
_FP8_MODES = {None: 0, "mx": 1, "row": 2}


def _norm_rows(t, shape, what, types):
    """Row pitch of a [rows, hidden] bf16 or float32 tensor whose rows are contiguous."""
    if t.dtype not in types:
        raise Fp4Error(ERR_DTYPE, "%s dtype %s" % (what, t.dtype))
    got = t.shape
    if len(got) != 2 or (shape is not None and got != shape):
        raise ValueError("%s must be %s, got %s" % (what, "2-D" if shape is None else list(shape), list(got)))
    rows, hidden = got
    ld, step = t.stride()
    if rows and hidden > 1 and step != 1:
        raise ValueError("%s rows must be contiguous (stride(1) == 1)" % what)
    return ld if rows > 1 else hidden


def _norm_weight(weight, hidden, types):
    if weight.dtype not in types:
        raise Fp4Error(ERR_DTYPE, "weight dtype %s" % weight.dtype)
    if weight.shape != (hidden,) or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous [%d]" % hidden)


def _out(t, shape, dtype, device, what, stream):
    """A given output, checked, or a new one."""
    if t is None:
        return _new(shape, dtype, device, stream)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous() or t.device != device:
        raise ValueError("%s must be a contiguous %s %s on %s" % (what, dtype, list(shape), device))
    return t


def fp4_add_rms_norm(x, weight, residual=None, *, eps=1e-6, fp8=None, y=None, y_dtype=None, out=None, stream=None):
    """h = x + residual and its root-mean-square norm times weight, in bf16 or float32, in 8 bits with
    scales, or both (see include/fp4q.h for the rounding).

    x, residual  bf16 or float32 [rows, hidden], each its own; views with a row pitch are accepted.
    fp8          None, "mx" (E4M3 with a UE8M0 scale byte for 32 values) or "row" (a float32
                 scale a row).
    y            whether the norm itself is returned; by default where fp8 is None.  y_dtype: bf16, or
                 float32.
    out          may supply any result; "residual" may be the given residual.
    Returns {"residual": h in residual's dtype (x itself without one), "rstd": float32 [rows], "y", "fp8": uint8
    [rows, hidden], "fp8_scales": uint8 [rows, hidden / 32] or float32 [rows]}; what was not asked for
    is None."""
    torch = _torch()
    types = (torch.bfloat16, torch.float32)
    if fp8 not in _FP8_MODES:
        raise ValueError("fp8 must be None, 'mx' or 'row', got %r" % (fp8,))
    ld_x = _norm_rows(x, None, "x", types)
    (rows, hidden), dev = x.shape, x.device
    if not x.is_cuda:
        raise ValueError("fp4q takes device tensors; got one on %s" % dev)
    ld_r = 0 if residual is None else _norm_rows(residual, x.shape, "residual", types)
    _norm_weight(weight, hidden, types)
    _same_device(dev, weight=weight, residual=residual)
    given = out or {}
    if y is None:
        y = fp8 is None
    y_dtype = y_dtype if y_dtype is not None else torch.bfloat16
    if y_dtype not in types:
        raise Fp4Error(ERR_DTYPE, "y dtype %s" % y_dtype)
    res = dict(residual=x, y=None, fp8=None, fp8_scales=None)
    if residual is not None:
        res["residual"] = _out(given.get("residual"), (rows, hidden), residual.dtype, dev, "residual", stream)
    res["rstd"] = _out(given.get("rstd"), (rows,), torch.float32, dev, "rstd", stream)
    if y:
        res["y"] = _out(given.get("y"), (rows, hidden), y_dtype, dev, "y", stream)
    if fp8 is not None:
        res["fp8"] = _out(given.get("fp8"), (rows, hidden), torch.uint8, dev, "fp8", stream)
        res["fp8_scales"] = _out(given.get("fp8_scales"), (rows, hidden // 32) if fp8 == "mx" else (rows,),
                                 torch.uint8 if fp8 == "mx" else torch.float32, dev, "fp8_scales", stream)
    kind = {torch.bfloat16: 0, torch.float32: 2}
    added = residual is not None
    a = _AddRmsNorm(x.data_ptr(), residual.data_ptr() if added else None, ld_x, ld_r, weight.data_ptr(),
                    res["residual"].data_ptr() if added else None, res["rstd"].data_ptr(), res["y"].data_ptr() if y else None,
                    res["fp8"].data_ptr() if fp8 else None, res["fp8_scales"].data_ptr() if fp8 else None, rows, hidden, eps,
                    kind[x.dtype], kind[residual.dtype] if added else 0, kind[weight.dtype], kind[y_dtype], _FP8_MODES[fp8], 0)
    _launch("fp4_add_rms_norm", lib().fp4_add_rms_norm, dev, ct.byref(a), _raw_stream(stream, dev))
    return res


def fp4q_add_rms_norm_backward_workspace_bytes(rows, hidden):
    return lib().fp4q_add_rms_norm_backward_workspace_bytes(int(rows), int(hidden))


def fp4_add_rms_norm_backward(dy, h, weight, rstd, *, dresidual=None, dx=None, dweight=None, workspace=None, stream=None):
    """The gradient of fp4_add_rms_norm from dy (that of y; bf16 or float32), what the call returned as
    "residual" (h) and "rstd", and dresidual, the gradient of "residual" (h's dtype; None: zero).
    Returns {"dx": the gradient of x, and of the residual, in h's dtype, "dweight": float32 [hidden]}.
    dx may be dresidual.  workspace: at least fp4q_add_rms_norm_backward_workspace_bytes(rows, hidden) bytes,
    else one is allocated where it is needed."""
    torch = _torch()
    types = (torch.bfloat16, torch.float32)
    ld_h = _norm_rows(h, None, "h", types)
    (rows, hidden), dev = h.shape, h.device
    if not h.is_cuda:
        raise ValueError("fp4q takes device tensors; got one on %s" % dev)
    ld_dy = _norm_rows(dy, h.shape, "dy", types)
    ld_dr = 0 if dresidual is None else _norm_rows(dresidual, h.shape, "dresidual", (h.dtype,))
    _norm_weight(weight, hidden, types)
    if rstd.dtype != torch.float32 or tuple(rstd.shape) != (rows,) or not rstd.is_contiguous():
        raise ValueError("rstd must be a contiguous float32 [%d]" % rows)
    _same_device(dev, dy=dy, weight=weight, rstd=rstd, dresidual=dresidual, workspace=workspace)
    dx = _out(dx, (rows, hidden), h.dtype, dev, "dx", stream)
    dweight = _out(dweight, (hidden,), torch.float32, dev, "dweight", stream)
    if workspace is None:
        need = lib().fp4q_add_rms_norm_backward_workspace_bytes(rows, hidden)
        if need:
            workspace = _new(need, torch.uint8, dev, stream)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    size, scratch = (0, None) if workspace is None else (workspace.nbytes, workspace.data_ptr())
    f32 = lambda t: 2 if t.dtype == torch.float32 else 0  # noqa: E731
    a = _RmsNormGrad(dy.data_ptr(), h.data_ptr(), None if dresidual is None else dresidual.data_ptr(), ld_dy, ld_h, ld_dr,
                     weight.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dweight.data_ptr(), rows, hidden, f32(dy), f32(h),
                     f32(weight), 0)
    _launch("fp4_add_rms_norm_backward", lib().fp4_add_rms_norm_backward, dev, ct.byref(a), scratch, size,
            _raw_stream(stream, dev))
    return {"dx": dx, "dweight": dweight}


class ErrorFeedback:
    """Per-tensor error-feedback state for quantised weights ("fp4-train"
    README, API: ErrorFeedback; Method: error feedback carries each step's
    quantisation error into the next step's value).

    One FP32 residual per name, created as zeros on the first call with the
    tensor's shape and device.  qdq(name, w, step) quantises RN(w + residual)
    and returns the dequantised tensor (w's dtype); the same kernel rewrites the
    residual in place with RN(value - dequantised value).  quantize() does the
    same and returns the packed codes and scales instead.  `step` is the
    stochastic-rounding counter of that call.  NVFP4 / AMD-FP4 only (MXFP4 has
    no error-feedback path).
    """

    def __init__(self, cfg=None, *, stochastic=False, seed=0, **cfg_kw):
        if cfg is None:
            cfg = make_cfg(rounding="stochastic" if stochastic else "rne", seed=seed, **cfg_kw)
        elif cfg_kw or stochastic or seed:
            raise ValueError("pass either cfg or its keyword settings, not both")
        if cfg.format == FORMATS["mxfp4"]:
            raise Fp4Error(ERR_UNSUPPORTED, "ErrorFeedback with MXFP4")
        self.cfg = cfg
        self._res = {}

    def _cfg(self, step):
        c = Cfg.from_buffer_copy(self.cfg)
        c.step = int(step)
        return c

    def residual(self, name, like=None):
        """The residual of `name` (created as zeros shaped like `like`)."""
        r = self._res.get(name)
        if r is None:
            if like is None:
                raise KeyError(name)
            torch = _torch()
            r = torch.zeros(like.shape, dtype=torch.float32, device=like.device)
            self._res[name] = r
        elif like is not None and (tuple(r.shape) != tuple(like.shape) or r.device != like.device):
            raise ValueError("residual of %r is %s on %s, tensor is %s on %s"
                             % (name, tuple(r.shape), r.device, tuple(like.shape), like.device))
        return r

    def qdq(self, name, w, step=0, **kw):
        return fp4_qdq(w, self._cfg(step), residual=self.residual(name, w), **kw)["y"]

    def quantize(self, name, w, step=0, **kw):
        return fp4_quantize(w, self._cfg(step), residual=self.residual(name, w), **kw)

    def reset(self, name=None):
        """Forget one residual (or all of them)."""
        if name is None:
            self._res.clear()
        else:
            self._res.pop(name, None)

    def state_dict(self):
        return {k: v.clone() for k, v in self._res.items()}

    def load_state_dict(self, state):
        torch = _torch()
        for k, v in state.items():
            if v.dtype != torch.float32 or v.dim() != 2:
                raise ValueError("residual %r must be a 2-D float32 tensor" % k)
        self._res = {k: v.clone().contiguous() for k, v in state.items()}
