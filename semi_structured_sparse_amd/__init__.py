"""Python binding of libnmsparse (N:M structured-sparse linear layers on MI355X / gfx950).

Thin ctypes layer: every function has the name of the C entry point it calls and only
marshals arguments (device pointers, sizes, leading dimensions, the current HIP stream).
All arithmetic runs in the library's HIP kernels.  torch tensors serve as device memory:
bf16 data may be any 2-byte dtype (torch.bfloat16, int16, uint16 holding bf16 bits).

The library must have been built (``semi_structured_sparse_amd.build.build()``); there is
no fallback: importing the binding without the shared library raises ImportError.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "NMError", "lib", "NM_OK", "NM_EINVAL", "NM_ESHAPE", "NM_EALIGN", "NM_EUNSUPPORTED", "NM_EHIP",
    "NM_META_U8", "NM_META_2BIT", "NM_W_BF16", "NM_W_FP8E4M3", "NM_ACT_DYNAMIC", "NM_ACT_COMPRESSED",
    "NM_W_COMPRESSED", "NM_W_SLIDE", "NM_ACT_MASKED", "nm_spmm_args", "nm_status_str", "nm_version", "nm_sparsify",
    "nm_sparsify_scored", "NM_SCORE_ACT_WEIGHTED", "NM_SCORE_WEIGHT", "route_taken", "ROUTE", "TAKEN",
    "route_bits", "taken_names", "make_spmm_args",
    "nm_compress", "nm_decompress", "nm_lower_slide", "nm_slide_lift", "nm_spmm",
    "nm_spmm_workspace_size", "nm_hybrid_pack", "nm_hybrid_pack_workspace_size", "nm_hybrid_gemm",
    "nm_hybrid_gemm_workspace_size", "lowered_k", "NM_SPENSE_LOSS", "NM_SPENSE_TAIL", "nm_spense_glu_order",
    "nm_spense_glu_order_workspace_size", "nm_spense_pack", "nm_spense_pack_workspace_size",
    "nm_spense_outsplit_gemm", "nm_spense_outsplit_workspace_size", "nm_quant_lift", "NM_PTS_DYNAMIC",
    "NM_PTS_STATIC", "NM_PTS_VAR", "nm_sparsify_pts", "nm_weight_sums", "NM_ESCRATCH", "nm_spmm_noalloc",
    "NM_NOALLOC_SCRATCH_BYTES", "nm_quant_i8", "nm_meta_block", "nm_meta_block_bytes", "nm_spmm_i8", "nm_glu_i8",
    "nm_i8_workspace_size", "NM_I8_MAX_K", "NM_I8_MAX_ROWS", "NM_Y_F32", "NM_Y_BF16", "NM_GLU_SILU", "NM_GLU_GELU_TANH",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnmsparse.so")

NM_OK, NM_EINVAL, NM_ESHAPE, NM_EALIGN, NM_EUNSUPPORTED, NM_EHIP, NM_ESCRATCH = range(7)
NM_NOALLOC_SCRATCH_BYTES = 64 << 20
NM_META_U8, NM_META_2BIT = 0, 1
NM_W_BF16, NM_W_FP8E4M3 = 0, 1
NM_SCORE_ACT_WEIGHTED, NM_SCORE_WEIGHT = 0, 1
NM_SPENSE_LOSS, NM_SPENSE_TAIL = 0, 1
NM_ACT_DYNAMIC, NM_ACT_COMPRESSED, NM_W_COMPRESSED, NM_W_SLIDE, NM_ACT_MASKED = range(5)
NM_PTS_DYNAMIC, NM_PTS_STATIC, NM_PTS_VAR = 1, 2, 4
NM_I8_MAX_K = 131071
NM_I8_MAX_ROWS = 1 << 27
NM_Y_F32, NM_Y_BF16 = 0, 1
NM_GLU_SILU, NM_GLU_GELU_TANH = 0, 1

# route hints (NM_ROUTE_*) and the report of what ran (NM_TAKEN_*), by lower-case name
ROUTE = {name: 1 << i for i, name in enumerate(
    ["act_fused", "act_mask", "act_sx", "no_few", "few_stream", "few_tile", "no_meta_block", "fp8_widen",
     "no_xlds", "no_few_select", "tile_lds", "tile_regs", "lift_copy", "act_sparse_x", "row_sx"])}
TAKEN = {name: 1 << i for i, name in enumerate(
    ["select", "few_stream", "few_xlds", "few_select", "tile_split", "reduce", "tile_lds", "tile_regs",
     "fused_select", "mask", "gather1", "lift", "meta_block", "permute", "quant", "widen", "decompress",
     "sparse_mma"])}


def route_bits(*names) -> int:
    """OR of the NM_ROUTE_* bits named (e.g. route_bits("few_stream", "no_xlds"))."""
    bits = 0
    for nm in names:
        bits |= ROUTE[nm]
    return bits


def taken_names(bits: int) -> set:
    """The NM_TAKEN_* names set in a route report."""
    return {nm for nm, b in TAKEN.items() if bits & b}


_i64 = ctypes.c_int64
_int = ctypes.c_int
_vp = ctypes.c_void_p


class nm_spmm_args(ctypes.Structure):
    _fields_ = [
        ("mode", _int), ("n", _int), ("m", _int), ("ns", _int),
        ("t", _i64), ("o", _i64), ("k", _i64),
        ("x", _vp), ("ldx", _i64), ("x_meta", _vp), ("x_meta_fmt", _int),
        ("w", _vp), ("ldw", _i64), ("w_dtype", _int), ("w_meta", _vp), ("w_meta_fmt", _int),
        ("w_scale", _vp), ("w_kmajor", _vp),
        ("y", _vp), ("ldy", _i64), ("accumulate", _int),
        ("x_mask_out", _vp), ("workspace", _vp), ("workspace_bytes", _i64),
        ("route", ctypes.c_uint32), ("few_wpb", ctypes.c_int32), ("few_splits", ctypes.c_int32),
        ("tile_wg", ctypes.c_int32), ("route_taken", _vp),
        ("pts", _int), ("pts_shift", _vp), ("col_shift", _vp), ("row_scale", _vp), ("row_shift", _vp),
    ]


class NMError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {nm_status_str(status)}")


_LIB = None


def lib() -> ctypes.CDLL:
    """Load libnmsparse.so once; raise ImportError if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with semi_structured_sparse_amd.build.build()")
    L = ctypes.CDLL(LIB_PATH)
    L.nm_status_str.restype = ctypes.c_char_p
    L.nm_status_str.argtypes = [_int]
    L.nm_version.restype = _int
    L.nm_version.argtypes = []
    L.nm_sparsify.restype = _int
    L.nm_sparsify.argtypes = [_vp, _i64, _i64, _i64, _int, _int, _vp, _i64, _vp, _vp]
    L.nm_sparsify_scored.restype = _int
    L.nm_sparsify_scored.argtypes = [_vp, _i64, _i64, _i64, _int, _int, _vp, _int, _vp, _i64, _vp, _vp]
    L.nm_sparsify_pts.restype = _int
    L.nm_sparsify_pts.argtypes = [_vp, _i64, _i64, _i64, _int, _int, _int, _vp, _vp, _i64, _vp, _vp, _vp, _vp]
    L.nm_weight_sums.restype = _int
    L.nm_weight_sums.argtypes = [_vp, _i64, _i64, _i64, _int, _vp, _vp, _vp, _vp]
    L.nm_compress.restype = _int
    L.nm_compress.argtypes = [_vp, _i64, _i64, _i64, _int, _int, _vp, _vp, _int, _vp, _vp]
    L.nm_decompress.restype = _int
    L.nm_decompress.argtypes = [_vp, _vp, _int, _i64, _i64, _int, _int, _vp, _i64, _vp]
    L.nm_lower_slide.restype = _int
    L.nm_lower_slide.argtypes = [_vp, _vp, _i64, _i64, _int, _vp, _vp, _int, _vp]
    L.nm_slide_lift.restype = _int
    L.nm_slide_lift.argtypes = [_vp, _i64, _i64, _i64, _int, _vp, _i64, _vp]
    L.nm_spmm.restype = _int
    L.nm_spmm.argtypes = [ctypes.POINTER(nm_spmm_args), _vp]
    L.nm_spmm_noalloc.restype = _int
    L.nm_spmm_noalloc.argtypes = [ctypes.POINTER(nm_spmm_args), _vp]
    L.nm_spmm_workspace_size.restype = _i64
    L.nm_spmm_workspace_size.argtypes = [ctypes.POINTER(nm_spmm_args)]
    L.nm_hybrid_pack.restype = _int
    L.nm_hybrid_pack.argtypes = [_vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _int, _vp, _i64, _vp, _i64, _vp]
    L.nm_hybrid_pack_workspace_size.restype = _i64
    L.nm_hybrid_pack_workspace_size.argtypes = [_i64]
    L.nm_hybrid_gemm.restype = _int
    L.nm_hybrid_gemm.argtypes = [_vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _int, _vp, _i64, _i64, _vp,
                                 _i64, _int, _vp, _i64, ctypes.c_uint32, _vp, _vp]
    L.nm_hybrid_gemm_workspace_size.restype = _i64
    L.nm_hybrid_gemm_workspace_size.argtypes = [_i64, _i64, _i64, _i64, _int, ctypes.c_uint32]
    L.nm_quant_lift.restype = _int
    L.nm_quant_lift.argtypes = [_vp, _i64, _i64, _i64, _int, _vp, _i64, _vp, _vp]
    L.nm_spense_glu_order.restype = _int
    L.nm_spense_glu_order.argtypes = [_vp, _vp, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _int, _vp, _vp, _vp,
                                      _i64, _vp]
    L.nm_spense_glu_order_workspace_size.restype = _i64
    L.nm_spense_glu_order_workspace_size.argtypes = [_i64]
    L.nm_spense_pack.restype = _int
    L.nm_spense_pack.argtypes = [_vp, _i64, _i64, _i64, _int, _vp, _i64, _vp, _vp, _int, _vp, _i64, _vp, _i64, _vp]
    L.nm_spense_pack_workspace_size.restype = _i64
    L.nm_spense_pack_workspace_size.argtypes = [_i64, _i64, _int, _i64]
    L.nm_spense_outsplit_gemm.restype = _int
    L.nm_spense_outsplit_gemm.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _int,
                                          _vp, _i64, _vp]
    L.nm_spense_outsplit_workspace_size.restype = _i64
    L.nm_spense_outsplit_workspace_size.argtypes = [_i64, _i64, _i64, _i64]
    L.nm_quant_i8.restype = _int
    L.nm_quant_i8.argtypes = [_vp, _i64, _i64, _i64, _int, _int, _int, _vp, _i64, _vp, _vp]
    L.nm_meta_block.restype = _int
    L.nm_meta_block.argtypes = [_vp, _i64, _i64, _vp, _vp]
    L.nm_meta_block_bytes.restype = _i64
    L.nm_meta_block_bytes.argtypes = [_i64, _i64]
    L.nm_spmm_i8.restype = _int
    L.nm_spmm_i8.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _int, _int,
                             _vp, _i64, ctypes.c_uint32, _vp, _vp]
    L.nm_glu_i8.restype = _int
    L.nm_glu_i8.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _int, _vp, _i64,
                            _int, _vp, _i64, ctypes.c_uint32, _vp, _vp]
    L.nm_i8_workspace_size.restype = _i64
    L.nm_i8_workspace_size.argtypes = [_i64, _i64, _i64, _int, _int, ctypes.c_uint32]
    _LIB = L
    return L


# ------------------------------------------------------------------- marshalling ---

def _ptr(t):
    """Device pointer of a tensor (None -> NULL).  Integers pass through as raw pointers."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _ld(t, default=0):
    if t is None:
        return default
    if t.dim() == 2:
        if t.stride(1) != 1:
            raise ValueError("innermost dimension must be contiguous")
        return t.stride(0)
    return default


_current_raw_stream = None      # device -> raw current stream
_current_device = None          # () -> the current device
# element types of the int8 layers: codes, rows of bf16 (or their bits), and fp16, which y must not be
_int8s = _bf16s = _half = None


def _bind_types(torch):
    global _int8s, _bf16s, _half
    _int8s, _bf16s, _half = (torch.int8, torch.uint8), (torch.bfloat16, torch.int16, torch.uint16), torch.float16


def _bind_torch():
    global _current_raw_stream, _current_device
    import torch
    _bind_types(torch)
    torch.cuda.current_stream()             # initialises the device
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    # building a Stream object costs 2.7 us a call, the raw handle 0.2 us (one-token calls take 6)
    # the stream lookup last: it tells other threads that all of it is there
    if raw is not None and device is not None:
        _current_device = device
        _current_raw_stream = raw
    else:
        _current_device = torch.cuda.current_device
        _current_raw_stream = lambda dev: torch.cuda.current_stream(dev).cuda_stream  # noqa: E731


def _current():
    """(current device, its raw current stream)"""
    if _current_raw_stream is None:
        _bind_torch()
    dev = _current_device()
    return dev, _current_raw_stream(dev)


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    return _current()[1]


def _check(status: int, where: str):
    if status != NM_OK:
        raise NMError(status, where)


def nm_status_str(status: int) -> str:
    return lib().nm_status_str(int(status)).decode()


def nm_version() -> int:
    return int(lib().nm_version())


def lowered_k(k: int, ns: int) -> int:
    """Reduction length after (2N-2):2N -> 2:4 lowering: k * (2N-2) / N."""
    return (k // (2 * ns)) * 4 * (ns - 1)


# ------------------------------------------------------------------- entry points ---

def nm_sparsify(x, n, m, y=None, mask=None, stream=None, *, rows=None, k=None, ldx=None, ldy=None, check=True):
    rows = x.shape[0] if rows is None else rows
    k = x.shape[1] if k is None else k
    st = lib().nm_sparsify(_ptr(x), rows, k, _ld(x) if ldx is None else ldx, n, m, _ptr(y),
                           _ld(y) if ldy is None else ldy, _ptr(mask), _stream(stream))
    if check:
        _check(st, "nm_sparsify")
    return st


def nm_sparsify_scored(x, n, m, col_score, mode=NM_SCORE_ACT_WEIGHTED, y=None, mask=None, stream=None, *,
                       rows=None, k=None, ldx=None, ldy=None, check=True):
    rows = x.shape[0] if rows is None else rows
    k = x.shape[1] if k is None else k
    st = lib().nm_sparsify_scored(_ptr(x), rows, k, _ld(x) if ldx is None else ldx, n, m, _ptr(col_score), mode,
                                  _ptr(y), _ld(y) if ldy is None else ldy, _ptr(mask), _stream(stream))
    if check:
        _check(st, "nm_sparsify_scored")
    return st


def nm_sparsify_pts(x, n, m, pts, y, mask=None, shift=None, row_shift=None, row_scale=None, stream=None, *,
                    rows=None, k=None, ldx=None, ldy=None, check=True):
    rows = x.shape[0] if rows is None else rows
    k = x.shape[1] if k is None else k
    st = lib().nm_sparsify_pts(_ptr(x), rows, k, _ld(x) if ldx is None else ldx, n, m, pts, _ptr(shift), _ptr(y),
                               _ld(y) if ldy is None else ldy, _ptr(mask), _ptr(row_shift), _ptr(row_scale),
                               _stream(stream))
    if check:
        _check(st, "nm_sparsify_pts")
    return st


def nm_weight_sums(w, out, w_dtype=NM_W_BF16, w_scale=None, shift=None, stream=None, *, o=None, k=None, ldw=None,
                   check=True):
    o = w.shape[0] if o is None else o
    k = w.shape[1] if k is None else k
    st = lib().nm_weight_sums(_ptr(w), o, k, _ld(w) if ldw is None else ldw, w_dtype, _ptr(w_scale), _ptr(shift),
                              _ptr(out), _stream(stream))
    if check:
        _check(st, "nm_weight_sums")
    return st


def nm_compress(x, n, m, values, meta, fmt=NM_META_U8, mask=None, stream=None, *, rows=None, k=None, ldx=None,
                check=True):
    rows = x.shape[0] if rows is None else rows
    k = x.shape[1] if k is None else k
    st = lib().nm_compress(_ptr(x), rows, k, _ld(x) if ldx is None else ldx, n, m, _ptr(values), _ptr(meta), fmt,
                           _ptr(mask), _stream(stream))
    if check:
        _check(st, "nm_compress")
    return st


def nm_decompress(values, meta, fmt, rows, k, n, m, y, stream=None, *, ldy=None, check=True):
    st = lib().nm_decompress(_ptr(values), _ptr(meta), fmt, rows, k, n, m, _ptr(y), _ld(y) if ldy is None else ldy,
                             _stream(stream))
    if check:
        _check(st, "nm_decompress")
    return st


def nm_lower_slide(values, idx, rows, k, ns, values_out, meta_out, fmt=NM_META_2BIT, stream=None, *, check=True):
    st = lib().nm_lower_slide(_ptr(values), _ptr(idx), rows, k, ns, _ptr(values_out), _ptr(meta_out), fmt,
                              _stream(stream))
    if check:
        _check(st, "nm_lower_slide")
    return st


def nm_slide_lift(x, ns, x_out, stream=None, *, t=None, k=None, ldx=None, ldo=None, check=True):
    t = x.shape[0] if t is None else t
    k = x.shape[1] if k is None else k
    st = lib().nm_slide_lift(_ptr(x), t, k, _ld(x) if ldx is None else ldx, ns, _ptr(x_out),
                             _ld(x_out) if ldo is None else ldo, _stream(stream))
    if check:
        _check(st, "nm_slide_lift")
    return st


def nm_spmm(args: nm_spmm_args, stream=None, *, check=True):
    st = lib().nm_spmm(ctypes.byref(args), _stream(stream))
    if check:
        _check(st, "nm_spmm")
    return st


def nm_spmm_noalloc(args: nm_spmm_args, stream=None, *, check=True):
    """nm_spmm with the library's own scratch (args.workspace must be NULL, bytes 0)."""
    st = lib().nm_spmm_noalloc(ctypes.byref(args), _stream(stream))
    if check:
        _check(st, "nm_spmm_noalloc")
    return st


def nm_spmm_workspace_size(args: nm_spmm_args) -> int:
    return int(lib().nm_spmm_workspace_size(ctypes.byref(args)))


def make_spmm_args(mode, t, o, k, x, w, y, *, n=2, m=4, ns=2, ldx=None, x_meta=None, x_meta_fmt=NM_META_U8,
                   ldw=None, w_dtype=NM_W_BF16, w_meta=None, w_meta_fmt=NM_META_2BIT, w_scale=None,
                   w_kmajor=None, ldy=None, accumulate=0, x_mask_out=None, workspace=None, workspace_bytes=0,
                   route=0, few_wpb=0, few_splits=0, tile_wg=0, pts=0, pts_shift=None, col_shift=None,
                   row_scale=None, row_shift=None):
    """Fill an nm_spmm_args from tensors (pointers and leading dimensions only).  The
    returned struct keeps references to the tensors so that their memory stays allocated
    while the struct is alive (it holds raw device pointers), and carries a report cell
    that route_taken(args) reads after a call."""
    a = nm_spmm_args()
    a._taken = ctypes.c_uint32(0)
    a.route, a.few_wpb, a.few_splits, a.tile_wg = route, few_wpb, few_splits, tile_wg
    a.route_taken = ctypes.addressof(a._taken)
    a._tensors = [v for v in (x, w, y, x_meta, w_meta, w_scale, w_kmajor, x_mask_out, workspace, pts_shift,
                              col_shift, row_scale, row_shift)
                  if v is not None and not isinstance(v, int)]
    a.pts, a.pts_shift, a.col_shift = pts, _ptr(pts_shift), _ptr(col_shift)
    a.row_scale, a.row_shift = _ptr(row_scale), _ptr(row_shift)
    a.mode, a.n, a.m, a.ns = mode, n, m, ns
    a.t, a.o, a.k = t, o, k
    a.x, a.ldx = _ptr(x), (_ld(x) if ldx is None else ldx)
    a.x_meta, a.x_meta_fmt = _ptr(x_meta), x_meta_fmt
    a.w, a.ldw, a.w_dtype = _ptr(w), (_ld(w) if ldw is None else ldw), w_dtype
    a.w_meta, a.w_meta_fmt = _ptr(w_meta), w_meta_fmt
    a.w_scale, a.w_kmajor = _ptr(w_scale), _ptr(w_kmajor)
    a.y, a.ldy, a.accumulate = _ptr(y), (_ld(y) if ldy is None else ldy), accumulate
    a.x_mask_out = _ptr(x_mask_out)
    a.workspace, a.workspace_bytes = _ptr(workspace), workspace_bytes
    return a


def nm_hybrid_pack(w, k_dense, sparse_cols, dense_cols, ws_values, ws_meta, fmt, wd, workspace, stream=None, *,
                   o=None, k=None, ldw=None, ldwd=None, workspace_bytes=None, check=True):
    o = w.shape[0] if o is None else o
    k = w.shape[1] if k is None else k
    wsb = (workspace.numel() * workspace.element_size()) if workspace_bytes is None else workspace_bytes
    st = lib().nm_hybrid_pack(_ptr(w), o, k, _ld(w) if ldw is None else ldw, k_dense, _ptr(sparse_cols),
                              _ptr(dense_cols), _ptr(ws_values), _ptr(ws_meta), fmt, _ptr(wd),
                              _ld(wd) if ldwd is None else ldwd, _ptr(workspace), wsb, _stream(stream))
    if check:
        _check(st, "nm_hybrid_pack")
    return st


def nm_hybrid_pack_workspace_size(k: int) -> int:
    return int(lib().nm_hybrid_pack_workspace_size(k))


def route_taken(args: nm_spmm_args) -> int:
    """NM_TAKEN_* bits reported by the calls made with args (made by make_spmm_args)."""
    return int(args._taken.value)


def nm_hybrid_gemm_workspace_size(t: int, k_s: int, k_d: int, o: int, gathered: bool, route: int = 0) -> int:
    return int(lib().nm_hybrid_gemm_workspace_size(t, k_s, k_d, o, 1 if gathered else 0, route))


def nm_quant_lift(x, ns, xq, xs, stream=None, *, t=None, k=None, ldx=None, ldq=None, check=True):
    t = x.shape[0] if t is None else t
    k = x.shape[1] if k is None else k
    st = lib().nm_quant_lift(_ptr(x), t, k, _ld(x) if ldx is None else ldx, ns, _ptr(xq),
                             _ld(xq) if ldq is None else ldq, _ptr(xs), _stream(stream))
    if check:
        _check(st, "nm_quant_lift")
    return st


def nm_spense_glu_order(w_gate, w_up, w_down, hs_in, hs_mid, n_dense, strategy, perm, workspace, scores=None,
                        stream=None, *, hidden=None, inter=None, ld_gu=None, ld_d=None, workspace_bytes=None,
                        check=True):
    inter = (w_gate.shape[0] if w_gate is not None else perm.shape[0]) if inter is None else inter
    hidden = (w_gate.shape[1] if w_gate is not None else 0) if hidden is None else hidden
    wsb = (workspace.numel() * workspace.element_size()) if workspace_bytes is None else workspace_bytes
    st = lib().nm_spense_glu_order(_ptr(w_gate), _ptr(w_up), (_ld(w_gate) if w_gate is not None else 0)
                                   if ld_gu is None else ld_gu, _ptr(w_down),
                                   (_ld(w_down) if w_down is not None else 0) if ld_d is None else ld_d, hidden,
                                   inter, _ptr(hs_in), _ptr(hs_mid), n_dense, strategy, _ptr(perm), _ptr(scores),
                                   _ptr(workspace), wsb, _stream(stream))
    if check:
        _check(st, "nm_spense_glu_order")
    return st


def nm_spense_glu_order_workspace_size(inter: int) -> int:
    return int(lib().nm_spense_glu_order_workspace_size(inter))


def nm_spense_pack(w, axis, perm, n_sparse, ws_values, ws_meta, fmt, wd, workspace=None, stream=None, *, o=None,
                   k=None, ldw=None, ldwd=None, workspace_bytes=None, check=True):
    o = w.shape[0] if o is None else o
    k = w.shape[1] if k is None else k
    wsb = (workspace.numel() * workspace.element_size() if workspace is not None else 0) \
        if workspace_bytes is None else workspace_bytes
    st = lib().nm_spense_pack(_ptr(w), o, k, _ld(w) if ldw is None else ldw, axis, _ptr(perm), n_sparse,
                              _ptr(ws_values), _ptr(ws_meta), fmt, _ptr(wd),
                              (_ld(wd) if wd is not None else 0) if ldwd is None else ldwd, _ptr(workspace), wsb,
                              _stream(stream))
    if check:
        _check(st, "nm_spense_pack")
    return st


def nm_spense_pack_workspace_size(o: int, k: int, axis: int, n_sparse: int) -> int:
    return int(lib().nm_spense_pack_workspace_size(o, k, axis, n_sparse))


def nm_spense_outsplit_gemm(x, ws_values, ws_meta, o_s, wd, o_d, y, accumulate=0, workspace=None, stream=None, *,
                            t=None, k=None, ldx=None, ldwd=None, ldy=None, workspace_bytes=None, check=True):
    t = x.shape[0] if t is None else t
    k = x.shape[1] if k is None else k
    wsb = (workspace.numel() * workspace.element_size() if workspace is not None else 0) \
        if workspace_bytes is None else workspace_bytes
    st = lib().nm_spense_outsplit_gemm(_ptr(x), t, k, _ld(x) if ldx is None else ldx, _ptr(ws_values),
                                       _ptr(ws_meta), o_s, _ptr(wd),
                                       (_ld(wd) if wd is not None else 0) if ldwd is None else ldwd, o_d, _ptr(y),
                                       _ld(y) if ldy is None else ldy, accumulate, _ptr(workspace), wsb,
                                       _stream(stream))
    if check:
        _check(st, "nm_spense_outsplit_gemm")
    return st


def nm_spense_outsplit_workspace_size(t: int, k: int, o_s: int, o_d: int) -> int:
    return int(lib().nm_spense_outsplit_workspace_size(t, k, o_s, o_d))


def nm_hybrid_gemm(x, sparse_cols, k_s, dense_cols, k_d, ws_values, ws_meta, fmt, wd, o, y, accumulate=0,
                   stream=None, *, t=None, ldx=None, ldwd=None, ldy=None, workspace=None, workspace_bytes=None,
                   route=0, taken=None, check=True):
    """taken: optional ctypes.c_uint32 that receives the NM_TAKEN_* report."""
    t = x.shape[0] if t is None else t
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None or isinstance(workspace, int) else \
            workspace.numel() * workspace.element_size()
    st = lib().nm_hybrid_gemm(_ptr(x), t, _ld(x) if ldx is None else ldx, _ptr(sparse_cols), k_s,
                              _ptr(dense_cols), k_d, _ptr(ws_values), _ptr(ws_meta), fmt, _ptr(wd),
                              _ld(wd) if ldwd is None else ldwd, o, _ptr(y), _ld(y) if ldy is None else ldy,
                              accumulate, _ptr(workspace), workspace_bytes, route,
                              ctypes.addressof(taken) if taken is not None else None, _stream(stream))
    if check:
        _check(st, "nm_hybrid_gemm")
    return st


# ------------------------------------------------------------------------ int8 layers ---

def _device_of(*ts):
    """The device the tensors have to be on where the caller names a stream; -1 where all of them
    are raw pointers."""
    for t in ts:
        if t is not None and type(t) is not int:
            if t.get_device() < 0:
                _refuse(t, 0, "")
            return _current()[0]
    return -1


def _refuse(t, dev, what):
    if t.get_device() != dev:
        raise ValueError("tensors must be on the current GPU")
    raise ValueError(what)


def _mat(t, dev, types, name):
    """(pointer, leading dimension) of a matrix with contiguous rows of one of the types."""
    if t is None or type(t) is int:
        return t, 0
    st = t.stride()
    if len(st) != 2 or st[1] != 1 or t.get_device() != dev or t.dtype not in types:
        _refuse(t, dev, f"a matrix with contiguous rows of {name} is needed")
    return t.data_ptr(), st[0]


def _holds(t, rows, cols, whole, ld):
    """Refuses a matrix with fewer rows or columns (counted up to a whole piece of `whole` elements,
    which a row's padding completes), or whose last row's pieces end past its storage."""
    sh = t.shape
    if sh[0] < rows or sh[1] + -sh[1] % whole < cols:
        raise ValueError(f"a matrix of {rows} rows of {cols} elements is needed")
    if rows > 0 and cols > 0:
        end = t.storage_offset() + (rows - 1) * ld + cols + -cols % whole
        if end * t.element_size() > t.untyped_storage().nbytes():
            raise ValueError(f"the storage ends inside the last of {rows} rows of {cols} elements, {ld} apart")


def _codes(m, sh, dev, rows, cols, ld):
    """(pointer, leading dimension) of int8 codes of shape sh that are read: `rows` rows of `cols`, in
    pieces of 16; ld: None, or a leading dimension in place of the tensor's."""
    if sh is None:
        return m, ld or 0
    st = m.stride()
    if len(st) != 2 or st[1] != 1 or m.get_device() != dev or m.dtype not in _int8s:
        _refuse(m, dev, "a matrix with contiguous rows of int8 codes is needed")
    if ld is None:
        ld = st[0] if cols else 0       # of no columns: torch has 1
    if sh[0] < rows or sh[1] < cols + -cols % 16 or ld != st[0]:
        _holds(m, rows, cols, 16, ld)
    return m.data_ptr(), ld


def _factors(t, n, dev):
    """Pointer of at least n contiguous fp32 values (None -> NULL, integers are raw pointers)."""
    if t is None or type(t) is int:
        return t
    if t.get_device() != dev or t.nbytes < 4 * n or t.element_size() != 4 or not t.is_contiguous():
        _refuse(t, dev, f"{n} contiguous fp32 factors are needed")
    return t.data_ptr()


def _i8_out(y, t, o, dev, ld, dtype):
    """(pointer, leading dimension, NM_Y_*) of an output of at least t rows of o (raw pointers: fp32
    unless dtype says otherwise); ld: None, or a leading dimension in place of the tensor's."""
    if y is None or type(y) is int:
        return y, ld or 0, NM_Y_F32 if dtype is None else dtype
    st, sh, size = y.stride(), y.shape, y.element_size()
    kind = NM_Y_F32 if size == 4 else NM_Y_BF16
    if (len(st) != 2 or st[1] != 1 or y.get_device() != dev or (size != 4 and size != 2) or y.dtype is _half
            or sh[0] < t or sh[1] < o or (dtype is not None and dtype != kind)):
        _refuse(y, dev, f"y of {t} contiguous rows of {o} fp32 or bf16 values is needed")
    if ld is None:
        return y.data_ptr(), st[0], kind
    _holds(y, t, o, 1, ld)
    return y.data_ptr(), ld, kind


def _packed(t, size, dev):
    """Pointer of at least `size` contiguous bytes of positions."""
    if t is None or type(t) is int:
        return t
    if t.get_device() != dev or t.nbytes < size or not t.is_contiguous():
        _refuse(t, dev, f"{size} contiguous bytes of positions are needed")
    return t.data_ptr()


def _meta(t, o, k, dev):
    """Pointer of blocked positions (nm_meta_block) of at least o rows over k."""
    return t if t is None else _packed(t, (k + 127) // 128 * o * 16, dev)


def _scratch(t, size, dev):
    """(pointer, bytes) of a workspace; size: None, or a part of it to use."""
    if t is None or type(t) is int:
        return t, size or 0
    have = t.nbytes
    if t.get_device() != dev or not t.is_contiguous() or (size is not None and size > have):
        _refuse(t, dev, "a contiguous workspace of at least the stated bytes is needed")
    return t.data_ptr(), have if size is None else size


def nm_quant_i8(x, q, scale, n=0, m=0, ns=2, stream=None, *, rows=None, k=None, ldx=None, ldq=None, check=True):
    """Rows of bf16 x -> int8 codes q and one fp32 scale per row (include/nm.h)."""
    if stream is None:
        dev, stream = _current()
    else:
        dev, stream = _device_of(x, q, scale), _stream(stream)
    xp, lx = _mat(x, dev, _bf16s, "bf16 values")
    qp, lq = _mat(q, dev, _int8s, "int8 codes")
    if ldx is not None:
        lx = ldx
    if ldq is not None:
        lq = ldq
    if xp is not x:                      # a tensor
        have, width = x.shape
        if rows is None:
            rows = have
        if k is None:
            k = width
        if width < k:
            raise ValueError(f"x of rows of {k} values is needed")
        if have < rows or width & 7 or ldx is not None:
            _holds(x, rows, k, 8, lx)
    if qp is not q:
        have, width = q.shape
        kq = k // (2 * ns) * 4 * (ns - 1) if ns > 2 else k
        if width < kq:
            raise ValueError(f"q of rows of {kq} codes is needed")
        if have < rows or width & 15 or ldq is not None:
            _holds(q, rows, kq, 16, lq)
    if k == 0:                           # torch has a leading dimension of 1 for no columns
        lx, lq = ldx or 0, ldq or 0
    st = lib().nm_quant_i8(xp, rows, k, lx, n, m, ns, qp, lq, _factors(scale, rows, dev), stream)
    if check and st:
        _check(st, "nm_quant_i8")
    return st


def nm_meta_block(meta, o, kc, out, stream=None, *, check=True):
    """2-bit positions in rows -> step blocks (include/nm.h); both tensors contiguous."""
    if stream is None:
        dev, stream = _current()
    else:
        dev, stream = _device_of(meta, out), _stream(stream)
    st = lib().nm_meta_block(_packed(meta, o * ((kc + 7) // 8), dev), o, kc, _meta(out, o, kc, dev), stream)
    if check:
        _check(st, "nm_meta_block")
    return st


def nm_meta_block_bytes(o: int, kc: int) -> int:
    return int(lib().nm_meta_block_bytes(o, kc))


def nm_i8_workspace_size(t: int, o: int, k: int, sparse: bool = False, glu: bool = False, route: int = 0) -> int:
    return int(lib().nm_i8_workspace_size(t, o, k, 1 if sparse else 0, 1 if glu else 0, route))


def nm_spmm_i8(x, x_scale, w, w_scale, y, w_meta=None, row_shift=None, col_shift=None, accumulate=0, workspace=None,
               stream=None, *, t=None, o=None, k=None, ldx=None, ldw=None, ldy=None, y_dtype=None,
               workspace_bytes=None, route=0, taken=None, check=True):
    """y = (x . w^T) * x_scale * w_scale (+ row_shift * col_shift) in 8-bit integers; w_meta (from
    nm_meta_block): 2:4 weights.  k: the reduction length where it is not x's width.
    taken: optional ctypes.c_uint32 that receives the NM_TAKEN_* report."""
    if stream is None:
        dev, stream = _current()
    else:
        dev, stream = _device_of(x, w, y, x_scale, w_scale, w_meta, row_shift, col_shift, workspace), _stream(stream)
    sx = None if x is None or type(x) is int else x.shape
    sw = None if w is None or type(w) is int else w.shape
    if t is None:
        t = sx[0]
    if o is None:
        o = sw[0]
    if k is None:
        k = sx[1]
    xp, lx = _codes(x, sx, dev, t, k, ldx)
    wp, lw = _codes(w, sw, dev, o, k if w_meta is None else k // 2, ldw)
    yp, ly, yd = _i8_out(y, t, o, dev, ldy, y_dtype)
    wsp, wsn = _scratch(workspace, workspace_bytes, dev)
    st = lib().nm_spmm_i8(xp, t, k, lx, _factors(x_scale, t, dev), wp, o,
                          lw, _factors(w_scale, o, dev), _meta(w_meta, o, k, dev),
                          _factors(row_shift, t, dev), _factors(col_shift, o, dev), yp, ly, yd, accumulate,
                          wsp, wsn, route, ctypes.addressof(taken) if taken is not None else None, stream)
    if check and st:
        _check(st, "nm_spmm_i8")
    return st


def nm_glu_i8(x, x_scale, w_gate, gate_scale, w_up, up_scale, y, act=NM_GLU_SILU, gate_meta=None, up_meta=None,
              workspace=None, stream=None, *, t=None, inter=None, k=None, ldx=None, ldw=None, ldy=None, y_dtype=None,
              workspace_bytes=None, route=0, taken=None, check=True):
    """y = act(x . w_gate^T) * (x . w_up^T), each with its scales, in 8-bit integers.
    taken: optional ctypes.c_uint32 that receives the NM_TAKEN_* report."""
    if stream is None:
        dev, stream = _current()
    else:
        dev, stream = _device_of(x, w_gate, y, w_up, x_scale, gate_scale, up_scale, gate_meta, up_meta,
                                 workspace), _stream(stream)
    sx = None if x is None or type(x) is int else x.shape
    sg = None if w_gate is None or type(w_gate) is int else w_gate.shape
    su = None if w_up is None or type(w_up) is int else w_up.shape
    if t is None:
        t = sx[0]
    if inter is None:
        inter = sg[0]
        if su is not None and su[0] != inter:
            raise ValueError("w_gate and w_up need the same rows")
    if k is None:
        k = sx[1]
    xp, lx = _codes(x, sx, dev, t, k, ldx)
    kw = k if gate_meta is None else k // 2
    gp, lg = _codes(w_gate, sg, dev, inter, kw, ldw)
    up, lu = _codes(w_up, su, dev, inter, kw, ldw)
    if lg != lu:
        raise ValueError("w_gate and w_up need the same leading dimension")
    yp, ly, yd = _i8_out(y, t, inter, dev, ldy, y_dtype)
    wsp, wsn = _scratch(workspace, workspace_bytes, dev)
    st = lib().nm_glu_i8(xp, t, k, lx, _factors(x_scale, t, dev), gp,
                         _factors(gate_scale, inter, dev), _meta(gate_meta, inter, k, dev), up,
                         _factors(up_scale, inter, dev), _meta(up_meta, inter, k, dev), inter, lg, act, yp, ly, yd,
                         wsp, wsn, route, ctypes.addressof(taken) if taken is not None else None, stream)
    if check and st:
        _check(st, "nm_glu_i8")
    return st
