"""Thin ctypes binding of libnabla.so (include/nabla.h).

Argument marshalling only: torch tensors provide device memory and the
current CUDA stream; every step runs in the library's kernels.  There is no
fallback: if the library is missing or a call fails, this module raises.
"""
import ctypes
import os
import struct

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libnabla.so")

OK = 0
ERR_SHAPE, ERR_ALIGN, ERR_PARAM, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_NULL = (
    -1, -2, -3, -4, -5, -6, -7)
NO_STA, FULL_STA, EMIT_COLS, DEBUG_SCORES, DEBUG_TIMEOUT = 1, 2, 4, 8, 0x100
OP_BUILD_MASK, OP_ATTN_FWD, OP_ATTN_BWD = 0, 1, 2
MASK_BITS, MASK_ROW_IDX, MASK_ROW_CNT, MASK_COL_IDX, MASK_COL_CNT, MASK_SCORES = 0, 1, 2, 3, 4, 5

# every symbol include/nabla.h declares
SYMBOLS = ("nabla_flatten", "nabla_workspace_size", "nabla_mask_bytes", "nabla_build_mask",
           "nabla_build_mask_grid", "nabla_build_mask_static", "nabla_build_mask_dr",
           "nabla_attn_fwd", "nabla_attn_bwd", "nabla_status", "nabla_strerror",
           "nabla_rope", "nabla_packed_workspace_size", "nabla_attn_packed_fwd",
           "nabla_attn_packed_bwd", "nabla_cache_append", "nabla_paged_workspace_size",
           "nabla_attn_paged")
DR_STATIC_RATIO, DR_THRESHOLD = 0, 1
ROPE_ADJACENT, ROPE_HALVES = 0, 1
ROPE_INVERSE, ROPE_FLAT_IN, ROPE_FLAT_OUT = 1, 2, 4
PACKED_FWD, PACKED_BWD = 0, 1
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class NablaError(RuntimeError):
    def __init__(self, status, what):
        super().__init__("%s failed: %s (%d)" % (what, strerror(status), status))
        self.status = status


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "heads", "T", "H", "W", "D", "P")]


class Params(ctypes.Structure):
    _fields_ = [("p", ctypes.c_float), ("sta_t", ctypes.c_int), ("sta_h", ctypes.c_int),
                ("sta_w", ctypes.c_int), ("scale", ctypes.c_float), ("flags", ctypes.c_uint)]


class DrParams(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("gamma", ctypes.c_double), ("lambda_", ctypes.c_double),
                ("tau", ctypes.c_float), ("sta_t", ctypes.c_int), ("sta_h", ctypes.c_int),
                ("sta_w", ctypes.c_int), ("scale", ctypes.c_float), ("flags", ctypes.c_uint)]


class MaskStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p)
                for n in ("bits", "row_idx", "row_cnt", "col_idx", "col_cnt", "scores")]


class View(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("head", ctypes.c_int64),
                ("token", ctypes.c_int64)]


class RopeParams(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("layout", ctypes.c_int), ("D", ctypes.c_int),
                ("pairs", ctypes.c_int * 3), ("theta", ctypes.c_double * 3),
                ("scale", ctypes.c_double * 3), ("offset", ctypes.c_double * 3),
                ("flags", ctypes.c_uint)]


class Packed(ctypes.Structure):
    _fields_ = [("seqs", ctypes.c_int), ("heads", ctypes.c_int), ("heads_kv", ctypes.c_int),
                ("D", ctypes.c_int), ("total_q", ctypes.c_int64), ("total_k", ctypes.c_int64),
                ("causal", ctypes.c_int), ("scale", ctypes.c_float)]


class Cache(ctypes.Structure):
    _fields_ = [("k", View), ("v", View), ("table", ctypes.c_void_p), ("pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("heads_kv", ctypes.c_int), ("D", ctypes.c_int),
                ("seqs", ctypes.c_int), ("table_width", ctypes.c_int)]


_lib = None


def lib():
    """Load libnabla.so; raises if it was not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libnabla.so is not built; run "
                               "`python -m adaptive_block_sparse_fractal_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        F = ctypes.c_float
        L.nabla_flatten.argtypes = [P, P, I64, I, I, I, I, I64, I, P]
        L.nabla_flatten.restype = I
        L.nabla_workspace_size.argtypes = [P, I]
        L.nabla_workspace_size.restype = SZ
        L.nabla_mask_bytes.argtypes = [P, I]
        L.nabla_mask_bytes.restype = SZ
        L.nabla_build_mask.argtypes = [P, P, P, P, P, P, SZ, P]
        L.nabla_build_mask.restype = I
        L.nabla_build_mask_grid.argtypes = [P, P, P, P, P, P, P, P, SZ, P]
        L.nabla_build_mask_grid.restype = I
        L.nabla_build_mask_static.argtypes = [P, P, P, P, P, P]
        L.nabla_build_mask_static.restype = I
        L.nabla_build_mask_dr.argtypes = [P, P, P, P, P, P, SZ, P]
        L.nabla_build_mask_dr.restype = I
        L.nabla_attn_fwd.argtypes = [P, P, P, P, P, P, P, P, P, SZ, P]
        L.nabla_attn_fwd.restype = I
        L.nabla_attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.nabla_attn_bwd.restype = I
        L.nabla_status.argtypes = [P, P]
        L.nabla_status.restype = I
        L.nabla_strerror.argtypes = [I]
        L.nabla_strerror.restype = ctypes.c_char_p
        L.nabla_rope.argtypes = [P, I, I, I, I, I, I, P, P, P, P, I64, I, P]
        L.nabla_rope.restype = I
        L.nabla_packed_workspace_size.argtypes = [P, I]
        L.nabla_packed_workspace_size.restype = SZ
        L.nabla_attn_packed_fwd.argtypes = [P, P, P, P, P, P, P, P, P, SZ, P]
        L.nabla_attn_packed_fwd.restype = I
        L.nabla_attn_packed_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.nabla_attn_packed_bwd.restype = I
        L.nabla_cache_append.argtypes = [P, P, P, I64, P, P, P, SZ, P]
        L.nabla_cache_append.restype = I
        L.nabla_paged_workspace_size.argtypes = [P, I]
        L.nabla_paged_workspace_size.restype = SZ
        L.nabla_attn_paged.argtypes = [P, I, F, P, P, P, P, P, SZ, P]
        L.nabla_attn_paged.restype = I
        _lib = L
    return _lib


def strerror(status):
    return lib().nabla_strerror(int(status)).decode()


def _check(status, what):
    if status != OK:
        raise NablaError(status, what)


def _stream(t):
    """The current stream of the tensor's device."""
    return torch._C._cuda_getCurrentRawStream(_device(t, "the workspace"))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, dtype, name):
    if not (t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise ValueError("%s must be a contiguous CUDA %s tensor" % (name, dtype))


def shape_of(B, heads, T, H, W, D, P=8):
    return Shape(B, heads, T, H, W, D, P)


def params_of(p, window=(3, 3, 3), scale=None, D=None, flags=0):
    if scale is None:
        scale = D ** -0.5
    return Params(float(p), int(window[0]), int(window[1]), int(window[2]), float(scale),
                  int(flags))


def dr_params_of(mode, gamma=1.0, lam=0.0, tau=0.0, window=(3, 3, 3), scale=None, D=None,
                 flags=0):
    if scale is None:
        scale = D ** -0.5
    return DrParams(int(mode), float(gamma), float(lam), float(tau), int(window[0]),
                    int(window[1]), int(window[2]), float(scale), int(flags))


def workspace_size(shape, op):
    return int(lib().nabla_workspace_size(ctypes.byref(shape), op))


def mask_bytes(shape, part):
    return int(lib().nabla_mask_bytes(ctypes.byref(shape), part))


def workspace(shape, op, device):
    n = workspace_size(shape, op)
    if n == 0:
        raise NablaError(ERR_SHAPE, "workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def alloc_mask(shape, device, cols=True, scores=False):
    BH, nb = shape.B * shape.heads, shape.T * (shape.H // shape.P) * (shape.W // shape.P)
    words = (nb + 31) // 32
    m = {"bits": torch.empty((BH, nb, words), dtype=torch.int32, device=device),
         "row_idx": torch.empty((BH, nb, nb), dtype=torch.int16, device=device),
         "row_cnt": torch.empty((BH, nb), dtype=torch.int32, device=device)}
    if cols:
        m["col_idx"] = torch.empty((BH, nb, nb), dtype=torch.int16, device=device)
        m["col_cnt"] = torch.empty((BH, nb), dtype=torch.int32, device=device)
    if scores:
        m["scores"] = torch.empty((BH, nb, nb), dtype=torch.float32, device=device)
    for part, key in ((MASK_BITS, "bits"), (MASK_ROW_IDX, "row_idx"), (MASK_ROW_CNT, "row_cnt"),
                      (MASK_COL_IDX, "col_idx"), (MASK_COL_CNT, "col_cnt"),
                      (MASK_SCORES, "scores")):
        if key in m:
            assert m[key].numel() * m[key].element_size() == mask_bytes(shape, part)
    return m


def _mask_struct(m):
    return MaskStruct(*(_ptr(m.get(k)) for k in ("bits", "row_idx", "row_cnt", "col_idx",
                                                  "col_cnt", "scores")))


def flatten(x, T, H, W, P=8, inverse=False, out=None):
    """x: contiguous CUDA tensor whose bytes are [outer, T*H*W, inner] in grid
    order (inverse=False) or flattened order (inverse=True); dim 0 is outer."""
    if not (x.is_cuda and x.is_contiguous()):
        raise ValueError("x must be a contiguous CUDA tensor")
    out = torch.empty_like(x) if out is None else out
    outer = x.shape[0]
    total = x.numel() * x.element_size()
    inner = total // (outer * T * H * W) if outer else 0
    _check(lib().nabla_flatten(_ptr(x), _ptr(out), outer, T, H, W, P, inner, int(inverse),
                               _stream(x)), "nabla_flatten")
    return out


def build_mask(shape, params, q, k, mask=None, ws=None):
    _need(q, torch.bfloat16, "q")
    _need(k, torch.bfloat16, "k")
    cols = bool(params.flags & EMIT_COLS)
    dbg = bool(params.flags & DEBUG_SCORES)
    mask = alloc_mask(shape, q.device, cols, dbg) if mask is None else mask
    ws = workspace(shape, OP_BUILD_MASK, q.device) if ws is None else ws
    ms = _mask_struct(mask)
    _check(lib().nabla_build_mask(ctypes.byref(shape), ctypes.byref(params), _ptr(q), _ptr(k),
                                  ctypes.byref(ms), _ptr(ws), ws.numel(), _stream(q)),
           "nabla_build_mask")
    return mask


def build_mask_dr(shape, params, q=None, k=None, mask=None, ws=None, device=None):
    """DynamicRad-style mask (static ratio or logit threshold) in the same
    format; q and k are needed by the threshold mode only."""
    thr = params.mode == DR_THRESHOLD
    if thr:
        _need(q, torch.bfloat16, "q")
        _need(k, torch.bfloat16, "k")
        device = q.device
    cols = bool(params.flags & EMIT_COLS)
    dbg = bool(params.flags & DEBUG_SCORES)
    mask = alloc_mask(shape, device, cols, dbg) if mask is None else mask
    if ws is None:
        ws = workspace(shape, OP_BUILD_MASK if thr else OP_ATTN_FWD, device)
    ms = _mask_struct(mask)
    stream = ctypes.c_void_p(torch.cuda.current_stream(ws.device).cuda_stream)
    _check(lib().nabla_build_mask_dr(ctypes.byref(shape), ctypes.byref(params), _ptr(q), _ptr(k),
                                     ctypes.byref(ms), _ptr(ws), ws.numel(), stream),
           "nabla_build_mask_dr")
    return mask


def build_mask_grid(shape, params, q_grid, k_grid, q=None, k=None, mask=None, ws=None):
    """Flatten q_grid, k_grid (grid order, any shape holding [B*h, T*H*W, D])
    into q, k and build the mask from them in one call; returns (q, k, mask)."""
    _need(q_grid, torch.bfloat16, "q_grid")
    _need(k_grid, torch.bfloat16, "k_grid")
    q = torch.empty_like(q_grid) if q is None else q
    k = torch.empty_like(k_grid) if k is None else k
    cols = bool(params.flags & EMIT_COLS)
    dbg = bool(params.flags & DEBUG_SCORES)
    mask = alloc_mask(shape, q_grid.device, cols, dbg) if mask is None else mask
    ws = workspace(shape, OP_BUILD_MASK, q_grid.device) if ws is None else ws
    ms = _mask_struct(mask)
    _check(lib().nabla_build_mask_grid(ctypes.byref(shape), ctypes.byref(params), _ptr(q_grid),
                                       _ptr(k_grid), _ptr(q), _ptr(k), ctypes.byref(ms), _ptr(ws),
                                       ws.numel(), _stream(q_grid)), "nabla_build_mask_grid")
    return q, k, mask


def attn_fwd(shape, params, q, k, v, mask, o=None, lse=None, ws=None, want_lse=True):
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, n)
    o = torch.empty_like(q) if o is None else o
    if lse is None and want_lse:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    ws = workspace(shape, OP_ATTN_FWD, q.device) if ws is None else ws
    ms = _mask_struct(mask)
    _check(lib().nabla_attn_fwd(ctypes.byref(shape), ctypes.byref(params), _ptr(q), _ptr(k),
                                _ptr(v), ctypes.byref(ms), _ptr(o), _ptr(lse), _ptr(ws),
                                ws.numel(), _stream(q)), "nabla_attn_fwd")
    return o, lse


def attn_bwd(shape, params, q, k, v, o, dout, lse, mask, dq=None, dk=None, dv=None, ws=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _need(t, torch.bfloat16, n)
    _need(lse, torch.float32, "lse")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    ws = workspace(shape, OP_ATTN_BWD, q.device) if ws is None else ws
    ms = _mask_struct(mask)
    _check(lib().nabla_attn_bwd(ctypes.byref(shape), ctypes.byref(params), _ptr(q), _ptr(k),
                                _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), ctypes.byref(ms),
                                _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), ws.numel(), _stream(q)),
           "nabla_attn_bwd")
    return dq, dk, dv


# ---------------------------------------------------------------------------
# rotary positions, packed-sequence attention, the paged cache
# ---------------------------------------------------------------------------
def _call(fn, what, dev, *args):
    """fn(*args, current stream of device dev), launched on that device."""
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status != OK:
        raise NablaError(status, what)


def _device(t, name):
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    return dev


# The structures of a call travel as packed bytes (half the cost of filling
# ctypes structures): nabla_view, nabla_packed, and nabla_cache behind its views.
_VIEW = struct.Struct("@Pqqq").pack
_PACKED = struct.Struct("@iiiiqqif").pack
_CACHE = struct.Struct("@Piiiiii").pack
_HEADS = struct.Struct("@ii").pack


def _view(t, name, dev, dims, dtype, shape=None):
    """nabla_view of a tensor of rows on device dev.  Its last dimension is
    contiguous; in front of it stand the tokens and heads ([tokens, heads, D],
    dims = 3) or pages, rows and heads (dims = 4)."""
    s = t.stride()
    if t.dtype != dtype or t.get_device() != dev or len(s) != dims or s[-1] != 1:
        raise ValueError("%s must be a %s tensor of %d dimensions on cuda:%d with a contiguous last "
                         "dimension" % (name, dtype, dims, dev))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    return _VIEW(t.data_ptr(), 0, s[1], s[0]) if dims == 3 else _VIEW(t.data_ptr(), s[0], s[2], s[1])


def _int32(t, name, dev, shape=None):
    if t.dtype != torch.int32 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor on cuda:%d" % (name, dev))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    return t.data_ptr()


def _lse(t, dev, shape):
    if t.dtype != torch.float32 or t.get_device() != dev or not t.is_contiguous() or t.shape != shape:
        raise ValueError("lse must be a contiguous float32 tensor %s on cuda:%d" % (tuple(shape), dev))
    return t.data_ptr()


def _work(ws, dev):
    if ws.dtype != torch.uint8 or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor on cuda:%d" % dev)
    return ws.data_ptr(), ws.numel()


def rope_params_of(pairs, theta=10000.0, scale=1.0, offset=0.0, layout=ROPE_ADJACENT,
                   inverse=False):
    """Rotary parameters: `pairs` turned by each of up to three axes (time,
    height, width); theta, scale and offset are one number or one per axis.
    dtype, D and the token order are filled in by rope()."""
    pairs = [int(n) for n in pairs]
    if not 1 <= len(pairs) <= 3:
        raise ValueError("pairs: one to three axes")

    def axes(x, name):
        x = [float(v) for v in x] if isinstance(x, (tuple, list)) else [float(x)] * len(pairs)
        if len(x) != len(pairs):
            raise ValueError("%s: one number, or one for each of the %d axes" % (name, len(pairs)))
        return tuple(x) + (1.0,) * (3 - len(x))  # (axes without pairs are not looked at)
    p = RopeParams()
    p.layout = int(layout)
    p.pairs = tuple(pairs) + (0,) * (3 - len(pairs))
    p.theta, p.scale, p.offset = axes(theta, "theta"), axes(scale, "scale"), axes(offset, "offset")
    p.flags = ROPE_INVERSE if inverse else 0
    return p


def rope(params, q, k=None, grid=None, pos=None, flat_in=False, flat_out=False, P=8, q_out=None,
         k_out=None):
    """Rotate q, or q and k ([B, heads, N, D] or [heads, N, D], any strides with
    contiguous rows; bf16, fp16 or fp32) by the positions of a (T, H, W) grid or
    by `pos` (int32 [N, axes] or [B, N, axes], in grid order).  flat_in /
    flat_out: that side is in flattened token order (needs `grid`).  Outputs may
    be the inputs (same order on both sides).  Returns q_out, or (q_out, k_out)."""
    shape = q.shape
    dims = len(shape)
    dtype = DTYPES.get(q.dtype)
    if dtype is None or dims not in (3, 4):
        raise ValueError("q must be [B, heads, N, D] or [heads, N, D] in bf16, fp16 or fp32")
    dev = _device(q, "q")
    heads, N, D = shape[-3:]
    B = shape[0] if dims == 4 else 1
    if grid is not None:
        T, H, W = grid
        if T * H * W != N:
            raise ValueError("grid %s does not hold %d tokens" % (tuple(grid), N))
    elif pos is None or flat_in or flat_out:
        raise ValueError("grid is needed without pos and for a flattened order")
    else:
        T, H, W = N, 1, 1
    if q_out is None:
        q_out = torch.empty_like(q)
    ins, outs = _rope_view(q, q, shape, dev), _rope_view(q_out, q, shape, dev)
    heads_k = 0
    if k is not None:
        shape_k = k.shape
        heads_k = shape_k[-3]
        if len(shape_k) != dims or shape_k[-2:] != (N, D) or (dims == 4 and shape_k[0] != B):
            raise ValueError("q and k must have the same batch, tokens and D")
        if k_out is None:
            k_out = torch.empty_like(k)
        ins += _rope_view(k, q, shape_k, dev)
        outs += _rope_view(k_out, q, shape_k, dev)
    pos_ptr, pos_batch, axes = None, 0, 0
    if pos is not None:
        axes = pos.shape[-1]
        pos_ptr = _int32(pos, "pos", dev, (N, axes) if pos.dim() == 2 else (B, N, axes))
        pos_batch = N * axes if pos.dim() == 3 else 0
    p = RopeParams.from_buffer_copy(params)
    p.dtype, p.D = dtype, D
    if flat_in or flat_out:
        p.flags |= (ROPE_FLAT_IN if flat_in else 0) | (ROPE_FLAT_OUT if flat_out else 0)
    _call(lib().nabla_rope, "nabla_rope", dev, ctypes.byref(p), B, T, H, W, P, 1 if k is None else 2,
          _HEADS(heads, heads_k), ins, outs, pos_ptr, pos_batch, axes)
    return q_out if k is None else (q_out, k_out)


def _rope_view(t, q, shape, dev):
    """nabla_view of [heads, N, D] or [B, heads, N, D] in q's type."""
    s = t.stride()
    if t.dtype != q.dtype or t.get_device() != dev or t.shape != shape or s[-1] != 1 != shape[-1]:
        raise ValueError("q, k and their outputs must be %s tensors on cuda:%d with contiguous rows, "
                         "outputs in their inputs' shapes" % (q.dtype, dev))
    return _VIEW(t.data_ptr(), 0, s[0], s[1]) if len(s) == 3 else _VIEW(t.data_ptr(), *s[:3])


def _packed_of(q, k, cu_q, causal, scale):
    shape = q.shape
    D = shape[-1]
    if k.shape[-1] != D or len(shape) != 3:
        raise ValueError("q must be [total_q, heads, D] and k [total_k, heads_kv, D]")
    return _PACKED(cu_q.shape[0] - 1, shape[1], k.shape[1], D, shape[0], k.shape[0],
                   1 if causal else 0, D ** -0.5 if scale is None else scale)


def packed_workspace(q, k, seqs, back=False):
    """Workspace of the packed calls for q [total_q, heads, D], k [total_k,
    heads_kv, D] and `seqs` sequences; back=True serves both directions.  It
    serves one call at a time."""
    s = _PACKED(int(seqs), q.shape[1], k.shape[1], q.shape[2], q.shape[0], k.shape[0], 0, 1.0)
    n = int(lib().nabla_packed_workspace_size(s, PACKED_BWD if back else PACKED_FWD))
    if n == 0:
        raise NablaError(ERR_SHAPE, "nabla_packed_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def attn_packed_fwd(q, k, v, cu_q, cu_k, causal=False, scale=None, o=None, lse=None, ws=None,
                    want_lse=True):
    """Attention of packed sequences: q [total_q, heads, D], k, v [total_k,
    heads_kv, D] (bf16, any strides of 16 bytes with contiguous rows), borders
    cu_q, cu_k int32 [seqs + 1].  causal aligns the last rows of q and k.
    Returns o (laid out like q) and lse float32 [heads, total_q]; rows of no
    sequence are left as they were, and hold anything where o is not given."""
    dev = _device(q, "q")
    bf = torch.bfloat16
    shape = _packed_of(q, k, cu_q, causal, scale)
    if o is None:
        o = torch.empty_like(q)
    qs = q.shape
    if lse is None and want_lse:
        lse = torch.empty_strided((qs[1], qs[0]), (qs[0], 1), dtype=torch.float32, device=q.device)
    lse_ptr = None if lse is None else _lse(lse, dev, (qs[1], qs[0]))
    ws, ws_bytes = _work(packed_workspace(q, k, cu_q.shape[0] - 1) if ws is None else ws, dev)
    _call(lib().nabla_attn_packed_fwd, "nabla_attn_packed_fwd", dev, shape, _view(q, "q", dev, 3, bf),
          _view(k, "k", dev, 3, bf), _view(v, "v", dev, 3, bf, k.shape), _int32(cu_q, "cu_q", dev),
          _int32(cu_k, "cu_k", dev, cu_q.shape), _view(o, "o", dev, 3, bf, qs), lse_ptr, ws, ws_bytes)
    return o, lse


def attn_packed_bwd(q, k, v, o, dout, lse, cu_q, cu_k, causal=False, scale=None, dq=None, dk=None,
                    dv=None, ws=None):
    """Gradients dq, dk, dv of attn_packed_fwd from its o and lse; rows of no
    sequence as there."""
    dev = _device(q, "q")
    bf = torch.bfloat16
    shape = _packed_of(q, k, cu_q, causal, scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    qs, ks = q.shape, k.shape
    lse_ptr = _lse(lse, dev, (qs[1], qs[0]))
    ws, ws_bytes = _work(packed_workspace(q, k, cu_q.shape[0] - 1, back=True) if ws is None else ws, dev)
    _call(lib().nabla_attn_packed_bwd, "nabla_attn_packed_bwd", dev, shape, _view(q, "q", dev, 3, bf),
          _view(k, "k", dev, 3, bf), _view(v, "v", dev, 3, bf, ks), _view(o, "o", dev, 3, bf, qs),
          _view(dout, "dout", dev, 3, bf, qs), lse_ptr, _int32(cu_q, "cu_q", dev),
          _int32(cu_k, "cu_k", dev, cu_q.shape), _view(dq, "dq", dev, 3, bf, qs),
          _view(dk, "dk", dev, 3, bf, ks), _view(dv, "dv", dev, 3, bf, ks), ws, ws_bytes)
    return dq, dk, dv


def _cache_of(k_cache, v_cache, table, seqs, dev):
    """nabla_cache, heads_kv and D."""
    pages, page, heads_kv, D = shape = k_cache.shape
    width = 1 if table is None else table.shape[-1]
    ptr = 0 if table is None else _int32(table, "table", dev, (seqs, width))
    c = (_view(k_cache, "k_cache", dev, 4, torch.bfloat16)
         + _view(v_cache, "v_cache", dev, 4, torch.bfloat16, shape)
         + _CACHE(ptr, pages, page, heads_kv, D, seqs, width))
    return c, heads_kv, D


def cache_workspace(device):
    """Workspace of cache_append (its status word)."""
    return torch.empty(256, dtype=torch.uint8, device=device)


def cache_append(k, v, k_cache, v_cache, table, starts, cu=None, ws=None):
    """Write rows k, v [total, heads_kv, D] of packed sequences (borders cu
    [seqs + 1]; None: one row each) into the pages [pages, page_size, heads_kv,
    D] behind the starts[s] rows that sequence s has.  table int32 [seqs,
    width].  Rows without a page are skipped; with `ws` (cache_workspace) they
    are reported by status(ws)."""
    dev = _device(k, "k")
    seqs = starts.numel()
    starts_ptr = _int32(starts, "starts", dev, (seqs,))
    cu_ptr = None if cu is None else _int32(cu, "cu", dev, (seqs + 1,))
    c, heads_kv, D = _cache_of(k_cache, v_cache, table, seqs, dev)
    shape = k.shape
    if shape[1:] != (heads_kv, D):
        raise ValueError("k must be [total, %d, %d]" % (heads_kv, D))
    ws, ws_bytes = (None, 0) if ws is None else _work(ws, dev)
    _call(lib().nabla_cache_append, "nabla_cache_append", dev, c, _view(k, "k", dev, 3, torch.bfloat16),
          _view(v, "v", dev, 3, torch.bfloat16, shape), shape[0], starts_ptr, cu_ptr, ws, ws_bytes)


def paged_workspace(q, k_cache):
    """Workspace of attn_paged; it serves one call at a time."""
    c, _, _ = _cache_of(k_cache, k_cache, None, 0, _device(k_cache, "k_cache"))
    n = int(lib().nabla_paged_workspace_size(c, q.shape[1]))
    if n == 0:
        raise NablaError(ERR_SHAPE, "nabla_paged_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def attn_paged(q, k_cache, v_cache, table, lens, scale=None, o=None, lse=None, ws=None,
               want_lse=True):
    """Attention of one new token per sequence, q [seqs, heads, D], over the
    first lens[s] rows of its pages.  Returns o and lse float32 [seqs, heads]."""
    dev = _device(q, "q")
    bf = torch.bfloat16
    shape = q.shape
    view = _view(q, "q", dev, 3, bf)
    seqs, heads, D = shape
    c, _, cache_D = _cache_of(k_cache, v_cache, table, seqs, dev)
    if cache_D != D:
        raise ValueError("q and the cache must have the same D")
    if o is None:
        o = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty_strided((seqs, heads), (heads, 1), dtype=torch.float32, device=q.device)
    lse_ptr = None if lse is None else _lse(lse, dev, (seqs, heads))
    ws, ws_bytes = _work(paged_workspace(q, k_cache) if ws is None else ws, dev)
    _call(lib().nabla_attn_paged, "nabla_attn_paged", dev, c, heads, D ** -0.5 if scale is None else scale,
          view, _int32(lens, "lens", dev, (seqs,)), _view(o, "o", dev, 3, bf, shape), lse_ptr, ws, ws_bytes)
    return o, lse


def status(ws):
    """Synchronise the current stream and return the workspace status word."""
    return int(lib().nabla_status(_ptr(ws), _stream(ws)))
