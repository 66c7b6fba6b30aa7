"""Python binding of libnvfp4moe.so, the MI355X (gfx950) NVFP4 MoE hot path.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in ``include/nvfp4moe.h``.  torch supplies
device memory (``data_ptr()``) and the current stream; nothing here computes
on the host.  If the shared library has not been built this module raises on
import -- there is no fallback path.
"""
import ctypes
import math
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4moe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
        "or `python quantization_nvfp4_quantize_amd/build.py` (needs hipcc for gfx950)")

_lib = ctypes.CDLL(LIB_PATH)

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t


class MoeArgs(ctypes.Structure):
    """Mirror of nvfp4_moe_args (include/nvfp4moe.h)."""
    _fields_ = [
        ("T", _i64), ("H", _i64), ("I", _i64), ("E", _i64), ("topk", _i64),
        ("x", _vp), ("x_gs_in", _vp), ("topk_ids", _vp), ("topk_w", _vp),
        ("w1_q", _vp), ("w1_sf", _vp), ("w1_gs", _vp),
        ("w2_q", _vp), ("w2_sf", _vp), ("w2_gs", _vp),
        ("a2_gs", _vp), ("out", _vp), ("out_dtype", ctypes.c_int),
        ("xq", _vp), ("xsf", _vp), ("x_gs_out", _vp),
        ("l1_c_bf16", _vp), ("l1_q", _vp), ("l1_sf", _vp), ("err_count", _vp),
        ("stage_events", ctypes.POINTER(_vp)),
        ("tile_rows", ctypes.c_int32),
        ("a2_gs_out", _vp),
        ("l1_unfused", ctypes.c_int32),
        ("aux_stream", _vp),
        ("aux_events", ctypes.POINTER(_vp)),
        ("w1_sf_paired", _vp), ("w2_sf_paired", _vp),
    ]


class CachePart(ctypes.Structure):
    """Mirror of kv_cache_part (include/nvfp4moe.h)."""
    _fields_ = [("rows", _vp), ("row_stride", _i64), ("R", _i64), ("q", _vp), ("s", _vp), ("gs", _vp)]


_SIG = {
    "nvfp4_version": (ctypes.c_int, []),
    "nvfp4_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "nvfp4_last_error": (ctypes.c_char_p, []),
    "nvfp4_quantize_workspace_size": (_sz, [_i64, _i64]),
    "nvfp4_quantize": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "nvfp4_dequantize": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, ctypes.c_int, _vp, _vp]),
    "nvfp4_pair_scales": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp]),
    "nvfp4_gemm_swiglu_quant_workspace_size": (_sz, [_i64, _i64, _i64]),
    "nvfp4_gemm_swiglu_quant": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _i64,
                                               _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "nvfp4_linear_workspace_size": (_sz, [_i64, _i64, _i64]),
    "nvfp4_linear": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _i64, ctypes.c_int, _vp, _vp,
                                    _vp, _sz, _vp]),
    "mxfp4_quantize": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "mxfp4_dequantize": (ctypes.c_int, [_vp, _vp, _i64, _i64, ctypes.c_int, _vp, _vp]),
    "mxfp4_linear_workspace_size": (_sz, [_i64, _i64, _i64]),
    "mxfp4_linear": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _i64, ctypes.c_int, _vp, _vp, _sz, _vp]),
    "nvfp4_lora_add_workspace_size": (_sz, [_i64, _i64, _i64, _i64, _i64]),
    "nvfp4_lora_add": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp,
                                      _vp, _sz, _vp]),
    "moe_router_logits_workspace_size": (_sz, [_i64, _i64, _i64, ctypes.c_int]),
    "moe_router_logits": (ctypes.c_int, [_vp, _i64, _i64, _vp, ctypes.c_int, _i64, _vp, _vp, _vp, _sz, _vp]),
    "moe_route": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, ctypes.c_int, _vp, _i64, _i64, ctypes.c_int,
                                 ctypes.c_int, ctypes.c_float, _vp, _vp, _vp, _vp]),
    "nvfp4_matvec": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp, _i64, ctypes.c_int, _vp, _vp]),
    "mxfp4_matvec": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _i64, ctypes.c_int, _vp, _vp]),
    "kv_cache_write": (ctypes.c_int, [ctypes.c_int, _vp, ctypes.c_int, _i64, _vp, _i64, _vp]),
    "kv_cache_read": (ctypes.c_int, [ctypes.c_int, _vp, ctypes.c_int, _i64, _vp, _i64,
                                     ctypes.c_int, _vp]),
    "kv_cache_read_pages": (ctypes.c_int, [ctypes.c_int, _vp, ctypes.c_int, _i64, _vp, _i64, _i64,
                                           _i64, _vp, _i64, ctypes.c_int, _vp]),
    "moe_expert_ffn_nvfp4_workspace_size": (_sz, [ctypes.POINTER(MoeArgs)]),
    "moe_expert_ffn_nvfp4": (ctypes.c_int, [ctypes.POINTER(MoeArgs), _vp, _sz, _vp]),
    "moe_expert_ffn_nvfp4_noalloc": (ctypes.c_int, [ctypes.POINTER(MoeArgs), _vp]),
}
for _name, (_res, _args) in _SIG.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTS = tuple(_SIG)


class Nvfp4Error(RuntimeError):
    def __init__(self, status, where):
        msg = _lib.nvfp4_last_error().decode() or _lib.nvfp4_status_string(status).decode()
        super().__init__(f"{where}: status {status}: {msg}")
        self.status = status


def _check(status, where):
    if status != 0:
        raise Nvfp4Error(status, where)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    if isinstance(device, torch.device) and device.index is not None:
        return torch._C._cuda_getCurrentRawStream(device.index)  # 2 us less than a Stream object
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _require(t, dtype, name):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(nbytes, device):
    """A fresh device workspace of at least nbytes for one call.

    It comes from torch's caching allocator on the current stream, so a block
    is handed out again only after the work queued on that stream has used
    it: calls on different streams never share one, and a graph captured
    around a call keeps its block in the graph's private pool for as long as
    the graph lives.  (The allocator caches freed blocks, so a call of the
    same size costs no device allocation.)"""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _ws_bytes(ws, device):
    """Size of a caller's workspace; its elements have to be memory of their own
    (an expanded view counts bytes that are not there)."""
    if ws.device != device:
        raise ValueError(f"ws must be on {device}, got {ws.device}")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws.numel() * ws.element_size()


def _require_all(device, *specs):
    """Each (tensor or None, dtype, shape, name) on the device and contiguous:
    _require in one pass over the tensors of a short call."""
    index = device.index  # None for host tensors, which get_device() calls -1
    for t, dtype, shape, name in specs:
        if t is None:
            continue
        if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
            _require(t, dtype, name)
            if t.shape != shape:
                raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
            raise ValueError(f"all tensors of a call must be on one device, got {device} and {t.device}")


def _launch(name, device, *args):
    """Call an entry point (its arguments but the stream) on a device's current
    stream, whatever the current device is."""
    index = device.index
    if torch._C._cuda_getDevice() == index:  # half a microsecond less than torch.cuda.current_device()
        status = getattr(_lib, name)(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = getattr(_lib, name)(*args, _stream(device))
    if status != 0:
        raise Nvfp4Error(status, name)


def _at(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ API
def quantize(x, gs=None, out=None):
    """bf16 [M][K] -> (q uint8 [M][K/2], sf uint8 [M][K/16], gs float32 [1]).

    gs: optional float32 [1] device tensor (supplied global scale); by default
    the global scale is max|x| / 2688 computed on the device."""
    _require(x, torch.bfloat16, "x")
    _require(gs, torch.float32, "gs")
    M, K = x.shape
    dev = x.device
    if out is None:
        q = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
        sf = torch.empty((M, K // 16), dtype=torch.uint8, device=dev)
        gs_out = torch.empty(1, dtype=torch.float32, device=dev) if gs is None else None
    else:
        q, sf, gs_out = out
        if gs is not None:
            gs_out = None  # the supplied scale is returned as is; nothing to copy
    wsz = _lib.nvfp4_quantize_workspace_size(M, K)
    ws = _workspace(wsz, dev)
    _check(_lib.nvfp4_quantize(_p(x), M, K, _p(gs), _p(q), _p(sf), _p(gs_out), _p(ws), ws.numel(),
                               _stream(dev)), "nvfp4_quantize")
    return q, sf, (gs if gs is not None else gs_out)


def dequantize(q, sf, gs, out_dtype=torch.bfloat16, out=None):
    """NVFP4 -> bf16 or float32 [M][K]."""
    _require(q, torch.uint8, "q")
    _require(sf, torch.uint8, "sf")
    _require(gs, torch.float32, "gs")
    M, K2 = q.shape
    K = 2 * K2
    if out is None:
        out = torch.empty((M, K), dtype=out_dtype, device=q.device)
    code = {torch.bfloat16: 0, torch.float32: 1}[out.dtype]
    _check(_lib.nvfp4_dequantize(_p(q), _p(sf), _p(gs), M, K, code, _p(out), _stream(q.device)),
           "nvfp4_dequantize")
    return out


def gemm_swiglu_quant(a_q, a_sf, a_gs, w_q, w_sf, w_gs, out_gs, want_bf16=True, out=None, expand_a=True):
    """One expert's L1 stage: returns (c bf16 [M][I] or None, c_q [M][I/2],
    c_sf [M][I/16]).  Weight rows are gate/up interleaved by 8.
    expand_a: pass a workspace (the activations are expanded to f16 once),
    else none (the GEMM dequantizes the NVFP4 activations into LDS)."""
    for t, n, d in ((a_q, "a_q", torch.uint8), (a_sf, "a_sf", torch.uint8), (a_gs, "a_gs", torch.float32),
                    (w_q, "w_q", torch.uint8), (w_sf, "w_sf", torch.uint8), (w_gs, "w_gs", torch.float32),
                    (out_gs, "out_gs", torch.float32)):
        _require(t, d, n)
    M, K = a_q.shape[0], a_q.shape[1] * 2
    N2 = w_q.shape[0]
    I = N2 // 2
    dev = a_q.device
    if out is None:
        c = torch.empty((M, I), dtype=torch.bfloat16, device=dev) if want_bf16 else None
        cq = torch.empty((M, I // 2), dtype=torch.uint8, device=dev)
        csf = torch.empty((M, I // 16), dtype=torch.uint8, device=dev)
    else:
        c, cq, csf = out
    ws = _workspace(_lib.nvfp4_gemm_swiglu_quant_workspace_size(M, K, N2), dev) if expand_a else None
    _check(_lib.nvfp4_gemm_swiglu_quant(_p(a_q), _p(a_sf), _p(a_gs), M, K, _p(w_q), _p(w_sf), _p(w_gs),
                                        N2, _p(out_gs), _p(c), _p(cq), _p(csf), _p(ws),
                                        0 if ws is None else ws.numel(), _stream(dev)), "nvfp4_gemm_swiglu_quant")
    return c, cq, csf


def linear(x, w_q, w_sf, w_gs, out_dtype=torch.bfloat16, x_gs=None, x_gs_out=None, out=None, ws=None):
    """Dense NVFP4 linear: y [M][N] = alpha * NVFP4(x) @ W^T (out_dtype bf16 or
    float32).  x bf16 [M][K]; w_q [N][K/2], w_sf [N][K/16], w_gs float32 [1];
    x_gs: supplied activation global scale (float32 [1]) or None (dynamic);
    x_gs_out: float32 [1] that receives the scale used."""
    _require(x, torch.bfloat16, "x")
    for t, n, d in ((w_q, "w_q", torch.uint8), (w_sf, "w_sf", torch.uint8), (w_gs, "w_gs", torch.float32),
                    (x_gs, "x_gs", torch.float32), (x_gs_out, "x_gs_out", torch.float32)):
        _require(t, d, n)
    M, K = x.shape
    N = w_q.shape[0]
    dev = x.device
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    code = {torch.bfloat16: 0, torch.float32: 1}[out.dtype]
    if ws is None:
        ws = _workspace(_lib.nvfp4_linear_workspace_size(M, K, N), dev)
    _check(_lib.nvfp4_linear(_p(x), M, K, _p(x_gs), _p(w_q), _p(w_sf), _p(w_gs), N, code, _p(out),
                             _p(x_gs_out), _p(ws), ws.numel(), _stream(dev)), "nvfp4_linear")
    return out


def linear_workspace(M, K, N, device):
    """A dedicated workspace for nvfp4_linear (e.g. for graph capture)."""
    return torch.empty(max(int(_lib.nvfp4_linear_workspace_size(M, K, N)), 256), dtype=torch.uint8,
                       device=device)


def lora_add(y, x, a, b, ids, scales=None, out=None, ws=None):
    """The low-rank adapters of many requests, added to the output y of a
    projection they share (linear, mx_linear or another):
    out[t] = y[t] + scales[id] * b[id] @ (a[id] @ x[t]) with id = ids[t], and
    out[t] = y[t] for tokens whose id is outside [0, L).

    y [T][N] bf16 or float32; x bf16 [T][K]: the projection's input; a bf16
    [L][r][K], b bf16 [L][N][r] (smaller ranks padded with zeros); ids int32
    [T]; scales float32 [L].  out: a new tensor by default; pass y to work in
    place (x's memory is fine, too).  ws: a workspace of lora_add_workspace,
    not shared by calls that may run at the same time."""
    if y.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"y must be bfloat16 or float32, got {y.dtype}")
    if y.dim() != 2 or x.dim() != 2 or a.dim() != 3:
        raise ValueError("y and x must be matrices, a [L][r][K] and b [L][N][r]")
    (T, N), K, (L, r, _), dev = y.shape, x.shape[1], a.shape, y.device
    _require_all(dev, (y, y.dtype, (T, N), "y"), (x, torch.bfloat16, (T, K), "x"),
                 (a, torch.bfloat16, (L, r, K), "a"), (b, torch.bfloat16, (L, N, r), "b"),
                 (ids, torch.int32, (T,), "ids"), (scales, torch.float32, (L,), "scales"), (out, y.dtype, (T, N), "out"))
    if out is None:
        out = torch.empty_like(y)
    if ws is None:
        ws = _workspace(_lib.nvfp4_lora_add_workspace_size(T, N, K, r, L), dev)
    nws = _ws_bytes(ws, dev)
    _launch("nvfp4_lora_add", dev, _at(y), 0 if y.dtype == torch.bfloat16 else 1, T, N, _at(x), K, _at(a), _at(b), r,
            L, _at(ids), _at(scales), _at(out), _at(ws), nws)
    return out


def lora_add_workspace(T, N, K, r, L, device):
    """A dedicated workspace for nvfp4_lora_add (e.g. for graph capture)."""
    return torch.empty(max(int(_lib.nvfp4_lora_add_workspace_size(T, N, K, r, L)), 256), dtype=torch.uint8,
                       device=device)


# ------------------------------------------------------------------ few tokens
_OUT_CODE = {torch.bfloat16: 0, torch.float32: 1}


def _out_code(dtype):
    if dtype not in _OUT_CODE:
        raise ValueError(f"the output must be bfloat16 or float32, got {dtype}")
    return _OUT_CODE[dtype]


def _matvec(name, x, w_q, w_s, w_gs, block, out_dtype, out):
    if x.dim() != 2 or w_q.dim() != 2:
        raise ValueError(f"x must be [M][K] and w_q [N][K/2], got {tuple(x.shape)} and {tuple(w_q.shape)}")
    (M, K), N, dev = x.shape, w_q.shape[0], x.device
    _require_all(dev, (x, torch.bfloat16, (M, K), "x"), (w_q, torch.uint8, (N, K // 2), "w_q"),
                 (w_s, torch.uint8, (N, K // block), "the scales"), (w_gs, torch.float32, (1,), "w_gs"))
    if out is None:
        code = _out_code(out_dtype)
        out = torch.empty(M, N, dtype=out_dtype, device=dev)  # sizes one by one: 0.3 us less than a tuple
    else:
        _require_all(dev, (out, out.dtype, (M, N), "out"))
        code = _out_code(out.dtype)
    if block == 16:
        _launch(name, dev, x.data_ptr(), M, K, w_q.data_ptr(), w_s.data_ptr(), w_gs.data_ptr(), N, code, out.data_ptr())
    else:
        _launch(name, dev, x.data_ptr(), M, K, w_q.data_ptr(), w_s.data_ptr(), N, code, out.data_ptr())
    return out


def matvec(x, w_q, w_sf, w_gs, out_dtype=torch.bfloat16, out=None):
    """Products of a few tokens with NVFP4 weights, the activations kept in bf16:
    y [M][N] = x @ deq(W)^T (bf16 or float32).  x bf16 [M][K], K % 32 == 0; w_q
    [N][K/2], w_sf [N][K/16], w_gs float32 [1] as linear takes them, any N.
    out: a tensor to fill, whose type then counts (as in linear).
    Made for M up to 64 (the weights are read once per 64 tokens)."""
    return _matvec("nvfp4_matvec", x, w_q, w_sf, w_gs, 16, out_dtype, out)


def mx_matvec(x, w_q, w_sc, out_dtype=torch.bfloat16, out=None):
    """The same with MXFP4 weights (w_sc [N][K/32] E8M0 codes, as mx_linear)."""
    return _matvec("mxfp4_matvec", x, w_q, w_sc, None, 32, out_dtype, out)


# ------------------------------------------------------------------ quantized cache
# format -> (code, elements per scale, elements per byte of q)
_CACHE = {"nvfp4": (0, 16, 2), "mxfp4": (1, 32, 2), "mxfp8": (2, 32, 1)}


def _cache_format(format):
    if format not in _CACHE:
        raise ValueError(f"format must be one of {sorted(_CACHE)}, got {format!r}")
    return _CACHE[format]


def cache_empty(n_slots, row_shape, format="mxfp8", device="cuda", gs=None):
    """A cache of n_slots rows of row_shape (for instance (heads, dim)), all zeros:
    (q, s), or (q, s, gs) for "nvfp4", whose global scale gs (float32 [1]) is
    supplied."""
    code, block, per = _cache_format(format)
    *lead, dim = row_shape
    if dim <= 0 or dim % block:
        raise ValueError(f"{format} rows need a last dimension that is a multiple of {block}, got {dim}")
    if (gs is None) == (code == 0):
        raise ValueError("a global scale gs goes with format nvfp4, and with no other")
    q = torch.zeros((n_slots, *lead, dim // per), dtype=torch.uint8, device=device)
    s = torch.zeros((n_slots, *lead, dim // block), dtype=torch.uint8, device=device)
    return (q, s) if gs is None else (q, s, gs)


def _cache_part(cache, form, dev):
    """(pointers to q, s and gs, row shape, slots) of one cache, checked.  (One
    condition over both tensors: half of what _require_all takes for them.)"""
    code, block, per = form
    if len(cache) != (2 if code else 3):
        raise ValueError("a cache is (q, s), for nvfp4 (q, s, gs)")
    q, s = cache[0], cache[1]
    if q.dim() < 2:
        raise ValueError("q must be [n_slots][...][bytes]")
    n, *lead, dim = q.shape
    dim *= per
    if dim % block or not dim:
        raise ValueError(f"the last dimension must be whole blocks of {block} elements, got {dim}")
    index = dev.index
    if (q.dtype is not torch.uint8 or s.dtype is not torch.uint8 or s.shape != (n, *lead, dim // block)
            or q.get_device() != index or s.get_device() != index or not q.is_contiguous() or not s.is_contiguous()):
        _require_all(dev, (q, torch.uint8, q.shape, "q"), (s, torch.uint8, (n, *lead, dim // block), "s"))
    if code:
        return (q.data_ptr(), s.data_ptr(), 0), (*lead, dim), n
    gs = cache[2]
    _require_all(dev, (gs, torch.float32, (1,), "gs"))
    return (q.data_ptr(), s.data_ptr(), gs.data_ptr()), (*lead, dim), n


def _pair(v, cache):
    """One tensor with its cache, or two of each -> lists, and whether it was one."""
    one = isinstance(cache[0], torch.Tensor)
    caches = [cache] if one else cache
    if not 1 <= len(caches) <= 2:
        raise ValueError("one cache, or two (keys and values)")
    tensors = [None] * len(caches) if v is None else [v] if isinstance(v, torch.Tensor) else v
    if len(tensors) != len(caches):
        raise ValueError(f"{len(tensors)} tensors for {len(caches)} caches")
    return tensors, caches, one


_PART = struct.Struct("QqqQQQ")  # kv_cache_part


def _rows_of(t, shape):
    """(elements between the rows of t [T][*shape], elements of a row); each row is contiguous."""
    if t.is_contiguous():
        R = math.prod(shape)
        return R, R
    R, strides = 1, t.stride()
    for k in range(len(shape) - 1, -1, -1):
        if strides[k + 1] != R and shape[k] != 1:
            raise ValueError(f"each row must be contiguous, got strides {strides}")
        R *= shape[k]
    return strides[0] if t.shape[0] > 1 else R, R


def _slots(slots):
    if slots.dim() != 1:
        raise ValueError(f"slots must be [T], got {list(slots.shape)}")
    if slots.dtype is not torch.int32 or not slots.is_cuda or not slots.is_contiguous():
        _require(slots, torch.int32, "slots")
    return slots.shape[0]


def cache_write(rows, slots, cache, format="mxfp8"):
    """Quantize rows into a cache: row t goes to slot slots[t] (int32 [T]; slots
    outside the cache are skipped, a slot may occur once).

    rows: bf16 [T][*row_shape]; each row contiguous, the rows any multiple of 8
    elements apart (keys and values may be columns of one projection's output).
    cache: as cache_empty makes it.  rows and cache may also be two of each
    (keys and values), written in one launch.  format: "nvfp4" (the bytes of
    quantize with the cache's gs), "mxfp4" (of mx_quantize) or "mxfp8" (E4M3
    elements, a power of two per 32 at which nothing saturates)."""
    rows, caches, _ = _pair(rows, cache)
    T, dev, form = _slots(slots), slots.device, _cache_format(format)
    parts, n_slots = b"", None
    for x, c in zip(rows, caches):
        held, shape, n = _cache_part(c, form, dev)
        if x.dtype is not torch.bfloat16 or x.shape != (T, *shape) or x.get_device() != dev.index:
            raise ValueError(f"rows must be bfloat16 {[T, *shape]} on {dev}, got {x.dtype} {list(x.shape)} on {x.device}")
        if n != n_slots and n_slots is not None:
            raise ValueError(f"the caches have {n_slots} and {n} slots")
        n_slots = n
        parts += _PART.pack(x.data_ptr(), *_rows_of(x, shape), *held)
    _launch("kv_cache_write", dev, form[0], parts, len(caches), T, slots.data_ptr(), n_slots)


def _cache_read(name, cache, T, format, out_dtype, out, dev, index):
    outs, caches, one = _pair(out, cache)
    form = _cache_format(format)
    code, parts, n_slots, got = _out_code(out_dtype), b"", None, []
    for o, c in zip(outs, caches):
        held, shape, n = _cache_part(c, form, dev)
        if o is None:
            o = torch.empty(T, *shape, dtype=out_dtype, device=dev)
        else:
            _require_all(dev, (o, out_dtype, (T, *shape), "out"))
        if n != n_slots and n_slots is not None:
            raise ValueError(f"the caches have {n_slots} and {n} slots")
        n_slots = n
        parts += _PART.pack(o.data_ptr(), 0, math.prod(shape), *held)
        got.append(o)
    _launch(name, dev, form[0], parts, len(caches), T, *index, n_slots, code)
    return got[0] if one else tuple(got)


def cache_read(cache, slots, format="mxfp8", out_dtype=torch.bfloat16, out=None):
    """Rows of a cache, dequantized: [T][*row_shape] (bf16 or float32) with row t
    from slot slots[t] (int32 [T]), zeros where that is outside the cache.  For
    two caches (keys and values) a pair.  out: tensor(s) to fill, of out_dtype
    (one of another type is refused)."""
    T = _slots(slots)
    return _cache_read("kv_cache_read", cache, T, format, out_dtype, out, slots.device, (slots.data_ptr(),))


def cache_read_pages(cache, pages, cu_lens, page_size, total, format="mxfp8", out_dtype=torch.bfloat16, out=None):
    """The rows of B sequences, one after the other: [total][*row_shape] with rows
    cu_lens[b] .. cu_lens[b + 1] (int32 [B + 1]) those of sequence b, of which
    row i is in slot pages[b][i // page_size] * page_size + i % page_size (pages
    int32 [B][P]).  Rows of pages outside the table or the cache are zeros; rows
    behind the last sequence are left as they were (new tensors: unset)."""
    if pages.dim() != 2:
        raise ValueError("pages must be [B][P]")
    (B, P), dev = pages.shape, pages.device
    _require_all(dev, (pages, torch.int32, (B, P), "pages"), (cu_lens, torch.int32, (B + 1,), "cu_lens"))
    return _cache_read("kv_cache_read_pages", cache, total, format, out_dtype, out, dev,
                       (pages.data_ptr(), B, P, page_size, cu_lens.data_ptr()))


# ------------------------------------------------------------------ MXFP4
# The separately labelled OCP MX v1.0 format (E8M0 scale per 32 elements) on
# the scaled FP4 MFMA; not the NVFP4 of the functions above.
def mx_quantize(x, out=None):
    """bf16 [M][K] (K % 32 == 0) -> (q uint8 [M][K/2], scale codes uint8 [M][K/32])."""
    _require(x, torch.bfloat16, "x")
    M, K = x.shape
    if out is None:
        out = (torch.empty((M, K // 2), dtype=torch.uint8, device=x.device),
               torch.empty((M, K // 32), dtype=torch.uint8, device=x.device))
    q, sc = out
    _check(_lib.mxfp4_quantize(_p(x), M, K, _p(q), _p(sc), _stream(x.device)), "mxfp4_quantize")
    return q, sc


def mx_dequantize(q, sc, out_dtype=torch.bfloat16, out=None):
    """MXFP4 -> bf16 or float32 [M][K]."""
    _require(q, torch.uint8, "q")
    _require(sc, torch.uint8, "scale")
    M, K = q.shape[0], 2 * q.shape[1]
    if out is None:
        out = torch.empty((M, K), dtype=out_dtype, device=q.device)
    code = {torch.bfloat16: 0, torch.float32: 1}[out.dtype]
    _check(_lib.mxfp4_dequantize(_p(q), _p(sc), M, K, code, _p(out), _stream(q.device)), "mxfp4_dequantize")
    return out


def mx_linear(x, w_q, w_sc, out_dtype=torch.bfloat16, out=None, ws=None):
    """Dense MXFP4 linear: y [M][N] = MXFP4(x) @ W^T with W MXFP4 [N][K]."""
    _require(x, torch.bfloat16, "x")
    _require(w_q, torch.uint8, "w_q")
    _require(w_sc, torch.uint8, "w_scale")
    M, K = x.shape
    N = w_q.shape[0]
    dev = x.device
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    code = {torch.bfloat16: 0, torch.float32: 1}[out.dtype]
    if ws is None:
        ws = _workspace(_lib.mxfp4_linear_workspace_size(M, K, N), dev)
    _check(_lib.mxfp4_linear(_p(x), M, K, _p(w_q), _p(w_sc), N, code, _p(out), _p(ws), ws.numel(),
                             _stream(dev)), "mxfp4_linear")
    return out


def mx_linear_workspace(M, K, N, device):
    """A dedicated workspace for mxfp4_linear (e.g. for graph capture)."""
    return torch.empty(max(int(_lib.mxfp4_linear_workspace_size(M, K, N)), 256), dtype=torch.uint8,
                       device=device)


# ------------------------------------------------------------------ router
def router_logits(x, w, bias=None, out=None, ws=None):
    """The router's gate projection: float32 logits [T][E] = x @ w^T (+ bias).
    x bf16 [T][H] (H % 32 == 0); w [E][H] bf16 or float32 (all its bits are
    used); bias float32 [E]."""
    if w.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"w must be bfloat16 or float32, got {w.dtype}")
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError(f"x must be [T][H] and w [E][H], got {tuple(x.shape)} and {tuple(w.shape)}")
    (T, H), E, dev = x.shape, w.shape[0], x.device
    _require_all(dev, (x, torch.bfloat16, (T, H), "x"), (w, w.dtype, (E, H), "w"), (bias, torch.float32, (E,), "bias"),
                 (out, torch.float32, (T, E), "out"))
    if out is None:
        out = torch.empty((T, E), dtype=torch.float32, device=dev)
    code = 0 if w.dtype == torch.bfloat16 else 1
    if ws is None:
        need = _lib.moe_router_logits_workspace_size(T, H, E, code)
        ws = _workspace(need, dev) if need else None
    nws = 0 if ws is None else _ws_bytes(ws, dev)
    _launch("moe_router_logits", dev, _at(x), T, H, _at(w), code, E, _at(bias), _at(out), _at(ws), nws)
    return out


_SCORING = {"softmax": 0, "sigmoid": 1}


def route(logits, topk, scoring="softmax", bias=None, n_group=1, topk_group=1, group_top=1, renormalize=True,
          scale=1.0, n_tokens=None, out=None):
    """Routing of tokens to experts: logits [T][E] (bf16 or float32) -> (ids
    int32 [T][topk], weights float32 [T][topk]), as moe_expert_ffn takes them.
    The logits start at a multiple of 16 bytes (a slice of rows with an odd E
    may need a copy).

    scoring: "softmax" (over the token's experts) or "sigmoid".  bias: float32
    [E], added to the scores for the choice only.  n_group, topk_group,
    group_top: the experts in n_group groups of consecutive ones, of which a
    token uses the topk_group with the largest sum of their group_top (1 or
    2) best choices.  renormalize: divide the chosen scores by their sum;
    scale: factor on the weights.  A NaN or -inf logit (or bias) masks an
    expert; where too few are left, ids are -1 and weights 0, which
    moe_expert_ffn skips.  Experts come best first, ties by the lowest index.
    n_tokens: int32 [1] on the device; rows behind it get id -1, weight 0.
    out: (ids, weights) to fill."""
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"logits must be bfloat16 or float32, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must be [T][E]")
    if scoring not in _SCORING:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}, got {scoring!r}")
    (T, E), dev = logits.shape, logits.device
    if out is None:
        shape = (T, max(topk, 0))
        out = (torch.empty(shape, dtype=torch.int32, device=dev), torch.empty(shape, dtype=torch.float32, device=dev))
    ids, weights = out
    _require_all(dev, (logits, logits.dtype, (T, E), "logits"), (bias, torch.float32, (E,), "bias"),
                 (n_tokens, torch.int32, (1,), "n_tokens"), (ids, torch.int32, (T, max(topk, 0)), "ids"),
                 (weights, torch.float32, (T, max(topk, 0)), "weights"))
    _launch("moe_route", dev, _at(logits), 0 if logits.dtype == torch.bfloat16 else 1, T, E, topk, _SCORING[scoring],
            _at(bias), n_group, topk_group, group_top, int(bool(renormalize)), scale, _at(n_tokens), _at(ids),
            _at(weights))
    return ids, weights


def pair_scales(sf, out=None):
    """A weight block-scale tensor [..., R, C] (uint8, C = K/16 bytes per row)
    in the row-paired layout of nvfp4_pair_scales (each 128-byte line holds
    64 bytes of rows 2j and 2j + 1), for the 32-row MoE tiles.  The leading
    dimensions are taken as more rows (the experts' rows are consecutive);
    needs an even row count per matrix and C % 64 == 0.  Returns a new
    tensor of the same shape (or fills out)."""
    _require(sf, torch.uint8, "sf")
    C = sf.shape[-1]
    R = sf.numel() // C if C else 0
    if out is None:
        out = torch.empty_like(sf)
    _require(out, torch.uint8, "out")
    _check(_lib.nvfp4_pair_scales(_p(sf), R, C, _p(out), _stream(sf.device)), "nvfp4_pair_scales")
    return out


def moe_args(x, topk_ids, topk_w, w1_q, w1_sf, w1_gs, w2_q, w2_sf, w2_gs, a2_gs, out,
             x_gs=None, xq=None, xsf=None, x_gs_out=None, l1_c=None, l1_q=None, l1_sf=None,
             err_count=None, tile_rows=0, a2_gs_out=None, l1_unfused=False, aux=None,
             w1_sf_paired=None, w2_sf_paired=None):
    """Build the nvfp4_moe_args struct from tensors.  The struct holds
    references to every tensor it points at, so they stay allocated for as
    long as the struct lives (a temporary passed here cannot be freed and its
    memory reused while a launch still reads it).
    tile_rows: 0 lets the library choose the GEMM tiles; 32 or 256 forces
    one tile height, 288 the mixed tiling (256-row tiles, each expert's last
    block of at most 64 rows on one or two 32-row tiles).
    a2_gs None: dynamic L1-output global scale (unfused flow); l1_unfused:
    True / 1 the unfused flow with the supplied a2_gs, "interleaved" / 2 the
    interleaved-output flow; a2_gs_out receives the scale.  aux: None, or
    (torch.cuda.Stream, (torch.cuda.Event, torch.cuda.Event)) on which the
    short tiles of the mixed tiling run concurrently (the events must have
    been recorded once, so that they exist); the struct then holds the event
    handle array, which the caller keeps alive with the struct.
    w1_sf_paired, w2_sf_paired: pair_scales(w1_sf), pair_scales(w2_sf), read
    by the 32-row tiles when H (resp. I) is a multiple of 1024."""
    _require(x, torch.bfloat16, "x")
    _require(topk_ids, torch.int32, "topk_ids")
    _require(topk_w, torch.float32, "topk_w")
    T, H = x.shape
    E, N2 = w1_q.shape[0], w1_q.shape[1]
    k = topk_ids.shape[1]
    code = {torch.bfloat16: 0, torch.float32: 1}[out.dtype]
    a = MoeArgs(T, H, N2 // 2, E, k, _p(x), _p(x_gs), _p(topk_ids), _p(topk_w),
                _p(w1_q), _p(w1_sf), _p(w1_gs), _p(w2_q), _p(w2_sf), _p(w2_gs), _p(a2_gs),
                _p(out), code, _p(xq), _p(xsf), _p(x_gs_out), _p(l1_c), _p(l1_q), _p(l1_sf),
                _p(err_count))
    _require(w1_sf_paired, torch.uint8, "w1_sf_paired")
    _require(w2_sf_paired, torch.uint8, "w2_sf_paired")
    a._refs = (x, topk_ids, topk_w, w1_q, w1_sf, w1_gs, w2_q, w2_sf, w2_gs, a2_gs, out, x_gs, xq, xsf, x_gs_out,
               l1_c, l1_q, l1_sf, err_count, a2_gs_out, w1_sf_paired, w2_sf_paired)
    a.w1_sf_paired = _p(w1_sf_paired)
    a.w2_sf_paired = _p(w2_sf_paired)
    a.tile_rows = int(tile_rows)
    a.a2_gs_out = _p(a2_gs_out)
    a.l1_unfused = {False: 0, True: 1, 0: 0, 1: 1, 2: 2, "interleaved": 2}[l1_unfused]
    if aux is not None:
        stream, (ev0, ev1) = aux
        a._aux_events = (ctypes.c_void_p * 2)(ev0.cuda_event, ev1.cuda_event)
        a.aux_stream = stream.cuda_stream
        a.aux_events = ctypes.cast(a._aux_events, ctypes.POINTER(ctypes.c_void_p))
    return a


def moe_workspace_size(args):
    return int(_lib.moe_expert_ffn_nvfp4_workspace_size(ctypes.byref(args)))


def moe_expert_ffn_raw(args, device, ws=None):
    """Launch with a prepared MoeArgs (the bench's hot loop uses this)."""
    need = moe_workspace_size(args)
    if ws is None:
        ws = _workspace(need, device)
    _check(_lib.moe_expert_ffn_nvfp4(ctypes.byref(args), _p(ws), ws.numel(), _stream(device)),
           "moe_expert_ffn_nvfp4")


def moe_expert_ffn_noalloc(args, device):
    """Launch with a prepared MoeArgs on the library's static per-GPU scratch
    buffer (moe_expert_ffn_nvfp4_noalloc): no workspace is allocated here
    or in the library.  Calls that overlap on one GPU race on that buffer."""
    _check(_lib.moe_expert_ffn_nvfp4_noalloc(ctypes.byref(args), _stream(device)), "moe_expert_ffn_nvfp4_noalloc")


def moe_expert_ffn(x, topk_ids, topk_w, w1_q, w1_sf, w1_gs, w2_q, w2_sf, w2_gs, a2_gs,
                   out_dtype=torch.bfloat16, x_gs=None, debug=False, tile_rows=0, l1_unfused=False,
                   aux=None, w1_sf_paired=None, w2_sf_paired=None):
    """NVFP4 MoE expert FFN.  Returns y [T][H] (out_dtype), plus with
    debug=True a dict of the intermediate outputs (xq, xsf, x_gs, l1_c,
    l1_q, l1_sf, err_count, a2_gs_out).  a2_gs None: dynamic L1-output
    global scale.  tile_rows, l1_unfused, aux, w1_sf_paired, w2_sf_paired:
    see moe_args."""
    T, H = x.shape
    I = w1_q.shape[1] // 2
    k = topk_ids.shape[1]
    P = T * k
    dev = x.device
    out = torch.empty((T, H), dtype=out_dtype, device=dev)
    dbg = {}
    if debug:
        dbg = dict(xq=torch.empty((T, H // 2), dtype=torch.uint8, device=dev),
                   xsf=torch.empty((T, H // 16), dtype=torch.uint8, device=dev),
                   x_gs_out=torch.empty(1, dtype=torch.float32, device=dev),
                   l1_c=torch.zeros((P, I), dtype=torch.bfloat16, device=dev),
                   l1_q=torch.zeros((P, I // 2), dtype=torch.uint8, device=dev),
                   l1_sf=torch.zeros((P, I // 16), dtype=torch.uint8, device=dev),
                   err_count=torch.zeros(1, dtype=torch.int32, device=dev),
                   a2_gs_out=torch.empty(1, dtype=torch.float32, device=dev))
    args = moe_args(x, topk_ids, topk_w, w1_q, w1_sf, w1_gs, w2_q, w2_sf, w2_gs, a2_gs, out,
                    x_gs=x_gs, tile_rows=tile_rows, l1_unfused=l1_unfused, aux=aux,
                    w1_sf_paired=w1_sf_paired, w2_sf_paired=w2_sf_paired, **dbg)
    moe_expert_ffn_raw(args, dev)
    if debug:
        return out, dbg
    return out


def quantize_experts(w, gs_out=None):
    """Quantize a stack of expert weight matrices [E][R][K] (bf16), each with
    its own dynamic global scale.  Returns (q [E][R][K/2], sf [E][R][K/16],
    gs float32 [E]).  Model preparation, not part of the hot path."""
    E, R, K = w.shape
    dev = w.device
    q = torch.empty((E, R, K // 2), dtype=torch.uint8, device=dev)
    sf = torch.empty((E, R, K // 16), dtype=torch.uint8, device=dev)
    gs = torch.empty(E, dtype=torch.float32, device=dev) if gs_out is None else gs_out
    for e in range(E):
        quantize(w[e], out=(q[e], sf[e], gs[e:e + 1]))
    return q, sf, gs
