"""ctypes binding of libmoe.so (the C ABI of include/moe.h).

Argument marshalling only: every step runs in the library's CUDA kernels.
There is no fallback — if libmoe.so is missing or cannot be loaded, every
call raises."""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE = 0, 1, 2, 3
MOE_ERR_CUDA, MOE_ERR_TIMEOUT, MOE_ERR_DEVICE_FAULT = 4, 5, 6
DTYPE_FP8, DTYPE_BF16, DTYPE_F32 = 0, 1, 2
EPI_SCATTER, EPI_STORE, EPI_SWIGLU, EPI_STORE_BF16 = 0, 1, 2, 3
SCHED_QUEUE, SCHED_STATIC = 0, 1
CTRL_BYTES = 256
ATTENTION_CTRL_BYTES = CTRL_BYTES + 65536   # MOE_ATTENTION_CTRL_BYTES
ATTENTION_WS_BYTES = 64 << 20               # MOE_ATTENTION_WS_BYTES

EXPORTS = ["moe_status_string", "moe_num_sms", "moe_route", "moe_layout", "moe_quant_gather",
           "moe_grouped_gemm", "moe_scatter", "moe_workspace_size", "moe_forward",
           "moe_forward_host", "moe_get_error", "moe_debug_set_pipeline_fault", "moe_forward_plan",
           "moe_last_cuda_error", "moe_grouped_gemm_noalloc", "moe_swiglu_quant",
           "moe_forward_workspace_map", "moe_gemm_cta_pairs", "moe_kv_write", "moe_kv_read",
           "moe_paged_attention", "moe_verify_draft"]
WS_NONE = (1 << 64) - 1   # MOE_WS_NONE


class MoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        detail = ""
        if code == MOE_ERR_CUDA:
            detail = " — " + lib().moe_last_cuda_error().decode()
        super().__init__(f"{what}: {status_string(code)} ({code}){detail}")
        self.code = code


class GemmArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("epilogue", ctypes.c_int), ("sched", ctypes.c_int),
                ("block_m", ctypes.c_int), ("E", ctypes.c_int), ("N", ctypes.c_int),
                ("K", ctypes.c_int), ("R", ctypes.c_int), ("M", ctypes.c_int),
                ("top_k", ctypes.c_int), ("a", ctypes.c_void_p), ("a_scales", ctypes.c_void_p),
                ("w", ctypes.c_void_p), ("w_scales", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("tile_offsets", ctypes.c_void_p),
                ("sorted_route_ids", ctypes.c_void_p), ("route_weights", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("k_splits", ctypes.c_int), ("num_ctas", ctypes.c_int),
                ("gather_rows", ctypes.c_int), ("out_scales", ctypes.c_void_p),
                ("cta_pairs", ctypes.c_int)]


class ForwardArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("M", ctypes.c_int), ("K", ctypes.c_int),
                ("N", ctypes.c_int), ("E", ctypes.c_int), ("top_k", ctypes.c_int),
                ("softcap", ctypes.c_float), ("renorm", ctypes.c_int),
                ("logits", ctypes.c_void_p), ("x", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("w_scales", ctypes.c_void_p), ("w2", ctypes.c_void_p),
                ("block_m", ctypes.c_int), ("sched", ctypes.c_int), ("k_splits", ctypes.c_int),
                ("use_graph", ctypes.c_int), ("gather_rows", ctypes.c_int),
                ("gated", ctypes.c_int), ("w2_scales", ctypes.c_void_p),
                ("cta_pairs", ctypes.c_int)]


class WorkspaceMap(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("ids", "weights", "counts", "offsets", "tile_offsets", "sorted_route_ids",
                 "route_slot", "a", "a_scales", "h_q", "h_scales")] + \
               [("a_rows", ctypes.c_int), ("block_m", ctypes.c_int)]


class KvCache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p)]


class AttentionArgs(ctypes.Structure):
    _fields_ = [("cache", KvCache), ("B", ctypes.c_int), ("T", ctypes.c_int),
                ("q_heads", ctypes.c_int), ("max_q", ctypes.c_int), ("max_kv", ctypes.c_int),
                ("table_stride", ctypes.c_int), ("q", ctypes.c_void_p),
                ("q_stride_t", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_stride_t", ctypes.c_int64),
                ("out_stride_h", ctypes.c_int64), ("lse", ctypes.c_void_p),
                ("cu_q", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("scale", ctypes.c_float),
                ("softcap", ctypes.c_float), ("window", ctypes.c_int), ("causal", ctypes.c_int)]


class VerifyArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", ctypes.c_int), ("n", ctypes.c_int),
                ("V", ctypes.c_int), ("p", ctypes.c_void_p), ("p_stride_b", ctypes.c_int64),
                ("p_stride_i", ctypes.c_int64), ("q", ctypes.c_void_p),
                ("q_stride_b", ctypes.c_int64), ("q_stride_i", ctypes.c_int64),
                ("draft", ctypes.c_void_p), ("draft_lens", ctypes.c_void_p),
                ("u_accept", ctypes.c_void_p), ("u_sample", ctypes.c_void_p),
                ("accepted", ctypes.c_void_p), ("tokens", ctypes.c_void_p)]


_lib = None


def lib():
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m mixture_experts_forward_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        L.moe_status_string.argtypes = [I]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_num_sms.restype = I
        L.moe_gemm_cta_pairs.restype = I
        L.moe_last_cuda_error.restype = ctypes.c_char_p
        L.moe_route.argtypes = [P, I, I, I, F, I, P, P, P]
        L.moe_layout.argtypes = [P, I, I, I, I, P, P, P, P, P, P, P]
        L.moe_quant_gather.argtypes = [P, I, I, I, P, P, P, P, I, P]
        L.moe_grouped_gemm.argtypes = [ctypes.POINTER(GemmArgs), P, ctypes.c_size_t, P]
        L.moe_grouped_gemm_noalloc.argtypes = [ctypes.POINTER(GemmArgs), P]
        L.moe_scatter.argtypes = [P, P, P, I, I, I, P, P, P]
        L.moe_swiglu_quant.argtypes = [P, I, I, P, P, P]
        L.moe_workspace_size.argtypes = [ctypes.POINTER(ForwardArgs)]
        L.moe_workspace_size.restype = ctypes.c_size_t
        L.moe_forward.argtypes = [ctypes.POINTER(ForwardArgs), P, P, ctypes.c_size_t, P]
        L.moe_forward_host.argtypes = [ctypes.POINTER(ForwardArgs), P, P, P, P, ctypes.c_size_t, P]
        L.moe_forward_plan.argtypes = [ctypes.POINTER(ForwardArgs), ctypes.POINTER(I),
                                       ctypes.POINTER(I)]
        L.moe_forward_workspace_map.argtypes = [ctypes.POINTER(ForwardArgs),
                                                ctypes.POINTER(WorkspaceMap)]
        L.moe_get_error.argtypes = [P, ctypes.POINTER(ctypes.c_int), P]
        L.moe_debug_set_pipeline_fault.argtypes = [I, ctypes.c_uint64]
        Z = ctypes.c_int64
        L.moe_kv_write.argtypes = [ctypes.POINTER(KvCache), P, P, I, Z, Z, Z, Z, P, P, P]
        L.moe_kv_read.argtypes = [ctypes.POINTER(KvCache), P, I, P, P, I, I, P, P, P, P]
        L.moe_paged_attention.argtypes = [ctypes.POINTER(AttentionArgs), P, ctypes.c_size_t, P]
        L.moe_verify_draft.argtypes = [ctypes.POINTER(VerifyArgs), P, P]
        for name in EXPORTS:
            if name not in ("moe_status_string", "moe_num_sms", "moe_workspace_size",
                            "moe_last_cuda_error", "moe_gemm_cta_pairs"):
                getattr(L, name).restype = I
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().moe_status_string(code).decode()


def _check(code: int, what: str):
    if code != MOE_OK:
        raise MoeError(code, what)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def new_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A zeroed device workspace (the control block must start zeroed)."""
    nbytes = max(int(nbytes), CTRL_BYTES)
    return torch.zeros((nbytes + 255) // 256 * 256, dtype=torch.uint8, device=device)


def _new(shape, dtype, device, stream):
    """An uninitialised result.  With a stream it comes from that stream's memory: a block of the
    current stream's may have been freed while work queued there still reads it.  It is usually
    read on the current stream later, so its release waits for that one too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(t.device)
    if current.cuda_stream != stream.cuda_stream:
        t.record_stream(current)
    return t


# ------------------------------------------------------------------ steps
def route(logits: torch.Tensor, k: int, softcap: float = 0.0, renorm: int = 1, stream=None):
    M, E = logits.shape
    ids = _new((M, k), torch.int32, logits.device, stream)
    w = _new((M, k), torch.float32, logits.device, stream)
    _check(lib().moe_route(_ptr(logits), M, E, k, float(softcap), int(renorm), _ptr(ids), _ptr(w),
                           _stream(stream)), "moe_route")
    return ids, w


def layout(ids: torch.Tensor, E: int, block_m: int, ws: torch.Tensor, stream=None):
    M, k = ids.shape
    R = M * k
    out = {name: _new((n,), torch.int32, ids.device, stream) for name, n in (
        ("counts", E), ("offsets", E + 1), ("sorted_route_ids", R), ("route_slot", R),
        ("tile_offsets", E + 1))}
    _check(lib().moe_layout(_ptr(ids), M, E, k, block_m, _ptr(out["counts"]), _ptr(out["offsets"]),
                            _ptr(out["sorted_route_ids"]), _ptr(out["route_slot"]),
                            _ptr(out["tile_offsets"]), _ptr(ws), _stream(stream)), "moe_layout")
    return out


def quant_gather(x: torch.Tensor, k: int, route_slot: torch.Tensor, zero_acc=None, stream=None):
    M, K = x.shape
    R = M * k
    a_q = _new((R, K), torch.uint8, x.device, stream)
    a_s = _new((K // 128, R), torch.float32, x.device, stream)
    zc = 0 if zero_acc is None else zero_acc.shape[1]
    _check(lib().moe_quant_gather(_ptr(x), M, K, k, _ptr(route_slot), _ptr(a_q), _ptr(a_s),
                                  _ptr(zero_acc), zc, _stream(stream)), "moe_quant_gather")
    return a_q, a_s


def grouped_gemm(*, dtype, epilogue, a, w, offsets, tile_offsets, out, ws, block_m,
                 a_scales=None, w_scales=None, sorted_route_ids=None, route_weights=None,
                 M=0, top_k=0, sched=SCHED_QUEUE, k_splits=0, num_ctas=0, gather_rows=0,
                 out_scales=None, cta_pairs=0, stream=None):
    """moe_grouped_gemm.  gather_rows=1: `a` (and FP8 a_scales) are token-major
    and compact slot s reads row sorted_route_ids[s] // top_k.  FP8 SWIGLU:
    out = u8 [R, N/2] codes of h, out_scales = f32 [N/256, R].  cta_pairs=-1:
    single CTAs only (0: CTA pairs wherever that form exists)."""
    E, N, K = w.shape
    R = sorted_route_ids.numel() if gather_rows else a.shape[0]
    g = GemmArgs(dtype=dtype, epilogue=epilogue, sched=sched, block_m=block_m, E=E, N=N, K=K,
                 R=R, M=M, top_k=top_k, a=a.data_ptr(),
                 a_scales=None if a_scales is None else a_scales.data_ptr(), w=w.data_ptr(),
                 w_scales=None if w_scales is None else w_scales.data_ptr(),
                 offsets=offsets.data_ptr(), tile_offsets=tile_offsets.data_ptr(),
                 sorted_route_ids=None if sorted_route_ids is None else sorted_route_ids.data_ptr(),
                 route_weights=None if route_weights is None else route_weights.data_ptr(),
                 out=out.data_ptr(), k_splits=k_splits, num_ctas=num_ctas,
                 gather_rows=gather_rows,
                 out_scales=None if out_scales is None else out_scales.data_ptr(),
                 cta_pairs=cta_pairs)
    _check(lib().moe_grouped_gemm(ctypes.byref(g), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_grouped_gemm")
    return out


def grouped_gemm_noalloc(*, dtype, epilogue, a, w, offsets, tile_offsets, out, block_m,
                         a_scales=None, w_scales=None, sorted_route_ids=None, route_weights=None,
                         M=0, top_k=0, sched=SCHED_QUEUE, k_splits=0, num_ctas=0,
                         out_scales=None, cta_pairs=0, stream=None):
    """moe_grouped_gemm_noalloc: the same GEMM with the library's own static
    scratch instead of a workspace (for callers that cannot allocate)."""
    E, N, K = w.shape
    g = GemmArgs(dtype=dtype, epilogue=epilogue, sched=sched, block_m=block_m, E=E, N=N, K=K,
                 R=a.shape[0], M=M, top_k=top_k, a=a.data_ptr(),
                 a_scales=None if a_scales is None else a_scales.data_ptr(), w=w.data_ptr(),
                 w_scales=None if w_scales is None else w_scales.data_ptr(),
                 offsets=offsets.data_ptr(), tile_offsets=tile_offsets.data_ptr(),
                 sorted_route_ids=None if sorted_route_ids is None else sorted_route_ids.data_ptr(),
                 route_weights=None if route_weights is None else route_weights.data_ptr(),
                 out=out.data_ptr(), k_splits=k_splits, num_ctas=num_ctas,
                 out_scales=None if out_scales is None else out_scales.data_ptr(),
                 cta_pairs=cta_pairs)
    _check(lib().moe_grouped_gemm_noalloc(ctypes.byref(g), _stream(stream)),
           "moe_grouped_gemm_noalloc")
    return out


def scatter(rows: torch.Tensor, route_slot: torch.Tensor, weights: torch.Tensor,
            ws: torch.Tensor, stream=None):
    """moe_scatter: out bf16 [M, N]; a route with an out-of-range slot records
    MOE_ERR_DEVICE_FAULT in ws's status word (get_error)."""
    M, k = weights.shape
    N = rows.shape[1]
    out = _new((M, N), torch.bfloat16, rows.device, stream)
    _check(lib().moe_scatter(_ptr(rows), _ptr(route_slot), _ptr(weights), M, N, k, _ptr(out),
                             _ptr(ws), _stream(stream)), "moe_scatter")
    return out


def swiglu_quant(gu: torch.Tensor, stream=None):
    """moe_swiglu_quant: gu f32 [R, 2I] (gate columns, then up columns) ->
    (h_q u8 [R, I], h_scales f32 [I/128, R])."""
    R, I2 = gu.shape
    I = I2 // 2
    h_q = _new((R, I), torch.uint8, gu.device, stream)
    h_s = _new((I // 128, R), torch.float32, gu.device, stream)
    _check(lib().moe_swiglu_quant(_ptr(gu), R, I, _ptr(h_q), _ptr(h_s), _stream(stream)),
           "moe_swiglu_quant")
    return h_q, h_s


# ------------------------------------------------------------------ serving
# These calls sit in a serving loop where single tokens cost a few microseconds
# on the device, so the binding itself is kept to plain attribute reads: no
# stream object, no tuple comparisons, one structure per call.
_U8, _BF16, _F32, _I32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32
_raw_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _bad(what: str, why: str):
    raise MoeError(MOE_ERR_INVALID_ARG, f"{what}: {why}")


def _raw_stream(stream, t) -> int:
    """The cudaStream_t of `stream`, or of the current stream of t's device."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream_of is not None and t.is_cuda:
        return _raw_stream_of(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def new_kv_cache(dtype, num_pages, page_size, heads, head_dim, device="cuda"):
    """(k, v, k_scales, v_scales) of a zeroed paged cache; the scales are None
    for DTYPE_BF16."""
    shape = (num_pages, heads, page_size, head_dim)
    fp8 = dtype == DTYPE_FP8
    kv = [torch.zeros(shape, dtype=torch.uint8 if fp8 else torch.bfloat16, device=device)
          for _ in range(2)]
    sc = [torch.zeros(shape[:3], dtype=torch.float32, device=device) if fp8 else None
          for _ in range(2)]
    return (*kv, *sc)


def _cache(what, k, v, k_scales, v_scales) -> KvCache:
    """The cache of these page tensors: u8 codes [P, H, page, D] with f32 scales
    [P, H, page], or bf16 pages without scales."""
    P, H, page, D = k.shape
    if not (v.shape == k.shape and v.dtype is k.dtype and k.is_contiguous() and
            v.is_contiguous()):
        _bad(what, "k and v pages must be contiguous, of one shape and type")
    if k.dtype is _BF16:
        return KvCache(DTYPE_BF16, P, page, H, D, k.data_ptr(), v.data_ptr(), None, None)
    if k.dtype is not _U8:
        _bad(what, "pages are uint8 (E4M3 codes) or bfloat16")
    rows = P * H * page
    if (k_scales is None or v_scales is None or k_scales.dtype is not _F32 or
            v_scales.dtype is not _F32 or k_scales.numel() != rows or v_scales.numel() != rows or
            not k_scales.is_contiguous() or not v_scales.is_contiguous()):
        _bad(what, "an FP8 cache needs f32 scales [pages, heads, page_size]")
    return KvCache(DTYPE_FP8, P, page, H, D, k.data_ptr(), v.data_ptr(), k_scales.data_ptr(),
                   v_scales.data_ptr())


def _ints(t, n) -> bool:
    return t.dtype is _I32 and t.numel() == n and t.is_contiguous()


def _table(what: str, t):
    """(B, table_stride) of a block table: int32 [B, entries], or the columns of a wider one (its
    rows are then as long as the wider table's, all within its storage)."""
    B, entries = t.shape
    if t.dtype is _I32:
        if t.is_contiguous():
            return B, entries
        row, one = t.stride()
        if (row >= entries and (one == 1 or entries == 1) and
                (t.storage_offset() + B * row) * 4 <= t.untyped_storage().nbytes()):
            return B, row
    _bad(what, "block_table is int32 [B, entries] with contiguous rows")


def _placed(what: str, cache, ws, *tensors):
    """Every tensor on the cache's GPU (a host address faults the kernel), and a workspace with
    room for the control block."""
    dev = cache.get_device()
    if dev < 0 or ws.get_device() != dev:
        _bad(what, "all tensors must be on one GPU")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            _bad(what, "all tensors must be on one GPU")
    if ws.numel() * ws.element_size() < CTRL_BYTES:
        raise MoeError(MOE_ERR_WORKSPACE, what)


def kv_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
             v_cache: torch.Tensor, ws: torch.Tensor, k_scales=None, v_scales=None, stream=None):
    """moe_kv_write: k, v bf16 [T, heads, head_dim] (strided views allowed, the
    last dimension contiguous) into the slots s32 [T] of a paged cache."""
    what = "moe_kv_write"
    c = _cache(what, k_cache, v_cache, k_scales, v_scales)
    T, H, D = k.shape
    kt, kh, kd = k.stride()
    vt, vh, vd = v.stride()
    if T == 1:                       # (a dimension of one has any stride)
        kt = vt = 0
    if H == 1:
        kh = vh = 0
    if not (H == c.heads and D == c.head_dim and v.shape == k.shape and k.dtype is _BF16 and
            v.dtype is _BF16 and kd == 1 and vd == 1):
        _bad(what, "k and v are bf16 [T, heads, head_dim] with contiguous rows")
    if not _ints(slots, T):
        _bad(what, "slots is int32 [T]")
    _placed(what, k_cache, ws, v_cache, k_scales, v_scales, k, v, slots)
    code = lib().moe_kv_write(c, k.data_ptr(), v.data_ptr(), T, kt, kh, vt, vh, slots.data_ptr(),
                              ws.data_ptr(), _raw_stream(stream, k))
    if code:
        _check(code, what)


def kv_read(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
            cu_rows: torch.Tensor, rows: int, ws: torch.Tensor, k_scales=None, v_scales=None,
            starts=None, stream=None):
    """moe_kv_read: (k, v) bf16 [rows, heads, head_dim]; rows = cu_rows[-1]."""
    what = "moe_kv_read"
    c = _cache(what, k_cache, v_cache, k_scales, v_scales)
    B, entries = _table(what, block_table)
    if not _ints(cu_rows, B + 1):
        _bad(what, "cu_rows is int32 [B+1]")
    if not (starts is None or _ints(starts, B)):
        _bad(what, "starts is int32 [B]")
    _placed(what, k_cache, ws, v_cache, k_scales, v_scales, block_table, cu_rows, starts)
    shape = (rows, c.heads, c.head_dim)
    k = _new(shape, _BF16, k_cache.device, stream)
    v = _new(shape, _BF16, k_cache.device, stream)
    code = lib().moe_kv_read(c, block_table.data_ptr(), entries, cu_rows.data_ptr(),
                             None if starts is None else starts.data_ptr(), B, rows, k.data_ptr(),
                             v.data_ptr(), ws.data_ptr(), _raw_stream(stream, k_cache))
    if code:
        _check(code, what)
    return k, v


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    block_table: torch.Tensor, cu_q: torch.Tensor, kv_lens: torch.Tensor,
                    ws: torch.Tensor, max_q: int, max_kv: int = 0, k_scales=None, v_scales=None,
                    scale: float = 0.0, softcap: float = 0.0, window: int = 0, causal=True,
                    out=None, lse: bool = False, stream=None):
    """moe_paged_attention: (out bf16 [T, q_heads, head_dim], lse f32 [T, q_heads]
    or None) of q bf16 [T, q_heads, head_dim].  ws: new_workspace(
    ATTENTION_WS_BYTES), kept by the caller for its attention calls."""
    what = "moe_paged_attention"
    c = _cache(what, k_cache, v_cache, k_scales, v_scales)
    T, Hq, D = q.shape
    qt, qh, qd = q.stride()
    B, entries = _table(what, block_table)
    if not (q.dtype is _BF16 and D == c.head_dim and qd == 1):
        _bad(what, "q is bf16 [T, q_heads, head_dim] with contiguous rows")
    if not (_ints(cu_q, B + 1) and _ints(kv_lens, B)):
        _bad(what, "cu_q is int32 [B+1], kv_lens int32 [B]")
    if T > 0 and (B == 0 or max_q <= 0):
        _bad(what, "rows of q, but no sequence or max_q = 0: nothing would write out")
    if out is not None and not (out.dtype is _BF16 and out.shape == q.shape and out.stride(2) == 1):
        _bad(what, "out is bf16, shaped like q, with contiguous rows")
    _placed(what, k_cache, ws, v_cache, k_scales, v_scales, q, block_table, cu_q, kv_lens, out)
    sums = _new((T, Hq), _F32, q.device, stream) if lse else None
    if out is None:
        out = _new((T, Hq, D), _BF16, q.device, stream)
        ot, oh = Hq * D, D
    else:
        ot, oh, _ = out.stride()
    if T == 1:
        qt = ot = 0
    if Hq == 1:
        qh = oh = 0
    a = AttentionArgs(c, B, T, Hq, max_q, max_kv, entries, q.data_ptr(), qt, qh, out.data_ptr(),
                      ot, oh, sums.data_ptr() if lse else None, cu_q.data_ptr(),
                      kv_lens.data_ptr(), block_table.data_ptr(), scale, softcap, window,
                      1 if causal else 0)
    code = lib().moe_paged_attention(a, ws.data_ptr(), ws.numel(), _raw_stream(stream, q))
    if code:
        _check(code, what)
    return out, sums


def verify_draft(p: torch.Tensor, q: torch.Tensor, draft: torch.Tensor, u_accept: torch.Tensor,
                 u_sample: torch.Tensor, ws: torch.Tensor, draft_lens=None, stream=None):
    """moe_verify_draft: (accepted s32 [B], tokens s32 [B, n+1]) of target
    probabilities p [B, n+1, V] and draft probabilities q [B, n, V] (f32 or bf16)."""
    what = "moe_verify_draft"
    B, n, V = q.shape
    pb, pi, pv = p.stride()
    qb, qi, qv = q.stride()
    f32 = q.dtype is _F32
    if not (p.shape == (B, n + 1, V) and p.dtype is q.dtype and (f32 or q.dtype is _BF16) and
            (V == 1 or (pv == 1 and qv == 1))):
        _bad(what, "p is [B, n+1, V] and q [B, n, V], f32 or bf16, with contiguous rows")
    if not (_ints(draft, B * n) and u_accept.dtype is _F32 and u_accept.numel() == B * n and
            u_accept.is_contiguous() and u_sample.dtype is _F32 and u_sample.numel() == B and
            u_sample.is_contiguous()):
        _bad(what, "draft is int32 [B, n], u_accept f32 [B, n], u_sample f32 [B]")
    if not (draft_lens is None or _ints(draft_lens, B)):
        _bad(what, "draft_lens is int32 [B]")
    _placed(what, p, ws, q, draft, draft_lens, u_accept, u_sample)
    accepted = _new((B,), _I32, p.device, stream)
    tokens = _new((B, n + 1), _I32, p.device, stream)
    a = VerifyArgs(DTYPE_F32 if f32 else DTYPE_BF16, B, n, V, p.data_ptr(), pb, pi, q.data_ptr(),
                   qb, qi, draft.data_ptr(), None if draft_lens is None else draft_lens.data_ptr(),
                   u_accept.data_ptr(), u_sample.data_ptr(), accepted.data_ptr(),
                   tokens.data_ptr())
    code = lib().moe_verify_draft(a, ws.data_ptr(), _raw_stream(stream, p))
    if code:
        _check(code, what)
    return accepted, tokens


# ------------------------------------------------------------------ forward
def forward_args(*, dtype, M, K, N, E, top_k, softcap=0.0, renorm=1, logits=None, x=None, w=None,
                 w_scales=None, w2=None, block_m=0, sched=SCHED_QUEUE, k_splits=0,
                 use_graph=1, gather_rows=0, gated=0, w2_scales=None, cta_pairs=0) -> ForwardArgs:
    """Arguments of moe_forward.  gated=1 with dtype FP8: the FP8 gated FFN
    (w = w_up codes [E,2N,K] + w_scales, w2 = w_down codes [E,K,N] + w2_scales).
    cta_pairs=-1: the grouped GEMMs on single CTAs only."""
    return ForwardArgs(dtype=dtype, M=M, K=K, N=N, E=E, top_k=top_k, softcap=float(softcap),
                       renorm=int(renorm), logits=None if logits is None else logits.data_ptr(),
                       x=None if x is None else x.data_ptr(),
                       w=None if w is None else w.data_ptr(),
                       w_scales=None if w_scales is None else w_scales.data_ptr(),
                       w2=None if w2 is None else w2.data_ptr(), block_m=block_m, sched=sched,
                       k_splits=k_splits, use_graph=use_graph, gather_rows=gather_rows,
                       gated=gated,
                       w2_scales=None if w2_scales is None else w2_scales.data_ptr(),
                       cta_pairs=cta_pairs)


def workspace_size(args: ForwardArgs) -> int:
    n = lib().moe_workspace_size(ctypes.byref(args))
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_workspace_size")
    return n


def forward_plan(args: ForwardArgs):
    """(block_m, k_splits) that moe_forward uses for these arguments."""
    bm, ks = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().moe_forward_plan(ctypes.byref(args), ctypes.byref(bm), ctypes.byref(ks)),
           "moe_forward_plan")
    return bm.value, ks.value


def workspace_map(args: ForwardArgs) -> dict:
    """moe_forward_workspace_map: byte offsets of the forward's intermediates
    in its workspace (None for a buffer the forward does not keep), plus
    a_rows and block_m."""
    m = WorkspaceMap()
    _check(lib().moe_forward_workspace_map(ctypes.byref(args), ctypes.byref(m)),
           "moe_forward_workspace_map")
    out = {}
    for name, _ in WorkspaceMap._fields_:
        v = getattr(m, name)
        out[name] = None if (name not in ("a_rows", "block_m") and v == WS_NONE) else v
    return out


def ws_view(ws: torch.Tensor, offset: int, dtype: torch.dtype, shape) -> torch.Tensor:
    """The workspace bytes at ``offset`` viewed as a tensor of dtype/shape
    (no copy)."""
    n = 1
    for s in shape:
        n *= int(s)
    nbytes = n * torch.empty((), dtype=dtype).element_size()
    return ws[offset:offset + nbytes].view(dtype).view(*shape)


def forward(args: ForwardArgs, out: torch.Tensor, ws: torch.Tensor, stream=None):
    _check(lib().moe_forward(ctypes.byref(args), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_forward")
    return out


def forward_host(args: ForwardArgs, host_logits: torch.Tensor, host_x: torch.Tensor,
                 host_out: torch.Tensor, ws: torch.Tensor, stream=None):
    _check(lib().moe_forward_host(ctypes.byref(args), _ptr(host_logits), _ptr(host_x),
                                  _ptr(host_out), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_forward_host")
    return host_out


def get_error(ws: torch.Tensor, stream=None) -> int:
    st = ctypes.c_int(0)
    _check(lib().moe_get_error(_ptr(ws), ctypes.byref(st), _stream(stream)), "moe_get_error")
    return st.value


def debug_set_pipeline_fault(drop_producer: bool, timeout_ns: int = 0):
    _check(lib().moe_debug_set_pipeline_fault(int(drop_producer), int(timeout_ns)),
           "moe_debug_set_pipeline_fault")


def num_sms() -> int:
    return lib().moe_num_sms()


def gemm_cta_pairs() -> int:
    """CTA pairs resident at once for the FP8 scatter GEMM at block_m 128 (0: not used)."""
    return lib().moe_gemm_cta_pairs()
