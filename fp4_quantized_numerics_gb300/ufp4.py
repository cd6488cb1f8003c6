"""Thin ctypes binding of libufp4 (include/ufp4.h).

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels.  PyTorch provides device memory and the current stream.  There
is no fallback: if libufp4.so is missing or a tensor is not on a CUDA device,
the calls raise.  The library launches on the current device: tensors and
streams of another one are refused (call under torch.cuda.device).

Where a call takes stream=, the results that it makes belong to that stream,
as if made under torch.cuda.stream(stream): work of another stream that uses
them waits for it and, if they may be dropped before it ends, marks them
(Tensor.record_stream).  The same holds the other way round for operands made
on another stream.

The functions carry the C names:
  ufp4_quantize(x, grid, ...) -> QTensor
  ufp4_dequantize(q, ...)     -> fp32 tensor
  ufp4_gemm(a, b, ...)        -> fp32 tensor (C = A B^T)
  ufp4_stats(x, q, ...)       -> dict
  ufp4_check(...), ufp4_status_string(...)
  ufp4_moe_sort(ids, n_experts) -> MoePlan;  ufp4_moe_dispatch / _combine / _combine_bwd
  ufp4_ckpt_save(x, fmt) -> Ckpt;  ufp4_ckpt_load(c) -> tensor
  ufp4_swiglu(gate, up, ...)  -> (h, Ckpt, Ckpt);  ufp4_swiglu_bwd(dh, ...) -> (dgate, dup)
  ufp4_gemv(x, w), ufp4_gemv_grouped(x, w, plan, rows) -> tensor (unquantized tokens times quantized weights)
  ufp4_cache_append(k, v, slots, cache);  ufp4_cache_load(cache, slots) -> (k, v)
  ufp4_cache_attn(q, cache, table, lens, ...) -> tensor, or (tensor, lse)
"""
import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libufp4.so")

UFP4_E2M1, UFP4_E1M2, UFP4_E2M1C, UFP4_MXFP4 = 0, 1, 2, 3
UFP4_BLOCK, UFP4_MX_BLOCK = 16, 32
UFP4_RTNE, UFP4_SR = 0, 1
UFP4_BF16, UFP4_FP32 = 0, 1
UFP4_CKPT_INT8, UFP4_CKPT_E4M3 = 0, 1
UFP4_CKPT_BLOCK = 32
UFP4_OK, UFP4_ERR_INVALID, UFP4_ERR_UNSUPPORTED, UFP4_ERR_NONFINITE, UFP4_ERR_CUDA, \
    UFP4_ERR_TIMEOUT = range(6)

EXPORTED = ["ufp4_kpad", "ufp4_codes_bytes", "ufp4_scales_bytes", "ufp4_workspace_bytes",
            "ufp4_quantize", "ufp4_check", "ufp4_dequantize", "ufp4_gemm", "ufp4_stats",
            "ufp4_status_string", "ufp4_quantize_noalloc", "ufp4_grouped_rows",
            "ufp4_grouped_kpad", "ufp4_quantize_grouped", "ufp4_gemm_grouped", "ufp4_quantize_dual",
            "ufp4_gemm_amax", "ufp4_quantize_stats", "ufp4_quantize_grouped_dual", "ufp4_moe_sort",
            "ufp4_moe_dispatch", "ufp4_moe_combine", "ufp4_moe_combine_bwd", "ufp4_ckpt_ld",
            "ufp4_ckpt_codes_bytes", "ufp4_ckpt_scales_bytes", "ufp4_ckpt_save", "ufp4_ckpt_load",
            "ufp4_swiglu", "ufp4_swiglu_bwd", "ufp4_gemv", "ufp4_gemv_grouped", "ufp4_cache_dim",
            "ufp4_cache_append", "ufp4_cache_load", "ufp4_cache_attn_workspace_bytes", "ufp4_cache_attn"]


class QParamsC(ctypes.Structure):
    _fields_ = [("grid", ctypes.c_int32), ("block", ctypes.c_int32), ("rht", ctypes.c_int32),
                ("round", ctypes.c_int32), ("rht_seed", ctypes.c_uint64),
                ("sr_seed", ctypes.c_uint64), ("sr_counter", ctypes.c_uint64),
                ("colwise", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("amax_in", ctypes.c_void_p)]


class QTensorC(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("tensor_scale", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("k", ctypes.c_int64), ("grid", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("eplane", ctypes.c_void_p)]


class StatsC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in
                ("alpha", "sqnr_db", "mean_bias", "sum_aq", "sum_aa", "sum_err2", "bias_count")]


class GemmGroupC(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("a_row", ctypes.c_int64), ("a_k", ctypes.c_int64), ("b_row", ctypes.c_int64),
                ("b_k", ctypes.c_int64), ("a_seg", ctypes.c_int32), ("b_seg", ctypes.c_int32),
                ("c", ctypes.c_void_p), ("ldc", ctypes.c_int64)]


class MoePlanC(ctypes.Structure):
    _fields_ = [("pos", ctypes.c_void_p), ("src", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("tokens", ctypes.c_int64), ("topk", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class CkptC(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("format", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class CacheC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "k_row_scale", "v_codes", "v_scales",
                                               "v_row_scale")] + \
               [("pages", ctypes.c_int64)] + \
               [(n, ctypes.c_int32) for n in ("heads", "page", "head_dim", "grid", "rht", "reserved")] + \
               [("rht_seed", ctypes.c_uint64)]


class UFP4Error(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        super().__init__("%s: %s (status %d)" % (what, ufp4_status_string(status), status))


_lib = None


def lib():
    """The loaded libufp4 (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libufp4.so is not built (run fp4_quantized_numerics_gb300.build.build())")
        L = ctypes.CDLL(LIB_PATH)
        i64, vp = ctypes.c_int64, ctypes.c_void_p
        L.ufp4_kpad.argtypes = [i64]
        L.ufp4_kpad.restype = i64
        L.ufp4_codes_bytes.argtypes = [i64, i64]
        L.ufp4_codes_bytes.restype = i64
        L.ufp4_scales_bytes.argtypes = [i64, i64]
        L.ufp4_scales_bytes.restype = i64
        L.ufp4_workspace_bytes.argtypes = []
        L.ufp4_workspace_bytes.restype = ctypes.c_size_t
        L.ufp4_quantize.argtypes = [vp, ctypes.c_int32, i64, i64, i64, ctypes.POINTER(QParamsC),
                                    ctypes.POINTER(QTensorC), vp, ctypes.c_size_t, vp]
        L.ufp4_quantize.restype = ctypes.c_int
        L.ufp4_quantize_dual.argtypes = [vp, ctypes.c_int32, i64, i64, i64, ctypes.POINTER(QParamsC),
                                         ctypes.POINTER(QParamsC), ctypes.POINTER(QTensorC),
                                         ctypes.POINTER(QTensorC), vp, ctypes.c_size_t, vp]
        L.ufp4_quantize_dual.restype = ctypes.c_int
        L.ufp4_check.argtypes = [vp, vp]
        L.ufp4_check.restype = ctypes.c_int
        L.ufp4_dequantize.argtypes = [ctypes.POINTER(QTensorC), ctypes.c_int32, ctypes.c_uint64,
                                      vp, i64, vp]
        L.ufp4_dequantize.restype = ctypes.c_int
        L.ufp4_gemm.argtypes = [ctypes.POINTER(QTensorC), ctypes.POINTER(QTensorC), vp, i64, vp]
        L.ufp4_gemm.restype = ctypes.c_int
        L.ufp4_gemm_amax.argtypes = [ctypes.POINTER(QTensorC), ctypes.POINTER(QTensorC), vp, i64,
                                     ctypes.c_int32, ctypes.c_uint64, vp, vp]
        L.ufp4_gemm_amax.restype = ctypes.c_int
        L.ufp4_stats.argtypes = [vp, ctypes.c_int32, i64, i64, i64, ctypes.POINTER(QParamsC),
                                 ctypes.POINTER(QTensorC), vp, ctypes.c_size_t,
                                 ctypes.POINTER(StatsC), vp]
        L.ufp4_stats.restype = ctypes.c_int
        L.ufp4_quantize_stats.argtypes = [vp, ctypes.c_int32, i64, i64, i64, ctypes.POINTER(QParamsC),
                                          ctypes.POINTER(QTensorC), vp, ctypes.c_size_t,
                                          ctypes.POINTER(StatsC), vp]
        L.ufp4_quantize_stats.restype = ctypes.c_int
        i64p = ctypes.POINTER(ctypes.c_int64)
        L.ufp4_grouped_rows.argtypes = [i64p, ctypes.c_int32]
        L.ufp4_grouped_rows.restype = i64
        L.ufp4_grouped_kpad.argtypes = [i64p, ctypes.c_int32]
        L.ufp4_grouped_kpad.restype = i64
        L.ufp4_quantize_grouped.argtypes = [vp, ctypes.c_int32, i64, i64, i64p, ctypes.c_int32,
                                            ctypes.POINTER(QParamsC), ctypes.POINTER(QTensorC), vp,
                                            ctypes.c_size_t, vp]
        L.ufp4_quantize_grouped.restype = ctypes.c_int
        L.ufp4_quantize_grouped_dual.argtypes = [vp, ctypes.c_int32, i64, i64, i64p, ctypes.c_int32,
                                                 ctypes.POINTER(QParamsC), ctypes.POINTER(QParamsC),
                                                 ctypes.POINTER(QTensorC), ctypes.POINTER(QTensorC), vp,
                                                 ctypes.c_size_t, vp]
        L.ufp4_quantize_grouped_dual.restype = ctypes.c_int
        L.ufp4_gemm_grouped.argtypes = [ctypes.POINTER(QTensorC), ctypes.POINTER(QTensorC),
                                        ctypes.POINTER(GemmGroupC), ctypes.c_int32, vp]
        L.ufp4_gemm_grouped.restype = ctypes.c_int
        i32, plan, ck = ctypes.c_int32, ctypes.POINTER(MoePlanC), ctypes.POINTER(CkptC)
        u64, qt, cache = ctypes.c_uint64, ctypes.POINTER(QTensorC), ctypes.POINTER(CacheC)
        for name, args in (
                ("ufp4_moe_sort", [vp, i32, plan, vp]),
                ("ufp4_moe_dispatch", [vp, i32, i64, i64, plan, vp, i64, vp]),
                ("ufp4_moe_combine", [vp, i32, i64, i64, plan, vp, vp, i32, i64, vp]),
                ("ufp4_moe_combine_bwd", [vp, i32, i64, vp, i32, i64, i64, plan, vp, vp, i32, i64, vp, vp]),
                ("ufp4_ckpt_save", [vp, i32, i64, ck, vp]),
                ("ufp4_ckpt_load", [ck, vp, i32, i64, vp]),
                ("ufp4_swiglu", [vp, i64, vp, i64, i32, i64, i64, vp, i32, i64, ck, ck, vp]),
                ("ufp4_swiglu_bwd", [vp, i32, i64, ck, ck, vp, i64, vp, i64, i32, vp]),
                ("ufp4_gemv", [vp, i32, i64, i64, qt, i32, u64, vp, i32, i64, vp]),
                ("ufp4_gemv_grouped", [vp, i32, i64, i32, qt, i64, plan, i32, u64, vp, i32, i64, vp]),
                ("ufp4_cache_append", [vp, vp, i32, i64, i64, i64, i64, i64, vp, cache, vp]),
                ("ufp4_cache_load", [cache, vp, i64, vp, vp, i32, i64, i64, i64, i64, vp]),
                ("ufp4_cache_attn", [vp, i32, i64, i64, i64, i32, i32, cache, vp, i64, i64, vp, vp, ctypes.c_float, vp,
                                     i32, i64, i64, vp, vp, ctypes.c_size_t, vp])):
            f = getattr(L, name)
            f.argtypes, f.restype = args, ctypes.c_int
        for name, args in (("ufp4_ckpt_ld", [i64]), ("ufp4_ckpt_codes_bytes", [i64, i64]),
                           ("ufp4_ckpt_scales_bytes", [i64, i64])):
            f = getattr(L, name)
            f.argtypes, f.restype = args, i64
        L.ufp4_cache_dim.argtypes, L.ufp4_cache_dim.restype = [i64], i64
        L.ufp4_cache_attn_workspace_bytes.argtypes = [i64, i32, i32, i64, cache]
        L.ufp4_cache_attn_workspace_bytes.restype = ctypes.c_size_t
        L.ufp4_status_string.argtypes = [ctypes.c_int]
        L.ufp4_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def ufp4_status_string(status):
    return lib().ufp4_status_string(int(status)).decode()


def _check(status, what):
    if status != UFP4_OK:
        raise UFP4Error(status, what)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    else:
        _here(stream.device_index, "stream")
    return ctypes.c_void_p(stream.cuda_stream)


def _for(stream):
    """Allocations for `stream` (None: the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    _here(stream.device_index, "stream")
    return torch.cuda.stream(stream)


def _on_gpu(t, name):
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError("%s must be a CUDA tensor (libufp4 has no CPU path)" % name)


def _cuda(t, name):
    _on_gpu(t, name)
    _here(t.get_device(), name)


def _here(index, name):
    if index != _current_device():
        raise ValueError("%s is on cuda:%d, the current device is cuda:%d" % (name, index, _current_device()))


_workspaces = {}


def workspace(device=None):
    """A per-device scratch buffer of ufp4_workspace_bytes() (allocated once);
    calls that may run at the same time on several streams need their own (ws=)."""
    dev = torch.device("cuda") if device is None else torch.device(device)
    if dev.index is None:
        dev = torch.device(dev.type, torch.cuda.current_device())
    key = (dev.type, dev.index)
    ws = _workspaces.get(key)
    if ws is None:
        ws = torch.empty(int(lib().ufp4_workspace_bytes()), dtype=torch.uint8, device=dev)
        _workspaces[key] = ws
    return ws


def _workspace_for(stream, device):
    with _for(stream):
        return workspace(device)


class QTensor:
    """Quantized tensor: device codes / scales / tensor scale in the layouts
    of include/ufp4.h, logical shape rows x k; E1M2 tensors may carry the
    correction plane (eplane) that the quantizer writes and the GEMM loads."""

    def __init__(self, codes, scales, tensor_scale, rows, k, grid, eplane=None):
        self.codes, self.scales, self.tensor_scale = codes, scales, tensor_scale
        self.rows, self.k, self.grid = int(rows), int(k), int(grid)
        self.eplane = eplane

    @classmethod
    def empty(cls, rows, k, grid, device="cuda", eplane=None):
        """eplane: allocate the E1M2 correction plane (default: for E1M2)."""
        L = lib()
        codes = torch.empty(max(int(L.ufp4_codes_bytes(rows, k)), 1), dtype=torch.uint8, device=device)
        scales = torch.empty(max(int(L.ufp4_scales_bytes(rows, k)), 1), dtype=torch.uint8, device=device)
        ts = torch.empty(1, dtype=torch.float32, device=device)
        if eplane is None:
            eplane = int(grid) == UFP4_E1M2
        ep = torch.empty_like(codes) if eplane and int(grid) == UFP4_E1M2 else None
        return cls(codes, scales, ts, rows, k, grid, ep)

    @property
    def kpad(self):
        return int(lib().ufp4_kpad(self.k))

    def c(self):
        return QTensorC(self.codes.data_ptr(), self.scales.data_ptr(), self.tensor_scale.data_ptr(),
                        self.rows, self.k, self.grid, 0,
                        None if self.eplane is None else self.eplane.data_ptr())

    def ungrouped(self):
        """Forgets the segments of a grouped quantization that was kept here before."""
        self.__dict__.pop("seg_rows", None)

    def codes_2d(self):
        """codes as uint8 [rows, kpad/2] (a view)."""
        return self.codes[: self.rows * (self.kpad // 2)].view(self.rows, self.kpad // 2)


def _dtype_code(x):
    if x.dtype == torch.bfloat16:
        return UFP4_BF16
    if x.dtype == torch.float32:
        return UFP4_FP32
    raise TypeError("libufp4 quantizes bf16 or fp32 tensors, got %s" % x.dtype)


def qparams(grid, rht=False, rht_seed=0, round=UFP4_RTNE, sr_seed=0, sr_counter=0,
            colwise=False, amax_in=None):
    block = UFP4_MX_BLOCK if int(grid) == UFP4_MXFP4 else UFP4_BLOCK
    return QParamsC(int(grid), block, int(bool(rht)), int(round), int(rht_seed) & (2**64 - 1),
                    int(sr_seed) & (2**64 - 1), int(sr_counter) & (2**64 - 1), int(bool(colwise)), 0,
                    None if amax_in is None else amax_in.data_ptr())


def ufp4_quantize(x, grid, rht=False, rht_seed=0, round=UFP4_RTNE, sr_seed=0, sr_counter=0,
                  colwise=False, amax_in=None, out=None, ws=None, stream=None):
    """Fused (RHT +) block quantization of a 2-D bf16/fp32 CUDA tensor.
    Row-wise: blocks along the last dim, result rows x cols.  colwise=True:
    blocks down the columns, result is the quantization of x.T."""
    _cuda(x, "x")
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit stride in its last dim")
    rows, cols = x.shape
    out_rows, k = (cols, rows) if colwise else (rows, cols)
    if out is None:
        with _for(stream):
            out = QTensor.empty(out_rows, k, grid, x.device)
    if ws is None:
        ws = _workspace_for(stream, x.device)
    p = qparams(grid, rht, rht_seed, round, sr_seed, sr_counter, colwise, amax_in)
    qc = out.c()
    st = lib().ufp4_quantize(x.data_ptr(), _dtype_code(x), rows, cols, x.stride(0), ctypes.byref(p),
                             ctypes.byref(qc), ws.data_ptr(), ws.numel(), _stream(stream))
    _check(st, "ufp4_quantize")
    out.ungrouped()
    return out


def ufp4_quantize_dual(x, grid, rht=False, rht_seed=0, round=UFP4_RTNE, sr_seed=0, sr_counter_row=0,
                       sr_counter_col=0, amax_row=None, amax_col=None, out_row=None, out_col=None, ws=None,
                       stream=None):
    """Row-wise and column-wise quantization of x (results x and x.T
    quantized along their last dim) from one read of x per pass."""
    _cuda(x, "x")
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit stride in its last dim")
    rows, cols = x.shape
    with _for(stream):
        if out_row is None:
            out_row = QTensor.empty(rows, cols, grid, x.device)
        if out_col is None:
            out_col = QTensor.empty(cols, rows, grid, x.device)
    if ws is None:
        ws = _workspace_for(stream, x.device)
    pr = qparams(grid, rht, rht_seed, round, sr_seed, sr_counter_row, False, amax_row)
    pc = qparams(grid, rht, rht_seed, round, sr_seed, sr_counter_col, True, amax_col)
    qr, qc = out_row.c(), out_col.c()
    st = lib().ufp4_quantize_dual(x.data_ptr(), _dtype_code(x), rows, cols, x.stride(0), ctypes.byref(pr),
                                  ctypes.byref(pc), ctypes.byref(qr), ctypes.byref(qc), ws.data_ptr(),
                                  ws.numel(), _stream(stream))
    _check(st, "ufp4_quantize_dual")
    out_row.ungrouped()
    out_col.ungrouped()
    return out_row, out_col


def ufp4_check(ws=None, stream=None):
    return lib().ufp4_check(None if ws is None else ws.data_ptr(), _stream(stream))


def ufp4_dequantize(q, inverse_rht=False, rht_seed=0, out=None, stream=None):
    _cuda(q.codes, "q.codes")
    if out is None:
        with _for(stream):
            out = torch.empty(q.rows, q.k, dtype=torch.float32, device=q.codes.device)
    qc = q.c()
    st = lib().ufp4_dequantize(ctypes.byref(qc), int(bool(inverse_rht)), int(rht_seed),
                               out.data_ptr(), out.stride(0), _stream(stream))
    _check(st, "ufp4_dequantize")
    return out


def ufp4_gemm(a, b, out=None, stream=None):
    """C = A B^T (fp32), A: M x K and B: N x K quantized along K."""
    _cuda(a.codes, "a.codes")
    _cuda(b.codes, "b.codes")
    if out is None:   # row stride rounded up to 4 floats (16 bytes), as the ABI requires
        ld = (b.rows + 3) // 4 * 4
        with _for(stream):
            out = torch.empty(a.rows, ld, dtype=torch.float32, device=a.codes.device)[:, : b.rows]
    ac, bc = a.c(), b.c()
    st = lib().ufp4_gemm(ctypes.byref(ac), ctypes.byref(bc), out.data_ptr(), out.stride(0),
                         _stream(stream))
    _check(st, "ufp4_gemm")
    return out


def ufp4_gemm_amax(a, b, rht=False, rht_seed=0, out=None, amax=None, stream=None):
    """C = A B^T as ufp4_gemm, and the tensor amax of C's row-wise
    quantization (rotated with rht_seed when rht) from the epilogue.
    Returns (C, amax); pass amax as the amax_in of ufp4_quantize(C, ...)."""
    _cuda(a.codes, "a.codes")
    _cuda(b.codes, "b.codes")
    with _for(stream):
        if out is None:
            ld = (b.rows + 3) // 4 * 4
            out = torch.empty(a.rows, ld, dtype=torch.float32, device=a.codes.device)[:, : b.rows]
        if amax is None:
            amax = torch.empty(1, dtype=torch.float32, device=a.codes.device)
    ac, bc = a.c(), b.c()
    st = lib().ufp4_gemm_amax(ctypes.byref(ac), ctypes.byref(bc), out.data_ptr(), out.stride(0),
                              int(bool(rht)), int(rht_seed) & (2**64 - 1), amax.data_ptr(), _stream(stream))
    _check(st, "ufp4_gemm_amax")
    return out, amax


def ufp4_quantize_stats(x, grid, rht=False, rht_seed=0, round=UFP4_RTNE, sr_seed=0, sr_counter=0,
                        colwise=False, amax_in=None, out=None, ws=None, stream=None):
    """ufp4_quantize and ufp4_stats of its result in one call (one read of x
    where the layout allows).  Returns (QTensor, stats dict); synchronises."""
    _cuda(x, "x")
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit stride in its last dim")
    rows, cols = x.shape
    out_rows, k = (cols, rows) if colwise else (rows, cols)
    if out is None:
        with _for(stream):
            out = QTensor.empty(out_rows, k, grid, x.device)
    if ws is None:
        ws = _workspace_for(stream, x.device)
    p = qparams(grid, rht, rht_seed, round, sr_seed, sr_counter, colwise, amax_in)
    qc = out.c()
    res = StatsC()
    st = lib().ufp4_quantize_stats(x.data_ptr(), _dtype_code(x), rows, cols, x.stride(0), ctypes.byref(p),
                                   ctypes.byref(qc), ws.data_ptr(), ws.numel(), ctypes.byref(res),
                                   _stream(stream))
    _check(st, "ufp4_quantize_stats")
    out.ungrouped()
    return out, {n: getattr(res, n) for n, _ in StatsC._fields_}


def ufp4_stats(x, q, rht=False, rht_seed=0, round=UFP4_RTNE, sr_seed=0, sr_counter=0,
               colwise=False, amax_in=None, ws=None, stream=None):
    """alpha, SQNR and mean rounding bias of quantization q of x (synchronises)."""
    _cuda(x, "x")
    rows, cols = x.shape
    if ws is None:
        ws = _workspace_for(stream, x.device)
    p = qparams(q.grid, rht, rht_seed, round, sr_seed, sr_counter, colwise, amax_in)
    qc = q.c()
    out = StatsC()
    st = lib().ufp4_stats(x.data_ptr(), _dtype_code(x), rows, cols, x.stride(0), ctypes.byref(p),
                          ctypes.byref(qc), ws.data_ptr(), ws.numel(), ctypes.byref(out),
                          _stream(stream))
    _check(st, "ufp4_stats")
    return {n: getattr(out, n) for n, _ in StatsC._fields_}


# ------------------------------------------------------------ grouped (MoE)
def _i64_array(vals):
    arr = (ctypes.c_int64 * len(vals))(*[int(v) for v in vals])
    return arr


def grouped_rows(seg_rows):
    return int(lib().ufp4_grouped_rows(_i64_array(seg_rows), len(seg_rows)))


def grouped_kpad(seg_rows):
    return int(lib().ufp4_grouped_kpad(_i64_array(seg_rows), len(seg_rows)))


def grouped_offsets(seg_rows, colwise):
    """Row offsets (row-wise) or k offsets (column-wise) of each segment."""
    offs, o = [], 0
    for t in seg_rows:
        offs.append(o)
        if t > 0:
            o += ((t + 63) // 64 * 64) if colwise else ((t + 127) // 128 * 128)
    return offs


def ufp4_quantize_grouped(x, grid, seg_rows, rht=False, rht_seed=0, round=UFP4_RTNE, sr_seed=0,
                          sr_counter=0, colwise=False, out=None, ws=None, stream=None):
    """Quantize the row segments of x, one tensor scale per segment (layouts:
    include/ufp4.h, grouped tensors).  Returns a QTensor whose tensor_scale
    holds one S_dec per segment."""
    _cuda(x, "x")
    cols = x.shape[1]
    n = len(seg_rows)
    if colwise:
        rows, k = cols, grouped_kpad(seg_rows)
    else:
        rows, k = grouped_rows(seg_rows), cols
    if out is None:
        with _for(stream):
            out = QTensor.empty(rows, k, grid, x.device)
            out.tensor_scale = torch.empty(max(n, 1), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = _workspace_for(stream, x.device)
    p = qparams(grid, rht, rht_seed, round, sr_seed, sr_counter, colwise)
    qc = out.c()
    st = lib().ufp4_quantize_grouped(x.data_ptr(), _dtype_code(x), cols, x.stride(0),
                                     _i64_array(seg_rows), n, ctypes.byref(p), ctypes.byref(qc),
                                     ws.data_ptr(), ws.numel(), _stream(stream))
    _check(st, "ufp4_quantize_grouped")
    out.seg_rows = list(seg_rows)
    return out


def ufp4_quantize_grouped_dual(x, grid, seg_rows, rht=False, rht_seed=0, round=UFP4_RTNE, sr_seed=0,
                               sr_counter_row=0, sr_counter_col=0, out_row=None, out_col=None, ws=None,
                               stream=None):
    """Row-wise and column-wise grouped quantization of x from one read of x
    per pass; each result as its own ufp4_quantize_grouped call."""
    _cuda(x, "x")
    cols = x.shape[1]
    n = len(seg_rows)
    with _for(stream):
        if out_row is None:
            out_row = QTensor.empty(grouped_rows(seg_rows), cols, grid, x.device)
            out_row.tensor_scale = torch.empty(max(n, 1), dtype=torch.float32, device=x.device)
        if out_col is None:
            out_col = QTensor.empty(cols, grouped_kpad(seg_rows), grid, x.device)
            out_col.tensor_scale = torch.empty(max(n, 1), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = _workspace_for(stream, x.device)
    pr = qparams(grid, rht, rht_seed, round, sr_seed, sr_counter_row, False)
    pc = qparams(grid, rht, rht_seed, round, sr_seed, sr_counter_col, True)
    qr, qc = out_row.c(), out_col.c()
    st = lib().ufp4_quantize_grouped_dual(x.data_ptr(), _dtype_code(x), cols, x.stride(0),
                                          _i64_array(seg_rows), n, ctypes.byref(pr), ctypes.byref(pc),
                                          ctypes.byref(qr), ctypes.byref(qc), ws.data_ptr(), ws.numel(),
                                          _stream(stream))
    _check(st, "ufp4_quantize_grouped_dual")
    out_row.seg_rows = list(seg_rows)
    out_col.seg_rows = list(seg_rows)
    return out_row, out_col


def ufp4_gemm_grouped(a, b, groups, stream=None):
    """groups: list of dicts with keys M, N, K, a_row, a_k, b_row, b_k, a_seg,
    b_seg and c (an fp32 CUDA tensor view of M x N with unit column stride)."""
    _cuda(a.codes, "a.codes")
    _cuda(b.codes, "b.codes")
    arr = (GemmGroupC * max(len(groups), 1))()
    for i, g in enumerate(groups):
        c = g["c"]
        arr[i] = GemmGroupC(g["M"], g["N"], g["K"], g["a_row"], g["a_k"], g["b_row"], g["b_k"],
                            g["a_seg"], g["b_seg"], c.data_ptr(), c.stride(0))
    ac, bc = a.c(), b.c()
    st = lib().ufp4_gemm_grouped(ctypes.byref(ac), ctypes.byref(bc), arr, len(groups), _stream(stream))
    _check(st, "ufp4_gemm_grouped")


# ------------------------------------------- around the grouped GEMMs (MoE)
# These calls are also made a token at a time, where the binding's own time
# counts: one stream query without a Stream object, results allocated by the
# shortest route torch offers (the one its own compiled code takes; measured
# 1.5 -> 0.9 us alone and 3 to 5 us less between other calls), no second check
# of buffers made here.
try:
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    _empty_strided_cuda = None
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_INT32, _INT64, _FLOAT32 = torch.int32, torch.int64, torch.float32


def _place(t, name):
    """Device index of a call's first operand: the current device."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        _on_gpu(t, name)
    dev = t.get_device()
    if dev != _current_device():
        _here(dev, name)
    return dev


def _same_place(index, dev, name):
    if index < 0:
        raise TypeError("%s must be a CUDA tensor (libufp4 has no CPU path)" % name)
    if index != dev:
        raise ValueError("%s is on cuda:%d, the other operands are on cuda:%d" % (name, index, dev))


def _streams(stream, dev):
    """The handle of the stream to launch on, and that stream where it is not
    the current one: results have to be made there, because the caching
    allocator gives out a block in the order of one stream's work."""
    if stream is None:
        return _current_raw_stream(dev), None
    _same_place(stream.device_index, dev, "stream")
    raw = stream.cuda_stream
    return raw, None if raw == _current_raw_stream(dev) else stream


def _empty(shape, dtype, dev, on=None):
    """A fresh contiguous tensor (one to three dims) on the current device, for
    use on stream `on` (None: the current one)."""
    global _empty_strided_cuda
    if on is not None:
        with torch.cuda.stream(on):
            return _empty(shape, dtype, dev)
    if _empty_strided_cuda is not None:
        try:
            return _empty_strided_cuda(shape, (shape[1], 1) if len(shape) == 2 else (1,) if len(shape) == 1 else
                                       (shape[1] * shape[2], shape[2], 1), dtype)
        except TypeError:
            pass
    out = torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev))
    _empty_strided_cuda = None   # (not there, or of a torch where it takes other arguments)
    return out


def _device(device):
    """A torch.device with its index."""
    device = torch.device(device)
    if device.type != "cuda":
        raise TypeError("libufp4 has no CPU path")
    return device if device.index is not None else torch.device("cuda", torch.cuda.current_device())


class MoePlan:
    """Expert order of a routed batch (layouts: include/ufp4.h): pos int32
    [tokens, topk], src int32 [tokens * topk], counts int64 [n_experts],
    offsets int64 [n_experts + 1].  counts.tolist() is the seg_rows of the
    grouped calls; rows past offsets[-1] belong to dropped slots."""

    def __init__(self, pos, src, counts, offsets):
        if not (pos.is_cuda and src.is_cuda and counts.is_cuda and offsets.is_cuda):
            raise TypeError("the plan's tensors must be CUDA tensors (libufp4 has no CPU path)")
        dev = pos.get_device()
        if not (src.get_device() == dev and counts.get_device() == dev and offsets.get_device() == dev):
            raise ValueError("the plan's tensors must be on one device")
        if not (pos.dtype is _INT32 and src.dtype is _INT32 and counts.dtype is _INT64 and offsets.dtype is _INT64):
            raise ValueError("pos and src must be int32, counts and offsets int64")
        if not (pos.is_contiguous() and src.is_contiguous() and counts.is_contiguous() and offsets.is_contiguous()):
            raise ValueError("the plan's tensors must be contiguous")
        if pos.dim() != 2:
            raise ValueError("pos must be [tokens, topk]")
        tokens, topk = pos.shape
        n_experts = counts.numel()
        if src.numel() != tokens * topk or offsets.numel() != n_experts + 1:
            raise ValueError("src must have pos's elements, offsets one more than counts")
        self._set(pos, src, counts, offsets, tokens, topk, n_experts, dev)

    def _set(self, pos, src, counts, offsets, tokens, topk, n_experts, dev):
        self.pos, self.src, self.counts, self.offsets = pos, src, counts, offsets
        self.tokens, self.topk, self.n_experts, self._dev = tokens, topk, n_experts, dev
        self._c = ctypes.byref(MoePlanC(pos.data_ptr(), src.data_ptr(), counts.data_ptr(), offsets.data_ptr(),
                                        tokens, topk, n_experts, 0))

    @classmethod
    def empty(cls, tokens, topk, n_experts, device="cuda"):
        device = _device(device)
        with torch.cuda.device(device):
            return cls._new(tokens, topk, n_experts, device.index)

    @classmethod
    def _new(cls, tokens, topk, n_experts, dev, on=None):
        plan = cls.__new__(cls)
        plan._set(_empty((tokens, topk), _INT32, dev, on), _empty((tokens * topk,), _INT32, dev, on),
                  _empty((n_experts,), _INT64, dev, on), _empty((n_experts + 1,), _INT64, dev, on),
                  tokens, topk, n_experts, dev)
        return plan

    def c(self):
        return self._c


_DTYPES = {torch.bfloat16: UFP4_BF16, torch.float32: UFP4_FP32}


def _rows2d(t, name, dev, rows=None, cols=None):
    """Checks a 2-D tensor on device `dev` with unit stride in its last dim, of
    the given shape.  Returns its pointer, dtype code, row stride, rows and cols."""
    if not isinstance(t, torch.Tensor):
        _on_gpu(t, name)
    if t.get_device() != dev:
        _same_place(t.get_device(), dev, name)
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must be 2-D" % name)
    r, c = shape
    ld, unit = t.stride()
    if unit != 1 and c > 1:
        raise ValueError("%s must have unit stride in its last dim" % name)
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError("%s must be %s x %s, got %d x %d" % (name, rows, cols, r, c))
    if r <= 1 and ld < c:   # the stride of a single row says nothing
        ld = c
    dt = _DTYPES.get(t.dtype)
    return t.data_ptr(), _dtype_code(t) if dt is None else dt, ld, r, c


def _result(out, name, rows, cols, dtype, default, dev, on):
    """A fresh rows x cols result (of `dtype`, or of the default's where that
    is None), or the caller's, checked: the tensor, its pointer, dtype code and
    row stride."""
    if out is None:
        dtype = dtype or default
        dt = _DTYPES.get(dtype)
        if dt is None:
            raise TypeError("%s must be bf16 or fp32, got %s" % (name, dtype))
        out = _empty((rows, cols), dtype, dev, on)
        return out, out.data_ptr(), dt, cols
    p, dt, ld, _, _ = _rows2d(out, name, dev, rows, cols)
    if dtype is not None and out.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, out.dtype))
    return out, p, dt, ld


def _struct(held, dev, name="plan"):
    """The C struct of a plan or checkpoint on device `dev`."""
    if held._dev != dev:
        _same_place(held._dev, dev, name)
    return held._c


def _plan_weights(weights, plan, dev, name="weights"):
    if weights.get_device() != dev:
        _same_place(weights.get_device(), dev, name)
    if weights.dtype is not _FLOAT32 or weights.shape != plan.pos.shape or not weights.is_contiguous():
        raise ValueError("%s must be contiguous fp32 [tokens, topk]" % name)
    return weights.data_ptr()


def ufp4_moe_sort(ids, n_experts, out=None, stream=None):
    """Stable sort of the slots of ids ([tokens, topk], int32 or int64) by
    expert; ids outside [0, n_experts) are dropped.  Returns a MoePlan."""
    dev = _place(ids, "ids")
    if ids.dim() != 2 or not ids.is_contiguous():
        raise ValueError("ids must be contiguous [tokens, topk]")
    size = 8 if ids.dtype is _INT64 else 4 if ids.dtype is _INT32 else 0
    if not size:
        raise TypeError("ids must be int32 or int64, got %s" % ids.dtype)
    tokens, topk = ids.shape
    s, on = _streams(stream, dev)
    if out is None:
        out = MoePlan._new(tokens, topk, n_experts, dev, on)
    elif (out.tokens, out.topk, out.n_experts) != (tokens, topk, n_experts):
        raise ValueError("out is a plan of another size")
    st = lib().ufp4_moe_sort(ids.data_ptr(), size, _struct(out, dev, "out"), s)
    _check(st, "ufp4_moe_sort")
    return out


def ufp4_moe_dispatch(x, plan, out=None, stream=None):
    """x ([tokens, hidden]) in expert order: [tokens * topk, hidden], dropped
    slots' rows (the last ones) zero.  Gradient: ufp4_moe_combine(dxs, plan)."""
    dev = _place(x, "x")
    pc, (s, on) = _struct(plan, dev), _streams(stream, dev)
    xp, dt, ld, _, hidden = _rows2d(x, "x", dev, plan.tokens)
    out, op, _, old = _result(out, "out", plan.tokens * plan.topk, hidden, x.dtype, None, dev, on)
    st = lib().ufp4_moe_dispatch(xp, dt, hidden, ld, pc, op, old, s)
    _check(st, "ufp4_moe_dispatch")
    return out


def ufp4_moe_combine(y, plan, weights=None, dtype=None, out=None, stream=None):
    """y ([tokens * topk, hidden], expert order) back in token order: the sum
    over each token's routed slots, times weights ([tokens, topk] fp32) if
    given.  dtype: the result's (y's by default)."""
    dev = _place(y, "y")
    pc, (s, on) = _struct(plan, dev), _streams(stream, dev)
    yp, dt, ld, _, hidden = _rows2d(y, "y", dev, plan.tokens * plan.topk)
    w = None if weights is None else _plan_weights(weights, plan, dev)
    out, op, odt, old = _result(out, "out", plan.tokens, hidden, dtype, y.dtype, dev, on)
    st = lib().ufp4_moe_combine(yp, dt, hidden, ld, pc, w, op, odt, old, s)
    _check(st, "ufp4_moe_combine")
    return out


def ufp4_moe_combine_bwd(dout, y, plan, weights, dtype=None, dy=None, dw=None, stream=None):
    """Gradients of ufp4_moe_combine(y, plan, weights): (dy, dw).  dtype: dy's
    (dout's by default)."""
    dev = _place(y, "y")
    pc, (s, on) = _struct(plan, dev), _streams(stream, dev)
    yp, ydt, yld, rows, hidden = _rows2d(y, "y", dev, plan.tokens * plan.topk)
    dp, ddt, dld, _, _ = _rows2d(dout, "dout", dev, plan.tokens, hidden)
    w = _plan_weights(weights, plan, dev)
    dwp = None if dw is None else _plan_weights(dw, plan, dev, "dw")
    dy, gp, gdt, gld = _result(dy, "dy", rows, hidden, dtype, dout.dtype, dev, on)
    if dw is None:
        dw = _empty((plan.tokens, plan.topk), _FLOAT32, dev, on)
        dwp = dw.data_ptr()
    st = lib().ufp4_moe_combine_bwd(dp, ddt, dld, yp, ydt, yld, hidden, pc, w, gp, gdt, gld, dwp, s)
    _check(st, "ufp4_moe_combine_bwd")
    return dy, dw


class Ckpt:
    """An activation kept in 8 bits (layouts: include/ufp4.h): codes uint8
    [rows, ufp4_ckpt_ld(cols)], scales uint8 [rows, ceil(cols / 32)]."""

    def __init__(self, codes, scales, rows, cols, format):
        for t, name, width in ((codes, "codes", self._ld(cols)), (scales, "scales", self._blocks(cols))):
            _on_gpu(t, name)
            if t.dtype != torch.uint8 or tuple(t.shape) != (rows, width) or not t.is_contiguous():
                raise ValueError("%s must be contiguous uint8 [%d, %d]" % (name, rows, width))
        _same_place(scales.get_device(), codes.get_device(), "scales")
        self._codes, self._scales = codes, scales
        self._set(codes.data_ptr(), scales.data_ptr(), rows, cols, format, codes.get_device())

    def _set(self, codes, scales, rows, cols, format, dev):
        self.rows, self.cols, self.format, self._dev = rows, cols, int(format), dev
        self._c = ctypes.byref(CkptC(codes, scales, rows, cols, self.format, 0))

    @staticmethod
    def _ld(cols):
        return (cols + 15) // 16 * 16

    @staticmethod
    def _blocks(cols):
        return (cols + UFP4_CKPT_BLOCK - 1) // UFP4_CKPT_BLOCK

    @classmethod
    def empty(cls, rows, cols, format, device="cuda"):
        device = _device(device)
        with torch.cuda.device(device):
            return cls._new(1, rows, cols, format, device.index)[0]

    @classmethod
    def _new(cls, count, rows, cols, format, dev, on=None):
        """`count` checkpoints of one shape in one buffer; the views of their
        codes and scales are made when asked for."""
        n = rows * cls._ld(cols)
        step = (n + rows * cls._blocks(cols) + 15) // 16 * 16
        buf = _empty((count * step,), torch.uint8, dev, on)
        at, made = buf.data_ptr(), []
        for k in range(count):
            c = cls.__new__(cls)
            c._buf, c._at, c._codes, c._scales = buf, k * step, None, None
            c._set(at + k * step, at + k * step + n, rows, cols, format, dev)
            made.append(c)
        return made

    def _view(self, first, rows, width):
        return self._buf[self._at + first:self._at + first + rows * width].view(rows, width)

    @property
    def device(self):
        return torch.device("cuda", self._dev)

    @property
    def codes(self):
        if self._codes is None:
            self._codes = self._view(0, self.rows, self._ld(self.cols))
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._scales = self._view(self.rows * self._ld(self.cols), self.rows, self._blocks(self.cols))
        return self._scales

    def c(self):
        return self._c


def ufp4_ckpt_save(x, format=UFP4_CKPT_INT8, out=None, stream=None):
    """x (2-D bf16 / fp32) in 8 bits with a power-of-two scale per 32
    elements of a row.  Returns a Ckpt."""
    dev = _place(x, "x")
    xp, dt, ld, rows, cols = _rows2d(x, "x", dev)
    s, on = _streams(stream, dev)
    if out is None:
        out = Ckpt._new(1, rows, cols, format, dev, on)[0]
    elif (out.rows, out.cols, out.format) != (rows, cols, format):
        raise ValueError("out is a checkpoint of another shape or format")
    st = lib().ufp4_ckpt_save(xp, dt, ld, _struct(out, dev, "out"), s)
    _check(st, "ufp4_ckpt_save")
    return out


def ufp4_ckpt_load(c, dtype=None, out=None, stream=None):
    """The values of a checkpoint (exact in bf16 and fp32).  dtype: the
    result's (bf16 by default)."""
    dev = c._dev
    _here(dev, "c")
    s, on = _streams(stream, dev)
    out, op, odt, old = _result(out, "out", c.rows, c.cols, dtype, torch.bfloat16, dev, on)
    st = lib().ufp4_ckpt_load(c._c, op, odt, old, s)
    _check(st, "ufp4_ckpt_load")
    return out


def ufp4_swiglu(gate, up, ckpt=None, dtype=None, out=None, keep=None, stream=None):
    """h = silu(gate) * up, and gate's and up's 8-bit checkpoints for the
    backward pass (ckpt: their format, or None to keep nothing; keep: a pair
    of Ckpts to write instead of new ones, of that format if it is given).
    Returns (h, keep_gate, keep_up), the latter two None if nothing is kept.
    dtype: h's (gate's by default).  New checkpoints share one buffer, which
    is held until both are dropped."""
    dev = _place(gate, "gate")
    gp, dt, gld, rows, cols = _rows2d(gate, "gate", dev)
    up_p, udt, uld, _, _ = _rows2d(up, "up", dev, rows, cols)
    if udt != dt:
        raise TypeError("gate and up must have one dtype")
    s, on = _streams(stream, dev)
    kg = ku = None
    if keep is not None:
        kg, ku = keep
        if ckpt is not None and not (kg and ku and kg.format == ku.format == ckpt):
            raise ValueError("keep must be two checkpoints of the format ckpt=%s" % ckpt)
    elif ckpt is not None:
        kg, ku = Ckpt._new(2, rows, cols, ckpt, dev, on)
    out, hp, hdt, hld = _result(out, "out", rows, cols, dtype, gate.dtype, dev, on)
    st = lib().ufp4_swiglu(gp, gld, up_p, uld, dt, rows, cols, hp, hdt, hld, kg and _struct(kg, dev, "keep"),
                           ku and _struct(ku, dev, "keep"), s)
    _check(st, "ufp4_swiglu")
    return out, kg, ku


def ufp4_swiglu_bwd(dh, keep_gate, keep_up, dtype=None, dgate=None, dup=None, stream=None):
    """Gradients of ufp4_swiglu from its checkpoints: (dgate, dup).  dtype:
    the gradients' (dh's by default)."""
    dev = _place(dh, "dh")
    kg, ku = _struct(keep_gate, dev, "keep_gate"), _struct(keep_up, dev, "keep_up")
    s, on = _streams(stream, dev)
    rows, cols = keep_gate.rows, keep_gate.cols
    dp, ddt, dld, _, _ = _rows2d(dh, "dh", dev, rows, cols)
    dgate, gp, gdt, gld = _result(dgate, "dgate", rows, cols, dtype, dh.dtype, dev, on)
    dup, up, udt, uld = _result(dup, "dup", rows, cols, dgate.dtype, None, dev, on)
    st = lib().ufp4_swiglu_bwd(dp, ddt, dld, kg, ku, gp, gld, up, uld, gdt, s)
    _check(st, "ufp4_swiglu_bwd")
    return dgate, dup


# --------------------------------------- answering with a quantized model
def _tokens(x, name, dev, k):
    """Checks a 2-D operand of k columns; its pointer, dtype code, row stride and rows."""
    p, dt, ld, rows, _ = _rows2d(x, name, dev, None, k)
    return p, dt, ld, rows


def _weights(w, dev):
    if w.codes.get_device() != dev:
        _same_place(w.codes.get_device(), dev, "w")
    return ctypes.byref(w.c())


def ufp4_gemv(x, w, rht=False, rht_seed=0, dtype=None, out=None, stream=None):
    """x W^T for a few tokens: x [tokens, k] bf16 or fp32, not quantized, and w
    a QTensor (rows x k; not a grouped one of several segments).  rht: w was
    quantized with that rotation, and x's 16-blocks are rotated to match.  Returns [tokens, rows] of `dtype` (x's by
    default)."""
    dev = _place(x, "x")
    if len(getattr(w, "seg_rows", ())) > 1:
        raise ValueError("w is a grouped tensor of %d segments, each with a tensor scale of its own" % len(w.seg_rows))
    xp, dt, ld, tokens = _tokens(x, "x", dev, w.k)
    wc, (s, on) = _weights(w, dev), _streams(stream, dev)
    out, yp, ydt, yld = _result(out, "out", tokens, w.rows, dtype, x.dtype, dev, on)
    st = lib().ufp4_gemv(xp, dt, tokens, ld, wc, 1 if rht else 0, rht_seed, yp, ydt, yld, s)
    _check(st, "ufp4_gemv")
    return out


def ufp4_gemv_grouped(x, w, plan, rows, gather=False, rht=False, rht_seed=0, dtype=None, out=None, stream=None):
    """ufp4_gemv by expert, the counts read on the device: w is a grouped
    row-wise QTensor of n_experts segments of `rows` rows.  x: [tokens * topk,
    k] in expert order, or with gather=True [tokens, k], each place taking its
    token's row.  Returns [tokens * topk, rows] in expert order; the rows of
    dropped slots are zeros."""
    dev = _place(x, "x")
    pc, (s, on) = _struct(plan, dev), _streams(stream, dev)
    slots = plan.tokens * plan.topk
    xp, dt, ld, _, _ = _rows2d(x, "x", dev, plan.tokens if gather else slots, w.k)
    wc = _weights(w, dev)
    if w.tensor_scale.numel() != plan.n_experts:
        raise ValueError("w must have one tensor scale for each of the plan's %d experts" % plan.n_experts)
    out, yp, ydt, yld = _result(out, "out", slots, rows, dtype, x.dtype, dev, on)
    st = lib().ufp4_gemv_grouped(xp, dt, ld, 1 if gather else 0, wc, rows, pc, 1 if rht else 0, rht_seed, yp, ydt, yld,
                                 s)
    _check(st, "ufp4_gemv_grouped")
    return out


class Cache:
    """Keys and values in 4 bits, in pages (layouts: include/ufp4.h): for each,
    codes uint8 [pages, heads, page, ufp4_cache_dim(head_dim) / 2], scales uint8
    [pages, heads, page, ufp4_cache_dim(head_dim) / 16] and row_scale fp32
    [pages, heads, page].  rht: kept rotated, with the signs of rht_seed."""

    def __init__(self, k_codes, k_scales, k_row_scale, v_codes, v_scales, v_row_scale, head_dim, grid, rht=False,
                 rht_seed=0):
        _on_gpu(k_codes, "k_codes")
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [pages, heads, page, width]")
        pages, heads, page, _ = k_codes.shape
        dev, pad = k_codes.get_device(), self._pad(head_dim)
        rows = (pages, heads, page)
        for shape, dtype, pair, names in ((rows + (pad // 2,), torch.uint8, (k_codes, v_codes), "codes"),
                                          (rows + (pad // 16,), torch.uint8, (k_scales, v_scales), "scales"),
                                          (rows, _FLOAT32, (k_row_scale, v_row_scale), "row_scale")):
            for t in pair:
                if t.get_device() != dev:
                    _same_place(t.get_device(), dev, names)
                if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
                    raise ValueError("%s must be contiguous %s %s" % (names, dtype, shape))
        self.k_codes, self.k_scales, self.k_row_scale = k_codes, k_scales, k_row_scale
        self.v_codes, self.v_scales, self.v_row_scale = v_codes, v_scales, v_row_scale
        self.pages, self.heads, self.page, self.head_dim, self._dev = pages, heads, page, head_dim, dev
        self.grid, self.rht, self.rht_seed = int(grid), bool(rht), rht_seed
        self._c = ctypes.byref(CacheC(k_codes.data_ptr(), k_scales.data_ptr(), k_row_scale.data_ptr(),
                                      v_codes.data_ptr(), v_scales.data_ptr(), v_row_scale.data_ptr(), pages, heads,
                                      page, head_dim, self.grid, 1 if rht else 0, 0, rht_seed))

    @staticmethod
    def _pad(head_dim):
        return 64 if head_dim <= 64 else 128 if head_dim <= 128 else 256

    @classmethod
    def empty(cls, pages, heads, page, head_dim, grid, rht=False, rht_seed=0, device="cuda"):
        device, pad = _device(device), cls._pad(head_dim)
        new = lambda *tail, dtype=torch.uint8: torch.empty((pages, heads, page) + tail, dtype=dtype,  # noqa: E731
                                                           device=device)
        return cls(new(pad // 2), new(pad // 16), new(dtype=_FLOAT32), new(pad // 2), new(pad // 16),
                   new(dtype=_FLOAT32), head_dim, grid, rht, rht_seed)

    @property
    def device(self):
        return torch.device("cuda", self._dev)

    def c(self):
        return self._c


def _heads3d(t, name, dev, heads, dim, tokens=None):
    """Checks a [tokens, heads, dim] tensor with unit stride in its last dim;
    its pointer, dtype code, token stride, head stride and tokens."""
    if not isinstance(t, torch.Tensor):
        _on_gpu(t, name)
    if t.get_device() != dev:
        _same_place(t.get_device(), dev, name)
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or (tokens is not None and shape[0] != tokens):
        raise ValueError("%s must be [%s, %d, %d], got %s" % (name, "tokens" if tokens is None else tokens, heads, dim,
                                                              tuple(shape)))
    ld, head, unit = t.stride()
    if unit != 1:
        raise ValueError("%s must have unit stride in its last dim" % name)
    if shape[0] <= 1 and ld < dim:   # (the stride of a single one says nothing)
        ld = dim
    if heads == 1 and head < dim:
        head = dim
    dt = _DTYPES.get(t.dtype)
    return t.data_ptr(), _dtype_code(t) if dt is None else dt, ld, head, shape[0]


def _slots(slots, dev, tokens=None):
    if slots.get_device() != dev:
        _same_place(slots.get_device(), dev, "slots")
    if slots.dtype is not _INT64 or slots.dim() != 1 or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous int64 vector")
    if tokens is not None and slots.numel() != tokens:
        raise ValueError("slots must have one place for each of the %d tokens" % tokens)
    return slots.data_ptr()


def ufp4_cache_append(k, v, slots, cache, stream=None):
    """Quantizes k and v ([tokens, heads, head_dim], bf16 or fp32) into the
    cache at places slots ([tokens] int64, page number * page + offset, all
    different); places outside the cache (-1) are skipped."""
    dev = _place(k, "k")
    cc, (s, _) = _struct(cache, dev, "cache"), _streams(stream, dev)
    kp, dt, kld, kh, tokens = _heads3d(k, "k", dev, cache.heads, cache.head_dim)
    vp, vdt, vld, vh, _ = _heads3d(v, "v", dev, cache.heads, cache.head_dim, tokens)
    if vdt != dt:
        raise TypeError("k and v must have one dtype")
    st = lib().ufp4_cache_append(kp, vp, dt, tokens, kld, kh, vld, vh, _slots(slots, dev, tokens), cc, s)
    _check(st, "ufp4_cache_append")


def ufp4_cache_load(cache, slots, dtype=None, k=None, v=None, stream=None):
    """The keys and values at places slots, as (k, v), each [tokens, heads,
    head_dim] of `dtype` (bf16 by default); zeros for places outside the cache.
    k, v: tensors to write, both or none."""
    dev = _place(slots, "slots")
    cc, (s, on) = _struct(cache, dev, "cache"), _streams(stream, dev)
    sp, shape = _slots(slots, dev), (slots.numel(), cache.heads, cache.head_dim)
    if (k is None) != (v is None):
        raise ValueError("give both k and v, or neither")
    if k is None:
        dtype = dtype or torch.bfloat16
        if dtype not in _DTYPES:
            raise TypeError("k and v must be bf16 or fp32, got %s" % dtype)
        k, v = _empty(shape, dtype, dev, on), _empty(shape, dtype, dev, on)
        kp, vp, dt, kh = k.data_ptr(), v.data_ptr(), _DTYPES[dtype], shape[2]
        kld = vld = shape[1] * kh
        vh = kh
    elif k.dtype is not v.dtype or (dtype is not None and k.dtype is not dtype):
        raise TypeError("k and v must be %s" % (dtype or "of one dtype"))
    else:
        kp, dt, kld, kh, _ = _heads3d(k, "k", dev, cache.heads, cache.head_dim, shape[0])
        vp, _, vld, vh, _ = _heads3d(v, "v", dev, cache.heads, cache.head_dim, shape[0])
    st = lib().ufp4_cache_load(cc, sp, shape[0], kp, vp, dt, kld, kh, vld, vh, s)
    _check(st, "ufp4_cache_load")
    return k, v


_attn_needs = {}     # scratch bytes by a call's sizes (and the device, by whose SMs the work is split)


def ufp4_cache_attn(q, cache, table, lens, mask=None, scale=None, dtype=None, out=None, lse=None, ws=None,
                    stream=None):
    """Attention of each sequence's last m tokens over its rows of the cache.
    q: [batch * m, heads, head_dim]; table: int32 [batch, width], the pages of
    each sequence; lens: int32 [batch], the m new tokens included; mask: int64
    [batch, m], bit r of a token's word set where it sees new token r (None:
    those up to itself); scale: 1 / sqrt(head_dim) by default.  lse: True or an
    fp32 [batch * m, heads] to write for the logarithms of the softmax's sums.
    ws: scratch of ufp4_cache_attn_workspace_bytes(...), contiguous and 16-byte
    aligned (a new one by default).
    Returns out [batch * m, heads, head_dim] of `dtype` (q's by default), or
    (out, lse)."""
    dev = _place(q, "q")
    cc, (s, on) = _struct(cache, dev, "cache"), _streams(stream, dev)
    shape, span = q.shape, table.shape
    if len(shape) != 3:
        raise ValueError("q must be [batch * m, heads, head_dim]")
    tokens, heads, dim = shape
    if table.get_device() != dev:
        _same_place(table.get_device(), dev, "table")
    if lens.get_device() != dev:
        _same_place(lens.get_device(), dev, "lens")
    if table.dtype is not _INT32 or lens.dtype is not _INT32:
        raise TypeError("table and lens must be int32, got %s and %s" % (table.dtype, lens.dtype))
    batch = lens.numel()
    if lens.dim() != 1 or not lens.is_contiguous():
        raise ValueError("lens must be a contiguous vector")
    if len(span) != 2 or span[0] != batch or (span[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be [batch, width] with unit stride in its last dim")
    width = span[1]
    if tokens % batch if batch else tokens:
        raise ValueError("q must have the same number of tokens for each of the %d sequences" % batch)
    m = tokens // batch if batch else 1
    qp, dt, qld, qh, _ = _heads3d(q, "q", dev, heads, cache.head_dim)
    mp = None
    if mask is not None:
        if mask.get_device() != dev:
            _same_place(mask.get_device(), dev, "mask")
        if mask.dtype is not _INT64 or mask.shape != (batch, m) or not mask.is_contiguous():
            raise ValueError("mask must be contiguous int64 [%d, %d]" % (batch, m))
        mp = mask.data_ptr()
    if out is None:
        dtype = dtype or q.dtype
        if dtype not in _DTYPES:
            raise TypeError("out must be bf16 or fp32, got %s" % dtype)
        out = _empty((tokens, heads, dim), dtype, dev, on)
        op, odt, old, oh = out.data_ptr(), _DTYPES[dtype], heads * dim, dim
    elif dtype is not None and out.dtype is not dtype:
        raise TypeError("out must be %s, got %s" % (dtype, out.dtype))
    else:
        op, odt, old, oh, _ = _heads3d(out, "out", dev, heads, dim, tokens)
    lp, want = None, lse is not None and lse is not False
    if want:
        if lse is True:
            lse = _empty((tokens, heads), _FLOAT32, dev, on)
        elif lse.get_device() != dev:
            _same_place(lse.get_device(), dev, "lse")
        if lse.dtype is not _FLOAT32 or lse.shape != (tokens, heads) or not lse.is_contiguous():
            raise ValueError("lse must be contiguous fp32 [%d, %d]" % (tokens, heads))
        lp = lse.data_ptr()
    L, sizes = lib(), None
    if ws is None:
        sizes = (dev, batch, m, heads, width, cache.heads, cache.page, dim)
        need = _attn_needs.get(sizes)
        if need is None:
            need = L.ufp4_cache_attn_workspace_bytes(batch, m, heads, width, cc)
        else:
            sizes = None
        ws = _empty((need,), torch.uint8, dev, on) if need else None
    elif ws.get_device() != dev:
        _same_place(ws.get_device(), dev, "ws")
    elif not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    st = L.ufp4_cache_attn(qp, dt, qld, qh, batch, m, heads, cc, table.data_ptr(),
                           table.stride(0) if batch > 1 else max(width, 1), width, lens.data_ptr(), mp,
                           dim ** -0.5 if scale is None else scale, op, odt, old, oh, lp,
                           None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel() * ws.element_size(),
                           s)
    _check(st, "ufp4_cache_attn")
    if sizes is not None:                # (of a cache that is refused the library says 0)
        if len(_attn_needs) >= 4096:
            _attn_needs.clear()
        _attn_needs[sizes] = need
    return (out, lse) if want else out
