"""Python binding of the C ABI of libbsg.so: the block-scaled GEMM (include/bsg.h), the paged NVFP4
key/value cache with its attention (include/bsg_kv.h) and the mixture-of-experts layer for few tokens
(include/bsg_moe.h).

Argument marshalling only: every step runs in the HIP library.  Tensors are passed as
device pointers (anything with .data_ptr(), or a plain int); streams as hipStream_t handles (an
object with .cuda_stream, an int, or None for torch's current stream).  PyTorch is used to find the
current stream, when present, and to know the types of the tensors that KVPlan and MoEPlan are given.

The library is loaded on first use and a missing build raises LibraryNotBuilt: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

__all__ = ["Plan", "BsgError", "LibraryNotBuilt", "load_library", "bench_loop", "null_loop", "run_noalloc", "NOALLOC_SCRATCH_BYTES", "decode_nvfp4_f16",
           "FORMATS", "OUT_DTYPES", "SCALE_LAYOUTS", "abi_version", "packed_strides", "Problem", "PROBLEM_V1_SIZE", "PROBLEM_V2_SIZE",
           "pack_scales", "scales_ktile_bytes",
           "KVPlan", "KVBatch", "kv_page_bytes", "rope_table", "MoEPlan"]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbsg.so")

FORMATS = {"mxfp8": 1, "nvfp4": 2}
OUT_DTYPES = {"bf16": 1, "f16": 2}
EPI_BIAS, EPI_SILU, SCALES_KTILE = 1, 2, 4
SCALE_LAYOUTS = ("linear", "ktile")  # row-major [rows][K/block], or K-tile-major (BSG_SCALES_KTILE)
SCALE_BLOCK = {"mxfp8": 32, "nvfp4": 16}

STATUS = {0: "BSG_OK", 1: "BSG_ERR_NULL", 2: "BSG_ERR_SHAPE", 3: "BSG_ERR_UNSUPPORTED", 4: "BSG_ERR_ALIGN",
          5: "BSG_ERR_DEVICE", 6: "BSG_ERR_HIP", 7: "BSG_ERR_ALLOC", 8: "BSG_ERR_ABI"}


class LibraryNotBuilt(RuntimeError):
    pass


class BsgError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        self.status_name = STATUS.get(status, f"status {status}")
        super().__init__(f"{self.status_name}: {message}")


class Problem(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("format", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("device", ctypes.c_int32), ("batch", ctypes.c_int32), ("stride_a", ctypes.c_int64),
                ("stride_b", ctypes.c_int64), ("stride_sa", ctypes.c_int64), ("stride_sb", ctypes.c_int64),
                ("stride_bias", ctypes.c_int64), ("stride_d", ctypes.c_int64),
                ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64), ("ldd", ctypes.c_int64)]


PROBLEM_V1_SIZE = 48  # sizeof(bsg_problem) of ABI 1, still accepted by bsg_plan_create
PROBLEM_V2_SIZE = 96  # ... and of ABI 2 (no leading dimensions)


def scales_ktile_bytes(rows: int, codes_per_row: int) -> int:
    """Bytes of one operand's scales in the K-tile-major layout: ceil(codes / 4) * rows * 4."""
    return 0 if rows < 1 or codes_per_row < 1 else (codes_per_row + 3) // 4 * rows * 4


def packed_strides(fmt: str, M: int, N: int, K: int, scale_layout: str = "linear", lda: int = 0, ldb: int = 0,
                   ldd: int = 0) -> dict:
    """Byte strides of back-to-back batched operands (bias shared by every problem): each problem's
    A, B and D take rows x leading dimension (0 = packed: K, K, N)."""
    elem, blk = (1.0, 32) if fmt == "mxfp8" else (0.5, 16)
    lda, ldb, ldd = lda or K, ldb or K, ldd or N
    if scale_layout == "ktile":
        sa, sb = scales_ktile_bytes(M, K // blk), scales_ktile_bytes(N, K // blk)
    else:
        sa, sb = M * K // blk, N * K // blk
    return dict(a=int(M * lda * elem), b=int(N * ldb * elem), sa=sa, sb=sb, bias=0, d=2 * M * ldd)


_HEADS = struct.Struct("@Pqq").pack  # bsg_heads: pointer, token stride, head stride


class KVProblem(ctypes.Structure):  # bsg_kv_problem
    _fields_ = [("struct_size", ctypes.c_uint32), ("dtype", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("max_tokens", ctypes.c_int64),
                ("flags", ctypes.c_uint32), ("rope_dim", ctypes.c_int32), ("window", ctypes.c_int32),
                ("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float), ("device", ctypes.c_int32)]


class KVBatchArgs(ctypes.Structure):  # bsg_kv_batch
    _fields_ = [("struct_size", ctypes.c_uint32), ("num_seqs", ctypes.c_int32), ("num_tokens", ctypes.c_int64),
                ("max_q", ctypes.c_int32), ("max_kv", ctypes.c_int32), ("q_start", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("pages", ctypes.c_void_p), ("pages_stride", ctypes.c_int64)]


class KVPlanInfo(ctypes.Structure):  # bsg_kv_plan_info
    _fields_ = [("struct_size", ctypes.c_uint32), ("reserved", ctypes.c_int32), ("page_bytes", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("workspace_bytes", ctypes.c_uint64)]


class MoEProblem(ctypes.Structure):  # bsg_moe_problem
    _fields_ = [("struct_size", ctypes.c_uint32), ("format", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("hidden", ctypes.c_int64), ("inter", ctypes.c_int64), ("max_tokens", ctypes.c_int64),
                ("device", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MoEWeights(ctypes.Structure):  # bsg_moe_weights
    _fields_ = [("struct_size", ctypes.c_uint32), ("reserved", ctypes.c_uint32), ("router", ctypes.c_void_p),
                ("w13", ctypes.c_void_p), ("s13", ctypes.c_void_p), ("w2", ctypes.c_void_p), ("s2", ctypes.c_void_p),
                ("alpha13", ctypes.c_void_p), ("alpha2", ctypes.c_void_p)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("variant", ctypes.c_char * 64), ("tile_m", ctypes.c_int32),
                ("tile_n", ctypes.c_int32), ("tile_k", ctypes.c_int32), ("grid_x", ctypes.c_uint32),
                ("grid_y", ctypes.c_uint32), ("grid_z", ctypes.c_uint32), ("block_x", ctypes.c_uint32),
                ("lds_bytes", ctypes.c_uint32), ("workspace_bytes", ctypes.c_uint64)]


_lib = None

_VP = ctypes.c_void_p
_SIGNATURES = {
    "bsg_plan_create": (ctypes.c_int, [ctypes.POINTER(Problem), ctypes.POINTER(_VP)]),
    "bsg_run": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_float, _VP, _VP]),
    "bsg_run_alpha_ptr": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "bsg_plan_destroy": (ctypes.c_int, [_VP]),
    "bsg_plan_query": (ctypes.c_int, [_VP, ctypes.POINTER(PlanInfo)]),
    "bsg_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "bsg_last_error": (ctypes.c_char_p, []),
    "bsg_abi_version": (ctypes.c_int, []),
    "bsg_test_decode_nvfp4_f16": (ctypes.c_int, [_VP, _VP, _VP, ctypes.c_int64, _VP]),
    "bsg_pack_scales": (ctypes.c_int, [_VP, _VP, ctypes.c_int64, ctypes.c_int64, _VP]),
    "bsg_scales_ktile_bytes": (ctypes.c_int64, [ctypes.c_int64, ctypes.c_int64]),
    "bsg_bench_loop": (ctypes.c_int, [_VP, ctypes.c_int, ctypes.POINTER(_VP), ctypes.POINTER(_VP),
                                      ctypes.POINTER(_VP), ctypes.POINTER(_VP), ctypes.POINTER(_VP),
                                      ctypes.POINTER(ctypes.c_float), ctypes.POINTER(_VP), ctypes.c_int,
                                      ctypes.c_int, _VP, ctypes.POINTER(ctypes.c_double),
                                      ctypes.POINTER(ctypes.c_double)]),
    "bsg_run_noalloc": (ctypes.c_int, [ctypes.POINTER(Problem), _VP, _VP, _VP, _VP, _VP, ctypes.c_float, _VP, _VP]),
    "bsg_kv_plan_create": (ctypes.c_int, [ctypes.POINTER(KVProblem), ctypes.POINTER(_VP)]),
    "bsg_kv_plan_destroy": (ctypes.c_int, [_VP]),
    "bsg_kv_plan_query": (ctypes.c_int, [_VP, ctypes.POINTER(KVPlanInfo)]),
    "bsg_kv_page_bytes": (ctypes.c_int64, [ctypes.c_int32] * 3),
    "bsg_kv_append": (ctypes.c_int, [_VP] * 7 + [ctypes.c_int64, _VP, _VP]),
    "bsg_kv_attend": (ctypes.c_int, [_VP] * 7),
    "bsg_kv_read": (ctypes.c_int, [_VP] * 6),
    "bsg_moe_plan_create": (ctypes.c_int, [ctypes.POINTER(MoEProblem), ctypes.POINTER(_VP)]),
    "bsg_moe_plan_destroy": (ctypes.c_int, [_VP]),
    "bsg_moe_run": (ctypes.c_int, [_VP, ctypes.c_int64, _VP, ctypes.c_int64, _VP, _VP, ctypes.c_int64, _VP, _VP, _VP]),
    "bsg_bench_null_loop": (ctypes.c_int, [ctypes.c_int, _VP, ctypes.POINTER(ctypes.c_double),
                                           ctypes.POINTER(ctypes.c_double)]),
}


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libbsg.so (once).  Raises LibraryNotBuilt if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise LibraryNotBuilt(f"{path} is missing: build it with `python -m block_scaled_precision_gemm_amd.build` "
                              "(or __graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def abi_version() -> int:
    return load_library().bsg_abi_version()


def _check(status: int) -> None:
    if status != 0:
        raise BsgError(status, load_library().bsg_last_error().decode(errors="replace"))


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_current_stream = None  # returns torch's current stream as a handle, once a GPU was seen through torch


def _find_current_stream():
    """How to ask torch for its current stream; None without torch or a GPU."""
    try:
        import torch
    except ImportError:
        return None
    if not torch.cuda.is_available():
        return None
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw and device:
        torch.cuda.current_stream()  # torch's own start-up
        return lambda: raw(device())
    return lambda: torch.cuda.current_stream().cuda_stream


def _stream(s) -> int | None:
    global _current_stream
    if s is None:
        if _current_stream is None:
            _current_stream = _find_current_stream()
        return _current_stream() if _current_stream else None
    if isinstance(s, int):
        return s
    return s.cuda_stream


class Plan:
    """A cached GEMM plan: D = epi(alpha * A x B^T (+ bias)) for one problem shape and variant.

    batch > 1: that many problems of this shape per call; problem z uses each pointer advanced by
    strides[key] * z bytes (keys a, b, sa, sb, bias, d; default: back-to-back operands, shared bias).
    scale_layout "ktile": sA and sB in the K-tile-major layout (pack_scales converts).
    lda, ldb, ldd: leading dimensions in elements (row pitch of A, B and D; 0 = packed).
    """

    def __init__(self, fmt: str, M: int, N: int, K: int, out: str = "bf16", bias: bool = False,
                 silu: bool = False, device: int = -1, batch: int = 1, strides: dict | None = None,
                 scale_layout: str = "linear", lda: int = 0, ldb: int = 0, ldd: int = 0):
        if scale_layout not in SCALE_LAYOUTS:
            raise ValueError(f"scale_layout must be one of {SCALE_LAYOUTS}")
        lib = load_library()
        self._lib = lib
        self._h = None
        self.fmt, self.M, self.N, self.K, self.out, self.bias, self.silu = fmt, M, N, K, out, bias, silu
        self.batch, self.scale_layout = batch, scale_layout
        st = packed_strides(fmt, M, N, K, scale_layout, lda, ldb, ldd)
        st.update(strides or {})
        self.strides = st
        self.lda, self.ldb, self.ldd = lda or K, ldb or K, ldd or N
        prob = Problem(ctypes.sizeof(Problem), FORMATS[fmt], OUT_DTYPES[out],
                       (EPI_BIAS if bias else 0) | (EPI_SILU if silu else 0)
                       | (SCALES_KTILE if scale_layout == "ktile" else 0), M, N, K, device, batch,
                       st["a"], st["b"], st["sa"], st["sb"], st["bias"], st["d"], lda, ldb, ldd)
        h = _VP()
        _check(lib.bsg_plan_create(ctypes.byref(prob), ctypes.byref(h)))
        self._h = h

    @property
    def handle(self) -> int:
        return self._h.value

    def run(self, A, B, sA, sB, D, alpha: float = 1.0, bias=None, stream=None) -> None:
        _check(self._lib.bsg_run(self._h, _ptr(A), _ptr(B), _ptr(sA), _ptr(sB), _ptr(bias), float(alpha), _ptr(D),
                                 _stream(stream)))

    def run_alpha_ptr(self, A, B, sA, sB, D, alpha_dev, bias=None, stream=None) -> None:
        _check(self._lib.bsg_run_alpha_ptr(self._h, _ptr(A), _ptr(B), _ptr(sA), _ptr(sB), _ptr(bias),
                                           _ptr(alpha_dev), _ptr(D), _stream(stream)))

    def info(self) -> dict:
        inf = PlanInfo()
        inf.struct_size = ctypes.sizeof(PlanInfo)
        _check(self._lib.bsg_plan_query(self._h, ctypes.byref(inf)))
        return dict(variant=inf.variant.decode(), tile=(inf.tile_m, inf.tile_n, inf.tile_k),
                    grid=(inf.grid_x, inf.grid_y, inf.grid_z), block=inf.block_x, lds_bytes=inf.lds_bytes,
                    workspace_bytes=inf.workspace_bytes)

    def close(self) -> None:
        if self._h is not None and self._h.value:
            _check(self._lib.bsg_plan_destroy(self._h))
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


NOALLOC_SCRATCH_BYTES = 32 << 20  # BSG_NOALLOC_SCRATCH_BYTES


def run_noalloc(fmt: str, M: int, N: int, K: int, A, B, sA, sB, D, alpha: float = 1.0, bias=None, out: str = "bf16",
                silu: bool = False, device: int = -1, stream=None) -> None:
    """One GEMM call through bsg_run_noalloc (no allocation; split-K partials in the library's static
    device scratch).  Packed, single-problem, row-major scales."""
    prob = Problem(ctypes.sizeof(Problem), FORMATS[fmt], OUT_DTYPES[out],
                   (EPI_BIAS if bias is not None else 0) | (EPI_SILU if silu else 0), M, N, K, device, 1,
                   0, 0, 0, 0, 0, 0, 0, 0, 0)
    _check(load_library().bsg_run_noalloc(ctypes.byref(prob), _ptr(A), _ptr(B), _ptr(sA), _ptr(sB), _ptr(bias),
                                          float(alpha), _ptr(D), _stream(stream)))


def bench_loop(plan: Plan, sets: list[dict], calls_per_set: int, mode: int, stream, with_submit: bool = False):
    """Native loop of len(sets) * calls_per_set bsg_run calls; returns the host wall time in us
    (with_submit: the pair (wall, enqueue-only time) in us).

    Each set is a dict with A, B, sA, sB, D, alpha and optional bias.  mode 0 = direct calls,
    mode 1 = one HIP graph per set (captured outside the timed region) replayed.
    """
    lib = load_library()
    n = len(sets)
    arr = lambda key: (_VP * n)(*[_ptr(s.get(key)) for s in sets])  # noqa: E731
    alphas = (ctypes.c_float * n)(*[float(s["alpha"]) for s in sets])
    has_bias = any(s.get("bias") is not None for s in sets)
    wall, submit = ctypes.c_double(), ctypes.c_double()
    _check(lib.bsg_bench_loop(plan._h, n, arr("A"), arr("B"), arr("sA"), arr("sB"), arr("bias") if has_bias else None,
                              alphas, arr("D"), calls_per_set, mode, _stream(stream), ctypes.byref(wall),
                              ctypes.byref(submit)))
    return (wall.value, submit.value) if with_submit else wall.value


def null_loop(n: int, stream) -> tuple[float, float]:
    """n back-to-back launches of an empty kernel from C++: (wall us, enqueue-only us)."""
    wall, submit = ctypes.c_double(), ctypes.c_double()
    _check(load_library().bsg_bench_null_loop(n, _stream(stream), ctypes.byref(wall), ctypes.byref(submit)))
    return wall.value, submit.value


def decode_nvfp4_f16(packed, scale_codes, out_f16, n_elements: int, stream=None) -> None:
    """out_f16[k] = device fp16 dequantisation of NVFP4 element k times 2^-8, through the GEMM
    kernels' routine (packed[k/2] nibble, scale_codes[k/16]); n_elements a multiple of 32."""
    _check(load_library().bsg_test_decode_nvfp4_f16(_ptr(packed), _ptr(scale_codes), _ptr(out_f16), n_elements,
                                                    _stream(stream)))


def pack_scales(src, dst, rows: int, codes_per_row: int, stream=None) -> None:
    """dst (scales_ktile_bytes(rows, codes_per_row) bytes, device) = the K-tile-major layout of the
    row-major scale codes src [rows][codes_per_row] (device); enqueued on `stream`."""
    _check(load_library().bsg_pack_scales(_ptr(src), _ptr(dst), rows, codes_per_row, _stream(stream)))


def _dtypes(name: str) -> tuple:
    """Types of tensors that hold 16-bit numbers of the named type: its own, or integers with their bits."""
    import torch
    return ({"bf16": torch.bfloat16, "f16": torch.float16}[name], torch.int16, torch.uint16)


def _f32_i32() -> tuple:
    import torch
    return torch.float32, torch.int32


KV_ROPE_INTERLEAVED, KV_NONCAUSAL = 1, 2
ROPE_LAYOUTS = ("half", "interleaved")


def kv_page_bytes(kv_heads: int, head_dim: int, page_tokens: int) -> int:
    """Bytes of one packed page of a paged NVFP4 cache (0 for a geometry without kernels)."""
    return load_library().bsg_kv_page_bytes(kv_heads, head_dim, page_tokens)


class KVBatch:
    """The new tokens of a call and where their sequences' positions live (bsg_kv_batch).

    q_start [seqs + 1], kv_len [seqs] and pages [seqs][entries]: int32 device tensors (kept alive here);
    num_tokens = q_start[-1]; max_q and max_kv bound every sequence's new tokens and context.
    """

    def __init__(self, q_start, kv_len, pages, num_tokens: int, max_q: int, max_kv: int):
        seqs = kv_len.shape[0]
        if q_start.shape[0] != seqs + 1 or pages.dim() != 2 or pages.shape[0] != seqs:
            raise ValueError("q_start needs one entry more than kv_len, and pages one row for each of its entries")
        for t in (q_start, kv_len, pages):
            if t.element_size() != 4 or t.is_floating_point() or (t.numel() and t.stride(-1) != 1):
                raise ValueError("q_start, kv_len and pages must be int32 with contiguous rows")
        self.num_tokens, self.max_kv, self.columns, self._held = num_tokens, max_kv, pages.shape[1], (q_start, kv_len, pages)
        stride = pages.stride(0) if seqs > 1 else pages.shape[1]
        self._args = KVBatchArgs(ctypes.sizeof(KVBatchArgs), seqs, num_tokens, max_q, max_kv, q_start.data_ptr(),
                                 kv_len.data_ptr(), pages.data_ptr(), stride)
        self._ref = ctypes.byref(self._args)


class KVPlan:
    """A plan of the paged NVFP4 cache and its attention for one geometry (bsg_kv.h): append, attend, read.

    The cache is a contiguous device tensor of num_pages * page_stride bytes (the last page's padding may be missing);
    page_bytes is what a page holds, page_stride the bytes from one to the next, the same unless page_stride is given.
    q, k, v and outputs: tensors [tokens][heads][head_dim] of `dtype` (or 16-bit integers that hold its bits), any
    token and head strides that are multiples of 8 elements.  window > 0: causal attention to the last `window`
    positions only.
    """

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, page_tokens: int, num_pages: int, max_tokens: int,
                 dtype: str = "bf16", scale: float = 0.0, causal: bool = True, window: int = 0, softcap: float = 0.0,
                 k_scale: float = 1.0, v_scale: float = 1.0, rope_dim: int = 0, rope_layout: str = "half",
                 page_stride: int = 0, device: int = -1):
        if rope_layout not in ROPE_LAYOUTS:
            raise ValueError(f"rope_layout must be one of {ROPE_LAYOUTS}")
        self._h = None
        self._lib = lib = load_library()
        self.q_heads, self.kv_heads, self.head_dim, self.rope_dim = q_heads, kv_heads, head_dim, rope_dim
        prob = KVProblem(ctypes.sizeof(KVProblem), OUT_DTYPES[dtype], q_heads, kv_heads, head_dim, page_tokens, num_pages,
                         page_stride, max_tokens, (KV_ROPE_INTERLEAVED if rope_layout == "interleaved" else 0)
                         | (0 if causal else KV_NONCAUSAL), rope_dim, window, scale, softcap, k_scale, v_scale, device)
        h = _VP()
        _check(lib.bsg_kv_plan_create(ctypes.byref(prob), ctypes.byref(h)))
        self._h = h
        info = self.info()
        self.page_tokens, self.page_bytes, self.page_stride = page_tokens, info["page_bytes"], info["page_stride"]
        self._cache_bytes = (num_pages - 1) * self.page_stride + self.page_bytes
        self._dtypes, (self._f32, _) = _dtypes(dtype), _f32_i32()

    def _heads(self, t, tokens: int, heads: int) -> bytes:
        token_stride, head_stride, one = t.stride() if t.dim() == 3 else (0, 0, 0)
        if one != 1 or t.shape != (tokens, heads, self.head_dim) or t.dtype not in self._dtypes:
            raise ValueError(f"expected a 16-bit tensor [{tokens}][{heads}][{self.head_dim}] of the plan's dtype with "
                             f"contiguous rows, got {t.dtype} {tuple(t.shape)} with strides {t.stride()}")
        return _HEADS(t.data_ptr(), token_stride, head_stride)

    def _cache(self, t) -> int | None:
        if t is None or isinstance(t, int):
            return t
        if t.nbytes < self._cache_bytes or not t.is_contiguous():
            raise ValueError(f"the cache must be contiguous and of {self._cache_bytes} bytes or more")
        return t.data_ptr()

    def _batch(self, batch: KVBatch):
        if batch.columns * self.page_tokens < batch.max_kv and batch.num_tokens:  # (the library sees only the rows' stride)
            raise BsgError(2, f"{batch.columns} pages of {self.page_tokens} positions must cover max_kv = {batch.max_kv}")
        return batch._ref

    def append(self, batch: KVBatch, k, v, cache, q=None, q_out=None, rope=None, stream=None) -> None:
        """Store the batch's keys (rotated) and values; with q, write rotated queries to q_out (q: in place).
        rope: float32 table [rows][2][rope_dim / 2] (rope_table makes one)."""
        n = batch.num_tokens
        if rope is not None and (rope.shape[1:] != (2, self.rope_dim // 2) or rope.dtype != self._f32
                                 or not rope.is_contiguous()):
            raise ValueError(f"rope must be a contiguous float32 tensor [rows][2][{self.rope_dim // 2}]")
        _check(self._lib.bsg_kv_append(
            self._h, self._batch(batch), None if q is None else self._heads(q, n, self.q_heads),
            self._heads(k, n, self.kv_heads), self._heads(v, n, self.kv_heads),
            None if q_out is None else self._heads(q_out, n, self.q_heads), _ptr(rope),
            0 if rope is None else rope.shape[0], self._cache(cache), _stream(stream)))

    def attend(self, batch: KVBatch, q, cache, out, lse=None, stream=None) -> None:
        """out = attention of the batch's queries over the cache; lse: float32 [tokens][q_heads] or None."""
        n = batch.num_tokens
        if lse is not None and (lse.shape != (n, self.q_heads) or lse.dtype != self._f32 or not lse.is_contiguous()):
            raise ValueError(f"lse must be a contiguous float32 tensor [{n}][{self.q_heads}]")
        _check(self._lib.bsg_kv_attend(self._h, self._batch(batch), self._heads(q, n, self.q_heads), self._cache(cache),
                                       self._heads(out, n, self.q_heads), _ptr(lse), _stream(stream)))

    def read(self, batch: KVBatch, cache, k, v, stream=None) -> None:
        """k, v = the values that the cache holds at the positions of the batch's new tokens."""
        n = batch.num_tokens
        _check(self._lib.bsg_kv_read(self._h, self._batch(batch), self._cache(cache), self._heads(k, n, self.kv_heads),
                                     self._heads(v, n, self.kv_heads), _stream(stream)))

    def info(self) -> dict:
        inf = KVPlanInfo()
        inf.struct_size = ctypes.sizeof(KVPlanInfo)
        _check(self._lib.bsg_kv_plan_query(self._h, ctypes.byref(inf)))
        return dict(page_bytes=inf.page_bytes, page_stride=inf.page_stride, workspace_bytes=inf.workspace_bytes)

    def close(self) -> None:
        if self._h is not None and self._h.value:
            _check(self._lib.bsg_kv_plan_destroy(self._h))
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


MOE_KEEP_PROBABILITIES = 1


class MoEPlan:
    """A plan of a mixture-of-experts layer for up to max_tokens (at most 64) tokens (bsg_moe.h).

    fmt: format of the experts' weights; dtype: of x, router and out.  renormalize: the chosen experts' weights
    are divided by their sum.
    """

    def __init__(self, fmt: str, experts: int, top_k: int, hidden: int, inter: int, max_tokens: int, dtype: str = "bf16",
                 renormalize: bool = True, device: int = -1):
        self._h = None
        self._lib = lib = load_library()
        self.fmt, self.experts, self.top_k, self.hidden, self.inter = fmt, experts, top_k, hidden, inter
        prob = MoEProblem(ctypes.sizeof(MoEProblem), FORMATS[fmt], OUT_DTYPES[dtype],
                          0 if renormalize else MOE_KEEP_PROBABILITIES, experts, top_k, hidden, inter, max_tokens, device, 0)
        h = _VP()
        _check(lib.bsg_moe_plan_create(ctypes.byref(prob), ctypes.byref(h)))
        self._h = h
        self._dtypes, (self._f32, self._i32) = _dtypes(dtype), _f32_i32()
        per, rows = 2 if fmt == "nvfp4" else 1, experts * inter * hidden
        self._nr = experts * hidden
        self._n13, self._ns13 = 2 * rows // per, 2 * rows // SCALE_BLOCK[fmt]
        self._n2, self._ns2 = rows // per, rows // SCALE_BLOCK[fmt]

    def run(self, x, router, w13, s13, w2, s2, out, alpha13=None, alpha2=None, ids=None, weights=None, stream=None) -> None:
        """out = the layer applied to x [tokens][hidden] (row-strided views are fine).  w13, s13, w2, s2: uint8 codes
        and row-major scale codes of every expert; alpha13, alpha2: float32 [experts] or None; ids (int32) and weights
        (float32) [tokens][top_k]: the routing, or None."""
        tokens = x.shape[0]
        for t in (x, out):
            if t.shape != (tokens, self.hidden) or t.dtype not in self._dtypes or t.stride(1) != 1:
                raise ValueError(f"expected 16-bit rows [{tokens}][{self.hidden}] of the plan's dtype, got {t.dtype} "
                                 f"{tuple(t.shape)} with strides {t.stride()}")
        choices = tokens * self.top_k
        if not (router.numel() == self._nr and router.dtype in self._dtypes and router.is_contiguous()
                and w13.numel() == self._n13 and w13.element_size() == 1 and w13.is_contiguous()
                and s13.numel() == self._ns13 and s13.element_size() == 1 and s13.is_contiguous()
                and w2.numel() == self._n2 and w2.element_size() == 1 and w2.is_contiguous()
                and s2.numel() == self._ns2 and s2.element_size() == 1 and s2.is_contiguous()):
            raise ValueError(f"router, w13, s13, w2 and s2 must be contiguous, of {self._nr} values of the plan's dtype and {self._n13}, "
                             f"{self._ns13}, {self._n2}, {self._ns2} bytes")
        f32, i32 = self._f32, self._i32
        for t, n, d in ((alpha13, self.experts, f32), (alpha2, self.experts, f32), (ids, choices, i32), (weights, choices, f32)):
            if t is not None and (t.numel() != n or t.dtype != d or not t.is_contiguous()):
                raise ValueError("alpha13 and alpha2 are float32 [experts], ids int32 and weights float32 [tokens][top_k]")
        w = MoEWeights(ctypes.sizeof(MoEWeights), 0, router.data_ptr(), w13.data_ptr(), s13.data_ptr(), w2.data_ptr(),
                       s2.data_ptr(), _ptr(alpha13), _ptr(alpha2))
        _check(self._lib.bsg_moe_run(self._h, tokens, x.data_ptr(), x.stride(0) if tokens > 1 else self.hidden,
                                     ctypes.byref(w), out.data_ptr(), out.stride(0) if tokens > 1 else self.hidden,
                                     _ptr(ids), _ptr(weights), _stream(stream)))

    def close(self) -> None:
        if self._h is not None and self._h.value:
            _check(self._lib.bsg_moe_plan_destroy(self._h))
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


def rope_table(rows: int, rope_dim: int, base: float = 10000.0, scaling: tuple | None = None):
    """The rotation table of positions 0 .. rows - 1: float32 array [rows][2][rope_dim / 2], cosines then sines.

    Pair i turns by position * base^(-2 i / rope_dim).  scaling, for contexts longer than a model was trained on:
      ("linear", f)        positions divided by f;
      ("base", f)          base multiplied by f^(R / (R - 2)): the slowest pair slows down by f, the fastest not at all;
      ("parts", f, n)      pairs that turn more than 32 times in the trained n positions stay, pairs that turn less than
                           once slow down by f, those between go from one to the other linearly in the pair's index;
                           cosines and sines are multiplied by 1 + 0.1 ln f.  The ends of that line are where a pair would
                           turn 32 times and once, not rounded to whole pairs: programs that round them give the pairs in
                           between slightly other speeds, and tables for models trained so are made elsewhere.
    Angles are formed in 64 bits (in 32, position 100000 would be off by 0.004 rad)."""
    import numpy as np

    if rope_dim < 2 or rope_dim % 2 or rows < 1:
        raise ValueError("rope_dim must be even and positive, rows positive")
    half = rope_dim // 2
    kind = scaling[0] if scaling else None
    if kind not in (None, "linear", "base", "parts"):
        raise ValueError('scaling must be None, ("linear", f), ("base", f) or ("parts", f, n)')
    if kind == "base":
        base = base * scaling[1] ** (rope_dim / max(rope_dim - 2, 1))
    freq = base ** (-np.arange(half, dtype=np.float64) / half)
    gain = 1.0
    if kind == "linear":
        freq = freq / scaling[1]
    elif kind == "parts":
        turns = freq * scaling[2] / (2.0 * np.pi)
        first = half * np.log(scaling[2] / (32 * 2.0 * np.pi)) / np.log(base)  # pair that turns 32 times
        last = half * np.log(scaling[2] / (2.0 * np.pi)) / np.log(base)        # pair that turns once
        slow = np.clip((np.arange(half) - first) / max(last - first, 1e-3), 0.0, 1.0)
        freq = np.where(turns >= 32, freq, np.where(turns <= 1, freq / scaling[1], freq * (1 - slow) + freq / scaling[1] * slow))
        gain = 1.0 + 0.1 * np.log(scaling[1])
    angle = np.arange(rows, dtype=np.float64)[:, None] * freq
    return np.stack((np.cos(angle) * gain, np.sin(angle) * gain), 1).astype(np.float32)
