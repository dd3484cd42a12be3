"""ctypes binding of libkvq8attn.so -- argument marshalling only.

Every entry point mirrors the C ABI in include/kvq8attn.h under the same name.  Tensors
are torch CUDA tensors; their data pointers and the current CUDA stream are passed
through unchanged, and every step of the computation runs in the library's kernels.
There is no fallback: a missing library raises, and a nonzero status raises
KVQ8Error with the library's own message.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

_lock = threading.Lock()
_lib = None

KVQ8_OK = 0
KVQ8_ERR_INVALID_ARG = 1
KVQ8_ERR_UNSUPPORTED = 2
KVQ8_ERR_MISALIGNED = 3
KVQ8_ERR_WORKSPACE = 4
KVQ8_ERR_CUDA = 5

# Entry points declared in include/kvq8attn.h.
EXPORTED = ("kvq8_quantize", "kvq8_append", "attn_verify_q8_workspace_bytes", "attn_verify_q8", "attn_verify_tree_q8",
            "attn_verify_append_q8_workspace_bytes", "attn_verify_append_q8", "attn_verify_q8_partials_count",
            "attn_verify_q8_partials", "attn_verify_append_q8_host_scratch_bytes", "attn_verify_append_q8_host",
            "kvf16_append", "attn_verify_f16_workspace_bytes", "attn_verify_f16", "kvk8v4_append", "attn_verify_k8v4",
            "attn_prompt_k8v4", "attn_prompt_f16_workspace_bytes", "attn_prompt_f16", "attn_combine",
            "attn_prompt_q8_workspace_bytes", "attn_prompt_q8", "attn_verify_q8_noalloc", "kvq8_device_error", "kvq8_status_str",
            "argmax_rows_top_prob_workspace_bytes", "argmax_rows_top_prob", "kvq8_selftest_convert",
            "kvq8_selftest_wait_timeout", "kvq8_paged_tables", "kvq8_paged_append", "kvq8_paged_read",
            "attn_verify_paged_q8_workspace_bytes", "attn_verify_paged_q8", "logits_adjust", "token_counts")
NOALLOC_SCRATCH_BYTES = 8 * 1024 * 1024


class KVQ8Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed with status {status}: {kvq8_status_str(status)}")


class kvf16_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("capacity", ctypes.c_int32)]


class kvk8v4_cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("capacity", ctypes.c_int32)]


class kvq8_cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("capacity", ctypes.c_int32)]


class kvq8_paged_cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", ctypes.c_int32)]


def library_path() -> str:
    return _build.LIB_PATH


def load_library():
    """Load the in-tree library (built by ``build.build()``); raises if it is missing."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(path)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        cp = ctypes.POINTER(kvq8_cache)
        lib.kvq8_quantize.argtypes = [vp, i32, i32, i32, vp, vp, i32, i32, vp]
        lib.kvq8_quantize.restype = i32
        lib.kvq8_append.argtypes = [vp, vp, i32, cp, i32, vp]
        lib.kvq8_append.restype = i32
        lib.attn_verify_q8_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.attn_verify_q8_workspace_bytes.restype = sz
        lib.attn_verify_q8.argtypes = [vp, i32, i32, cp, i32, i32, f32, vp, vp, sz, i32, vp]
        lib.attn_verify_q8.restype = i32
        lib.attn_verify_tree_q8.argtypes = [vp, i32, i32, cp, i32, i32, vp, f32, vp, vp, sz, i32, vp]
        lib.attn_verify_tree_q8.restype = i32
        lib.attn_verify_q8_partials_count.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.attn_verify_q8_partials_count.restype = i32
        lib.attn_verify_q8_partials.argtypes = [vp, i32, i32, cp, i32, i32, f32, vp, vp, i32, vp]
        lib.attn_verify_q8_partials.restype = i32
        lib.attn_verify_append_q8_host_scratch_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.attn_verify_append_q8_host_scratch_bytes.restype = sz
        lib.attn_verify_append_q8_host.argtypes = [vp, i32, i32, cp, i32, f32, vp, vp, sz, i32, vp]
        lib.attn_verify_append_q8_host.restype = i32
        c44 = ctypes.POINTER(kvk8v4_cache)
        lib.kvk8v4_append.argtypes = [vp, vp, i32, c44, i32, vp]
        lib.kvk8v4_append.restype = i32
        lib.attn_verify_k8v4.argtypes = [vp, i32, i32, c44, i32, i32, f32, vp, vp, sz, i32, vp]
        lib.attn_verify_k8v4.restype = i32
        lib.attn_prompt_k8v4.argtypes = [vp, i32, i32, c44, i32, i32, f32, vp, vp, sz, vp]
        lib.attn_prompt_k8v4.restype = i32
        cf = ctypes.POINTER(kvf16_cache)
        lib.kvf16_append.argtypes = [vp, vp, i32, cf, i32, vp]
        lib.kvf16_append.restype = i32
        lib.attn_verify_f16_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.attn_verify_f16_workspace_bytes.restype = sz
        lib.attn_verify_f16.argtypes = [vp, i32, i32, cf, i32, i32, f32, vp, vp, sz, i32, vp]
        lib.attn_verify_f16.restype = i32
        lib.attn_prompt_f16.argtypes = [vp, i32, i32, cf, i32, i32, f32, vp, vp, sz, vp]
        lib.attn_prompt_f16.restype = i32
        lib.attn_verify_append_q8_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.attn_verify_append_q8_workspace_bytes.restype = sz
        lib.attn_verify_append_q8.argtypes = [vp, vp, vp, i32, i32, cp, i32, f32, vp, vp, sz, i32, vp]
        lib.attn_verify_append_q8.restype = i32
        lib.argmax_rows_top_prob_workspace_bytes.argtypes = [i32, i32]
        lib.argmax_rows_top_prob_workspace_bytes.restype = sz
        lib.argmax_rows_top_prob.argtypes = [vp, i32, i32, vp, vp, vp, sz, vp]
        lib.argmax_rows_top_prob.restype = i32
        lib.kvq8_selftest_convert.argtypes = [i32, vp, vp, i32, vp]
        lib.kvq8_selftest_convert.restype = i32
        lib.kvq8_selftest_wait_timeout.argtypes = [i32, vp]
        lib.kvq8_selftest_wait_timeout.restype = i32
        lib.attn_combine.argtypes = [vp, vp, i32, i32, i32, vp, vp]
        lib.attn_combine.restype = i32
        lib.attn_prompt_q8_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.attn_prompt_q8_workspace_bytes.restype = sz
        lib.attn_prompt_f16_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.attn_prompt_f16_workspace_bytes.restype = sz
        lib.attn_prompt_q8.argtypes = [vp, i32, i32, cp, i32, i32, f32, vp, vp, sz, vp]
        lib.attn_prompt_q8.restype = i32
        lib.attn_verify_q8_noalloc.argtypes = [vp, i32, i32, cp, i32, i32, f32, vp, i32, vp]
        lib.attn_verify_q8_noalloc.restype = i32
        cpg, i64 = ctypes.POINTER(kvq8_paged_cache), ctypes.c_int64
        lib.kvq8_paged_tables.argtypes = [vp, vp, vp, i32, i32, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp, i32, vp, vp]
        lib.kvq8_paged_tables.restype = i32
        lib.kvq8_paged_append.argtypes = [vp, vp, i32, i32, i64, i64, cpg, vp, vp]
        lib.kvq8_paged_append.restype = i32
        lib.kvq8_paged_read.argtypes = [cpg, vp, i32, i32, vp, vp, ctypes.POINTER(i64), ctypes.POINTER(i64), vp]
        lib.kvq8_paged_read.restype = i32
        lib.attn_verify_paged_q8_workspace_bytes.argtypes = [i32, i32, i32, i32]
        lib.attn_verify_paged_q8_workspace_bytes.restype = sz
        lib.attn_verify_paged_q8.argtypes = [vp, i32, i64, i32, i32, cpg, vp, i32, vp, vp, i32, i32, vp, f32, vp, vp, sz, vp]
        lib.attn_verify_paged_q8.restype = i32
        lib.logits_adjust.argtypes = [vp, i32, i64, i32, i32, vp, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp, i32, vp, i32,
                                      vp, vp, i64, vp]
        lib.logits_adjust.restype = i32
        lib.token_counts.argtypes = [vp, vp, i32, i32, vp, vp, i32, vp, i32, i32, vp]
        lib.token_counts.restype = i32
        lib.kvq8_device_error.argtypes = [i32]
        lib.kvq8_device_error.restype = i32
        lib.kvq8_status_str.argtypes = [i32]
        lib.kvq8_status_str.restype = ctypes.c_char_p
        _lib = lib
        return lib


def kvq8_status_str(status: int) -> str:
    return load_library().kvq8_status_str(int(status)).decode()


def kvq8_device_error(reset: bool = False) -> int:
    """The library's device error flag (nonzero: a kernel timed out on an internal wait).
    Synchronises the current device."""
    return int(load_library().kvq8_device_error(1 if reset else 0))


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream))


def _empty(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """Memory that a call takes for itself or returns, taken on the stream that the call runs on, a raw handle's too: the
    allocator gives it out again in that stream's order, while the current stream may be far ahead or behind."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):  # a handle, or another library's object with one
        handle = int(getattr(stream, "cuda_stream", stream))
        # 1 is another name of the default stream, 0
        stream = torch.cuda.ExternalStream(0 if handle == 1 else handle, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _scratch(nbytes: int, device, stream) -> torch.Tensor:
    return _empty(nbytes, torch.uint8, device, stream)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _check(fn: str, status: int) -> None:
    if status != KVQ8_OK:
        raise KVQ8Error(fn, status)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype) -> None:
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor (got {t.dtype}, {t.device})")


class KVCacheQ8:
    """Caller-owned Q8_0 K/V planes on one device (the layout of include/kvq8attn.h):
    codes int8 [n_kv_heads][capacity][head_dim], scales fp16 [n_kv_heads][capacity][head_dim/32]."""

    def __init__(self, n_kv_heads: int, head_dim: int, capacity: int, device="cuda"):
        self.n_kv_heads, self.head_dim, self.capacity = n_kv_heads, head_dim, capacity
        nb = head_dim // 32
        self.k_codes = torch.zeros((n_kv_heads, capacity, head_dim), dtype=torch.int8, device=device)
        self.v_codes = torch.zeros((n_kv_heads, capacity, head_dim), dtype=torch.int8, device=device)
        self.k_scales = torch.zeros((n_kv_heads, capacity, nb), dtype=torch.float16, device=device)
        self.v_scales = torch.zeros((n_kv_heads, capacity, nb), dtype=torch.float16, device=device)

    @classmethod
    def from_planes(cls, k_codes, k_scales, v_codes, v_scales):
        c = cls.__new__(cls)
        c.n_kv_heads, c.capacity, c.head_dim = k_codes.shape
        c.k_codes, c.k_scales, c.v_codes, c.v_scales = k_codes, k_scales, v_codes, v_scales
        return c

    def struct(self) -> kvq8_cache:
        return kvq8_cache(self.k_codes.data_ptr(), self.k_scales.data_ptr(), self.v_codes.data_ptr(),
                          self.v_scales.data_ptr(), self.n_kv_heads, self.head_dim, self.capacity)

    def append(self, k: torch.Tensor, v: torch.Tensor, pos0: int, stream=None) -> None:
        """Quantise K and V values [n_tok][n_kv_heads][head_dim] (fp32) into positions pos0..
        (one kvq8_append launch for both planes)."""
        kvq8_append(k, v, self, pos0, stream)


class KVCacheK8V4:
    """Caller-owned K8V4 pool on one device (kvk8v4_cache of include/kvq8attn.h): K as Q8_0
    planes, V as 4-bit nibbles v_codes uint8 [n_kv_heads][capacity][head_dim/2] with fp16
    scales v_scales [n_kv_heads][capacity][head_dim/32]."""

    def __init__(self, n_kv_heads: int, head_dim: int, capacity: int, device="cuda"):
        self.n_kv_heads, self.head_dim, self.capacity = n_kv_heads, head_dim, capacity
        nb = head_dim // 32
        self.k_codes = torch.zeros((n_kv_heads, capacity, head_dim), dtype=torch.int8, device=device)
        self.k_scales = torch.zeros((n_kv_heads, capacity, nb), dtype=torch.float16, device=device)
        self.v_codes = torch.full((n_kv_heads, capacity, head_dim // 2), 0x88, dtype=torch.uint8, device=device)
        self.v_scales = torch.zeros((n_kv_heads, capacity, nb), dtype=torch.float16, device=device)

    def struct(self) -> kvk8v4_cache:
        return kvk8v4_cache(self.k_codes.data_ptr(), self.k_scales.data_ptr(), self.v_codes.data_ptr(),
                            self.v_scales.data_ptr(), self.n_kv_heads, self.head_dim, self.capacity)

    def append(self, k: torch.Tensor, v: torch.Tensor, pos0: int, stream=None) -> None:
        """Quantise K (Q8_0) and V (4-bit) values [n_tok][n_kv_heads][head_dim] (fp32) at pos0.."""
        kvk8v4_append(k, v, self, pos0, stream)


def kvk8v4_append(k: torch.Tensor, v: torch.Tensor, cache: KVCacheK8V4, pos0: int, stream=None) -> None:
    _need(k, "k", torch.float32)
    _need(v, "v", torch.float32)
    if k.shape != v.shape or k.dim() != 3 or k.shape[1:] != (cache.n_kv_heads, cache.head_dim):
        raise ValueError(f"k and v must both be [n_tok][{cache.n_kv_heads}][{cache.head_dim}]")
    st = load_library().kvk8v4_append(_ptr(k), _ptr(v), k.shape[0], ctypes.byref(cache.struct()), int(pos0),
                                      _stream(stream))
    _check("kvk8v4_append", st)


def attn_verify_k8v4(q: torch.Tensor, cache: KVCacheK8V4, kv_len: int, q_pos0: int, softmax_scale: float,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, n_split: int = 0,
                     stream=None) -> torch.Tensor:
    """Verify attention of fp32 q [T][Hq][hd] over a K8V4 pool; returns fp32 [T][Hq][hd]."""
    _need(q, "q", torch.float32)
    n_rows, n_q_heads, head_dim = q.shape
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _need(out, "out", torch.float32)
    if workspace is None:
        nbytes = attn_verify_q8_workspace_bytes(n_rows, n_q_heads, head_dim, kv_len, cache.n_kv_heads, n_split)
        workspace = _scratch(max(nbytes, 16), q.device, stream)
    st = load_library().attn_verify_k8v4(_ptr(q), n_rows, n_q_heads, ctypes.byref(cache.struct()), int(kv_len),
                                         int(q_pos0), float(softmax_scale), _ptr(out), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), int(n_split), _stream(stream))
    _check("attn_verify_k8v4", st)
    return out


def attn_prompt_k8v4(q: torch.Tensor, cache: KVCacheK8V4, kv_len: int, q_pos0: int, softmax_scale: float,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Prompt-chunk attention of fp16 q [n_q][Hq][hd] over a K8V4 pool; returns fp32 [n_q][Hq][hd]."""
    _need(q, "q", torch.float16)
    n_q, n_q_heads, head_dim = q.shape
    if out is None:
        out = _empty(q.shape, torch.float32, q.device, stream)
    _need(out, "out", torch.float32)
    if workspace is None:
        nbytes = attn_prompt_q8_workspace_bytes(n_q, n_q_heads, head_dim, kv_len, q_pos0, cache.n_kv_heads)
        workspace = _scratch(max(nbytes, 16), q.device, stream)
    st = load_library().attn_prompt_k8v4(_ptr(q), n_q, n_q_heads, ctypes.byref(cache.struct()), int(kv_len),
                                         int(q_pos0), float(softmax_scale), _ptr(out), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _stream(stream))
    _check("attn_prompt_k8v4", st)
    return out


class KVCacheF16:
    """Caller-owned fp16 KV pool on one device (kvf16_cache of include/kvq8attn.h):
    k, v fp16 [n_kv_heads][capacity][head_dim]."""

    def __init__(self, n_kv_heads: int, head_dim: int, capacity: int, device="cuda"):
        self.n_kv_heads, self.head_dim, self.capacity = n_kv_heads, head_dim, capacity
        self.k = torch.zeros((n_kv_heads, capacity, head_dim), dtype=torch.float16, device=device)
        self.v = torch.zeros((n_kv_heads, capacity, head_dim), dtype=torch.float16, device=device)

    def struct(self) -> kvf16_cache:
        return kvf16_cache(self.k.data_ptr(), self.v.data_ptr(), self.n_kv_heads, self.head_dim, self.capacity)

    def append(self, k: torch.Tensor, v: torch.Tensor, pos0: int, stream=None) -> None:
        """Round K and V values [n_tok][n_kv_heads][head_dim] (fp32) to fp16 at positions pos0.."""
        kvf16_append(k, v, self, pos0, stream)


def kvf16_append(k: torch.Tensor, v: torch.Tensor, cache: KVCacheF16, pos0: int, stream=None) -> None:
    _need(k, "k", torch.float32)
    _need(v, "v", torch.float32)
    if k.shape != v.shape or k.dim() != 3 or k.shape[1:] != (cache.n_kv_heads, cache.head_dim):
        raise ValueError(f"k and v must both be [n_tok][{cache.n_kv_heads}][{cache.head_dim}]")
    st = load_library().kvf16_append(_ptr(k), _ptr(v), k.shape[0], ctypes.byref(cache.struct()), int(pos0),
                                     _stream(stream))
    _check("kvf16_append", st)


def attn_verify_f16_workspace_bytes(n_rows: int, n_q_heads: int, head_dim: int, kv_len: int, n_kv_heads: int,
                                    n_split: int = 0) -> int:
    return int(load_library().attn_verify_f16_workspace_bytes(n_rows, n_q_heads, head_dim, kv_len, n_kv_heads,
                                                              n_split))


def attn_verify_f16(q: torch.Tensor, cache: KVCacheF16, kv_len: int, q_pos0: int, softmax_scale: float,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, n_split: int = 0,
                    stream=None) -> torch.Tensor:
    """Verify attention of fp32 q [T][Hq][hd] over an fp16 pool; returns fp32 [T][Hq][hd]."""
    _need(q, "q", torch.float32)
    n_rows, n_q_heads, head_dim = q.shape
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _need(out, "out", torch.float32)
    if workspace is None:
        nbytes = attn_verify_f16_workspace_bytes(n_rows, n_q_heads, head_dim, kv_len, cache.n_kv_heads, n_split)
        workspace = _scratch(max(nbytes, 16), q.device, stream)
    st = load_library().attn_verify_f16(_ptr(q), n_rows, n_q_heads, ctypes.byref(cache.struct()), int(kv_len),
                                        int(q_pos0), float(softmax_scale), _ptr(out), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), int(n_split), _stream(stream))
    _check("attn_verify_f16", st)
    return out


def attn_prompt_f16(q: torch.Tensor, cache: KVCacheF16, kv_len: int, q_pos0: int, softmax_scale: float,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Prompt-chunk attention of fp16 q [n_q][Hq][hd] over an fp16 pool; returns fp32 [n_q][Hq][hd]."""
    _need(q, "q", torch.float16)
    n_q, n_q_heads, head_dim = q.shape
    if out is None:
        out = _empty(q.shape, torch.float32, q.device, stream)
    _need(out, "out", torch.float32)
    if workspace is None:
        nbytes = attn_prompt_f16_workspace_bytes(n_q, n_q_heads, head_dim, kv_len, q_pos0, cache.n_kv_heads)
        workspace = _scratch(max(nbytes, 16), q.device, stream)
    st = load_library().attn_prompt_f16(_ptr(q), n_q, n_q_heads, ctypes.byref(cache.struct()), int(kv_len),
                                        int(q_pos0), float(softmax_scale), _ptr(out), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(stream))
    _check("attn_prompt_f16", st)
    return out


def kvq8_quantize(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, pos0: int, stream=None) -> None:
    _need(x, "x", torch.float32)
    _need(codes, "codes", torch.int8)
    _need(scales, "scales", torch.float16)
    n_tok, n_kv_heads, head_dim = x.shape
    capacity = codes.shape[1]
    st = load_library().kvq8_quantize(_ptr(x), n_tok, n_kv_heads, head_dim, _ptr(codes), _ptr(scales),
                                      capacity, int(pos0), _stream(stream))
    _check("kvq8_quantize", st)


def kvq8_append(k: torch.Tensor, v: torch.Tensor, cache: "KVCacheQ8", pos0: int, stream=None) -> None:
    """Quantise K and V values [n_tok][n_kv_heads][head_dim] (fp32) into both planes of
    `cache` at positions pos0.. in one launch."""
    _need(k, "k", torch.float32)
    _need(v, "v", torch.float32)
    if k.shape != v.shape or k.dim() != 3 or k.shape[1:] != (cache.n_kv_heads, cache.head_dim):
        raise ValueError(f"k and v must both be [n_tok][{cache.n_kv_heads}][{cache.head_dim}]")
    st = load_library().kvq8_append(_ptr(k), _ptr(v), k.shape[0], ctypes.byref(cache.struct()), int(pos0),
                                    _stream(stream))
    _check("kvq8_append", st)


def attn_verify_q8_workspace_bytes(n_rows: int, n_q_heads: int, head_dim: int, kv_len: int, n_kv_heads: int,
                                   n_split: int = 0) -> int:
    return int(load_library().attn_verify_q8_workspace_bytes(n_rows, n_q_heads, head_dim, kv_len, n_kv_heads,
                                                             n_split))


def attn_verify_q8(q: torch.Tensor, cache: KVCacheQ8, kv_len: int, q_pos0: int, softmax_scale: float,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, n_split: int = 0,
                   stream=None) -> torch.Tensor:
    """Verify attention of fp32 q [T][Hq][hd] over the cache; returns fp32 [T][Hq][hd]."""
    _need(q, "q", torch.float32)
    n_rows, n_q_heads, head_dim = q.shape
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _need(out, "out", torch.float32)
    if workspace is None:
        nbytes = attn_verify_q8_workspace_bytes(n_rows, n_q_heads, head_dim, kv_len, cache.n_kv_heads, n_split)
        workspace = _scratch(max(nbytes, 16), q.device, stream)
    st = load_library().attn_verify_q8(_ptr(q), n_rows, n_q_heads, ctypes.byref(cache.struct()), int(kv_len),
                                       int(q_pos0), float(softmax_scale), _ptr(out), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), int(n_split), _stream(stream))
    _check("attn_verify_q8", st)
    return out


def attn_verify_tree_q8(q: torch.Tensor, cache: KVCacheQ8, kv_len: int, q_pos0: int, window_mask: torch.Tensor,
                        softmax_scale: float, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        n_split: int = 0, stream=None) -> torch.Tensor:
    """Verify attention of a tree-shaped window: fp32 q [T][Hq][hd]; window_mask int32 [T] on
    the device, bit j of row i's word = row i sees key q_pos0 + j (keys before q_pos0 are
    always visible).  Returns fp32 [T][Hq][hd]."""
    _need(q, "q", torch.float32)
    _need(window_mask, "window_mask", torch.int32)
    n_rows, n_q_heads, head_dim = q.shape
    if window_mask.shape != (n_rows,):
        raise ValueError(f"window_mask must hold one word per row ({n_rows})")
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _need(out, "out", torch.float32)
    if workspace is None:
        nbytes = attn_verify_q8_workspace_bytes(n_rows, n_q_heads, head_dim, kv_len, cache.n_kv_heads, n_split)
        workspace = _scratch(max(nbytes, 16), q.device, stream)
    st = load_library().attn_verify_tree_q8(_ptr(q), n_rows, n_q_heads, ctypes.byref(cache.struct()), int(kv_len),
                                            int(q_pos0), _ptr(window_mask), float(softmax_scale), _ptr(out),
                                            _ptr(workspace), workspace.numel() * workspace.element_size(),
                                            int(n_split), _stream(stream))
    _check("attn_verify_tree_q8", st)
    return out


def attn_verify_q8_partials_count(n_rows: int, n_q_heads: int, head_dim: int, kv_len: int, n_kv_heads: int,
                                  n_split: int = 0) -> int:
    return int(load_library().attn_verify_q8_partials_count(n_rows, n_q_heads, head_dim, kv_len, n_kv_heads,
                                                            n_split))


def attn_verify_q8_partials(q: torch.Tensor, cache: KVCacheQ8, kv_len: int, q_pos0: int, softmax_scale: float,
                            n_split: int = 0, part_o: torch.Tensor | None = None,
                            part_ml: torch.Tensor | None = None, stream=None):
    """Per-slice partials of verify attention of fp32 q [T][Hq][hd] over cache positions
    [0, kv_len), row i seeing positions <= q_pos0 + i (q_pos0 may be negative).  Returns
    (part_o fp32 [n][T*Hq][hd], part_ml fp32 [n][T*Hq][2]) in attn_combine's layout."""
    _need(q, "q", torch.float32)
    n_rows, n_q_heads, head_dim = q.shape
    n = attn_verify_q8_partials_count(n_rows, n_q_heads, head_dim, kv_len, cache.n_kv_heads, n_split)
    if n <= 0:
        raise KVQ8Error("attn_verify_q8_partials_count", KVQ8_ERR_INVALID_ARG)
    rows = n_rows * n_q_heads
    if part_o is None:
        part_o = _empty((n, rows, head_dim), torch.float32, q.device, stream)
    if part_ml is None:
        part_ml = _empty((n, rows, 2), torch.float32, q.device, stream)
    _need(part_o, "part_o", torch.float32)
    _need(part_ml, "part_ml", torch.float32)
    if part_o.shape != (n, rows, head_dim) or part_ml.shape != (n, rows, 2):
        raise ValueError(f"part_o / part_ml must be [{n}][{rows}][{head_dim}] / [{n}][{rows}][2]")
    st = load_library().attn_verify_q8_partials(_ptr(q), n_rows, n_q_heads, ctypes.byref(cache.struct()), int(kv_len),
                                                int(q_pos0), float(softmax_scale), _ptr(part_o), _ptr(part_ml),
                                                int(n_split), _stream(stream))
    _check("attn_verify_q8_partials", st)
    return part_o, part_ml


def attn_verify_append_q8_workspace_bytes(n_rows: int, n_q_heads: int, head_dim: int, q_pos0: int,
                                          n_kv_heads: int, n_split: int = 0) -> int:
    return int(load_library().attn_verify_append_q8_workspace_bytes(n_rows, n_q_heads, head_dim, q_pos0,
                                                                    n_kv_heads, n_split))


def attn_verify_append_q8(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, cache: KVCacheQ8, q_pos0: int,
                          softmax_scale: float, out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, n_split: int = 0, stream=None) -> torch.Tensor:
    """Append the window's fp32 keys and values [T][Hkv][hd] to the cache at q_pos0.. and run
    verify attention of fp32 q [T][Hq][hd] over q_pos0 + T keys, in one call; returns fp32
    [T][Hq][hd]."""
    _need(q, "q", torch.float32)
    _need(k_new, "k_new", torch.float32)
    _need(v_new, "v_new", torch.float32)
    n_rows, n_q_heads, head_dim = q.shape
    if k_new.shape != v_new.shape or k_new.shape != (n_rows, cache.n_kv_heads, cache.head_dim):
        raise ValueError(f"k_new and v_new must both be [{n_rows}][{cache.n_kv_heads}][{cache.head_dim}]")
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _need(out, "out", torch.float32)
    if workspace is None:
        nbytes = attn_verify_append_q8_workspace_bytes(n_rows, n_q_heads, head_dim, q_pos0, cache.n_kv_heads,
                                                       n_split)
        workspace = _scratch(max(nbytes, 16), q.device, stream)
    st = load_library().attn_verify_append_q8(_ptr(q), _ptr(k_new), _ptr(v_new), n_rows, n_q_heads,
                                              ctypes.byref(cache.struct()), int(q_pos0), float(softmax_scale),
                                              _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                              int(n_split), _stream(stream))
    _check("attn_verify_append_q8", st)
    return out


def attn_verify_append_q8_host_scratch_bytes(n_rows: int, n_q_heads: int, head_dim: int, q_pos0: int,
                                             n_kv_heads: int, n_split: int = 0) -> int:
    return int(load_library().attn_verify_append_q8_host_scratch_bytes(n_rows, n_q_heads, head_dim, q_pos0,
                                                                       n_kv_heads, n_split))


def attn_verify_append_q8_host(h_in: torch.Tensor, n_rows: int, n_q_heads: int, cache: KVCacheQ8, q_pos0: int,
                               softmax_scale: float, h_out: torch.Tensor, scratch: torch.Tensor, n_split: int = 0,
                               stream=None) -> None:
    """attn_verify_append_q8 from and to host tensors: h_in (CPU fp32) holds q [T][Hq][hd] then
    k_new and v_new [T][Hkv][hd]; h_out (CPU fp32 [T][Hq][hd]) is written once the stream gets
    there.  Pinned tensors are read by a copy kernel and written in place by the merge;
    pageable ones go through copy-engine transfers.  scratch: device bytes from the
    scratch-size query."""
    for t, name in ((h_in, "h_in"), (h_out, "h_out")):
        if t.device.type != "cpu" or t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CPU float32 tensor")
    hd, hkv = cache.head_dim, cache.n_kv_heads
    if h_in.numel() != n_rows * (n_q_heads + 2 * hkv) * hd or h_out.numel() != n_rows * n_q_heads * hd:
        raise ValueError("h_in / h_out sizes do not match the shape")
    if scratch.device.type != "cuda" or not scratch.is_contiguous():
        raise ValueError("scratch must be a contiguous device tensor")
    st = load_library().attn_verify_append_q8_host(h_in.data_ptr(), n_rows, n_q_heads, ctypes.byref(cache.struct()),
                                                   int(q_pos0), float(softmax_scale), h_out.data_ptr(),
                                                   _ptr(scratch), scratch.numel() * scratch.element_size(),
                                                   int(n_split), _stream(stream))
    _check("attn_verify_append_q8_host", st)


class PreparedAppendVerifyHost:
    """attn_verify_append_q8_host with its arguments marshalled once, for a loop that repeats
    one call (same buffers, cache and window position): calling it is one C-ABI call.  The
    tensors must stay alive and in place while the object is used."""

    def __init__(self, h_in: torch.Tensor, n_rows: int, n_q_heads: int, cache: KVCacheQ8, q_pos0: int,
                 softmax_scale: float, h_out: torch.Tensor, scratch: torch.Tensor, n_split: int = 0, stream=None):
        for t, name in ((h_in, "h_in"), (h_out, "h_out")):
            if t.device.type != "cpu" or t.dtype != torch.float32 or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous CPU float32 tensor")
        hd, hkv = cache.head_dim, cache.n_kv_heads
        if h_in.numel() != n_rows * (n_q_heads + 2 * hkv) * hd or h_out.numel() != n_rows * n_q_heads * hd:
            raise ValueError("h_in / h_out sizes do not match the shape")
        if scratch.device.type != "cuda" or not scratch.is_contiguous():
            raise ValueError("scratch must be a contiguous device tensor")
        self._keep = (h_in, h_out, scratch, cache)
        self._struct = cache.struct()
        self._fn = load_library().attn_verify_append_q8_host
        self._args = (ctypes.c_void_p(h_in.data_ptr()), ctypes.c_int(n_rows), ctypes.c_int(n_q_heads),
                      ctypes.byref(self._struct), ctypes.c_int(int(q_pos0)), ctypes.c_float(float(softmax_scale)),
                      ctypes.c_void_p(h_out.data_ptr()), _ptr(scratch),
                      ctypes.c_size_t(scratch.numel() * scratch.element_size()), ctypes.c_int(int(n_split)),
                      _stream(stream))

    def __call__(self) -> None:
        st = self._fn(*self._args)
        if st != KVQ8_OK:
            raise KVQ8Error("attn_verify_append_q8_host", st)


def argmax_rows_top_prob(logits: torch.Tensor, workspace: torch.Tensor | None = None, argmax=None, top_prob=None,
                         stream=None):
    """Verify-head acceptance over fp32 logits [T][V] on the device: returns (argmax int32 [T],
    top_prob fp32 [T]) -- the first index of each row's maximum and softmax(row) there."""
    _need(logits, "logits", torch.float32)
    if logits.dim() != 2:
        raise ValueError("logits must be [T][V]")
    n_rows, vocab = logits.shape
    if argmax is None:
        argmax = _empty(n_rows, torch.int32, logits.device, stream)
    if top_prob is None:
        top_prob = _empty(n_rows, torch.float32, logits.device, stream)
    _need(argmax, "argmax", torch.int32)
    _need(top_prob, "top_prob", torch.float32)
    lib = load_library()
    if workspace is None:
        workspace = _scratch(max(int(lib.argmax_rows_top_prob_workspace_bytes(n_rows, vocab)), 16), logits.device,
                             stream)
    st = lib.argmax_rows_top_prob(_ptr(logits), n_rows, vocab, _ptr(argmax), _ptr(top_prob), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream))
    _check("argmax_rows_top_prob", st)
    return argmax, top_prob


def kvq8_selftest_convert(kind: int, words: torch.Tensor, stream=None) -> torch.Tensor:
    """Run the kernels' code -> fp16 conversion `kind` (0-3, see the header) over int32 words on the
    device; returns the fp16 pairs as int32 words (2 per input word for kinds 0 and 1, 4 for 2 and 3)."""
    _need(words, "words", torch.int32)
    n = words.numel()
    out = _empty(n * (2 if kind in (0, 1) else 4), torch.int32, words.device, stream)
    st = load_library().kvq8_selftest_convert(int(kind), _ptr(words), _ptr(out), n, _stream(stream))
    _check("kvq8_selftest_convert", st)
    return out


def kvq8_selftest_wait_timeout(polls: int = 4096, stream=None) -> None:
    """One launch whose bounded wait on a barrier that nothing arrives on gives up after `polls`
    polls and sets the device error flag (read it with kvq8_device_error)."""
    st = load_library().kvq8_selftest_wait_timeout(int(polls), _stream(stream))
    _check("kvq8_selftest_wait_timeout", st)


def attn_combine(part_o: torch.Tensor, part_ml: torch.Tensor, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """Merge partials part_o [n_split][rows][hd], part_ml [n_split][rows][2] -> out [rows][hd] (fp32)."""
    _need(part_o, "part_o", torch.float32)
    _need(part_ml, "part_ml", torch.float32)
    n_split, rows, head_dim = part_o.shape
    if out is None:
        out = _empty((rows, head_dim), torch.float32, part_o.device, stream)
    _need(out, "out", torch.float32)
    st = load_library().attn_combine(_ptr(part_o), _ptr(part_ml), n_split, rows, head_dim, _ptr(out),
                                     _stream(stream))
    _check("attn_combine", st)
    return out


def attn_prompt_q8_workspace_bytes(n_q: int, n_q_heads: int, head_dim: int, kv_len: int, q_pos0: int,
                                   n_kv_heads: int) -> int:
    return int(load_library().attn_prompt_q8_workspace_bytes(n_q, n_q_heads, head_dim, kv_len, q_pos0, n_kv_heads))


def attn_prompt_f16_workspace_bytes(n_q: int, n_q_heads: int, head_dim: int, kv_len: int, q_pos0: int,
                                    n_kv_heads: int) -> int:
    return int(load_library().attn_prompt_f16_workspace_bytes(n_q, n_q_heads, head_dim, kv_len, q_pos0, n_kv_heads))


def attn_prompt_q8(q: torch.Tensor, cache: KVCacheQ8, kv_len: int, q_pos0: int, softmax_scale: float,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Prompt-chunk attention of fp16 q [n_q][Hq][hd] over the cache; returns fp32 [n_q][Hq][hd]."""
    _need(q, "q", torch.float16)
    n_q, n_q_heads, head_dim = q.shape
    if out is None:
        out = _empty(q.shape, torch.float32, q.device, stream)
    _need(out, "out", torch.float32)
    if workspace is None:
        nbytes = attn_prompt_q8_workspace_bytes(n_q, n_q_heads, head_dim, kv_len, q_pos0, cache.n_kv_heads)
        workspace = _scratch(max(nbytes, 16), q.device, stream)
    st = load_library().attn_prompt_q8(_ptr(q), n_q, n_q_heads, ctypes.byref(cache.struct()), int(kv_len),
                                       int(q_pos0), float(softmax_scale), _ptr(out), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream))
    _check("attn_prompt_q8", st)
    return out


def attn_verify_q8_noalloc(q: torch.Tensor, cache: KVCacheQ8, kv_len: int, q_pos0: int, softmax_scale: float,
                           out: torch.Tensor | None = None, n_split: int = 0, stream=None) -> torch.Tensor:
    """attn_verify_q8 without a workspace, for callers that cannot allocate device memory at
    call time: the library keeps the split partials in its own static device array.  The
    first call on a device must come before any stream capture; calls that overlap on the
    GPU share that array and must be serialised by the caller.  `out` must be given by such
    callers (it is only allocated here when omitted, as a convenience)."""
    _need(q, "q", torch.float32)
    n_rows, n_q_heads, _ = q.shape
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _need(out, "out", torch.float32)
    st = load_library().attn_verify_q8_noalloc(_ptr(q), n_rows, n_q_heads, ctypes.byref(cache.struct()),
                                               int(kv_len), int(q_pos0), float(softmax_scale), _ptr(out),
                                               int(n_split), _stream(stream))
    _check("attn_verify_q8_noalloc", st)
    return out


# ---------------------------------------------------------------- serving a batch over a paged cache

_DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def _addr(t, name: str, dtype: torch.dtype, shape: tuple, device: int) -> int:
    """The address of a contiguous tensor of this type and shape on this device.  These calls serve steps of a few
    microseconds, so the good case is tested with the fewest calls into torch."""
    if t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{device} "
                     f"(got {t.dtype}, {tuple(t.shape)}, {t.device})")


def _maybe(t, name: str, dtype: torch.dtype, shape: tuple, device: int):
    return None if t is None else _addr(t, name, dtype, shape, device)


def _launch_on(device: int, stream) -> int:
    """The raw stream to launch on, after checking that the tensors live on the current device."""
    if device < 0:
        raise ValueError("tensors must be on a CUDA device")
    if torch.cuda.current_device() != device:
        raise ValueError(f"the tensors are on cuda:{device}, which is not the current device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if hasattr(stream, "device") and stream.device.index != device:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to cuda:{device}")
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


class KVPagedCacheQ8:
    """Caller-owned paged Q8_0 K/V planes on one device (kvq8_paged_cache of include/kvq8attn.h): codes
    int8 [n_pages][n_kv_heads][page_size][head_dim], scales fp16 [n_pages][n_kv_heads][page_size][head_dim/32]."""

    def __init__(self, n_kv_heads: int, head_dim: int, page_size: int, n_pages: int, device="cuda"):
        rows = (n_pages, n_kv_heads, page_size)
        self._set(torch.zeros(rows + (head_dim,), dtype=torch.int8, device=device),
                  torch.zeros(rows + (head_dim // 32,), dtype=torch.float16, device=device),
                  torch.zeros(rows + (head_dim,), dtype=torch.int8, device=device),
                  torch.zeros(rows + (head_dim // 32,), dtype=torch.float16, device=device))

    @classmethod
    def from_planes(cls, k_codes, k_scales, v_codes, v_scales):
        c = cls.__new__(cls)
        c._set(k_codes, k_scales, v_codes, v_scales)
        return c

    def _set(self, k_codes, k_scales, v_codes, v_scales):
        shape = tuple(k_codes.shape)
        n_pages, n_kv_heads, page_size, head_dim = shape
        index = k_codes.get_device()
        for t, name in ((k_codes, "k_codes"), (v_codes, "v_codes")):
            _addr(t, name, torch.int8, shape, index)
        for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            _addr(t, name, torch.float16, shape[:3] + (head_dim // 32,), index)
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = shape
        self.device, self._index = k_codes.device, index
        self._planes = {"k_codes": k_codes, "k_scales": k_scales, "v_codes": v_codes, "v_scales": v_scales}
        self._struct = kvq8_paged_cache(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
                                        n_kv_heads, head_dim, page_size, n_pages)

    def _plane(name: str):
        # the C struct is kept, so a plane that is replaced has to reach it; one of another shape, type or device raises
        return property(lambda self: self._planes[name], lambda self, t: self._set(**{**self._planes, name: t}))

    k_codes, k_scales, v_codes, v_scales = _plane("k_codes"), _plane("k_scales"), _plane("v_codes"), _plane("v_scales")
    del _plane

    def struct(self) -> kvq8_paged_cache:
        return self._struct


def kvq8_paged_tables(lens: torch.Tensor, n_new: torch.Tensor, held: torch.Tensor, page_table: torch.Tensor,
                      free_ring: torch.Tensor, ring_state: torch.Tensor, page_size: int, row_starts: torch.Tensor,
                      slots: torch.Tensor, positions: torch.Tensor, status: torch.Tensor,
                      held_out: torch.Tensor | None = None, ring_out: torch.Tensor | None = None, stream=None) -> None:
    """Pages and slots of a step's new tokens from the requests' lengths: int32 lens, n_new, held [n], page_table
    [n][max_pages] and free_ring [n_pages] (both updated), ring_state [2]; outputs row_starts int32 [n + 1], slots
    int64 [n_rows], positions int32 [n_rows], status int32 [1].  held and ring_state are updated in place unless
    held_out / ring_out are given."""
    n, dev, i32 = lens.shape[0], lens.get_device(), torch.int32
    if page_table.dim() != 2 or free_ring.dim() != 1 or slots.dim() != 1:
        raise ValueError("page_table must be [n][max_pages], free_ring [n_pages] and slots [n_rows]")
    mp, n_pages, n_rows = page_table.shape[1], free_ring.shape[0], slots.shape[0]
    st = (_lib or load_library()).kvq8_paged_tables(
        _addr(lens, "lens", i32, (n,), dev), _addr(n_new, "n_new", i32, (n,), dev), _addr(held, "held", i32, (n,), dev),
        n, int(page_size), _addr(page_table, "page_table", i32, (n, mp), dev), mp,
        _addr(free_ring, "free_ring", i32, (n_pages,), dev), n_pages, _addr(ring_state, "ring_state", i32, (2,), dev),
        _addr(held if held_out is None else held_out, "held_out", i32, (n,), dev),
        _addr(ring_state if ring_out is None else ring_out, "ring_out", i32, (2,), dev),
        _addr(row_starts, "row_starts", i32, (n + 1,), dev), _addr(slots, "slots", torch.int64, (n_rows,), dev),
        _addr(positions, "positions", i32, (n_rows,), dev), n_rows, _addr(status, "status", i32, (1,), dev),
        _launch_on(dev, stream))
    _check("kvq8_paged_tables", st)


def _token_stride(t: torch.Tensor, name: str, cache: KVPagedCacheQ8) -> int:
    if t.dim() != 3 or t.shape[1:] != (cache.n_kv_heads, cache.head_dim) or t.get_device() != cache._index:
        raise ValueError(f"{name} must be [n_tok][{cache.n_kv_heads}][{cache.head_dim}] on {cache.device}")
    if t.stride(2) != 1 or (t.stride(1) != cache.head_dim and cache.n_kv_heads > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else cache.n_kv_heads * cache.head_dim


def kvq8_paged_append(k: torch.Tensor, v: torch.Tensor, cache: KVPagedCacheQ8, slots: torch.Tensor, stream=None) -> None:
    """Quantise K and V values [n_tok][n_kv_heads][head_dim] (fp32, fp16 or bf16; tokens may be strided) into the
    cache at int64 slots [n_tok], which are distinct; slots outside the cache are skipped."""
    if k.dtype is not v.dtype or k.dtype not in _DTYPE or k.shape != v.shape:
        raise ValueError("k and v must have one shape and one type (float32, float16 or bfloat16)")
    ks, vs = _token_stride(k, "k", cache), _token_stride(v, "v", cache)
    st = (_lib or load_library()).kvq8_paged_append(k.data_ptr(), v.data_ptr(), _DTYPE[k.dtype], k.shape[0], ks, vs,
                                          cache._struct, _addr(slots, "slots", torch.int64, (k.shape[0],), cache._index),
                                          _launch_on(cache._index, stream))
    _check("kvq8_paged_append", st)


def kvq8_paged_read(cache: KVPagedCacheQ8, slots: torch.Tensor, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    """Write the values of int64 slots [n_tok] into k and v [n_tok][n_kv_heads][head_dim] (fp32, fp16 or bf16; tokens
    and heads may be strided, so a KVCacheF16's planes can be given as k.transpose(0, 1)[:n_tok])."""
    n = slots.shape[0]
    if k.dtype is not v.dtype or k.dtype not in _DTYPE:
        raise ValueError("k and v must have one type (float32, float16 or bfloat16)")
    strides = []
    for t, name in ((k, "k"), (v, "v")):
        if t.shape != (n, cache.n_kv_heads, cache.head_dim) or t.stride(2) != 1 or t.get_device() != cache._index:
            raise ValueError(f"{name} must be [{n}][{cache.n_kv_heads}][{cache.head_dim}] with contiguous dims on {cache.device}")
        strides.append((ctypes.c_int64 * 2)(t.stride(0) if n > 1 else cache.head_dim,
                                            t.stride(1) if cache.n_kv_heads > 1 else cache.head_dim))
    st = (_lib or load_library()).kvq8_paged_read(cache._struct, _addr(slots, "slots", torch.int64, (n,), cache._index), n,
                                        _DTYPE[k.dtype], k.data_ptr(), v.data_ptr(), strides[0], strides[1],
                                        _launch_on(cache._index, stream))
    _check("kvq8_paged_read", st)


def attn_verify_paged_q8_workspace_bytes(n_q_heads: int, n_kv_heads: int, head_dim: int, max_rows: int) -> int:
    return int((_lib or load_library()).attn_verify_paged_q8_workspace_bytes(n_q_heads, n_kv_heads, head_dim, max_rows))


def attn_verify_paged_q8(q: torch.Tensor, cache: KVPagedCacheQ8, page_table: torch.Tensor, lens: torch.Tensor,
                         row_starts: torch.Tensor, max_rows: int, softmax_scale: float,
                         window_mask: torch.Tensor | None = None, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Verify attention of a batch's windows: fp16 or bf16 q [n_rows][Hq][hd] (rows may be strided), page_table int32
    [n][max_pages], lens int32 [n], row_starts int32 [n + 1], window_mask int64 [n_rows] (bit j of a row's word = it
    sees window key j) or None for chains.  Returns out, of q's type; rows of no request are left as they were."""
    dev = cache._index
    if q.dim() != 3 or q.dtype not in (torch.float16, torch.bfloat16) or q.get_device() != dev or q.shape[2] != cache.head_dim:
        raise ValueError(f"q must be float16 or bfloat16 [n_rows][n_q_heads][{cache.head_dim}] on {cache.device}")
    n_rows, hq, hd = q.shape
    if q.stride(2) != 1 or (q.stride(1) != hd and hq > 1):
        raise ValueError("q: the heads of a row must be contiguous")
    n, mp = page_table.shape
    if out is None:
        out = _empty((n_rows, hq, hd), q.dtype, q.device, stream)
    lib = (_lib or load_library())
    if workspace is None:
        workspace = _scratch(max(lib.attn_verify_paged_q8_workspace_bytes(hq, cache.n_kv_heads, hd, int(max_rows)), 16), q.device,
                             stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {cache.device}")
    st = lib.attn_verify_paged_q8(
        q.data_ptr(), _DTYPE[q.dtype], q.stride(0) if n_rows > 1 else hq * hd, n_rows, hq, cache._struct,
        _addr(page_table, "page_table", torch.int32, (n, mp), dev), mp, _addr(lens, "lens", torch.int32, (n,), dev),
        _addr(row_starts, "row_starts", torch.int32, (n + 1,), dev), n, int(max_rows),
        _maybe(window_mask, "window_mask", torch.int64, (n_rows,), dev), float(softmax_scale),
        _addr(out, "out", q.dtype, (n_rows, hq, hd), dev), workspace.data_ptr(), workspace.nbytes, _launch_on(dev, stream))
    _check("attn_verify_paged_q8", st)
    return out


def logits_adjust(logits: torch.Tensor, row_starts: torch.Tensor, penalties: torch.Tensor | None = None,
                  counts: torch.Tensor | None = None, state_of: torch.Tensor | None = None,
                  window_tokens: torch.Tensor | None = None, window_mask: torch.Tensor | None = None,
                  bias_starts: torch.Tensor | None = None, bias_tokens: torch.Tensor | None = None,
                  bias_values: torch.Tensor | None = None, grammar: torch.Tensor | None = None,
                  grammar_of: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Logits [n_rows][V] (fp32, fp16 or bf16; rows may be strided) bent by the requests' penalties fp32 [n][3]
    (repetition, frequency, presence) over counts int32 [n_states][V] and the drafted window_tokens int32 [n_rows],
    by biases and by grammar masks int32 [n_grammar][ceil(V/32)]; see include/kvq8attn.h.  Returns fp32 out [n_rows][V]
    (out=logits works in place for fp32); rows of no request are left as they were."""
    dev, i32, f32 = logits.get_device(), torch.int32, torch.float32
    if logits.dim() != 2 or logits.dtype not in _DTYPE or logits.stride(1) != 1 and logits.shape[1] > 1:
        raise ValueError("logits must be [n_rows][V] of float32, float16 or bfloat16 with contiguous rows")
    rows, vocab = logits.shape
    n = row_starts.shape[0] - 1
    if out is None:
        out = _empty((rows, vocab), f32, logits.device, stream)
    if out.dtype is not f32 or out.shape != logits.shape or out.get_device() != dev or (out.stride(1) != 1 and vocab > 1):
        raise ValueError(f"out must be float32 [{rows}][{vocab}] with contiguous rows on {logits.device}")
    n_states = 0 if counts is None else counts.shape[0]
    n_bias = 0 if bias_tokens is None else bias_tokens.shape[0]
    n_grammar = 0 if grammar is None else grammar.shape[0]
    st = (_lib or load_library()).logits_adjust(
        logits.data_ptr(), _DTYPE[logits.dtype], logits.stride(0) if rows > 1 else vocab, rows, vocab,
        _addr(row_starts, "row_starts", i32, (n + 1,), dev), n, _maybe(penalties, "penalties", f32, (n, 3), dev),
        _maybe(counts, "counts", i32, (n_states, vocab), dev), n_states,
        _maybe(state_of, "state_of", i32, (n,), dev), _maybe(window_tokens, "window_tokens", i32, (rows,), dev),
        _maybe(window_mask, "window_mask", torch.int64, (rows,), dev),
        _maybe(bias_starts, "bias_starts", i32, (n + 1,), dev),
        _maybe(bias_tokens, "bias_tokens", i32, (n_bias,), dev),
        _maybe(bias_values, "bias_values", f32, (n_bias,), dev), n_bias,
        _maybe(grammar, "grammar", i32, (n_grammar, (vocab + 31) // 32), dev), n_grammar,
        _maybe(grammar_of, "grammar_of", i32, (rows,), dev), out.data_ptr(), out.stride(0) if rows > 1 else vocab,
        _launch_on(dev, stream))
    _check("logits_adjust", st)
    return out


def token_counts(tokens: torch.Tensor, token_starts: torch.Tensor, counts: torch.Tensor,
                 prompt_lens: torch.Tensor | None = None, state_of: torch.Tensor | None = None, clear: bool = False,
                 stream=None) -> torch.Tensor:
    """Count int32 tokens [n_tokens], list i = [token_starts[i], token_starts[i + 1]), into counts int32 [n_states][V]
    (bit 31: in the prompt; bits 0-30: times generated); clear: the lists' rows start from zero.  Returns counts."""
    dev, i32 = counts.get_device(), torch.int32
    n = token_starts.shape[0] - 1
    if counts.dim() != 2 or tokens.dim() != 1:
        raise ValueError("counts must be [n_states][V] and tokens [n_tokens]")
    st = (_lib or load_library()).token_counts(
        _addr(tokens, "tokens", i32, tuple(tokens.shape), dev), _addr(token_starts, "token_starts", i32, (n + 1,), dev), n,
        tokens.shape[0], _maybe(prompt_lens, "prompt_lens", i32, (n,), dev),
        _maybe(state_of, "state_of", i32, (n,), dev), 1 if clear else 0,
        _addr(counts, "counts", i32, tuple(counts.shape), dev), counts.shape[0], counts.shape[1], _launch_on(dev, stream))
    _check("token_counts", st)
    return counts
