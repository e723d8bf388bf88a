"""W8A8 FP8 block-scaled linear layer for B200 (sm_100a).

Python binding of the C ABI in ``include/fp8bq.h`` (library ``libfp8bq.so``
built in this directory by ``build.py``).  This module only marshals torch
tensors (device memory and the current CUDA stream) into the C calls; every
step of the computation runs in the library's CUDA kernels.  There is no CPU
fallback: if the library is missing or no sm_100 device is current, the calls
raise.

Functions (names follow the C ABI without the ``fp8bq_`` prefix):

* ``quantize_act(x)``        BF16 [M, K] -> (E4M3 codes uint8 [M, K], FP32 [M, K/128])
* ``quantize_weight(w)``     BF16 [N, K] -> (E4M3 codes uint8 [N, K], FP32 [N/128, K/128])
* ``gemm(qa, sa, qw, sw)``   -> BF16 [M, N]
* ``linear(x, qw, sw)``      -> BF16 [M, N], activation quantization fused into the call
* ``kv_write_e4m3(k, v, loc, k_cache, v_cache)``  E4M3 unit-scale KV-cache write (in place)
* ``silu_mul_quantize(gu)``  BF16 [M, 2I] gate|up -> (codes [M, I], FP32 [M, I/128])
* ``rms_norm_quantize(x, weight, eps, residual)``  norm (+ residual) -> (codes, FP32 scales);
  ``rms_norm(...)`` -> BF16
* ``rope_inv_freq(rot_dim, base, scaling, ...)``  -> (FP32 frequencies, factor on cos and sin)
* ``rope_kv_write_e4m3(qkv, positions, inv_freq, loc, k_cache, v_cache)``  rotated queries BF16;
  rotated keys and values to the E4M3 cache (in place)
* ``paged_attention(q, k_cache, v_cache, page_table, seq_lens, cu_q, ...)``  attention of new
  tokens over the paged E4M3 cache -> BF16
* ``nvfp4_quantize_weight(w)`` BF16 [N, K] -> (packed uint8 [N, K/2], E4M3 uint8 [N, K/16], FP32 [1])
* ``nvfp4_gemm_a16(x, packed, sb, g)`` BF16 [M, K] x NVFP4 W -> BF16 [M, N]
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

__all__ = [
    "Fp8bqError", "lib", "quantize_act", "quantize_weight", "gemm", "gemm_noalloc", "linear",
    "workspace_size", "new_workspace", "workspace_init", "last_device_status",
    "launch_count", "status_string", "selftest_timeout", "OP_GEMM", "OP_LINEAR", "OP_GEMM_SILU",
    "LIB_PATH", "kv_write_e4m3", "silu_mul_quantize", "gemm_silu_mul_quantize",
    "nvfp4_quantize_weight", "nvfp4_gemm_a16", "rms_norm_quantize", "rms_norm", "rope_inv_freq",
    "rope_kv_write_e4m3", "paged_attention", "attention_workspace_size", "new_attention_workspace",
    "HEAD_DIM", "WORKSPACE_HEADER",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfp8bq.so")
OP_GEMM = 0
OP_LINEAR = 1
OP_GEMM_SILU = 2
HEAD_DIM = 128  # channels of a head in paged_attention
WORKSPACE_HEADER = 16384  # bytes of counters at the start of every workspace
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3, "yarn_exact": 4}

STATUS_NAMES = {
    0: "FP8BQ_OK", 1: "FP8BQ_ERR_INVALID_ARG", 2: "FP8BQ_ERR_UNSUPPORTED_SHAPE",
    3: "FP8BQ_ERR_MISALIGNED", 4: "FP8BQ_ERR_WORKSPACE", 5: "FP8BQ_ERR_CUDA",
    6: "FP8BQ_ERR_TIMEOUT", 7: "FP8BQ_ERR_NO_DEVICE", 8: "FP8BQ_ERR_INDEX",
}

_lock = threading.Lock()
_lib = None


class Fp8bqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


def lib() -> ctypes.CDLL:
    """Loads libfp8bq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:  # loaded: no lock on the per-call path
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m fp8_block_scaled_09_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        st = ctypes.c_int
        L.fp8bq_quantize_act.argtypes = [P, I, I, P, P, P]
        L.fp8bq_quantize_weight.argtypes = [P, I, I, P, P, P]
        L.fp8bq_gemm.argtypes = [P, P, P, P, I, I, I, P, P, S, P]
        L.fp8bq_linear.argtypes = [P, P, P, I, I, I, P, P, S, P]
        L.fp8bq_gemm_noalloc.argtypes = [P, P, P, P, I, I, I, P, P]
        L.fp8bq_selftest_timeout.argtypes = [ctypes.c_uint32, P]
        L.fp8bq_kv_write_e4m3.argtypes = [P, P, I, I, I, P, P, P, I, I, P]
        L.fp8bq_silu_mul_quantize.argtypes = [P, I, I, P, P, P, P]
        L.fp8bq_gemm_silu_mul_quantize.argtypes = [P, P, P, P, I, I, I, P, P, P, P, S, P]
        L.fp8bq_nvfp4_quantize_weight.argtypes = [P, I, I, P, P, P, P]
        L.fp8bq_nvfp4_gemm_a16.argtypes = [P, P, P, P, I, I, I, P, P]
        F, D, N = ctypes.c_float, ctypes.c_double, ctypes.c_int
        L.fp8bq_rms_norm_quantize.argtypes = [P, P, P, F, I, I, P, P, P, P, P]
        L.fp8bq_rope_inv_freq.argtypes = [I, D, N, D, D, D, D, P, P]
        L.fp8bq_rope_kv_write_e4m3.argtypes = [P, I, I, I, I, I, P, P, I, N, F, P, P, I, P, P, I, I, P]
        L.fp8bq_paged_attention.argtypes = [P, I, P, P, I, I, P, I, I, I, P, P, I, I, I, I, I, F, N,
                                            P, I, P, P, S, P]
        L.fp8bq_paged_attention_workspace_size.argtypes = [I, I, I, I, I]
        L.fp8bq_paged_attention_workspace_size.restype = S
        L.fp8bq_workspace_size.argtypes = [ctypes.c_int, I, I, I]
        L.fp8bq_workspace_size.restype = S
        L.fp8bq_workspace_init.argtypes = [P, S, P]
        L.fp8bq_last_device_status.argtypes = [P]
        L.fp8bq_status_string.argtypes = [st]
        L.fp8bq_status_string.restype = ctypes.c_char_p
        L.fp8bq_launch_count.argtypes = []
        L.fp8bq_launch_count.restype = ctypes.c_uint64
        L.fp8bq_version.argtypes = []
        L.fp8bq_version.restype = ctypes.c_int
        L.fp8bq_clear_cache.argtypes = []
        L.fp8bq_clear_cache.restype = None
        for name in ("fp8bq_quantize_act", "fp8bq_quantize_weight", "fp8bq_gemm", "fp8bq_linear",
                     "fp8bq_workspace_init", "fp8bq_last_device_status", "fp8bq_gemm_noalloc",
                     "fp8bq_selftest_timeout", "fp8bq_kv_write_e4m3", "fp8bq_silu_mul_quantize",
                     "fp8bq_gemm_silu_mul_quantize",
                     "fp8bq_nvfp4_quantize_weight", "fp8bq_nvfp4_gemm_a16",
                     "fp8bq_rms_norm_quantize", "fp8bq_rope_inv_freq", "fp8bq_rope_kv_write_e4m3",
                     "fp8bq_paged_attention"):
            getattr(L, name).restype = st
        _lib = L
        return L


def status_string(status: int) -> str:
    return lib().fp8bq_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != 0:
        raise Fp8bqError(status, what)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# Pointers and stream handles are passed as plain Python ints (or None for
# NULL): every argument is declared c_void_p, so ctypes converts them without a
# c_void_p object per argument (a few microseconds per call on the host).
def _stream(t: torch.Tensor) -> int:
    # the current stream's handle without building a torch.cuda.Stream object
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t: torch.Tensor | None) -> int | None:
    return t.data_ptr() if t is not None else None


def _codes(t: torch.Tensor) -> torch.Tensor:
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise TypeError(f"E4M3 codes must be uint8 or float8_e4m3fn, got {t.dtype}")
    return t


def _need(t: torch.Tensor, dtype: torch.dtype, name: str) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")


def workspace_size(op: int, M: int, N: int, K: int) -> int:
    return int(lib().fp8bq_workspace_size(op, M, N, K))


def new_workspace(op: int, M: int, N: int, K: int, device) -> torch.Tensor:
    """A zero-filled (initial-state) workspace for this operation and shape."""
    return torch.zeros(max(workspace_size(op, M, N, K), 256), dtype=torch.uint8, device=device)


def workspace_init(ws: torch.Tensor) -> None:
    _check(lib().fp8bq_workspace_init(_ptr(ws), ws.numel(), _stream(ws)), "fp8bq_workspace_init")


def quantize_act(x: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None):
    _need(x, torch.bfloat16, "x")
    M, K = x.shape
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.empty((M, K // 128), dtype=torch.float32, device=x.device)
    _check(lib().fp8bq_quantize_act(_ptr(x), M, K, _ptr(q), _ptr(s), _stream(x)),
           "fp8bq_quantize_act")
    return q, s


def quantize_weight(w: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None):
    _need(w, torch.bfloat16, "w")
    N, K = w.shape
    if q is None:
        q = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    if s is None:
        s = torch.empty((N // 128, K // 128), dtype=torch.float32, device=w.device)
    _check(lib().fp8bq_quantize_weight(_ptr(w), N, K, _ptr(q), _ptr(s), _stream(w)),
           "fp8bq_quantize_weight")
    return q, s


def gemm(qa: torch.Tensor, sa: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor,
         out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    qa, qw = _codes(qa), _codes(qw)
    _need(qa, torch.uint8, "qa")
    _need(qw, torch.uint8, "qw")
    _need(sa, torch.float32, "sa")
    _need(sw, torch.float32, "sw")
    M, K = qa.shape
    N = qw.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=qa.device)
    if workspace is None:
        workspace = new_workspace(OP_GEMM, M, N, K, qa.device)
    _check(lib().fp8bq_gemm(_ptr(qa), _ptr(sa), _ptr(qw), _ptr(sw), M, N, K, _ptr(out),
                            _ptr(workspace), workspace.numel(), _stream(qa)), "fp8bq_gemm")
    return out


def gemm_noalloc(qa: torch.Tensor, sa: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor,
                 out: torch.Tensor) -> torch.Tensor:
    """fp8bq_gemm_noalloc: the GEMM with the library's built-in scratch instead of a
    workspace, for callers that cannot allocate device memory.  `out` must be given
    (this call allocates nothing); calls must not overlap on the GPU."""
    qa, qw = _codes(qa), _codes(qw)
    _need(qa, torch.uint8, "qa")
    _need(qw, torch.uint8, "qw")
    _need(sa, torch.float32, "sa")
    _need(sw, torch.float32, "sw")
    _need(out, torch.bfloat16, "out")
    M, K = qa.shape
    N = qw.shape[0]
    _check(lib().fp8bq_gemm_noalloc(_ptr(qa), _ptr(sa), _ptr(qw), _ptr(sw), M, N, K, _ptr(out),
                                    _stream(qa)), "fp8bq_gemm_noalloc")
    return out


def linear(x: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor, out: torch.Tensor | None = None,
           workspace: torch.Tensor | None = None) -> torch.Tensor:
    qw = _codes(qw)
    _need(x, torch.bfloat16, "x")
    _need(qw, torch.uint8, "qw")
    _need(sw, torch.float32, "sw")
    M, K = x.shape
    N = qw.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = new_workspace(OP_LINEAR, M, N, K, x.device)
    _check(lib().fp8bq_linear(_ptr(x), _ptr(qw), _ptr(sw), M, N, K, _ptr(out), _ptr(workspace),
                              workspace.numel(), _stream(x)), "fp8bq_linear")
    return out


def last_device_status(device=None) -> int:
    """Synchronizes the current stream and returns/clears the device status word."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    s = ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
    return int(lib().fp8bq_last_device_status(s))


def selftest_timeout(limit_us: int = 20000) -> None:
    """Enqueues the bounded-wait self-test (see fp8bq_selftest_timeout)."""
    dev = torch.device("cuda", torch.cuda.current_device())
    _check(lib().fp8bq_selftest_timeout(limit_us,
                                        ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)),
           "fp8bq_selftest_timeout")


def clear_cache() -> None:
    """Empties the library's cache of encoded TMA descriptors."""
    lib().fp8bq_clear_cache()


def launch_count() -> int:
    return int(lib().fp8bq_launch_count())


def kv_write_e4m3(k: torch.Tensor, v: torch.Tensor, loc: torch.Tensor, k_cache: torch.Tensor,
                  v_cache: torch.Tensor) -> None:
    """fp8bq_kv_write_e4m3: k_cache[loc[t], :W] = e4m3(k[t]) and the same for v, with
    unit scales.  k, v: BF16 [T, W] with unit column stride and a shared row stride (e.g.
    column slices of the fused QKV output); loc: int64 [T]; caches: uint8 or
    float8_e4m3fn [num_slots, slot_bytes], slot_bytes >= W.  Out-of-range slots are
    skipped on the device and reported through last_device_status()."""
    for t, name in ((k, "k"), (v, "v")):
        if t.dtype != torch.bfloat16 or t.device.type != "cuda" or t.dim() != 2 or t.stride(1) != 1:
            raise ValueError(f"{name} must be a 2-D CUDA BF16 tensor with unit column stride")
    if k.shape != v.shape or k.stride(0) != v.stride(0):
        raise ValueError("k and v must have the same shape and row stride")
    k_cache, v_cache = _codes(k_cache), _codes(v_cache)
    _need(k_cache, torch.uint8, "k_cache")
    _need(v_cache, torch.uint8, "v_cache")
    _need(loc, torch.int64, "loc")
    if k_cache.shape != v_cache.shape or k_cache.dim() != 2:
        raise ValueError("k_cache and v_cache must be [num_slots, slot_bytes] of the same shape")
    T, W = k.shape
    if loc.shape != (T,):
        raise ValueError("loc must be int64 [T]")
    _check(lib().fp8bq_kv_write_e4m3(_ptr(k), _ptr(v), k.stride(0), T, W, _ptr(loc),
                                     _ptr(k_cache), _ptr(v_cache), k_cache.shape[0],
                                     k_cache.shape[1], _stream(k)), "fp8bq_kv_write_e4m3")


def silu_mul_quantize(gu: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None,
                      h: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """fp8bq_silu_mul_quantize: gu BF16 [M, 2I] (gate, then up) -> the group-128
    quantization of h = BF16(silu(gate) * up): (codes uint8 [M, I], scales FP32
    [M, I/128]).  Pass h (BF16 [M, I]) to also receive h itself."""
    _need(gu, torch.bfloat16, "gu")
    M, two_i = gu.shape
    if two_i % 2:
        raise ValueError("gu must have an even number of columns (gate | up)")
    I = two_i // 2
    if q is None:
        q = torch.empty((M, I), dtype=torch.uint8, device=gu.device)
    if s is None:
        s = torch.empty((M, I // 128 if I % 128 == 0 else 0), dtype=torch.float32, device=gu.device)
    q = _codes(q)
    _need(q, torch.uint8, "q")
    _need(s, torch.float32, "s")
    if h is not None:
        _need(h, torch.bfloat16, "h")
    _check(lib().fp8bq_silu_mul_quantize(_ptr(gu), M, I, _ptr(q), _ptr(s), _ptr(h), _stream(gu)),
           "fp8bq_silu_mul_quantize")
    return q, s


def gemm_silu_mul_quantize(qa: torch.Tensor, sa: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor,
                           q: torch.Tensor | None = None, s: torch.Tensor | None = None,
                           h: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """fp8bq_gemm_silu_mul_quantize: the gate/up GEMM (fused weight codes qw [2I, K],
    gate rows first) with the SiLU-gated product quantized in its epilogue ->
    (codes uint8 [M, I], scales FP32 [M, I/128]), the same as
    silu_mul_quantize(gemm(qa, sa, qw, sw)).  Pass h (BF16 [M, I]) to also receive h."""
    qa, qw = _codes(qa), _codes(qw)
    _need(qa, torch.uint8, "qa")
    _need(qw, torch.uint8, "qw")
    _need(sa, torch.float32, "sa")
    _need(sw, torch.float32, "sw")
    M, K = qa.shape
    two_i = qw.shape[0]
    if two_i % 2:
        raise ValueError("qw must have an even number of rows (gate | up)")
    I = two_i // 2
    if q is None:
        q = torch.empty((M, I), dtype=torch.uint8, device=qa.device)
    if s is None:
        s = torch.empty((M, I // 128 if I % 128 == 0 else 0), dtype=torch.float32, device=qa.device)
    q = _codes(q)
    _need(q, torch.uint8, "q")
    _need(s, torch.float32, "s")
    if h is not None:
        _need(h, torch.bfloat16, "h")
    if workspace is None:
        workspace = new_workspace(OP_GEMM_SILU, M, two_i, K, qa.device)
    _check(lib().fp8bq_gemm_silu_mul_quantize(_ptr(qa), _ptr(sa), _ptr(qw), _ptr(sw), M, I, K,
                                              _ptr(q), _ptr(s), _ptr(h), _ptr(workspace),
                                              workspace.numel(), _stream(qa)),
           "fp8bq_gemm_silu_mul_quantize")
    return q, s


def nvfp4_quantize_weight(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """fp8bq_nvfp4_quantize_weight: BF16 W [N, K] -> (packed E2M1 uint8 [N, K/2], E4M3
    block scales uint8 [N, K/16], global scale FP32 [1]), plain min-max."""
    _need(w, torch.bfloat16, "w")
    N, K = w.shape
    packed = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    sb = torch.empty((N, K // 16), dtype=torch.uint8, device=w.device)
    g = torch.empty(1, dtype=torch.float32, device=w.device)
    _check(lib().fp8bq_nvfp4_quantize_weight(_ptr(w), N, K, _ptr(packed), _ptr(sb), _ptr(g),
                                             _stream(w)), "fp8bq_nvfp4_quantize_weight")
    return packed, sb, g


def nvfp4_gemm_a16(x: torch.Tensor, packed: torch.Tensor, sb: torch.Tensor, g: torch.Tensor,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """fp8bq_nvfp4_gemm_a16: BF16 X [M, K] times the NVFP4 weight (packed [N, K/2], sb
    [N, K/16], g FP32 [1]) transposed -> BF16 [M, N]."""
    _need(x, torch.bfloat16, "x")
    _need(packed, torch.uint8, "packed")
    sb = _codes(sb)
    _need(sb, torch.uint8, "sb")
    _need(g, torch.float32, "g")
    M, K = x.shape
    N = packed.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, "out")
    _check(lib().fp8bq_nvfp4_gemm_a16(_ptr(x), _ptr(packed), _ptr(sb), _ptr(g), M, N, K, _ptr(out),
                                      _stream(x)), "fp8bq_nvfp4_gemm_a16")
    return out


# The calls below take several tensors of one device, which need not be the
# current one.  A check that passes costs one expression (a few hundred
# nanoseconds) and gives the pointer; _refuse finds what is wrong otherwise.
def _refuse(t, dtype, shape, dev, name) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous (row-major)")


def _dense(t: torch.Tensor, dtype: torch.dtype, shape: tuple, dev: int, name: str) -> int:
    """The pointer of a contiguous tensor of this type and shape on this device."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, dtype, shape, dev, name)


def _rows(t: torch.Tensor, cols: int, rows: int, dev: int, name: str) -> int:
    """Row stride of a BF16 [rows, cols] tensor with unit column stride.  A single row may have any."""
    if t.dtype is not torch.bfloat16 or t.shape != (rows, cols) or t.get_device() != dev:
        _refuse(t, torch.bfloat16, (rows, cols), dev, name)
    step, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    return step if rows > 1 or (step >= cols and step % 8 == 0) else cols


def _first(t: torch.Tensor, name: str) -> int:
    """The device of a call, from its first tensor: on a GPU, two dimensions."""
    dev = t.get_device()
    if dev < 0 or t.dim() != 2:
        raise ValueError(f"{name} must be a CUDA tensor of two dimensions, got {tuple(t.shape)} on {t.device}")
    return dev


_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_stream_of = _raw_stream or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _call(dev: int, f, *args) -> None:
    """Calls a library function with this device current and its current stream as the last argument."""
    if dev == _get_device():
        status = f(*args, _stream_of(dev))
    else:
        with torch.cuda.device(dev):
            status = f(*args, _stream_of(dev))
    if status != 0:
        raise Fp8bqError(status, f.__name__)


def _norm(x, weight, eps, residual, residual_out, q, s, h) -> None:
    dev = _first(x, "x")
    shape = x.shape
    M, K = shape
    px = _dense(x, torch.bfloat16, shape, dev, "x")
    pw = _dense(weight, torch.bfloat16, (K,), dev, "weight")
    pr = po = None
    if residual is not None:
        pr = po = _dense(residual, torch.bfloat16, shape, dev, "residual")
        if residual_out is not None:
            po = _dense(residual_out, torch.bfloat16, shape, dev, "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    pq = ps = None
    if q is not None:
        pq = _dense(_codes(q), torch.uint8, shape, dev, "q")
        ps = _dense(s, torch.float32, (M, K // 128), dev, "s")
    ph = None if h is None else _dense(h, torch.bfloat16, shape, dev, "h")
    _call(dev, (_lib or lib()).fp8bq_rms_norm_quantize, px, pr, pw, eps, M, K, po, pq, ps, ph)


def rms_norm_quantize(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5,
                      residual: torch.Tensor | None = None,
                      residual_out: torch.Tensor | None = None, q: torch.Tensor | None = None,
                      s: torch.Tensor | None = None,
                      h: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """fp8bq_rms_norm_quantize: the group-128 quantization of the root-mean-square norm of
    r = BF16(x + residual) -> (codes uint8 [M, K], scales FP32 [M, K/128]).  x, residual: BF16
    [M, K]; weight: BF16 [K].  r goes to residual_out, or in place of residual when that is
    not given.  Pass h (BF16 [M, K]) to also receive the norm itself."""
    if q is None or s is None:
        _first(x, "x")
        M, K = x.shape
        if q is None:
            q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
        if s is None:
            s = torch.empty((M, K // 128), dtype=torch.float32, device=x.device)
    _norm(x, weight, eps, residual, residual_out, q, s, h)
    return q, s


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5,
             residual: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
             h: torch.Tensor | None = None) -> torch.Tensor:
    """fp8bq_rms_norm_quantize without codes: the BF16 norm of r = BF16(x + residual), e.g.
    before the BF16 output head.  Arguments as rms_norm_quantize."""
    if h is None:
        h = torch.empty_like(x)
    _norm(x, weight, eps, residual, residual_out, None, None, h)
    return h


def rope_inv_freq(rot_dim: int, base: float, scaling: str = "plain", factor: float = 1.0,
                  old_context: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                  device=None) -> tuple[torch.Tensor, float]:
    """fp8bq_rope_inv_freq: (FP32 frequencies [rot_dim / 2] on `device`, factor on cos and sin).
    scaling: "plain", "linear", "ntk", "yarn" or "yarn_exact" (both also need old_context;
    "yarn" rounds the ends of its ramp to whole pairs, as checkpoints have it)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    f = torch.empty(max(0, int(rot_dim) // 2), dtype=torch.float32)
    m = ctypes.c_float()
    _check(lib().fp8bq_rope_inv_freq(rot_dim, base, ROPE_SCALINGS[scaling], factor, old_context,
                                     beta_fast, beta_slow, _ptr(f), ctypes.addressof(m)),
           "fp8bq_rope_inv_freq")
    return (f if device is None else f.to(device)), m.value


def _caches(k_cache, v_cache, dev) -> tuple[int, int, int, int]:
    """Pointers, slots and slot bytes of the two E4M3 caches."""
    shape = k_cache.shape
    if len(shape) != 2:
        raise ValueError("k_cache and v_cache must be [num_slots, slot_bytes]")
    if k_cache.dtype is not torch.uint8:
        k_cache = _codes(k_cache)
    if v_cache.dtype is not torch.uint8:
        v_cache = _codes(v_cache)
    return (_dense(k_cache, torch.uint8, shape, dev, "k_cache"),
            _dense(v_cache, torch.uint8, shape, dev, "v_cache"), shape[0], shape[1])


def rope_kv_write_e4m3(qkv: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor,
                       loc: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       head_dim: int = HEAD_DIM, kv_heads: int | None = None,
                       interleaved: bool = False, mscale: float = 1.0,
                       q_out: torch.Tensor | None = None) -> torch.Tensor:
    """fp8bq_rope_kv_write_e4m3: rotates the query and key heads of the fused QKV output (BF16
    [T, (q_heads + 2 kv_heads) head_dim], rows may be strided) by positions (int64 [T]) and
    writes keys and values to slots loc (int64 [T], -1: padding) of the E4M3 caches (uint8 or
    float8_e4m3fn [num_slots, slot_bytes]).  kv_heads defaults to slot_bytes / head_dim.
    Returns the rotated queries q_out (BF16 [T, q_heads head_dim], new unless given; may be
    qkv's own query columns)."""
    dev = _first(qkv, "qkv")
    T, cols = qkv.shape
    step = _rows(qkv, cols, T, dev, "qkv")
    pk, pv, slots, slot_bytes = _caches(k_cache, v_cache, dev)
    if head_dim <= 0 or cols % head_dim:
        raise ValueError("qkv columns must be a multiple of head_dim")
    if kv_heads is None:
        kv_heads = slot_bytes // head_dim
    q_heads = cols // head_dim - 2 * kv_heads
    if q_heads <= 0:
        raise ValueError(f"qkv of {cols} columns has no query heads beside 2 x {kv_heads} kv heads")
    pp = _dense(positions, torch.int64, (T,), dev, "positions")
    pl = _dense(loc, torch.int64, (T,), dev, "loc")
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be FP32 [rot_dim / 2]")
    pairs = inv_freq.shape[0]
    pf = _dense(inv_freq, torch.float32, (pairs,), dev, "inv_freq")
    if q_out is None:
        q_out = torch.empty((T, q_heads * head_dim), dtype=torch.bfloat16, device=qkv.device)
    out_step = _rows(q_out, q_heads * head_dim, T, dev, "q_out")
    if T == 1 and q_out.data_ptr() == qkv.data_ptr():  # in place, whatever the row's stride
        out_step = step
    _call(dev, (_lib or lib()).fp8bq_rope_kv_write_e4m3, qkv.data_ptr(), step, T, q_heads, kv_heads,
          head_dim, pp, pf, 2 * pairs, 1 if interleaved else 0, mscale, pl, q_out.data_ptr(), out_step,
          pk, pv, slots, slot_bytes)
    return q_out


def attention_workspace_size(T: int, B: int, q_heads: int, kv_heads: int, max_q_len: int) -> int:
    return int(lib().fp8bq_paged_attention_workspace_size(T, B, q_heads, kv_heads, max_q_len))


def new_attention_workspace(T: int, B: int, q_heads: int, kv_heads: int, max_q_len: int,
                            device) -> torch.Tensor:
    """A workspace in its initial state for paged_attention of this batch: the counters at its
    start are zero, the rest (up to 42 MB) is as it was allocated."""
    ws = torch.empty(max(attention_workspace_size(T, B, q_heads, kv_heads, max_q_len), 256),
                     dtype=torch.uint8, device=device)
    ws[:WORKSPACE_HEADER].zero_()
    return ws


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    page_table: torch.Tensor, seq_lens: torch.Tensor, cu_q: torch.Tensor,
                    page_size: int, q_heads: int, kv_heads: int, max_q_len: int,
                    scale: float | None = None, causal: bool = True,
                    out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """fp8bq_paged_attention: attention of the new tokens q (BF16 [T, q_heads 128], rows may be
    strided) over the paged E4M3 caches (uint8 or float8_e4m3fn [num_slots, slot_bytes]) ->
    BF16 [T, q_heads 128].  Sequence b has rows cu_q[b] .. cu_q[b+1] - 1 of q, seq_lens[b] cache
    positions (its new tokens' among them) and pages page_table[b] (int32 [B, max_pages]; rows
    may be strided); seq_lens int32 [B], cu_q int32 [B + 1].  scale defaults to 128^-1/2.  Pass
    lse (FP32 [T, q_heads]) to also receive the log of the softmax's denominator.  Without a
    workspace (new_attention_workspace) each call makes its own.  Out-of-range
    pages and lengths are reported through last_device_status()."""
    dev = _first(q, "q")
    T, width = q.shape[0], q_heads * HEAD_DIM
    step = _rows(q, width, T, dev, "q")
    pk, pv, slots, slot_bytes = _caches(k_cache, v_cache, dev)
    if page_table.dtype is not torch.int32 or page_table.dim() != 2:
        raise TypeError("page_table must be int32 [B, max_pages]")
    if page_table.get_device() != dev:
        raise ValueError(f"page_table must be on cuda:{dev}, got {page_table.device}")
    B, pages = page_table.shape
    table_step, unit = page_table.stride()
    if pages > 1 and unit != 1 and B > 0:
        raise ValueError("page_table must have unit column stride")
    pl = _dense(seq_lens, torch.int32, (B,), dev, "seq_lens")
    pc = _dense(cu_q, torch.int32, (B + 1,), dev, "cu_q")
    if out is None:
        out = torch.empty((T, width), dtype=torch.bfloat16, device=q.device)
    out_step = _rows(out, width, T, dev, "out")
    pe = None if lse is None else _dense(lse, torch.float32, (T, q_heads), dev, "lse")
    if workspace is None:
        workspace = new_attention_workspace(T, B, q_heads, kv_heads, max_q_len, q.device)
    pw = _dense(workspace, torch.uint8, workspace.shape, dev, "workspace")
    _call(dev, (_lib or lib()).fp8bq_paged_attention, q.data_ptr(), step, pk, pv, slots, slot_bytes,
          page_table.data_ptr(), table_step if B > 1 else max(pages, table_step), pages, page_size,
          pl, pc, B, T, q_heads, kv_heads, max_q_len, HEAD_DIM ** -0.5 if scale is None else scale,
          1 if causal else 0, out.data_ptr(), out_step, pe, pw, workspace.numel())
    return out
