"""bit_gemv_gemm_gb300 -- Python binding of libtern (GB300 ternary-g128 product).

A thin ctypes layer over the C ABI in ``include/tern.h``: it checks tensor
types, passes ``data_ptr()`` and the current CUDA stream, and turns status codes
into exceptions.  Every step of the computation runs in the library's CUDA
kernels; PyTorch only allocates device memory and supplies streams.  There is
no fallback: if the library is not built, or the device is not an sm_103 GPU,
the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libtern.so")

TERN_OK = 0
_STATUS = {0: "ok", 1: "null pointer", 2: "bad shape", 3: "misaligned pointer", 4: "workspace too small",
           5: "CUDA error", 6: "device is not sm_103", 7: "device-side error"}

_lock = threading.Lock()
_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_LL = ctypes.c_longlong
_F = ctypes.c_float
_D = ctypes.c_double

EXPORTS = {
    "tern_status_str": (ctypes.c_char_p, [_I]),
    "tern_packed_bytes": (_SZ, [_I, _I]),
    "tern_pack": (_I, [_P, _I, _I, _P, _P, _P]),
    "tern_pack_host": (_I, [_P, _I, _I, _P, _P]),
    "tern_unpack_host": (_I, [_P, _I, _I, _P, _P]),
    "tern_validate_host": (_I, [_P, _I, _I, _P]),
    "tern_gemv_workspace_bytes": (_SZ, [_I, _I, _I]),
    "tern_gemv": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "tern_fwht": (_I, [_P, _P, _P, _I, _I, _P]),
    "tern_fwht_gemm": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "tern_gemm_workspace_bytes": (_SZ, [_I, _I, _I]),
    "tern_gemm": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "tern_device_error": (_I, [_P]),
    "tern_last_launch_count": (_I, []),
    "tern_gemv_noalloc": (_I, [_P, _P, _P, _P, _I, _I, _I, _P]),
    "tern_gemv_pair_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "tern_gemv_pair": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "tern_wait_selftest": (_I, [_I, _I, _P]),
    "tern_bin_packed_bytes": (_SZ, [_I, _I]),
    "tern_scales_from_g64": (_I, [_P, _I, _I, _P, _P, _P]),
    "tern_scales_from_g64_host": (_I, [_P, _I, _I, _P, _P]),
    "tern_bin_pack": (_I, [_P, _I, _I, _P, _P, _P]),
    "tern_bin_pack_host": (_I, [_P, _I, _I, _P, _P]),
    "tern_bin_unpack_host": (_I, [_P, _I, _I, _P]),
    "tern_bin_gemv": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "tern_bin_gemm": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "tern_affine_gemv": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "tern_affine_gemm": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "tern_f3_packed_bytes": (_SZ, [_I, _I]),
    "tern_f3_pack": (_I, [_P, _I, _I, _P, _P, _P]),
    "tern_f3_gemv": (_I, [_P, _P, _P, _P, _I, _I, _I, _P]),
    "tern_rope_frequencies_host": (_I, [_I, _D, _I, _D, _I, _D, _D, _P, _P]),
    "tern_rope_append": (_I, [_P, _P, _P, _I, _LL, _LL, _LL, _P, _P, _P, _F, _I, _I, _I, _I, _P, _P, _P, _P, _P]),
    "tern_paged_attention_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "tern_paged_attention": (_I, [_P, _LL, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _F, _I, _P, _P, _P, _SZ, _P]),
    "tern_attention_mass": (_I, [_P, _LL, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _F, _I, _P, _F, _P, _P, _P]),
    "tern_cache_evict": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P, _P, _P, _P, _P, _I, _P, _P, _P]),
}


class TernError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {_STATUS.get(status, 'unknown')} (status {status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded libtern.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libtern.so is not built ({LIB_PATH}); run "
                                   "`python -m bit_gemv_gemm_gb300.build` or __graft_entry__.build()")
            l = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in EXPORTS.items():
                fn = getattr(l, name)
                fn.restype = res
                fn.argtypes = args
            _lib = l
    return _lib


def _check(fn: str, st: int) -> None:
    if st != TERN_OK:
        raise TernError(fn, st)


def _stream(stream) -> int:
    if stream is None:
        # the raw handle: building a Stream object takes longer than a small call's launch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _covers(**need) -> None:
    """name=(tensor, elements): each tensor must hold at least the elements the
    call reads or writes through its pointer (the library sees only pointers
    and sizes, so a short tensor would be read or written past its end)."""
    for name, (t, n) in need.items():
        if t is not None and t.numel() < n:
            raise ValueError(f"{name} holds {t.numel()} elements; the call needs {n}")


def _dev(t: torch.Tensor, dtype, name: str) -> int:
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# ---------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------

def packed_bytes(N: int, K: int) -> int:
    return int(lib().tern_packed_bytes(N, K))


def gemv_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().tern_gemv_workspace_bytes(M, N, K))


def gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().tern_gemm_workspace_bytes(M, N, K))


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zero-filled device byte buffer usable as a libtern workspace (torch's
    allocations are 256-byte aligned)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


# What a call allocates itself has to be ready on the stream that the call runs on,
# which need not be the current one: memory that was freed on the current stream
# may still be in use there, and a fill there is not ordered before the kernel.

def _there(stream):
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                             else torch.cuda.ExternalStream(stream.cuda_stream))


def _scratch(nbytes: int, device, stream, counters: int | None = None) -> torch.Tensor:
    """A workspace for one call on `stream`, of which the first `counters` bytes
    (all if not given) have to be zero."""
    if stream is not None:
        with _there(stream):
            return _scratch(nbytes, device, None, counters)
    # (filling a small one takes less than the host needs for a view of its counters: a call of
    # one token 31 us, not 35)
    if counters is None or nbytes <= 8 << 20:
        return workspace(nbytes, device)
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    ws[:counters].zero_()
    return ws


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """An output of a call on `stream`, which the current stream will use too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _there(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream()
    if t.is_cuda and here.cuda_stream != stream.cuda_stream:
        t.record_stream(here)
    return t


# ---------------------------------------------------------------------------
# packing
# ---------------------------------------------------------------------------

def pack(t: torch.Tensor, codes: torch.Tensor | None = None, bad_count: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """Device packer: int8 trits [N, K] -> uint32 codes [N, K/16] (as int32 storage).

    If ``bad_count`` (int32 CUDA tensor of one element) is given, the number of
    entries outside {-1, 0, +1} is added to it."""
    N, K = t.shape
    if codes is None:
        codes = _new((N, K // 16), torch.int32, t.device, stream)
    _covers(codes=(codes, N * (K // 16)), bad_count=(bad_count, 1))
    bp = _dev(bad_count, torch.int32, "bad_count") if bad_count is not None else None
    _check("tern_pack", lib().tern_pack(_dev(t, torch.int8, "t"), N, K, _dev(codes, torch.int32, "codes"),
                                        bp, _stream(stream)))
    return codes


def scales_from_g64(s64: torch.Tensor, K: int, mismatch: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Scales of the group-size-64 pack (fp16 [N, K/64], each g128 scale
    repeated) -> g128 scales fp16 [N, K/128]; differing halves are counted."""
    N = s64.shape[0]
    out = _new((N, K // 128), torch.float16, s64.device, stream)
    _covers(s64=(s64, N * (K // 64)), mismatch=(mismatch, 1))
    mp = _dev(mismatch, torch.int32, "mismatch") if mismatch is not None else None
    _check("tern_scales_from_g64", lib().tern_scales_from_g64(_dev(s64, torch.float16, "s64"), N, K,
                                                              _dev(out, torch.float16, "s128"), mp, _stream(stream)))
    return out


def scales_from_g64_host(s64: np.ndarray, K: int) -> tuple[np.ndarray, int]:
    s64 = np.ascontiguousarray(s64, dtype=np.float16)
    N = s64.shape[0]
    out = np.empty((N, K // 128), dtype=np.float16)
    bad = ctypes.c_longlong(0)
    _check("tern_scales_from_g64_host", lib().tern_scales_from_g64_host(s64.ctypes.data, N, K, out.ctypes.data,
                                                                        ctypes.byref(bad)))
    return out, int(bad.value)


def bin_pack(t: torch.Tensor, words: torch.Tensor | None = None, bad_count: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    """Device packer of the 1-bit format: int8 [N, K] in {-1, +1} -> uint32
    words [N, K/32] (as int32 storage), bit k%32 of word k/32 set for +1."""
    N, K = t.shape
    if words is None:
        words = _new((N, K // 32), torch.int32, t.device, stream)
    _covers(words=(words, N * (K // 32)), bad_count=(bad_count, 1))
    bp = _dev(bad_count, torch.int32, "bad_count") if bad_count is not None else None
    _check("tern_bin_pack", lib().tern_bin_pack(_dev(t, torch.int8, "t"), N, K, _dev(words, torch.int32, "words"),
                                                bp, _stream(stream)))
    return words


def f3_pack(t: torch.Tensor, packed: torch.Tensor | None = None, bad_count: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """Device packer of the base-3 format: int8 [N, K] in {-1, 0, +1} -> uint8
    [N, 26 K/128], five trits per byte (q0 + 3 q1 + 9 q2 + 27 q3 + 81 q4)."""
    N, K = t.shape
    nbytes = int(lib().tern_f3_packed_bytes(N, K))
    if packed is None:
        packed = _new((N, 26 * (K // 128)), torch.uint8, t.device, stream)
    _covers(packed=(packed, nbytes), bad_count=(bad_count, 1))
    bp = _dev(bad_count, torch.int32, "bad_count") if bad_count is not None else None
    _check("tern_f3_pack", lib().tern_f3_pack(_dev(t, torch.int8, "t"), N, K, _dev(packed, torch.uint8, "packed"),
                                              bp, _stream(stream)))
    return packed


def f3_gemv(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, y: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """y (fp32 [M, N]) = x W^T on a base-3 pack, M = 1..16; x bf16 [M, K],
    packed uint8 [N, 26 K/128], scales fp16 [N, K/128].  No workspace."""
    M, K = x.shape
    N = packed.shape[0]
    if y is None:
        y = _new((M, N), torch.float32, x.device, stream)
    _covers(packed=(packed, N * 26 * (K // 128)), scales=(scales, N * (K // 128)), y=(y, M * N))
    _check("tern_f3_gemv", lib().tern_f3_gemv(
        _dev(x, torch.bfloat16, "x"), _dev(packed, torch.uint8, "packed"), _dev(scales, torch.float16, "scales"),
        _dev(y, torch.float32, "y"), M, N, K, _stream(stream)))
    return y


def bin_pack_host(t: np.ndarray) -> tuple[np.ndarray, int]:
    t = np.ascontiguousarray(t, dtype=np.int8)
    N, K = t.shape
    words = np.empty((N, K // 32), dtype=np.uint32)
    bad = ctypes.c_longlong(0)
    _check("tern_bin_pack_host", lib().tern_bin_pack_host(t.ctypes.data, N, K, words.ctypes.data,
                                                          ctypes.byref(bad)))
    return words, int(bad.value)


def bin_unpack_host(words: np.ndarray, K: int) -> np.ndarray:
    words = np.ascontiguousarray(words, dtype=np.uint32)
    N = words.shape[0]
    t = np.empty((N, K), dtype=np.int8)
    _check("tern_bin_unpack_host", lib().tern_bin_unpack_host(words.ctypes.data, N, K, t.ctypes.data))
    return t


def pack_host(t: np.ndarray) -> tuple[np.ndarray, int]:
    t = np.ascontiguousarray(t, dtype=np.int8)
    N, K = t.shape
    codes = np.empty((N, K // 16), dtype=np.uint32)
    bad = ctypes.c_longlong(0)
    _check("tern_pack_host", lib().tern_pack_host(t.ctypes.data, N, K, codes.ctypes.data, ctypes.byref(bad)))
    return codes, int(bad.value)


def unpack_host(codes: np.ndarray, K: int) -> tuple[np.ndarray, int]:
    codes = np.ascontiguousarray(codes, dtype=np.uint32)
    N = codes.shape[0]
    t = np.empty((N, K), dtype=np.int8)
    bad = ctypes.c_longlong(0)
    _check("tern_unpack_host", lib().tern_unpack_host(codes.ctypes.data, N, K, t.ctypes.data, ctypes.byref(bad)))
    return t, int(bad.value)


def validate_host(codes: np.ndarray, K: int) -> int:
    codes = np.ascontiguousarray(codes, dtype=np.uint32)
    bad = ctypes.c_longlong(0)
    _check("tern_validate_host", lib().tern_validate_host(codes.ctypes.data, codes.shape[0], K, ctypes.byref(bad)))
    return int(bad.value)


# ---------------------------------------------------------------------------
# products and rotation
# ---------------------------------------------------------------------------

def gemv(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, y: torch.Tensor | None = None,
         ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y (fp32 [M, N]) = x W^T for M = 1..16; x bf16 [M, K], codes int32 [N, K/16], scales fp16 [N, K/128]."""
    M, K = x.shape
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), torch.float32, x.device, stream)
    _covers(codes=(codes, N * (K // 16)), scales=(scales, N * (K // 128)), y=(y, M * N))
    if ws is None:
        ws = _scratch(gemv_workspace_bytes(M, N, K), x.device, stream)
    _check("tern_gemv", lib().tern_gemv(
        _dev(x, torch.bfloat16, "x"), _dev(codes, torch.int32, "codes"), _dev(scales, torch.float16, "scales"),
        _dev(y, torch.float32, "y"), M, N, K, _dev(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))
    return y


def bin_gemv(x: torch.Tensor, words: torch.Tensor, scales: torch.Tensor, y: torch.Tensor | None = None,
             ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The 1-bit sibling: y (fp32 [M, N]) = x W^T for M = 1..16, W = (2b - 1) s;
    x bf16 [M, K], words int32 [N, K/32], scales fp16 [N, K/128]."""
    M, K = x.shape
    N = words.shape[0]
    if y is None:
        y = _new((M, N), torch.float32, x.device, stream)
    _covers(words=(words, N * (K // 32)), scales=(scales, N * (K // 128)), y=(y, M * N))
    if ws is None:
        ws = _scratch(gemv_workspace_bytes(M, N, K), x.device, stream)
    _check("tern_bin_gemv", lib().tern_bin_gemv(
        _dev(x, torch.bfloat16, "x"), _dev(words, torch.int32, "words"), _dev(scales, torch.float16, "scales"),
        _dev(y, torch.float32, "y"), M, N, K, _dev(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))
    return y


def gemv_pair(x: torch.Tensor, codes_a: torch.Tensor, scales_a: torch.Tensor, codes_b: torch.Tensor,
              scales_b: torch.Tensor, y_a: torch.Tensor | None = None, y_b: torch.Tensor | None = None,
              ws: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Two products of the same activation in one launch: (x W_a^T, x W_b^T)."""
    M, K = x.shape
    Na, Nb = codes_a.shape[0], codes_b.shape[0]
    if y_a is None:
        y_a = _new((M, Na), torch.float32, x.device, stream)
    if y_b is None:
        y_b = _new((M, Nb), torch.float32, x.device, stream)
    _covers(codes_a=(codes_a, Na * (K // 16)), scales_a=(scales_a, Na * (K // 128)), y_a=(y_a, M * Na),
            codes_b=(codes_b, Nb * (K // 16)), scales_b=(scales_b, Nb * (K // 128)), y_b=(y_b, M * Nb))
    if ws is None:
        ws = _scratch(int(lib().tern_gemv_pair_workspace_bytes(M, Na, Nb, K)), x.device, stream)
    _check("tern_gemv_pair", lib().tern_gemv_pair(
        _dev(x, torch.bfloat16, "x"), _dev(codes_a, torch.int32, "codes_a"), _dev(scales_a, torch.float16, "scales_a"),
        _dev(y_a, torch.float32, "y_a"), Na, _dev(codes_b, torch.int32, "codes_b"),
        _dev(scales_b, torch.float16, "scales_b"), _dev(y_b, torch.float32, "y_b"), Nb, M, K,
        _dev(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))
    return y_a, y_b


def gemv_noalloc(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, y: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """tern_gemv without a workspace: the library's fixed scratch array is used."""
    M, K = x.shape
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), torch.float32, x.device, stream)
    _covers(codes=(codes, N * (K // 16)), scales=(scales, N * (K // 128)), y=(y, M * N))
    _check("tern_gemv_noalloc", lib().tern_gemv_noalloc(
        _dev(x, torch.bfloat16, "x"), _dev(codes, torch.int32, "codes"), _dev(scales, torch.float16, "scales"),
        _dev(y, torch.float32, "y"), M, N, K, _stream(stream)))
    return y


def fwht(x: torch.Tensor, signs: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y (bf16 [M, K]) = H_4096 (signs * x) / 64 per 4096-block of the last dimension."""
    M, K = x.shape
    if y is None:
        y = _new(x.shape, x.dtype, x.device, stream)
    _covers(signs=(signs, K), y=(y, M * K))
    _check("tern_fwht", lib().tern_fwht(_dev(x, torch.bfloat16, "x"), _dev(signs, torch.int8, "signs"),
                                        _dev(y, torch.bfloat16, "y"), M, K, _stream(stream)))
    return y


def fwht_gemm(x: torch.Tensor, signs: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
              y: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y (fp32 [M, N]) = rotate(x) W^T with the rotation fused into the product's prologue."""
    M, K = x.shape
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), torch.float32, x.device, stream)
    _covers(signs=(signs, K), codes=(codes, N * (K // 16)), scales=(scales, N * (K // 128)), y=(y, M * N))
    if ws is None:
        ws = _scratch(gemv_workspace_bytes(M, N, K), x.device, stream)
    _check("tern_fwht_gemm", lib().tern_fwht_gemm(
        _dev(x, torch.bfloat16, "x"), _dev(signs, torch.int8, "signs"), _dev(codes, torch.int32, "codes"),
        _dev(scales, torch.float16, "scales"), _dev(y, torch.float32, "y"), M, N, K,
        _dev(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))
    return y


def gemm(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, y: torch.Tensor | None = None,
         out_dtype=torch.float32, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y ([M, N], fp32 or bf16) = x W^T on the tcgen05 tensor cores, any M >= 1."""
    M, K = x.shape
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), out_dtype, x.device, stream)
    if y.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("y must be float32 or bfloat16")
    _covers(codes=(codes, N * (K // 16)), scales=(scales, N * (K // 128)), y=(y, M * N))
    if ws is None:
        ws = _scratch(gemm_workspace_bytes(M, N, K), x.device, stream)
    _check("tern_gemm", lib().tern_gemm(
        _dev(x, torch.bfloat16, "x"), _dev(codes, torch.int32, "codes"), _dev(scales, torch.float16, "scales"),
        _dev(y, y.dtype, "y"), 1 if y.dtype == torch.bfloat16 else 0, M, N, K,
        _dev(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))
    return y


def device_error() -> int:
    """Reads and clears the device-side error word (synchronizes the device)."""
    code = ctypes.c_int(0)
    _check("tern_device_error", lib().tern_device_error(ctypes.byref(code)))
    return int(code.value)


SELFTEST_RANGE_FLAG, SELFTEST_MBARRIER = 0, 1
DEVERR_GEMM_MMA_WAIT, DEVERR_GEMV_RANGE_FLAG_WAIT, DEVERR_GEMV_ACTIVATION_RANGE = 0x103, 0x202, 0x203
DEVERR_CACHE_PAGE, DEVERR_CACHE_SEQUENCE, DEVERR_CACHE_SLOT = 0x301, 0x302, 0x303
DEVERR_ATTN_WAIT = 0x311


def wait_selftest(which: int, limit_us: int, stream=None) -> None:
    """Runs one bounded wait on something nothing completes (tern_wait_selftest);
    the code it reports is read with device_error()."""
    _check("tern_wait_selftest", lib().tern_wait_selftest(which, limit_us, _stream(stream)))


def last_launch_count() -> int:
    return int(lib().tern_last_launch_count())


def bin_gemm(x: torch.Tensor, words: torch.Tensor, scales: torch.Tensor, y: torch.Tensor | None = None,
             out_dtype=torch.float32, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The 1-bit sibling format on the tcgen05 tensor cores: y ([M, N], fp32 or
    bf16) = x W^T, W = (2b - 1) s, any M >= 1."""
    M, K = x.shape
    N = words.shape[0]
    if y is None:
        y = _new((M, N), out_dtype, x.device, stream)
    if y.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("y must be float32 or bfloat16")
    _covers(words=(words, N * (K // 32)), scales=(scales, N * (K // 128)), y=(y, M * N))
    if ws is None:
        ws = _scratch(gemm_workspace_bytes(M, N, K), x.device, stream)
    _check("tern_bin_gemm", lib().tern_bin_gemm(
        _dev(x, torch.bfloat16, "x"), _dev(words, torch.int32, "words"), _dev(scales, torch.float16, "scales"),
        _dev(y, y.dtype, "y"), 1 if y.dtype == torch.bfloat16 else 0, M, N, K,
        _dev(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))
    return y


def affine_gemv(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor,
                y: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """An affine pack: y (fp32 [M, N]) = x W^T for M = 1..16, W = s q + b per
    group of 128; x bf16 [M, K], codes int32 [N, K/16] (every code 0..3),
    scales and biases fp16 [N, K/128]."""
    M, K = x.shape
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), torch.float32, x.device, stream)
    _covers(codes=(codes, N * (K // 16)), scales=(scales, N * (K // 128)), biases=(biases, N * (K // 128)),
            y=(y, M * N))
    if ws is None:
        ws = _scratch(gemv_workspace_bytes(M, N, K), x.device, stream)
    _check("tern_affine_gemv", lib().tern_affine_gemv(
        _dev(x, torch.bfloat16, "x"), _dev(codes, torch.int32, "codes"), _dev(scales, torch.float16, "scales"),
        _dev(biases, torch.float16, "biases"), _dev(y, torch.float32, "y"), M, N, K,
        _dev(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))
    return y


def affine_gemm(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor,
                y: torch.Tensor | None = None, out_dtype=torch.float32, ws: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """An affine pack on the tcgen05 tensor cores: y ([M, N], fp32 or bf16) =
    x W^T, W = s q + b per group of 128, any M >= 1."""
    M, K = x.shape
    N = codes.shape[0]
    if y is None:
        y = _new((M, N), out_dtype, x.device, stream)
    if y.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("y must be float32 or bfloat16")
    _covers(codes=(codes, N * (K // 16)), scales=(scales, N * (K // 128)), biases=(biases, N * (K // 128)),
            y=(y, M * N))
    if ws is None:
        ws = _scratch(gemm_workspace_bytes(M, N, K), x.device, stream)
    _check("tern_affine_gemm", lib().tern_affine_gemm(
        _dev(x, torch.bfloat16, "x"), _dev(codes, torch.int32, "codes"), _dev(scales, torch.float16, "scales"),
        _dev(biases, torch.float16, "biases"), _dev(y, y.dtype, "y"), 1 if y.dtype == torch.bfloat16 else 0,
        M, N, K, _dev(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))
    return y


# ---------------------------------------------------------------------------
# the paged key/value cache
# ---------------------------------------------------------------------------

class CacheLayout(ctypes.Structure):
    """tern_cache_layout: strides in elements."""
    _fields_ = [("pages", _I), ("page_size", _I), ("kv_heads", _I), ("head_dim", _I),
                ("page_stride", _LL), ("head_stride", _LL), ("slot_stride", _LL)]


# What the calls below learn from shapes and strides alone is kept by shape: a
# decode step makes the same small calls over and over, and the checks would take
# longer than the launch.

def _steps(shape, stride):
    """The strides with those of axes of one element, which say nothing (a view may
    hold any there), as in a contiguous array."""
    dense = [1] * len(shape)
    for i in range(len(shape) - 2, -1, -1):
        dense[i] = dense[i + 1] * shape[i + 1]
    return tuple(d if n == 1 else s for n, s, d in zip(shape, stride, dense))


@functools.lru_cache(maxsize=1024)
def _layout(name: str, shape, stride, like=None) -> CacheLayout:
    """The layout of one cache array, bf16 [pages, kv_heads, page_size, head_dim]
    with any strides over contiguous heads (a permuted [pages, page_size,
    kv_heads, head_dim] array is one); `like`: the shape and strides of its K array."""
    if len(shape) != 4 or stride[3] != 1:
        raise ValueError(f"{name} must be [pages, kv_heads, page_size, head_dim] with contiguous heads")
    stride = _steps(shape, stride)
    if like is not None and (shape, stride) != (like[0], _steps(*like)):
        raise ValueError(f"{name} must have the shape and strides of its K array")
    return CacheLayout(shape[0], shape[2], shape[1], shape[3], stride[0], stride[1], stride[2])


def _here(names: str, *tensors) -> None:
    """Each tensor (None left out) lies on the current device, whose kernel the call
    launches.  (A kernel can reach another GPU's memory where peer access is on,
    which is no way to run these.)"""
    now = torch.cuda.current_device()
    for i, t in enumerate(tensors):
        if t is not None and t.get_device() != now and t.is_cuda:   # (a CPU tensor: _dev says so)
            raise ValueError(f"{names.split()[i]} is on cuda:{t.get_device()}, the current device is cuda:{now}")


def _caches(k: torch.Tensor, v: torch.Tensor | None, kn: str, vn: str) -> CacheLayout:
    ks, kt = k.shape, k.stride()
    lay = _layout(kn, ks, kt)
    if v is not None:
        _layout(vn, v.shape, v.stride(), (ks, kt))
    if not k.is_cuda or k.dtype != torch.bfloat16:
        raise TypeError(f"{kn} must be a bfloat16 CUDA tensor")
    if v is not None:
        if not v.is_cuda or v.dtype != torch.bfloat16:
            raise TypeError(f"{vn} must be a bfloat16 CUDA tensor")
    return lay


@functools.lru_cache(maxsize=4096)
def _token_stride(name: str, shape, stride, heads, dim: int) -> int:
    """The token stride of [T, heads, dim] with each token's heads contiguous."""
    if len(shape) != 3 or stride[2] != 1 or (shape[1] > 1 and stride[1] != shape[2]):
        raise ValueError(f"{name} must be [tokens, heads, head_dim] with each token's heads contiguous")
    if shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must hold {'' if heads is None else heads} heads of {dim}, got {tuple(shape[1:])}")
    return stride[0] if shape[0] > 1 else shape[1] * shape[2]


def _tokens(t: torch.Tensor, dtype, name: str, heads, dim: int) -> int:
    stride = _token_stride(name, t.shape, t.stride(), heads, dim)
    if not t.is_cuda or t.dtype != dtype:
        raise TypeError(f"{name} must be a CUDA tensor of type {dtype}")
    return stride


_ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_len: int = 0, turns_fast: float = 32.0, turns_slow: float = 1.0):
    """(inv_freq, attn_factor) of a rotation over rot_dim values: fp32 numpy
    [rot_dim / 2] and a float.  scaling: "none", "linear" (positions divided by
    factor), "ntk" (a larger base) or "yarn" (by parts, with original_len)."""
    if scaling not in _ROPE_SCALING:
        raise ValueError(f"scaling must be one of {sorted(_ROPE_SCALING)}")
    out = np.empty(max(rot_dim // 2, 1), dtype=np.float32)
    af = ctypes.c_float(1.0)
    _check("tern_rope_frequencies_host", lib().tern_rope_frequencies_host(
        rot_dim, base, _ROPE_SCALING[scaling], factor, original_len, turns_fast, turns_slow, out.ctypes.data,
        ctypes.byref(af)))
    return out, float(af.value)


def rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
                inv_freq: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                q_out: torch.Tensor | None = None, interleaved: bool = False, attn_factor: float = 1.0,
                stream=None) -> torch.Tensor:
    """Turns q and k by their positions and appends k and v to the paged cache.

    q [T, q_heads, D], k and v [T, kv_heads, D]: all fp32 or all bf16, views of
    one product output included; positions int32 [T]; slots int64 [T] (page *
    page_size + slot, negative: not stored); inv_freq fp32 [rot_dim / 2], its
    length setting how much of a head turns; the caches bf16 [pages, kv_heads,
    page_size, D].  Returns the turned q, bf16 [T, q_heads, D]."""
    lay = _caches(k_cache, v_cache, "k_cache", "v_cache")
    D, Hk, kind = lay.head_dim, lay.kv_heads, q.dtype
    if kind not in (torch.float32, torch.bfloat16):
        raise TypeError("q must be float32 or bfloat16")
    qs, ks, vs = _tokens(q, kind, "q", None, D), _tokens(k, kind, "k", Hk, D), _tokens(v, kind, "v", Hk, D)
    T, Hq = q.shape[:2]
    if k.shape[0] != T or v.shape[0] != T:
        raise ValueError("q, k and v must hold the same number of tokens")
    if q_out is None:
        q_out = _new((T, Hq, D), torch.bfloat16, q.device, stream)
    _covers(positions=(positions, T), slots=(slots, T), q_out=(q_out, T * Hq * D))
    _here("q k v positions slots inv_freq k_cache v_cache q_out",
          q, k, v, positions, slots, inv_freq, k_cache, v_cache, q_out)
    _check("tern_rope_append", lib().tern_rope_append(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), 1 if kind == torch.float32 else 0, qs, ks, vs,
        _dev(positions, torch.int32, "positions"), _dev(slots, torch.int64, "slots"),
        _dev(inv_freq, torch.float32, "inv_freq"), attn_factor, 2 * inv_freq.numel(), 1 if interleaved else 0, T, Hq,
        _dev(q_out, torch.bfloat16, "q_out"), k_cache.data_ptr(), v_cache.data_ptr(), ctypes.addressof(lay),
        _stream(stream)))
    return q_out


ATTENTION_COUNTER_BYTES = 8192   # of the workspace, that have to be zero before its first use


def paged_attention_workspace_bytes(B: int, T: int, max_new: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().tern_paged_attention_workspace_bytes(B, T, max_new, q_heads, kv_heads, head_dim))


def _sequences(q, lay, table, lens, q_start, max_new):
    """(token stride, T, q_heads, B, table width, q_start pointer, max_new)."""
    qs = _tokens(q, torch.bfloat16, "q", None, lay.head_dim)
    T, Hq = q.shape[:2]
    if table.dim() != 2:
        raise ValueError("table must be [B, pages per sequence]")
    B, W = table.shape
    _covers(lens=(lens, B), q_start=(q_start, B + 1))
    if q_start is None:
        return qs, T, Hq, B, W, None, 0
    return qs, T, Hq, B, W, _dev(q_start, torch.int32, "q_start"), T if max_new is None else max_new


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor,
                    lens: torch.Tensor, q_start: torch.Tensor | None = None, max_new: int | None = None,
                    scale: float | None = None, window: int = 0, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of new tokens (one, a few or a chunk for each sequence) over a
    paged cache that already holds their keys.

    q bf16 [T, q_heads, D] (any token stride); table int32 [B, W]; lens int32
    [B], the new tokens included; q_start int32 [B + 1] (None: T / B tokens
    each) with max_new, the most tokens of one sequence (T if not given);
    scale 1/sqrt(D) if not given; window 0 or the number of last keys a query
    sees.  Returns out bf16 [T, q_heads, D]; lse fp32 [T, q_heads] if given."""
    lay = _caches(k_cache, v_cache, "k_cache", "v_cache")
    qs, T, Hq, B, W, start, max_new = _sequences(q, lay, table, lens, q_start, max_new)
    D = lay.head_dim
    if out is None:
        out = _new((T, Hq, D), torch.bfloat16, q.device, stream)
    _covers(out=(out, T * Hq * D), lse=(lse, T * Hq))
    _here("q k_cache v_cache table lens q_start out lse ws", q, k_cache, v_cache, table, lens, q_start, out, lse, ws)
    if ws is None:
        ws = _scratch(paged_attention_workspace_bytes(B, T, max_new if start else T // B, Hq, lay.kv_heads, D),
                      q.device, stream, ATTENTION_COUNTER_BYTES)
    _check("tern_paged_attention", lib().tern_paged_attention(
        q.data_ptr(), qs, k_cache.data_ptr(), v_cache.data_ptr(), ctypes.addressof(lay),
        _dev(table, torch.int32, "table"), W, _dev(lens, torch.int32, "lens"), start, B, T, max_new, Hq,
        D ** -0.5 if scale is None else scale, window, _dev(out, torch.bfloat16, "out"),
        None if lse is None else _dev(lse, torch.float32, "lse"), _dev(ws, torch.uint8, "ws"), ws.numel(),
        _stream(stream)))
    return out


def attention_mass(q: torch.Tensor, k_cache: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                   lse: torch.Tensor, mass: torch.Tensor, out: torch.Tensor | None = None,
                   q_start: torch.Tensor | None = None, max_new: int | None = None, scale: float | None = None,
                   window: int = 0, decay: float = 1.0, stream=None) -> torch.Tensor:
    """Adds the attention weight each cached key received from the new tokens
    to its running mass: out = decay * mass + sum exp(s - lse), fp32 [pages,
    kv_heads, page_size]; out defaults to mass itself.  The other arguments as
    paged_attention's, lse its output.  No page may stand in two sequences'
    tables: one's sum would overwrite the other's."""
    lay = _caches(k_cache, None, "k_cache", "")
    qs, T, Hq, B, W, start, max_new = _sequences(q, lay, table, lens, q_start, max_new)
    if out is None:
        out = mass
    need = lay.pages * lay.kv_heads * lay.page_size
    _covers(lse=(lse, T * Hq), mass=(mass, need), out=(out, need))
    _here("q k_cache table lens q_start lse mass out", q, k_cache, table, lens, q_start, lse, mass, out)
    _check("tern_attention_mass", lib().tern_attention_mass(
        q.data_ptr(), qs, k_cache.data_ptr(), ctypes.addressof(lay), _dev(table, torch.int32, "table"), W,
        _dev(lens, torch.int32, "lens"), start, B, T, max_new, Hq, lay.head_dim ** -0.5 if scale is None else scale,
        window, _dev(lse, torch.float32, "lse"), decay, _dev(mass, torch.float32, "mass"),
        _dev(out, torch.float32, "out"), _stream(stream)))
    return out


def cache_evict(k_cache: torch.Tensor, v_cache: torch.Tensor, mass: torch.Tensor, table: torch.Tensor,
                lens: torch.Tensor, budget: int, recent: int, dst_k: torch.Tensor, dst_v: torch.Tensor,
                dst_mass: torch.Tensor, dst_table: torch.Tensor, keep: torch.Tensor | None = None,
                dst_lens: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Keeps `budget` keys of each sequence and head, the `recent` last and the
    heaviest before them, and moves them (K, V and mass) to the pages
    dst_table of the destination arrays.  Returns (keep int32 [B, kv_heads,
    budget], the kept keys' old indices with -1 past the last, and the new
    lengths int32 [B]).  The call needs no workspace; `ws` is accepted as by the
    other calls and left alone."""
    lay = _caches(k_cache, v_cache, "k_cache", "v_cache")
    dlay = _caches(dst_k, dst_v, "dst_k", "dst_v")
    if table.dim() != 2 or dst_table.dim() != 2 or dst_table.shape[0] != table.shape[0]:
        raise ValueError("table and dst_table must be [B, pages per sequence]")
    B, H = table.shape[0], lay.kv_heads
    if keep is None:
        keep = _new((B, H, budget), torch.int32, mass.device, stream)
    if dst_lens is None:
        dst_lens = _new(B, torch.int32, mass.device, stream)
    _covers(mass=(mass, lay.pages * H * lay.page_size), lens=(lens, B), keep=(keep, B * H * budget),
            dst_mass=(dst_mass, dlay.pages * dlay.kv_heads * dlay.page_size), dst_lens=(dst_lens, B))
    _here("k_cache v_cache mass table lens dst_k dst_v dst_mass dst_table keep dst_lens",
          k_cache, v_cache, mass, table, lens, dst_k, dst_v, dst_mass, dst_table, keep, dst_lens)
    _check("tern_cache_evict", lib().tern_cache_evict(
        k_cache.data_ptr(), v_cache.data_ptr(), ctypes.addressof(lay), _dev(mass, torch.float32, "mass"),
        _dev(table, torch.int32, "table"), table.shape[1], _dev(lens, torch.int32, "lens"), B, budget, recent,
        dst_k.data_ptr(), dst_v.data_ptr(), ctypes.addressof(dlay), _dev(dst_mass, torch.float32, "dst_mass"),
        _dev(dst_table, torch.int32, "dst_table"), dst_table.shape[1], _dev(keep, torch.int32, "keep"),
        _dev(dst_lens, torch.int32, "dst_lens"), _stream(stream)))
    return keep, dst_lens
