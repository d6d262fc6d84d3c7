"""Python binding of the gfx950 RHT + lattice + bit-strip + Rice codec (``libhq.so``).

Argument marshalling only: every step of the method runs in the HIP kernels behind the C ABI
declared in ``include/hq.h``.  PyTorch provides device memory and the stream.  There is no CPU
fallback: if the library is missing the calls raise.

Entry points mirror the C ABI: ``hq_encode``, ``hq_decode``, ``hq_rate``, ``hq_codes``,
``hq_status``, ``hq_fallbacks``, ``hq_workspace_size``, ``hq_stream_fixed_bytes``, ``hq_encode_bound``,
``hq_version``, ``hq_strerror``; the paged SRFT cache: ``hq_kv_cache``, ``hq_kv_append``, ``hq_kv_read``,
``hq_kv_attend``, ``hq_kv_evict``.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhq.so")

HQ_OK, HQ_ERR_INVALID_ARG, HQ_ERR_UNSUPPORTED, HQ_ERR_NONFINITE = 0, -1, -2, -3
HQ_ERR_CAPACITY, HQ_ERR_CORRUPT, HQ_ERR_RATE, HQ_ERR_HIP, HQ_ERR_TIMEOUT, HQ_ERR_SCRATCH = -4, -5, -6, -7, -8, -9
HQ_Z, HQ_D4, HQ_E8, HQ_A2 = 0, 1, 2, 3
HQ_F32, HQ_BF16 = 0, 1
LATTICES = {"z": HQ_Z, "d4": HQ_D4, "e8": HQ_E8, "a2": HQ_A2}

EXPORTS = ("hq_version", "hq_strerror", "hq_workspace_size", "hq_stream_fixed_bytes", "hq_encode_bound", "hq_rate",
           "hq_encode", "hq_encode_noalloc", "hq_decode", "hq_status", "hq_fallbacks", "hq_codes",
           "hq_gemv_workspace_size", "hq_gemv",
           "hq_haar_matrix", "hq_rotate", "hq_srft_encode", "hq_srft_decode",
           "hq_kv_append", "hq_kv_read", "hq_kv_attend_workspace_size", "hq_kv_attend", "hq_kv_evict")


class HqParams(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_uint32), ("lattice", ctypes.c_int32), ("target_bps", ctypes.c_float),
                ("seed", ctypes.c_uint64), ("dither", ctypes.c_uint32), ("step", ctypes.c_float),
                ("rice_k", ctypes.c_int32)]


class HqInfo(ctypes.Structure):
    _fields_ = [("step", ctypes.c_float), ("rice_k", ctypes.c_int32), ("bytes", ctypes.c_uint64),
                ("payload_bits", ctypes.c_uint64), ("payload_bps", ctypes.c_double),
                ("side_bps", ctypes.c_double), ("total_bps", ctypes.c_double)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class HqKvCache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("pages", ctypes.c_uint32), ("heads", ctypes.c_uint32),
                ("page", ctypes.c_uint32), ("bits", ctypes.c_int32), ("seed", ctypes.c_uint64),
                ("lambda_k", ctypes.c_void_p), ("lambda_v", ctypes.c_void_p)]


class HqKvAttendArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("q_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("q_stride_token", ctypes.c_int64), ("q_stride_head", ctypes.c_int64), ("total_q", ctypes.c_uint64),
                ("q_heads", ctypes.c_uint32), ("seqs", ctypes.c_uint32), ("max_q", ctypes.c_uint32), ("max_len", ctypes.c_uint32),
                ("q_start", ctypes.c_void_p), ("table", ctypes.c_void_p), ("table_width", ctypes.c_uint32),
                ("lens", ctypes.c_void_p), ("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("causal", ctypes.c_int32),
                ("window", ctypes.c_uint32), ("weights", ctypes.c_void_p), ("weights_stride", ctypes.c_uint64)]


class HqKvEvictArgs(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("weights", ctypes.c_void_p),
                ("weights_stride", ctypes.c_uint64), ("seqs", ctypes.c_uint32), ("table_width", ctypes.c_uint32),
                ("max_len", ctypes.c_uint32), ("budget", ctypes.c_uint32), ("sink", ctypes.c_uint32), ("recent", ctypes.c_uint32),
                ("dst_table", ctypes.c_void_p), ("dst_width", ctypes.c_uint32), ("kept", ctypes.c_void_p),
                ("new_lens", ctypes.c_void_p), ("new_weights", ctypes.c_void_p)]


class HqError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} ({code})")
        self.code = code


_lib = None


def lib():
    """Load ``libhq.so`` (built in-tree by ``kv_quantization_tile_amd/build.py``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with kv_quantization_tile_amd/build.py")
        L = ctypes.CDLL(LIB_PATH)
        P, u64, i32, sz = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int32, ctypes.c_size_t
        L.hq_version.restype = ctypes.c_uint32
        L.hq_strerror.argtypes = [ctypes.c_int]
        L.hq_strerror.restype = ctypes.c_char_p
        L.hq_workspace_size.argtypes = [u64, P, ctypes.POINTER(sz)]
        L.hq_stream_fixed_bytes.argtypes = [u64, i32, i32, ctypes.c_uint32, ctypes.POINTER(u64)]
        L.hq_encode_bound.argtypes = [u64, P, ctypes.POINTER(u64)]
        L.hq_rate.argtypes = [P, i32, u64, P, P, P, sz, P]
        L.hq_encode.argtypes = [P, i32, u64, P, P, u64, P, P, P, sz, P]
        L.hq_encode_noalloc.argtypes = [P, i32, u64, P, P, u64, P, P, P]
        L.hq_decode.argtypes = [P, u64, P, i32, u64, P, sz, P]
        L.hq_status.argtypes = [P, P]
        L.hq_fallbacks.argtypes = [P, P, ctypes.POINTER(ctypes.c_uint32)]
        L.hq_codes.argtypes = [P, i32, u64, P, P, P, P, sz, P]
        L.hq_gemv_workspace_size.argtypes = [u64, u64, ctypes.POINTER(sz)]
        L.hq_gemv.argtypes = [P, u64, u64, u64, P, i32, P, P, sz, P]
        L.hq_haar_matrix.argtypes = [u64, P]
        L.hq_rotate.argtypes = [P, u64, P, i32, P, P]
        L.hq_srft_encode.argtypes = [P, i32, u64, u64, P, i32, P, P, P]
        L.hq_srft_decode.argtypes = [P, P, u64, u64, P, i32, P, i32, P]
        L.hq_kv_append.argtypes = [P, P, P, i32, u64, P, P, P]
        L.hq_kv_read.argtypes = [P, P, u64, P, P, i32, P]
        L.hq_kv_attend_workspace_size.argtypes = [P, P, ctypes.POINTER(sz)]
        L.hq_kv_attend.argtypes = [P, P, P, sz, P]
        L.hq_kv_evict.argtypes = [P, P, P]
        for name in EXPORTS:
            getattr(L, name).restype = getattr(L, name).restype or ctypes.c_int
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().hq_strerror(code).decode()


def hq_version() -> int:
    return int(lib().hq_version())


def _check(rc: int, what: str):
    if rc != HQ_OK:
        raise HqError(rc, what)


# Dither flags: bit 0 on; bit 1 the dither's Philox calls take 7 rounds instead of 10; bit 2 a
# 24-bit draw instead of 16.  True / False mean 1 / 0.
HQ_DITHER, HQ_DITHER_PHILOX7, HQ_DITHER_24BIT = 1, 2, 4


def dither_flags(dither) -> int:
    return (1 if dither else 0) if isinstance(dither, bool) else int(dither)


def make_params(lattice="e8", target_bps=4.0, seed=0, dither=False, step=0.0, rice_k=-1, tile=128) -> HqParams:
    lat = LATTICES[lattice] if isinstance(lattice, str) else int(lattice)
    return HqParams(tile=tile, lattice=lat, target_bps=float(target_bps), seed=int(seed),
                    dither=dither_flags(dither), step=float(step), rice_k=int(rice_k))


def hq_workspace_size(n: int, params: HqParams | None = None) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().hq_workspace_size(n, ctypes.byref(params) if params else None, ctypes.byref(out)),
           "hq_workspace_size")
    return out.value


def hq_stream_fixed_bytes(n: int, lattice, rice_k: int, tile: int = 128) -> int:
    out = ctypes.c_uint64(0)
    lat = LATTICES[lattice] if isinstance(lattice, str) else int(lattice)
    _check(lib().hq_stream_fixed_bytes(n, lat, rice_k, tile, ctypes.byref(out)), "hq_stream_fixed_bytes")
    return out.value


def hq_encode_bound(n: int, lattice="e8", step=0.0, rice_k=-1, dither=False, tile=128) -> int:
    """Worst-case stream bytes of an encode of n values (host only; see include/hq.h)."""
    out = ctypes.c_uint64(0)
    p = make_params(lattice, 4.0, 0, dither, step, rice_k, tile)
    _check(lib().hq_encode_bound(n, ctypes.byref(p), ctypes.byref(out)), "hq_encode_bound")
    return out.value


# ---- torch-side helpers (device memory and streams only) ------------------------------------------

def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return HQ_F32
    if t.dtype == torch.bfloat16:
        return HQ_BF16
    raise TypeError("input must be float32 or bfloat16")


def _stream_handle(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def workspace(n: int, device="cuda"):
    torch = _torch()
    return torch.empty(hq_workspace_size(n), dtype=torch.uint8, device=device)


def capacity_estimate(n: int, lattice, target_bps: float, rice_k: int = -1, step: float = 0.0,
                      tile: int = 128) -> int:
    """A starting output size: the fixed plane at a generous Rice k plus 4 unary bits per value."""
    if rice_k >= 0:
        k = rice_k
    elif step > 0:
        k = 15
    else:
        k = min(15, int(target_bps) + 3)
    return hq_stream_fixed_bytes(n, lattice, k, tile) + n // 2 + 4096


def hq_encode(x, lattice="e8", target_bps=4.0, seed=0, dither=False, step=0.0, rice_k=-1, out=None,
              ws=None, stream=None, blocking=True, tile=128):
    """Encode a contiguous CUDA tensor (fp32 or bf16, numel a multiple of the tile length 64, 128
    or 256).

    Returns (stream bytes as a uint8 CUDA tensor, info dict).  With blocking=False the call only
    enqueues work and returns (out, None); the size is then in the stream header.  Without `out`,
    the asynchronous call sizes the buffer with hq_encode_bound: at the given step (step > 0), or,
    with rate control (step == 0), at the operating point of a blocking hq_rate on the workspace,
    which the asynchronous encode then uses (step == -1)."""
    torch = _torch()
    assert x.is_cuda and x.is_contiguous()
    n = x.numel()
    p = make_params(lattice, target_bps, seed, dither, step, rice_k, tile)
    if ws is None:
        ws = workspace(n, x.device)
    sh = _stream_handle(stream)
    if out is None and not blocking:
        if step > 0:
            cap = hq_encode_bound(n, p.lattice, step, rice_k, p.dither, tile)
        elif step == 0:
            point = hq_rate(x, lattice, target_bps, seed, dither, 0.0, rice_k, ws=ws, stream=stream, tile=tile)
            cap = hq_encode_bound(n, p.lattice, point["step"], point["rice_k"], p.dither, tile)
            p = make_params(lattice, target_bps, seed, dither, -1.0, rice_k, tile)
        else:
            raise ValueError("an asynchronous encode at the workspace's operating point (step=-1) needs `out`")
        out = torch.empty(cap, dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty(capacity_estimate(n, p.lattice, target_bps, rice_k, step, tile), dtype=torch.uint8,
                          device=x.device)
    assert out.is_cuda and out.is_contiguous() and out.dtype == torch.uint8
    if not blocking:
        _check(lib().hq_encode(ctypes.c_void_p(x.data_ptr()), _dtype_code(x), n, ctypes.byref(p),
                               ctypes.c_void_p(out.data_ptr()), out.numel(), None, None,
                               ctypes.c_void_p(ws.data_ptr()), ws.numel(), sh), "hq_encode")
        return out, None
    info = HqInfo()
    nbytes = ctypes.c_uint64(0)
    while True:
        rc = lib().hq_encode(ctypes.c_void_p(x.data_ptr()), _dtype_code(x), n, ctypes.byref(p),
                             ctypes.c_void_p(out.data_ptr()), out.numel(), ctypes.byref(nbytes),
                             ctypes.byref(info), ctypes.c_void_p(ws.data_ptr()), ws.numel(), sh)
        if rc == HQ_ERR_CAPACITY and nbytes.value > out.numel():
            out = torch.empty(nbytes.value, dtype=torch.uint8, device=x.device)
            continue
        _check(rc, "hq_encode")
        break
    return out[: nbytes.value], info.as_dict()


def hq_decode(stream_bytes, n: int, out_dtype=None, out=None, ws=None, stream=None, check=True):
    """Decode a uint8 CUDA tensor holding a stream into n values (bf16 by default)."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    assert stream_bytes.is_cuda and stream_bytes.is_contiguous() and stream_bytes.dtype == torch.uint8
    if out is None:
        out = torch.empty(n, dtype=out_dtype, device=stream_bytes.device)
    # the kernels write n values of out's type: a shorter or strided tensor would be written past
    assert out.is_cuda and out.is_contiguous() and out.numel() >= n, "out must be a contiguous CUDA tensor of n values"
    assert out.dtype in (torch.float32, torch.bfloat16), "out must be float32 or bfloat16"
    if ws is None:
        ws = workspace(0, stream_bytes.device)
    sh = _stream_handle(stream)
    _check(lib().hq_decode(ctypes.c_void_p(stream_bytes.data_ptr()), stream_bytes.numel(),
                           ctypes.c_void_p(out.data_ptr()), _dtype_code(out), n,
                           ctypes.c_void_p(ws.data_ptr()), ws.numel(), sh), "hq_decode")
    if check:
        _check(lib().hq_status(ctypes.c_void_p(ws.data_ptr()), sh), "hq_decode")
    return out


def hq_gemv_workspace_size(rows: int, cols: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().hq_gemv_workspace_size(rows, cols, ctypes.byref(out)), "hq_gemv_workspace_size")
    return out.value


def hq_gemv(stream_bytes, rows: int, cols: int, x, y=None, ws=None, stream=None, check=True):
    """y = W_hat x for a stream of a [rows][cols] matrix: fused decode + matrix-vector product
    (float32 output)."""
    torch = _torch()
    assert x.is_cuda and x.is_contiguous() and x.numel() == cols
    assert stream_bytes.is_cuda and stream_bytes.is_contiguous() and stream_bytes.dtype == torch.uint8
    if y is None:
        y = torch.empty(rows, dtype=torch.float32, device=x.device)
    # the kernels write `rows` binary32 values
    assert y.is_cuda and y.is_contiguous() and y.dtype == torch.float32 and y.numel() >= rows, \
        "y must be a contiguous float32 CUDA tensor of `rows` values"
    if ws is None:
        ws = torch.empty(hq_gemv_workspace_size(rows, cols), dtype=torch.uint8, device=x.device)
    sh = _stream_handle(stream)
    _check(lib().hq_gemv(ctypes.c_void_p(stream_bytes.data_ptr()), stream_bytes.numel(), rows, cols,
                         ctypes.c_void_p(x.data_ptr()), _dtype_code(x), ctypes.c_void_p(y.data_ptr()),
                         ctypes.c_void_p(ws.data_ptr()), ws.numel(), sh), "hq_gemv")
    if check:
        _check(lib().hq_status(ctypes.c_void_p(ws.data_ptr()), sh), "hq_gemv")
    return y


def hq_haar_matrix(seed: int):
    """The per-layer Haar-uniform rotation Q of a seed, as a float32 numpy array [128, 128]."""
    import numpy as np
    q = np.zeros(128 * 128, dtype=np.float32)
    _check(lib().hq_haar_matrix(seed, ctypes.c_void_p(q.ctypes.data)), "hq_haar_matrix")
    return q.reshape(128, 128)


def hq_rotate(x, q, transpose: bool = False, out=None, stream=None):
    """y_v = Q x_v (or Q^T x_v) for the 128-value bf16 vectors of x; q a float32 CUDA tensor [128, 128]."""
    torch = _torch()
    assert x.is_cuda and x.is_contiguous() and x.dtype == torch.bfloat16
    assert q.is_cuda and q.is_contiguous() and q.dtype == torch.float32 and q.numel() == 128 * 128
    if out is None:
        out = torch.empty_like(x)
    assert out.is_cuda and out.is_contiguous() and out.dtype == torch.bfloat16 and out.numel() >= x.numel()
    _check(lib().hq_rotate(ctypes.c_void_p(x.data_ptr()), x.numel(), ctypes.c_void_p(q.data_ptr()),
                           1 if transpose else 0, ctypes.c_void_p(out.data_ptr()), _stream_handle(stream)),
           "hq_rotate")
    return out


def _host_lambda(lam):
    import numpy as np
    if lam is None:
        return None, None
    a = np.ascontiguousarray(np.asarray(lam, dtype=np.float32).reshape(-1))
    if a.size != 128:
        raise ValueError("lambda holds one scale per coordinate: 128 values")
    return a, ctypes.c_void_p(a.ctypes.data)


def hq_srft_encode(x, seed: int = 0, bits: int = 4, lam=None, codes=None, scales=None, stream=None):
    """SRFT fixed-rate codes of x (bf16 or float32 CUDA tensor, numel % 128 == 0): returns (codes
    uint8 [vectors][64 | 128], scales int16 view of binary16 [vectors][16]).  lam: 128 host floats."""
    torch = _torch()
    assert x.is_cuda and x.is_contiguous()
    n = x.numel()
    nv = n // 128
    if codes is None:
        codes = torch.empty((nv, 64 if bits == 4 else 128), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((nv, 16), dtype=torch.int16, device=x.device)
    assert codes.is_cuda and codes.is_contiguous() and codes.numel() * codes.element_size() >= nv * (64 if bits == 4 else 128)
    assert scales.is_cuda and scales.is_contiguous() and scales.numel() * scales.element_size() >= nv * 32
    keep, lp = _host_lambda(lam)
    _check(lib().hq_srft_encode(ctypes.c_void_p(x.data_ptr()), _dtype_code(x), n, int(seed), lp, int(bits),
                                ctypes.c_void_p(codes.data_ptr()), ctypes.c_void_p(scales.data_ptr()),
                                _stream_handle(stream)), "hq_srft_encode")
    return codes, scales


def hq_srft_decode(codes, scales, n: int, seed: int = 0, bits: int = 4, lam=None, out=None,
                   out_dtype=None, stream=None):
    """Decode n values from SRFT codes and scales (CUDA tensors) into bf16 (default) or float32."""
    torch = _torch()
    assert codes.is_cuda and scales.is_cuda and codes.is_contiguous() and scales.is_contiguous()
    if out is None:
        out = torch.empty(n, dtype=out_dtype or torch.bfloat16, device=codes.device)
    assert out.is_cuda and out.is_contiguous() and out.numel() >= n and out.dtype in (torch.float32, torch.bfloat16)
    keep, lp = _host_lambda(lam)
    _check(lib().hq_srft_decode(ctypes.c_void_p(codes.data_ptr()), ctypes.c_void_p(scales.data_ptr()), n,
                                int(seed), lp, int(bits), ctypes.c_void_p(out.data_ptr()), _dtype_code(out),
                                _stream_handle(stream)), "hq_srft_decode")
    return out


# ---- the paged SRFT cache (for inference: no gradient passes through these calls) --------------------

def hq_kv_token_bytes(bits: int = 4) -> int:
    """Bytes of one token of one head, K and V."""
    return 2 * (16 * bits + 32)


def hq_kv_cache(pages: int, heads: int, page: int = 64, bits: int = 4, device="cuda"):
    """A layer's empty paged cache: uint8 [pages][heads][page bytes] (layout in include/hq.h)."""
    torch = _torch()
    if bits not in (4, 8) or page < 16 or page > 4096 or page & (page - 1):
        raise ValueError("bits is 4 or 8, page a power of two from 16 to 4096")
    return torch.zeros(pages, heads, page * hq_kv_token_bytes(bits), dtype=torch.uint8, device=device)


def _cache_arg(cache, bits, seed, lam_k, lam_v):
    """The C description of a cache tensor, and what has to outlive the call."""
    if cache.dtype != _torch().uint8 or cache.dim() != 3 or not (cache.is_cuda and cache.is_contiguous()):
        raise TypeError("cache must be a contiguous uint8 CUDA tensor [pages][heads][page bytes]")
    if bits != 4 and bits != 8:
        raise ValueError("bits is 4 or 8")
    pages, heads, size = cache.shape
    page, rest = divmod(size, 2 * (16 * bits + 32))
    if rest:
        raise ValueError("the cache's last dimension is not a whole number of tokens at these bits")
    if lam_k is None and lam_v is None:
        return HqKvCache(cache.data_ptr(), pages, heads, page, bits, seed, None, None), None
    keep_k, pk = _host_lambda(lam_k)
    keep_v, pv = _host_lambda(lam_v)
    return HqKvCache(cache.data_ptr(), pages, heads, page, bits, seed, pk, pv), (keep_k, keep_v)


def _check_tensor(t, name, dtype, shape, device):
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _size(v, name: str) -> int:
    if not 0 <= v <= 0xFFFFFFFF:
        raise ValueError(f"{name} must be a 32-bit size, not {v}")
    return v


def _empty(shape, dtype, device, stream):
    """A buffer of the call's own, from the pool of the stream the call runs on."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _launch(what, device, stream, call, *args):
    """Calls `call`(*args, stream's handle) with `device` current: the handle of `stream`, or of the device's current stream
    (without the Stream object, which takes 3 us to make)."""
    torch = _torch()
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device.index)
    elif stream.device == device:
        handle = stream.cuda_stream
    else:
        raise ValueError(f"{what}: the stream is on {stream.device}, the cache on {device}")
    if torch.cuda.current_device() == device.index:
        _check(call(*args, handle), what)
    else:
        with torch.cuda.device(device):
            _check(call(*args, handle), what)


def _row_strides(t, name, heads, device):
    """Token and head strides of t [tokens][heads][128] (heads None: any)."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != 128 or (heads is not None and shape[1] != heads) or t.device != device or (strides[2] != 1 and shape[0]):
        raise ValueError(f"{name} must be [tokens][{heads or 'heads'}][128] on {device}, its last dimension contiguous")
    return strides


_Strides4 = ctypes.c_int64 * 4


def hq_kv_append(cache, k, v, slots, bits: int = 4, seed: int = 0, lam_k=None, lam_v=None, stream=None):
    """Encode K and V of new tokens ([tokens][heads][128] bf16 or float32, any token and head strides) into
    their slots (int64 [tokens]: page * P + offset; a slot outside the cache, -1 say, writes nothing)."""
    c, keep = _cache_arg(cache, bits, seed, lam_k, lam_v)
    dev, tokens = cache.device, k.shape[0]
    ks, vs = _row_strides(k, "k", c.heads, dev), _row_strides(v, "v", c.heads, dev)
    if k.dtype != v.dtype or v.shape[0] != tokens:
        raise ValueError("k and v must have one type and length")
    _check_tensor(slots, "slots", _torch().int64, (tokens,), dev)
    _launch("hq_kv_append", dev, stream, lib().hq_kv_append, ctypes.byref(c), k.data_ptr(), v.data_ptr(), _dtype_code(k), tokens,
            _Strides4(ks[0], ks[1], vs[0], vs[1]), slots.data_ptr())
    return cache


def hq_kv_read(cache, slots, bits: int = 4, seed: int = 0, lam_k=None, lam_v=None, out_dtype=None, k=None, v=None,
               stream=None):
    """Decode slots (int64 [tokens]) into (k, v), each [tokens][heads][128] bf16 (default) or float32; a slot
    outside the cache reads as zeros."""
    torch = _torch()
    c, keep = _cache_arg(cache, bits, seed, lam_k, lam_v)
    dev, tokens = cache.device, slots.numel()
    _check_tensor(slots, "slots", torch.int64, (tokens,), dev)
    shape, dt = (tokens, c.heads, 128), out_dtype or torch.bfloat16
    if k is None:
        k = _empty(shape, dt, dev, stream)
    else:
        _check_tensor(k, "k", dt, shape, dev)
    if v is None:
        v = _empty(shape, dt, dev, stream)
    else:
        _check_tensor(v, "v", dt, shape, dev)
    _launch("hq_kv_read", dev, stream, lib().hq_kv_read, ctypes.byref(c), slots.data_ptr(), tokens, k.data_ptr(), v.data_ptr(), _dtype_code(k))
    return k, v


def hq_kv_attend(cache, q, table, lens, q_start=None, max_q=None, max_len=None, bits: int = 4, seed: int = 0, lam_k=None,
                 lam_v=None, scale=None, causal: bool = True, window: int = 0, softcap: float = 0.0, weights=None, out=None,
                 ws=None, stream=None):
    """Softmax attention of q ([queries][q heads][128] bf16 or float32, any strides but the last) over the cache.

    table int32 [seqs][width], lens int32 [seqs] (tokens cached, the queries' own among them); q_start int32
    [seqs + 1] offsets of each sequence's queries (None: as many each); max_q, max_len bounds on a sequence's
    queries and tokens (None: all queries, what the table's width or the weights hold): further queries are not computed,
    and a longer length counts as max_len.  weights float32
    [seqs][heads][>= max_len] gets each token's softmax weights added (and has the scores computed in two parts, so out may
    differ in its last bits).  Returns out ([queries][q heads][128], bf16 unless given)."""
    torch = _torch()
    c, keep = _cache_arg(cache, bits, seed, lam_k, lam_v)
    dev = cache.device
    strides = _row_strides(q, "q", None, dev)
    total, heads, _ = q.shape
    if heads == 0 or heads % c.heads:
        raise ValueError("q must be [queries][q heads][128], q heads a multiple of the cache's heads")
    seqs, width = lens.numel(), table.shape[-1]
    _check_tensor(lens, "lens", torch.int32, (seqs,), dev)
    _check_tensor(table, "table", torch.int32, (seqs, width), dev)
    if q_start is not None:
        _check_tensor(q_start, "q_start", torch.int32, (seqs + 1,), dev)
    if max_q is None:
        max_q = total if q_start is not None else total // max(seqs, 1)
    if out is None:
        out = _empty((total, heads, 128), torch.bfloat16, dev, stream)
    else:
        _check_tensor(out, "out", out.dtype, (total, heads, 128), dev)
    stride = 0
    if weights is not None:
        if weights.dim() != 3:
            raise ValueError("weights must be [seqs][heads][tokens]")
        stride = weights.shape[2]
        _check_tensor(weights, "weights", torch.float32, (seqs, c.heads, stride), dev)
    if max_len is None:
        max_len = width * c.page if weights is None else min(stride, width * c.page)
    a = HqKvAttendArgs(q.data_ptr(), out.data_ptr(), _dtype_code(q), _dtype_code(out), strides[0], strides[1], total, heads, seqs,
                       _size(max_q, "max_q"), _size(max_len, "max_len"), q_start.data_ptr() if q_start is not None else None,
                       table.data_ptr(), width, lens.data_ptr(), 128 ** -0.5 if scale is None else scale, softcap, 1 if causal else 0,
                       _size(window, "window"), weights.data_ptr() if weights is not None else None, stride)
    L, cp, ap = lib(), ctypes.byref(c), ctypes.byref(a)
    if ws is None:
        need = ctypes.c_size_t()
        _check(L.hq_kv_attend_workspace_size(cp, ap, ctypes.byref(need)), "hq_kv_attend")
        ws = _empty(need.value, torch.uint8, dev, stream)
    elif not (ws.is_contiguous() and ws.device == dev and ws.dtype == torch.uint8):
        raise ValueError(f"ws must be a contiguous uint8 tensor on {dev}")
    _launch("hq_kv_attend", dev, stream, L.hq_kv_attend, cp, ap, ws.data_ptr(), ws.numel())
    return out


def hq_kv_evict(cache, table, lens, weights, budget: int, sink: int, recent: int, dst_table, bits: int = 4, max_len=None,
                kept=None, new_lens=None, new_weights=None, stream=None):
    """Keep, of each (sequence, head)'s tokens, at most `budget`: the first `sink`, the last `recent`, and the
    others of most weight (ties to the lowest index), moved in order into the pages of dst_table (int32 [seqs][width],
    none of them in `table`).  max_len bounds a sequence's tokens (None: what the table's width and the weights hold);
    tokens past it are not kept, so weights has to reach over every length.  Returns (kept int32 [seqs][heads][budget], -1 past the end; new_lens int32 [seqs];
    new_weights float32 [seqs][heads][budget])."""
    torch = _torch()
    c, _ = _cache_arg(cache, bits, 0, None, None)
    dev, heads, seqs, width, dst_width, top = cache.device, c.heads, lens.numel(), table.shape[-1], dst_table.shape[-1], weights.shape[-1]
    _check_tensor(lens, "lens", torch.int32, (seqs,), dev)
    _check_tensor(table, "table", torch.int32, (seqs, width), dev)
    _check_tensor(weights, "weights", torch.float32, (seqs, heads, top), dev)
    _check_tensor(dst_table, "dst_table", torch.int32, (seqs, dst_width), dev)
    shape = (seqs, heads, _size(budget, "budget"))
    if budget > dst_width * c.page:
        raise ValueError("budget is more than dst_table's pages hold")
    if kept is None:
        kept = _empty(shape, torch.int32, dev, stream)
    else:
        _check_tensor(kept, "kept", torch.int32, shape, dev)
    if new_lens is None:
        new_lens = _empty((seqs,), torch.int32, dev, stream)
    else:
        _check_tensor(new_lens, "new_lens", torch.int32, (seqs,), dev)
    if new_weights is None:
        new_weights = _empty(shape, torch.float32, dev, stream)
    else:
        _check_tensor(new_weights, "new_weights", torch.float32, shape, dev)
    a = HqKvEvictArgs(table.data_ptr(), lens.data_ptr(), weights.data_ptr(), top, seqs, width,
                      min(top, width * c.page) if max_len is None else _size(max_len, "max_len"), budget, _size(sink, "sink"),
                      _size(recent, "recent"), dst_table.data_ptr(), dst_width, kept.data_ptr(), new_lens.data_ptr(),
                      new_weights.data_ptr())
    _launch("hq_kv_evict", dev, stream, lib().hq_kv_evict, ctypes.byref(c), ctypes.byref(a))
    return kept, new_lens, new_weights


def hq_rate(x, lattice="e8", target_bps=4.0, seed=0, dither=False, step=0.0, rice_k=-1, ws=None, stream=None,
            blocking=True, tile=128):
    """Rate control alone.  blocking=False only enqueues it; a following hq_encode(..., step=-1,
    ws=<same workspace>) then encodes at the chosen operating point."""
    assert x.is_cuda and x.is_contiguous()
    n = x.numel()
    p = make_params(lattice, target_bps, seed, dither, step, rice_k, tile)
    if ws is None:
        ws = workspace(n, x.device)
    info = HqInfo()
    _check(lib().hq_rate(ctypes.c_void_p(x.data_ptr()), _dtype_code(x), n, ctypes.byref(p),
                         ctypes.byref(info) if blocking else None, ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                         _stream_handle(stream)), "hq_rate")
    return info.as_dict() if blocking else None


def hq_codes(x, step: float, lattice="e8", seed=0, dither=False, ws=None, stream=None, tile=128):
    """Integer lattice codes (int32, per value) and bf16 tile-scale bits (int16 view, per tile)."""
    torch = _torch()
    assert x.is_cuda and x.is_contiguous()
    n = x.numel()
    p = make_params(lattice, 4.0, seed, dither, step, -1, tile)
    if ws is None:
        ws = workspace(0, x.device)
    codes = torch.empty(n, dtype=torch.int32, device=x.device)
    scales = torch.empty(max(n // tile, 1), dtype=torch.int16, device=x.device)
    sh = _stream_handle(stream)
    _check(lib().hq_codes(ctypes.c_void_p(x.data_ptr()), _dtype_code(x), n, ctypes.byref(p),
                          ctypes.c_void_p(codes.data_ptr()), ctypes.c_void_p(scales.data_ptr()),
                          ctypes.c_void_p(ws.data_ptr()), ws.numel(), sh), "hq_codes")
    _check(lib().hq_status(ctypes.c_void_p(ws.data_ptr()), sh), "hq_codes")
    return codes, scales[: n // tile]


def hq_status(ws, stream=None) -> int:
    return int(lib().hq_status(ctypes.c_void_p(ws.data_ptr()), _stream_handle(stream)))


# bits of hq_fallbacks
FALLBACK_LOOKBACK, FALLBACK_CENTRE, FALLBACK_PRIVATE = 1, 2, 4


def hq_fallbacks(ws, stream=None) -> int:
    """Which bounded waits of the workspace's last call took their (slower, same-result) fallback:
    bit 0 a look-back aggregate, bit 1 pass A's centre, bit 2 a pass's private evaluation."""
    f = ctypes.c_uint32(0)
    _check(lib().hq_fallbacks(ctypes.c_void_p(ws.data_ptr()), _stream_handle(stream), ctypes.byref(f)),
           "hq_fallbacks")
    return int(f.value)


def header_fields(stream_bytes_host) -> dict:
    """Parse the 128-byte stream header (host bytes) into a dict."""
    import struct
    b = bytes(stream_bytes_host[:128])
    magic, ver, lat, flags, tile, k, clog, step_bits = struct.unpack_from("<IHBBHBBI", b, 0)
    seed, n, T = struct.unpack_from("<QQQ", b, 16)
    chunks, F = struct.unpack_from("<II", b, 40)
    fixed_off, unary_off, words, ubits, payload, total = struct.unpack_from("<QQQQQQ", b, 48)
    return dict(magic=magic, version=ver, lattice=lat, dither=flags, tile=tile, k=k, chunk_log2=clog,
                step_bits=step_bits, seed=seed, n=n, tiles=T, chunks=chunks, F=F, fixed_off=fixed_off,
                unary_off=unary_off, unary_words=words, unary_bits=ubits, payload_bits=payload,
                total_bytes=total)
