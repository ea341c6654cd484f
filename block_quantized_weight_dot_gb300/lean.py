"""ctypes binding of ``liblean_qmatmul.so`` (C ABI in ``include/lean_qmatmul.h``,
``include/lean_quant.h``, ``include/lean_step.h`` and ``include/lean_cache.h``).

Argument marshalling only: every computation of the product runs in the CUDA
library.  Functions keep the C names.  Buffers may be given as torch tensors
(their ``data_ptr()`` is passed), numpy arrays (host calls only) or raw integer
addresses.  A non-OK status raises :class:`LeanError`.  If the library has not
been built the import fails: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblean_qmatmul.so")
# the LEAN_DEBUG build of the same ABI (build.build(debug=True)): every kernel
# checks its global-memory indices; for test runs (open_library / use_library)
DEBUG_LIB_PATH = os.path.join(_HERE, "liblean_qmatmul_debug.so")

LEAN_Q4_0, LEAN_Q8_0, LEAN_I8_B64, LEAN_Q6_K = 0, 1, 2, 3
(LEAN_OK, LEAN_ERR_FORMAT, LEAN_ERR_SHAPE, LEAN_ERR_NULL, LEAN_ERR_ALIGN, LEAN_ERR_CUDA,
 LEAN_ERR_KERNEL_BOUNDS, LEAN_ERR_DEVICE) = range(8)
LEAN_FLAG_EARLY_WEIGHTS = 1
LEAN_FLAG_X_PLANES = 2
LEAN_FLAG_STREAM = 4
LEAN_FLAG_X_INT8 = 8

LEAN_F32, LEAN_BF16, LEAN_F16, LEAN_I8 = 0, 1, 2, 3
(LEAN_ROPE_PLAIN, LEAN_ROPE_LINEAR, LEAN_ROPE_BASE, LEAN_ROPE_RAMP, LEAN_ROPE_BANDS) = range(5)
LEAN_MAX_TOP = 64

# every symbol the headers declare, with (restype, argtypes)
_i64, _int, _vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
SIGNATURES = {
    "lean_block_elems": (_int, [_int]),
    "lean_block_bytes": (_i64, [_int]),
    "lean_canonical_bytes": (_i64, [_int, _i64, _i64]),
    "lean_packed_bytes": (_i64, [_int, _i64, _i64]),
    "lean_pack": (_int, [_int, _vp, _vp, _i64, _i64]),
    "lean_unpack_canonical": (_int, [_int, _vp, _vp, _i64, _i64]),
    "lean_dequant": (_int, [_int, _vp, _vp, _i64, _i64, _vp]),
    "lean_embed_rows": (_int, [_int, _vp, _vp, _vp, _i64, _i64, _i64, _vp]),
    "lean_qmatmul_swiglu": (_int, [_int, _vp, _vp, _vp, _vp, _i64, _i64, ctypes.c_uint, _vp]),
    "lean_qmatmul": (_int, [_int, _vp, _vp, _vp, _i64, _i64, _i64, _vp]),
    "lean_qmatmul_ex": (_int, [_int, _vp, _vp, _vp, _i64, _i64, _i64, ctypes.c_uint, _vp]),
    "lean_qmatmul_workspace_bytes": (_i64, [_int, _i64, _i64, _i64]),
    "lean_tensor_core_min_m": (_int, [_int]),
    "lean_qmatmul_ws": (_int, [_int, _vp, _vp, _vp, _i64, _i64, _i64, ctypes.c_uint, _vp, _i64,
                               _vp]),
    "lean_batch_workspace_bytes": (_i64, [_int, _int, _vp]),
    "lean_qmatmul_batch": (_int, [_int, _int, _vp, ctypes.c_uint, _vp, _i64, _vp]),
    "lean_device_error": (ctypes.c_uint, [_int]),
    "lean_device_status": (_int, [_int]),
    "lean_debug_build": (_int, []),
    "lean_wait_selftest": (_int, [ctypes.c_uint, _vp]),
    "lean_quantize": (_int, [_int, _vp, _vp, _i64, _i64, _int]),
    "lean_qmatmul_fixed_ws": (_int, [_int, _vp, _vp, _vp, _i64, _i64, ctypes.c_uint, _vp]),
    "lean_fixed_workspace_bytes": (_i64, []),
    "lean_status_str": (ctypes.c_char_p, [_int]),
    "lean_residual_norm": (_int, [_vp, _vp]),
    "lean_rope_turns": (_int, [_vp, _i64, _vp]),
    "lean_rope_frequencies": (_int, [_int, _i64] + [ctypes.c_double] * 5 + [_vp]),
    "lean_rope_append": (_int, [_vp, _vp]),
    "lean_kv_pages": (_int, [_vp, _vp]),
    "lean_kv_read": (_int, [_vp, _vp]),
    "lean_paged_attention": (_int, [_vp, _vp]),
    "lean_paged_attention_workspace_bytes": (_i64, [_i64] * 4),
    "lean_prefix_attention": (_int, [_vp, _vp]),
    "lean_prefix_attention_workspace_bytes": (_i64, [_i64] * 5),
    "lean_token_logprobs": (_int, [_vp, _vp]),
    "lean_token_logprobs_workspace_bytes": (_i64, [_i64] * 3),
}
LEAN_MAX_BATCH = 256


class lean_problem(ctypes.Structure):
    """One product of a batch: device pointers and its shape (C struct lean_problem)."""
    _fields_ = [("W", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class LeanError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (fn, status_str(status), status))


def open_library(path: str):
    """A ctypes handle on a build of this ABI (the product library or its
    LEAN_DEBUG build), with every declared signature set."""
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("liblean_qmatmul.so is not built: run "
                          "`python -c \"import __graft_entry__ as g; g.build()\"`")
    return open_library(LIB_PATH)


_lib = _load()


def use_library(lib):
    """Route every call of this module through `lib` (a handle from
    open_library); returns the handle used until now."""
    global _lib
    prev, _lib = _lib, lib
    return prev


def _addr(buf):
    """Address of a buffer: torch tensor, numpy array, int or None."""
    if buf is None:
        return None
    if isinstance(buf, int):
        return buf
    if isinstance(buf, np.ndarray):
        return buf.ctypes.data
    if hasattr(buf, "data_ptr"):
        return buf.data_ptr()
    raise TypeError("unsupported buffer type %r" % type(buf))


_raw_stream = None  # torch's current stream without the Stream object around it (0.2 us instead of 3.8)


def _stream(stream):
    global _raw_stream
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream()
        try:
            import torch
            if torch.cuda.is_available():
                st = torch.cuda.current_stream().cuda_stream
                c = torch._C
                if hasattr(c, "_cuda_getCurrentRawStream") and hasattr(c, "_cuda_getDevice"):
                    get, dev = c._cuda_getCurrentRawStream, c._cuda_getDevice
                    _raw_stream = lambda: get(dev())  # noqa: E731
                return st
        except ImportError:
            pass
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream  # torch.cuda.Stream


def _check(fn, status):
    if status != LEAN_OK:
        raise LeanError(fn, status)


def status_str(status: int) -> str:
    return _lib.lean_status_str(status).decode()


lean_status_str = status_str


def lean_block_elems(fmt: int) -> int:
    return _lib.lean_block_elems(fmt)


def lean_block_bytes(fmt: int) -> int:
    return _lib.lean_block_bytes(fmt)


def lean_canonical_bytes(fmt: int, N: int, K: int) -> int:
    return _lib.lean_canonical_bytes(fmt, N, K)


def lean_packed_bytes(fmt: int, N: int, K: int) -> int:
    return _lib.lean_packed_bytes(fmt, N, K)


def lean_pack(fmt: int, canon, N: int, K: int, packed=None) -> np.ndarray:
    """Canonical host bytes -> packed host bytes (a new uint8 array unless given)."""
    canon = np.ascontiguousarray(canon, dtype=np.uint8)
    nb = lean_packed_bytes(fmt, N, K)
    if nb < 0:
        raise LeanError("lean_pack", LEAN_ERR_SHAPE)
    if canon.size != lean_canonical_bytes(fmt, N, K):
        raise ValueError("canonical buffer has %d bytes, expected %d"
                         % (canon.size, lean_canonical_bytes(fmt, N, K)))
    if packed is None:
        packed = np.empty(nb, dtype=np.uint8)
    _check("lean_pack", _lib.lean_pack(fmt, _addr(canon), _addr(packed), N, K))
    return packed


def lean_unpack_canonical(fmt: int, packed, N: int, K: int) -> np.ndarray:
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    if packed.size != lean_packed_bytes(fmt, N, K):
        raise ValueError("packed buffer has the wrong size")
    canon = np.empty(lean_canonical_bytes(fmt, N, K), dtype=np.uint8)
    _check("lean_unpack_canonical", _lib.lean_unpack_canonical(fmt, _addr(packed), _addr(canon), N, K))
    return canon


def lean_dequant(fmt: int, W_packed_dev, w_dev, N: int, K: int, stream=None) -> None:
    _check("lean_dequant", _lib.lean_dequant(fmt, _addr(W_packed_dev), _addr(w_dev), N, K,
                                             _stream(stream)))


def lean_embed_rows(fmt: int, W_packed_dev, ids_dev, out_dev, n_ids: int, N: int, K: int,
                    stream=None) -> None:
    """out[i][k] = w[ids[i]][k] (an embedding lookup); ids: int32 device tensor."""
    _check("lean_embed_rows", _lib.lean_embed_rows(fmt, _addr(W_packed_dev), _addr(ids_dev),
                                                   _addr(out_dev), n_ids, N, K, _stream(stream)))


def lean_qmatmul_swiglu(fmt: int, W_gate_dev, W_up_dev, x_dev, h_dev, N: int, K: int,
                        flags: int = 0, stream=None) -> None:
    """h = silu(W_gate x) * (W_up x) in one launch (M = 1)."""
    _check("lean_qmatmul_swiglu", _lib.lean_qmatmul_swiglu(
        fmt, _addr(W_gate_dev), _addr(W_up_dev), _addr(x_dev), _addr(h_dev), N, K, flags,
        _stream(stream)))


def lean_qmatmul(fmt: int, W_packed_dev, x_dev, y_dev, N: int, K: int, M: int,
                 stream=None) -> None:
    """y[M][N] = x[M][K] . W[N][K]^T on the device, asynchronously on `stream`."""
    _check("lean_qmatmul", _lib.lean_qmatmul(fmt, _addr(W_packed_dev), _addr(x_dev),
                                             _addr(y_dev), N, K, M, _stream(stream)))


def lean_qmatmul_ex(fmt: int, W_packed_dev, x_dev, y_dev, N: int, K: int, M: int,
                    flags: int = 0, stream=None) -> None:
    """lean_qmatmul with launch flags (LEAN_FLAG_EARLY_WEIGHTS, LEAN_FLAG_X_PLANES)."""
    _check("lean_qmatmul_ex", _lib.lean_qmatmul_ex(fmt, _addr(W_packed_dev), _addr(x_dev),
                                                   _addr(y_dev), N, K, M, flags, _stream(stream)))


def lean_qmatmul_workspace_bytes(fmt: int, N: int, K: int, M: int) -> int:
    return _lib.lean_qmatmul_workspace_bytes(fmt, N, K, M)


def lean_tensor_core_min_m(fmt: int) -> int:
    """Rows of x from which the product of format fmt runs on the tensor cores."""
    return _lib.lean_tensor_core_min_m(fmt)


def lean_qmatmul_ws(fmt: int, W_packed_dev, x_dev, y_dev, N: int, K: int, M: int,
                    flags: int = 0, workspace=None, workspace_bytes: int = 0,
                    stream=None) -> None:
    """lean_qmatmul with flags and a caller-owned, once-zeroed device workspace."""
    _check("lean_qmatmul_ws", _lib.lean_qmatmul_ws(fmt, _addr(W_packed_dev), _addr(x_dev),
                                                   _addr(y_dev), N, K, M, flags,
                                                   _addr(workspace), workspace_bytes,
                                                   _stream(stream)))


def make_problems(items):
    """ctypes array of lean_problem from (W, x, y, N, K) tuples."""
    arr = (lean_problem * len(items))()
    for i, (W, x, y, N, K) in enumerate(items):
        arr[i] = lean_problem(_addr(W), _addr(x), _addr(y), N, K)
    return arr


def lean_batch_workspace_bytes(fmt: int, problems) -> int:
    return _lib.lean_batch_workspace_bytes(fmt, len(problems), ctypes.cast(problems, _vp))


def lean_qmatmul_batch(fmt: int, problems, flags: int = 0, workspace=None,
                       workspace_bytes: int = 0, stream=None) -> None:
    """Independent M = 1 products in one launch; `problems` from make_problems()."""
    _check("lean_qmatmul_batch", _lib.lean_qmatmul_batch(fmt, len(problems),
                                                         ctypes.cast(problems, _vp), flags,
                                                         _addr(workspace), workspace_bytes,
                                                         _stream(stream)))


def lean_qmatmul_fixed_ws(fmt: int, W_packed_dev, x_dev, y_dev, N: int, K: int, flags: int = 0,
                          stream=None) -> None:
    """M = 1 product whose scratch is the library's own fixed device array (no
    allocation by the caller; calls overlapping on the GPU must be serialised)."""
    _check("lean_qmatmul_fixed_ws", _lib.lean_qmatmul_fixed_ws(fmt, _addr(W_packed_dev),
                                                               _addr(x_dev), _addr(y_dev), N, K,
                                                               flags, _stream(stream)))


def lean_fixed_workspace_bytes() -> int:
    return _lib.lean_fixed_workspace_bytes()


def lean_device_error(clear: bool = True) -> int:
    """Device error word (non-zero: a kernel's bounded wait timed out)."""
    return _lib.lean_device_error(1 if clear else 0)


def lean_quantize(fmt: int, w, N: int, K: int, threads: int = 0):
    """Canonical blocks (uint8 array, ready for lean_pack) of fp32 w[N][K]
    quantized on the host to Q4_0, Q8_0 or I8_B64 (rule in lean_quant.h)."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    if w.size != N * K:
        raise ValueError("w has %d elements, expected %d" % (w.size, N * K))
    nbytes = lean_canonical_bytes(fmt, N, K)
    out = np.zeros(max(nbytes, 1), dtype=np.uint8)  # a bad shape is reported by the call
    _check("lean_quantize", _lib.lean_quantize(fmt, w.ctypes.data, out.ctypes.data, N, K,
                                                threads))
    return out[:nbytes]


def lean_device_status(clear: bool = True) -> int:
    """The device error word as a status (LEAN_OK, LEAN_ERR_KERNEL_BOUNDS,
    LEAN_ERR_DEVICE or LEAN_ERR_CUDA); returned, not raised."""
    return _lib.lean_device_status(1 if clear else 0)


def lean_debug_build() -> int:
    return _lib.lean_debug_build()


def lean_wait_selftest(limit_us: int, stream=None) -> None:
    """Launch the bounded-wait self-test: a block waits on a barrier nothing
    completes, gives up after limit_us and sets bit 8 of the error word."""
    _check("lean_wait_selftest", _lib.lean_wait_selftest(limit_us, _stream(stream)))


# ---- the operators of a serving step (include/lean_step.h, include/lean_cache.h) ----
#
# These take torch tensors on the GPU and read sizes, strides and element types
# off them (a caller without torch fills the C structs); every output is the
# caller's.  A tensor of a wrong shape or type, or on another device than the
# current GPU, is a ValueError, what the library refuses a LeanError.

_NORM = struct.Struct("<4qQqQqQqQQQqQq2dq")
_ROPE = struct.Struct("<8q" + "Q2q" * 5 + "3Q2Q5qdq" + "2Q3q")
_PAGES = struct.Struct("<3q3Q2qQqQ2Q5Qq")
_ATTENTION = struct.Struct("<6qQ2q2Q5qQ2qQQ2qQdqQqq" + "2Q3q")
_KV_READ = struct.Struct("<5q2Q5q2Q3qQQ2qQ2qq")
_PREFIX = struct.Struct("<6qQ2q2Q5q2Q3qqQ2q3Q2qQQ2qQdQqq")
_LOGPROBS = struct.Struct("<3qQqQdq5QQqq")
_dtypes = {}
_i32 = _f32 = _i64t = _u8 = _i8 = None  # torch's, once a call has needed them
_NO_SCALES = (0,) * 5
_device = None


def _here():
    """Index of the current GPU, as tensors on it have it; -2 without any."""
    global _i32, _f32, _i64t, _u8, _i8, _device
    if _device is not None:
        return _device()
    import torch
    _dtypes.update({torch.float32: LEAN_F32, torch.bfloat16: LEAN_BF16, torch.float16: LEAN_F16})
    _i32, _f32, _i64t, _u8, _i8 = torch.int32, torch.float32, torch.int64, torch.uint8, torch.int8
    if not torch.cuda.is_available():
        return -2
    here = torch.cuda.current_device()
    _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return here


def _dtype(t):
    code = _dtypes.get(t.dtype)
    if code is None:
        raise ValueError("element type %s: float32, bfloat16 or float16 is wanted" % t.dtype)
    return code


def _array(t, shape, dtype, name, here):
    """(address, stride of each dimension but the last) of a tensor on the current GPU of
    that shape and element type, its last dimension contiguous; zeros for None."""
    if t is None:
        return (0,) * len(shape)
    st = t.stride()
    if t.shape == shape and t.dtype is dtype and t.get_device() == here and (st[-1] == 1 or shape[-1] == 1):
        return (t.data_ptr(),) + st[:-1]
    raise ValueError("%s is %s %s on %s, strides %s: %s %s on the current GPU is wanted, the last dimension contiguous"
                     % (name, t.dtype, tuple(t.shape), t.device, st, dtype, tuple(shape)))


def _cache_dtype(t):
    """Code of a cache's element type, int8 among them."""
    return LEAN_I8 if t.dtype is _i8 else _dtype(t)


def _scales(cache, k_scales, v_scales, here):
    """The addresses and the three strides of the scales of caches in 8 bits, [pages, page_size, kv heads] float32;
    zeros for caches of 16 bits, which have none."""
    if k_scales is None and v_scales is None:
        return _NO_SCALES
    if cache is None or cache.dtype is not _i8:
        raise ValueError("k_scales and v_scales go with caches of int8")
    shape, out, at = cache.shape[:3], None, []
    for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
        if t is None:
            at.append(0)
            continue
        if t.shape != shape or t.dtype is not _f32 or t.get_device() != here:
            raise ValueError("%s is %s %s on %s: %s %s on the current GPU is wanted"
                             % (name, t.dtype, tuple(t.shape), t.device, _f32, tuple(shape)))
        st = t.stride()
        if out is not None and st != out:
            raise ValueError("k_scales and v_scales have different strides")
        out = st
        at.append(t.data_ptr())
    return (*at, *out)


def _plain(t, size, dtype, name, here):
    """Address of a contiguous tensor on the current GPU of `size` elements of that type; 0 for None."""
    if t is None:
        return 0
    if t.dtype is dtype and t.numel() == size and t.get_device() == here and t.is_contiguous():
        return t.data_ptr()
    raise ValueError("%s is %s %s on %s: %d contiguous elements of %s on the current GPU are wanted"
                     % (name, t.dtype, tuple(t.shape), t.device, size, dtype))


def _rows(t, rows, size, dtype, name, here):
    """As _plain, for `size` elements of each row: [rows, size], or all in one dimension."""
    if t is not None and t.dim() != 1 and t.shape != (rows, size):
        raise ValueError("%s is %s: [%d, %d] is wanted" % (name, tuple(t.shape), rows, size))
    return _plain(t, rows * size, dtype, name, here)


def _workspace(t, here):
    """(address, bytes) of a workspace; zeros for None."""
    if t is None:
        return 0, 0
    if t.dtype is _u8 and t.get_device() == here and t.is_contiguous():
        return t.data_ptr(), t.numel()
    raise ValueError("workspace is %s %s on %s, strides %s: contiguous bytes (uint8) on the current GPU are wanted"
                     % (t.dtype, tuple(t.shape), t.device, t.stride()))


def lean_residual_norm(x, h, w, h_out, y, eps: float = 1e-6, post_w=None, gate=None,
                       res_scale: float = 1.0, flags: int = 0, stream=None) -> None:
    """h_out = h + res_scale * gate * norm(x) and y = w * norm(h_out), rows of
    [rows, width]: x a block's output (None: none), h the residual (None: none),
    post_w the weights of the norm after the block (None: x as it is), gate
    [rows, width] or [width] (None: 1), w of the norm before the next one.
    h_out or y may be None."""
    here = _here()
    one = x if x is not None else h
    if one is None or one.dim() != 2:
        raise ValueError("x or h: [rows, width] is wanted")
    act = x if x is not None else y if y is not None else h
    res = h if h is not None else h_out if h_out is not None else act
    shape = one.shape
    rows, width = shape
    at, rt = act.dtype, res.dtype
    if gate is None:
        g = (0, 0)
    elif gate.dim() == 1 or gate.shape[0] == 1:
        g = _array(gate.reshape(1, -1), (1, width), at, "gate", here)[0], 0
    else:
        g = _array(gate, shape, at, "gate", here)
    args = _NORM.pack(rows, width, _dtype(act), _dtype(res), *_array(x, shape, at, "x", here),
                      *_array(h, shape, rt, "h", here), *g, _plain(post_w, width, _f32, "post_w", here),
                      _plain(w, width, _f32, "w", here),
                      *_array(h_out, shape, rt, "h_out", here), *_array(y, shape, at, "y", here), eps, res_scale, flags)
    st = _lib.lean_residual_norm(args, _stream(stream))
    if st:
        raise LeanError("lean_residual_norm", st)


def lean_rope_frequencies(kind: int, rot_dim: int, base: float, factor: float = 1.0, trained_len: float = 0.0,
                          slow: float = 1.0, fast: float = 32.0) -> np.ndarray:
    """Radians per position of each rotated pair (LEAN_ROPE_*), float64."""
    freq = np.zeros(max(1, rot_dim // 2))
    _check("lean_rope_frequencies", _lib.lean_rope_frequencies(kind, rot_dim, base, factor, trained_len, slow, fast,
                                                               freq.ctypes.data))
    return freq


def lean_rope_turns(freq) -> np.ndarray:
    """The whole-number form of frequencies that lean_rope_append takes: 2^-64
    turns per position, as int64 (the bits of uint64)."""
    freq = np.ascontiguousarray(freq, dtype=np.float64)
    turns = np.zeros(freq.shape, dtype=np.int64)
    _check("lean_rope_turns", _lib.lean_rope_turns(freq.ctypes.data, freq.size, turns.ctypes.data))
    return turns


def lean_rope_append(q, k, v, positions, slots, turns, q_out, k_cache, v_cache, rot_dim: int,
                     interleaved: bool = False, rot_scale: float = 1.0, k_out=None, flags: int = 0,
                     stream=None, k_scales=None, v_scales=None) -> None:
    """Rotate the first rot_dim elements of each head of q and k ([tokens, heads,
    dim]) to `positions`, into q_out (and k_out), and store k and v at `slots` of
    the caches ([pages, page_size, kv_heads, dim], strides of their own).  Caches
    of int8 are written in 8 bits, with a scale for each token and kv head in
    k_scales and v_scales ([pages, page_size, kv_heads] float32, any strides)."""
    here = _here()
    one = q if q is not None else k
    if one is None or one.dim() != 3:
        raise ValueError("q or k: [tokens, heads, dim] is wanted")
    n, _, dim = one.shape
    at = one.dtype
    hq = q.shape[1] if q is not None else 0
    hkv = k.shape[1] if k is not None else 0
    qs, ks = (n, hq, dim), (n, hkv, dim)
    some = k_cache if k_cache is not None else v_cache
    if some is not None:  # (one alone is refused by the library)
        pages, page = some.shape[:2]
        kc, vc = (_array(t, (pages, page, hkv, dim), some.dtype, name, here)
                  for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")))
        if kc[0] and vc[0] and vc[1:] != kc[1:]:
            raise ValueError("k_cache and v_cache have different strides")
        cache, cdt = (pages, page) + (kc if kc[0] else vc)[1:], _cache_dtype(some)
    else:
        cache, cdt, kc, vc = (0,) * 5, 0, (0,), (0,)
    args = _ROPE.pack(n, hq, hkv, dim, rot_dim, 1 if interleaved else 0, _dtype(one), cdt,
                      *_array(q, qs, at, "q", here), *_array(k, ks, at, "k", here), *_array(v, ks, at, "v", here),
                      *_array(q_out, qs, at, "q_out", here), *_array(k_out, ks, at, "k_out", here),
                      _plain(positions, n, _i32, "positions", here), _plain(slots, n, _i32, "slots", here),
                      _plain(turns, rot_dim // 2, _i64t, "turns", here), kc[0], vc[0], *cache, rot_scale, flags,
                      *_scales(some, k_scales, v_scales, here))
    st = _lib.lean_rope_append(args, _stream(stream))
    if st:
        raise LeanError("lean_rope_append", st)


def lean_kv_pages(lens, targets, block_table, free_ring, ring_state, page_size: int, lens_out, ring_state_out,
                  status, token_starts, slots=None, positions=None, token_seqs=None, flags: int = 0,
                  stream=None, max_tokens=None) -> None:
    """Sequences go from `lens` to `targets` tokens: pages are taken from and
    given back to the free ring, block_table [seqs, width] follows, and the new
    tokens' slots, positions and sequences are written as one packed batch
    (int32 throughout).  Each of the three may be left out.  max_tokens: the most
    new tokens of a call, past which sequences fail; None: as many as the maps
    given hold (without any: 0, so that only sequences that do not grow succeed;
    2 ** 31 - 1 sets no limit)."""
    here = _here()
    n = lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise ValueError("block_table: [%d, width] is wanted" % n)
    some = slots if slots is not None else positions if positions is not None else token_seqs
    most = max_tokens if max_tokens is not None else some.numel() if some is not None else 0
    i32 = _i32
    table, stride = _array(block_table, block_table.shape, i32, "block_table", here)
    args = _PAGES.pack(n, page_size, most, _plain(lens, n, i32, "lens", here), _plain(targets, n, i32, "targets", here),
                       table, block_table.shape[1], stride,
                       _plain(free_ring, free_ring.numel(), i32, "free_ring", here), free_ring.numel(),
                       _plain(ring_state, 2, i32, "ring_state", here), _plain(lens_out, n, i32, "lens_out", here),
                       _plain(ring_state_out, 2, i32, "ring_state_out", here), _plain(status, n, i32, "status", here),
                       _plain(token_starts, n + 1, i32, "token_starts", here), _plain(slots, most, i32, "slots", here),
                       _plain(positions, most, i32, "positions", here),
                       _plain(token_seqs, most, i32, "token_seqs", here), flags)
    st = _lib.lean_kv_pages(args, _stream(stream))
    if st:
        raise LeanError("lean_kv_pages", st)


def lean_kv_read(k_cache, v_cache, slots, k_out, v_out, k_scales=None, v_scales=None, flags: int = 0,
                 stream=None) -> None:
    """The tokens at `slots` of the caches ([pages, page_size, kv_heads, dim]) as
    rows of k_out and v_out [tokens, kv_heads, dim], float32, bfloat16 or float16,
    whatever the caches are (int8 with k_scales and v_scales as for
    lean_rope_append).  Either cache may be None with its output."""
    here = _here()
    some, out = (k_cache, k_out) if k_cache is not None else (v_cache, v_out)
    if some is None or out is None or some.dim() != 4:
        raise ValueError("k_cache with k_out or v_cache with v_out: [pages, page_size, kv_heads, dim] and"
                         " [tokens, kv_heads, dim] are wanted")
    shape, ct = some.shape, some.dtype
    n, rows = slots.numel(), (slots.numel(),) + shape[2:]
    kc, vc = _array(k_cache, shape, ct, "k_cache", here), _array(v_cache, shape, ct, "v_cache", here)
    if kc[0] and vc[0] and vc[1:] != kc[1:]:
        raise ValueError("k_cache and v_cache have different strides")
    args = _KV_READ.pack(n, *shape[2:], _dtype(out), _cache_dtype(some), kc[0], vc[0], *shape[:2],
                         *(kc if kc[0] else vc)[1:], *_scales(some, k_scales, v_scales, here),
                         _plain(slots, n, _i32, "slots", here), *_array(k_out, rows, out.dtype, "k_out", here),
                         *_array(v_out, rows, out.dtype, "v_out", here), flags)
    st = _lib.lean_kv_read(args, _stream(stream))
    if st:
        raise LeanError("lean_kv_read", st)


def lean_paged_attention_workspace_bytes(n_seqs: int, n_q_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return _lib.lean_paged_attention_workspace_bytes(n_seqs, n_q_heads, n_kv_heads, head_dim)


def lean_paged_attention(q, k_cache, v_cache, block_table, seq_lens, out, scale: float, window: int = 0, lse=None,
                         workspace=None, flags: int = 0, stream=None, k_scales=None, v_scales=None) -> None:
    """Attention of one new token per sequence: q and out [seqs, heads, dim], the
    caches (and scales) as for lean_rope_append, block_table [seqs, width], lse [seqs, heads]
    (None: not wanted); workspace: a uint8 tensor of
    lean_paged_attention_workspace_bytes."""
    here = _here()
    shape, at, ct = q.shape, q.dtype, k_cache.dtype
    n, hq, dim = shape
    pages, page, hkv = k_cache.shape[:3]
    kc = _array(k_cache, (pages, page, hkv, dim), ct, "k_cache", here)
    vc = _array(v_cache, (pages, page, hkv, dim), ct, "v_cache", here)
    if vc[1:] != kc[1:]:
        raise ValueError("k_cache and v_cache have different strides")
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise ValueError("block_table: [%d, width] is wanted" % n)
    table = _array(block_table, block_table.shape, _i32, "block_table", here)
    args = _ATTENTION.pack(n, hq, hkv, dim, _dtype(q), _cache_dtype(k_cache), *_array(q, shape, at, "q", here), kc[0], vc[0],
                           pages, page, *kc[1:], table[0], block_table.shape[1], table[1],
                           _plain(seq_lens, n, _i32, "seq_lens", here), *_array(out, shape, at, "out", here),
                           _rows(lse, n, hq, _f32, "lse", here), scale, window, *_workspace(workspace, here), flags,
                           *_scales(k_cache, k_scales, v_scales, here))
    st = _lib.lean_paged_attention(args, _stream(stream))
    if st:
        raise LeanError("lean_paged_attention", st)


def lean_prefix_attention_workspace_bytes(n_seqs: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                                          n_prefixes: int) -> int:
    return _lib.lean_prefix_attention_workspace_bytes(n_seqs, n_q_heads, n_kv_heads, head_dim, n_prefixes)


def lean_prefix_attention(q, k_cache, v_cache, prefix_table, prefix_lens, seq_starts, block_table, seq_lens, out,
                          scale: float, lse=None, workspace=None, flags: int = 0, stream=None, k_scales=None,
                          v_scales=None) -> None:
    """Attention of one new token per sequence where sequences seq_starts[p] ..
    seq_starts[p + 1] - 1 begin with prefix p: prefix_table [prefixes, width] and
    prefix_lens [prefixes] have its pages and length, block_table [seqs, width] and
    seq_lens [seqs] those of the sequences' own tokens after it; the rest as for
    lean_paged_attention.  workspace: a uint8 tensor of
    lean_prefix_attention_workspace_bytes."""
    here = _here()
    shape, at, ct = q.shape, q.dtype, k_cache.dtype
    n, hq, dim = shape
    pages, page, hkv = k_cache.shape[:3]
    kc = _array(k_cache, (pages, page, hkv, dim), ct, "k_cache", here)
    vc = _array(v_cache, (pages, page, hkv, dim), ct, "v_cache", here)
    if vc[1:] != kc[1:]:
        raise ValueError("k_cache and v_cache have different strides")
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise ValueError("block_table: [%d, width] is wanted" % n)
    if prefix_table.dim() != 2:
        raise ValueError("prefix_table: [prefixes, width] is wanted")
    prefixes = prefix_table.shape[0]
    shared = _array(prefix_table, prefix_table.shape, _i32, "prefix_table", here)
    table = _array(block_table, block_table.shape, _i32, "block_table", here)
    args = _PREFIX.pack(n, hq, hkv, dim, _dtype(q), _cache_dtype(k_cache), *_array(q, shape, at, "q", here), kc[0], vc[0],
                        pages, page, *kc[1:], *_scales(k_cache, k_scales, v_scales, here), prefixes, shared[0],
                        prefix_table.shape[1], shared[1], _plain(prefix_lens, prefixes, _i32, "prefix_lens", here),
                        _plain(seq_starts, prefixes + 1, _i32, "seq_starts", here), table[0], block_table.shape[1], table[1],
                        _plain(seq_lens, n, _i32, "seq_lens", here), *_array(out, shape, at, "out", here),
                        _rows(lse, n, hq, _f32, "lse", here), scale, *_workspace(workspace, here), flags)
    st = _lib.lean_prefix_attention(args, _stream(stream))
    if st:
        raise LeanError("lean_prefix_attention", st)


def lean_token_logprobs_workspace_bytes(rows: int, vocab: int, top_k: int) -> int:
    return _lib.lean_token_logprobs_workspace_bytes(rows, vocab, top_k)


def lean_token_logprobs(logits, ids, logprobs, ranks=None, entropy=None, top_ids=None, top_logprobs=None,
                        scale: float = 1.0, workspace=None, flags: int = 0, stream=None) -> None:
    """Log probabilities of ids [rows] under softmax(scale * logits [rows, vocab]),
    how many logits are larger, the entropy, and the top_ids.shape[1] most likely
    ids with theirs.  Outputs that are None are left out; workspace: a uint8 tensor
    of lean_token_logprobs_workspace_bytes."""
    here = _here()
    rows, vocab = logits.shape
    k = 0 if top_ids is None else top_ids.shape[1] if top_ids.dim() == 2 else top_ids.numel() // max(1, rows)
    x = _array(logits, (rows, vocab), logits.dtype, "logits", here)
    f32 = _f32
    args = _LOGPROBS.pack(rows, vocab, _dtype(logits), *x, _plain(ids, rows, _i32, "ids", here), scale, k,
                          _plain(logprobs, rows, f32, "logprobs", here), _plain(ranks, rows, _i32, "ranks", here),
                          _plain(entropy, rows, f32, "entropy", here), _rows(top_ids, rows, k, _i32, "top_ids", here),
                          _rows(top_logprobs, rows, k, f32, "top_logprobs", here), *_workspace(workspace, here), flags)
    st = _lib.lean_token_logprobs(args, _stream(stream))
    if st:
        raise LeanError("lean_token_logprobs", st)


# ---- torch conveniences (device memory via PyTorch; compute via the library) ----

def upload_packed(fmt: int, canon, N: int, K: int, device="cuda"):
    """Pack canonical host bytes and copy them to a new uint8 device tensor."""
    import torch
    packed = lean_pack(fmt, canon, N, K)
    return torch.from_numpy(packed).to(device)


def qmatmul(fmt: int, W_packed_dev, x, N: int, K: int, out=None, stream=None):
    """Allocate y (or use `out`) and run lean_qmatmul; x is a [M, K] fp32 cuda tensor."""
    import torch
    x = x.contiguous()
    M = x.numel() // K
    y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=x.device)
    lean_qmatmul(fmt, W_packed_dev, x, y, N, K, M, stream)
    return y
