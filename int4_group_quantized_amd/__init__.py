"""Python binding of libq4g128 (int4 group-128 GEMV family for MI355X).

Argument marshalling only: every entry point checks tensor devices, dtypes,
shapes and contiguity, then passes raw device pointers, sizes and the
current HIP stream of the tensors' device to the C ABI of the same name
(include/q4g128.h).  All arithmetic runs in the library's HIP kernels; there
is no fallback path.  Importing this package fails loudly if the library is
not built, and the cache and attention calls if their compiled binding is not.

PyTorch provides device memory and streams: fp16 arguments are torch.float16
tensors (the C ABI receives their bit patterns), codes/packed are torch.uint8,
outputs are torch.float32.
"""
from __future__ import annotations

import ctypes
import os

import torch  # noqa: F401  (loads torch's HIP runtime before the library binds to it)

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "libq4g128.so")

Q4_OK = 0
Q4_EINVAL = -1
Q4_ESHAPE = -2
Q4_EALIGN = -3
Q4_EDEVICE = -4
GROUP = 128
MAX_K = 32768
MAX_BATCH = 16
INT8_MAX_K = 8192
MAX_GROUPED = 65536
ATTN_COUNTER_BYTES = 4096
MAX_DRAFT = 64
LATENT_ROT = 64


class GemvDesc(ctypes.Structure):
    """struct q4g128_gemv_desc of include/q4g128.h."""
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("mins", ctypes.c_void_p),
                ("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("n", ctypes.c_int64), ("k", ctypes.c_int64)]

class KvCache(ctypes.Structure):
    """struct q4g128_kv_cache of include/q4g128.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("table", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64), ("sequences", ctypes.c_int64),
                ("table_cols", ctypes.c_int64), ("kv_heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("page", ctypes.c_int32)]


class LatentCache(ctypes.Structure):
    """struct q4g128_latent_cache of include/q4g128.h."""
    _fields_ = [("rows", ctypes.c_void_p), ("table", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("stride", ctypes.c_int64), ("sequences", ctypes.c_int64), ("table_cols", ctypes.c_int64),
                ("latent", ctypes.c_int32), ("page", ctypes.c_int32)]


class AttnOptions(ctypes.Structure):
    """struct q4g128_attn_options of include/q4g128.h."""
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", ctypes.c_int64),
                ("slopes", ctypes.c_void_p), ("prefix", ctypes.c_void_p)]


EXPORTED = (
    "q4g128_pack",
    "q4g128_quantize",
    "q4g128_gemv",
    "q4g128_gemv_grouped",
    "q4g128_gemm_small_batch",
    "q4g128_gemm_prefill",
    "q4g128_gemm_prefill_epilogue",
    "q4g128_gemv_int8",
    "q4g128_rope_append",
    "q4g128_rope_append_slots",
    "q4g128_cache_keep",
    "q4g128_attn_decode_workspace",
    "q4g128_attn_decode",
    "q4g128_attn_prefill_workspace",
    "q4g128_attn_prefill",
    "q4g128_attn_tree_workspace",
    "q4g128_attn_tree",
    "q4g128_latent_append",
    "q4g128_latent_keep",
    "q4g128_latent_attn_workspace",
    "q4g128_latent_attn",
    "q4g128_latent_expand",
    "q4g128_latent_prefill_workspace",
    "q4g128_latent_prefill",
    "q4g128_status_string",
    "q4g128_last_hip_error",
)


class Q4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.q4g128_status_string(status).decode()
        if status == Q4_EDEVICE:
            msg += f" (hipError_t {_lib.q4g128_last_hip_error()})"
        super().__init__(f"{where}: {msg}")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python int4_group_quantized_amd/build.py` "
            "(or __graft_entry__.build()); there is no fallback implementation"
        )
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    lib.q4g128_pack.argtypes = [vp, vp, i64, i64, vp]
    lib.q4g128_quantize.argtypes = [vp, vp, vp, vp, i64, i64, vp]
    lib.q4g128_gemv.argtypes = [vp, vp, vp, vp, vp, i64, i64, vp]
    lib.q4g128_gemv_grouped.argtypes = [ctypes.POINTER(GemvDesc), i64, vp]
    lib.q4g128_gemm_small_batch.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
    lib.q4g128_gemm_prefill.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
    lib.q4g128_gemv_int8.argtypes = [vp, vp, vp, vp, i64, i64, vp]
    lib.q4g128_gemm_prefill_epilogue.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
    i32, f32 = ctypes.c_int32, ctypes.c_float
    cache, options = ctypes.POINTER(KvCache), ctypes.POINTER(AttnOptions)
    lib.q4g128_rope_append.argtypes = [vp, i64, i64, i32, cache, vp, vp, vp, i32, i32, f32, vp, vp, f32, vp, vp]
    lib.q4g128_rope_append_slots.argtypes = [vp, i64, i64, i32, cache, vp, vp, vp, vp, i32, i32, f32, vp, vp, f32, vp,
                                             vp]
    lib.q4g128_cache_keep.argtypes = [cache, vp, vp, vp, i64, i64, vp]
    lib.q4g128_attn_tree_workspace.argtypes = [i64, i64, i32, i32, i32, i64, i64]
    lib.q4g128_attn_tree.argtypes = [vp, cache, vp, vp, vp, i64, i64, i64, i64, i32, options, vp, vp, i64, vp]
    latent = ctypes.POINTER(LatentCache)
    lib.q4g128_latent_append.argtypes = [vp, i64, i64, latent, vp, vp, vp, vp, i32, f32, vp, f32, vp, i64, i64, i32, vp,
                                         i64, i64, i32, vp, vp]
    lib.q4g128_latent_keep.argtypes = [latent, vp, vp, vp, i64, i64, vp]
    lib.q4g128_latent_attn_workspace.argtypes = [i32, i32, i64]
    lib.q4g128_latent_attn.argtypes = [vp, latent, vp, vp, vp, i64, i64, i64, i64, i32, f32, vp, vp, i64, vp]
    lib.q4g128_latent_expand.argtypes = [latent, vp, vp, i64, i64, vp, vp, vp, cache, vp]
    lib.q4g128_latent_prefill_workspace.argtypes = [i64, i64, i32, i32, i64]
    lib.q4g128_latent_prefill.argtypes = [vp, cache, vp, vp, i64, i64, i64, f32, vp, vp, i64, vp]
    lib.q4g128_attn_decode_workspace.argtypes = [i64, i32, i32]
    lib.q4g128_attn_decode.argtypes = [vp, cache, vp, i64, i64, i32, options, vp, vp, i64, vp]
    lib.q4g128_attn_prefill_workspace.argtypes = [i64, i64, i32, i32, i32, i64]
    lib.q4g128_attn_prefill.argtypes = [vp, cache, vp, vp, i64, i64, i64, i32, options, vp, vp, i64, vp]
    for name in ("q4g128_pack", "q4g128_quantize", "q4g128_gemv", "q4g128_gemv_grouped", "q4g128_gemm_small_batch",
                 "q4g128_gemm_prefill",
                 "q4g128_gemv_int8", "q4g128_gemm_prefill_epilogue", "q4g128_rope_append", "q4g128_attn_decode",
                 "q4g128_attn_prefill", "q4g128_rope_append_slots", "q4g128_cache_keep", "q4g128_attn_tree",
                 "q4g128_latent_append", "q4g128_latent_keep", "q4g128_latent_attn",
                 "q4g128_latent_expand", "q4g128_latent_prefill"):
        getattr(lib, name).restype = ctypes.c_int32
    for name in ("q4g128_attn_decode_workspace", "q4g128_attn_prefill_workspace", "q4g128_attn_tree_workspace",
                 "q4g128_latent_attn_workspace", "q4g128_latent_prefill_workspace"):
        getattr(lib, name).restype = ctypes.c_int64
    lib.q4g128_status_string.argtypes = [ctypes.c_int32]
    lib.q4g128_status_string.restype = ctypes.c_char_p
    lib.q4g128_last_hip_error.argtypes = []
    lib.q4g128_last_hip_error.restype = ctypes.c_int32
    return lib


_lib = _load()


class _NoBinding:
    """In place of the compiled module: its calls say why it could not be loaded."""

    def __init__(self, error: ImportError):
        self.error = error

    def __getattr__(self, call):
        raise ImportError(f"q4g128_{call}: {self.error}: build the binding with "
                          "`python int4_group_quantized_amd/build.py`") from self.error


# The cache and attention calls' checks and calls are compiled (csrc/binding.cpp),
# for one torch and Python; their module links to the library loaded above.
# The products do without it.
try:
    from . import _binding
except ImportError as e:
    _binding = _NoBinding(e)


def library() -> ctypes.CDLL:
    return _lib


def _check(status: int, where: str) -> None:
    if status != Q4_OK:
        raise Q4Error(status, where)


def _dev_tensor(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live on a GPU (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _same_device(*ts: torch.Tensor) -> torch.device:
    dev = ts[0].device
    for t in ts[1:]:
        if t.device != dev:
            raise ValueError("all tensors must be on the same GPU")
    return dev


def _stream(dev: torch.device, stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    return stream.cuda_stream


def _weights(packed, scales, mins):
    if packed.dim() != 2:
        raise ValueError("packed must be [N][K/2]")
    n, half_k = packed.shape
    k = 2 * half_k
    _dev_tensor(packed, "packed", torch.uint8, (n, half_k))
    _dev_tensor(scales, "scales", torch.float16, (n, k // GROUP))
    _dev_tensor(mins, "mins", torch.float16, (n, k // GROUP))
    return n, k


def q4g128_pack(codes: torch.Tensor, packed: torch.Tensor = None, stream=None) -> torch.Tensor:
    """codes uint8 [N][K] (low 4 bits used) -> packed uint8 [N][K/2]."""
    if codes.dim() != 2:
        raise ValueError("codes must be [N][K]")
    n, k = codes.shape
    _dev_tensor(codes, "codes", torch.uint8, (n, k))
    if packed is None:
        packed = torch.empty((n, k // 2), dtype=torch.uint8, device=codes.device)
    _dev_tensor(packed, "packed", torch.uint8, (n, k // 2))
    dev = _same_device(codes, packed)
    with torch.cuda.device(dev):
        _check(_lib.q4g128_pack(codes.data_ptr(), packed.data_ptr(), n, k, _stream(dev, stream)), "q4g128_pack")
    return packed


def q4g128_quantize(W: torch.Tensor, packed=None, scales=None, mins=None, stream=None):
    """float32 W [N][K] -> (packed uint8 [N][K/2], scales fp16 [N][K/128], mins fp16 [N][K/128])."""
    if W.dim() != 2:
        raise ValueError("W must be [N][K]")
    n, k = W.shape
    _dev_tensor(W, "W", torch.float32, (n, k))
    g = k // GROUP
    if packed is None:
        packed = torch.empty((n, k // 2), dtype=torch.uint8, device=W.device)
    if scales is None:
        scales = torch.empty((n, g), dtype=torch.float16, device=W.device)
    if mins is None:
        mins = torch.empty((n, g), dtype=torch.float16, device=W.device)
    _dev_tensor(packed, "packed", torch.uint8, (n, k // 2))
    _dev_tensor(scales, "scales", torch.float16, (n, g))
    _dev_tensor(mins, "mins", torch.float16, (n, g))
    dev = _same_device(W, packed, scales, mins)
    with torch.cuda.device(dev):
        _check(_lib.q4g128_quantize(W.data_ptr(), packed.data_ptr(), scales.data_ptr(), mins.data_ptr(), n, k,
                                    _stream(dev, stream)), "q4g128_quantize")
    return packed, scales, mins


def q4g128_gemv(packed, scales, mins, x, y=None, stream=None) -> torch.Tensor:
    """y[N] fp32 = W x for fp16 x [K]."""
    n, k = _weights(packed, scales, mins)
    _dev_tensor(x, "x", torch.float16, (k,))
    if y is None:
        y = torch.empty((n,), dtype=torch.float32, device=packed.device)
    _dev_tensor(y, "y", torch.float32, (n,))
    dev = _same_device(packed, scales, mins, x, y)
    with torch.cuda.device(dev):
        _check(_lib.q4g128_gemv(packed.data_ptr(), scales.data_ptr(), mins.data_ptr(), x.data_ptr(),
                                y.data_ptr(), n, k, _stream(dev, stream)), "q4g128_gemv")
    return y


def gemv_descs(projections, ys):
    """ctypes array of q4g128_gemv_desc for [(packed, scales, mins, x)] and outputs ys (shapes checked)."""
    arr = (GemvDesc * len(projections))()
    for i, ((packed, scales, mins, x), y) in enumerate(zip(projections, ys)):
        n, k = _weights(packed, scales, mins)
        _dev_tensor(x, f"x[{i}]", torch.float16, (k,))
        _dev_tensor(y, f"y[{i}]", torch.float32, (n,))
        _same_device(projections[0][0], packed, scales, mins, x, y)
        arr[i] = GemvDesc(packed.data_ptr(), scales.data_ptr(), mins.data_ptr(), x.data_ptr(), y.data_ptr(), n, k)
    return arr


def q4g128_gemv_grouped(projections, ys=None, stream=None):
    """[y_i = W_i x_i] for independent projections [(packed, scales, mins, x)], in few launches.

    Each y_i is bit-identical to q4g128_gemv on projection i.  Returns the list of outputs.
    """
    projections = list(projections)
    if not projections:
        raise ValueError("projections must not be empty")
    if ys is None:
        ys = [torch.empty((p[0].shape[0],), dtype=torch.float32, device=p[0].device) for p in projections]
    if len(ys) != len(projections):
        raise ValueError("one output per projection")
    arr = gemv_descs(projections, ys)
    dev = projections[0][0].device
    with torch.cuda.device(dev):
        _check(_lib.q4g128_gemv_grouped(arr, len(projections), _stream(dev, stream)), "q4g128_gemv_grouped")
    return ys


def q4g128_gemm_small_batch(packed, scales, mins, X, Y=None, stream=None) -> torch.Tensor:
    """Y[B][N] fp32 = X W^T for fp16 X [B][K], 1 <= B <= 16; row b equals q4g128_gemv(X[b])."""
    n, k = _weights(packed, scales, mins)
    if X.dim() != 2:
        raise ValueError("X must be [B][K]")
    b = X.shape[0]
    _dev_tensor(X, "X", torch.float16, (b, k))
    if Y is None:
        Y = torch.empty((b, n), dtype=torch.float32, device=packed.device)
    _dev_tensor(Y, "Y", torch.float32, (b, n))
    dev = _same_device(packed, scales, mins, X, Y)
    with torch.cuda.device(dev):
        _check(_lib.q4g128_gemm_small_batch(packed.data_ptr(), scales.data_ptr(), mins.data_ptr(),
                                            X.data_ptr(), Y.data_ptr(), n, k, b, _stream(dev, stream)),
               "q4g128_gemm_small_batch")
    return Y


def q4g128_gemm_prefill(packed, scales, mins, X, Y=None, stream=None) -> torch.Tensor:
    """Y[M][N] fp32 = X fp16(W)^T for fp16 X [M][K] on the matrix cores."""
    n, k = _weights(packed, scales, mins)
    if X.dim() != 2:
        raise ValueError("X must be [M][K]")
    m = X.shape[0]
    _dev_tensor(X, "X", torch.float16, (m, k))
    if Y is None:
        Y = torch.empty((m, n), dtype=torch.float32, device=packed.device)
    _dev_tensor(Y, "Y", torch.float32, (m, n))
    dev = _same_device(packed, scales, mins, X, Y)
    with torch.cuda.device(dev):
        _check(_lib.q4g128_gemm_prefill(packed.data_ptr(), scales.data_ptr(), mins.data_ptr(),
                                        X.data_ptr(), Y.data_ptr(), n, k, m, _stream(dev, stream)),
               "q4g128_gemm_prefill")
    return Y


def q4g128_gemm_prefill_epilogue(packed, scales, mins, X, Y=None, stream=None) -> torch.Tensor:
    """Y[M][N] fp32 = X W^T for fp16 X [M][K]: exact codes on the matrix cores, scale and min per group on the result."""
    n, k = _weights(packed, scales, mins)
    if X.dim() != 2:
        raise ValueError("X must be [M][K]")
    m = X.shape[0]
    _dev_tensor(X, "X", torch.float16, (m, k))
    if Y is None:
        Y = torch.empty((m, n), dtype=torch.float32, device=packed.device)
    _dev_tensor(Y, "Y", torch.float32, (m, n))
    dev = _same_device(packed, scales, mins, X, Y)
    with torch.cuda.device(dev):
        _check(_lib.q4g128_gemm_prefill_epilogue(packed.data_ptr(), scales.data_ptr(), mins.data_ptr(),
                                                 X.data_ptr(), Y.data_ptr(), n, k, m, _stream(dev, stream)),
               "q4g128_gemm_prefill_epilogue")
    return Y


def q4g128_gemv_int8(q, scales, x, y=None, stream=None) -> torch.Tensor:
    """y[N] fp32 = scale[n] * (q x) for int8 q [N][K], fp16 scales [N], fp16 x [K]."""
    if q.dim() != 2:
        raise ValueError("q must be [N][K]")
    n, k = q.shape
    _dev_tensor(q, "q", torch.int8, (n, k))
    _dev_tensor(scales, "scales", torch.float16, (n,))
    _dev_tensor(x, "x", torch.float16, (k,))
    if y is None:
        y = torch.empty((n,), dtype=torch.float32, device=q.device)
    _dev_tensor(y, "y", torch.float32, (n,))
    dev = _same_device(q, scales, x, y)
    with torch.cuda.device(dev):
        _check(_lib.q4g128_gemv_int8(q.data_ptr(), scales.data_ptr(), x.data_ptr(), y.data_ptr(), n, k,
                                     _stream(dev, stream)), "q4g128_gemv_int8")
    return y


def _answer(got, where):
    """The output tensor of a compiled call, or its status as an error."""
    if type(got) is int:
        raise Q4Error(got, where)
    return got


def q4g128_rope_append(qkv, k_cache, v_cache, table, positions, inv_freq, heads, seq=None, q_norm=None, k_norm=None,
                       eps=1e-6, interleaved=False, mscale=1.0, q=None, stream=None, slots=None) -> torch.Tensor:
    """Head norm, rotary position and cache write of new tokens; returns q fp16 [T][heads][dim].

    qkv: fp32 [T][>= (heads + 2 kv_heads) dim], rows may be strided (a product's output: columns after the
    value heads are left alone).  k_cache fp16 [pages][kv_heads][page][dim], v_cache fp16
    [pages][kv_heads][dim][page], table int32 [sequences][cols]; a page is contiguous, the pages may be a strided
    slice of a larger pool.  positions int32 [T]; slots int32 [T]: the positions that are written, where they are not
    those that heads are turned by (drafted tokens of a tree); seq int32 [T] (None: token t is of sequence t).  inv_freq fp32
    [rot / 2] (None: no rotation).  q_norm, k_norm fp16 [dim] or None.
    """
    if stream is not None:
        with torch.cuda.stream(stream):  # new memory is the stream's too
            return q4g128_rope_append(qkv, k_cache, v_cache, table, positions, inv_freq, heads, seq, q_norm, k_norm,
                                      eps, interleaved, mscale, q, slots=slots)
    return _answer(_binding.rope_append(qkv, k_cache, v_cache, table, positions, inv_freq, heads, seq, q_norm, k_norm,
                                        eps, interleaved, mscale, q, slots), "q4g128_rope_append")


def q4g128_attn_decode_workspace(batch, heads, dim) -> int:
    """Bytes of workspace that q4g128_attn_decode needs."""
    return _lib.q4g128_attn_decode_workspace(batch, heads, dim)


def q4g128_attn_prefill_workspace(tokens, count, heads, kv_heads, dim, max_length) -> int:
    """Bytes of workspace that q4g128_attn_prefill needs (0: none)."""
    return _lib.q4g128_attn_prefill_workspace(tokens, count, heads, kv_heads, dim, max_length)


def q4g128_attn_decode(q, k_cache, v_cache, table, lengths, scale=None, softcap=0.0, window=0, slopes=None,
                       max_length=None, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Attention of one new token per sequence: q fp16 [B][heads][dim] -> out fp16 [B][heads][dim].

    lengths int32 [B] counts the cached positions of sequence b (row b of table), the new one included.
    scale: dim ** -0.5 by default; softcap, window, slopes as in include/q4g128.h.  max_length: an upper bound on
    the lengths (default: what the table holds).  workspace: uint8 of q4g128_attn_decode_workspace bytes, its first
    ATTN_COUNTER_BYTES zero before its first use (default: one that the binding keeps for the stream, or in a graph
    capture one of the graph's own).
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return q4g128_attn_decode(q, k_cache, v_cache, table, lengths, scale, softcap, window, slopes, max_length,
                                      out, workspace)
    return _answer(_binding.attn_decode(q, k_cache, v_cache, table, lengths, scale, softcap, window, slopes,
                                        max_length, out, workspace), "q4g128_attn_decode")


def q4g128_attn_prefill(q, k_cache, v_cache, table, q_starts, lengths, scale=None, softcap=0.0, window=0, slopes=None,
                        prefix=None, max_length=None, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Causal attention of prompt tokens packed over sequences: q fp16 [T][heads][dim] -> out, same shape.

    Rows q_starts[s]..q_starts[s+1]-1 (int32 [S + 1]) are the last positions of sequence s, which holds lengths[s]
    positions (int32 [S]), these included.  prefix int32 [S]: positions below prefix[s] are seen by every token of
    the sequence (not together with a window).  Other arguments as q4g128_attn_decode.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return q4g128_attn_prefill(q, k_cache, v_cache, table, q_starts, lengths, scale, softcap, window, slopes,
                                       prefix, max_length, out, workspace)
    return _answer(_binding.attn_prefill(q, k_cache, v_cache, table, q_starts, lengths, scale, softcap, window, slopes,
                                         prefix, max_length, out, workspace), "q4g128_attn_prefill")


def q4g128_attn_tree_workspace(tokens, count, heads, kv_heads, dim, max_new, max_length) -> int:
    """Bytes of workspace that q4g128_attn_tree needs (0: none)."""
    return _lib.q4g128_attn_tree_workspace(tokens, count, heads, kv_heads, dim, max_new, max_length)


def q4g128_attn_tree(q, k_cache, v_cache, table, q_starts, lengths, masks=None, scale=None, softcap=0.0, window=0,
                     slopes=None, max_new=None, max_length=None, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Attention of drafted tokens packed over sequences: q fp16 [T][heads][dim] -> out, same shape.

    Rows q_starts[s]..q_starts[s+1]-1 (int32 [S + 1]), at most 64 of a sequence, are the last of its lengths[s] cached
    positions (int32 [S]).  masks int64 [T]: a token sees every position before its sequence's draft, and drafted
    token k where bit k of its mask is set (a tree: its ancestors and itself); None: the tokens up to itself.
    max_new: an upper bound on a sequence's tokens (default: 64, or T).  Other arguments as q4g128_attn_decode.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return q4g128_attn_tree(q, k_cache, v_cache, table, q_starts, lengths, masks, scale, softcap, window, slopes,
                                    max_new, max_length, out, workspace)
    return _answer(_binding.attn_tree(q, k_cache, v_cache, table, q_starts, lengths, masks, scale, softcap, window,
                                      slopes, max_new, max_length, out, workspace), "q4g128_attn_tree")


def q4g128_cache_keep(k_cache, v_cache, table, starts, keep_starts, keep, stream=None) -> None:
    """Accepted drafted tokens moved together, in place: position starts[s] + keep[i] becomes starts[s] + i.

    starts int32 [S]: the committed positions of each sequence; keep int32 [n]: for sequence s the numbers
    keep[keep_starts[s]:keep_starts[s + 1]] of its accepted tokens within the draft, strictly ascending; keep_starts
    int32 [S + 1].
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return q4g128_cache_keep(k_cache, v_cache, table, starts, keep_starts, keep)
    _check(_binding.cache_keep(k_cache, v_cache, table, starts, keep_starts, keep), "q4g128_cache_keep")


def q4g128_latent_append(kv, cache, table, positions, inv_freq, seq=None, slots=None, norm=None, eps=1e-6,
                         interleaved=False, mscale=1.0, q_main=None, q_rot=None, q=None, stream=None):
    """New tokens' latent rows into the cache; returns their queries fp16 [T][heads][main + 64], or None without any.

    kv: fp32 [T][>= latent + 64], rows may be strided.  cache fp16 [pages][page][latent + 64], each page contiguous;
    table int32 [sequences][cols].  positions, slots, seq as q4g128_rope_append; inv_freq fp32 [32] or None (nothing is
    turned); norm fp16 [latent] or None.  q_main fp32 [T][heads][main] and q_rot fp32 [T][heads][64], both or none, may
    be views of larger tensors.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return q4g128_latent_append(kv, cache, table, positions, inv_freq, seq, slots, norm, eps, interleaved, mscale,
                                        q_main, q_rot, q)
    return _answer(_binding.latent_append(kv, cache, table, positions, inv_freq, seq, slots, norm, eps, interleaved,
                                          mscale, q_main, q_rot, q), "q4g128_latent_append")


def q4g128_latent_keep(cache, table, starts, keep_starts, keep, stream=None) -> None:
    """q4g128_cache_keep for a latent cache."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return q4g128_latent_keep(cache, table, starts, keep_starts, keep)
    _check(_binding.latent_keep(cache, table, starts, keep_starts, keep), "q4g128_latent_keep")


def q4g128_latent_attn_workspace(heads, latent, max_new) -> int:
    """Bytes of workspace that q4g128_latent_attn needs."""
    return _lib.q4g128_latent_attn_workspace(heads, latent, max_new)


def q4g128_latent_attn(q, cache, table, q_starts, lengths, scale, masks=None, max_new=None, max_length=None, out=None,
                       workspace=None, stream=None) -> torch.Tensor:
    """Attention over the latent rows themselves: q fp16 [T][heads][latent + 64] -> out fp16 [T][heads][latent].

    q_starts, lengths, masks and max_new as q4g128_attn_tree; without masks a sequence may have any number of rows, and
    max_new is T by default.  Give it for several sequences, 1 for single tokens: the work is shared out as if every
    sequence had max_new rows (64 sequences of 8,192 positions and 16 heads: 115 us with 1, 290 with the default).  Other
    arguments as q4g128_attn_decode.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return q4g128_latent_attn(q, cache, table, q_starts, lengths, scale, masks, max_new, max_length, out,
                                      workspace)
    return _answer(_binding.latent_attn(q, cache, table, q_starts, lengths, scale, masks, max_new, max_length, out,
                                        workspace), "q4g128_latent_attn")


def q4g128_latent_expand(cache, table, lengths, packed, scales, mins, k_cache, v_cache, expanded_table, firsts=None,
                         max_length=None, stream=None) -> None:
    """Keys and values of every head from latent rows by int4 weights, into pages that q4g128_latent_prefill reads.

    packed, scales, mins: the format of q4g128_quantize for [heads * 2 * value][latent], each head's key rows before its
    value rows.  k_cache fp16 [pages][heads][page][value + 64], v_cache fp16 [pages][heads][value][page], expanded_table
    int32 [sequences][cols] (value 64 or 128).  Positions firsts[s] (int32 [S]; None: 0) to lengths[s] - 1 are written.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return q4g128_latent_expand(cache, table, lengths, packed, scales, mins, k_cache, v_cache, expanded_table,
                                        firsts, max_length)
    _check(_binding.latent_expand(cache, table, lengths, packed, scales, mins, k_cache, v_cache, expanded_table, firsts,
                                  max_length), "q4g128_latent_expand")


def q4g128_latent_prefill_workspace(tokens, count, heads, value, max_length) -> int:
    """Bytes of workspace that q4g128_latent_prefill needs (0: none)."""
    return _lib.q4g128_latent_prefill_workspace(tokens, count, heads, value, max_length)


def q4g128_latent_prefill(q, k_cache, v_cache, table, q_starts, lengths, scale, max_length=None, out=None, workspace=None,
                          stream=None) -> torch.Tensor:
    """Causal attention of prompt tokens over expanded keys and values: q fp16 [T][heads][value + 64] -> out fp16
    [T][heads][value].  Caches as q4g128_latent_expand, other arguments as q4g128_attn_prefill."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return q4g128_latent_prefill(q, k_cache, v_cache, table, q_starts, lengths, scale, max_length, out, workspace)
    return _answer(_binding.latent_prefill(q, k_cache, v_cache, table, q_starts, lengths, scale, max_length, out,
                                           workspace), "q4g128_latent_prefill")


def q4g128_status_string(status: int) -> str:
    return _lib.q4g128_status_string(status).decode()
