"""Python binding of libbitnet_w2a8.so (MI355X / gfx950 W2A8 ternary product).

Argument marshalling only: every step of the path runs in the library's HIP
kernels or, for the offline packer, in its host C++ code.  torch supplies
device memory and streams.  The C ABI and the tile layout are specified in
``include/bitnet_w2a8.h``; the functions below carry the same names.

If the library is not built, every call raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbitnet_w2a8.so")

BITNET_OK, BITNET_ERR_INVALID_ARG, BITNET_ERR_UNSUPPORTED_SHAPE, BITNET_ERR_HIP = 0, 1, 2, 3
BITNET_DT_BF16, BITNET_DT_F32, BITNET_DT_F32_FOLD2, BITNET_DT_F32_RELU2_GLU = 0, 1, 2, 3
BITNET_JUNCTION_NONE, BITNET_JUNCTION_SUM, BITNET_JUNCTION_RELU2_GLU = 0, 1, 2
BITNET_ACT_NONE, BITNET_ACT_RELU, BITNET_ACT_RELU2, BITNET_ACT_SILU, BITNET_ACT_GELU = 0, 1, 2, 3, 4
_ACTS = {None: 0, "none": 0, "relu": 1, "relu2": 2, "silu": 3, "gelu": 4}
_JUNCTIONS = {False: 0, None: 0, "none": 0, True: 1, "sum": 1, "relu2_glu": 2, 0: 0, 1: 1, 2: 2}


def junction_code(j) -> int:
    """Junction of a two-half input: False/None/"none" -> 0, True/"sum" -> 1 (lo + hi),
    "relu2_glu" -> 2 (relu(lo)^2 * hi); the integers 0..2 map to themselves."""
    try:
        return _JUNCTIONS[j]
    except (KeyError, TypeError):
        raise ValueError(f"unknown junction {j!r}") from None
BLOCK_K = 128
TILE_N = 16
GEMV_MAX_M = 16


class BitnetError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {bitnet_status_str(status)} (status {status})")
        self.status = status


_lib = None

_SIGS = {
    "bitnet_status_str": ([ctypes.c_int], ctypes.c_char_p),
    "bitnet_check_shape": ([ctypes.c_int64, ctypes.c_int64], ctypes.c_int),
    "bitnet_gemv_split": ([ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                           ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)], ctypes.c_int),
    "bitnet_packed_bytes": ([ctypes.c_int64, ctypes.c_int64], ctypes.c_size_t),
    "bitnet_scale_count": ([ctypes.c_int64, ctypes.c_int64], ctypes.c_size_t),
    "bitnet_ternarize_absmean": ([ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                  ctypes.c_void_p], ctypes.c_int),
    "bitnet_pack_i2s": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                         ctypes.c_void_p], ctypes.c_int),
    "bitnet_repack_i2s": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                           ctypes.c_void_p], ctypes.c_int),
    "bitnet_unpack_i2s": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                           ctypes.c_void_p], ctypes.c_int),
    "bitnet_quant_act": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                          ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "bitnet_quant_act_fold": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                               ctypes.c_void_p], ctypes.c_int),
    "bitnet_quant_act_relu2_glu": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_void_p], ctypes.c_int),
    "bitnet_w2a8_gemv": ([ctypes.c_void_p] * 5 + [ctypes.c_int] * 3 + [ctypes.c_void_p], ctypes.c_int),
    "bitnet_w2a8_gemm": ([ctypes.c_void_p] * 5 + [ctypes.c_int] * 4 + [ctypes.c_void_p], ctypes.c_int),
    "bitnet_scale_count_g": ([ctypes.c_int64, ctypes.c_int64, ctypes.c_int], ctypes.c_size_t),
    "bitnet_probe_stream_read_sink_len": ([ctypes.c_size_t], ctypes.c_size_t),
    "bitnet_probe_stream_read": ([ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int,
                                  ctypes.c_void_p], ctypes.c_int),
    "bitnet_ternarize_absmean_g": ([ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                    ctypes.c_void_p], ctypes.c_int),
    "bitnet_pack_i2s_g": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                           ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "bitnet_repack_i2s_g": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                             ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "bitnet_unpack_i2s_g": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                             ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "bitnet_w2a8_gemv_g": ([ctypes.c_void_p] * 5 + [ctypes.c_int] * 4 + [ctypes.c_void_p], ctypes.c_int),
    "bitnet_w2a8_gemm_g": ([ctypes.c_void_p] * 5 + [ctypes.c_int] * 5 + [ctypes.c_void_p], ctypes.c_int),
    "bitnet_w2a8_gemv_act": ([ctypes.c_void_p] * 3 + [ctypes.c_int] + [ctypes.c_void_p] * 3 + [ctypes.c_int] * 3
                             + [ctypes.c_void_p], ctypes.c_int),
    "bitnet_w2a8_acc_i32": ([ctypes.c_void_p] * 3 + [ctypes.c_int] * 3 + [ctypes.c_void_p], ctypes.c_int),
    "bitnet_w2a8_gemv_lut": ([ctypes.c_void_p] * 6 + [ctypes.c_int] * 3 + [ctypes.c_void_p], ctypes.c_int),
    "bitnet_w2a8_chain_workspace_bytes": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_int], ctypes.c_size_t),
    "bitnet_w2a8_chain": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                           ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p], ctypes.c_int),
    "bitnet_w2a8_chain_static_max_bytes": ([], ctypes.c_size_t),
    "bitnet_w2a8_persist_table_bytes": ([ctypes.c_int], ctypes.c_size_t),
    "bitnet_w2a8_persist_prepare": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int64,
                                     ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
    "bitnet_w2a8_chain_persistent": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p], ctypes.c_int),
    "bitnet_w2a8_chain_persistent_ex": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                                         ctypes.c_void_p], ctypes.c_int),
    "bitnet_w2a8_chain_static": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                  ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "bitnet_kv_cache_bytes": ([ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int], ctypes.c_size_t),
    "bitnet_rope_table": ([ctypes.c_int64, ctypes.c_int, ctypes.c_double, ctypes.c_double, ctypes.c_int64,
                           ctypes.c_void_p], ctypes.c_int),
    "bitnet_rope_append_kv": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                               ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                               ctypes.c_int, ctypes.c_int] + [ctypes.c_void_p] * 4, ctypes.c_int),
    "bitnet_attn_decode_workspace_bytes": ([ctypes.c_int] * 5, ctypes.c_size_t),
    "bitnet_attn_decode": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                            ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                            ctypes.c_size_t, ctypes.c_void_p], ctypes.c_int),
    "bitnet_attn_prompt": ([ctypes.c_void_p, ctypes.c_int64] * 3 + [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64]
                           + [ctypes.c_int] * 5 + [ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "bitnet_add_norm": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                         ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_int, ctypes.c_int]
                        + [ctypes.c_void_p] * 4 + [ctypes.c_int, ctypes.c_void_p], ctypes.c_int),
    "bitnet_w2a8_linear": ([ctypes.c_void_p] * 5 + [ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]
                           + [ctypes.c_int] * 4 + [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p], ctypes.c_int),
    "bitnet_w2a8_linear_workspace_bytes": ([ctypes.c_int] * 3, ctypes.c_size_t),
    "bitnet_w2a8_grouped_workspace_bytes": ([ctypes.c_int] * 5, ctypes.c_size_t),
    "bitnet_w2a8_grouped": ([ctypes.c_void_p] * 4 + [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                             ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p] + [ctypes.c_int] * 3
                            + [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p], ctypes.c_int),
    "bitnet_route_workspace_bytes": ([ctypes.c_int] * 3, ctypes.c_size_t),
    "bitnet_route": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_int64] + [ctypes.c_int] * 4 + [ctypes.c_void_p] * 6
                     + [ctypes.c_size_t, ctypes.c_void_p], ctypes.c_int),
}


class KVCacheStruct(ctypes.Structure):
    """bitnet_kv_cache_t"""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("table", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("page", ctypes.c_int),
                ("batch", ctypes.c_int), ("slots", ctypes.c_int)]


class ChainLayer(ctypes.Structure):
    """bitnet_chain_layer_t"""
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("fold_input", ctypes.c_int)]


def lib():
    """The loaded library (ctypes.CDLL).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        # The kernels must run on the HIP runtime that owns the device memory and
        # streams passed in.  torch bundles its own libamdhip64 under the same
        # soname; with torch loaded first the dynamic linker binds this library to
        # that copy, while loading this library first would map the system runtime
        # and torch would then load a second one beside it.
        try:
            import torch  # noqa: F401
        except ImportError:
            pass
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"HIP library not built: {LIB_PATH} is missing "
                               "(run `python -m bit_gemv_i2_amd.build`)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _lib = handle
    return _lib


def _ok(status: int, what: str):
    if status != BITNET_OK:
        raise BitnetError(status, what)


def _np_ptr(a: np.ndarray):
    return a.ctypes.data_as(ctypes.c_void_p)


def _dev_ptr(t, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _check(t, name: str, dtype, numel: int | None = None, shape: tuple | None = None):
    """Raises ValueError unless tensor t has the given dtype and exactly `numel`
    elements (or exactly `shape`).  Runs on metadata only, before any pointer is
    taken or any launch is made: a buffer whose size disagrees with the library's
    size authorities (bitnet_packed_bytes, bitnet_scale_count[_g], M*K, M*N) is
    never handed to a kernel."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, not {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} elements, not {t.numel()}")


def _check_weights(packed, scales, N: int, K: int, scale_block: int = 128):
    """packed / scales against bitnet_packed_bytes and bitnet_scale_count[_g]."""
    import torch
    nb = bitnet_packed_bytes(N, K)
    ns = bitnet_scale_count(N, K) if scale_block == 128 else bitnet_scale_count_g(N, K, scale_block)
    if nb == 0 or ns == 0:
        raise BitnetError(BITNET_ERR_UNSUPPORTED_SHAPE if nb == 0 else BITNET_ERR_INVALID_ARG,
                          f"weights of shape {N} x {K} (scale_block {scale_block})")
    _check(packed, "packed", torch.uint8, numel=nb)
    if scales is not None:
        _check(scales, "scales", torch.float32, numel=ns)


def _check_acts(q, s_a, K: int):
    """q int8 [M][K] and s_a fp32 [M]; returns M."""
    import torch
    if q.dim() != 2 or q.shape[1] != K:
        raise ValueError(f"q must be [M][{K}], not {tuple(q.shape)}")
    _check(q, "q", torch.int8)
    M = q.shape[0]
    if s_a is not None:
        _check(s_a, "s_a", torch.float32, numel=M)
    return M


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# ------------------------------------------------------------------ sizes
def bitnet_status_str(status: int) -> str:
    return lib().bitnet_status_str(int(status)).decode()


def bitnet_check_shape(N: int, K: int) -> int:
    return lib().bitnet_check_shape(N, K)


def bitnet_gemv_split(N: int, K: int, cus: int = 0, wave_slots: int = 0):
    """(waves per 16-row workgroup, 128-weight blocks per wave) of the decode products for an
    N x K matrix on a device with `cus` CUs holding `wave_slots` waves (0, 0: the base split)."""
    w, p = ctypes.c_int(0), ctypes.c_int(0)
    _ok(lib().bitnet_gemv_split(int(N), int(K), int(cus), int(wave_slots), ctypes.byref(w), ctypes.byref(p)),
        "bitnet_gemv_split")
    return w.value, p.value


def bitnet_packed_bytes(N: int, K: int) -> int:
    return lib().bitnet_packed_bytes(N, K)


def bitnet_scale_count(N: int, K: int) -> int:
    return lib().bitnet_scale_count(N, K)


# ------------------------------------------------------------------ offline, host
def bitnet_ternarize_absmean(w: np.ndarray):
    """fp32 [N][K] -> (ternary int8 [N][K], scales fp32 [N][K/128])."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    N, K = w.shape
    t = np.empty((N, K), np.int8)
    s = np.empty((N, K // BLOCK_K), np.float32)
    _ok(lib().bitnet_ternarize_absmean(_np_ptr(w), N, K, _np_ptr(t), _np_ptr(s)), "bitnet_ternarize_absmean")
    return t, s


def bitnet_pack_i2s(ternary: np.ndarray, scales: np.ndarray):
    """ternary int8 [N][K], scales fp32 [N][K/128] -> (packed uint8 [N*K/4], tiled scales fp32 [N*K/128])."""
    ternary = np.ascontiguousarray(ternary, dtype=np.int8)
    scales = np.ascontiguousarray(scales, dtype=np.float32)
    N, K = ternary.shape
    if scales.shape != (N, K // BLOCK_K):
        raise ValueError("scales must be [N][K/128]")
    nb = bitnet_packed_bytes(N, K)
    if nb == 0:
        raise BitnetError(BITNET_ERR_UNSUPPORTED_SHAPE, "bitnet_pack_i2s")
    packed = np.empty(nb, np.uint8)
    st = np.empty(bitnet_scale_count(N, K), np.float32)
    _ok(lib().bitnet_pack_i2s(_np_ptr(ternary), _np_ptr(scales), N, K, _np_ptr(packed), _np_ptr(st)),
        "bitnet_pack_i2s")
    return packed, st


def bitnet_repack_i2s(i2s: np.ndarray, scales: np.ndarray, K: int):
    """canonical i2_s bytes uint8 [N][K/4] + scales [N][K/128] -> (packed, tiled scales)."""
    i2s = np.ascontiguousarray(i2s, dtype=np.uint8)
    scales = np.ascontiguousarray(scales, dtype=np.float32)
    N = i2s.shape[0]
    if i2s.shape != (N, K // 4) or scales.shape != (N, K // BLOCK_K):
        raise ValueError("bad i2s / scales shape")
    nb = bitnet_packed_bytes(N, K)
    if nb == 0:
        raise BitnetError(BITNET_ERR_UNSUPPORTED_SHAPE, "bitnet_repack_i2s")
    packed = np.empty(nb, np.uint8)
    st = np.empty(bitnet_scale_count(N, K), np.float32)
    _ok(lib().bitnet_repack_i2s(_np_ptr(i2s), _np_ptr(scales), N, K, _np_ptr(packed), _np_ptr(st)),
        "bitnet_repack_i2s")
    return packed, st


def bitnet_unpack_i2s(packed: np.ndarray, scales_tiled: np.ndarray | None, N: int, K: int):
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    t = np.empty((N, K), np.int8)
    s = None
    sp = None
    if scales_tiled is not None:
        scales_tiled = np.ascontiguousarray(scales_tiled, dtype=np.float32)
        s = np.empty((N, K // BLOCK_K), np.float32)
        sp = _np_ptr(scales_tiled)
    _ok(lib().bitnet_unpack_i2s(_np_ptr(packed), sp, N, K, _np_ptr(t), None if s is None else _np_ptr(s)),
        "bitnet_unpack_i2s")
    return t, s


# ------------------------------------------------------------------ scale granularity
# scale_block: 128 (x86 i2_s blocks, the default everywhere else), 64 (ARM
# blocks) or 0 (one scale for the whole matrix).
def scale_shape(N: int, K: int, scale_block: int):
    return (1,) if scale_block == 0 else (N, K // scale_block)


def bitnet_scale_count_g(N: int, K: int, scale_block: int) -> int:
    return lib().bitnet_scale_count_g(N, K, scale_block)


def bitnet_ternarize_absmean_g(w: np.ndarray, scale_block: int):
    """fp32 [N][K] -> (ternary int8 [N][K], scales fp32 scale_shape(N, K, scale_block))."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    N, K = w.shape
    t = np.empty((N, K), np.int8)
    s = np.empty(scale_shape(N, K, scale_block), np.float32)
    _ok(lib().bitnet_ternarize_absmean_g(_np_ptr(w), N, K, scale_block, _np_ptr(t), _np_ptr(s)),
        "bitnet_ternarize_absmean_g")
    return t, s


def _pack_g(name, src, scales, N, K, scale_block):
    scales = np.ascontiguousarray(scales, dtype=np.float32)
    if scales.shape != scale_shape(N, K, scale_block):
        raise ValueError("scales must have shape %s" % (scale_shape(N, K, scale_block),))
    nb, ns = bitnet_packed_bytes(N, K), bitnet_scale_count_g(N, K, scale_block)
    if nb == 0 or ns == 0:
        raise BitnetError(BITNET_ERR_UNSUPPORTED_SHAPE, name)
    packed = np.empty(nb, np.uint8)
    st = np.empty(ns, np.float32)
    _ok(getattr(lib(), name)(_np_ptr(src), _np_ptr(scales), N, K, scale_block, _np_ptr(packed), _np_ptr(st)), name)
    return packed, st


def bitnet_pack_i2s_g(ternary: np.ndarray, scales: np.ndarray, scale_block: int):
    """As bitnet_pack_i2s, scales of shape scale_shape(N, K, scale_block)."""
    ternary = np.ascontiguousarray(ternary, dtype=np.int8)
    N, K = ternary.shape
    return _pack_g("bitnet_pack_i2s_g", ternary, scales, N, K, scale_block)


def bitnet_repack_i2s_g(i2s: np.ndarray, scales: np.ndarray, K: int, scale_block: int):
    """Canonical bytes of the given format uint8 [N][K/4] + scales -> (packed, tiled scales)."""
    i2s = np.ascontiguousarray(i2s, dtype=np.uint8)
    N = i2s.shape[0]
    if i2s.shape != (N, K // 4):
        raise ValueError("bad i2s shape")
    return _pack_g("bitnet_repack_i2s_g", i2s, scales, N, K, scale_block)


def bitnet_unpack_i2s_g(packed: np.ndarray, scales_tiled, N: int, K: int, scale_block: int):
    packed = np.ascontiguousarray(packed, dtype=np.uint8)
    t = np.empty((N, K), np.int8)
    s = sp = None
    if scales_tiled is not None:
        scales_tiled = np.ascontiguousarray(scales_tiled, dtype=np.float32)
        s = np.empty(scale_shape(N, K, scale_block), np.float32)
        sp = _np_ptr(scales_tiled)
    _ok(lib().bitnet_unpack_i2s_g(_np_ptr(packed), sp, N, K, scale_block, _np_ptr(t),
                                  None if s is None else _np_ptr(s)), "bitnet_unpack_i2s_g")
    return t, s


# ------------------------------------------------------------------ device, async
def bitnet_quant_act(x, q=None, s_a=None, stream=None):
    """x: device [M][K] bf16 or fp32 -> (q int8 [M][K], s_a fp32 [M])."""
    import torch
    M, K = x.shape
    xdt = {torch.bfloat16: BITNET_DT_BF16, torch.float32: BITNET_DT_F32}.get(x.dtype)
    if xdt is None:
        raise ValueError("x must be bf16 or fp32")
    if q is None:
        q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if s_a is None:
        s_a = torch.empty((M,), dtype=torch.float32, device=x.device)
    _check(q, "q", torch.int8, numel=M * K)
    _check(s_a, "s_a", torch.float32, numel=M)
    _ok(lib().bitnet_quant_act(_dev_ptr(x, "x"), xdt, M, K, _dev_ptr(q, "q"), _dev_ptr(s_a, "s_a"),
                               _stream(stream)), "bitnet_quant_act")
    return q, s_a


def _quant_two_half(name, y, q, s_a, stream):
    import torch
    M, H2 = y.shape
    H = H2 // 2
    if y.dtype != torch.float32 or H2 % 2:
        raise ValueError("y must be fp32 [M][2H]")
    if q is None:
        q = torch.empty((M, H), dtype=torch.int8, device=y.device)
    if s_a is None:
        s_a = torch.empty((M,), dtype=torch.float32, device=y.device)
    _check(q, "q", torch.int8, numel=M * H)
    _check(s_a, "s_a", torch.float32, numel=M)
    _ok(getattr(lib(), name)(_dev_ptr(y, "y"), M, H, _dev_ptr(q, "q"), _dev_ptr(s_a, "s_a"), _stream(stream)), name)
    return q, s_a


def bitnet_quant_act_fold(y, q=None, s_a=None, stream=None):
    """y: device fp32 [M][2H] -> h = y[:, :H] + y[:, H:] quantised: (q int8 [M][H], s_a fp32 [M])."""
    return _quant_two_half("bitnet_quant_act_fold", y, q, s_a, stream)


def bitnet_quant_act_relu2_glu(y, q=None, s_a=None, stream=None):
    """y: device fp32 [M][2H] (gate | up) -> h = relu(gate)^2 * up quantised: (q int8 [M][H], s_a fp32 [M])."""
    return _quant_two_half("bitnet_quant_act_relu2_glu", y, q, s_a, stream)


def bitnet_w2a8_gemv(packed, scales, q, s_a, N: int, K: int, y=None, stream=None):
    """Decode product (M <= 16): y fp32 [M][N]."""
    import torch
    _check_weights(packed, scales, N, K)
    M = _check_acts(q, s_a, K)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=q.device)
    _check(y, "y", torch.float32, numel=M * N)
    _ok(lib().bitnet_w2a8_gemv(_dev_ptr(packed, "packed"), _dev_ptr(scales, "scales"), _dev_ptr(q, "q"),
                               _dev_ptr(s_a, "s_a"), _dev_ptr(y, "y"), M, N, K, _stream(stream)),
        "bitnet_w2a8_gemv")
    return y


def bitnet_w2a8_gemv_act(packed, scales, x, N: int, K: int, fold: bool = False, y=None, q_out=None,
                         s_a_out=None, stream=None):
    """Decode step in one launch: quantise x (bf16/fp32 [M][K], or fp32 [M][2K]
    brought to width K by a junction: fold=True or "sum" for lo + hi,
    "relu2_glu" for relu(lo)^2 * hi) and multiply.  Optional q_out / s_a_out
    receive the int8 activations and dequant factors.  Returns y fp32 [M][N]."""
    import torch
    M = x.shape[0]
    jc = junction_code(fold)
    if jc:
        if x.dtype != torch.float32 or x.shape[1] != 2 * K:
            raise ValueError("a junction needs fp32 x of shape [M][2K]")
        xdt = BITNET_DT_F32_FOLD2 if jc == BITNET_JUNCTION_SUM else BITNET_DT_F32_RELU2_GLU
    else:
        xdt = {torch.bfloat16: BITNET_DT_BF16, torch.float32: BITNET_DT_F32}.get(x.dtype)
        if xdt is None or x.shape[1] != K:
            raise ValueError("x must be bf16 or fp32 [M][K]")
    _check_weights(packed, scales, N, K)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _check(y, "y", torch.float32, numel=M * N)
    if q_out is not None:
        _check(q_out, "q_out", torch.int8, numel=M * K)
    if s_a_out is not None:
        _check(s_a_out, "s_a_out", torch.float32, numel=M)
    qp = None if q_out is None else _dev_ptr(q_out, "q_out")
    sp = None if s_a_out is None else _dev_ptr(s_a_out, "s_a_out")
    _ok(lib().bitnet_w2a8_gemv_act(_dev_ptr(packed, "packed"), _dev_ptr(scales, "scales"), _dev_ptr(x, "x"), xdt,
                                   _dev_ptr(y, "y"), qp, sp, M, N, K, _stream(stream)), "bitnet_w2a8_gemv_act")
    return y


def bitnet_w2a8_gemm(packed, scales, q, s_a, N: int, K: int, out_dtype=None, y=None, stream=None):
    """Prefill product (any M): y [M][N] in bf16 (default) or fp32."""
    import torch
    _check_weights(packed, scales, N, K)
    M = _check_acts(q, s_a, K)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if y is None else y.dtype
    ydt = {torch.bfloat16: BITNET_DT_BF16, torch.float32: BITNET_DT_F32}.get(out_dtype)
    if ydt is None:
        raise ValueError("out_dtype must be bf16 or fp32")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=q.device)
    _check(y, "y", out_dtype, numel=M * N)
    _ok(lib().bitnet_w2a8_gemm(_dev_ptr(packed, "packed"), _dev_ptr(scales, "scales"), _dev_ptr(q, "q"),
                               _dev_ptr(s_a, "s_a"), _dev_ptr(y, "y"), ydt, M, N, K, _stream(stream)),
        "bitnet_w2a8_gemm")
    return y


def bitnet_w2a8_gemv_g(packed, scales, q, s_a, N: int, K: int, scale_block: int, y=None, stream=None):
    """Decode product at scale granularity scale_block (tiled scales of bitnet_pack_i2s_g)."""
    import torch
    _check_weights(packed, scales, N, K, scale_block)
    M = _check_acts(q, s_a, K)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=q.device)
    _check(y, "y", torch.float32, numel=M * N)
    _ok(lib().bitnet_w2a8_gemv_g(_dev_ptr(packed, "packed"), _dev_ptr(scales, "scales"), _dev_ptr(q, "q"),
                                 _dev_ptr(s_a, "s_a"), _dev_ptr(y, "y"), M, N, K, scale_block, _stream(stream)),
        "bitnet_w2a8_gemv_g")
    return y


def bitnet_w2a8_gemm_g(packed, scales, q, s_a, N: int, K: int, scale_block: int, out_dtype=None, y=None,
                       stream=None):
    """Prefill product at scale granularity scale_block."""
    import torch
    _check_weights(packed, scales, N, K, scale_block)
    M = _check_acts(q, s_a, K)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if y is None else y.dtype
    ydt = {torch.bfloat16: BITNET_DT_BF16, torch.float32: BITNET_DT_F32}.get(out_dtype)
    if ydt is None:
        raise ValueError("out_dtype must be bf16 or fp32")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=q.device)
    _check(y, "y", out_dtype, numel=M * N)
    _ok(lib().bitnet_w2a8_gemm_g(_dev_ptr(packed, "packed"), _dev_ptr(scales, "scales"), _dev_ptr(q, "q"),
                                 _dev_ptr(s_a, "s_a"), _dev_ptr(y, "y"), ydt, M, N, K, scale_block,
                                 _stream(stream)), "bitnet_w2a8_gemm_g")
    return y


def bitnet_w2a8_acc_i32(packed, q, N: int, K: int, acc=None, stream=None):
    """Exact int32 product acc [M][N] through the decode (M <= 16) or prefill kernel."""
    import torch
    _check_weights(packed, None, N, K)
    M = _check_acts(q, None, K)
    if acc is None:
        acc = torch.empty((M, N), dtype=torch.int32, device=q.device)
    _check(acc, "acc", torch.int32, numel=M * N)
    _ok(lib().bitnet_w2a8_acc_i32(_dev_ptr(packed, "packed"), _dev_ptr(q, "q"), _dev_ptr(acc, "acc"), M, N, K,
                                  _stream(stream)), "bitnet_w2a8_acc_i32")
    return acc


def bitnet_w2a8_gemv_lut(packed, scales, q, s_a, N: int, K: int, tiles_per_group: int = 0, y=None, acc=None,
                         with_acc: bool = False, stream=None):
    """Table-lookup decode product for one token: y fp32 [1][N] (and, with
    with_acc or a given acc, the exact int32 sums [1][N]).  Returns y, or (y, acc)."""
    import torch
    if q.dim() != 2 or q.shape[0] != 1:
        raise ValueError("q must be int8 [1][K]")
    _check_weights(packed, scales, N, K)
    _check_acts(q, s_a, K)
    if y is None:
        y = torch.empty((1, N), dtype=torch.float32, device=q.device)
    if acc is None and with_acc:
        acc = torch.empty((1, N), dtype=torch.int32, device=q.device)
    _check(y, "y", torch.float32, numel=N)
    if acc is not None:
        _check(acc, "acc", torch.int32, numel=N)
    accp = _dev_ptr(acc, "acc") if acc is not None else None
    _ok(lib().bitnet_w2a8_gemv_lut(_dev_ptr(packed, "packed"), _dev_ptr(scales, "scales"), _dev_ptr(q, "q"),
                                   _dev_ptr(s_a, "s_a"), _dev_ptr(y, "y"), accp, N, K, tiles_per_group,
                                   _stream(stream)), "bitnet_w2a8_gemv_lut")
    return (y, acc) if acc is not None else y


# ------------------------------------------------------------------ attention side of a decoder layer
def bitnet_kv_cache_bytes(pages: int, kv_heads: int, head_dim: int, page: int) -> int:
    for n, name in ((kv_heads, "kv_heads"), (head_dim, "head_dim"), (page, "page")):
        _bound(n, name)
    return lib().bitnet_kv_cache_bytes(int(pages), int(kv_heads), int(head_dim), int(page))


def bitnet_rope_table(positions: int, rot: int, base: float = 10000.0, factor: float = 1.0, trained: int = 0):
    """Rotary table, fp32 numpy [positions][rot] (cosines, then sines).  factor > 1 stretches the
    positions: all rates by 1/factor, or by parts when `trained` gives the context length of the training."""
    if positions < 1 or rot < 1:
        raise BitnetError(BITNET_ERR_UNSUPPORTED_SHAPE, "bitnet_rope_table")
    _bound(positions, "positions")
    _bound(rot, "rot")
    if not -1 << 63 <= trained < 1 << 63:
        raise ValueError("trained must be below 2^63")
    t = np.empty((positions, rot), np.float32)
    _ok(lib().bitnet_rope_table(int(positions), int(rot), float(base), float(factor), int(trained), _np_ptr(t)),
        "bitnet_rope_table")
    return t


_torch = None


def _import_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _cache_struct(torch, k_cache, v_cache, k_scale, v_scale, table):
    """(bitnet_kv_cache_t over the given tensors, their device index), each tensor checked against the layout of the
    header.  One combined test first: a serving step makes this call for every layer."""
    i8, f32 = torch.int8, torch.float32
    dev = k_cache.get_device()
    if k_cache.dim() == 4 and table.dim() == 2:
        pages, heads, page, dim = k_cache.shape
        per_page = (pages, heads)
        if (k_cache.dtype is i8 and v_cache.dtype is i8 and k_scale.dtype is f32 and v_scale.dtype is f32
                and table.dtype is torch.int32 and v_cache.shape == (pages, heads, dim, page)
                and k_scale.shape == per_page and v_scale.shape == per_page
                and dev == v_cache.get_device() == k_scale.get_device() == v_scale.get_device() == table.get_device()
                and dev >= 0 and k_cache.is_contiguous() and v_cache.is_contiguous() and k_scale.is_contiguous()
                and v_scale.is_contiguous() and table.is_contiguous()):
            batch, slots = table.shape
            return KVCacheStruct(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                 table.data_ptr(), pages, heads, dim, page, batch, slots), dev
    # something is wrong: say what
    if k_cache.dim() != 4 or table.dim() != 2:
        raise ValueError("k_cache must be [pages][kv_heads][page][head_dim] and table [batch][slots]")
    pages, heads, page, dim = k_cache.shape
    _check(k_cache, "k_cache", i8)
    _check(v_cache, "v_cache", i8, shape=(pages, heads, dim, page))
    _check(k_scale, "k_scale", f32, shape=(pages, heads))
    _check(v_scale, "v_scale", f32, shape=(pages, heads))
    _check(table, "table", torch.int32)
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache"), (k_scale, "k_scale"), (v_scale, "v_scale"),
                    (table, "table")):
        _on_device(t, name, dev)
    raise ValueError("the cache's tensors do not fit together")


def _on_device(t, name: str, dev: int, dtype=None, shape=None):
    """Pointer of a contiguous tensor on device `dev`, of the given dtype and shape where they are named."""
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a device tensor" if t.get_device() < 0 else
                         f"{name} must be on the device of the other tensors")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if (dtype is not None and t.dtype is not dtype) or (shape is not None and t.shape != shape):
        _check(t, name, dtype, shape=shape)
    return t.data_ptr()


def _launch_stream(torch, stream, dev: int):
    """The stream handle of a launch on device `dev`, which has to be the current one and the stream's."""
    if torch._C._cuda_getDevice() != dev:
        raise ValueError(f"the tensors are on device {dev}, the current device is {torch._C._cuda_getDevice()}")
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"the tensors are on device {dev}, the stream is of device {stream.device.index}")
    # the handle alone: current_stream() builds an object around it, for as long as a launch takes
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _rows_ptr(t, name: str, inner: int, dev: int):
    """(pointer, elements from row to row) of a device tensor whose rows hold `inner` elements side by side:
    contiguous, or a slice of wider rows."""
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a device tensor" if t.get_device() < 0 else
                         f"{name} must be on the device of the other tensors")
    if t.is_contiguous():
        return t.data_ptr(), inner
    stride = t.stride()
    if len(stride) == 3 and stride[2] == 1 and stride[1] == t.shape[2] and t.shape[0] > 1:
        return t.data_ptr(), stride[0]
    want = 1
    for size, step in zip(reversed(t.shape[1:]), reversed(stride[1:])):
        if size != 1 and step != want:
            raise ValueError(f"{name} must have its heads and channels side by side in a row")
        want *= size
    return t.data_ptr(), stride[0] if t.shape[0] > 1 else inner


def _empty(torch, like, shape, dtype, stream):
    """Memory on `like`'s device for a call on `stream`, taken from that stream's pool so that nothing still pending
    elsewhere uses it."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _bound(n: int, name: str):
    """ctypes would cut a count to its low 32 bits without a word."""
    if not -0x80000000 <= n <= 0x7FFFFFFF:
        raise ValueError(f"{name} must be below 2^31 and not below -2^31")


def _float_dt(torch, t, name: str) -> int:
    if t.dtype is torch.bfloat16:
        return BITNET_DT_BF16
    if t.dtype is torch.float32:
        return BITNET_DT_F32
    raise ValueError(f"{name} must be bf16 or fp32")


def bitnet_rope_append_kv(qkv, rope, k_cache, v_cache, k_scale, v_scale, table, starts, before, max_new: int,
                          q_heads: int, interleaved: bool = False, with_k: bool = False, q_out=None, k_out=None,
                          stream=None):
    """Turns the queries and keys of the fused projection qkv [T][(q_heads + 2 kv_heads) * head_dim] by their
    positions and appends keys and values to the paged int8 cache.  rope: fp32 [positions][rot] on the device, or
    None; starts int32 [batch + 1], before int32 [batch].  Returns (q [T][q_heads][head_dim], k or None); k,
    the turned keys, is made when with_k or k_out asks for it."""
    torch = _torch or _import_torch()
    _bound(max_new, "max_new")
    c, dev = _cache_struct(torch, k_cache, v_cache, k_scale, v_scale, table)
    dt = _float_dt(torch, qkv, "qkv")
    hk, dim, batch = c.kv_heads, c.head_dim, c.batch
    width = (q_heads + 2 * hk) * dim
    if qkv.dim() != 2 or qkv.shape[1] != width:
        raise ValueError(f"qkv must be [T][{width}], not {tuple(qkv.shape)}")
    T = qkv.shape[0]
    sp = _on_device(starts, "starts", dev, torch.int32, (batch + 1,))
    bp = _on_device(before, "before", dev, torch.int32, (batch,))
    rot = rows = 0
    rp = None
    if rope is not None:
        if rope.dim() != 2:
            raise ValueError("rope must be [positions][rot]")
        rp = _on_device(rope, "rope", dev, torch.float32)
        rows, rot = rope.shape
    xp, stride = _rows_ptr(qkv, "qkv", width, dev)
    if q_out is None:
        q_out = _empty(torch, qkv, (T, q_heads, dim), qkv.dtype, stream)
    else:
        _check(q_out, "q_out", qkv.dtype, numel=T * q_heads * dim)
    if k_out is not None:
        _check(k_out, "k_out", qkv.dtype, numel=T * hk * dim)
    elif with_k:
        k_out = _empty(torch, qkv, (T, hk, dim), qkv.dtype, stream)
    _ok(lib().bitnet_rope_append_kv(xp, dt, stride, rp, rows, rot, bool(interleaved), sp, bp, T, max_new, q_heads,
                                    ctypes.byref(c), _on_device(q_out, "q_out", dev),
                                    None if k_out is None else _on_device(k_out, "k_out", dev),
                                    _launch_stream(torch, stream, dev)), "bitnet_rope_append_kv")
    return q_out, k_out


def bitnet_attn_decode_workspace_bytes(batch: int, q_heads: int, kv_heads: int, head_dim: int, max_len: int) -> int:
    for n, name in ((batch, "batch"), (q_heads, "q_heads"), (kv_heads, "kv_heads"), (head_dim, "head_dim"), (max_len, "max_len")):
        _bound(n, name)
    return lib().bitnet_attn_decode_workspace_bytes(int(batch), int(q_heads), int(kv_heads), int(head_dim),
                                                    int(max_len))


def bitnet_attn_decode(q, k_cache, v_cache, k_scale, v_scale, table, lengths, max_len: int, scale: float | None = None,
                       out=None, out_dtype=None, workspace=None, stream=None):
    """Attention of one query token per sequence, q [batch][q_heads][head_dim], over the paged int8 cache; `lengths`
    int32 [batch] counts the cached tokens, max_len bounds them.  scale defaults to 1/sqrt(head_dim).  Returns
    [batch][q_heads][head_dim] in out_dtype (q's by default).  The workspace is allocated unless given."""
    torch = _torch or _import_torch()
    _bound(max_len, "max_len")
    c, dev = _cache_struct(torch, k_cache, v_cache, k_scale, v_scale, table)
    qdt = _float_dt(torch, q, "q")
    batch, dim = c.batch, c.head_dim
    if q.dim() != 3 or q.shape[0] != batch or q.shape[2] != dim:
        raise ValueError(f"q must be [{batch}][q_heads][{dim}], not {tuple(q.shape)}")
    hq = q.shape[1]
    qp, stride = _rows_ptr(q, "q", hq * dim, dev)
    lp = _on_device(lengths, "lengths", dev, torch.int32, (batch,))
    if out is None:
        out = _empty(torch, q, (batch, hq, dim), out_dtype or q.dtype, stream)
    else:
        _check(out, "out", out_dtype or out.dtype, numel=batch * hq * dim)
    odt = _float_dt(torch, out, "out")
    need = lib().bitnet_attn_decode_workspace_bytes(batch, hq, c.kv_heads, dim, max_len)
    if workspace is None and need:
        workspace = _empty(torch, q, (need,), torch.uint8, stream)
    wp, nb = None, 0
    if workspace is not None:
        wp, nb = _on_device(workspace, "workspace", dev, torch.uint8), workspace.numel()
        if nb < need:
            raise ValueError(f"workspace must hold at least {need} bytes")
    _ok(lib().bitnet_attn_decode(qp, qdt, stride, ctypes.byref(c), lp, max_len, hq,
                                 dim ** -0.5 if scale is None else scale, _on_device(out, "out", dev), odt, wp, nb,
                                 _launch_stream(torch, stream, dev)), "bitnet_attn_decode")
    return out


def bitnet_attn_prompt(q, k, v, starts, max_len: int, causal: bool = True, scale: float | None = None, out=None,
                       stream=None):
    """Attention over whole prompts packed one behind the other: q [T][q_heads][head_dim], k and v
    [T][kv_heads][head_dim], bf16, tokens at any stride; starts int32 [batch + 1], max_len the longest prompt.
    Returns bf16 [T][q_heads][head_dim]."""
    torch = _torch or _import_torch()
    _bound(max_len, "max_len")
    if q.dim() != 3 or k.dim() != 3 or k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2] or v.shape != k.shape:
        raise ValueError("q must be [T][q_heads][head_dim], k and v [T][kv_heads][head_dim]")
    bf16 = torch.bfloat16
    if q.dtype is not bf16 or k.dtype is not bf16 or v.dtype is not bf16:
        raise ValueError("q, k and v must be bf16")
    if starts.dim() != 1 or starts.shape[0] < 2:
        raise ValueError("starts must be [batch + 1]")
    T, hq, dim = q.shape
    hk = k.shape[1]
    dev = q.get_device()
    qp, qs = _rows_ptr(q, "q", hq * dim, dev)
    kp, ks = _rows_ptr(k, "k", hk * dim, dev)
    vp, vs = _rows_ptr(v, "v", hk * dim, dev)
    sp = _on_device(starts, "starts", dev, torch.int32)
    if out is None:
        out = _empty(torch, q, (T, hq, dim), bf16, stream)
    else:
        _check(out, "out", bf16, numel=T * hq * dim)
    _ok(lib().bitnet_attn_prompt(qp, qs, kp, ks, vp, vs, sp, starts.shape[0] - 1, T, max_len, hq, hk, dim, bool(causal),
                                 dim ** -0.5 if scale is None else scale, _on_device(out, "out", dev),
                                 _launch_stream(torch, stream, dev)), "bitnet_attn_prompt")
    return out


# ------------------------------------------------------------------ between the products of a decoder layer
def _add_norm(name, x, weight, eps, add, slots, gates, x_out, q, s_a, h, h_dtype, stream):
    """The checks and the launch behind bitnet_add_norm_quant (h_dtype None) and bitnet_add_norm."""
    torch = _torch or _import_torch()
    if x.dim() != 2:
        raise ValueError("x must be [M][K]")
    M, K = x.shape
    _bound(M, "M")
    _bound(K, "K")
    dev = x.get_device()
    xp, xdt = _on_device(x, "x", dev), _float_dt(torch, x, "x")
    ap = adt = sp = gp = rows = parts = 0
    if slots is not None and add is None or (slots is None) != (gates is None):
        raise ValueError("slots and gates come together, and with add")
    if add is not None:
        ap, adt = _on_device(add, "add", dev), _float_dt(torch, add, "add")
        if slots is None:
            if add.shape != x.shape:
                raise ValueError(f"add must be [{M}][{K}], not {tuple(add.shape)}")
        else:
            if add.dim() != 2 or add.shape[1] != K or slots.dim() != 2 or slots.shape[0] != M:
                raise ValueError(f"with slots [{M}][parts] add must be [rows][{K}]")
            rows, parts = add.shape[0], slots.shape[1]
            _bound(parts, "parts")
            sp = _on_device(slots, "slots", dev, torch.int32)
            gp = _on_device(gates, "gates", dev, torch.float32, slots.shape)
        if x_out is None:
            x_out = _empty(torch, x, (M, K), x.dtype, stream)
            op = x_out.data_ptr()
        else:
            op = _on_device(x_out, "x_out", dev, x.dtype, x.shape)
    else:
        if x_out is not None:
            raise ValueError("x_out comes with add")
        x_out, op = x, None
    wp = None if weight is None else _on_device(weight, "weight", dev, torch.float32, (K,))
    qp = sap = hp = None
    hdt = 0
    if h_dtype is None:
        if q is None:
            q = _empty(torch, x, (M, K), torch.int8, stream)
            qp = q.data_ptr()
        else:
            qp = _on_device(q, "q", dev, torch.int8, x.shape)
        if s_a is None:
            s_a = _empty(torch, x, (M,), torch.float32, stream)
            sap = s_a.data_ptr()
        else:
            sap = _on_device(s_a, "s_a", dev, torch.float32, (M,))
    else:
        if h is None:
            h = _empty(torch, x, (M, K), h_dtype, stream)
        hp, hdt = _on_device(h, "h", dev, h_dtype, x.shape), _float_dt(torch, h, "h")
    _ok(lib().bitnet_add_norm(xp, xdt, ap or None, adt, rows, sp or None, gp or None, parts, wp, eps, M, K, op, qp, sap, hp, hdt,
                              _launch_stream(torch, stream, dev)), name)
    return q, s_a, h, x_out


def bitnet_add_norm_quant(x, weight=None, eps: float = 1e-5, add=None, slots=None, gates=None, x_out=None, q=None, s_a=None,
                          stream=None):
    """Residual addition, root-mean-square norm and int8 quantisation: x [M][K] bf16 or fp32, plus add [M][K] (or, with
    slots int32 [M][parts] and gates fp32 [M][parts], plus the gated sum of those rows of add [rows][K]).  Returns
    (q int8 [M][K], s_a fp32 [M], the new stream); the last is x itself without add, else x_out (allocated unless given;
    x serves)."""
    q, s_a, _, x_out = _add_norm("bitnet_add_norm_quant", x, weight, eps, add, slots, gates, x_out, q, s_a, None, None, stream)
    return q, s_a, x_out


def bitnet_add_norm(x, weight=None, eps: float = 1e-5, add=None, slots=None, gates=None, x_out=None, out_dtype=None, h=None,
                    stream=None):
    """bitnet_add_norm_quant without the quantiser, as before a product of other types: returns (h [M][K] in out_dtype,
    x's by default, and the new stream).  x itself serves as h where it is not x_out."""
    _, _, h, x_out = _add_norm("bitnet_add_norm", x, weight, eps, add, slots, gates, x_out, None, None, h,
                               out_dtype or (x.dtype if h is None else h.dtype), stream)
    return h, x_out


def _act_code(act) -> int:
    try:
        return _ACTS[act]
    except (KeyError, TypeError):
        raise ValueError(f"unknown activation {act!r}") from None


def _product_ptrs(torch, packed, scales, q, s_a, N, K, matrices):
    """(device, packed, scales, q, s_a pointers, tokens) of `matrices` weights N x K one behind the other and activations."""
    dev = q.get_device()
    pp, sp = _on_device(packed, "packed", dev, torch.uint8), _on_device(scales, "scales", dev, torch.float32)
    if N < 1 or K < 1 or packed.numel() * 4 != matrices * N * K or scales.numel() * 128 != matrices * N * K:
        if bitnet_packed_bytes(_i64(N), _i64(K)) == 0:
            raise BitnetError(BITNET_ERR_UNSUPPORTED_SHAPE, f"weights of shape {N} x {K}")
        _check(packed, "packed", torch.uint8, numel=matrices * N * K // 4)
        _check(scales, "scales", torch.float32, numel=matrices * N * K // 128)
    _bound(N, "N")
    _bound(K, "K")
    if q.dim() != 2 or q.shape[1] != K:
        raise ValueError(f"q must be [M][{K}], not {tuple(q.shape)}")
    M = q.shape[0]
    _bound(M, "M")
    return dev, pp, sp, _on_device(q, "q", dev, torch.int8), _on_device(s_a, "s_a", dev, torch.float32, (M,)), M


def _workspace(torch, given, need: int, like, dev: int, stream):
    """(pointer, bytes) of the workspace given, or of one made where any is needed."""
    if given is None:
        if not need:
            return None, 0
        given = _empty(torch, like, (need,), torch.uint8, stream)
    elif given.numel() < need:
        raise ValueError(f"workspace must hold at least {need} bytes")
    return _on_device(given, "workspace", dev, torch.uint8), given.numel()


def _i64(n: int) -> int:
    if not -1 << 63 <= n < 1 << 63:
        raise ValueError("a size must be below 2^63")
    return n


def bitnet_w2a8_linear(packed, scales, q, s_a, N: int, K: int, bias=None, act="none", gated: bool = False, residual=None,
                       out_dtype=None, y=None, workspace=None, stream=None):
    """W2A8 product with an epilogue, any number of tokens: act(z) + residual, or gated act(z[:, :N/2]) * z[:, N/2:] + residual, with
    z = product + bias.  act: "none", "relu", "relu2", "silu" or "gelu"; bias fp32 [N]; residual bf16 or fp32 of y's shape (y itself
    serves).  Returns y [M][N, or N/2 when gated] in out_dtype (y's, else the residual's, else bf16)."""
    torch = _torch or _import_torch()
    code = _act_code(act)
    dev, pp, sp, qp, sap, M = _product_ptrs(torch, packed, scales, q, s_a, N, K, 1)
    shape = (M, N // 2 if gated else N)
    bp = None if bias is None else _on_device(bias, "bias", dev, torch.float32, (N,))
    rp, rdt = None, 0
    if residual is not None:
        rp, rdt = _on_device(residual, "residual", dev, None, None), _float_dt(torch, residual, "residual")
        if residual.shape != shape:
            raise ValueError(f"residual must be {list(shape)}, not {tuple(residual.shape)}")
    if y is None:
        y = _empty(torch, q, shape, out_dtype or (torch.bfloat16 if residual is None else residual.dtype), stream)
        yp = y.data_ptr()
    else:
        yp = _on_device(y, "y", dev, out_dtype, shape)
    ydt = _float_dt(torch, y, "y")
    wp, nb = _workspace(torch, workspace, lib().bitnet_w2a8_linear_workspace_bytes(M, N, K), q, dev, stream)
    _ok(lib().bitnet_w2a8_linear(pp, sp, qp, sap, bp, code, bool(gated), rp, rdt, yp, ydt, M, N, K, wp, nb,
                                 _launch_stream(torch, stream, dev)), "bitnet_w2a8_linear")
    return y


# ------------------------------------------------------------------ a layer of experts
def bitnet_route_workspace_bytes(tokens: int, experts: int, k: int) -> int:
    for n, name in ((tokens, "tokens"), (experts, "experts"), (k, "k")):
        _bound(n, name)
    return lib().bitnet_route_workspace_bytes(int(tokens), int(experts), int(k))


def bitnet_route(logits, k: int, over_all: bool = False, out=None, workspace=None, stream=None):
    """The k experts of each token and the plan that sorts tokens by expert: logits [T][E] bf16 or fp32, rows at any stride.
    Returns (chosen int32 [T][k], gates fp32 [T][k], starts int32 [E + 1], rows int32 [T * k], slots int32 [T][k]); `out` gives
    these five.  Gates are the softmax of the chosen logits, or with over_all their share of the softmax over all experts."""
    torch = _torch or _import_torch()
    _bound(k, "k")
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be [T][E] with the experts side by side")
    dt = _float_dt(torch, logits, "logits")
    T, E = logits.shape
    _bound(T, "T")
    _bound(E, "E")
    dev = logits.get_device()
    if dev < 0:
        raise ValueError("logits must be a device tensor")
    need = lib().bitnet_route_workspace_bytes(T, E, k)
    if out is None:
        if T < 1 or not 1 <= k <= E:
            raise BitnetError(BITNET_ERR_UNSUPPORTED_SHAPE, "bitnet_route")
        i32 = torch.int32
        out = (_empty(torch, logits, (T, k), i32, stream), _empty(torch, logits, (T, k), torch.float32, stream),
               _empty(torch, logits, (E + 1,), i32, stream), _empty(torch, logits, (T * k,), i32, stream),
               _empty(torch, logits, (T, k), i32, stream))
        ptrs = [t.data_ptr() for t in out]
    else:
        if len(out) != 5:
            raise ValueError("out must be (chosen, gates, starts, rows, slots)")
        shapes = ((T, k), (T, k), (E + 1,), (T * k,), (T, k))
        ptrs = [_on_device(t, n, dev, torch.float32 if n == "gates" else torch.int32, s)
                for t, n, s in zip(out, ("chosen", "gates", "starts", "rows", "slots"), shapes)]
    wp, nb = _workspace(torch, workspace, need, logits, dev, stream)
    _ok(lib().bitnet_route(logits.data_ptr(), dt, logits.stride(0) if T > 1 else E, T, E, k, bool(over_all), *ptrs, wp, nb,
                           _launch_stream(torch, stream, dev)), "bitnet_route")
    return tuple(out)


def bitnet_w2a8_grouped(packed, scales, q, s_a, starts, N: int, K: int, rows=None, bias=None, act="none", gated: bool = False,
                        out_dtype=None, y=None, workspace=None, stream=None):
    """bitnet_w2a8_linear by expert: packed and scales hold the experts' matrices one behind the other, starts int32 [E + 1] says
    which rows of y are whose, rows int32 [slots] which token each is of (without it row i is token i); bias fp32 [E][N].
    Returns y [slots][N, or N/2 when gated] in out_dtype (bf16 by default); rows of no expert are not written."""
    torch = _torch or _import_torch()
    code = _act_code(act)
    if starts.dim() != 1 or starts.shape[0] < 2:
        raise ValueError("starts must be [experts + 1]")
    E = starts.shape[0] - 1
    dev, pp, sp, qp, sap, tokens = _product_ptrs(torch, packed, scales, q, s_a, N, K, E)
    stp = _on_device(starts, "starts", dev, torch.int32)
    rp, slots = None, tokens
    if rows is not None:
        rp = _on_device(rows, "rows", dev, torch.int32)
        slots = rows.numel()
        _bound(slots, "slots")
    shape = (slots, N // 2 if gated else N)
    bp = None if bias is None else _on_device(bias, "bias", dev, torch.float32, (E, N))
    if y is None:
        y = _empty(torch, q, shape, out_dtype or torch.bfloat16, stream)
        yp = y.data_ptr()
    else:
        yp = _on_device(y, "y", dev, out_dtype, shape)
    ydt = _float_dt(torch, y, "y")
    wp, nb = _workspace(torch, workspace, lib().bitnet_w2a8_grouped_workspace_bytes(tokens, slots, E, N, K), q, dev, stream)
    _ok(lib().bitnet_w2a8_grouped(pp, sp, qp, sap, tokens, stp, rp, E, slots, bp, code, bool(gated), yp, ydt, N, K, wp, nb,
                                  _launch_stream(torch, stream, dev)), "bitnet_w2a8_grouped")
    return y


# ------------------------------------------------------------------ convenience
@dataclass
class KVCache:
    """A paged int8 cache resident in device memory, in the layout of bitnet_kv_cache_t."""
    k: object        # torch int8 [pages][kv_heads][page][head_dim]
    v: object        # torch int8 [pages][kv_heads][head_dim][page]
    k_scale: object  # torch fp32 [pages][kv_heads]
    v_scale: object

    @classmethod
    def empty(cls, pages: int, kv_heads: int, head_dim: int, page: int = 64, device="cuda"):
        import torch
        if bitnet_kv_cache_bytes(pages, kv_heads, head_dim, page) == 0:
            raise BitnetError(BITNET_ERR_UNSUPPORTED_SHAPE, "bitnet_kv_cache_bytes")
        return cls(torch.zeros((pages, kv_heads, page, head_dim), dtype=torch.int8, device=device),
                   torch.zeros((pages, kv_heads, head_dim, page), dtype=torch.int8, device=device),
                   torch.zeros((pages, kv_heads), dtype=torch.float32, device=device),
                   torch.zeros((pages, kv_heads), dtype=torch.float32, device=device))

    def append(self, qkv, rope, table, starts, before, max_new, q_heads, **kw):
        return bitnet_rope_append_kv(qkv, rope, self.k, self.v, self.k_scale, self.v_scale, table, starts, before,
                                     max_new, q_heads, **kw)

    def attend(self, q, table, lengths, max_len, **kw):
        return bitnet_attn_decode(q, self.k, self.v, self.k_scale, self.v_scale, table, lengths, max_len, **kw)


@dataclass
class PackedWeight:
    """A ternary weight matrix resident in device memory in the tile layout."""
    packed: object   # torch uint8 [N*K/4] on device
    scales: object   # torch fp32 [N*K/128] on device (tiled order)
    N: int
    K: int

    @classmethod
    def from_ternary(cls, ternary: np.ndarray, scales: np.ndarray, device="cuda"):
        import torch
        p, s = bitnet_pack_i2s(ternary, scales)
        N, K = ternary.shape
        return cls(torch.from_numpy(p).to(device), torch.from_numpy(s).to(device), N, K)

    def gemv(self, q, s_a, y=None, stream=None):
        return bitnet_w2a8_gemv(self.packed, self.scales, q, s_a, self.N, self.K, y=y, stream=stream)

    def gemv_act(self, x, fold=False, y=None, q_out=None, s_a_out=None, stream=None):
        return bitnet_w2a8_gemv_act(self.packed, self.scales, x, self.N, self.K, fold=fold, y=y, q_out=q_out,
                                    s_a_out=s_a_out, stream=stream)

    def gemm(self, q, s_a, out_dtype=None, y=None, stream=None):
        return bitnet_w2a8_gemm(self.packed, self.scales, q, s_a, self.N, self.K, out_dtype=out_dtype, y=y,
                                stream=stream)

    def linear(self, q, s_a, **kw):
        return bitnet_w2a8_linear(self.packed, self.scales, q, s_a, self.N, self.K, **kw)


@dataclass
class PackedExperts:
    """Ternary weight matrices of one shape, an expert each, one behind the other in device memory in the tile layout."""
    packed: object   # torch uint8 [experts * N*K/4] on device
    scales: object   # torch fp32 [experts * N*K/128] on device (tiled order)
    experts: int
    N: int
    K: int

    @classmethod
    def from_ternary(cls, ternary: np.ndarray, scales: np.ndarray, device="cuda"):
        """ternary int8 [experts][N][K], scales fp32 [experts][N][K/128]."""
        import torch
        E, N, K = ternary.shape
        # rows of 16 and their scales lie one behind the other, so the experts are packed as one tall matrix
        p, s = bitnet_pack_i2s(ternary.reshape(E * N, K), scales.reshape(E * N, -1))
        if bitnet_packed_bytes(N, K) == 0:
            raise BitnetError(BITNET_ERR_UNSUPPORTED_SHAPE, "PackedExperts")
        return cls(torch.from_numpy(p).to(device), torch.from_numpy(s).to(device), E, N, K)

    def grouped(self, q, s_a, starts, **kw):
        if starts.shape[0] != self.experts + 1:
            raise ValueError(f"starts must be [{self.experts + 1}]")
        return bitnet_w2a8_grouped(self.packed, self.scales, q, s_a, starts, self.N, self.K, **kw)


# ------------------------------------------------------------------ chained decode
class Chain:
    """A stack of W2A8 layers run by bitnet_w2a8_chain.  `weights` are
    PackedWeight objects; `folds[i]` is the junction in front of layer i
    (False: none; True or "sum": previous output folded h = lo + hi;
    "relu2_glu": h = relu(lo)^2 * hi)."""

    def __init__(self, weights, folds=None):
        self.weights = list(weights)
        self.folds = [0] * len(self.weights) if folds is None else [junction_code(f) for f in folds]
        n = len(self.weights)
        self._arr = (ChainLayer * n)()
        for i, (w, f) in enumerate(zip(self.weights, self.folds)):
            self._arr[i] = ChainLayer(w.packed.data_ptr(), w.scales.data_ptr(), w.N, w.K, int(f))
        self._ws = {}

    def workspace_bytes(self, M: int) -> int:
        return lib().bitnet_w2a8_chain_workspace_bytes(ctypes.cast(self._arr, ctypes.c_void_p), len(self.weights), M)

    def workspace(self, M: int, device="cuda"):
        import torch
        if M not in self._ws:
            nb = self.workspace_bytes(M)
            if nb == 0:
                raise BitnetError(BITNET_ERR_UNSUPPORTED_SHAPE, "bitnet_w2a8_chain_workspace_bytes")
            self._ws[M] = torch.empty(nb, dtype=torch.uint8, device=device)
        return self._ws[M]

    def __call__(self, x, y=None, stream=None):
        import torch
        M = x.shape[0]
        xdt = {torch.bfloat16: BITNET_DT_BF16, torch.float32: BITNET_DT_F32}.get(x.dtype)
        if xdt is None:
            raise ValueError("x must be bf16 or fp32")
        if x.dim() != 2 or x.shape[1] != self.weights[0].K:
            raise ValueError(f"x must be [M][{self.weights[0].K}], not {tuple(x.shape)}")
        if y is None:
            y = torch.empty((M, self.weights[-1].N), dtype=torch.float32, device=x.device)
        _check(y, "y", torch.float32, numel=M * self.weights[-1].N)
        ws = self.workspace(M, x.device)
        _ok(lib().bitnet_w2a8_chain(ctypes.cast(self._arr, ctypes.c_void_p), len(self.weights), _dev_ptr(x, "x"), xdt,
                                    M, _dev_ptr(y, "y"), _dev_ptr(ws, "workspace"), ws.numel(), _stream(stream)),
            "bitnet_w2a8_chain")
        return y


    def plan_persistent(self, M: int = 1, xdt: int = BITNET_DT_BF16, cus: int = 0, device="cuda"):
        key = ("persistent", M, xdt, cus)
        if key not in self._ws:
            self._ws[key] = PersistentPlan(self, M, xdt, cus, device)
        return self._ws[key]

    def persistent(self, x, y=None, stream=None, workspace=None, spin_limit: int = 0, withhold: int = -1):
        """The same decode pass as one persistent launch (bitnet_w2a8_chain_persistent, batch 1).
        Returns y; the workspace (which the binding allocates unless one is given) then
        holds the status word (int32 at offset 0: 0; the layer index + 1 of a wait that
        gave up; minus (layer index + 1) of a table entry that does not fit the workspace)
        and every intermediate layer's output.  spin_limit / withhold are the
        test-only knobs of bitnet_w2a8_chain_persistent_ex."""
        import torch
        M = x.shape[0]
        xdt = {torch.bfloat16: BITNET_DT_BF16, torch.float32: BITNET_DT_F32}.get(x.dtype)
        if xdt is None:
            raise ValueError("x must be bf16 or fp32")
        if x.dim() != 2 or x.shape[1] != self.weights[0].K:
            raise ValueError(f"x must be [M][{self.weights[0].K}], not {tuple(x.shape)}")
        plan = self.plan_persistent(M, xdt, device=x.device)
        if y is None:
            y = torch.empty((M, self.weights[-1].N), dtype=torch.float32, device=x.device)
        _check(y, "y", torch.float32, numel=M * self.weights[-1].N)
        if workspace is None:
            wkey = ("persistent_ws", M, xdt)
            if wkey not in self._ws:
                self._ws[wkey] = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=x.device)
            workspace = self._ws[wkey]
        _check(workspace, "workspace", torch.uint8)
        if workspace.numel() < plan.workspace_bytes:
            raise ValueError(f"workspace must hold at least {plan.workspace_bytes} bytes")
        _ok(lib().bitnet_w2a8_chain_persistent_ex(_dev_ptr(plan.table, "table"), plan.n, _dev_ptr(x, "x"), xdt, M,
                                                  _dev_ptr(y, "y"), _dev_ptr(workspace, "workspace"),
                                                  workspace.numel(), int(spin_limit), int(withhold), _stream(stream)),
            "bitnet_w2a8_chain_persistent")
        return y

    def persistent_layer_outputs(self, M: int = 1, xdt: int = BITNET_DT_BF16, workspace=None):
        """Host views (fp32 [M][N]) of every intermediate layer's output as the last
        persistent call left them in its workspace (the caller's, if one was passed to that
        call, else the binding's), and the status word."""
        plan = self.plan_persistent(M, xdt)
        if workspace is None:
            key = ("persistent_ws", M, xdt)
            if key not in self._ws:
                raise ValueError("no persistent call with the binding's workspace has been made for this batch and type")
            workspace = self._ws[key]
        import torch
        _check(workspace, "workspace", torch.uint8)
        if workspace.numel() < plan.workspace_bytes:
            raise ValueError(f"workspace must hold at least {plan.workspace_bytes} bytes")
        ws = workspace.cpu().numpy()
        table = plan.host_table.view(np.int64).reshape(plan.n, 8)  # out_off is the 4th 8-byte field
        outs = []
        for i in range(plan.n - 1):
            off = int(table[i, 3])
            N = self.weights[i].N
            outs.append(ws[off:off + 4 * M * N].view(np.float32).reshape(M, N).copy())
        return outs, int(ws[:4].view(np.int32)[0])

    def call_static(self, x, y=None, stream=None):
        """The same pass through bitnet_w2a8_chain_static: no workspace is allocated (the
        library's per-GPU array serves), for callers that cannot allocate."""
        import torch
        M = x.shape[0]
        xdt = {torch.bfloat16: BITNET_DT_BF16, torch.float32: BITNET_DT_F32}.get(x.dtype)
        if xdt is None:
            raise ValueError("x must be bf16 or fp32")
        if x.dim() != 2 or x.shape[1] != self.weights[0].K:
            raise ValueError(f"x must be [M][{self.weights[0].K}], not {tuple(x.shape)}")
        if y is None:
            y = torch.empty((M, self.weights[-1].N), dtype=torch.float32, device=x.device)
        _check(y, "y", torch.float32, numel=M * self.weights[-1].N)
        _ok(lib().bitnet_w2a8_chain_static(ctypes.cast(self._arr, ctypes.c_void_p), len(self.weights),
                                           _dev_ptr(x, "x"), xdt, M, _dev_ptr(y, "y"), _stream(stream)),
            "bitnet_w2a8_chain_static")
        return y


class PersistentPlan:
    """The layer table and workspace size of the one-launch (persistent) form of a chain,
    from bitnet_w2a8_persist_prepare (host), with the table copied to the device once:
    the weights' addresses are fixed, so a plan serves every later call."""

    def __init__(self, chain: "Chain", M: int, xdt: int, cus: int = 0, device="cuda"):
        import torch
        n = len(chain.weights)
        nb = lib().bitnet_w2a8_persist_table_bytes(n)
        host = np.zeros(nb, np.uint8)
        ws = ctypes.c_size_t(0)
        _ok(lib().bitnet_w2a8_persist_prepare(ctypes.cast(chain._arr, ctypes.c_void_p), n, M, xdt, cus,
                                              _np_ptr(host), nb, ctypes.byref(ws)), "bitnet_w2a8_persist_prepare")
        self.host_table = host
        self.table = torch.from_numpy(host).to(device)
        self.workspace_bytes = ws.value
        self.n = n


def bitnet_w2a8_chain_static_max_bytes() -> int:
    return lib().bitnet_w2a8_chain_static_max_bytes()


# ------------------------------------------------------------------ measurement helper
def bitnet_probe_stream_read(src, sink=None, mode=0, stream=None):
    """One pass of 16-byte non-temporal loads over the device tensor `src` (not part of
    the product path; the benchmark's attainable-bandwidth reference).  mode 0:
    returns the uint32 sink whose sum (mod 2^32) is the sum of src's 32-bit
    words; mode 1: no output (the read-only floor), the sink is left as it was."""
    import torch
    nbytes = src.numel() * src.element_size()
    nsink = lib().bitnet_probe_stream_read_sink_len(nbytes)
    if sink is None:
        sink = torch.empty((nsink,), dtype=torch.int32, device=src.device)
    _check(sink, "sink", torch.int32)
    if sink.numel() < nsink:
        raise ValueError(f"sink must hold at least {nsink} entries, not {sink.numel()}")
    _ok(lib().bitnet_probe_stream_read(_dev_ptr(src, "src"), nbytes, _dev_ptr(sink, "sink"), sink.numel(), int(mode),
                                       _stream(stream)), "bitnet_probe_stream_read")
    return sink
