"""Python binding of the W4A16 GB300 library (libw4a16.so, C ABI in include/w4a16.h).

The functions here carry the C entry points' names and only marshal arguments: torch
CUDA tensors (or raw integer device addresses) become pointers, the current torch
stream becomes the cudaStream_t.  Every step of the computation runs in the library's
CUDA kernels.  There is no fallback: if the shared library is missing, importing the
binding's functions raises.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libw4a16.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "w4a16.h")
HEADERS = [HEADER, os.path.join(os.path.dirname(HERE), "include", "w4a8.h"),
           os.path.join(os.path.dirname(HERE), "include", "mxfp.h"),
           os.path.join(os.path.dirname(HERE), "include", "decode.h")]

W4A16_OK = 0
W4A16_ERR_INVALID_ARG = -1
W4A16_ERR_UNSUPPORTED = -2
W4A16_ERR_CUDA = -3
W4A16_ERR_DEVICE_TIMEOUT = -4
W4A16_ERR_FORMAT = -5

W4A16_FP16 = 0
W4A16_BF16 = 1

W4A16_KERNEL_AUTO = 0
W4A16_KERNEL_TC = 1
W4A16_KERNEL_SIMT = 2

W4A16_ACT_NONE = 0
W4A16_ACT_RELU = 1
W4A16_ACT_SILU = 2

W4A16_GEMM_NO_PDL = 1
W4A16_GEMM_NO_WEIGHT_PREFETCH = 2
W4A16_GEMM_DEQUANT_LUT = 4
W4A16_GEMM_DEQUANT_INT = 8

DEC_KV_FP16 = 0
DEC_KV_BF16 = 1
DEC_KV_E4M3 = 2

DEC_ROPE_HALF = 0
DEC_ROPE_INTERLEAVED = 1

DEC_ROPE_SCALE_NONE = 0
DEC_ROPE_SCALE_LINEAR = 1
DEC_ROPE_SCALE_BASE = 2
DEC_ROPE_SCALE_RAMP = 3

_lock = threading.Lock()
_lib = None


class W4A16Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class GemmConfig(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("split_k", ctypes.c_int), ("tile_m", ctypes.c_int),
                ("stages", ctypes.c_int), ("flags", ctypes.c_int),
                ("reserved", ctypes.c_int * 3)]


class KvCache(ctypes.Structure):
    """dec_kv_cache: where a paged cache lies (kv_cache() fills it from tensors)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("k_page_stride", ctypes.c_int64), ("k_slot_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("v_page_stride", ctypes.c_int64),
                ("v_slot_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("dtype", ctypes.c_int), ("reserved", ctypes.c_int)]


class RopeScaling(ctypes.Structure):
    """dec_rope_scaling."""
    _fields_ = [("kind", ctypes.c_int), ("factor", ctypes.c_float), ("low", ctypes.c_float),
                ("high", ctypes.c_float), ("original_len", ctypes.c_float),
                ("magnitude", ctypes.c_float)]


class RopeConfig(ctypes.Structure):
    """dec_rope_config (rope_config() fills it)."""
    _fields_ = [("q_heads", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int), ("rot_dim", ctypes.c_int),
                ("layout", ctypes.c_int), ("table_len", ctypes.c_int),
                ("reserved", ctypes.c_int), ("table", ctypes.c_void_p),
                ("ldq", ctypes.c_int64), ("ldk", ctypes.c_int64), ("ldv", ctypes.c_int64),
                ("ldqo", ctypes.c_int64), ("ldko", ctypes.c_int64)]


class AttnConfig(ctypes.Structure):
    """dec_attn_config (attn_config() fills it)."""
    _fields_ = [("q_heads", ctypes.c_int), ("dtype", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("window", ctypes.c_int), ("scale", ctypes.c_float), ("reserved", ctypes.c_int),
                ("ldq", ctypes.c_int64), ("ldo", ctypes.c_int64), ("ld_table", ctypes.c_int64)]


def lib() -> ctypes.CDLL:
    """Loads libw4a16.so (built by weight_only_int4_tma_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: run weight_only_int4_tma_gb300.build "
                                   "(or __graft_entry__.build()) first")
            L = ctypes.CDLL(LIB_PATH)
            P, I, U, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t
            L.w4a16_abi_version.restype = I
            L.w4a16_status_string.argtypes = [I]
            L.w4a16_status_string.restype = ctypes.c_char_p
            L.w4a16_packed_bytes.argtypes = [I, I, I, I, I]
            L.w4a16_packed_bytes.restype = Z
            L.w4a16_repack.argtypes = [P, P, P, P, I, I, I, I, P, Z, P]
            L.w4a16_repack.restype = I
            L.w4a16_gemm.argtypes = [P, P, I, I, I, I, I, P, P]
            L.w4a16_gemm.restype = I
            L.w4a16_gemm_ex.argtypes = [P, P, I, I, I, I, I, P, ctypes.POINTER(GemmConfig), P]
            L.w4a16_gemm_ex.restype = I
            L.w4a16_gemm_epilogue.argtypes = [P, P, I, I, I, I, I, P, P, I, P,
                                              ctypes.POINTER(GemmConfig), P]
            L.w4a16_gemm_epilogue.restype = I
            L.w4a16_gemm_plan.argtypes = [I, I, I, I, I, ctypes.POINTER(GemmConfig),
                                          ctypes.POINTER(GemmConfig)]
            L.w4a16_gemm_plan.restype = I
            L.w4a16_dequant_debug.argtypes = [P, I, I, I, I, P, P]
            L.w4a16_dequant_debug.restype = I
            L.w4a16_get_device_status.argtypes = [P]
            L.w4a16_get_device_status.restype = I
            L.w4a16_debug_timeout_probe.argtypes = [U, P]
            L.w4a16_debug_timeout_probe.restype = I
            L.w4a16_debug_splitk_timeout_probe.argtypes = [P, P, I, I, I, I, I, P, U, P]
            L.w4a16_debug_splitk_timeout_probe.restype = I
            L.w4a8_packed_bytes.argtypes = [I, I]
            L.w4a8_packed_bytes.restype = Z
            L.w4a8_repack.argtypes = [P, P, P, P, I, I, P, Z, P]
            L.w4a8_repack.restype = I
            L.w4a8_quantize_act.argtypes = [P, I, I, I, P, P, P]
            L.w4a8_quantize_act.restype = I
            L.w4a8_gemm.argtypes = [P, P, P, I, I, I, I, P, P]
            L.w4a8_gemm.restype = I
            L.w4a8_dequant_debug.argtypes = [P, I, I, P, P]
            L.w4a8_dequant_debug.restype = I
            L.mx_packed_bytes.argtypes = [I, I]
            L.mx_packed_bytes.restype = Z
            L.mx_repack.argtypes = [P, P, I, I, P, Z, P]
            L.mx_repack.restype = I
            L.mx_gemm.argtypes = [P, P, P, I, I, I, I, P, P]
            L.mx_gemm.restype = I
            J, F, D = ctypes.c_int64, ctypes.c_float, ctypes.c_double
            L.dec_rms_norm.argtypes = [P, J, P, J, P, I, I, I, F, P, P, J, P]
            L.dec_rms_norm.restype = I
            L.dec_rms_norm_i8.argtypes = [P, J, P, J, P, I, I, I, F, P, P, P, P]
            L.dec_rms_norm_i8.restype = I
            L.dec_rms_norm_mx.argtypes = [P, J, P, J, P, I, I, I, F, P, P, P, P]
            L.dec_rms_norm_mx.restype = I
            L.dec_rope_table.argtypes = [I, D, ctypes.POINTER(RopeScaling), P, I, P]
            L.dec_rope_table.restype = I
            L.dec_rope_append.argtypes = [ctypes.POINTER(RopeConfig), ctypes.POINTER(KvCache),
                                          P, P, P, I, P, P, P, P, P]
            L.dec_rope_append.restype = I
            L.dec_attn_workspace_bytes.argtypes = [ctypes.POINTER(AttnConfig),
                                                   ctypes.POINTER(KvCache)]
            L.dec_attn_workspace_bytes.restype = Z
            L.dec_attn_paged.argtypes = [ctypes.POINTER(AttnConfig), ctypes.POINTER(KvCache),
                                         P, P, P, I, P, P, P, Z, P]
            L.dec_attn_paged.restype = I
            _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions the public headers (include/w4a16.h, w4a8.h, mxfp.h, decode.h)
    declare."""
    names = set()
    for h in HEADERS:
        src = re.sub(r"/\*.*?\*/", "", open(h).read(), flags=re.S)
        names.update(re.findall(r"\b((?:w4a16|w4a8|mx|dec)_[a-z_0-9]+)\s*\(", src))
    return sorted(names)


def status_string(status: int) -> str:
    return lib().w4a16_status_string(int(status)).decode()


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _current_stream() -> int:
    """The current torch stream's handle.  The first call binds torch's raw accessors: the
    Stream object of torch.cuda.current_stream() costs 3 us, most of a small launch."""
    global _current_stream
    import torch
    torch.cuda.current_stream()  # initialises CUDA
    device, raw = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _current_stream = lambda: raw(device())  # noqa: E731
    return _current_stream()


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str) -> int:
    if rc != W4A16_OK:
        raise W4A16Error(rc, where)
    return rc


def w4a16_abi_version() -> int:
    return lib().w4a16_abi_version()


def w4a16_packed_bytes(N: int, K: int, group: int, has_zeros: bool,
                       has_channel_scale: bool = False) -> int:
    return int(lib().w4a16_packed_bytes(N, K, group, int(bool(has_zeros)),
                                        int(bool(has_channel_scale))))


def w4a16_repack(qweight, scales, qzeros, channel_scale, N: int, K: int, group: int,
                 dtype: int, packed, packed_bytes: int | None = None, stream=None) -> None:
    if packed_bytes is None:
        packed_bytes = packed.numel() * packed.element_size()
    _check(lib().w4a16_repack(_ptr(qweight), _ptr(scales), _ptr(qzeros), _ptr(channel_scale),
                              N, K, group, dtype, _ptr(packed), packed_bytes, _stream(stream)),
           "w4a16_repack")


def w4a16_gemm(A, packed, M: int, N: int, K: int, group: int, dtype: int, Y,
               stream=None) -> None:
    _check(lib().w4a16_gemm(_ptr(A), _ptr(packed), M, N, K, group, dtype, _ptr(Y),
                            _stream(stream)), "w4a16_gemm")


def w4a16_gemm_ex(A, packed, M: int, N: int, K: int, group: int, dtype: int, Y, *,
                  kernel: int = W4A16_KERNEL_AUTO, split_k: int = 0, tile_m: int = 0,
                  stages: int = 0, flags: int = 0, stream=None) -> None:
    cfg = GemmConfig(kernel, split_k, tile_m, stages, flags)
    _check(lib().w4a16_gemm_ex(_ptr(A), _ptr(packed), M, N, K, group, dtype, _ptr(Y),
                               ctypes.byref(cfg), _stream(stream)), "w4a16_gemm_ex")


def w4a16_gemm_epilogue(A, packed, M: int, N: int, K: int, group: int, dtype: int, bias,
                        residual, act: int, Y, *, kernel: int = W4A16_KERNEL_AUTO,
                        split_k: int = 0, tile_m: int = 0, stages: int = 0, flags: int = 0,
                        stream=None) -> None:
    cfg = GemmConfig(kernel, split_k, tile_m, stages, flags)
    _check(lib().w4a16_gemm_epilogue(_ptr(A), _ptr(packed), M, N, K, group, dtype, _ptr(bias),
                                     _ptr(residual), act, _ptr(Y), ctypes.byref(cfg),
                                     _stream(stream)), "w4a16_gemm_epilogue")


def w4a16_gemm_plan(M: int, N: int, K: int, group: int, dtype: int, *,
                    kernel: int = W4A16_KERNEL_AUTO, split_k: int = 0, tile_m: int = 0,
                    stages: int = 0, flags: int = 0) -> dict:
    """The resolved launch choice of w4a16_gemm_ex for these arguments (no launch)."""
    cfg = GemmConfig(kernel, split_k, tile_m, stages, flags)
    out = GemmConfig()
    _check(lib().w4a16_gemm_plan(M, N, K, group, dtype, ctypes.byref(cfg), ctypes.byref(out)),
           "w4a16_gemm_plan")
    return {"kernel": out.kernel, "split_k": out.split_k, "tile_m": out.tile_m,
            "stages": out.stages, "w_stages": out.reserved[0], "groups": out.reserved[1],
            "whole_blocks": bool(out.reserved[2]), "flags": out.flags}


def w4a16_dequant_debug(packed, N: int, K: int, group: int, dtype: int, W_out,
                        stream=None) -> None:
    _check(lib().w4a16_dequant_debug(_ptr(packed), N, K, group, dtype, _ptr(W_out),
                                     _stream(stream)), "w4a16_dequant_debug")


def w4a16_get_device_status(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status word."""
    return int(lib().w4a16_get_device_status(_stream(stream)))


def w4a16_debug_timeout_probe(timeout_us: int, stream=None) -> None:
    _check(lib().w4a16_debug_timeout_probe(timeout_us, _stream(stream)),
           "w4a16_debug_timeout_probe")


def w4a16_debug_splitk_timeout_probe(A, packed, M: int, N: int, K: int, group: int,
                                     dtype: int, Y, timeout_us: int, stream=None) -> None:
    _check(lib().w4a16_debug_splitk_timeout_probe(_ptr(A), _ptr(packed), M, N, K, group, dtype,
                                                  _ptr(Y), timeout_us, _stream(stream)),
           "w4a16_debug_splitk_timeout_probe")


def w4a8_packed_bytes(N: int, K: int) -> int:
    return int(lib().w4a8_packed_bytes(N, K))


def w4a8_repack(qweight, s_u8, a, s_w, N: int, K: int, packed, packed_bytes: int | None = None,
                stream=None) -> None:
    if packed_bytes is None:
        packed_bytes = packed.numel() * packed.element_size()
    _check(lib().w4a8_repack(_ptr(qweight), _ptr(s_u8), _ptr(a), _ptr(s_w), N, K, _ptr(packed),
                             packed_bytes, _stream(stream)), "w4a8_repack")


def w4a8_quantize_act(A, M: int, K: int, dtype: int, A_i8, s_a, stream=None) -> None:
    _check(lib().w4a8_quantize_act(_ptr(A), M, K, dtype, _ptr(A_i8), _ptr(s_a),
                                   _stream(stream)), "w4a8_quantize_act")


def w4a8_gemm(A_i8, s_a, packed, M: int, N: int, K: int, dtype: int, Y, stream=None) -> None:
    _check(lib().w4a8_gemm(_ptr(A_i8), _ptr(s_a), _ptr(packed), M, N, K, dtype, _ptr(Y),
                           _stream(stream)), "w4a8_gemm")


def w4a8_dequant_debug(packed, N: int, K: int, W_out, stream=None) -> None:
    _check(lib().w4a8_dequant_debug(_ptr(packed), N, K, _ptr(W_out), _stream(stream)),
           "w4a8_dequant_debug")


def mx_packed_bytes(N: int, K: int) -> int:
    return int(lib().mx_packed_bytes(N, K))


def mx_repack(w_codes, w_scales, N: int, K: int, packed, packed_bytes: int | None = None,
              stream=None) -> None:
    if packed_bytes is None:
        packed_bytes = packed.numel() * packed.element_size()
    _check(lib().mx_repack(_ptr(w_codes), _ptr(w_scales), N, K, _ptr(packed), packed_bytes,
                           _stream(stream)), "mx_repack")


def mx_gemm(a_codes, a_scales, packed, M: int, N: int, K: int, dtype: int, Y,
            stream=None) -> None:
    _check(lib().mx_gemm(_ptr(a_codes), _ptr(a_scales), _ptr(packed), M, N, K, dtype, _ptr(Y),
                         _stream(stream)), "mx_gemm")


def dec_rms_norm(x, residual, weight, M: int, H: int, dtype: int, eps: float, residual_out, y, *,
                 ldx: int = 0, ldr: int = 0, ldy: int = 0, stream=None) -> None:
    _check(lib().dec_rms_norm(_ptr(x), ldx, _ptr(residual), ldr, _ptr(weight), M, H, dtype, eps,
                              _ptr(residual_out), _ptr(y), ldy, _stream(stream)), "dec_rms_norm")


def dec_rms_norm_i8(x, residual, weight, M: int, H: int, dtype: int, eps: float, residual_out,
                    y_i8, s_y, *, ldx: int = 0, ldr: int = 0, stream=None) -> None:
    _check(lib().dec_rms_norm_i8(_ptr(x), ldx, _ptr(residual), ldr, _ptr(weight), M, H, dtype,
                                 eps, _ptr(residual_out), _ptr(y_i8), _ptr(s_y),
                                 _stream(stream)), "dec_rms_norm_i8")


def dec_rms_norm_mx(x, residual, weight, M: int, H: int, dtype: int, eps: float, residual_out,
                    y_codes, y_scales, *, ldx: int = 0, ldr: int = 0, stream=None) -> None:
    _check(lib().dec_rms_norm_mx(_ptr(x), ldx, _ptr(residual), ldr, _ptr(weight), M, H, dtype,
                                 eps, _ptr(residual_out), _ptr(y_codes), _ptr(y_scales),
                                 _stream(stream)), "dec_rms_norm_mx")


def dec_rope_table(rot_dim: int, base: float, scaling: RopeScaling | None, table,
                   table_len: int, stream=None) -> None:
    _check(lib().dec_rope_table(rot_dim, base, scaling, _ptr(table), table_len,
                                _stream(stream)), "dec_rope_table")


def dec_rope_append(cfg: RopeConfig, cache: KvCache | None, q, k, v, T: int, positions, slots,
                    q_out, k_out=None, stream=None) -> None:
    _check(lib().dec_rope_append(cfg, cache, _ptr(q), _ptr(k), _ptr(v), T, _ptr(positions),
                                 _ptr(slots), _ptr(q_out), _ptr(k_out), _stream(stream)),
           "dec_rope_append")


def dec_attn_workspace_bytes(cfg: AttnConfig, cache: KvCache) -> int:
    return int(lib().dec_attn_workspace_bytes(cfg, cache))


def dec_attn_paged(cfg: AttnConfig, cache: KvCache, q, block_table, lens, B: int, out, lse,
                   workspace, ws_bytes: int | None = None, stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().dec_attn_paged(cfg, cache, _ptr(q), _ptr(block_table), _ptr(lens), B, _ptr(out),
                                _ptr(lse), _ptr(workspace), ws_bytes, _stream(stream)),
           "dec_attn_paged")


# ---- torch-friendly helpers (allocation + the calls above) ---------------------------

def repack(qweight, scales, qzeros, N: int, K: int, group: int, dtype: int,
           channel_scale=None, stream=None):
    """Allocates the packed blob on qweight's device and fills it; returns a uint8 tensor."""
    import torch
    nbytes = w4a16_packed_bytes(N, K, group, qzeros is not None, channel_scale is not None)
    if nbytes == 0:
        raise W4A16Error(W4A16_ERR_UNSUPPORTED, "w4a16_packed_bytes")
    packed = torch.empty(nbytes, dtype=torch.uint8, device=qweight.device)
    w4a16_repack(qweight, scales, qzeros, channel_scale, N, K, group, dtype, packed, nbytes,
                 stream)
    return packed


def gemm(A, packed, N: int, K: int, group: int, dtype: int, out=None, stream=None, **ex):
    """Y = A . W^T for a 2-D A on the GPU; returns Y (allocated unless `out` is given)."""
    import torch
    M = A.shape[0]
    Y = out if out is not None else torch.empty((M, N), dtype=A.dtype, device=A.device)
    if ex:
        w4a16_gemm_ex(A, packed, M, N, K, group, dtype, Y, stream=stream, **ex)
    else:
        w4a16_gemm(A, packed, M, N, K, group, dtype, Y, stream)
    return Y


def kv_cache(k, v, k_scale=None, v_scale=None) -> KvCache:
    """The paged cache in tensors k and v of shape [pages, page_size, kv_heads, head_dim], in
    any order of strides as long as head_dim is contiguous (pass a permuted view of a cache
    stored as [pages, kv_heads, page_size, head_dim]).  float16, bfloat16 or float8_e4m3fn,
    the last with optional float32 scales [kv_heads].  The struct keeps addresses, not the
    tensors: they have to outlive it."""
    import torch
    kinds = {torch.float16: DEC_KV_FP16, torch.bfloat16: DEC_KV_BF16,
             torch.float8_e4m3fn: DEC_KV_E4M3}
    if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.dtype not in kinds \
            or k.stride(3) != 1 or v.stride(3) != 1:
        raise W4A16Error(W4A16_ERR_UNSUPPORTED, "kv_cache")
    pages, size, heads, dim = k.shape
    for s in (k_scale, v_scale):
        if s is not None and (k.dtype != torch.float8_e4m3fn or s.dtype != torch.float32
                              or s.shape != (heads,) or not s.is_contiguous()):
            raise W4A16Error(W4A16_ERR_UNSUPPORTED, "kv_cache")
    return KvCache(k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale),
                   k.stride(0), k.stride(1), k.stride(2), v.stride(0), v.stride(1), v.stride(2),
                   pages, size, heads, dim, kinds[k.dtype], 0)


def rope_config(q_heads: int, kv_heads: int, head_dim: int, dtype: int, table, rot_dim: int,
                layout: int = DEC_ROPE_HALF, *, ldq: int = 0, ldk: int = 0, ldv: int = 0,
                ldqo: int = 0, ldko: int = 0) -> RopeConfig:
    """dec_rope_append's settings; table: contiguous float32 [positions, rot_dim] or [positions, 2,
    rot_dim / 2] (it has to outlive the struct), or None with rot_dim 0 and no rotation (any
    non-negative position)."""
    import torch
    if rot_dim and (table is None or table.dtype != torch.float32 or table.dim() < 2
                    or table.shape[1:].numel() != rot_dim or not table.is_contiguous()):
        raise W4A16Error(W4A16_ERR_UNSUPPORTED, "rope_config")
    n = table.shape[0] if table is not None else 0x7FFFFFFF
    return RopeConfig(q_heads, kv_heads, head_dim, dtype, rot_dim, layout, n, 0, _ptr(table),
                      ldq, ldk, ldv, ldqo, ldko)


def attn_config(q_heads: int, dtype: int, scale: float, max_pages: int, *, window: int = 0,
                ldq: int = 0, ldo: int = 0, ld_table: int = 0) -> AttnConfig:
    """dec_attn_paged's settings."""
    return AttnConfig(q_heads, dtype, max_pages, window, scale, 0, ldq, ldo, ld_table)


def attn_workspace(cfg: AttnConfig, cache: KvCache, device="cuda"):
    """A zero-filled workspace for dec_attn_paged (a uint8 tensor)."""
    import torch
    nbytes = dec_attn_workspace_bytes(cfg, cache)
    if nbytes == 0:
        raise W4A16Error(W4A16_ERR_UNSUPPORTED, "dec_attn_workspace_bytes")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)
