"""Python binding of libqmv.so, the sm_103a group-quantized mat-vec (affine and mxfp4).

Argument marshalling only: every step of the computation runs in the CUDA
library. The names match the C ABI of ``include/qmv.h``. Device buffers may be
given as torch tensors (their ``data_ptr()`` is passed) or as integer device
addresses; streams as ``torch.cuda.Stream``, an integer handle, or ``None``
(torch's current stream on the current device).

Raises ``QmvError`` for any non-OK status, and ``RuntimeError`` when the
library has not been built -- there is no fallback implementation.
"""

from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libqmv.so")

QMV_TILE_M = 16
QMV_MAX_M = 256
F32_OUT = 0x1
FORCE_M1_PER_COLUMN = 0x2
PDL = 0x4
SB_INTERLEAVED = 0x8
MOE_GELU = 0x10
MOE_SOFTMAX_ALL = 0x20
VERIFY_F32_LOGITS = 0x40
ROPE_F32_IN = 0x80
ROPE_NEIGHBOURS = 0x100
ROPE_NORM_PLUS_ONE = 0x200

STATUS = {
    0: "QMV_OK", 1: "QMV_ERR_NULL", 2: "QMV_ERR_BITS", 3: "QMV_ERR_GROUP", 4: "QMV_ERR_SHAPE",
    5: "QMV_ERR_M_RANGE", 6: "QMV_ERR_ALIGN", 7: "QMV_ERR_CUDA", 8: "QMV_ERR_WORKSPACE",
    9: "QMV_ERR_VALUE", 10: "QMV_ERR_FLAGS",
    11: "QMV_ERR_COUNT",
}

EXPORTED = ("qmv_packed_words", "qmv_pack", "qmv_unpack", "qmv_pack_sb", "qmv_split_count", "qmv_workspace_size",
            "qmv_run", "qmv_run_ex", "qmv_run_noalloc", "qmv_mxfp4_run", "qmv_workspace_init", "qmv_lora_workspace_size", "qmv_lora_run",
            "qmv_moe_workspace_size", "qmv_moe_run", "qmv_verify_workspace_size", "qmv_verify_run", "qmv_rope_run",
            "qmv_attend_workspace_size", "qmv_attend_run", "qmv_device_error", "qmv_last_cuda_error",
            "qmv_status_string")


class QmvError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = f"{where}: {qmv_status_string(code)}"
        if code == 7:
            msg += f" [{qmv_last_cuda_error()}]"
        super().__init__(msg)


_lock = threading.Lock()
_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libqmv.so (built by ``python -m group_quantized_mat_gb300.build``)."""
    global _lib
    if path is None and _lib is not None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is not built: run `python -m group_quantized_mat_gb300.build`")
        lib = ctypes.CDLL(p)
        P, I, I64, SZ, U = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_uint
        lib.qmv_packed_words.restype = SZ
        lib.qmv_packed_words.argtypes = [I64, I64, I]
        lib.qmv_pack.restype = I
        lib.qmv_pack.argtypes = [P, P, I64, I64, I]
        lib.qmv_unpack.restype = I
        lib.qmv_unpack.argtypes = [P, P, I64, I64, I]
        lib.qmv_pack_sb.restype = I
        lib.qmv_pack_sb.argtypes = [P, P, P, I64, I64]
        lib.qmv_split_count.restype = I
        lib.qmv_split_count.argtypes = [I, I, I, I]
        lib.qmv_workspace_size.restype = SZ
        lib.qmv_workspace_size.argtypes = [I, I, I, I, I]
        lib.qmv_run.restype = I
        lib.qmv_run.argtypes = [P, P, P, P, P, I, I, I, I, I, P]
        lib.qmv_run_ex.restype = I
        lib.qmv_run_ex.argtypes = [P, P, P, P, P, I, I, I, I, I, P, SZ, U, P]
        lib.qmv_run_noalloc.restype = I
        lib.qmv_run_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, I, P]
        lib.qmv_mxfp4_run.restype = I
        lib.qmv_mxfp4_run.argtypes = [P, P, P, P, I, I, I, U, P]
        lib.qmv_lora_workspace_size.restype = SZ
        lib.qmv_lora_workspace_size.argtypes = [I] * 6
        lib.qmv_lora_run.restype = I
        lib.qmv_lora_run.argtypes = [P] * 9 + [I] * 7 + [P, SZ, U, P]
        lib.qmv_moe_workspace_size.restype = SZ
        lib.qmv_moe_workspace_size.argtypes = [I] * 7
        lib.qmv_moe_run.restype = I
        lib.qmv_moe_run.argtypes = [P] * 11 + [I] * 7 + [P, SZ, U, P]
        lib.qmv_verify_workspace_size.restype = SZ
        lib.qmv_verify_workspace_size.argtypes = [I] * 3
        lib.qmv_verify_run.restype = I
        lib.qmv_verify_run.argtypes = [P] * 10 + [I] * 3 + [I64] * 3 + [P, SZ, U, P]
        F = ctypes.c_float
        lib.qmv_rope_run.restype = I
        lib.qmv_rope_run.argtypes = [P] * 10 + [I] * 8 + [F] + [I64] * 4 + [U, P]
        lib.qmv_attend_workspace_size.restype = SZ
        lib.qmv_attend_workspace_size.argtypes = [I] * 10
        lib.qmv_attend_run.restype = I
        lib.qmv_attend_run.argtypes = [P] * 8 + [I] * 9 + [F, I, I] + [I64] * 5 + [P, SZ, U, P]
        lib.qmv_workspace_init.restype = I
        lib.qmv_workspace_init.argtypes = [P, SZ, P]
        lib.qmv_device_error.restype = I
        lib.qmv_device_error.argtypes = [ctypes.POINTER(U)]
        lib.qmv_last_cuda_error.restype = ctypes.c_char_p
        lib.qmv_last_cuda_error.argtypes = []
        lib.qmv_status_string.restype = ctypes.c_char_p
        lib.qmv_status_string.argtypes = [I]
        if path is None:
            _lib = lib
        return lib


def _ptr(a) -> int | None:
    if a is None or type(a) is int:
        return a
    try:
        return a.data_ptr()  # torch.Tensor
    except AttributeError:
        if isinstance(a, np.ndarray):
            return a.ctypes.data
        if isinstance(a, int):
            return int(a)
        raise  # a float or a text is no address


def _stream(s) -> int | None:
    if s is None:
        import torch
        try:
            # the handle that torch.cuda.current_stream() wraps, in a tenth of its 3 us
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        except AttributeError:
            return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def _check(code: int, where: str) -> None:
    if code != 0:
        raise QmvError(code, where)


def qmv_status_string(code: int) -> str:
    try:
        return load().qmv_status_string(int(code)).decode()
    except RuntimeError:
        return STATUS.get(int(code), f"status {code}")


# ----------------------------------------------------------------- codec --
def qmv_packed_words(N: int, K: int, bits: int) -> int:
    return int(load().qmv_packed_words(N, K, bits))


def qmv_pack(q: np.ndarray, bits: int) -> np.ndarray:
    """Pack host q[N, K] (uint8, values < 2**bits) into uint32 [N, K*bits/32]."""
    q = np.ascontiguousarray(q, dtype=np.uint8)
    N, K = q.shape
    if (K * bits) % 32:
        raise QmvError(4, "qmv_pack")
    out = np.empty((N, K * bits // 32), dtype=np.uint32)
    _check(load().qmv_pack(q.ctypes.data, out.ctypes.data, N, K, bits), "qmv_pack")
    return out


def qmv_unpack(w_q: np.ndarray, K: int, bits: int) -> np.ndarray:
    w_q = np.ascontiguousarray(w_q, dtype=np.uint32)
    N = w_q.shape[0]
    out = np.empty((N, K), dtype=np.uint8)
    _check(load().qmv_unpack(w_q.ctypes.data, out.ctypes.data, N, K, bits), "qmv_unpack")
    return out


def qmv_pack_sb(scales: np.ndarray, biases: np.ndarray) -> np.ndarray:
    """Interleave host bf16 bit patterns scales, biases [N, G] (uint16) into
    uint32 [N, G]: scale in the low half of each word, bias in the high half."""
    s = np.ascontiguousarray(scales, dtype=np.uint16)
    b = np.ascontiguousarray(biases, dtype=np.uint16)
    if s.shape != b.shape or s.ndim != 2:
        raise QmvError(4, "qmv_pack_sb")
    out = np.empty(s.shape, dtype=np.uint32)
    _check(load().qmv_pack_sb(s.ctypes.data, b.ctypes.data, out.ctypes.data, s.shape[0], s.shape[1]), "qmv_pack_sb")
    return out


# ------------------------------------------------------------------ plan --
def qmv_split_count(N: int, K: int, bits: int, group_size: int) -> int:
    return int(load().qmv_split_count(N, K, bits, group_size))


def qmv_workspace_size(M: int, N: int, K: int, bits: int, group_size: int) -> int:
    return int(load().qmv_workspace_size(M, N, K, bits, group_size))


# ------------------------------------------------------------------- run --
def qmv_run(w_q, scales, biases, x, y, M: int, N: int, K: int, bits: int, group_size: int, stream=None) -> None:
    """y[M, N] (bf16) = W x, enqueued on ``stream``; see include/qmv.h."""
    code = load().qmv_run(_ptr(w_q), _ptr(scales), _ptr(biases), _ptr(x), _ptr(y), M, N, K, bits, group_size,
                          _stream(stream))
    _check(code, "qmv_run")


def qmv_run_ex(w_q, scales, biases, x, y, M: int, N: int, K: int, bits: int, group_size: int,
               workspace=None, workspace_bytes: int = 0, flags: int = 0, stream=None) -> None:
    code = load().qmv_run_ex(_ptr(w_q), _ptr(scales), _ptr(biases), _ptr(x), _ptr(y), M, N, K, bits, group_size,
                             _ptr(workspace), int(workspace_bytes), int(flags), _stream(stream))
    _check(code, "qmv_run_ex")


NOALLOC_SCRATCH_BYTES = 8 << 20


def qmv_run_noalloc(w_q, scales, biases, x, y, M: int, N: int, K: int, bits: int, group_size: int,
                    stream=None) -> None:
    """qmv_run without any device allocation (fixed scratch array in the library)."""
    code = load().qmv_run_noalloc(_ptr(w_q), _ptr(scales), _ptr(biases), _ptr(x), _ptr(y), M, N, K, bits,
                                  group_size, _stream(stream))
    _check(code, "qmv_run_noalloc")


def qmv_mxfp4_run(w_q, scales, x, y, M: int, N: int, K: int, flags: int = 0, stream=None) -> None:
    """y[M, N] = W x in the mxfp4 mode (E2M1 codes packed by ``qmv_pack(q, 4)``,
    uint8 E8M0 scales [N, K/32]); see include/qmv.h."""
    code = load().qmv_mxfp4_run(_ptr(w_q), _ptr(scales), _ptr(x), _ptr(y), M, N, K, int(flags), _stream(stream))
    _check(code, "qmv_mxfp4_run")


# ------------------------------------------- operators of a decode step --
def qmv_lora_workspace_size(M: int, N: int, K: int, bits: int, group_size: int, rank: int) -> int:
    return int(load().qmv_lora_workspace_size(M, N, K, bits, group_size, rank))


def qmv_lora_run(w_q, scales, biases, x, lora_a, lora_b, adapter, lora_scale, y, M: int, N: int, K: int, bits: int,
                 group_size: int, adapters: int, rank: int, workspace=None, workspace_bytes: int = 0, flags: int = 0,
                 stream=None) -> None:
    """y[M, N] = W x + scale_a B_a (A_a x) with each vector's own adapter a, enqueued on ``stream``; see include/qmv.h."""
    code = load().qmv_lora_run(_ptr(w_q), _ptr(scales), _ptr(biases), _ptr(x), _ptr(lora_a), _ptr(lora_b),
                               _ptr(adapter), _ptr(lora_scale), _ptr(y), M, N, K, bits, group_size, adapters, rank,
                               _ptr(workspace), workspace_bytes, flags, _stream(stream))
    _check(code, "qmv_lora_run")


def qmv_moe_workspace_size(M: int, K: int, inter: int, experts: int, top_k: int, bits: int, group_size: int) -> int:
    return int(load().qmv_moe_workspace_size(M, K, inter, experts, top_k, bits, group_size))


def qmv_moe_run(x, router, gu_w, gu_scales, gu_biases, dn_w, dn_scales, dn_biases, y, topk_ids, topk_weights, M: int,
                K: int, inter: int, experts: int, top_k: int, bits: int, group_size: int, workspace=None,
                workspace_bytes: int = 0, flags: int = 0, stream=None) -> None:
    """y[M, K] of a whole mixture-of-experts layer, and the routing if ``topk_ids`` / ``topk_weights`` are given."""
    code = load().qmv_moe_run(_ptr(x), _ptr(router), _ptr(gu_w), _ptr(gu_scales), _ptr(gu_biases), _ptr(dn_w),
                              _ptr(dn_scales), _ptr(dn_biases), _ptr(y), _ptr(topk_ids), _ptr(topk_weights), M, K,
                              inter, experts, top_k, bits, group_size, _ptr(workspace), workspace_bytes, flags,
                              _stream(stream))
    _check(code, "qmv_moe_run")


def qmv_verify_workspace_size(B: int, S: int, V: int) -> int:
    return int(load().qmv_verify_workspace_size(B, S, V))


def qmv_verify_run(target, draft, draft_tokens, draft_len, temperature, uniform, noise, tokens, accepted, logprob,
                   B: int, S: int, V: int, ld_target: int | None = None, ld_draft: int | None = None,
                   ld_noise: int | None = None, workspace=None, workspace_bytes: int = 0, flags: int = 0,
                   stream=None) -> None:
    """Accepted prefix of the drafted tokens, the token after it and their log-probabilities; see include/qmv.h.
    The row strides default to V."""
    code = load().qmv_verify_run(_ptr(target), _ptr(draft), _ptr(draft_tokens), _ptr(draft_len), _ptr(temperature),
                                 _ptr(uniform), _ptr(noise), _ptr(tokens), _ptr(accepted), _ptr(logprob), B, S, V,
                                 V if ld_target is None else ld_target, V if ld_draft is None else ld_draft,
                                 V if ld_noise is None else ld_noise, _ptr(workspace), workspace_bytes, flags,
                                 _stream(stream))
    _check(code, "qmv_verify_run")


# --------------------------------------------- an attention layer's part --
def qmv_rope_run(qkv, q_norm, k_norm, positions, inv_freq, axis, slots, q, k_cache, v_cache, T: int, heads: int,
                 kv_heads: int, head_dim: int, rope_dim: int, page_size: int, pages: int, axes: int = 1,
                 eps: float = 1e-6, ld_qkv: int | None = None, page_stride: int | None = None,
                 token_stride: int | None = None, head_stride: int | None = None, flags: int = 0, stream=None) -> None:
    """Norms and rotation of each head's query and key, and the new keys and values put into the paged cache; see
    include/qmv.h. The strides default to those of whole rows and of a cache [pages, page_size, kv_heads, head_dim]."""
    code = load().qmv_rope_run(_ptr(qkv), _ptr(q_norm), _ptr(k_norm), _ptr(positions), _ptr(inv_freq), _ptr(axis),
                               _ptr(slots), _ptr(q), _ptr(k_cache), _ptr(v_cache), T, heads, kv_heads, head_dim,
                               rope_dim, page_size, pages, axes, eps,
                               (heads + 2 * kv_heads) * head_dim if ld_qkv is None else ld_qkv,
                               page_size * kv_heads * head_dim if page_stride is None else page_stride,
                               kv_heads * head_dim if token_stride is None else token_stride,
                               head_dim if head_stride is None else head_stride, flags, _stream(stream))
    _check(code, "qmv_rope_run")


def qmv_attend_workspace_size(B: int, T: int, max_new: int, heads: int, kv_heads: int, head_dim: int, page_size: int,
                              max_pages: int, window: int = 0, sinks: int = 0) -> int:
    return int(load().qmv_attend_workspace_size(B, T, max_new, heads, kv_heads, head_dim, page_size, max_pages, window,
                                                sinks))


def qmv_attend_run(q, k_cache, v_cache, page_table, q_start, kv_len, out, lse, B: int, T: int, max_new: int, heads: int,
                   kv_heads: int, head_dim: int, page_size: int, pages: int, max_pages: int, scale: float | None = None,
                   window: int = 0, sinks: int = 0, ld_q: int | None = None, ld_out: int | None = None,
                   page_stride: int | None = None, token_stride: int | None = None, head_stride: int | None = None,
                   workspace=None, workspace_bytes: int = 0, flags: int = 0, stream=None) -> None:
    """Attention of new tokens over a paged cache; see include/qmv.h. The scale defaults to head_dim ** -0.5, the
    strides to those of whole rows and of a cache [pages, page_size, kv_heads, head_dim]."""
    if scale is None:
        scale = head_dim ** -0.5 if head_dim > 0 else 1.0
    code = load().qmv_attend_run(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(q_start), _ptr(kv_len),
                                 _ptr(out), _ptr(lse), B, T, max_new, heads, kv_heads, head_dim, page_size, pages,
                                 max_pages, scale, window, sinks,
                                 heads * head_dim if ld_q is None else ld_q, heads * head_dim if ld_out is None else ld_out,
                                 page_size * kv_heads * head_dim if page_stride is None else page_stride,
                                 kv_heads * head_dim if token_stride is None else token_stride,
                                 head_dim if head_stride is None else head_stride, _ptr(workspace), workspace_bytes,
                                 flags, _stream(stream))
    _check(code, "qmv_attend_run")


def qmv_workspace_init(workspace, nbytes: int, stream=None) -> None:
    _check(load().qmv_workspace_init(_ptr(workspace), int(nbytes), _stream(stream)), "qmv_workspace_init")


def qmv_last_cuda_error() -> str:
    return load().qmv_last_cuda_error().decode()


def qmv_device_error() -> int:
    w = ctypes.c_uint(0)
    _check(load().qmv_device_error(ctypes.byref(w)), "qmv_device_error")
    return int(w.value)
