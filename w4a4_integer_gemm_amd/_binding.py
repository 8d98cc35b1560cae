"""ctypes binding of libfq (include/fq.h).  Argument marshalling only.

Device entry points take torch tensors that already live on the GPU and pass
their data pointers plus the current HIP stream; every step of the layer runs
in libfq's kernels.  Host entry points take numpy arrays.  There is no
fallback: if libfq.so is missing or a call fails, an exception says why.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import sys
from typing import Optional

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
# FQ_LIB selects another build of the same library (the host-sanitizer build)
LIB_PATH = os.environ.get("FQ_LIB") or os.path.join(HERE, "libfq.so")

E2M3 = 6  # FQ_CODES_E2M3: the 4-bit codes stored as FP6 E2M3 (include/fq.h)

# scaling rules of fq_rope_freqs (include/fq.h)
ROPE_PLAIN, ROPE_LINEAR, ROPE_BASE, ROPE_BANDS, ROPE_RAMP, ROPE_PAIRS = range(6)

FQ_OK = 0
_STATUS = {0: "FQ_OK", 1: "FQ_ERR_ARG", 2: "FQ_ERR_SHAPE", 3: "FQ_ERR_UNSUPPORTED", 4: "FQ_ERR_ALIGN",
           5: "FQ_ERR_DEVICE"}

# exported symbols and their signatures (must match include/fq.h)
_P, _I32, _I64, _F, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "fq_last_error": ([], ctypes.c_char_p),
    "fq_abi_version": ([], ctypes.c_int),
    "fq_device_init": ([], ctypes.c_int),
    "fq_test_hook": ([ctypes.c_char_p], ctypes.c_int),
    "fq_weight_bytes": ([_I32, _I32, _I32], _SZ),
    "fq_act_bytes": ([_I32, _I32, _I32], _SZ),
    "fq_fold_gain": ([_P, _P, _I32, _P], ctypes.c_int),
    "fq_pack_weights": ([_P, _I32, _I32, _P, _I32, _I32, _I32, _P, _P], ctypes.c_int),
    "fq_dequant_rows": ([_P, _P, _I32, _I32, _P, _I32, _I32, _I32, _P], ctypes.c_int),
    "fq_prologue": ([_P, _I32, _I32, _I64, _P, _F, _P, _I32, _I32, _I32, _P, _P, _P], ctypes.c_int),
    "fq_gemm": ([_P, _P, _I32, _I32, _P, _P, _I32, _I32, _I32, _P, _P, _I64, _P, _I64, _P, _P], ctypes.c_int),
    "fq_geglu": ([_P, _I32, _I32, _I64, _P, _I64, _P], ctypes.c_int),
    "fq_gemm_heads": ([_P, _P, _I32, _I32, _P, _P, _I32, _I32, _I32, _P, _P, _I64, _I32, _P, _P, _P], ctypes.c_int),
    "fq_linear_workspace_bytes": ([_I32, _I32, _I32], _SZ),
    "fq_linear": ([_P, _I32, _I32, _I64, _P, _F, _P, _I32, _I32, _I32, _P, _P, _I32, _I32, _P, _P, _I64, _P,
                   _I64, _P, _SZ, _P], ctypes.c_int),
    "fq_linear_noalloc": ([_P, _I32, _I32, _I64, _P, _F, _P, _I32, _I32, _I32, _P, _P, _I32, _I32, _P, _P, _I64, _P,
                           _I64, _P], ctypes.c_int),
    "fq_linear_noalloc_max_bytes": ([], _SZ),
    "fq_linear_heads": ([_P, _I32, _I32, _I64, _P, _F, _P, _I32, _I32, _I32, _P, _P, _I32, _I32, _P, _P, _I64,
                         _I32, _P, _P, _SZ, _P], ctypes.c_int),
    "fq_fp8_ascale_count": ([_I32, _I32], _SZ),
    "fq_fp8_wscale_count": ([_I32, _I32], _SZ),
    "fq_fp8_pack_weights": ([_P, _I32, _I32, _P, _P], ctypes.c_int),
    "fq_fp8_dequant_rows": ([_P, _P, _I32, _I32, _P], ctypes.c_int),
    "fq_fp8_prologue": ([_P, _I32, _I32, _I64, _P, _F, _P, _P, _P], ctypes.c_int),
    "fq_fp8_gemm": ([_P, _P, _I32, _P, _P, _I32, _I32, _P, _P, _I64, _I32, _P, _I64, _P], ctypes.c_int),
    "fq_fp8_linear_workspace_bytes": ([_I32, _I32], _SZ),
    "fq_fp8_linear": ([_P, _I32, _I32, _I64, _P, _F, _P, _P, _I32, _P, _P, _I64, _I32, _P, _I64, _P, _SZ, _P],
                      ctypes.c_int),
    "fq_block_norm": ([_I32, _I32, _P, _I64, _P, _F, _P, _I64, _F, _P, _I64, _P, _I64, _I32, _P, _F, _P, _P, _I64, _I32,
                       _P, _I64, _P, _P, _P], ctypes.c_int),
    "fq_rope_freqs": ([_I32, ctypes.c_double, _I32, ctypes.c_double, _I32, ctypes.c_double, ctypes.c_double, _P, _P, _P],
                      ctypes.c_int),
    "fq_rope": ([_P, _I64, _I64, _I32, _I32, _I32, _I32, _I32, _I32, _P, _F, _P, _I32, _I32, _P, _I64, _I64, _P],
                ctypes.c_int),
    "fq_qk_norm_rope": ([_P, _I64, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _F, _I32, _I32, _P, _F, _P, _I32, _P, _I64,
                         _I64, _P], ctypes.c_int),
    "fq_kv_write": ([_P, _I64, _I64, _P, _I64, _I64, _P, _I32, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P],
                    ctypes.c_int),
    "fq_kv_read": ([_P, _P, _P, _P, _I32, _I32, _I32, _P, _I32, _I32, _I32, _P, _I64, _I64, _P, _I64, _I64, _P],
                   ctypes.c_int),
    "fq_attn_prefill": ([_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _I32, _I32, _P, _P, _I32, _I32, _I32, _I32, _F,
                         _I32, _P, _I64, _I64, _P], ctypes.c_int),
    "fq_attn_decode_workspace_bytes": ([_I32, _I32, _I32, _I32, _I32], _SZ),
    "fq_attn_decode": ([_P, _I64, _I64, _I32, _I32, _I32, _I32, _F, _P, _P, _P, _P, _I32, _I32, _I32, _P, _I32, _P, _P,
                        _I64, _I64, _P, _SZ, _P], ctypes.c_int),
}


class FqError(RuntimeError):
    """A libfq call returned a status other than FQ_OK."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status
        self.message = message


_lib = None


def _load_hip_runtime():
    """torch brings a HIP runtime of its own, and a host call of this library before `import
    torch` (a packer, a rotary plan) would load the system's, which then sees no device.
    The one that torch will use is loaded first, without torch's import (1 to 2 s, which
    callers of the host entry points alone do not need)."""
    if "torch" in sys.modules:
        return
    spec = importlib.util.find_spec("torch")
    path = spec and spec.origin and os.path.join(os.path.dirname(spec.origin), "lib", "libamdhip64.so")
    if path and os.path.exists(path):
        try:
            ctypes.CDLL(path)
        except OSError:
            pass  # a torch that cannot be loaded: the host entry points need none


def lib() -> ctypes.CDLL:
    """Load libfq.so from the package directory (built by build.py)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libfq.so not found at {LIB_PATH}; build it with "
                               "`python w4a4_integer_gemm_amd/build.py` (hipcc, gfx950)")
        _load_hip_runtime()
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(rc: int):
    if rc != FQ_OK:
        raise FqError(rc, lib().fq_last_error().decode())


def last_error() -> str:
    return lib().fq_last_error().decode()


def abi_version() -> int:
    return lib().fq_abi_version()


def fq_device_init():
    """Per-device set-up of the current device (optional; see include/fq.h)."""
    _check(lib().fq_device_init())


def fq_test_hook(spec: Optional[str]):
    """Force kernel choices for the tests ("gemm_tile=64x128,gemm_mfma=32,gemv=split"; "" resets)."""
    _check(lib().fq_test_hook(None if spec is None else spec.encode()))


# ------------------------------------------------------------------ host entry points
def _np_ptr(a: Optional[np.ndarray]):
    return None if a is None else a.ctypes.data_as(ctypes.c_void_p)


def fq_weight_bytes(N: int, K: int, wbits: int) -> int:
    return lib().fq_weight_bytes(N, K, wbits)


def fq_act_bytes(M: int, K: int, abits: int) -> int:
    return lib().fq_act_bytes(M, K, abits)


def fq_linear_workspace_bytes(M: int, K: int, abits: int) -> int:
    return lib().fq_linear_workspace_bytes(M, K, abits)


def fq_fold_gain(gamma: np.ndarray, ascale: Optional[np.ndarray]) -> np.ndarray:
    g = np.ascontiguousarray(gamma, dtype=np.float32)
    a = None if ascale is None else np.ascontiguousarray(ascale, dtype=np.float32)
    out = np.empty_like(g)
    _check(lib().fq_fold_gain(_np_ptr(g), _np_ptr(a), g.size, _np_ptr(out)))
    return out


def fq_pack_weights(W: np.ndarray, ascale: Optional[np.ndarray], fold_after: int, hblock: int, wbits: int):
    """Host packer; returns (codes uint8 [N][K, K/2 or 3K/4 (E2M3)], wscale float32 [N])."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    a = None if ascale is None else np.ascontiguousarray(ascale, dtype=np.float32)
    nbytes = fq_weight_bytes(N, K, wbits)
    codes = np.zeros((N, nbytes // N if nbytes else 0), np.uint8)
    ws = np.empty(N, np.float32)
    _check(lib().fq_pack_weights(_np_ptr(W), N, K, _np_ptr(a), fold_after, hblock, wbits, _np_ptr(codes),
                                 _np_ptr(ws)))
    return codes, ws


def fq_dequant_rows(codes: np.ndarray, wscale: np.ndarray, K: int, ascale: Optional[np.ndarray], fold_after: int,
                    hblock: int, wbits: int) -> np.ndarray:
    """Host dequantisation to float rows in the original frame; returns float32 [N][K]."""
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    ws = np.ascontiguousarray(wscale, dtype=np.float32)
    N = ws.shape[0]
    a = None if ascale is None else np.ascontiguousarray(ascale, dtype=np.float32)
    out = np.empty((N, K), np.float32)
    _check(lib().fq_dequant_rows(_np_ptr(codes), _np_ptr(ws), N, K, _np_ptr(a), fold_after, hblock, wbits,
                                 _np_ptr(out)))
    return out


def fq_fp8_ascale_count(M: int, K: int) -> int:
    return lib().fq_fp8_ascale_count(M, K)


def fq_fp8_wscale_count(N: int, K: int) -> int:
    return lib().fq_fp8_wscale_count(N, K)


def fq_fp8_linear_workspace_bytes(M: int, K: int) -> int:
    return lib().fq_fp8_linear_workspace_bytes(M, K)


def fq_fp8_pack_weights(W: np.ndarray):
    """Host packer; returns (codes uint8 [N][K], wscale float32 [ceil(N / 128)][K / 128])."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    codes = np.zeros((N, K), np.uint8)
    ws = np.zeros((-(-N // 128), max(K // 128, 0)), np.float32)
    _check(lib().fq_fp8_pack_weights(_np_ptr(W), N, K, _np_ptr(codes), _np_ptr(ws)))
    return codes, ws


def fq_fp8_dequant_rows(codes: np.ndarray, wscale: np.ndarray) -> np.ndarray:
    """Host dequantisation; returns float32 [N][K]."""
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    ws = np.ascontiguousarray(wscale, dtype=np.float32)
    N, K = codes.shape
    if ws.size != fq_fp8_wscale_count(N, K):
        raise ValueError(f"wscale has {ws.size} values, not {fq_fp8_wscale_count(N, K)} for N={N} K={K}")
    out = np.empty((N, K), np.float32)
    _check(lib().fq_fp8_dequant_rows(_np_ptr(codes), _np_ptr(ws), N, K, _np_ptr(out)))
    return out


def fq_rope_freqs(rot_dim: int, base: float = 10000.0, kind: int = ROPE_PLAIN, factor: float = 1.0,
                  trained_len: int = 1, low: float = 1.0, high: float = 32.0,
                  pair_factors: Optional[np.ndarray] = None):
    """Host plan; returns (freq uint64 [rot_dim / 2], factor on cos and sin)."""
    pf = None if pair_factors is None else np.ascontiguousarray(pair_factors, dtype=np.float32)
    if pf is not None and pf.size != rot_dim // 2:
        raise ValueError(f"pair_factors has {pf.size} values, not {rot_dim // 2}")
    freq = np.zeros(max(rot_dim // 2, 1), np.uint64)
    scale = ctypes.c_float()
    _check(lib().fq_rope_freqs(rot_dim, base, kind, factor, trained_len, low, high, _np_ptr(pf), _np_ptr(freq),
                               ctypes.byref(scale)))
    return freq, scale.value


# ------------------------------------------------------------------ device entry points
def _dptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device entry points need GPU tensors")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    """The hipStream_t of `stream`, or of the current device's current stream.
    (torch.cuda.current_stream() builds a Stream object: about 2.7 us per call,
    a fifth of a small layer's host time; the raw accessor returns the handle.)"""
    import torch
    if stream is not None:
        return stream.cuda_stream
    C = torch._C
    if hasattr(C, "_cuda_getCurrentRawStream"):
        return C._cuda_getCurrentRawStream(C._cuda_getDevice())
    return torch.cuda.current_stream().cuda_stream


def fq_prologue(x, M: int, K: int, ldx: int, gamma_folded, eps: float, ascale, fold_after: int, hblock: int,
                abits: int, act_codes, act_scale, stream=None):
    _check(lib().fq_prologue(_dptr(x), M, K, ldx, _dptr(gamma_folded), eps, _dptr(ascale), fold_after, hblock,
                             abits, _dptr(act_codes), _dptr(act_scale), _stream(stream)))


def fq_gemm(act_codes, act_scale, M: int, abits: int, w_codes, wscale, N: int, K: int, wbits: int, bias,
            residual, ldr: int, y, ldy: int, acc=None, stream=None):
    _check(lib().fq_gemm(_dptr(act_codes), _dptr(act_scale), M, abits, _dptr(w_codes), _dptr(wscale), N, K, wbits,
                         _dptr(bias), _dptr(residual), ldr, _dptr(y), ldy, _dptr(acc), _stream(stream)))


def fq_linear(x, M: int, K: int, ldx: int, gamma_folded, eps: float, ascale, fold_after: int, hblock: int,
              abits: int, w_codes, wscale, N: int, wbits: int, bias, residual, ldr: int, y, ldy: int, workspace,
              workspace_bytes: int, stream=None):
    _check(lib().fq_linear(_dptr(x), M, K, ldx, _dptr(gamma_folded), eps, _dptr(ascale), fold_after, hblock, abits,
                           _dptr(w_codes), _dptr(wscale), N, wbits, _dptr(bias), _dptr(residual), ldr, _dptr(y),
                           ldy, _dptr(workspace), workspace_bytes, _stream(stream)))


def fq_linear_noalloc(x, M: int, K: int, ldx: int, gamma_folded, eps: float, ascale, fold_after: int, hblock: int,
                      abits: int, w_codes, wscale, N: int, wbits: int, bias, residual, ldr: int, y, ldy: int,
                      stream=None):
    _check(lib().fq_linear_noalloc(_dptr(x), M, K, ldx, _dptr(gamma_folded), eps, _dptr(ascale), fold_after, hblock,
                                   abits, _dptr(w_codes), _dptr(wscale), N, wbits, _dptr(bias), _dptr(residual), ldr,
                                   _dptr(y), ldy, _stream(stream)))


def fq_linear_noalloc_max_bytes() -> int:
    return lib().fq_linear_noalloc_max_bytes()


def fq_gemm_heads(act_codes, act_scale, M: int, abits: int, w_codes, wscale, N: int, K: int, wbits: int, bias,
                  residual, ldr: int, head_dim: int, y, acc=None, stream=None):
    _check(lib().fq_gemm_heads(_dptr(act_codes), _dptr(act_scale), M, abits, _dptr(w_codes), _dptr(wscale), N, K,
                               wbits, _dptr(bias), _dptr(residual), ldr, head_dim, _dptr(y), _dptr(acc),
                               _stream(stream)))


def fq_linear_heads(x, M: int, K: int, ldx: int, gamma_folded, eps: float, ascale, fold_after: int, hblock: int,
                    abits: int, w_codes, wscale, N: int, wbits: int, bias, residual, ldr: int, head_dim: int, y,
                    workspace, workspace_bytes: int, stream=None):
    _check(lib().fq_linear_heads(_dptr(x), M, K, ldx, _dptr(gamma_folded), eps, _dptr(ascale), fold_after, hblock,
                                 abits, _dptr(w_codes), _dptr(wscale), N, wbits, _dptr(bias), _dptr(residual), ldr,
                                 head_dim, _dptr(y), _dptr(workspace), workspace_bytes, _stream(stream)))


def fq_geglu(gateup, M: int, F: int, ld_in: int, h, ld_out: int, stream=None):
    _check(lib().fq_geglu(_dptr(gateup), M, F, ld_in, _dptr(h), ld_out, _stream(stream)))


def fq_fp8_prologue(x, M: int, K: int, ldx: int, gamma, eps: float, act_codes, act_scale, stream=None):
    _check(lib().fq_fp8_prologue(_dptr(x), M, K, ldx, _dptr(gamma), eps, _dptr(act_codes), _dptr(act_scale),
                                 _stream(stream)))


def fq_fp8_gemm(act_codes, act_scale, M: int, w_codes, wscale, N: int, K: int, bias, residual, ldr: int,
                head_dim: int, y, ldy: int, stream=None):
    _check(lib().fq_fp8_gemm(_dptr(act_codes), _dptr(act_scale), M, _dptr(w_codes), _dptr(wscale), N, K, _dptr(bias),
                             _dptr(residual), ldr, head_dim, _dptr(y), ldy, _stream(stream)))


def fq_fp8_linear(x, M: int, K: int, ldx: int, gamma, eps: float, w_codes, wscale, N: int, bias, residual, ldr: int,
                  head_dim: int, y, ldy: int, workspace, workspace_bytes: int, stream=None):
    _check(lib().fq_fp8_linear(_dptr(x), M, K, ldx, _dptr(gamma), eps, _dptr(w_codes), _dptr(wscale), N, _dptr(bias),
                               _dptr(residual), ldr, head_dim, _dptr(y), ldy, _dptr(workspace), workspace_bytes,
                               _stream(stream)))


def fq_block_norm(M: int, K: int, x, ldx: int, post_gamma, post_eps: float, gate, ld_gate: int, res_scale: float,
                  stream_in, ld_in: int, stream_out, ld_out: int, stream_f32: int, pre_gamma, pre_eps: float, mod_scale,
                  mod_shift, ld_mod: int, rows_per_cond: int, h, ld_h: int, act_codes=None, act_scale=None,
                  stream=None):
    _check(lib().fq_block_norm(M, K, _dptr(x), ldx, _dptr(post_gamma), post_eps, _dptr(gate), ld_gate, res_scale,
                               _dptr(stream_in), ld_in, _dptr(stream_out), ld_out, stream_f32, _dptr(pre_gamma),
                               pre_eps, _dptr(mod_scale), _dptr(mod_shift), ld_mod, rows_per_cond, _dptr(h), ld_h,
                               _dptr(act_codes), _dptr(act_scale), _stream(stream)))


def fq_rope(x, x_token: int, x_head: int, M: int, heads: int, rot_heads: int, head_dim: int, rot_dim: int,
            interleaved: int, freq, attn_scale: float, positions, pos0: int, inverse: int, y, y_token: int, y_head: int,
            stream=None):
    _check(lib().fq_rope(_dptr(x), x_token, x_head, M, heads, rot_heads, head_dim, rot_dim, interleaved, _dptr(freq),
                         attn_scale, _dptr(positions), pos0, inverse, _dptr(y), y_token, y_head, _stream(stream)))


def fq_qk_norm_rope(x, x_token: int, x_head: int, M: int, heads: int, q_heads: int, k_heads: int, head_dim: int, q_gamma,
                    k_gamma, eps: float, rot_dim: int, interleaved: int, freq, attn_scale: float, positions, pos0: int, y,
                    y_token: int, y_head: int, stream=None):
    _check(lib().fq_qk_norm_rope(_dptr(x), x_token, x_head, M, heads, q_heads, k_heads, head_dim, _dptr(q_gamma),
                                 _dptr(k_gamma), eps, rot_dim, interleaved, _dptr(freq), attn_scale, _dptr(positions), pos0,
                                 _dptr(y), y_token, y_head, _stream(stream)))


def fq_kv_write(k, k_token: int, k_head: int, v, v_token: int, v_head: int, slots, M: int, kv_heads: int, head_dim: int,
                kv_bits: int, pages: int, page_size: int, k_cache, v_cache, k_scale, v_scale, stream=None):
    _check(lib().fq_kv_write(_dptr(k), k_token, k_head, _dptr(v), v_token, v_head, _dptr(slots), M, kv_heads, head_dim,
                             kv_bits, pages, page_size, _dptr(k_cache), _dptr(v_cache), _dptr(k_scale), _dptr(v_scale),
                             _stream(stream)))


def fq_kv_read(k_cache, v_cache, k_scale, v_scale, kv_bits: int, pages: int, page_size: int, slots, M: int, kv_heads: int,
               head_dim: int, k, k_token: int, k_head: int, v, v_token: int, v_head: int, stream=None):
    _check(lib().fq_kv_read(_dptr(k_cache), _dptr(v_cache), _dptr(k_scale), _dptr(v_scale), kv_bits, pages, page_size,
                            _dptr(slots), M, kv_heads, head_dim, _dptr(k), k_token, k_head, _dptr(v), v_token, v_head,
                            _stream(stream)))


def fq_attn_prefill(q, q_token: int, q_head: int, k, k_token: int, k_head: int, v, v_token: int, v_head: int, M: int,
                    M_k: int, cu_q, cu_k, seqs: int, q_heads: int, kv_heads: int, head_dim: int, scale: float, causal: int,
                    o, o_token: int, o_head: int, stream=None):
    _check(lib().fq_attn_prefill(_dptr(q), q_token, q_head, _dptr(k), k_token, k_head, _dptr(v), v_token, v_head, M, M_k,
                                 _dptr(cu_q), _dptr(cu_k), seqs, q_heads, kv_heads, head_dim, scale, causal, _dptr(o),
                                 o_token, o_head, _stream(stream)))


def fq_attn_decode_workspace_bytes(seqs: int, q_heads: int, kv_heads: int, head_dim: int, max_len: int) -> int:
    return lib().fq_attn_decode_workspace_bytes(seqs, q_heads, kv_heads, head_dim, max_len)


def fq_attn_decode(q, q_token: int, q_head: int, seqs: int, q_heads: int, kv_heads: int, head_dim: int, scale: float,
                   k_cache, v_cache, k_scale, v_scale, kv_bits: int, pages: int, page_size: int, page_table, max_pages: int,
                   lens, o, o_token: int, o_head: int, workspace, workspace_bytes: int, stream=None):
    _check(lib().fq_attn_decode(_dptr(q), q_token, q_head, seqs, q_heads, kv_heads, head_dim, scale, _dptr(k_cache),
                                _dptr(v_cache), _dptr(k_scale), _dptr(v_scale), kv_bits, pages, page_size,
                                _dptr(page_table), max_pages, _dptr(lens), _dptr(o), o_token, o_head, _dptr(workspace),
                                workspace_bytes, _stream(stream)))
