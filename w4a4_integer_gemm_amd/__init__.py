"""FoldQuant W8A8/W4A4 integer linear layers for AMD Instinct MI355X (gfx950).

The layer (the vla.cpp FoldQuant page's act + gemm nodes) runs in libfq.so:
hand-written HIP kernels behind the C ABI declared in include/fq.h.  This
package only loads that library and marshals arguments; torch provides device
memory and streams.
"""
from ._binding import (E2M3, ROPE_BANDS, ROPE_BASE, ROPE_LINEAR, ROPE_PAIRS, ROPE_PLAIN, ROPE_RAMP, FqError,
                       abi_version, fq_act_bytes, fq_attn_decode, fq_attn_decode_workspace_bytes, fq_attn_prefill,
                       fq_block_norm, fq_dequant_rows, fq_device_init, fq_fold_gain,
                       fq_fp8_ascale_count, fq_fp8_dequant_rows, fq_fp8_gemm, fq_fp8_linear,
                       fq_fp8_linear_workspace_bytes, fq_fp8_pack_weights, fq_fp8_prologue, fq_fp8_wscale_count,
                       fq_geglu, fq_gemm, fq_gemm_heads, fq_kv_read, fq_kv_write, fq_linear, fq_linear_heads, fq_linear_noalloc,
                       fq_linear_noalloc_max_bytes, fq_linear_workspace_bytes, fq_pack_weights, fq_prologue,
                       fq_qk_norm_rope, fq_rope,
                       fq_rope_freqs, fq_test_hook, fq_weight_bytes, last_error, lib)
from .cache import KVCache
from .site import DeviceSite, Fp8Site

__all__ = [
    "E2M3", "FqError", "abi_version", "fq_act_bytes", "fq_device_init", "fq_fold_gain", "fq_test_hook", "fq_geglu",
    "fq_gemm", "fq_gemm_heads", "fq_linear", "fq_linear_heads", "fq_linear_noalloc", "fq_linear_noalloc_max_bytes",
    "fq_linear_workspace_bytes",
    "fq_pack_weights", "fq_dequant_rows", "fq_prologue", "fq_weight_bytes", "last_error", "lib", "DeviceSite",
    "fq_fp8_ascale_count", "fq_fp8_wscale_count", "fq_fp8_pack_weights", "fq_fp8_dequant_rows", "fq_fp8_prologue",
    "fq_fp8_gemm", "fq_fp8_linear", "fq_fp8_linear_workspace_bytes", "Fp8Site",
    "fq_block_norm",
    "fq_rope", "fq_rope_freqs", "ROPE_PLAIN", "ROPE_LINEAR", "ROPE_BASE", "ROPE_BANDS", "ROPE_RAMP", "ROPE_PAIRS",
    "fq_qk_norm_rope", "fq_kv_write", "fq_kv_read", "fq_attn_prefill", "fq_attn_decode", "fq_attn_decode_workspace_bytes",
    "KVCache",
]
