// C ABI of the operators around the integer sites: FP8 sites with block
// scales, the norms before and after a block, rotary positions.  Validation
// and dispatch; every check runs before any HIP call.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/fq.h"
#include "fq_check.h"
#include "fq_internal.h"

namespace {

// One workgroup per row.
fq_status check_norm_launch(const char* fn, int32_t M, int32_t K, bool f32) {
    if (int64_t(M) * fq::block_norm_threads(K, M, f32) >= kMaxThreads)
        return fail(FQ_ERR_SHAPE, fmt("%s: M=%d rows of K=%d are too many for one launch (M x %d threads >= 2^32)", fn, M,
                                      K, fq::block_norm_threads(K, M, f32)));
    return FQ_OK;
}

size_t scale_bytes(int32_t M, int32_t K) { return size_t(K / 128) * size_t(fq::fp8_scale_ld(M)) * sizeof(float); }

fq_status validate_fp8_prologue(const char* fn, const void* x, int32_t M, int32_t K, int64_t ldx, const float* gamma,
                                float eps, const void* codes, const float* scale) {
    if (!x) return fail(FQ_ERR_ARG, fmt("%s: x_bf16 is NULL", fn));
    if (!codes) return fail(FQ_ERR_ARG, fmt("%s: act_codes is NULL", fn));
    if (!scale) return fail(FQ_ERR_ARG, fmt("%s: act_scale is NULL", fn));
    FQ_TRY(check_m(fn, M));
    FQ_TRY(check_k(fn, K, kGemmK));
    FQ_TRY(check_norm_launch(fn, M, K, false));
    FQ_TRY(check_rows(fn, "x_bf16", "ldx", x, ldx, K, 8));
    if (gamma) FQ_TRY(check_eps(fn, "eps", eps));
    FQ_TRY(check_vector(fn, "gamma", gamma));
    FQ_TRY(check_vector(fn, "act_codes", codes));
    return check_vector(fn, "act_scale", scale);
}

fq_status validate_fp8_gemm(const char* fn, const void* act, const float* act_scale, int32_t M, const void* w,
                            const float* wscale, int32_t N, int32_t K, const float* bias, const void* residual,
                            int64_t ldr, int32_t head_dim, const void* y, int64_t ldy) {
    if (!act) return fail(FQ_ERR_ARG, fmt("%s: act_codes is NULL", fn));
    if (!act_scale) return fail(FQ_ERR_ARG, fmt("%s: act_scale is NULL", fn));
    if (!w) return fail(FQ_ERR_ARG, fmt("%s: w_codes is NULL", fn));
    if (!wscale) return fail(FQ_ERR_ARG, fmt("%s: wscale is NULL", fn));
    if (!y) return fail(FQ_ERR_ARG, fmt("%s: y_bf16 is NULL", fn));
    FQ_TRY(check_m(fn, M));
    if (N < 8 || N % 8 || N > INT32_MAX - 512)
        return fail(FQ_ERR_SHAPE, fmt("%s: N=%d is not a positive multiple of 8 (%d/8 = %.3f)", fn, N, N, N / 8.0));
    FQ_TRY(check_k(fn, K, kGemmK));
    // a workgroup of 512 threads per tile of at least 64 x 64 outputs, fewer than 2^32 threads in all
    if (((int64_t(M) + 63) / 64) * ((int64_t(N) + 63) / 64) >= kMaxThreads / 512)
        return fail(FQ_ERR_SHAPE, fmt("%s: M=%d x N=%d is too large for one launch", fn, M, N));
    if (head_dim < 0) return fail(FQ_ERR_SHAPE, fmt("%s: head_dim=%d must be >= 0", fn, head_dim));
    if (head_dim % 8) return fail(FQ_ERR_SHAPE, fmt("%s: head_dim=%d is not a multiple of 8", fn, head_dim));
    if (head_dim > 0 && N % head_dim)
        return fail(FQ_ERR_SHAPE, fmt("%s: N=%d is not a whole number of heads of head_dim=%d (%d/%d = %.3f)", fn, N,
                                      head_dim, N, head_dim, double(N) / head_dim));
    if (head_dim == 0)
        FQ_TRY(check_rows(fn, "y_bf16", "ldy", y, ldy, N, 8));
    else
        FQ_TRY(check_vector(fn, "y_bf16", y));
    if (residual) FQ_TRY(check_rows(fn, "residual_bf16", "ldr", residual, ldr, N, 8));
    // y over the residual: each output has to replace the value that it adds (one token has one layout)
    if (residual == y && M > 1 && (head_dim == 0 ? ldr != ldy : head_dim != N || ldr != N))
        return fail(FQ_ERR_SHAPE, fmt("%s: y_bf16 is residual_bf16 in another layout (M=%d, ldr=%lld, ldy=%lld, head_dim=%d)",
                                      fn, M, (long long)ldr, (long long)ldy, head_dim));
    FQ_TRY(check_vector(fn, "act_codes", act));
    FQ_TRY(check_vector(fn, "act_scale", act_scale));
    FQ_TRY(check_vector(fn, "w_codes", w));
    if (!aligned(wscale, 4)) return fail(FQ_ERR_ALIGN, fmt("%s: wscale is not 4-byte aligned", fn));
    return check_vector(fn, "bias", bias);
}

fq::NormArgs prologue_args(const void* x, int32_t M, int32_t K, int64_t ldx, const float* gamma, float eps, void* codes,
                           float* scale) {
    fq::NormArgs a{};
    a.M = M;
    a.K = K;
    a.r_in = x;
    a.ld_rin = ldx;
    a.pre_norm = gamma != nullptr;
    a.pre_gamma = gamma;
    a.pre_eps = eps;
    a.rows_per_cond = 1;
    a.codes = static_cast<uint8_t*>(codes);
    a.act_scale = scale;
    return a;
}

fq_status run_fp8_gemm(const char* fn, const fq::Fp8Args& g, const fq::DeviceInfo& dev, hipStream_t stream) {
    if (fq::fp8_decode_codes_takes(g)) return device_status(fn, fq::launch_fp8_decode_codes(g, stream));
    return device_status(fn, fq::fp8_gemv_takes(g, dev) ? fq::launch_fp8_gemv(g, dev, stream)
                                                        : fq::launch_fp8_gemm(g, dev, stream));
}

}  // namespace

extern "C" {

size_t fq_fp8_ascale_count(int32_t M, int32_t K) {
    if (M < 1 || M > kMaxM || K < 128 || K > kMaxK || K % 128) return 0;
    return scale_bytes(M, K) / sizeof(float);
}

size_t fq_fp8_linear_workspace_bytes(int32_t M, int32_t K) {
    if (!fq_fp8_ascale_count(M, K)) return 0;
    const size_t tile = size_t(fq::kSplitEdge) * fq::kSplitEdge * sizeof(float);
    const size_t parts = fq::fp8_may_split(M, K) ? fq::kSplitTiles * tile : 0;
    return round_up(size_t(M) * size_t(K), 256) + round_up(scale_bytes(M, K), 256) + parts;
}

fq_status fq_fp8_prologue(const void* x_bf16, int32_t M, int32_t K, int64_t ldx, const float* gamma, float eps,
                          void* act_codes, float* act_scale, void* stream) {
    fq::clear_error();
    const char* fn = "fq_fp8_prologue";
    FQ_TRY(validate_fp8_prologue(fn, x_bf16, M, K, ldx, gamma, eps, act_codes, act_scale));
    const fq::DeviceInfo* dev = nullptr;
    FQ_TRY(prepare(fn, &dev));
    return device_status(fn, fq::launch_block_norm(prologue_args(x_bf16, M, K, ldx, gamma, eps, act_codes, act_scale),
                                                   static_cast<hipStream_t>(stream)));
}

fq_status fq_fp8_gemm(const void* act_codes, const float* act_scale, int32_t M, const void* w_codes,
                      const float* wscale, int32_t N, int32_t K, const float* bias, const void* residual_bf16,
                      int64_t ldr, int32_t head_dim, void* y_bf16, int64_t ldy, void* stream) {
    fq::clear_error();
    const char* fn = "fq_fp8_gemm";
    FQ_TRY(validate_fp8_gemm(fn, act_codes, act_scale, M, w_codes, wscale, N, K, bias, residual_bf16, ldr, head_dim,
                             y_bf16, ldy));
    const fq::DeviceInfo* dev = nullptr;
    FQ_TRY(prepare(fn, &dev));
    fq::Fp8Args g{static_cast<const uint8_t*>(act_codes), act_scale, M, static_cast<const uint8_t*>(w_codes), wscale,
                  N, K, bias, static_cast<const uint16_t*>(residual_bf16), ldr, static_cast<uint16_t*>(y_bf16), ldy,
                  head_dim};
    return run_fp8_gemm(fn, g, *dev, static_cast<hipStream_t>(stream));
}

fq_status fq_fp8_linear(const void* x_bf16, int32_t M, int32_t K, int64_t ldx, const float* gamma, float eps,
                        const void* w_codes, const float* wscale, int32_t N, const float* bias,
                        const void* residual_bf16, int64_t ldr, int32_t head_dim, void* y_bf16, int64_t ldy,
                        void* workspace, size_t workspace_bytes, void* stream) {
    fq::clear_error();
    const char* fn = "fq_fp8_linear";
    if (!workspace) return fail(FQ_ERR_ARG, fmt("%s: workspace is NULL", fn));
    if (!aligned(workspace, 256)) return fail(FQ_ERR_ALIGN, fmt("%s: workspace is not 256-byte aligned", fn));
    FQ_TRY(check_m(fn, M));
    FQ_TRY(check_k(fn, K, kGemmK));
    const size_t need = fq_fp8_linear_workspace_bytes(M, K);
    if (workspace_bytes < need)
        return fail(FQ_ERR_ARG, fmt("%s: workspace_bytes=%zu < %zu needed for M=%d K=%d", fn, workspace_bytes, need, M, K));
    uint8_t* const codes = static_cast<uint8_t*>(workspace);
    float* const scales = reinterpret_cast<float*>(codes + round_up(size_t(M) * size_t(K), 256));
    FQ_TRY(validate_fp8_prologue(fn, x_bf16, M, K, ldx, gamma, eps, codes, scales));
    FQ_TRY(validate_fp8_gemm(fn, codes, scales, M, w_codes, wscale, N, K, bias, residual_bf16, ldr, head_dim, y_bf16,
                             ldy));
    const fq::DeviceInfo* dev = nullptr;
    FQ_TRY(prepare(fn, &dev));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    fq::Fp8Args g{codes, scales, M, static_cast<const uint8_t*>(w_codes), wscale, N, K, bias,
                  static_cast<const uint16_t*>(residual_bf16), ldr, static_cast<uint16_t*>(y_bf16), ldy, head_dim};
    const fq::NormArgs a = prologue_args(x_bf16, M, K, ldx, gamma, eps, codes, scales);
    if (fq::fp8_decode_takes(a, g)) return device_status(fn, fq::launch_fp8_decode(a, g, *dev, s));
    FQ_TRY(device_status(fn, fq::launch_block_norm(a, s)));
    const fq::Fp8Split how = fq::fp8_split(g, *dev);
    if (how.splits > 1) {
        float* const part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(scales) + round_up(scale_bytes(M, K), 256));
        return device_status(fn, fq::launch_fp8_split(g, how, part, s));
    }
    return run_fp8_gemm(fn, g, *dev, s);
}

fq_status fq_block_norm(int32_t M, int32_t K, const void* x_bf16, int64_t ldx, const float* post_gamma, float post_eps,
                        const void* gate_bf16, int64_t ld_gate, float res_scale, const void* stream_in,
                        int64_t ld_in, void* stream_out, int64_t ld_out, int32_t stream_f32, const float* pre_gamma,
                        float pre_eps, const void* mod_scale_bf16, const void* mod_shift_bf16, int64_t ld_mod,
                        int32_t rows_per_cond, void* h_bf16, int64_t ld_h, void* act_codes, float* act_scale,
                        void* stream) {
    fq::clear_error();
    const char* fn = "fq_block_norm";
    FQ_TRY(check_m(fn, M));
    FQ_TRY(check_k(fn, K, act_codes ? kGemmK : 8));
    FQ_TRY(check_norm_launch(fn, M, K, stream_f32 != 0));
    if (stream_f32 != 0 && stream_f32 != 1)
        return fail(FQ_ERR_ARG, fmt("%s: stream_f32=%d must be 0 or 1", fn, stream_f32));
    if (!stream_in) return fail(FQ_ERR_ARG, fmt("%s: stream_in is NULL", fn));
    if (!x_bf16 && (post_gamma || gate_bf16 || stream_out))
        return fail(FQ_ERR_ARG, fmt("%s: post_gamma, gate_bf16 and stream_out need x_bf16", fn));
    if (x_bf16 && !stream_out) return fail(FQ_ERR_ARG, fmt("%s: stream_out is NULL", fn));
    if (!x_bf16 && !h_bf16 && !act_codes)
        return fail(FQ_ERR_ARG, fmt("%s: nothing to write: x_bf16, h_bf16 and act_codes are NULL", fn));
    if (!act_codes != !act_scale)
        return fail(FQ_ERR_ARG, fmt("%s: act_codes and act_scale come together", fn));
    if (!h_bf16 && !act_codes && (pre_gamma || mod_scale_bf16 || mod_shift_bf16))
        return fail(FQ_ERR_ARG, fmt("%s: pre_gamma, mod_scale_bf16 and mod_shift_bf16 need h_bf16 or act_codes", fn));
    const int mult = stream_f32 ? 4 : 8;
    FQ_TRY(check_rows(fn, "stream_in", "ld_in", stream_in, ld_in, K, mult));
    if (x_bf16) {
        FQ_TRY(check_rows(fn, "x_bf16", "ldx", x_bf16, ldx, K, 8));
        FQ_TRY(check_rows(fn, "stream_out", "ld_out", stream_out, ld_out, K, mult));
        if (stream_out == stream_in && ld_out != ld_in)
            return fail(FQ_ERR_SHAPE, fmt("%s: an update in place needs ld_out=%lld equal to ld_in=%lld", fn,
                                          (long long)ld_out, (long long)ld_in));
        if (!std::isfinite(res_scale))
            return fail(FQ_ERR_ARG, fmt("%s: res_scale=%g must be finite", fn, double(res_scale)));
    }
    if (post_gamma) FQ_TRY(check_eps(fn, "post_eps", post_eps));
    if (h_bf16 || act_codes) FQ_TRY(check_eps(fn, "pre_eps", pre_eps));
    if (gate_bf16 || mod_scale_bf16 || mod_shift_bf16) {
        if (rows_per_cond < 1) return fail(FQ_ERR_SHAPE, fmt("%s: rows_per_cond=%d must be >= 1", fn, rows_per_cond));
        if (gate_bf16) FQ_TRY(check_rows(fn, "gate_bf16", "ld_gate", gate_bf16, ld_gate, K, 8));
        if (mod_scale_bf16) FQ_TRY(check_rows(fn, "mod_scale_bf16", "ld_mod", mod_scale_bf16, ld_mod, K, 8));
        if (mod_shift_bf16) FQ_TRY(check_rows(fn, "mod_shift_bf16", "ld_mod", mod_shift_bf16, ld_mod, K, 8));
    }
    FQ_TRY(check_vector(fn, "post_gamma", post_gamma));
    FQ_TRY(check_vector(fn, "pre_gamma", pre_gamma));
    if (h_bf16) FQ_TRY(check_rows(fn, "h_bf16", "ld_h", h_bf16, ld_h, K, 8));
    FQ_TRY(check_vector(fn, "act_codes", act_codes));
    FQ_TRY(check_vector(fn, "act_scale", act_scale));
    const fq::DeviceInfo* dev = nullptr;
    FQ_TRY(prepare(fn, &dev));
    fq::NormArgs a{M, K, static_cast<const uint16_t*>(x_bf16), ldx, post_gamma, post_eps,
                   static_cast<const uint16_t*>(gate_bf16), ld_gate, res_scale, stream_in, ld_in, stream_out, ld_out,
                   stream_f32, 1, pre_gamma, pre_eps, static_cast<const uint16_t*>(mod_scale_bf16),
                   static_cast<const uint16_t*>(mod_shift_bf16), ld_mod, rows_per_cond < 1 ? 1 : rows_per_cond,
                   static_cast<uint16_t*>(h_bf16), ld_h, static_cast<uint8_t*>(act_codes), act_scale};
    return device_status(fn, fq::launch_block_norm(a, static_cast<hipStream_t>(stream)));
}

fq_status fq_rope(const void* x_bf16, int64_t x_token, int64_t x_head, int32_t M, int32_t heads, int32_t rot_heads,
                  int32_t head_dim, int32_t rot_dim, int32_t interleaved, const uint64_t* freq, float attn_scale,
                  const int32_t* positions, int32_t pos0, int32_t inverse, void* y_bf16, int64_t y_token,
                  int64_t y_head, void* stream) {
    fq::clear_error();
    const char* fn = "fq_rope";
    if (!x_bf16) return fail(FQ_ERR_ARG, fmt("%s: x_bf16 is NULL", fn));
    if (!y_bf16) return fail(FQ_ERR_ARG, fmt("%s: y_bf16 is NULL", fn));
    if (!freq) return fail(FQ_ERR_ARG, fmt("%s: freq is NULL", fn));
    FQ_TRY(check_m(fn, M));
    if (heads < 1 || heads > 65535) return fail(FQ_ERR_SHAPE, fmt("%s: heads=%d outside [1, 65535]", fn, heads));
    if (rot_heads < 0 || rot_heads > heads)
        return fail(FQ_ERR_SHAPE, fmt("%s: rot_heads=%d outside [0, heads=%d]", fn, rot_heads, heads));
    if (head_dim < 8 || head_dim > kMaxK || head_dim % 8)
        return fail(FQ_ERR_SHAPE, fmt("%s: head_dim=%d must be a multiple of 8 in [8, %d]", fn, head_dim, kMaxK));
    if (rot_dim < 2 || rot_dim > head_dim || rot_dim % 2)
        return fail(FQ_ERR_SHAPE, fmt("%s: rot_dim=%d must be even and in [2, head_dim=%d]", fn, rot_dim, head_dim));
    if (int64_t(M) * (head_dim / 2) + 256 >= kMaxThreads)
        return fail(FQ_ERR_SHAPE, fmt("%s: M=%d x head_dim=%d is too large for one launch", fn, M, head_dim));
    if (interleaved != 0 && interleaved != 1)
        return fail(FQ_ERR_ARG, fmt("%s: interleaved=%d must be 0 or 1", fn, interleaved));
    if (inverse != 0 && inverse != 1) return fail(FQ_ERR_ARG, fmt("%s: inverse=%d must be 0 or 1", fn, inverse));
    if (!std::isfinite(attn_scale))
        return fail(FQ_ERR_ARG, fmt("%s: attn_scale=%g must be finite", fn, double(attn_scale)));
    if (!positions && int64_t(pos0) + M - 1 > INT32_MAX)
        return fail(FQ_ERR_ARG, fmt("%s: pos0=%d + M=%d passes the last position 2^31 - 1", fn, pos0, M));
    FQ_TRY(check_head_strides(fn, "x_token", x_token, "x_head", x_head, head_dim));
    FQ_TRY(check_head_strides(fn, "y_token", y_token, "y_head", y_head, head_dim));
    FQ_TRY(check_heads_apart(fn, "y_token", y_token, "y_head", y_head, heads, M, head_dim));
    if (x_bf16 == y_bf16 && (x_token != y_token || x_head != y_head))
        return fail(FQ_ERR_SHAPE, fmt("%s: a rotation in place needs the strides of x and y equal", fn));
    FQ_TRY(check_vector(fn, "x_bf16", x_bf16));
    FQ_TRY(check_vector(fn, "y_bf16", y_bf16));
    if (!aligned(freq, 16)) return fail(FQ_ERR_ALIGN, fmt("%s: freq is not 16-byte aligned", fn));
    if (!aligned(positions, 4)) return fail(FQ_ERR_ALIGN, fmt("%s: positions is not 4-byte aligned", fn));
    const fq::DeviceInfo* dev = nullptr;
    FQ_TRY(prepare(fn, &dev));
    fq::RopeArgs a{static_cast<const uint16_t*>(x_bf16), x_token, x_head, M, heads, rot_heads, head_dim, rot_dim,
                   interleaved, freq, attn_scale, positions, pos0, inverse, static_cast<uint16_t*>(y_bf16), y_token,
                   y_head};
    return device_status(fn, fq::launch_rope(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
