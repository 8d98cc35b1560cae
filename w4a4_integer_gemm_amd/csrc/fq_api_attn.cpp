// C ABI of the operators between the qkv site and the o site: norms of query
// and key heads with their rotation, the paged cache, attention.  Validation and
// dispatch; every check runs before any HIP call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/fq.h"
#include "fq_check.h"
#include "fq_internal.h"
#include "fq_paged.h"

namespace {

constexpr int32_t kMaxHeadDim = 256, kMaxHeads = 65535, kMaxKvHeads = 32767, kMaxPage = 32768;
constexpr int64_t kMaxKeyStride = 1 << 24;  // a tile's 64 rows stay inside a 32-bit byte offset

fq_status check_attn_head_dim(const char* fn, int32_t head_dim) {
    if (head_dim < 16 || head_dim > kMaxHeadDim || head_dim % 16)
        return fail(FQ_ERR_SHAPE, fmt("%s: head_dim=%d must be a multiple of 16 in [16, %d]", fn, head_dim, kMaxHeadDim));
    return FQ_OK;
}

fq_status check_groups(const char* fn, int32_t q_heads, int32_t kv_heads) {
    if (q_heads < 1 || q_heads > kMaxHeads)
        return fail(FQ_ERR_SHAPE, fmt("%s: q_heads=%d outside [1, %d]", fn, q_heads, kMaxHeads));
    if (kv_heads < 1 || kv_heads > kMaxKvHeads)
        return fail(FQ_ERR_SHAPE, fmt("%s: kv_heads=%d outside [1, %d]", fn, kv_heads, kMaxKvHeads));
    if (q_heads % kv_heads)
        return fail(FQ_ERR_SHAPE, fmt("%s: q_heads=%d is not a whole number of groups of kv_heads=%d (%d/%d = %.3f)", fn,
                                      q_heads, kv_heads, q_heads, kv_heads, double(q_heads) / kv_heads));
    return FQ_OK;
}

// Heads of `heads` x M rows: pointer and strides; `out`: they must not overlap.
fq_status check_head_rows(const char* fn, const char* name, const void* p, const char* token_name, int64_t token,
                          const char* head_name, int64_t head, int32_t heads, int32_t M, int32_t head_dim, bool out) {
    if (!p) return fail(FQ_ERR_ARG, fmt("%s: %s is NULL", fn, name));
    FQ_TRY(check_head_strides(fn, token_name, token, head_name, head, head_dim));
    if (out) FQ_TRY(check_heads_apart(fn, token_name, token, head_name, head, heads, M, head_dim));
    return check_vector(fn, name, p);
}

fq_status check_int32s(const char* fn, const char* name, const int32_t* p) {
    if (!p) return fail(FQ_ERR_ARG, fmt("%s: %s is NULL", fn, name));
    if (!aligned(p, 4)) return fail(FQ_ERR_ALIGN, fmt("%s: %s is not 4-byte aligned", fn, name));
    return FQ_OK;
}

fq_status check_cache(const char* fn, const void* k, const void* v, const float* ks, const float* vs, int32_t kv_bits,
                      int32_t pages, int32_t page_size, int32_t kv_heads, int32_t head_dim) {
    if (!k) return fail(FQ_ERR_ARG, fmt("%s: k_cache is NULL", fn));
    if (!v) return fail(FQ_ERR_ARG, fmt("%s: v_cache is NULL", fn));
    if (kv_bits != 8 && kv_bits != 16)
        return fail(FQ_ERR_UNSUPPORTED, fmt("%s: kv_bits=%d is not a supported width (8 or 16)", fn, kv_bits));
    if (kv_bits == 8 && (!ks || !vs)) return fail(FQ_ERR_ARG, fmt("%s: kv_bits=8 needs k_scale and v_scale", fn));
    if (kv_bits == 16 && (ks || vs)) return fail(FQ_ERR_ARG, fmt("%s: kv_bits=16 takes no k_scale and v_scale", fn));
    FQ_TRY(check_attn_head_dim(fn, head_dim));
    if (kv_heads < 1 || kv_heads > kMaxKvHeads)
        return fail(FQ_ERR_SHAPE, fmt("%s: kv_heads=%d outside [1, %d]", fn, kv_heads, kMaxKvHeads));
    if (page_size < 16 || page_size > kMaxPage || page_size % 16)
        return fail(FQ_ERR_SHAPE, fmt("%s: page_size=%d must be a multiple of 16 in [16, %d]", fn, page_size, kMaxPage));
    if (pages < 1 || int64_t(pages) * page_size > INT32_MAX)
        return fail(FQ_ERR_SHAPE, fmt("%s: pages=%d of page_size=%d must be at least 1 and hold fewer than 2^31 tokens", fn,
                                      pages, page_size));
    FQ_TRY(check_vector(fn, "k_cache", k));
    FQ_TRY(check_vector(fn, "v_cache", v));
    FQ_TRY(check_vector(fn, "k_scale", ks));
    return check_vector(fn, "v_scale", vs);
}

fq::KvCache cache_of(const void* k, const void* v, const float* ks, const float* vs, int32_t pages, int32_t page_size,
                     int32_t kv_heads, int32_t head_dim) {
    return fq::KvCache{const_cast<void*>(k), const_cast<void*>(v), const_cast<float*>(ks), const_cast<float*>(vs),
                       pages, page_size, kv_heads, head_dim};
}

// Rows of M tokens' heads that a launch takes a few lanes each.
fq_status check_kv_launch(const char* fn, int32_t M, int32_t head_dim) {
    if (int64_t(M) * (head_dim / 4) + 256 >= kMaxThreads)
        return fail(FQ_ERR_SHAPE, fmt("%s: M=%d x head_dim=%d is too large for one launch", fn, M, head_dim));
    return FQ_OK;
}

}  // namespace

extern "C" {

fq_status fq_qk_norm_rope(const void* x_bf16, int64_t x_token, int64_t x_head, int32_t M, int32_t heads,
                          int32_t q_heads, int32_t k_heads, int32_t head_dim, const float* q_gamma,
                          const float* k_gamma, float eps, int32_t rot_dim, int32_t interleaved, const uint64_t* freq,
                          float attn_scale, const int32_t* positions, int32_t pos0, void* y_bf16, int64_t y_token,
                          int64_t y_head, void* stream) {
    fq::clear_error();
    const char* fn = "fq_qk_norm_rope";
    FQ_TRY(check_m(fn, M));
    FQ_TRY(check_attn_head_dim(fn, head_dim));
    if (heads < 1 || heads > kMaxHeads) return fail(FQ_ERR_SHAPE, fmt("%s: heads=%d outside [1, %d]", fn, heads, kMaxHeads));
    if (q_heads < 0 || k_heads < 0 || int64_t(q_heads) + k_heads > heads)
        return fail(FQ_ERR_SHAPE, fmt("%s: q_heads=%d and k_heads=%d must be >= 0 and at most heads=%d together", fn, q_heads,
                                      k_heads, heads));
    if (int64_t(M) * 64 + 256 >= kMaxThreads)
        return fail(FQ_ERR_SHAPE, fmt("%s: M=%d is too large for one launch", fn, M));
    FQ_TRY(check_eps(fn, "eps", eps));
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 2)
        return fail(FQ_ERR_SHAPE, fmt("%s: rot_dim=%d must be even and in [0, head_dim=%d]", fn, rot_dim, head_dim));
    if (interleaved != 0 && interleaved != 1)
        return fail(FQ_ERR_ARG, fmt("%s: interleaved=%d must be 0 or 1", fn, interleaved));
    if (rot_dim) {
        if (!freq) return fail(FQ_ERR_ARG, fmt("%s: freq is NULL", fn));
        if (!std::isfinite(attn_scale))
            return fail(FQ_ERR_ARG, fmt("%s: attn_scale=%g must be finite", fn, double(attn_scale)));
        if (!positions && int64_t(pos0) + M - 1 > INT32_MAX)
            return fail(FQ_ERR_ARG, fmt("%s: pos0=%d + M=%d passes the last position 2^31 - 1", fn, pos0, M));
    }
    FQ_TRY(check_head_rows(fn, "x_bf16", x_bf16, "x_token", x_token, "x_head", x_head, heads, M, head_dim, false));
    FQ_TRY(check_head_rows(fn, "y_bf16", y_bf16, "y_token", y_token, "y_head", y_head, heads, M, head_dim, true));
    if (x_bf16 == y_bf16 && (x_token != y_token || x_head != y_head))
        return fail(FQ_ERR_SHAPE, fmt("%s: an update in place needs the strides of x and y equal", fn));
    FQ_TRY(check_vector(fn, "q_gamma", q_gamma));
    FQ_TRY(check_vector(fn, "k_gamma", k_gamma));
    FQ_TRY(check_vector(fn, "freq", freq));
    if (!aligned(positions, 4)) return fail(FQ_ERR_ALIGN, fmt("%s: positions is not 4-byte aligned", fn));
    const fq::DeviceInfo* dev = nullptr;
    FQ_TRY(prepare(fn, &dev));
    const fq::QkNormArgs a{static_cast<const uint16_t*>(x_bf16), x_token, x_head, M, heads, q_heads, k_heads, head_dim,
                           q_gamma, k_gamma, eps, rot_dim, interleaved, freq, attn_scale, positions, pos0,
                           static_cast<uint16_t*>(y_bf16), y_token, y_head};
    return device_status(fn, fq::launch_qk_norm(a, static_cast<hipStream_t>(stream)));
}

fq_status fq_kv_write(const void* k_bf16, int64_t k_token, int64_t k_head, const void* v_bf16, int64_t v_token,
                      int64_t v_head, const int32_t* slots, int32_t M, int32_t kv_heads, int32_t head_dim,
                      int32_t kv_bits, int32_t pages, int32_t page_size, void* k_cache, void* v_cache, float* k_scale,
                      float* v_scale, void* stream) {
    fq::clear_error();
    const char* fn = "fq_kv_write";
    FQ_TRY(check_m(fn, M));
    FQ_TRY(check_cache(fn, k_cache, v_cache, k_scale, v_scale, kv_bits, pages, page_size, kv_heads, head_dim));
    FQ_TRY(check_kv_launch(fn, M, head_dim));
    FQ_TRY(check_head_rows(fn, "k_bf16", k_bf16, "k_token", k_token, "k_head", k_head, kv_heads, M, head_dim, false));
    FQ_TRY(check_head_rows(fn, "v_bf16", v_bf16, "v_token", v_token, "v_head", v_head, kv_heads, M, head_dim, false));
    FQ_TRY(check_int32s(fn, "slots", slots));
    const fq::DeviceInfo* dev = nullptr;
    FQ_TRY(prepare(fn, &dev));
    const fq::KvCache c = cache_of(k_cache, v_cache, k_scale, v_scale, pages, page_size, kv_heads, head_dim);
    const fq::KvRows k{static_cast<uint16_t*>(const_cast<void*>(k_bf16)), k_token, k_head};
    const fq::KvRows v{static_cast<uint16_t*>(const_cast<void*>(v_bf16)), v_token, v_head};
    return device_status(fn, fq::launch_kv_write(c, k, v, slots, M, static_cast<hipStream_t>(stream)));
}

fq_status fq_kv_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                     int32_t kv_bits, int32_t pages, int32_t page_size, const int32_t* slots, int32_t M,
                     int32_t kv_heads, int32_t head_dim, void* k_bf16, int64_t k_token, int64_t k_head, void* v_bf16,
                     int64_t v_token, int64_t v_head, void* stream) {
    fq::clear_error();
    const char* fn = "fq_kv_read";
    FQ_TRY(check_m(fn, M));
    FQ_TRY(check_cache(fn, k_cache, v_cache, k_scale, v_scale, kv_bits, pages, page_size, kv_heads, head_dim));
    FQ_TRY(check_kv_launch(fn, M, head_dim));
    FQ_TRY(check_head_rows(fn, "k_bf16", k_bf16, "k_token", k_token, "k_head", k_head, kv_heads, M, head_dim, true));
    FQ_TRY(check_head_rows(fn, "v_bf16", v_bf16, "v_token", v_token, "v_head", v_head, kv_heads, M, head_dim, true));
    if (k_bf16 == v_bf16) return fail(FQ_ERR_ARG, fmt("%s: k_bf16 and v_bf16 are the same", fn));
    FQ_TRY(check_int32s(fn, "slots", slots));
    const fq::DeviceInfo* dev = nullptr;
    FQ_TRY(prepare(fn, &dev));
    const fq::KvCache c = cache_of(k_cache, v_cache, k_scale, v_scale, pages, page_size, kv_heads, head_dim);
    const fq::KvRows k{static_cast<uint16_t*>(k_bf16), k_token, k_head}, v{static_cast<uint16_t*>(v_bf16), v_token, v_head};
    return device_status(fn, fq::launch_kv_read(c, k, v, slots, M, static_cast<hipStream_t>(stream)));
}

fq_status fq_attn_prefill(const void* q_bf16, int64_t q_token, int64_t q_head, const void* k_bf16, int64_t k_token,
                          int64_t k_head, const void* v_bf16, int64_t v_token, int64_t v_head, int32_t M, int32_t M_k,
                          const int32_t* cu_q, const int32_t* cu_k, int32_t seqs, int32_t q_heads, int32_t kv_heads,
                          int32_t head_dim, float scale, int32_t causal, void* o_bf16, int64_t o_token, int64_t o_head,
                          void* stream) {
    fq::clear_error();
    const char* fn = "fq_attn_prefill";
    FQ_TRY(check_m(fn, M));
    if (M_k < 1 || M_k > kMaxM) return fail(FQ_ERR_SHAPE, fmt("%s: M_k=%d must be in [1, %d]", fn, M_k, kMaxM));
    if (seqs < 1 || seqs > (1 << 20)) return fail(FQ_ERR_SHAPE, fmt("%s: seqs=%d outside [1, %d]", fn, seqs, 1 << 20));
    FQ_TRY(check_groups(fn, q_heads, kv_heads));
    FQ_TRY(check_attn_head_dim(fn, head_dim));
    if (!std::isfinite(scale)) return fail(FQ_ERR_ARG, fmt("%s: scale=%g must be finite", fn, double(scale)));
    if (causal != 0 && causal != 1) return fail(FQ_ERR_ARG, fmt("%s: causal=%d must be 0 or 1", fn, causal));
    const fq::PrefillArgs a{static_cast<const uint16_t*>(q_bf16), q_token, q_head, static_cast<const uint16_t*>(k_bf16),
                            k_token, k_head, static_cast<const uint16_t*>(v_bf16), v_token, v_head, M, M_k, cu_q,
                            cu_k ? cu_k : cu_q, seqs, q_heads, kv_heads, head_dim, scale, causal,
                            static_cast<uint16_t*>(o_bf16), o_token, o_head};
    const int forced = fq::hooks().attn_prefill.load(std::memory_order_relaxed);
    if ((int64_t(M) / fq::kPrefillRows + seqs) * q_heads >= kMaxThreads / 512 ||
        (forced >= 0 && fq::attn_prefill_threads(a, forced) >= kMaxThreads))
        return fail(FQ_ERR_SHAPE, fmt("%s: M=%d rows of %d sequences x q_heads=%d are too many for one launch", fn, M, seqs,
                                      q_heads));
    FQ_TRY(check_head_rows(fn, "q_bf16", q_bf16, "q_token", q_token, "q_head", q_head, q_heads, M, head_dim, false));
    FQ_TRY(check_head_rows(fn, "k_bf16", k_bf16, "k_token", k_token, "k_head", k_head, kv_heads, M_k, head_dim, false));
    FQ_TRY(check_head_rows(fn, "v_bf16", v_bf16, "v_token", v_token, "v_head", v_head, kv_heads, M_k, head_dim, false));
    FQ_TRY(check_head_rows(fn, "o_bf16", o_bf16, "o_token", o_token, "o_head", o_head, q_heads, M, head_dim, true));
    if (k_token > kMaxKeyStride || v_token > kMaxKeyStride)
        return fail(FQ_ERR_SHAPE, fmt("%s: k_token=%lld and v_token=%lld must be at most 2^24", fn, (long long)k_token,
                                      (long long)v_token));
    FQ_TRY(check_int32s(fn, "cu_q", cu_q));
    if (!aligned(cu_k, 4)) return fail(FQ_ERR_ALIGN, fmt("%s: cu_k is not 4-byte aligned", fn));
    const fq::DeviceInfo* dev = nullptr;
    FQ_TRY(prepare(fn, &dev));
    return device_status(fn, fq::launch_attn_prefill(a, *dev, static_cast<hipStream_t>(stream)));
}

size_t fq_attn_decode_workspace_bytes(int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t max_len) {
    if (seqs < 1 || q_heads < 1 || q_heads > kMaxHeads || kv_heads < 1 || kv_heads > kMaxKvHeads || q_heads % kv_heads ||
        head_dim < 16 || head_dim > kMaxHeadDim || head_dim % 16 || max_len < 1 || max_len > fq::kDecodeMaxLen)
        return 0;
    return fq::decode_workspace(seqs, q_heads, kv_heads, head_dim, max_len).bytes;
}

fq_status fq_attn_decode(const void* q_bf16, int64_t q_token, int64_t q_head, int32_t seqs, int32_t q_heads,
                         int32_t kv_heads, int32_t head_dim, float scale, const void* k_cache, const void* v_cache,
                         const float* k_scale, const float* v_scale, int32_t kv_bits, int32_t pages, int32_t page_size,
                         const int32_t* page_table, int32_t max_pages, const int32_t* lens, void* o_bf16,
                         int64_t o_token, int64_t o_head, void* workspace, size_t workspace_bytes, void* stream) {
    fq::clear_error();
    const char* fn = "fq_attn_decode";
    if (seqs < 1) return fail(FQ_ERR_SHAPE, fmt("%s: seqs=%d must be >= 1", fn, seqs));
    FQ_TRY(check_groups(fn, q_heads, kv_heads));
    FQ_TRY(check_cache(fn, k_cache, v_cache, k_scale, v_scale, kv_bits, pages, page_size, kv_heads, head_dim));
    if (max_pages < 1 || int64_t(max_pages) * page_size > fq::kDecodeMaxLen)
        return fail(FQ_ERR_SHAPE, fmt("%s: max_pages=%d of page_size=%d must be at least 1 and hold at most 2^30 tokens", fn,
                                      max_pages, page_size));
    if (!std::isfinite(scale)) return fail(FQ_ERR_ARG, fmt("%s: scale=%g must be finite", fn, double(scale)));
    FQ_TRY(check_head_rows(fn, "q_bf16", q_bf16, "q_token", q_token, "q_head", q_head, q_heads, seqs, head_dim, false));
    FQ_TRY(check_head_rows(fn, "o_bf16", o_bf16, "o_token", o_token, "o_head", o_head, q_heads, seqs, head_dim, true));
    FQ_TRY(check_int32s(fn, "page_table", page_table));
    FQ_TRY(check_int32s(fn, "lens", lens));
    const int32_t max_len = max_pages * page_size;
    const int64_t parts = fq::decode_parts(seqs, q_heads, kv_heads, max_len);
    if (parts * kv_heads * fq::decode_head_tiles(q_heads, kv_heads) >= kMaxThreads / 256 ||
        int64_t(seqs) * q_heads >= kMaxThreads / 256)
        return fail(FQ_ERR_SHAPE, fmt("%s: seqs=%d x q_heads=%d are too many for one launch", fn, seqs, q_heads));
    if (!workspace) return fail(FQ_ERR_ARG, fmt("%s: workspace is NULL", fn));
    if (!aligned(workspace, 256)) return fail(FQ_ERR_ALIGN, fmt("%s: workspace is not 256-byte aligned", fn));
    const fq::DecodeWorkspace ws = fq::decode_workspace(seqs, q_heads, kv_heads, head_dim, max_len);
    if (workspace_bytes < ws.bytes)
        return fail(FQ_ERR_ARG, fmt("%s: workspace_bytes=%zu < %zu needed for seqs=%d q_heads=%d kv_heads=%d head_dim=%d "
                                    "max_pages=%d page_size=%d", fn, workspace_bytes, ws.bytes, seqs, q_heads, kv_heads,
                                    head_dim, max_pages, page_size));
    const fq::DeviceInfo* dev = nullptr;
    FQ_TRY(prepare(fn, &dev));
    uint8_t* const base = static_cast<uint8_t*>(workspace);
    const fq::DecodeArgs a{static_cast<const uint16_t*>(q_bf16), q_token, q_head, seqs, q_heads, scale,
                           cache_of(k_cache, v_cache, k_scale, v_scale, pages, page_size, kv_heads, head_dim), page_table,
                           max_pages, lens, static_cast<uint16_t*>(o_bf16), o_token, o_head,
                           static_cast<int2*>(workspace), reinterpret_cast<float2*>(base + ws.stats),
                           reinterpret_cast<float*>(base + ws.sums), int32_t(parts)};
    return device_status(fn, fq::launch_attn_decode(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
