// The paged cache of keys and values: tokens written, as bf16 or as e4m3 codes
// with a scale for a token's head, and read back (gfx950, wave64).
//
// Bound by moving the rows once.  A row is one token's key (or value) of one
// head; head_dim / 8 lanes hold 8 values each and sit in 2 to 32 consecutive
// lanes (a power of two), which find the row's maximum with lane moves.
// Consecutive rows are consecutive tokens of one head: they lie behind one
// another in the head layout and in a page, so that a wave reads and writes whole
// lines.  blockIdx.y: 2 * head + (0: key, 1: value).
//
// e4m3: s = max|h| / 448 in float32, q = e4m3(h / s) with one rounding to nearest even; read back as
// bf16(s q), one rounding more.  A row's scale is one store of the lane that holds its first piece.
// 4580 tokens, 4 heads of 128, e4m3: written in 4.7 us (14 MB, 3.0 TB/s); 4571 tokens, 8 heads, read in 6.9 us
// (28 MB, 4.1 TB/s).  Both are one round of waves: slot, row and store are three latencies in
// a chain.  A thread with two or four tokens of a head, all loaded before the first store, was slower (8.0 us
// for the reading).
#include <hip/hip_runtime.h>

#include "fq_device.h"
#include "fq_fp8.h"
#include "fq_internal.h"
#include "fq_paged.h"
#include "fq_row_norm.h"
#include "fq_token.h"

namespace fq {
namespace {

// Maximum over L consecutive lanes (a power of two up to 32, aligned) of values >= 0 or NaN.
template <int L>
__device__ __forceinline__ float lanes_max_nonneg(float x) {
    uint32_t v = __float_as_uint(x);
    if constexpr (L > 1) v = max(v, uint32_t(dpp_i<0xB1>(int(v))));   // quad_perm [1,0,3,2]
    if constexpr (L > 2) v = max(v, uint32_t(dpp_i<0x4E>(int(v))));   // quad_perm [2,3,0,1]
    if constexpr (L > 4) v = max(v, uint32_t(dpp_i<0x141>(int(v))));  // row_half_mirror
    if constexpr (L > 8) v = max(v, uint32_t(dpp_i<0x140>(int(v))));  // row_mirror
    if constexpr (L > 16) v = max(v, uint32_t(__shfl_xor(int(v), 16)));
    return __uint_as_float(v);
}

template <int L, bool FP8>
__global__ __launch_bounds__(256) void kv_write_kernel(KvCache c, KvRows k, KvRows v, const int32_t* slots, int32_t M) {
    const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
    const uint32_t m = idx / L;
    if (m >= uint32_t(M)) return;
    const int e = 8 * int(idx % L), head = blockIdx.y >> 1;
    const bool value = blockIdx.y & 1, active = e < c.head_dim;
    const KvRows& src = value ? v : k;
    const int32_t slot = slots[m];
    if (slot < 0 || slot >= c.pages * c.page_size) return;  // (all lanes of a row)
    const uint4 x = active ? *reinterpret_cast<const uint4*>(src.p + m * src.token + head * src.head + e)
                           : make_uint4(0, 0, 0, 0);
    const int32_t page = slot / c.page_size;
    const int64_t row = paged_row(page, slot - page * c.page_size, head, c.kv_heads, c.page_size);
    uint8_t* const rows = static_cast<uint8_t*>(value ? c.v : c.k);
    if constexpr (!FP8) {
        if (active) *reinterpret_cast<uint4*>(rows + 2 * (row * c.head_dim + e)) = x;
    } else {
        float h[8], top = 0.0f;
        unpack8(x, h);
        uint32_t t = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) t = max(t, __float_as_uint(h[j]) & 0x7FFFFFFFu);
        top = lanes_max_nonneg<L>(__uint_as_float(t));
        const float s = fp8_scale(top);
        if (active) *reinterpret_cast<uint2*>(rows + row * c.head_dim + e) = fp8_codes8(h, s);
        if (e == 0) (value ? c.v_scale : c.k_scale)[row] = s;
    }
}

template <int L, bool FP8>
__global__ __launch_bounds__(256) void kv_read_kernel(KvCache c, KvRows k, KvRows v, const int32_t* slots, int32_t M) {
    const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
    const uint32_t m = idx / L;
    const int e = 8 * int(idx % L), head = blockIdx.y >> 1;
    if (m >= uint32_t(M) || e >= c.head_dim) return;
    const bool value = blockIdx.y & 1;
    const KvRows& dst = value ? v : k;
    const int32_t slot = slots[m];
    uint4 x = make_uint4(0, 0, 0, 0);
    if (slot >= 0 && slot < c.pages * c.page_size) {
        const int32_t page = slot / c.page_size;
        const int64_t row = paged_row(page, slot - page * c.page_size, head, c.kv_heads, c.page_size);
        const uint8_t* const rows = static_cast<const uint8_t*>(value ? c.v : c.k);
        if constexpr (!FP8) {
            x = *reinterpret_cast<const uint4*>(rows + 2 * (row * c.head_dim + e));
        } else {
            const uint2 q = *reinterpret_cast<const uint2*>(rows + row * c.head_dim + e);
            const float s = (value ? c.v_scale : c.k_scale)[row];
            const uint32_t w[2] = {q.x, q.y};
            float h[8];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(w[j]), false);
                const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(w[j]), true);
                h[4 * j] = lo[0] * s, h[4 * j + 1] = lo[1] * s, h[4 * j + 2] = hi[0] * s, h[4 * j + 3] = hi[1] * s;
            }
            x = pack8(h);
        }
    }
    *reinterpret_cast<uint4*>(dst.p + m * dst.token + head * dst.head + e) = x;
}

template <int L>
hipError_t launch_lanes(bool write, const KvCache& c, const KvRows& k, const KvRows& v, const int32_t* slots, int32_t M,
                        hipStream_t st) {
    const dim3 grid(uint32_t((int64_t(M) * L + 255) / 256), uint32_t(2 * c.kv_heads));
    if (write && c.k_scale)
        hipLaunchKernelGGL((kv_write_kernel<L, true>), grid, dim3(256), 0, st, c, k, v, slots, M);
    else if (write)
        hipLaunchKernelGGL((kv_write_kernel<L, false>), grid, dim3(256), 0, st, c, k, v, slots, M);
    else if (c.k_scale)
        hipLaunchKernelGGL((kv_read_kernel<L, true>), grid, dim3(256), 0, st, c, k, v, slots, M);
    else
        hipLaunchKernelGGL((kv_read_kernel<L, false>), grid, dim3(256), 0, st, c, k, v, slots, M);
    return hipGetLastError();
}

hipError_t launch(bool write, const KvCache& c, const KvRows& k, const KvRows& v, const int32_t* slots, int32_t M,
                  hipStream_t st) {
    const int pieces = c.head_dim / 8;
    if (pieces <= 2) return launch_lanes<2>(write, c, k, v, slots, M, st);
    if (pieces <= 4) return launch_lanes<4>(write, c, k, v, slots, M, st);
    if (pieces <= 8) return launch_lanes<8>(write, c, k, v, slots, M, st);
    if (pieces <= 16) return launch_lanes<16>(write, c, k, v, slots, M, st);
    return launch_lanes<32>(write, c, k, v, slots, M, st);
}

}  // namespace

hipError_t launch_kv_write(const KvCache& c, const KvRows& k, const KvRows& v, const int32_t* slots, int32_t M,
                           hipStream_t stream) {
    return launch(true, c, k, v, slots, M, stream);
}

hipError_t launch_kv_read(const KvCache& c, const KvRows& k, const KvRows& v, const int32_t* slots, int32_t M,
                          hipStream_t stream) {
    return launch(false, c, k, v, slots, M, stream);
}

}  // namespace fq
