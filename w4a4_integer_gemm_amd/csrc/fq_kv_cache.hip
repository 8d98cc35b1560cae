// The paged cache of keys and values: tokens written, as bf16 or as e4m3 codes
// with a scale for a token's head, and read back (gfx950, wave64).
//
// Bound by moving the rows once.  A row is one token's key (or value) of one
// head; head_dim / 8 lanes hold 8 values each and sit in 2 to 32 consecutive
// lanes (a power of two), which find the row's maximum with lane moves.
// Consecutive rows are consecutive tokens of one head: they lie behind one
// another in the head layout and in a page, so that a wave reads and writes whole
// lines.  A thread takes a piece of the key and the same of the value (blockIdx.y: the
// head), whose loads are in flight together.
//
// e4m3: s = max|h| / 448 in float32, q = e4m3(h / s) with one rounding to nearest even; read back as
// bf16(s q), one rounding more.  A row's scale is one store of the lane that holds its first piece.
// 32768 tokens, 8 heads of 128, e4m3: written in 39 us, read in 34 to 39 (204 MB, 5.2 and 5.3 to 5.9 TB/s; with a
// thread each for key and value 46.5 and 43.1); bf16 53 and 41 (269 MB, 5.1 and 6.5 TB/s, the Infinity Cache
// helping).  4571 tokens read in 6.9 us, 4580 of 4 heads written in 5.1: one round of waves, slot, row and store three
// latencies in a chain.
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

// Index of a slot's row of a head.
__device__ __forceinline__ int64_t slot_row(const KvCache& c, int32_t slot, int head) {
    const int32_t page = slot / c.page_size;
    return paged_row(page, slot - page * c.page_size, head, c.kv_heads, c.page_size);
}

template <int L, bool FP8>
__global__ __launch_bounds__(256) void kv_write_kernel(KvCache c, KvRows k, KvRows v, const int32_t* slots, int32_t M) {
    const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
    const uint32_t m = idx / L;
    if (m >= uint32_t(M)) return;
    const int e = 8 * int(idx % L), head = blockIdx.y;
    const bool active = e < c.head_dim;
    const int32_t slot = slots[m];
    const int at = active ? e : 0;
    const uint4 x = *reinterpret_cast<const uint4*>(k.p + m * k.token + head * k.head + at);
    const uint4 y = *reinterpret_cast<const uint4*>(v.p + m * v.token + head * v.head + at);
    if (slot < 0 || slot >= c.pages * c.page_size) return;  // (all lanes of a row)
    const int64_t row = slot_row(c, slot, head);
    if constexpr (!FP8) {
        if (!active) return;
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(c.k) + 2 * (row * c.head_dim + e)) = x;
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(c.v) + 2 * (row * c.head_dim + e)) = y;
    } else {
        auto one = [&](const uint4& in, void* rows, float* scales) {
            float h[8];
            unpack8(in, h);
            uint32_t t = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) t = max(t, __float_as_uint(h[j]) & 0x7FFFFFFFu);
            const float s = fp8_scale(lanes_max_nonneg<L>(__uint_as_float(t)));
            if (active) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(rows) + row * c.head_dim + e) = fp8_codes8(h, s);
            if (e == 0) scales[row] = s;
        };
        one(x, c.k, c.k_scale);
        one(y, c.v, c.v_scale);
    }
}

template <int L, bool FP8>
__global__ __launch_bounds__(256) void kv_read_kernel(KvCache c, KvRows k, KvRows v, const int32_t* slots, int32_t M) {
    const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
    const uint32_t m = idx / L;
    const int e = 8 * int(idx % L), head = blockIdx.y;
    if (m >= uint32_t(M) || e >= c.head_dim) return;
    const int32_t slot = slots[m];
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (slot >= 0 && slot < c.pages * c.page_size) {
        const int64_t row = slot_row(c, slot, head);
        if constexpr (!FP8) {
            x = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c.k) + 2 * (row * c.head_dim + e));
            y = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c.v) + 2 * (row * c.head_dim + e));
        } else {
            const uint2 p = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.k) + row * c.head_dim + e);
            const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.v) + row * c.head_dim + e);
            const float ps = c.k_scale[row], qs = c.v_scale[row];
            auto one = [](const uint2& q, float s) {
                const uint32_t w[2] = {q.x, q.y};
                float h[8];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(w[j]), false);
                    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(w[j]), true);
                    h[4 * j] = lo[0] * s, h[4 * j + 1] = lo[1] * s, h[4 * j + 2] = hi[0] * s, h[4 * j + 3] = hi[1] * s;
                }
                return pack8(h);
            };
            x = one(p, ps);
            y = one(q, qs);
        }
    }
    *reinterpret_cast<uint4*>(k.p + m * k.token + head * k.head + e) = x;
    *reinterpret_cast<uint4*>(v.p + m * v.token + head * v.head + e) = y;
}

template <int L>
hipError_t launch_lanes(bool write, const KvCache& c, const KvRows& k, const KvRows& v, const int32_t* slots, int32_t M,
                        hipStream_t st) {
    const dim3 grid(uint32_t((int64_t(M) * L + 255) / 256), uint32_t(c.kv_heads));
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
