// Pieces shared by the attention kernels (gfx950, wave64): matrix instructions
// on bf16, lane exchanges, the softmax's base.
//
// Scores are kept in the base of two: p = 2^(s - max), s = scale log2(e) <q, k>.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fq_device.h"
#include "fq_paged.h"

namespace fq {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 0x1.715476p+0f;

// D[16][16] (+)= A[16][32] B[32][16]: lane l gives row (column) l % 16 and the same
// 8 of the 32 k on both sides, and holds D[4 (l / 16) + i][l % 16] in register i.
__device__ __forceinline__ v4f mfma_bf16_16(v8bf a, v8bf b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// D[32][32] (+)= A[32][16] B[16][32]: lane l gives row (column) l % 32 and 8 of the 16
// k, and holds D[8 (i / 4) + 4 (l / 32) + i % 4][l % 32] in register i.
__device__ __forceinline__ v16f mfma_bf16_32(v8bf a, v8bf b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ v8bf as_bf(uint4 v) { return __builtin_bit_cast(v8bf, v); }

// The value of lane l xor 32 (16) joined with the own one.
__device__ __forceinline__ float max_over_halves(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_int(x), __float_as_int(x), false, false);
    return fmaxf(__int_as_float(a[0]), __int_as_float(a[1]));
}
__device__ __forceinline__ float sum_over_halves(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_int(x), __float_as_int(x), false, false);
    return __int_as_float(a[0]) + __int_as_float(a[1]);
}
__device__ __forceinline__ float max_over_rows(float x) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_int(x), __float_as_int(x), false, false);
    return max_over_halves(fmaxf(__int_as_float(a[0]), __int_as_float(a[1])));
}
__device__ __forceinline__ float sum_over_rows(float x) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_int(x), __float_as_int(x), false, false);
    return sum_over_halves(__int_as_float(a[0]) + __int_as_float(a[1]));
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// A uniform load that the vector loads in flight need not be waited for.
typedef const int32_t __attribute__((address_space(4)))* const_i32;
__device__ __forceinline__ int32_t scalar_load(const int32_t* p, int64_t i) {
    return reinterpret_cast<const_i32>(reinterpret_cast<uintptr_t>(p))[i];
}

// The sequence that block b of a packed launch belongs to: sequence s has the blocks
// first(s), which grows by at least one with s, and the ones behind it.  -1: none.
template <class First>
__device__ __forceinline__ int find_sequence(int seqs, int64_t b, First first) {
    if (seqs == 1) return 0;
    const int lane = threadIdx.x & 63;
    return __builtin_amdgcn_readfirstlane(last_not_past(seqs, [&](int at, int step, int probes) {
        return __popcll(__ballot(lane < probes && first(at + lane * step) <= b));
    }));
}
// Rows of sequence s, cut off at [0, M].
struct Rows {
    int begin, count;
};
__device__ __forceinline__ Rows sequence_rows(const int32_t* cu, int s, int M) {
    const int begin = max(0, min(scalar_load(cu, s), M));
    return Rows{begin, max(0, min(scalar_load(cu, s + 1), M) - begin)};
}

}  // namespace fq
