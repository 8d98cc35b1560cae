// E4M3 codes with one float32 scale for 128 values (gfx950, wave64): the
// quantisation shared by the kernels that write them.
//
//   s = max|h| / 448 (IEEE float32), q = e4m3(h / s), rounded to nearest, ties
//   to even, clamped to +-448; a group whose scale is zero has zero codes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fq_device.h"
#include "fq_token.h"

namespace fq {

// Maximum over 16 consecutive lanes (a DPP row) of values that are >= 0 and not NaN.
__device__ __forceinline__ float max16_nonneg(float x) {
    uint32_t v = __float_as_uint(x);
    v = max(v, uint32_t(dpp_i<0xB1>(int(v))));   // quad_perm [1,0,3,2]
    v = max(v, uint32_t(dpp_i<0x4E>(int(v))));   // quad_perm [2,3,0,1]
    v = max(v, uint32_t(dpp_i<0x141>(int(v))));  // row_half_mirror
    v = max(v, uint32_t(dpp_i<0x140>(int(v))));  // row_mirror
    return __uint_as_float(v);
}

__device__ __forceinline__ float fp8_scale(float amax) { return amax / 448.0f; }

// The codes of four values, each already divided by its scale and within +-448.
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

// Codes of 8 values with scale s = fp8_scale(their group's maximum).
//
// Where r = 1/s is normal and the remainder cannot underflow (s in [2^-100,
// 2^100]) the quotient is q0 = h r corrected by fma(fma(-s, q0, h), r, q0): the
// IEEE quotient (Markstein), 3 operations instead of a divide's ten.  There
// |h| / s <= 448 (1 + 2^-23), which rounds to 448: the clamp is implied.  Other
// scales (a maximum below 2^-91, above 2^108, zero or not finite) divide and
// clamp each value; the comparisons keep a NaN.
__device__ __forceinline__ uint2 fp8_codes8(const float (&h)[8], float s) {
    float q[8];
    if (s >= 0x1p-100f && s <= 0x1p+100f) {
        const float r = 1.0f / s;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q0 = h[i] * r;
            q[i] = __builtin_fmaf(__builtin_fmaf(-s, q0, h[i]), r, q0);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = s == 0.0f ? (h[i] == h[i] ? 0.0f : h[i]) : h[i] / s;
            q[i] = d > 448.0f ? 448.0f : d < -448.0f ? -448.0f : d;
        }
    }
    return make_uint2(fp8_pack4(q[0], q[1], q[2], q[3]), fp8_pack4(q[4], q[5], q[6], q[7]));
}

}  // namespace fq
