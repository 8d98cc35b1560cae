// cos and sin of a rotary position's angles, shared by the kernels that rotate (gfx950).
//
// The angle is computed in integers: freq[i] is the turns per position as a
// 64-bit fraction (a whole turn = 2^64), so position * freq modulo 2^64 is the
// angle's fraction of a turn with no rounding at all, at any position; its top
// 32 bits give the angle to 2^-32 turns.  cos and sin come from their Taylor
// series on an eighth of a turn around the nearest quarter (remainders below
// 2^-28), in float32: its conversion moves the angle by up to 2^-26 turns.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fq {

// cos and sin of `turns` * 2 pi, turns given as a fraction of 2^32.
__device__ __forceinline__ void cos_sin_turns(uint32_t turns, float* c, float* s) {
    const uint32_t quarter = (turns + 0x20000000u) >> 30;
    const int32_t off = int32_t(turns - (quarter << 30));  // in [-2^29, 2^29): an eighth of a turn each way
    const float x = float(off) * 0x1.921fb6p-30f;          // 2 pi / 2^32 (float32 nearest)
    const float x2 = x * x;
    float sn = __builtin_fmaf(x2, 1.0f / 362880.0f, -1.0f / 5040.0f);
    sn = __builtin_fmaf(x2, sn, 1.0f / 120.0f);
    sn = __builtin_fmaf(x2, sn, -1.0f / 6.0f);
    sn = __builtin_fmaf(x * x2, sn, x);
    float cs = __builtin_fmaf(x2, -1.0f / 3628800.0f, 1.0f / 40320.0f);
    cs = __builtin_fmaf(x2, cs, -1.0f / 720.0f);
    cs = __builtin_fmaf(x2, cs, 1.0f / 24.0f);
    cs = __builtin_fmaf(x2, cs, -0.5f);
    cs = __builtin_fmaf(x2, cs, 1.0f);
    const float cq = (quarter & 1) ? sn : cs, sq = (quarter & 1) ? cs : sn;
    // quarters 0..3: (c, s), (-s, c), (-c, -s), (s, -c)
    *c = (quarter == 1 || quarter == 2) ? -cq : cq;
    *s = (quarter & 2) ? -sq : sq;
}

__device__ __forceinline__ uint32_t angle(uint64_t f, int32_t pos) {
    return uint32_t((f * uint64_t(int64_t(pos))) >> 32);
}

}  // namespace fq
