// Addresses of the FP8 GEMM's copies from global memory into a stage of LDS.
// Plain arithmetic, also compiled by the host compiler, where it is checked.
//
// A copy moves 8 rows of 128 codes with one buffer load of 16 bytes a lane.  A
// buffer load adds two offsets to its descriptor's base: one of the lane, which
// the range check against the descriptor's size always sees, and one common to
// the wave, which the check may leave out, or subtract from the size first.  So
// the rows are in the lane's offset alone: a row past the operand's last lies
// at or beyond the size whatever the check does with the other one, which holds
// the stage's place along k, less than a row.
#pragma once

#include <cstdint>

#if defined(__HIPCC__)
#define FQ_COPY_FN __host__ __device__ __forceinline__
#else
#define FQ_COPY_FN inline
#endif

namespace fq {

// LDS layout of a 128-byte row rho: chunk c of 16 bytes at slot 8 rho + (c ^ swizzle).
FQ_COPY_FN int fp8_swizzle(int rho) { return (rho >> 1) & 7; }

struct Fp8CopyOffset {
    uint32_t lane;    // of the lane: row and chunk
    uint32_t common;  // of the wave: place along k
};

// The lane's offset in the 8 rows of a copy: lane l fills the slot of row l / 8,
// chunk (l % 8) ^ swizzle; `odd`: the copy's first row is an odd multiple of 8.
FQ_COPY_FN uint32_t fp8_copy_lane(int lane, int odd, int K) {
    return uint32_t((lane >> 3) * K + 16 * ((lane & 7) ^ fp8_swizzle(8 * odd + (lane >> 3))));
}

// Rows row .. row + 7 (from the descriptor's first), unit `unit` of 128 k.
FQ_COPY_FN Fp8CopyOffset fp8_copy_at(uint32_t copy_lane, int row, int unit, int K) {
    return Fp8CopyOffset{copy_lane + uint32_t(row * K), uint32_t(128 * unit)};
}

}  // namespace fq
