// Rotary positions on the heads of a projection's output (gfx950, wave64).
//
// Pair i of a rotated head turns by the angle of freq[i] turns per position:
//   (a, b) -> (a c - b s, b c + a s),  c = scale cos, s = scale sin,
// a and b being elements i and i + rot_dim/2 of the head, or 2 i and 2 i + 1
// (interleaved); elements from rot_dim on and the heads from rot_heads on are
// copied.  `inverse` applies the transposed map (s negated).
//
// The angle is computed in integers: freq[i] is the turns per position as a
// 64-bit fraction (a whole turn = 2^64), so position * freq modulo 2^64 is the
// angle's fraction of a turn with no rounding at all, at any position; its top
// 32 bits give the angle to 2^-32 turns.  cos and sin come from their Taylor
// series on an eighth of a turn around the nearest quarter (remainders below
// 2^-28), in float32.
//
// Bound by reading and writing the heads once.  A thread owns one 16-byte piece
// of `a` and one of `b` (interleaved: two pieces) of one token, computes its 8
// angles once and applies them to its share of the heads.
#include <hip/hip_runtime.h>

#include "fq_device.h"
#include "fq_internal.h"
#include "fq_token.h"

namespace fq {
namespace {

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

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }
__device__ __forceinline__ uint16_t to_bf16(float v) { return uint16_t(pack_bf16x2(v, 0.0f)); }

// One element pair (or copied pair of elements) per thread: any even rot_dim.
__global__ __launch_bounds__(256) void rope_pairs_kernel(RopeArgs a) {
    const int half = a.head_dim / 2, rh = a.rot_dim / 2;
    const int64_t idx = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (idx >= int64_t(a.M) * half) return;
    const int m = int(idx / half), i = int(idx % half);
    const bool rot = i < rh;
    float c = 1.0f, s = 0.0f;
    int e0 = 2 * i, e1 = 2 * i + 1;  // (past rot_dim: two copied elements)
    if (rot) {
        const int32_t pos = a.positions ? a.positions[m] : a.pos0 + m;
        cos_sin_turns(angle(a.freq[i], pos), &c, &s);
        c *= a.attn_scale;
        s *= a.inverse ? -a.attn_scale : a.attn_scale;
        if (!a.interleaved) e0 = i, e1 = i + rh;
    }
    for (int h = blockIdx.y; h < a.heads; h += gridDim.y) {
        const uint16_t* xp = a.x + m * a.x_token + h * a.x_head;
        uint16_t* yp = a.y + m * a.y_token + h * a.y_head;
        const uint16_t u = xp[e0], v = xp[e1];
        if (rot && h < a.rot_heads) {
            const float p = bf16_value(u), q = bf16_value(v);
            yp[e0] = to_bf16(__builtin_fmaf(p, c, -(q * s)));
            yp[e1] = to_bf16(__builtin_fmaf(q, c, p * s));
        } else if (xp != yp) {
            yp[e0] = u;
            yp[e1] = v;
        }
    }
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
    const int64_t threads = int64_t(a.M) * (a.head_dim / 2);
    hipLaunchKernelGGL(rope_pairs_kernel, dim3(uint32_t((threads + 255) / 256), a.heads), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace fq
