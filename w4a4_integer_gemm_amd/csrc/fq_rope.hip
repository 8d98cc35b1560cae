// Rotary positions on the heads of a projection's output (gfx950, wave64).
//
// Pair i of a rotated head turns by the angle of freq[i] turns per position:
//   (a, b) -> (a c - b s, b c + a s),  c = scale cos, s = scale sin,
// a and b being elements i and i + rot_dim/2 of the head, or 2 i and 2 i + 1
// (interleaved); elements from rot_dim on and the heads from rot_heads on are
// copied.  `inverse` applies the transposed map (s negated).
//
// Bound by reading and writing the heads once.  A thread owns one item of one
// token: with halves the 16-byte piece of 8 `a` elements and the piece of their
// 8 `b` elements, interleaved one piece of 4 pairs, past rot_dim one copied piece.
// It computes the item's angles once and applies them to its share of the heads,
// UN heads' loads ahead of their stores.  (rot_dim not a multiple of 16, or of 8
// interleaved, has pieces that are neither: those sizes, and small calls, take
// a thread per pair of every head.  Where such a call is large, its two-byte accesses
// and an angle for every head cost twice the time: 24571 tokens x 18 heads x 80 with
// halves of rot_dim 40 70 us, 2.0 TB/s, against 31 us with rot_dim 32.)
#include <hip/hip_runtime.h>

#include "fq_angle.h"
#include "fq_device.h"
#include "fq_internal.h"
#include "fq_row_norm.h"
#include "fq_token.h"

namespace fq {
namespace {

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }
__device__ __forceinline__ uint16_t to_bf16(float v) { return uint16_t(pack_bf16x2(v, 0.0f)); }

__device__ __forceinline__ void angles(const RopeArgs& a, int32_t pos, int i0, int n, float* c, float* s) {
#pragma unroll
    for (int j = 0; j < n; ++j) {
        cos_sin_turns(angle(a.freq[i0 + j], pos), &c[j], &s[j]);
        c[j] *= a.attn_scale;
        s[j] *= a.inverse ? -a.attn_scale : a.attn_scale;
    }
}

// Rotates the pieces u, v (halves) or u alone (interleaved).
template <bool INTER>
__device__ __forceinline__ void rotate(uint4& u, uint4& v, const float (&c)[8], const float (&s)[8]) {
    float p[8], q[8];
    unpack8(u, p);
    if constexpr (INTER) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            q[2 * j] = __builtin_fmaf(p[2 * j], c[j], -(p[2 * j + 1] * s[j]));
            q[2 * j + 1] = __builtin_fmaf(p[2 * j + 1], c[j], p[2 * j] * s[j]);
        }
        u = pack8(q);
    } else {
        float r[8];
        unpack8(v, q);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[j] = __builtin_fmaf(p[j], c[j], -(q[j] * s[j]));
            q[j] = __builtin_fmaf(q[j], c[j], p[j] * s[j]);
        }
        u = pack8(r);
        v = pack8(q);
    }
}

// blockIdx.y: heads [y * share, (y + 1) * share); UN of them at a time.
template <bool INTER, int UN>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, uint32_t items, int share) {
    const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
    const uint32_t m = idx / items, item = idx - m * items;
    if (m >= uint32_t(a.M)) return;
    const uint32_t rot_items = uint32_t(a.rot_dim) / (INTER ? 8u : 16u);
    const bool rot = item < rot_items;
    // element of u, and the distance from u to v
    const int e = 8 * int(rot || INTER ? item : item + rot_items);
    const int dv = !INTER && rot ? a.rot_dim / 2 : 0;
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = 1.0f, s[j] = 0.0f;
    if (rot) {
        const int32_t pos = a.positions ? a.positions[m] : a.pos0 + int32_t(m);
        angles(a, pos, INTER ? 4 * int(item) : 8 * int(item), INTER ? 4 : 8, c, s);
    }
    const int h0 = blockIdx.y * share, h1 = h0 + share < a.heads ? h0 + share : a.heads;
    const uint16_t* const xp = a.x + m * a.x_token + e;
    uint16_t* const yp = a.y + m * a.y_token + e;
    const bool in_place = a.x == a.y;
    for (int h = h0; h < h1; h += UN) {
        uint4 u[UN], v[UN];
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            const int hk = h + k < h1 ? h + k : h1 - 1;  // (past the share: loaded again, not stored)
            u[k] = *reinterpret_cast<const uint4*>(xp + hk * a.x_head);
            if (!INTER) v[k] = *reinterpret_cast<const uint4*>(xp + hk * a.x_head + dv);
        }
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            const bool turn = rot && h + k < a.rot_heads;
            if (h + k >= h1 || (in_place && !turn)) continue;
            if (turn) rotate<INTER>(u[k], v[k], c, s);
            *reinterpret_cast<uint4*>(yp + (h + k) * a.y_head) = u[k];
            if (!INTER && rot) *reinterpret_cast<uint4*>(yp + (h + k) * a.y_head + dv) = v[k];
        }
    }
}

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
    const int h = blockIdx.y;
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

}  // namespace

// Few pairs take a thread each, whose chain is one angle instead of eight
// (graph-replayed, us, pairs against items: 1 x 12 x 256 1.93 / 2.55, 56 x 36 x
// 128 2.2 / 2.65, 512 x 36 x 128 4.98 / 3.78).
constexpr int64_t kFewPairs = 128 * 1024;
// Heads per thread: all of them where the tokens alone fill the chip (the angles
// are then computed once), fewer below kFill threads, one for a few tokens.
constexpr int64_t kFill = 256 * 1024;

template <bool INTER>
hipError_t launch_items(const RopeArgs& a, hipStream_t st) {
    const uint32_t items = INTER ? a.head_dim / 8 : a.rot_dim / 16 + (a.head_dim - a.rot_dim) / 8;
    const int64_t threads = int64_t(a.M) * items;
    int64_t parts = kFill / threads;
    parts = parts < 1 ? 1 : parts > a.heads ? a.heads : parts;
    const int share = int((a.heads + parts - 1) / parts);
    const dim3 grid(uint32_t((threads + 255) / 256), uint32_t((a.heads + share - 1) / share));
    if (share == 1)
        hipLaunchKernelGGL((rope_kernel<INTER, 1>), grid, dim3(256), 0, st, a, items, share);
    else if (share <= 3)
        hipLaunchKernelGGL((rope_kernel<INTER, 2>), grid, dim3(256), 0, st, a, items, share);
    else
        hipLaunchKernelGGL((rope_kernel<INTER, 4>), grid, dim3(256), 0, st, a, items, share);
    return hipGetLastError();
}

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
    const bool few = int64_t(a.M) * a.heads * (a.head_dim / 2) <= kFewPairs;
    if (!few && a.interleaved && a.rot_dim % 8 == 0) return launch_items<true>(a, stream);
    if (!few && !a.interleaved && a.rot_dim % 16 == 0) return launch_items<false>(a, stream);
    const int64_t threads = int64_t(a.M) * (a.head_dim / 2);
    hipLaunchKernelGGL(rope_pairs_kernel, dim3(uint32_t((threads + 255) / 256), a.heads), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace fq
