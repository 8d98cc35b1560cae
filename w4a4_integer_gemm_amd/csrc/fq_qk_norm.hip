// Norm of the query and key heads of every token and their rotation in one pass (gfx950, wave64).
//
//   n = x * (1/sqrt(mean(x^2) + eps)) * gamma,  (a, b) -> (a c - b s, b c + a s)
//
// over the head_dim values of a head; heads behind the queries and keys are
// copied.  Bound by reading and writing the heads once.  As in fq_rope a thread
// owns one item of one token, two 16-byte pieces: with halves the pieces of 8 `a`
// elements and of their 8 `b` elements, so that every pair is inside a thread,
// otherwise two neighbouring pieces.  head_dim / 16 items make a head; they sit
// in 1 to 16 consecutive lanes (a power of two), which add their sums of squares
// with lane moves.  A thread computes its item's angles once and applies them to
// its share of the heads, UN heads' loads ahead of their stores.  Sum, root, gain and rotation
// are float32, one rounding to bf16 at the end.
//
// 4571 tokens of 36 heads of 128: 15.5 us for 84 MB (5.4 TB/s, the Infinity Cache helping).
// One token of 12 heads of 256: 3.8 us, a launch, one memory latency and eight pairs' angles in turn.
#include <hip/hip_runtime.h>

#include "fq_angle.h"
#include "fq_device.h"
#include "fq_internal.h"
#include "fq_row_norm.h"
#include "fq_token.h"

namespace fq {
namespace {

// Sum over L consecutive lanes (a power of two up to 32, aligned).
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
    if constexpr (L > 1) v += __int_as_float(dpp_i<0xB1>(__float_as_int(v)));   // quad_perm [1,0,3,2]
    if constexpr (L > 2) v += __int_as_float(dpp_i<0x4E>(__float_as_int(v)));   // quad_perm [2,3,0,1]
    if constexpr (L > 4) v += __int_as_float(dpp_i<0x141>(__float_as_int(v)));  // row_half_mirror
    if constexpr (L > 8) v += __int_as_float(dpp_i<0x140>(__float_as_int(v)));  // row_mirror
    if constexpr (L > 16) v += __shfl_xor(v, 16);
    return v;
}

__device__ __forceinline__ float sumsq16(const float (&p)[8], const float (&q)[8]) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = __builtin_fmaf(p[j], p[j], s);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = __builtin_fmaf(q[j], q[j], s);
    return s;
}

__device__ __forceinline__ void load_gain(const float* g, int e, float (&o)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = g ? g[e + j] : 1.0f;
}

// blockIdx.y: heads [y * share, (y + 1) * share); UN of them at a time.
// Pieces are whole: rot_dim a multiple of 16 with halves, of 8 interleaved.
template <bool INTER, int L, int UN>
__global__ __launch_bounds__(256) void qk_norm_kernel(QkNormArgs a, int share) {
    const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
    const uint32_t m = idx / L;
    if (m >= uint32_t(a.M)) return;
    const int items = a.head_dim / 16, rot_items = a.rot_dim / 16;
    const bool active = int(idx % L) < items;
    const int item = active ? int(idx % L) : items - 1;  // (the lanes past the last item repeat it and store nothing)
    // elements of the two pieces
    const bool halves = !INTER && item < rot_items;
    const int ea = halves ? 8 * item : 16 * item, eb = halves ? ea + a.rot_dim / 2 : ea + 8;
    const bool rot_a = INTER ? ea < a.rot_dim : halves, rot_b = INTER ? eb < a.rot_dim : halves;
    float c[8], s[8];  // of the 8 pairs; interleaved: of the 4 pairs of each piece
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = 1.0f, s[j] = 0.0f;
    if (rot_a) {
        const int32_t pos = a.positions ? a.positions[m] : a.pos0 + int32_t(m);
        uint64_t f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = a.freq[8 * item + (!INTER || rot_b || j < 4 ? j : 0)];  // (one that exists)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            cos_sin_turns(angle(f[j], pos), &c[j], &s[j]);
            c[j] *= a.attn_scale;
            s[j] *= a.attn_scale;
            if (INTER && j >= 4 && !rot_b) c[j] = 1.0f, s[j] = 0.0f;
        }
    }
    const int h0 = blockIdx.y * share, h1 = h0 + share < a.heads ? h0 + share : a.heads;
    const int normed = a.q_heads + a.k_heads;
    const uint16_t* const xp = a.x + m * a.x_token;
    uint16_t* const yp = a.y + m * a.y_token;
    const bool in_place = a.x == a.y;
    float ga[8], gb[8];
    bool have_k = h0 >= a.q_heads;
    load_gain(have_k ? a.k_gamma : a.q_gamma, ea, ga);
    load_gain(have_k ? a.k_gamma : a.q_gamma, eb, gb);
    for (int h = h0; h < h1; h += UN) {
        uint4 u[UN], v[UN];
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            const int hk = h + k < h1 ? h + k : h1 - 1;  // (past the share: loaded again, not stored)
            u[k] = *reinterpret_cast<const uint4*>(xp + hk * a.x_head + ea);
            v[k] = *reinterpret_cast<const uint4*>(xp + hk * a.x_head + eb);
        }
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            if (h + k >= h1) break;
            if (h + k < normed) {
                if (!have_k && h + k >= a.q_heads) {
                    have_k = true;
                    load_gain(a.k_gamma, ea, ga);
                    load_gain(a.k_gamma, eb, gb);
                }
                float p[8], q[8], r[8], t[8];
                unpack8(u[k], p);
                unpack8(v[k], q);
                const float ss = lanes_sum<L>(active ? sumsq16(p, q) : 0.0f);
                const float inv = 1.0f / sqrtf(ss / float(a.head_dim) + a.eps);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    p[j] = p[j] * inv * ga[j];
                    q[j] = q[j] * inv * gb[j];
                }
                if constexpr (INTER) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        r[2 * j] = __builtin_fmaf(p[2 * j], c[j], -(p[2 * j + 1] * s[j]));
                        r[2 * j + 1] = __builtin_fmaf(p[2 * j + 1], c[j], p[2 * j] * s[j]);
                        t[2 * j] = __builtin_fmaf(q[2 * j], c[4 + j], -(q[2 * j + 1] * s[4 + j]));
                        t[2 * j + 1] = __builtin_fmaf(q[2 * j + 1], c[4 + j], q[2 * j] * s[4 + j]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        r[j] = __builtin_fmaf(p[j], c[j], -(q[j] * s[j]));
                        t[j] = __builtin_fmaf(q[j], c[j], p[j] * s[j]);
                    }
                }
                u[k] = pack8(r);
                v[k] = pack8(t);
            } else if (in_place) {
                continue;
            }
            if (active) {
                *reinterpret_cast<uint4*>(yp + (h + k) * a.y_head + ea) = u[k];
                *reinterpret_cast<uint4*>(yp + (h + k) * a.y_head + eb) = v[k];
            }
        }
    }
}

// Any even rot_dim: an element's partner may be in any lane, so a head's normed values pass
// through LDS.  A thread owns 8 consecutive elements of one token, L lanes a head.  20000 tokens of 18
// heads of 80, 40 of them rotated in halves: 54 to 56 us for 115 MB (2.1 TB/s); with 32 in halves, which the kernel
// above takes, 25.2.
template <int L>
__global__ __launch_bounds__(256) void qk_norm_any_kernel(QkNormArgs a, int share) {
    // (the lanes of a head are in one wave, whose LDS accesses stay in order)
    __shared__ __attribute__((aligned(16))) float rows[256 / L][8 * L + 4];
    const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
    const uint32_t m = idx / L;
    if (m >= uint32_t(a.M)) return;
    const bool active = int(idx % L) < a.head_dim / 8;
    const int e = active ? 8 * int(idx % L) : 0, rh = a.rot_dim / 2;  // (the lanes past the head repeat its first piece)
    float* const row = rows[threadIdx.x / L];
    int partner[8];
    uint64_t f[8];
    float c[8], s[8];  // y = n c + partner s
    const int32_t pos = a.positions ? a.positions[m] : a.pos0 + int32_t(m);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int x = e + j;
        const bool rotated = x < a.rot_dim;
        partner[j] = !rotated ? x : a.interleaved ? x ^ 1 : x < rh ? x + rh : x - rh;
        f[j] = a.freq[!rotated ? 0 : a.interleaved ? x / 2 : x < rh ? x : x - rh];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        cos_sin_turns(angle(f[j], pos), &c[j], &s[j]);
        c[j] *= a.attn_scale;
        s[j] *= e + j < partner[j] ? -a.attn_scale : a.attn_scale;
        if (e + j >= a.rot_dim) c[j] = 1.0f, s[j] = 0.0f;
    }
    const int h0 = blockIdx.y * share, h1 = h0 + share < a.heads ? h0 + share : a.heads;
    const uint16_t* const xp = a.x + m * a.x_token + e;
    uint4 next[2];  // the two heads behind the current one
#pragma unroll
    for (int k = 0; k < 2; ++k) next[k] = *reinterpret_cast<const uint4*>(xp + min(h0 + k, h1 - 1) * a.x_head);
    for (int h = h0; h < h1; ++h) {
        uint4 u = next[0];
        next[0] = next[1];
        next[1] = *reinterpret_cast<const uint4*>(xp + min(h + 2, h1 - 1) * a.x_head);
        if (h < a.q_heads + a.k_heads) {
            const float* const g = h < a.q_heads ? a.q_gamma : a.k_gamma;
            float p[8];
            unpack8(u, p);
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(p[j], p[j], ss);
            ss = lanes_sum<L>(active ? ss : 0.0f);
            const float inv = 1.0f / sqrtf(ss / float(a.head_dim) + a.eps);
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = p[j] * inv * (g ? g[e + j] : 1.0f);
            if (active) {
                *reinterpret_cast<float4*>(row + e) = make_float4(p[0], p[1], p[2], p[3]);
                *reinterpret_cast<float4*>(row + e + 4) = make_float4(p[4], p[5], p[6], p[7]);
            }
            asm volatile("" ::: "memory");
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = __builtin_fmaf(p[j], c[j], row[partner[j]] * s[j]);
            asm volatile("" ::: "memory");
            u = pack8(p);
        } else if (a.x == a.y) {
            continue;
        }
        if (active) *reinterpret_cast<uint4*>(a.y + m * a.y_token + h * a.y_head + e) = u;
    }
}

// Heads per thread: as in fq_rope, all of them where the tokens alone fill the
// chip (the angles are then computed once), fewer below kFill threads.
constexpr int64_t kFill = 256 * 1024;

template <bool INTER, int L>
hipError_t launch_items(const QkNormArgs& a, hipStream_t st) {
    const int64_t threads = int64_t(a.M) * L;
    int64_t parts = kFill / threads;
    parts = parts < 1 ? 1 : parts > a.heads ? a.heads : parts;
    const int share = int((a.heads + parts - 1) / parts);
    const dim3 grid(uint32_t((threads + 255) / 256), uint32_t((a.heads + share - 1) / share));
    if (share == 1)
        hipLaunchKernelGGL((qk_norm_kernel<INTER, L, 1>), grid, dim3(256), 0, st, a, share);
    else
        hipLaunchKernelGGL((qk_norm_kernel<INTER, L, 2>), grid, dim3(256), 0, st, a, share);
    return hipGetLastError();
}

template <bool INTER>
hipError_t launch_lanes(const QkNormArgs& a, hipStream_t st) {
    const int items = a.head_dim / 16;
    if (items <= 1) return launch_items<INTER, 1>(a, st);
    if (items <= 2) return launch_items<INTER, 2>(a, st);
    if (items <= 4) return launch_items<INTER, 4>(a, st);
    if (items <= 8) return launch_items<INTER, 8>(a, st);
    return launch_items<INTER, 16>(a, st);
}

template <int L>
hipError_t launch_any(const QkNormArgs& a, hipStream_t st) {
    const int64_t threads = int64_t(a.M) * L;
    int64_t parts = kFill / threads;
    parts = parts < 1 ? 1 : parts > a.heads ? a.heads : parts;
    const int share = int((a.heads + parts - 1) / parts);
    hipLaunchKernelGGL((qk_norm_any_kernel<L>), dim3(uint32_t((threads + 255) / 256), uint32_t((a.heads + share - 1) / share)),
                       dim3(256), 0, st, a, share);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_norm(const QkNormArgs& a, hipStream_t stream) {
    if (a.interleaved && a.rot_dim % 8 == 0) return launch_lanes<true>(a, stream);
    if (!a.interleaved && a.rot_dim % 16 == 0) return launch_lanes<false>(a, stream);
    if (a.head_dim <= 16) return launch_any<2>(a, stream);
    if (a.head_dim <= 32) return launch_any<4>(a, stream);
    if (a.head_dim <= 64) return launch_any<8>(a, stream);
    if (a.head_dim <= 128) return launch_any<16>(a, stream);
    return launch_any<32>(a, stream);
}

}  // namespace fq
