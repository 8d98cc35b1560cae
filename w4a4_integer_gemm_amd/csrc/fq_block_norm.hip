// Norms before and after a block, with the gate, the residual scale and the
// stream update between them, in one pass over the rows (gfx950, wave64); the
// same kernel is the FP8 sites' prologue with a norm (no block output, codes out).
//
//   p  = x * (1/sqrt(mean(x^2) + post_eps)) * post_gamma      (post norm, optional)
//   p  = p * gate[m / rows_per_cond]                          (optional)
//   r' = r + res_scale * p, rounded to the stream's type      (only with x)
//   h  = r' * (1/sqrt(mean(r'^2) + pre_eps)) * pre_gamma      (the rounded r')
//   h  = h * (1 + mod_scale[m / rows_per_cond]) + mod_shift[m / rows_per_cond]
// and h leaves as bf16 and/or as e4m3 codes q = rne(h / s) with one scale
// s = max|h| / 448 for every 128 consecutive values.  float32 throughout with
// one rounding per operation; both sums of squares are float64 (the squares
// are exact there), mean = (float)(sum / K).
//
// One workgroup per row; lane t holds pieces t, t + T, ... of 8 consecutive
// values, so every access of a wave covers contiguous memory and the 128
// values of one scale group sit in 16 consecutive lanes, whose maximum takes
// four DPP steps.  The row stays in registers between the two norms: x and r
// are read once, r' and h written once.  (Rows of more than 32768 values, eight
// pieces a lane, spill 14 to 63 registers to scratch on the way: 1024 x 40960 to bf16
// 47 us, 3.6 TB/s, to codes 83 us, where 1024 x 32768 takes 29, 4.7 TB/s, and 30.)
#include <hip/hip_runtime.h>

#include <type_traits>

#include "fq_device.h"
#include "fq_fp8.h"
#include "fq_internal.h"
#include "fq_row_norm.h"
#include "fq_token.h"

namespace fq {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxWaves = kMaxThreads / 64;

// A row's vectors that a lane needs, by piece: gains float32, conditions bf16.
template <int P>
struct Vectors {
    float4 post[P][2], pre[P][2];
    uint4 gate[P], scale[P], shift[P];
};

// P pieces of 8 values per lane; F32: the stream is float32; CODES: e4m3 codes
// go out.  kAhead: every vector is requested with the row, before the first
// reduction, so that one memory latency covers them all; otherwise each is
// requested where it is used, which takes 38 registers less and lets a CU hold
// more rows.
template <int P, bool F32, bool CODES, bool kAhead>
__global__ __launch_bounds__(kMaxThreads) void block_norm_kernel(NormArgs a, double rk) {
    __shared__ double red[2][kMaxWaves];
    const int m = blockIdx.x;
    const int t = threadIdx.x, T = blockDim.x, nwaves = T >> 6;
    const int pieces = a.K / 8;
    const int64_t cond = m / a.rows_per_cond;

    int kk[P];  // first value of each piece (lanes past the row: the row's first piece, left out below)
    bool on[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        on[j] = t + T * j < pieces;
        kk[j] = on[j] ? 8 * (t + T * j) : 0;
    }

    uint4 xr[P];
    float4 rr[P][2];
    Vectors<P> w;
    auto load4 = [](const float* p, int k, float4 (&o)[2]) {
        o[0] = *reinterpret_cast<const float4*>(p + k);
        o[1] = *reinterpret_cast<const float4*>(p + k + 4);
    };
    auto load8 = [](const uint16_t* p, int k) { return *reinterpret_cast<const uint4*>(p + k); };
    if (a.x) {
#pragma unroll
        for (int j = 0; j < P; ++j) xr[j] = load8(a.x + int64_t(m) * a.ldx, kk[j]);
    }
#pragma unroll
    for (int j = 0; j < P; ++j) {
        if constexpr (F32) {
            load4(static_cast<const float*>(a.r_in) + int64_t(m) * a.ld_rin, kk[j], rr[j]);
        } else {
            const uint4 u = load8(static_cast<const uint16_t*>(a.r_in) + int64_t(m) * a.ld_rin, kk[j]);
            rr[j][0] = *reinterpret_cast<const float4*>(&u);  // (bits; unpacked below)
        }
    }
    auto load_post = [&](int j) { load4(a.post_gamma, kk[j], w.post[j]); };
    auto load_gate = [&](int j) { w.gate[j] = load8(a.gate + cond * a.ld_gate, kk[j]); };
    auto load_pre = [&](int j) { load4(a.pre_gamma, kk[j], w.pre[j]); };
    auto load_scale = [&](int j) { w.scale[j] = load8(a.mod_scale + cond * a.ld_mod, kk[j]); };
    auto load_shift = [&](int j) { w.shift[j] = load8(a.mod_shift + cond * a.ld_mod, kk[j]); };
    if constexpr (kAhead) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            if (a.post_gamma) load_post(j);
            if (a.gate) load_gate(j);
            if (a.pre_gamma) load_pre(j);
            if (a.mod_scale) load_scale(j);
            if (a.mod_shift) load_shift(j);
        }
    }

    float r[P][8];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        if constexpr (F32) {
            unpack4(rr[j], r[j]);
        } else {
            unpack8(*reinterpret_cast<const uint4*>(&rr[j][0]), r[j]);
        }
    }

    if (a.x) {
        float rinv = 0.0f;
        if (a.post_gamma) {
            double ss = 0.0;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                float p[8];
                unpack8(xr[j], p);
                ss += on[j] ? lane_sumsq<8>(p) : 0.0;
            }
            rinv = inv_rms(block_sum(ss, nwaves, red[0]), a.K, rk, a.post_eps);
        }
#pragma unroll
        for (int j = 0; j < P; ++j) {
            float p[8], g[8];
            unpack8(xr[j], p);
            if (a.post_gamma) {
                if constexpr (!kAhead) load_post(j);
                unpack4(w.post[j], g);
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] = (p[i] * rinv) * g[i];
            }
            if (a.gate) {
                if constexpr (!kAhead) load_gate(j);
                unpack8(w.gate[j], g);
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] = p[i] * g[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) r[j][i] = r[j][i] + a.res_scale * p[i];
            if constexpr (F32) {
                if (on[j]) {
                    float* o = static_cast<float*>(a.r_out) + int64_t(m) * a.ld_rout + kk[j];
                    *reinterpret_cast<float4*>(o) = make_float4(r[j][0], r[j][1], r[j][2], r[j][3]);
                    *reinterpret_cast<float4*>(o + 4) = make_float4(r[j][4], r[j][5], r[j][6], r[j][7]);
                }
            } else {
                const uint4 u = pack8(r[j]);
                if (on[j]) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.r_out) + int64_t(m) * a.ld_rout + kk[j]) = u;
                unpack8(u, r[j]);  // the norm reads the stream as it is stored
            }
        }
    }

    if (!a.h && !CODES) return;
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < P; ++j) ss += on[j] ? lane_sumsq<8>(r[j]) : 0.0;
    const float rinv = inv_rms(block_sum(ss, nwaves, red[1]), a.K, rk, a.pre_eps);
#pragma unroll
    for (int j = 0; j < P; ++j) {
        float (&h)[8] = r[j];
        float g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = h[i] * rinv;
        if (a.pre_gamma) {
            if constexpr (!kAhead) load_pre(j);
            unpack4(w.pre[j], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = h[i] * g[i];
        }
        if (a.mod_scale) {
            if constexpr (!kAhead) load_scale(j);
            unpack8(w.scale[j], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = h[i] * (1.0f + g[i]);
        }
        if (a.mod_shift) {
            if constexpr (!kAhead) load_shift(j);
            unpack8(w.shift[j], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = h[i] + g[i];
        }
        if (a.h && on[j]) *reinterpret_cast<uint4*>(a.h + int64_t(m) * a.ld_h + kk[j]) = pack8(h);
        if constexpr (CODES) {
            // (K is a multiple of 128: the 16 lanes of a group are all on or all off)
            const float s = fp8_scale(max16_nonneg(lane_absmax<8>(h)));
            const uint2 q = fp8_codes8(h, s);
            if (on[j]) {
                *reinterpret_cast<uint2*>(a.codes + int64_t(m) * a.K + kk[j]) = q;
                if ((t & 15) == 0) a.act_scale[int64_t(kk[j] / 128) * fp8_scale_ld(a.M) + m] = s;
            }
        }
    }
}

// Rows that are at most one per CU request their vectors ahead (one row of 2048,
// gated and modulated: 3.04 us against 3.49, graph-replayed); more rows do not
// (1024 x 3584 to codes: 9.4 us against 10.1).
constexpr int kAheadRows = 256;

template <int P, bool F32>
hipError_t launch_p(const NormArgs& a, int T, hipStream_t st) {
    constexpr bool kMayAhead = P <= 2;  // (wider rows have no registers for it)
    const double rk = 1.0 / double(a.K);
    if (kMayAhead && a.M <= kAheadRows) {
        if (a.codes)
            hipLaunchKernelGGL((block_norm_kernel<P, F32, true, kMayAhead>), dim3(a.M), dim3(T), 0, st, a, rk);
        else
            hipLaunchKernelGGL((block_norm_kernel<P, F32, false, kMayAhead>), dim3(a.M), dim3(T), 0, st, a, rk);
    } else {
        if (a.codes)
            hipLaunchKernelGGL((block_norm_kernel<P, F32, true, false>), dim3(a.M), dim3(T), 0, st, a, rk);
        else
            hipLaunchKernelGGL((block_norm_kernel<P, F32, false, false>), dim3(a.M), dim3(T), 0, st, a, rk);
    }
    return hipGetLastError();
}

template <bool F32>
hipError_t launch_f(const NormArgs& a, hipStream_t st) {
    const int T = block_norm_threads(a.K, a.M, F32);
    if (T > kMaxThreads) return hipErrorInvalidValue;
    switch (block_norm_pieces(a.K, a.M, F32)) {
        case 1: return launch_p<1, F32>(a, T, st);
        case 2: return launch_p<2, F32>(a, T, st);
        case 4: return launch_p<4, F32>(a, T, st);
        default: return launch_p<8, F32>(a, T, st);
    }
}

// Codes of bf16 rows as they are (the prologue of a site without a norm).  The
// groups of 128 values are independent, so a row spreads over as many workgroups
// as it fills, a piece of 8 values per lane: bound by the bytes (4096 x 8192 20.4
// us, 4.9 TB/s; 23 x 16384 2.2 us, where one workgroup per row took 3.7).
constexpr int kQuantThreads = 256;
constexpr uint32_t kQuantGrid = 1u << 23;  // blocks along x (their threads below 2^32); further ones along y
__global__ __launch_bounds__(kQuantThreads) void quant_rows_kernel(NormArgs a, uint32_t per_row) {
    const uint32_t b = blockIdx.y * kQuantGrid + blockIdx.x, m = b / per_row;
    const int k = 8 * int((b - m * per_row) * kQuantThreads + threadIdx.x);
    // (K is a multiple of 128: a group's 16 lanes go on together)
    if (m >= uint32_t(a.M) || k >= a.K) return;
    float h[8];
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.r_in) + int64_t(m) * a.ld_rin + k), h);
    const float s = fp8_scale(max16_nonneg(lane_absmax<8>(h)));
    *reinterpret_cast<uint2*>(a.codes + int64_t(m) * a.K + k) = fp8_codes8(h, s);
    if ((threadIdx.x & 15) == 0) a.act_scale[int64_t(k / 128) * fp8_scale_ld(a.M) + m] = s;
}

hipError_t launch_quant_rows(const NormArgs& a, hipStream_t st) {
    const uint32_t per_row = (a.K / 8 + kQuantThreads - 1) / kQuantThreads, blocks = uint32_t(a.M) * per_row;
    const dim3 grid(blocks < kQuantGrid ? blocks : kQuantGrid, (blocks + kQuantGrid - 1) / kQuantGrid);
    hipLaunchKernelGGL(quant_rows_kernel, grid, dim3(kQuantThreads), 0, st, a, per_row);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, hipStream_t stream) {
    if (!a.pre_norm) return launch_quant_rows(a, stream);
    return a.stream_f32 ? launch_f<true>(a, stream) : launch_f<false>(a, stream);
}

}  // namespace fq
