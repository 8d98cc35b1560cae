// Norms before and after a block, with the gate, the residual scale and the
// stream update between them, in one pass over the rows (gfx950, wave64); the
// same kernel is the FP8 sites' prologue (no block output, codes out).
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
// are read once, r' and h written once.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "fq_device.h"
#include "fq_fp8.h"
#include "fq_internal.h"
#include "fq_token.h"

namespace fq {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxWaves = kMaxThreads / 64;

// Sum over the workgroup; every thread gets the same value.  `red` is used by
// one call only (no barrier separates two uses).
__device__ __forceinline__ double block_sum(double v, int nwaves, double* red) {
    v = wave_sum(v);
    if (nwaves > 1) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0;
        for (int w = 0; w < nwaves; ++w) v += red[w];
    }
    return v;
}

// 1 / sqrt(mean + eps) from a row's float64 sum of squares.  ss / K correctly
// rounded without a divide: Markstein's correction of ss * RN(1/K), rk.
__device__ __forceinline__ float inv_rms(double ss, int K, double rk, float eps) {
    const double q0 = ss * rk;
    const float ms = float(__builtin_fma(__builtin_fma(-q0, double(K), ss), rk, q0));
    return 1.0f / sqrtf(ms + eps);
}

__device__ __forceinline__ void load_gain(const float* __restrict__ g, int k, float (&o)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(g + k), b = *reinterpret_cast<const float4*>(g + k + 4);
    o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w;
    o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

// P pieces of 8 values per lane; F32: the stream is float32; CODES: e4m3 codes go out.
template <int P, bool F32, bool CODES>
__global__ __launch_bounds__(kMaxThreads) void block_norm_kernel(NormArgs a, double rk) {
    __shared__ double red[2][kMaxWaves];
    const int m = blockIdx.x;
    const int t = threadIdx.x, T = blockDim.x, nwaves = T >> 6;
    const int pieces = a.K / 8;
    const int64_t cond = m / a.rows_per_cond;

    float r[P][8];
    bool on[P];
#pragma unroll
    for (int j = 0; j < P; ++j) on[j] = t + T * j < pieces;

    // the stream
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int k = 8 * (t + T * j);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[j][i] = 0.0f;
        if (on[j]) {
            if constexpr (F32)
                load_gain(static_cast<const float*>(a.r_in) + int64_t(m) * a.ld_rin, k, r[j]);
            else
                unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.r_in) + int64_t(m) * a.ld_rin + k),
                        r[j]);
        }
    }

    if (a.x) {
        float p[P][8];
#pragma unroll
        for (int j = 0; j < P; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[j][i] = 0.0f;
            if (on[j]) unpack8(*reinterpret_cast<const uint4*>(a.x + int64_t(m) * a.ldx + 8 * (t + T * j)), p[j]);
        }
        if (a.post_gamma) {
            double ss = 0.0;
#pragma unroll
            for (int j = 0; j < P; ++j) ss += lane_sumsq<8>(p[j]);
            const float rinv = inv_rms(block_sum(ss, nwaves, red[0]), a.K, rk, a.post_eps);
#pragma unroll
            for (int j = 0; j < P; ++j)
                if (on[j]) {
                    float g[8];
                    load_gain(a.post_gamma, 8 * (t + T * j), g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[j][i] = (p[j][i] * rinv) * g[i];
                }
        }
        if (a.gate) {
#pragma unroll
            for (int j = 0; j < P; ++j)
                if (on[j]) {
                    float g[8];
                    unpack8(*reinterpret_cast<const uint4*>(a.gate + cond * a.ld_gate + 8 * (t + T * j)), g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[j][i] = p[j][i] * g[i];
                }
        }
#pragma unroll
        for (int j = 0; j < P; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[j][i] = r[j][i] + a.res_scale * p[j][i];
            const int k = 8 * (t + T * j);
            if constexpr (F32) {
                if (on[j] && a.r_out) {
                    float* o = static_cast<float*>(a.r_out) + int64_t(m) * a.ld_rout + k;
                    *reinterpret_cast<float4*>(o) = make_float4(r[j][0], r[j][1], r[j][2], r[j][3]);
                    *reinterpret_cast<float4*>(o + 4) = make_float4(r[j][4], r[j][5], r[j][6], r[j][7]);
                }
            } else {
                const uint4 w = pack8(r[j]);
                if (on[j] && a.r_out)
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.r_out) + int64_t(m) * a.ld_rout + k) = w;
                unpack8(w, r[j]);  // the norm reads the stream as it is stored
            }
        }
    }

    if (!a.h && !CODES) return;
    if (a.pre_norm) {
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < P; ++j) ss += lane_sumsq<8>(r[j]);
        const float rinv = inv_rms(block_sum(ss, nwaves, red[1]), a.K, rk, a.pre_eps);
#pragma unroll
        for (int j = 0; j < P; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[j][i] = r[j][i] * rinv;
            if (on[j] && a.pre_gamma) {
                float g[8];
                load_gain(a.pre_gamma, 8 * (t + T * j), g);
#pragma unroll
                for (int i = 0; i < 8; ++i) r[j][i] = r[j][i] * g[i];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int k = 8 * (t + T * j);
        if (on[j] && a.mod_scale) {
            float s[8];
            unpack8(*reinterpret_cast<const uint4*>(a.mod_scale + cond * a.ld_mod + k), s);
#pragma unroll
            for (int i = 0; i < 8; ++i) r[j][i] = r[j][i] * (1.0f + s[i]);
        }
        if (on[j] && a.mod_shift) {
            float s[8];
            unpack8(*reinterpret_cast<const uint4*>(a.mod_shift + cond * a.ld_mod + k), s);
#pragma unroll
            for (int i = 0; i < 8; ++i) r[j][i] = r[j][i] + s[i];
        }
        if (on[j] && a.h) *reinterpret_cast<uint4*>(a.h + int64_t(m) * a.ld_h + k) = pack8(r[j]);
        if constexpr (CODES) {
            // (K is a multiple of 128: the 16 lanes of a group are all on or all off)
            const float s = fp8_scale(max16_nonneg(lane_absmax<8>(r[j])));
            const uint2 q = fp8_codes8(r[j], s);
            if (on[j]) {
                *reinterpret_cast<uint2*>(a.codes + int64_t(m) * a.K + k) = q;
                if ((t & 15) == 0) a.act_scale[int64_t(k / 128) * fp8_scale_ld(a.M) + m] = s;
            }
        }
    }
}

template <int P, bool F32>
hipError_t launch_p(const NormArgs& a, int T, hipStream_t st) {
    if (a.codes)
        hipLaunchKernelGGL((block_norm_kernel<P, F32, true>), dim3(a.M), dim3(T), 0, st, a, 1.0 / double(a.K));
    else
        hipLaunchKernelGGL((block_norm_kernel<P, F32, false>), dim3(a.M), dim3(T), 0, st, a, 1.0 / double(a.K));
    return hipGetLastError();
}

template <bool F32>
hipError_t launch_f(const NormArgs& a, hipStream_t st) {
    const int T = block_norm_threads(a.K);
    if (T > kMaxThreads) return hipErrorInvalidValue;
    switch (block_norm_pieces(a.K)) {
        case 1: return launch_p<1, F32>(a, T, st);
        case 2: return launch_p<2, F32>(a, T, st);
        case 4: return launch_p<4, F32>(a, T, st);
        default: return launch_p<8, F32>(a, T, st);
    }
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, hipStream_t stream) {
    return a.stream_f32 ? launch_f<true>(a, stream) : launch_f<false>(a, stream);
}

}  // namespace fq
