// FP8 sites for a few tokens in one launch (fq_fp8_linear): the prologue and the
// weight-streaming GEMV fused, so that the tokens' quantisation overlaps the
// weight stream instead of preceding it.
//
// (fq_fp8_gemm runs the same kernel from codes where K is long.)
//
// Every workgroup quantises the tokens itself, with the prologue's arithmetic in
// the prologue's order (pieces of 8 values, 64 consecutive ones of a token to a
// wave; fq_row_norm.h, fq_fp8.h: the same codes bit for bit), while its weight
// loads are in flight: the tokens' loads are issued first and the weights' right
// after them, all unconditional, so the wait for the tokens leaves the weights
// in flight.  The codes go to LDS; workgroup 0 also writes them and the scales
// to the caller's workspace.  S of the 8 waves share the K range of R groups of
// 16 weight rows, up to C units of 128 k of a wave being requested at once, and
// the partial tiles meet in LDS.
//
// Measured (us, this launch / the two; one token): K = 3584, N = 37888 with the
// norm 26.7 / 29.2, K = 3584, N = 4608 6.8 / 9.6, K = 8192, N = 14336 27.1 / 28.2,
// without the norm 24.4 / 26.6; K = 16384, N = 2048 without 11.4 / 12.6.  One row
// group a workgroup instead of two: 27.7 at N = 37888, 6.5 against 6.2 at N =
// 6144; below one group for each CU the other way round (K = 896, N = 1024: 3.8
// against 5.3).
#include <hip/hip_runtime.h>

#include "fq_device.h"
#include "fq_fp8.h"
#include "fq_fp8_tile.h"
#include "fq_internal.h"
#include "fq_row_norm.h"

namespace fq {
namespace {

constexpr int kWaves = 8;
constexpr int kSpan = kWaves * 64 * 8;  // values in one piece of every lane

// Waves of 64 pieces that hold one token.
__host__ __device__ inline int token_waves(int K) { return (K + 511) / 512; }

// What the tokens come as: rows to quantise, rows to normalise and quantise, codes.
constexpr int kRows = 0, kNorm = 1, kCodes = 2;

// S waves share the K range of each of the 8 / S sets of R row groups; MT tiles
// of 16 tokens; P pieces per lane: piece j of wave w is wave v = 8 j + w of all
// tokens' waves, token v / token_waves(K); C units requested at once.
template <int SRC, int MT, int S, int R, int P, int C>
__global__ __launch_bounds__(64 * kWaves) void fp8_decode_kernel(NormArgs p, Fp8Args g, double rk) {
    constexpr bool NORM = SRC == kNorm;
    constexpr int G = kWaves / S;
    __shared__ double red_d[kWaves * (NORM ? P : 1)];
    __shared__ __attribute__((aligned(16))) uint8_t codes[kSpan * P];
    __shared__ float scales[kSpan * P / 128];
    __shared__ v4f red[kWaves][R][MT][64];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), ks = wave % S;
    const int K = g.K, nu = K / 128, per = (nu + S - 1) / S, tw = token_waves(K);
    const int u_begin = ks * per, u_end = u_begin + per < nu ? u_begin + per : nu;
    // a token's 16-byte chunk c of unit u; chunks of neighbouring tokens in other banks
    auto slot = [&](int m, int u, int c) { return m * K + u * 128 + 16 * (c ^ ((m >> 1) & 7)); };

    // the tokens' loads first (pieces past them: a token's first, left out below) ...
    int tok[P], k[P];
    bool on[P];
    uint4 xr[P];
    float4 gr[NORM ? P : 1][2];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int v = kWaves * j + wave;
        tok[j] = v / tw;
        k[j] = 8 * ((v - tok[j] * tw) * 64 + lane);
        on[j] = tok[j] < g.M && k[j] < K;
        if (!on[j]) k[j] = 0;
        if (tok[j] >= g.M) tok[j] = 0;
        if constexpr (SRC == kCodes) {
            const uint2 c = *reinterpret_cast<const uint2*>(g.act + int64_t(tok[j]) * K + k[j]);
            const float s = g.act_scale[int64_t(k[j] / 128) * fp8_scale_ld(g.M) + tok[j]];
            xr[j] = make_uint4(c.x, c.y, __float_as_uint(s), 0);
        } else {
            xr[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.r_in) + tok[j] * p.ld_rin + k[j]);
        }
    }
    if constexpr (NORM) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            gr[j][0] = *reinterpret_cast<const float4*>(p.pre_gamma + k[j]);
            gr[j][1] = *reinterpret_cast<const float4*>(p.pre_gamma + k[j] + 4);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    // ... then this wave's first weight units
    const int n0 = (blockIdx.x * G + wave / S) * 16 * R;
    const uint8_t* wp[R];
    const float* swp[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        int row = n0 + 16 * r + (lane & 15);
        row = row < g.N ? row : g.N - 1;  // rows past N load a valid row; their outputs are not stored
        wp[r] = g.w + int64_t(row) * K + 16 * q;
        const int first = n0 + 16 * r < g.N ? n0 + 16 * r : g.N - 1;
        swp[r] = g.wscale + int64_t(first / 128) * nu;
    }
    uint4 w[R][C][2];
    float sw[R][C];
    auto request = [&](int u0) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int v = u0 + i < u_end ? u0 + i : u_end - 1;
                const int u = v > 0 ? v : 0;  // repeated units are loaded but not used (a wave may have none)
                w[r][i][0] = *reinterpret_cast<const uint4*>(wp[r] + u * 128);
                w[r][i][1] = *reinterpret_cast<const uint4*>(wp[r] + u * 128 + 64);
                sw[r][i] = swp[r][u];
            }
    };
    request(u_begin);
    __builtin_amdgcn_sched_barrier(0);

    if constexpr (NORM) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            float x[8];
            unpack8(xr[j], x);
            const double v = wave_sum(on[j] ? lane_sumsq<8>(x) : 0.0);
            if (lane == 0) red_d[wave + kWaves * j] = v;
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < P; ++j) {
        if constexpr (SRC == kCodes) {
            if (on[j]) {
                const int u = k[j] / 128;
                *reinterpret_cast<uint2*>(codes + slot(tok[j], u, (k[j] / 16) & 7) + (k[j] & 8)) = make_uint2(xr[j].x, xr[j].y);
                if ((lane & 15) == 0) scales[u * g.M + tok[j]] = __uint_as_float(xr[j].z);
            }
            continue;
        }
        float h[8];
        unpack8(xr[j], h);
        if constexpr (NORM) {
            double ss = 0.0;
            if (g.M == 1) {  // (waves past the token hold 0; the reads go out at once)
#pragma unroll
                for (int i = 0; i < kWaves * P; ++i) ss += red_d[i];
            } else {
                for (int i = 0; i < tw; ++i) ss += red_d[tok[j] * tw + i];
            }
            const float rinv = inv_rms(ss, K, rk, p.pre_eps);
            float gv[8];
            unpack4(gr[j], gv);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = h[i] * rinv * gv[i];
        }
        const float s = fp8_scale(max16_nonneg(lane_absmax<8>(h)));
        const uint2 c = fp8_codes8(h, s);
        if (on[j]) {
            const int u = k[j] / 128;
            *reinterpret_cast<uint2*>(codes + slot(tok[j], u, (k[j] / 16) & 7) + (k[j] & 8)) = c;
            if ((lane & 15) == 0) scales[u * g.M + tok[j]] = s;
            if (blockIdx.x == 0) {
                *reinterpret_cast<uint2*>(p.codes + int64_t(tok[j]) * K + k[j]) = c;
                if ((lane & 15) == 0) p.act_scale[int64_t(u) * fp8_scale_ld(g.M) + tok[j]] = s;
            }
        }
    }
    __syncthreads();

    // the products (columns past M: the last token again, not stored)
    int col[MT];
    v4f acc[R][MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        col[t] = 16 * t + (lane & 15) < g.M ? 16 * t + (lane & 15) : g.M - 1;
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    for (int u0 = u_begin; u0 < u_end; u0 += C) {
        if (u0 > u_begin) request(u0);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int u = u0 + i;
            if (u >= u_end) break;  // wave-uniform
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const v8i a = join(*reinterpret_cast<const uint4*>(codes + slot(col[t], u, q)),
                                   *reinterpret_cast<const uint4*>(codes + slot(col[t], u, 4 + q)));
                const float sa = scales[u * g.M + col[t]];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const v4f d = mfma_e4m3(join(w[r][i][0], w[r][i][1]), a, v4f{0.f, 0.f, 0.f, 0.f});
                    const float ps = sa * sw[r][i];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[r][t][e] = __builtin_fmaf(d[e], ps, acc[r][t][e]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t) red[wave][r][t][lane] = acc[r][t];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if (ks != (r * MT + t) % S) continue;
            v4f sum[1][1] = {{red[wave - ks][r][t][lane]}};
#pragma unroll
            for (int i = 1; i < S; ++i) sum[0][0] += red[wave - ks + i][r][t][lane];
            const int mm[1] = {16 * t + (lane & 15)}, nn[1] = {n0 + 16 * r + 4 * q};
            fp8_store_tiles<1, 1>(sum, mm, nn, g);
        }
}

template <int SRC, int MT, int S, int R, int P, int C>
hipError_t launch(const NormArgs& p, const Fp8Args& g, hipStream_t st) {
    constexpr int rows = 16 * R * (kWaves / S);
    hipLaunchKernelGGL((fp8_decode_kernel<SRC, MT, S, R, P, C>), dim3((g.N + rows - 1) / rows), dim3(64 * kWaves), 0,
                       st, p, g, 1.0 / double(g.K));
    return hipGetLastError();
}

// K beyond four units a wave: three units at a time where that requests fewer past
// a wave's share, as in the GEMV (fq_fp8_gemv.hip).
template <int SRC, int P>
hipError_t launch_long(const NormArgs& p, const Fp8Args& g, hipStream_t st) {
    const int per = (g.K / 128 + kWaves - 1) / kWaves;
    return (per + 2) / 3 * 3 < (per + 3) / 4 * 4 ? launch<SRC, 1, 8, 1, P, 3>(p, g, st)
                                                 : launch<SRC, 1, 8, 1, P, 4>(p, g, st);
}

// One row group a workgroup where there is at most one for each CU, else two; S
// as in the GEMV.
template <int SRC, int MT, int P>
hipError_t launch_p(const NormArgs& p, const Fp8Args& g, const DeviceInfo& dev, hipStream_t st) {
    const int nu = g.K / 128, groups = (g.N + 15) / 16, per = (nu + kWaves - 1) / kWaves;
    if constexpr (P > 1 && MT == 1)  // (one piece per lane, or more than 16 tokens: short K)
        if (per > 4) return launch_long<SRC, P>(p, g, st);
    if constexpr (P > 4) return hipErrorInvalidValue;  // (one token of more than 16384 values)
    if constexpr (MT == 1 && P <= 4) {
        if (groups > dev.cus && nu > 16) return launch<SRC, MT, 8, 2, P, 4>(p, g, st);
        if (groups > dev.cus && nu > 8) return launch<SRC, MT, 4, 2, P, 4>(p, g, st);
    }
    if constexpr (P <= 4) {
        if (groups > dev.cus) return launch<SRC, MT, 2, 2, P, 4>(p, g, st);
        return launch<SRC, MT, 8, 1, P, 4>(p, g, st);
    }
}

template <int SRC>
hipError_t launch_n(const NormArgs& p, const Fp8Args& g, const DeviceInfo& dev, hipStream_t st) {
    const int waves = g.M * token_waves(g.K);
    if (waves <= 8) return launch_p<SRC, 1, 1>(p, g, dev, st);
    if (waves <= 16) return launch_p<SRC, 1, 2>(p, g, dev, st);
    if constexpr (SRC == kRows) {
        if (waves <= 32) return g.M > 16 ? launch_p<SRC, 2, 4>(p, g, dev, st) : launch_p<SRC, 1, 4>(p, g, dev, st);
        return launch_p<SRC, 1, 8>(p, g, dev, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace

// By the pieces that every workgroup quantises, and one token always.  Measured
// (us, this launch / the two): with the norm and two pieces per lane 2 x 3584 x
// 37888 29.0 / 29.4, 4 x 2048 x 8192 8.1 / 8.5, 16 x 256 x 512 4.9 / 5.0; with four
// 4 x 3584 x 37888 48.6 / 30.7, 16 x 896 x 1024 7.0 / 6.4, 2 x 8192 x 8192 17.7 /
// 18.8.  Without it and four 4 x 3584 x 37888 28.7 / 29.9, 16 x 896 x 1024 4.9 / 5.9.  (With the norm beyond 8192
// values the order of the prologue's sum is another.)
bool fp8_decode_takes(const NormArgs& p, const Fp8Args& g) {
    if (g.M > kGemvMaxM || hooks().fp8_tile.load(std::memory_order_relaxed) >= 0) return false;
    const int waves = g.M * token_waves(g.K);
    return waves <= (p.pre_norm ? 16 : g.M > 1 ? 32 : 64);
}

hipError_t launch_fp8_decode(const NormArgs& p, const Fp8Args& g, const DeviceInfo& dev, hipStream_t stream) {
    if (!fp8_decode_takes(p, g)) return hipErrorInvalidValue;
    return p.pre_norm ? launch_n<kNorm>(p, g, dev, stream) : launch_n<kRows>(p, g, dev, stream);
}

// From codes the LDS copy is worth its barrier where K is long: one token K = 5120,
// N = 5120 8.4 us against 9.4 with the codes read from L2, K = 18944, N = 3584 15.4
// against 17.7, two tokens 5120 x 5120 8.8 against 9.7; K = 2048, N = 8192 6.5 against
// 5.2.
bool fp8_decode_codes_takes(const Fp8Args& g) {
    if (g.K <= kSpan || g.M > 16 || hooks().fp8_tile.load(std::memory_order_relaxed) >= 0) return false;
    return g.M * token_waves(g.K) <= (g.M > 1 ? 32 : 64);
}

hipError_t launch_fp8_decode_codes(const Fp8Args& g, hipStream_t stream) {
    if (!fp8_decode_codes_takes(g)) return hipErrorInvalidValue;
    const int waves = g.M * token_waves(g.K);
    const NormArgs none{};
    if (waves <= 16) return launch_long<kCodes, 2>(none, g, stream);
    return waves <= 32 ? launch_long<kCodes, 4>(none, g, stream) : launch_long<kCodes, 8>(none, g, stream);
}

}  // namespace fq
