// One-token FP8 sites in one launch (fq_fp8_linear with M = 1): the prologue and
// the weight-streaming GEMV fused, so that the token's quantisation overlaps the
// weight stream instead of preceding it.
//
// Every workgroup quantises the token itself, with the prologue's arithmetic in
// the prologue's order (piece t of 8 values in lane t, fq_row_norm.h, fq_fp8.h:
// the same codes bit for bit), while its weight loads are in flight: the
// token's loads are issued first and the weights' right after them, all
// unconditional, so the wait for the token leaves the weights in flight.  The
// codes go to LDS; workgroup 0 also writes them and the scales to the caller's
// workspace.  S of the 8 waves share the K range of R groups of 16 weight rows, up
// to C units of 128 k of a wave being requested at once (all of them for K <=
// 4096), and the partial tiles meet in LDS.
//
// Measured (us, this launch / the two; one token): K = 3584, N = 37888 with the
// norm 26.4 / 29.4, K = 3584, N = 4608 6.2 / 9.6, K = 8192, N = 14336 26.7 / 28.9,
// without the norm 24.1 / 27.9; K = 16384, N = 2048 without 10.7 / 16.7.  One row
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
constexpr int kSpan = kWaves * 64 * 8;  // token values in a piece for every lane

// S waves share the K range of each of the 8 / S sets of R row groups; P token
// pieces per lane (with the norm at most two: the prologue holds a row of up to
// 8192 values at one piece per lane, and its sum of squares is taken here in its
// order, lanes of a wave first, then wave by wave); C units requested at once.
template <bool NORM, int S, int R, int P, int C>
__global__ __launch_bounds__(64 * kWaves) void fp8_decode1_kernel(NormArgs p, Fp8Args g, double rk) {
    static_assert(!NORM || P <= 2, "the order of the prologue's sums");
    constexpr int G = kWaves / S;
    __shared__ double red_d[kWaves * (NORM ? P : 1)];
    __shared__ __attribute__((aligned(16))) uint8_t codes[kSpan * P];
    __shared__ float scales[kSpan * P / 128];
    __shared__ v4f red[kWaves][R][64];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), ks = wave % S;
    const int K = g.K, nu = K / 128, per = (nu + S - 1) / S;
    const int u_begin = ks * per, u_end = u_begin + per < nu ? u_begin + per : nu;

    // the token's loads first (pieces past the token: its first, left out below) ...
    uint4 xr[P];
    float4 gr[NORM ? P : 1][2];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int k = 8 * (tid + 64 * kWaves * j);
        xr[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.r_in) + (k < K ? k : 0));
    }
    if constexpr (NORM) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int k = 8 * (tid + 64 * kWaves * j);
            const float* const gp = p.pre_gamma + (k < K ? k : 0);
            gr[j][0] = *reinterpret_cast<const float4*>(gp);
            gr[j][1] = *reinterpret_cast<const float4*>(gp + 4);
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

    float rinv = 1.0f;
    if constexpr (NORM) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            float x[8];
            unpack8(xr[j], x);
            const double v = wave_sum(8 * (tid + 64 * kWaves * j) < K ? lane_sumsq<8>(x) : 0.0);
            if (lane == 0) red_d[wave + kWaves * j] = v;
        }
        __syncthreads();
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < kWaves * P; ++i) ss += red_d[i];  // (waves past the token add 0)
        rinv = inv_rms(ss, K, rk, p.pre_eps);
    }
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int k = 8 * (tid + 64 * kWaves * j);
        const bool on = k < K;
        float h[8];
        unpack8(xr[j], h);
        if constexpr (NORM) {
            float gv[8];
            unpack4(gr[j], gv);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = h[i] * rinv * gv[i];
        }
        const float s = fp8_scale(max16_nonneg(lane_absmax<8>(h)));
        const uint2 c = fp8_codes8(h, s);
        if (on) {
            *reinterpret_cast<uint2*>(codes + k) = c;
            if ((tid & 15) == 0) scales[k / 128] = s;
            if (blockIdx.x == 0) {
                *reinterpret_cast<uint2*>(p.codes + k) = c;
                if ((tid & 15) == 0) p.act_scale[int64_t(k / 128) * fp8_scale_ld(1)] = s;
            }
        }
    }
    __syncthreads();

    // the products: all 16 columns are the token (one address for the 16 lanes of a
    // quarter); column 0 is stored
    v4f acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int u0 = u_begin; u0 < u_end; u0 += C) {
        if (u0 > u_begin) request(u0);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int u = u0 + i;
            if (u >= u_end) break;  // wave-uniform
            const v8i a = join(*reinterpret_cast<const uint4*>(codes + u * 128 + 16 * q),
                               *reinterpret_cast<const uint4*>(codes + u * 128 + 64 + 16 * q));
            const float sa = scales[u];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const v4f d = mfma_e4m3(join(w[r][i][0], w[r][i][1]), a, v4f{0.f, 0.f, 0.f, 0.f});
                const float ps = sa * sw[r][i];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[r][e] = __builtin_fmaf(d[e], ps, acc[r][e]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) red[wave][r][lane] = acc[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (ks != r % S) continue;
        v4f sum[1][1] = {{red[wave - ks][r][lane]}};
#pragma unroll
        for (int i = 1; i < S; ++i) sum[0][0] += red[wave - ks + i][r][lane];
        const int mm[1] = {lane & 15}, nn[1] = {n0 + 16 * r + 4 * q};
        fp8_store_tiles<1, 1>(sum, mm, nn, g);
    }
}

template <bool NORM, int S, int R, int P, int C>
hipError_t launch(const NormArgs& p, const Fp8Args& g, hipStream_t st) {
    constexpr int rows = 16 * R * (kWaves / S);
    hipLaunchKernelGGL((fp8_decode1_kernel<NORM, S, R, P, C>), dim3((g.N + rows - 1) / rows), dim3(64 * kWaves), 0, st, p,
                       g, 1.0 / double(p.K));
    return hipGetLastError();
}

template <bool NORM, int P>
hipError_t launch_long(const NormArgs& p, const Fp8Args& g, hipStream_t st) {  // (units per request as in the GEMV)
    const int per = (g.K / 128 + kWaves - 1) / kWaves;
    return (per + 2) / 3 * 3 < (per + 3) / 4 * 4 ? launch<NORM, 8, 1, P, 3>(p, g, st) : launch<NORM, 8, 1, P, 4>(p, g, st);
}

// One row group a workgroup where there is at most one for each CU, else two; S
// as in the GEMV (fq_fp8_gemv.hip), so that a wave has up to four units.
template <bool NORM>
hipError_t launch_short(const NormArgs& p, const Fp8Args& g, const DeviceInfo& dev, hipStream_t st) {
    const int nu = g.K / 128, groups = (g.N + 15) / 16;
    if (groups <= dev.cus) return launch<NORM, 8, 1, 1, 4>(p, g, st);
    if (nu > 16) return launch<NORM, 8, 2, 1, 4>(p, g, st);
    if (nu > 8) return launch<NORM, 4, 2, 1, 4>(p, g, st);
    return launch<NORM, 2, 2, 1, 4>(p, g, st);
}

}  // namespace

// (with the norm beyond 8192 values the order of the prologue's sum is another)
bool fp8_decode1_takes(const NormArgs& p, const Fp8Args& g) {
    return g.M == 1 && g.K <= (p.pre_norm ? 2 : 8) * kSpan && hooks().fp8_tile.load(std::memory_order_relaxed) < 0;
}

hipError_t launch_fp8_decode1(const NormArgs& p, const Fp8Args& g, const DeviceInfo& dev, hipStream_t stream) {
    if (!fp8_decode1_takes(p, g)) return hipErrorInvalidValue;
    if (g.K > 4 * kSpan) return launch_long<false, 8>(p, g, stream);
    if (g.K > kSpan) return p.pre_norm ? launch_long<true, 2>(p, g, stream) : launch_long<false, 4>(p, g, stream);
    return p.pre_norm ? launch_short<true>(p, g, dev, stream) : launch_short<false>(p, g, dev, stream);
}

}  // namespace fq
