// FP8 sites for decode-sized M (at most 32 tokens, more for narrow layers): the
// weight-streaming GEMV that reads the tokens' codes from L2.
//
// Bound by reading the weight codes once.  S waves of a workgroup share the K
// range of a group of 16 weight rows, in units of 128 (one scale group): per
// unit a lane loads 2 x 16 bytes of weight codes and of each token tile's codes,
// one v_mfma_f32_16x16x128_f8f6f4 multiplies 16 rows by 16 tokens, and the product
// is added to the float32 sums times sa * sw.  A wave requests C units before it
// uses the first; the S partial tiles meet in LDS in a fixed order.
//
// What costs beside the weights is the codes, read again for every row group:
// K = 3584, N = 37888 (26.6 us at copy rate): 25.7 us with one token, 26.9 with
// 4, 30 with 8, beyond which the tiled GEMM takes over (fp8_gemv_takes).
// From codes narrow layers keep it up to 32 tokens: K = 16384, N = 2048 16.9 us with
// 16 tokens, 17.1 with 32 (the GEMM 35), bound by what a CU keeps in flight: 16 waves
// on a row group took the same time, and so did groups of 8 rows on twice the CUs.
// (fq_fp8_linear has a workspace and cuts K there: 14.3 and 14.7 with its prologue; one
// or two tokens of such K take the kernel of fq_fp8_decode.hip.)
#include <hip/hip_runtime.h>

#include "fq_device.h"
#include "fq_fp8_tile.h"
#include "fq_internal.h"

namespace fq {
namespace {

constexpr int kWaves = 8;

// MT token tiles of 16, C units loaded before any is used
template <int MT, int S, int C>
__global__ __launch_bounds__(64 * kWaves) void fp8_gemv_kernel(Fp8Args g, int per) {
    constexpr int G = kWaves / S;  // row groups of a workgroup
    __shared__ v4f red[kWaves][MT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, ks = wave % S;
    const int n0 = (blockIdx.x * G + wave / S) * 16, m0 = blockIdx.y * 16 * MT;
    const int nu = g.K / 128;
    const int u_begin = ks * per, u_end = u_begin + per < nu ? u_begin + per : nu;
    const int lda = fp8_scale_ld(g.M);

    int row = n0 + (lane & 15);
    row = row < g.N ? row : g.N - 1;  // rows past N load a valid row; their outputs are not stored
    const uint8_t* const wp = g.w + int64_t(row) * g.K + 16 * q;
    const float* const swp = g.wscale + int64_t((n0 < g.N ? n0 : g.N - 1) / 128) * nu;
    const uint8_t* ap[MT];
    int tok[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        tok[t] = m0 + 16 * t + (lane & 15);
        tok[t] = tok[t] < g.M ? tok[t] : g.M - 1;  // (columns past M are not stored)
        ap[t] = g.act + int64_t(tok[t]) * g.K + 16 * q;
    }
    v4f acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};

    for (int u0 = u_begin; u0 < u_end; u0 += C) {
        uint4 w[C][2], a[C][MT][2];
        float sa[C][MT], sw[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int u = u0 + c < u_end ? u0 + c : u_end - 1;  // repeated units are loaded but not used
            w[c][0] = *reinterpret_cast<const uint4*>(wp + int64_t(u) * 128);
            w[c][1] = *reinterpret_cast<const uint4*>(wp + int64_t(u) * 128 + 64);
            sw[c] = swp[u];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                a[c][t][0] = *reinterpret_cast<const uint4*>(ap[t] + int64_t(u) * 128);
                a[c][t][1] = *reinterpret_cast<const uint4*>(ap[t] + int64_t(u) * 128 + 64);
                sa[c][t] = g.act_scale[int64_t(u) * lda + tok[t]];
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (u0 + c < u_end) {  // wave-uniform
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const v4f d = mfma_e4m3(join(w[c][0], w[c][1]), join(a[c][t][0], a[c][t][1]),
                                            v4f{0.f, 0.f, 0.f, 0.f});
                    const float p = sa[c][t] * sw[c];
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(d[i], p, acc[t][i]);
                }
            }
    }

#pragma unroll
    for (int t = 0; t < MT; ++t) red[wave][t][lane] = acc[t];
    __syncthreads();
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        if (ks != t % S) continue;
        v4f sum[1][1] = {{red[wave - ks][t][lane]}};
#pragma unroll
        for (int i = 1; i < S; ++i) sum[0][0] += red[wave - ks + i][t][lane];
        const int mm[1] = {m0 + 16 * t + (lane & 15)}, nn[1] = {n0 + 4 * q};
        fp8_store_tiles<1, 1>(sum, mm, nn, g);
    }
}

// More than 16 tokens: two tiles of 16 in one workgroup share its weights; one tile
// each where that only fills idle CUs (K = 16384, N = 2048, 23 tokens: 16.7 us
// against 21.0; K = N = 4096: 9.1 against 7.4).
template <int S, int C>
hipError_t launch_c(const Fp8Args& g, const DeviceInfo& dev, int per, hipStream_t st) {
    constexpr int rows = 16 * (kWaves / S);
    const int blocks = (g.N + rows - 1) / rows;
    const dim3 block(64 * kWaves);
    if (fp8_gemv_tokens(g.M, g.N, dev.cus) == 16)
        hipLaunchKernelGGL((fp8_gemv_kernel<1, S, C>), dim3(blocks, (g.M + 15) / 16), block, 0, st, g, per);
    else
        hipLaunchKernelGGL((fp8_gemv_kernel<2, S, C>), dim3(blocks, (g.M + 31) / 32), block, 0, st, g, per);
    return hipGetLastError();
}

// Four units at a time, three where that requests fewer units past a wave's share.
template <int S>
hipError_t launch_s(const Fp8Args& g, const DeviceInfo& dev, hipStream_t st) {
    const int per = (g.K / 128 + S - 1) / S;
    return (per + 2) / 3 * 3 < (per + 3) / 4 * 4 ? launch_c<S, 3>(g, dev, per, st) : launch_c<S, 4>(g, dev, per, st);
}

}  // namespace

// Waves that share a row group: 8 where a wave then still has more than two
// units, or where there is at most one group for each CU; otherwise 4, 2 or 1, so
// that a wave's loads in flight are not cut short by its share (M = 1, K = 2048,
// N = 32768: 22.6 us with 8, 14.0 with 4, 15.5 with 2; K = 1024, N = 16384: 9.2, 7.2,
// 5.2; K = 3584, N = 37888: 26.0, 29.0, 33.9; K = 896, N = 1024: 3.5, 4.1, 4.3).
hipError_t launch_fp8_gemv(const Fp8Args& g, const DeviceInfo& dev, hipStream_t stream) {
    if (!fp8_gemv_tokens(g.M, g.N, dev.cus)) return hipErrorInvalidValue;
    const int nu = g.K / 128, groups = (g.N + 15) / 16;
    if (nu > 16 || groups <= dev.cus) return launch_s<8>(g, dev, stream);
    if (nu > 8) return launch_s<4>(g, dev, stream);
    if (nu > 4) return launch_s<2>(g, dev, stream);
    return launch_s<1>(g, dev, stream);
}

}  // namespace fq
