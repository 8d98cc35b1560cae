// FP8 sites for decode-sized M (at most 32 tokens): a weight-streaming GEMV.
//
// Bound by reading the weight codes once.  A workgroup owns one group of 16
// weight rows; its waves split K in units of 128 (one scale group): per unit a
// lane loads 2 x 16 bytes of weight codes and of each token tile's codes, one
// v_mfma_f32_16x16x128_f8f6f4 multiplies 16 rows by 16 tokens, and the product
// is added to the float32 sums times sa * sw.  The waves' partial tiles meet
// in LDS; one wave per token tile runs the epilogue.
#include <hip/hip_runtime.h>

#include "fq_device.h"
#include "fq_fp8_tile.h"
#include "fq_internal.h"

namespace fq {
namespace {

constexpr int kWaves = 8;

__device__ __forceinline__ v8i join(uint4 a, uint4 b) {
    return v8i{int(a.x), int(a.y), int(a.z), int(a.w), int(b.x), int(b.y), int(b.z), int(b.w)};
}

// MT token tiles of 16, C units loaded before any is used
template <int MT, int C>
__global__ __launch_bounds__(64 * kWaves) void fp8_gemv_kernel(Fp8Args g, int per) {
    __shared__ v4f red[kWaves][MT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int nu = g.K / 128;
    const int u_begin = wave * per;
    const int u_end = u_begin + per < nu ? u_begin + per : nu;
    const int lda = fp8_scale_ld(g.M);

    int row = n0 + (lane & 15);
    row = row < g.N ? row : g.N - 1;  // rows past N load a valid row; their outputs are not stored
    const uint8_t* const wp = g.w + int64_t(row) * g.K + 16 * q;
    const float* const swp = g.wscale + int64_t(n0 / 128) * nu;
    const uint8_t* ap[MT];
    int tok[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        tok[t] = 16 * t + (lane & 15);
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
    if (wave >= MT) return;
    v4f sum[1][1] = {{red[0][wave][lane]}};
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum[0][0] += red[w][wave][lane];
    const int mm[1] = {16 * wave + (lane & 15)};
    const int nn[1] = {n0 + 4 * q};
    fp8_store_tiles<1, 1>(sum, mm, nn, g);
}

}  // namespace

hipError_t launch_fp8_gemv(const Fp8Args& g, hipStream_t stream) {
    if (g.M > kGemvMaxM) return hipErrorInvalidValue;
    const int nu = g.K / 128;
    const int per = (nu + kWaves - 1) / kWaves;
    const dim3 grid((g.N + 15) / 16), block(64 * kWaves);
    if (g.M <= 16)
        hipLaunchKernelGGL((fp8_gemv_kernel<1, 4>), grid, block, 0, stream, g, per);
    else
        hipLaunchKernelGGL((fp8_gemv_kernel<2, 4>), grid, block, 0, stream, g, per);
    return hipGetLastError();
}

}  // namespace fq
