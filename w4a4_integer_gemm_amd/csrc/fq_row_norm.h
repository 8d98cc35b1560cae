// The sums and the normalisation of a row held by one workgroup (gfx950,
// wave64): shared by the kernels whose codes have to agree bit for bit.
#pragma once

#include <hip/hip_runtime.h>

#include "fq_token.h"

namespace fq {

// Sum over the workgroup (of at most 16 waves) in the order of its waves; every
// thread gets the same value.  `red` has 16 entries and is used by one call only
// (no barrier separates two uses).  Up to 4 or 8 waves the entries past the last
// hold 0 and all reads go out at once (one row of 2048 with both norms 3.06 us,
// 3.26 with a read after the other; rows of 16 waves took 0.1 us longer that way).
template <int N>
__device__ __forceinline__ double sum_entries(const double* red) {
    double v = red[0];
#pragma unroll
    for (int w = 1; w < N; ++w) v += red[w];
    return v;
}
__device__ __forceinline__ double block_sum(double v, int nwaves, double* red) {
    v = wave_sum(v);
    if (nwaves == 1) return v;
    const int t = threadIdx.x;
    if ((t & 63) == 0) red[t >> 6] = v;
    if (t >= nwaves && t < 8) red[t] = 0.0;
    __syncthreads();
    if (nwaves <= 4) return sum_entries<4>(red);
    if (nwaves <= 8) return sum_entries<8>(red);
    v = 0.0;
    for (int w = 0; w < nwaves; ++w) v += red[w];
    return v;
}

// 1 / sqrt(mean + eps) from a row's float64 sum of squares.  ss / K correctly
// rounded without a divide: Markstein's correction of ss * RN(1/K), rk.
__device__ __forceinline__ float inv_rms(double ss, int K, double rk, float eps) {
    const double q0 = ss * rk;
    const float ms = float(__builtin_fma(__builtin_fma(-q0, double(K), ss), rk, q0));
    return 1.0f / sqrtf(ms + eps);
}

__device__ __forceinline__ void unpack4(const float4 (&v)[2], float (&o)[8]) {
    o[0] = v[0].x, o[1] = v[0].y, o[2] = v[0].z, o[3] = v[0].w;
    o[4] = v[1].x, o[5] = v[1].y, o[6] = v[1].z, o[7] = v[1].w;
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

}  // namespace fq
