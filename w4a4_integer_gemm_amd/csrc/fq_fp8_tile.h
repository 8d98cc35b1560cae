// Pieces shared by the FP8 GEMM and GEMV (gfx950, wave64): the matrix
// instruction, the LDS layout of an operand stage and the epilogue.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fq_device.h"
#include "fq_internal.h"

namespace fq {

// D[16 rows][16 tokens] = sum over 128 k.  Lane l gives row (token) l % 16 of
// each operand and 32 of its codes; the instruction sums over k in any order,
// so the operands only have to present the same k in the same register bytes.
// Lane l holds D[4 (l / 16) + i][l % 16] in register i.  (Zero scale operands
// select the form without block scales.)
//
// Precision, measured with powers of two on this chip: the products of 8
// consecutive codes of a lane are aligned to the largest exponent sum E among
// them and what lies below 2^(E - 13) is dropped; the sums of 8 are added in
// float32.  Two e4m3 codes multiply to a last bit of 2^(e - 6), so only a
// product 2^8 times smaller than its largest neighbour loses bits: a choice of
// the instruction, far below the codes' own rounding (2^-4).
__device__ __forceinline__ v4f mfma_e4m3(const v8i& w, const v8i& a, const v4f& c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 0, 0, 0, 0, 0, 0);
}

// LDS layout of a 128-byte row rho: chunk c of 16 bytes at slot 8 rho + (c ^ swizzle).
__device__ __forceinline__ int fp8_swizzle(int rho) { return (rho >> 1) & 7; }
// Byte offset of chunk q (0 .. 3) of a row; chunk q + 4 is at this offset ^ 64
// (the swizzle flips bits of the chunk number).
__device__ __forceinline__ uint32_t fp8_slot(int rho, int q) {
    return uint32_t(128 * rho + 16 * (q ^ fp8_swizzle(rho)));
}
typedef __attribute__((address_space(3))) const v4i lds_cv4i;
// A lane's 32 codes of a fragment: chunks q and q + 4 of its row.
__device__ __forceinline__ v8i fp8_read_frag(uint32_t addr) {
    const v4i a = *reinterpret_cast<lds_cv4i*>(uintptr_t(addr));
    const v4i b = *reinterpret_cast<lds_cv4i*>(uintptr_t(addr ^ 64u));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ uint16_t* fp8_out_ptr(const Fp8Args& g, int m, int n) {
    if (g.head_dim > 0) {
        const int h = n / g.head_dim;
        return g.y + (int64_t(h) * g.M + m) * g.head_dim + (n - h * g.head_dim);
    }
    return g.y + int64_t(m) * g.ldy + n;
}

// Epilogue of a wave's tiles: tile (i, j) holds features n[i] .. n[i] + 3 (a
// multiple of 4 inside one head) of token m[j].  Every operand is loaded
// before the first store (stores count in the loads' memory counter).
template <int TN, int TM>
__device__ __forceinline__ void fp8_store_tiles(const v4f (&acc)[TN][TM], const int (&m)[TM], const int (&n)[TN],
                                                const Fp8Args& g) {
    float4 bs[TN];
#pragma unroll
    for (int i = 0; i < TN; ++i)
        bs[i] = (g.bias && n[i] < g.N) ? *reinterpret_cast<const float4*>(g.bias + n[i])
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
    uint2 rs[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
            rs[i][j] = (g.residual && n[i] < g.N && m[j] < g.M)
                           ? *reinterpret_cast<const uint2*>(g.residual + int64_t(m[j]) * g.ldr + n[i])
                           : make_uint2(0, 0);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            if (m[j] >= g.M || n[i] >= g.N) continue;
            v4f t = acc[i][j];
            if (g.bias) {
                t[0] = t[0] + bs[i].x;
                t[1] = t[1] + bs[i].y;
                t[2] = t[2] + bs[i].z;
                t[3] = t[3] + bs[i].w;
            }
            if (g.residual) {
                t[0] = t[0] + bf16_lo(rs[i][j].x);
                t[1] = t[1] + bf16_hi(rs[i][j].x);
                t[2] = t[2] + bf16_lo(rs[i][j].y);
                t[3] = t[3] + bf16_hi(rs[i][j].y);
            }
            *reinterpret_cast<uint2*>(fp8_out_ptr(g, m[j], n[i])) =
                make_uint2(pack_bf16x2(t[0], t[1]), pack_bf16x2(t[2], t[3]));
        }
}

}  // namespace fq
