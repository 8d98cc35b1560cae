// Pieces shared by the FP8 GEMM and GEMV (gfx950, wave64): the matrix
// instruction, the LDS layout of an operand stage and the epilogue.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fq_device.h"
#include "fq_fp8_copy.h"
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

// Byte offset of chunk q (0 .. 3) of a row; chunk q + 4 is at this offset ^ 64
// (the swizzle flips bits of the chunk number).
__device__ __forceinline__ uint32_t fp8_slot(int rho, int q) {
    return uint32_t(128 * rho + 16 * (q ^ fp8_swizzle(rho)));
}
typedef __attribute__((address_space(3))) const v4i lds_cv4i;
// A lane's 32 codes of a fragment: chunks q and q + 4 of its row.
__device__ __forceinline__ v8i fp8_read_frag(uint32_t lo, uint32_t hi) {
    const v4i a = *reinterpret_cast<lds_cv4i*>(uintptr_t(lo));
    const v4i b = *reinterpret_cast<lds_cv4i*>(uintptr_t(hi));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The 32 codes of a fragment from the two 16-byte pieces.
__device__ __forceinline__ v8i join(uint4 a, uint4 b) {
    return v8i{int(a.x), int(a.y), int(a.z), int(a.w), int(b.x), int(b.y), int(b.z), int(b.w)};
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

// Epilogue of a wave's TW x TF fragments (weight rows n0 .. n0 + 16 TW - 1,
// tokens m0 .. m0 + 16 TF - 1) from the registers.  A lane holds 4 consecutive
// features of each fragment; exchanging the odd 16-lane rows of fragment n with
// the even rows of fragment n + 1 leaves every lane 8 consecutive features of
// one of the two (fragment n + q % 2, features 8 (q / 2) .. + 7, q = lane / 16),
// so it stores 16 bytes and four lanes store 64 consecutive bytes of a row.
// The addresses of a fragment pair are the row's plus a constant; the options
// (bias, residual) are decided once, outside the loops.
template <bool EXTRAS, int TW, int TF>
__device__ __forceinline__ void fp8_store_pairs(const v4f (&acc)[TW][TF], int m0, int n0, int lane, const Fp8Args& g) {
    const int q = lane >> 4;
    const int c0 = n0 + 16 * (q & 1) + 8 * (q >> 1);  // column of pair 0
    // y of (m, c0 + 32 pair): rows ld apart; a pair's column offset is 32 pair,
    // or with heads that of its head
    const int64_t row_step = g.head_dim > 0 ? g.head_dim : g.ldy;
    uint16_t* yp[(TW + 1) / 2];
#pragma unroll
    for (int n = 0; n + 1 < TW; n += 2) {
        const int col = c0 + 16 * n;
        yp[n / 2] = fp8_out_ptr(g, m0 + (lane & 15), col);
    }
    float bs[EXTRAS ? (TW + 1) / 2 : 1][8];
    if constexpr (EXTRAS) {
#pragma unroll
        for (int n = 0; n + 1 < TW; n += 2) {
            const int col = c0 + 16 * n;
            const bool on = g.bias && col < g.N;
            const float4 a = on ? *reinterpret_cast<const float4*>(g.bias + col) : make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 b = on ? *reinterpret_cast<const float4*>(g.bias + col + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
            bs[n / 2][0] = a.x, bs[n / 2][1] = a.y, bs[n / 2][2] = a.z, bs[n / 2][3] = a.w;
            bs[n / 2][4] = b.x, bs[n / 2][5] = b.y, bs[n / 2][6] = b.z, bs[n / 2][7] = b.w;
        }
    }
#pragma unroll
    for (int f = 0; f < TF; ++f) {
        const int m = m0 + 16 * f + (lane & 15);
        uint4 rs[EXTRAS ? (TW + 1) / 2 : 1];
        if constexpr (EXTRAS) {
#pragma unroll
            for (int n = 0; n + 1 < TW; n += 2) {
                const int col = c0 + 16 * n;
                rs[n / 2] = (g.residual && m < g.M && col < g.N)
                                ? *reinterpret_cast<const uint4*>(g.residual + int64_t(m) * g.ldr + col)
                                : make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int n = 0; n + 1 < TW; n += 2) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[n][f][i]),
                                                                __float_as_uint(acc[n + 1][f][i]), false, false);
                v[i] = __uint_as_float(r[0]);
                v[4 + i] = __uint_as_float(r[1]);
            }
            if constexpr (EXTRAS) {
                if (g.bias) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] += bs[n / 2][i];
                }
                if (g.residual) {
                    const uint4 r = rs[n / 2];
                    v[0] += bf16_lo(r.x), v[1] += bf16_hi(r.x), v[2] += bf16_lo(r.y), v[3] += bf16_hi(r.y);
                    v[4] += bf16_lo(r.z), v[5] += bf16_hi(r.z), v[6] += bf16_lo(r.w), v[7] += bf16_hi(r.w);
                }
            }
            if (m < g.M && c0 + 16 * n < g.N)
                *reinterpret_cast<uint4*>(yp[n / 2] + 16 * f * row_step) =
                    make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                               pack_bf16x2(v[6], v[7]));
        }
    }
    if constexpr (TW % 2 == 1) {  // the last fragment alone: 4 features per lane
#pragma unroll
        for (int f = 0; f < TF; ++f) {
            const v4f one[1][1] = {{acc[TW - 1][f]}};
            const int mm[1] = {m0 + 16 * f + (lane & 15)}, nn[1] = {n0 + 16 * (TW - 1) + 4 * q};
            fp8_store_tiles<1, 1>(one, mm, nn, g);
        }
    }
}
// A wave's float32 sums as they are, to part[m][n].
template <int TW, int TF>
__device__ __forceinline__ void fp8_store_part(const v4f (&acc)[TW][TF], int m0, int n0, int lane, const Fp8Args& g,
                                               float* part) {
#pragma unroll
    for (int f = 0; f < TF; ++f)
#pragma unroll
        for (int n = 0; n < TW; ++n) {
            const int m = m0 + 16 * f + (lane & 15), at = n0 + 16 * n + 4 * (lane >> 4);
            if (m < g.M && at < g.N) *reinterpret_cast<v4f*>(part + int64_t(m) * g.N + at) = acc[n][f];
        }
}
template <int TW, int TF>
__device__ __forceinline__ void fp8_store_tile(const v4f (&acc)[TW][TF], int m0, int n0, int lane, const Fp8Args& g) {
    if (g.bias || g.residual)
        fp8_store_pairs<true>(acc, m0, n0, lane, g);
    else
        fp8_store_pairs<false>(acc, m0, n0, lane, g);
}

}  // namespace fq
