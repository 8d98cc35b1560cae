// Attention of 16 columns (query heads, or rows, that share a key head) by the waves of a
// workgroup, straight from global memory (gfx950, wave64).
//
// The waves take tiles of 32 keys in turn, each with its own running maximum, sum
// and output, and join at the end.  Both products are matrix instructions over the columns:
//   S^T[key][column] = K Q^T     lane l: key l % 16 of a unit of 16 keys, 8 of 32 d
//   O^T[d][column]   = V^T P^T   lane l: one d, 8 of the tile's 32 keys
// A lane holds its column's scores of keys 4 (l / 16) + 0 .. 3 of both units, and those
// are the 8 keys that it has to present to the second product: the weights never
// leave their lane.  The other operand needs 8 keys of one d in a lane; lane l loads
// 8 consecutive d of each of these 8 keys and pairs them up in registers, the d's of
// its piece going to eight products.  e4m3 codes are exact in bf16; the key's scale
// multiplies the score, the value's the weight, in float32.
//
// Both products are the matrix instruction's bf16 ones with float32 sums.  Its operand holds 8 bits of a weight, so
// that a weight goes in as two of them, its rounding to bf16 and that of what is left: off by 2^-16 of itself at most,
// where one would be off by 2^-8, as much as the output's own rounding.  The second product reads nothing more, and the
// matrix unit is idle for nine cycles of ten here: without / with it, decode of 64 ragged sequences 25.0 / 25.6 us, of
// 131071 tokens 102.4 / 102.3, of 1024 8.6 / 8.8; 50 rows on 866 keys 13.3 / 13.6, on 8050 69.3 / 71.4 (28 heads of 128
// 47.1 / 50.2).
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "fq_attn.h"
#include "fq_device.h"
#include "fq_paged.h"

namespace fq {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
// Two of a dword's four codes as bf16, times a power of two.
template <bool HI>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w, float times = 1.0f) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, times, HI));
}
// Codes of keys are multiplied as 2^-8 of themselves, 1.75 at most, and their scales as 2^8 of themselves (a bf16 key's
// is below 2^120): sums that the key's scale meets only afterwards then stay within those of the query's own values.
constexpr float kKeyCode = 0x1p-8f;

// 8 keys of one d, for the d's of dword c of a lane's piece (bf16: two; codes: four), from rows of 8 keys.
__device__ __forceinline__ void transpose_dword(const uint4 (&r)[8], int c, v8bf (&out)[2]) {
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint4 &x = r[2 * p], &y = r[2 * p + 1];
        const uint32_t a = c == 0 ? x.x : c == 1 ? x.y : c == 2 ? x.z : x.w, b = c == 0 ? y.x : c == 1 ? y.y : c == 2 ? y.z : y.w;
        lo[p] = __builtin_amdgcn_perm(b, a, 0x05040100u);
        hi[p] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    }
    out[0] = as_bf(make_uint4(lo[0], lo[1], lo[2], lo[3]));
    out[1] = as_bf(make_uint4(hi[0], hi[1], hi[2], hi[3]));
}
__device__ __forceinline__ void transpose_dword(const uint2 (&r)[8], int c, v8bf (&out)[4]) {
    uint32_t w[4][4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t a = c ? r[2 * p].y : r[2 * p].x, b = c ? r[2 * p + 1].y : r[2 * p + 1].x;
        const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x05010400u), hi = __builtin_amdgcn_perm(b, a, 0x07030602u);
        w[0][p] = codes_bf16<false>(lo);
        w[1][p] = codes_bf16<true>(lo);
        w[2][p] = codes_bf16<false>(hi);
        w[3][p] = codes_bf16<true>(hi);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) out[t] = as_bf(make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]));
}

// DP: head_dim rounded up to a size with code of its own.  Pieces past head_dim
// are read as the row's first piece: the query's zeros meet them in the first product, and
// the outputs of the second are not stored.
// WHOLE: every unit has its 16 rows (a page's units do).
// PARTS: workgroups that share a head's values and outputs, 128 d each (every one computes all weights).
template <int DP, bool FP8, bool WHOLE, int PARTS = 1>
struct Columns {
    static constexpr int ES = FP8 ? 1 : 2;                     // bytes of a value
    static constexpr int LEAST = DP == 64 ? 16 : DP == 96 ? 80 : DP == 128 ? 112 : DP == 192 ? 144 : 208;  // head_dim
    static constexpr int KL = FP8 ? (DP + 63) / 64 : DP / 32;  // 16-byte pieces of a lane's key
    static constexpr int KM = FP8 ? 2 * KL : KL;               // products of a unit
    // Keys pass through LDS: they are loaded a few whole rows at a time, since 16 rows in
    // 16 neighbouring lanes, as the product wants them, cost the address unit four times as much.
    static constexpr int PIECES = DP * ES <= 64 ? 4 : DP * ES <= 128 ? 8 : DP * ES <= 256 ? 16 : 32;  // of a row in LDS
    static constexpr int ROWS = 64 / PIECES, LOADS = kDecodeUnit / ROWS;  // rows of a load, loads of a unit
    static constexpr int HV = (DP + 127) / 128 / PARTS;        // pieces of 8 d of a lane's value
    static_assert(HV >= 1 && (PARTS == 1 || HV == 1), "a part is a piece of every lane");
    static constexpr int VD = PARTS == 1 ? DP : 128;           // d of the values that a workgroup takes
    static constexpr int LD = VD + 4;                          // (floats; a column's row in LDS starts on another bank)
    // The query in LDS where its registers would cost a wave's place on the SIMD.
    static constexpr bool QL = !FP8 && DP > 128;
    using vpiece = std::conditional_t<FP8, uint2, uint4>;

    // 16 rows of keys and of values, from the first; the scales of theirs that the lane needs.
    struct Unit {
        const uint8_t *k, *v;
        const float *ks, *vs;
        int last;  // row that the ones behind it are read as, with WHOLE 15
    };

    v8bf q[QL ? 1 : KM];
    u32x4 kf[2 * LOADS];
    vpiece vf[HV][8];
    float4 ks[2], vs[2];
    v4f acc[HV][8];
    float m = -INFINITY, l = 0.0f;

    // What the waves share: their parts' outputs, maxima and sums, and the query.
    template <int WAVES>
    struct Shared {
        union {
            float part[WAVES][kDecodeHeads][LD];
            u32x4 keys[WAVES][kDecodeTile * (PIECES + 1)];  // (a wave's own)
        };
        float stat[2][WAVES][kDecodeHeads];
        uint4 query[QL ? KM : 1][64];
    };
    // Place of piece c of key r: a row is one piece longer than an even number of them, so that 16
    // rows' pieces of one number lie in different banks.
    static __device__ __forceinline__ int key_place(int r, int c) { return r * (PIECES + 1) + c; }

    // The column's query (nullptr: zeros).  With QL a barrier has to follow.
    template <int WAVES>
    __device__ __forceinline__ void load_query(const uint16_t* p, int D, Shared<WAVES>& lds) {
        const int lane = threadIdx.x & 63, g = lane >> 4;
        if (!QL || threadIdx.x < 64) {
#pragma unroll
            for (int j = 0; j < KM; ++j) {
                const int d = FP8 ? 64 * (j / 2) + 16 * g + 8 * (j % 2) : 32 * j + 8 * g;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (p && d < D) v = *reinterpret_cast<const uint4*>(p + d);
                if constexpr (QL)
                    lds.query[j][lane] = v;
                else
                    q[j] = as_bf(v);
            }
        }
#pragma unroll
        for (int i = 0; i < HV; ++i)
#pragma unroll
            for (int t = 0; t < 8; ++t) acc[i][t] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    template <int WAVES>
    __device__ __forceinline__ v8bf query(const Shared<WAVES>& lds, int j, int lane) const {
        if constexpr (QL)
            return as_bf(lds.query[j][lane]);
        else
            return q[j];
    }

    // kstride, vstride: bytes from row to row.  (Both sides of a branch issue the same loads, so
    // that the waits behind it know how many are in flight.)
    __device__ __forceinline__ void load_k(const Unit (&u)[2], int D, uint32_t kstride) {
        const int lane = threadIdx.x & 63, g = lane >> 4, row = lane / PIECES, at = 16 * (lane % PIECES);
        const uint32_t piece = at < D * ES ? at : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (WHOLE || u[i].last == 15) {
#pragma unroll
                for (int j = 0; j < LOADS; ++j)
                    kf[LOADS * i + j] = *reinterpret_cast<const u32x4*>(u[i].k + uint64_t(ROWS * j) * kstride + (row * kstride + piece));
            } else {
#pragma unroll
                for (int j = 0; j < LOADS; ++j)
                    kf[LOADS * i + j] = *reinterpret_cast<const u32x4*>(u[i].k + (uint32_t(min(ROWS * j + row, u[i].last)) * kstride + piece));
            }
            if constexpr (FP8) {
                ks[i] = *reinterpret_cast<const float4*>(u[i].ks + 4 * g);
                vs[i] = *reinterpret_cast<const float4*>(u[i].vs + 4 * g);
            }
        }
    }
    // D: of the values that the workgroup takes, whose first the units' rows are.
    __device__ __forceinline__ void load_v(const Unit (&u)[2], int D, uint32_t vstride) {
        const int col = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int hv = 0; hv < HV; ++hv) {
                    const bool there = (PARTS == 1 && 128 * hv + 120 < LEAST) || 128 * hv + 8 * col < D;
                    const uint32_t piece = there ? 8 * ES * col : 0;
                    const uint8_t* const p = u[i].v + (there ? 128 * ES * hv : 0);
                    if (WHOLE || u[i].last == 15)
                        vf[hv][4 * i + j] = *reinterpret_cast<const vpiece*>(p + uint64_t(j) * vstride + (4 * g * vstride + piece));
                    else
                        vf[hv][4 * i + j] = *reinterpret_cast<const vpiece*>(p + (uint32_t(min(4 * g + j, u[i].last)) * vstride + piece));
                }
    }

    // The scores of the loaded keys, times c (and the key's scale), and the values' scales.
    template <int WAVES>
    __device__ __forceinline__ void scores(Shared<WAVES>& lds, int wave, float c, float (&x)[8], float (&w)[8]) {
        const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
        u32x4* const keys = lds.keys[wave];
#pragma unroll
        for (int n = 0; n < 2 * LOADS; ++n) keys[key_place(ROWS * n + lane / PIECES, lane % PIECES)] = kf[n];
        int at = lane;
        if constexpr (QL) asm volatile("" : "+v"(at));  // (so that the query is read again for every tile)
        v4f s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            s[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < KL; ++j) {
                const u32x4 k = keys[key_place(kDecodeUnit * i + col, 4 * j + g)];
                if constexpr (FP8) {
                    auto half = [&](uint32_t a, uint32_t b) {
                        return as_bf(make_uint4(codes_bf16<false>(a, kKeyCode), codes_bf16<true>(a, kKeyCode),
                                                codes_bf16<false>(b, kKeyCode), codes_bf16<true>(b, kKeyCode)));
                    };
                    s[i] = mfma_bf16_16(half(k[0], k[1]), query(lds, 2 * j, at), s[i]);
                    s[i] = mfma_bf16_16(half(k[2], k[3]), query(lds, 2 * j + 1, at), s[i]);
                } else {
                    s[i] = mfma_bf16_16(__builtin_bit_cast(v8bf, k), query(lds, j, at), s[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 &kq = ks[i / 4], &vq = vs[i / 4];
            const float ki = i % 4 == 0 ? kq.x : i % 4 == 1 ? kq.y : i % 4 == 2 ? kq.z : kq.w;
            x[i] = (FP8 ? s[i / 4][i % 4] * (ki * (1.0f / kKeyCode)) : s[i / 4][i % 4]) * c;
            w[i] = FP8 ? (i % 4 == 0 ? vq.x : i % 4 == 1 ? vq.y : i % 4 == 2 ? vq.z : vq.w) : 1.0f;
        }
    }
    // Key i of the lane (0 .. 7) is not seen by any column, and its place may hold anything.
    __device__ __forceinline__ void drop(int i, float (&x)[8], float (&w)[8]) {
        x[i] = -INFINITY;
        w[i] = 0.0f;
#pragma unroll
        for (int hv = 0; hv < HV; ++hv) vf[hv][i] = vpiece{};
    }
    // The weights of the scores x, and the loaded values with them.
    __device__ __forceinline__ void add(float (&x)[8], const float (&w)[8]) {
        float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        top = fmaxf(m, max_over_rows(top));
        if (__any(top > m)) {
            const float f = top == -INFINITY ? 1.0f : exp2_fast(m - top);
            l *= f;
#pragma unroll
            for (int hv = 0; hv < HV; ++hv)
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[hv][k] *= f;
            m = top;
        }
        const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = exp2_fast(x[i] - base);
            l += x[i];
            if constexpr (FP8) x[i] *= w[i];
        }
        // p: the weights in bf16; rest: what that leaves of them, in bf16 again
        uint32_t w0[4], w1[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w0[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
            w1[i] = pack_bf16x2(x[2 * i] - __uint_as_float(w0[i] << 16), x[2 * i + 1] - __uint_as_float(w0[i] & 0xFFFF0000u));
        }
        const v8bf p = as_bf(make_uint4(w0[0], w0[1], w0[2], w0[3])), rest = as_bf(make_uint4(w1[0], w1[1], w1[2], w1[3]));
#pragma unroll
        for (int hv = 0; hv < HV; ++hv) {
            constexpr int EACH = FP8 ? 4 : 2;  // d's of a dword
#pragma unroll
            for (int w = 0; w < 8 / EACH; ++w) {
                v8bf vt[EACH];
                transpose_dword(vf[hv], w, vt);
#pragma unroll
                for (int k = 0; k < EACH; ++k) acc[hv][EACH * w + k] = mfma_bf16_16(vt[k], p, acc[hv][EACH * w + k]);
#pragma unroll
                for (int k = 0; k < EACH; ++k) acc[hv][EACH * w + k] = mfma_bf16_16(vt[k], rest, acc[hv][EACH * w + k]);
            }
        }
    }

    // The waves' parts, each scaled to the common maximum, meet in LDS.
    template <int WAVES>
    __device__ __forceinline__ void meet(Shared<WAVES>& lds, int wave) {
        const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
        l = sum_over_rows(l);  // (the barrier below is behind every wave's last reading of its keys)
        if (g == 0) {
            lds.stat[0][wave][col] = m;
            lds.stat[1][wave][col] = l;
        }
        __syncthreads();
        float top = lds.stat[0][0][col];
#pragma unroll
        for (int i = 1; i < WAVES; ++i) top = fmaxf(top, lds.stat[0][i][col]);
        const float f = top == -INFINITY ? 0.0f : exp2_fast(m - top);
        // register r of product k: d = 128 hv + 32 g + 8 r + k
#pragma unroll
        for (int hv = 0; hv < HV; ++hv)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = 128 * hv + 32 * g + 8 * r;
                if (d >= VD) continue;
                float* const out = &lds.part[wave][col][d];
                *reinterpret_cast<float4*>(out) =
                    make_float4(acc[hv][0][r] * f, acc[hv][1][r] * f, acc[hv][2][r] * f, acc[hv][3][r] * f);
                *reinterpret_cast<float4*>(out + 4) =
                    make_float4(acc[hv][4][r] * f, acc[hv][5][r] * f, acc[hv][6][r] * f, acc[hv][7][r] * f);
            }
        __syncthreads();
    }
    // Four d of a column from there: the sums over the waves, their maximum and the weights' sum.
    template <int WAVES>
    static __device__ __forceinline__ float4 joined(const Shared<WAVES>& lds, int column, int d, float& top, float& sum) {
        top = lds.stat[0][0][column];
        sum = 0.0f;
#pragma unroll
        for (int w = 1; w < WAVES; ++w) top = fmaxf(top, lds.stat[0][w][column]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(&lds.part[w][column][d]);
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            sum += lds.stat[1][w][column] * (top == -INFINITY ? 0.0f : exp2_fast(lds.stat[0][w][column] - top));
        }
        return v;
    }
};

}  // namespace fq
