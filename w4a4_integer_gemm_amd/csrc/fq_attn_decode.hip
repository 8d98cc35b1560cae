// Attention of one new token of each sequence over the paged cache (gfx950, wave64).
//
//   o[s][h] = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - max),  s_j = scale log2(e) <q[s][h], k_j>
//
// Bound by reading the visible keys and values once.  A workgroup takes up to 16
// query heads of one key head, so that they share the reading, and one part of a
// sequence; its four waves take tiles of 32 tokens in turn, each with its own
// running maximum, sum and output, and join at the end.  All parts of a batch have
// one length, found from its lengths by every workgroup, so that sequences of any lengths keep
// the chip equally busy.  Parts of a sequence meet in the workspace and are joined by a
// second launch.
//
// Both products are matrix instructions over 16 heads:
//   S^T[key][head] = K Q^T     lane l: key l % 16 of a unit of 16 tokens, 8 of 32 d
//   O^T[d][head]   = V^T P^T   lane l: one d, 8 of the tile's 32 keys
// A lane holds its head's scores of keys 4 (l / 16) + 0 .. 3 of both units, and those
// are the 8 keys that it has to present to the second product: the weights never
// leave their lane.  The other operand needs 8 keys of one d in a lane; lane l loads
// 8 consecutive d of each of these 8 keys and pairs them up in registers, the d's of
// its piece going to eight products.  e4m3 codes are exact in bf16; the key's scale
// multiplies the score, the value's the weight before it is rounded to bf16.
#include <hip/hip_runtime.h>

#include "fq_attn.h"
#include "fq_device.h"
#include "fq_internal.h"
#include "fq_paged.h"
#include "fq_token.h"

namespace fq {
namespace {

// A uniform load that the vector loads in flight need not be waited for.
typedef const int32_t __attribute__((address_space(4)))* const_i32;
__device__ __forceinline__ int32_t scalar_load(const int32_t* p, int64_t i) {
    return reinterpret_cast<const_i32>(reinterpret_cast<uintptr_t>(p))[i];
}

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
// Two of a dword's four codes as bf16.
template <bool HI>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}

// 8 keys of one d (eight times, for 8 consecutive d) from rows of 8 keys.
__device__ __forceinline__ void transpose8(const uint4 (&r)[8], v8bf (&out)[8]) {
    uint32_t w[8][4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t a[4] = {r[2 * p].x, r[2 * p].y, r[2 * p].z, r[2 * p].w};
        const uint32_t b[4] = {r[2 * p + 1].x, r[2 * p + 1].y, r[2 * p + 1].z, r[2 * p + 1].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            w[2 * c][p] = __builtin_amdgcn_perm(b[c], a[c], 0x05040100u);
            w[2 * c + 1][p] = __builtin_amdgcn_perm(b[c], a[c], 0x07060302u);
        }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) out[t] = as_bf(make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]));
}
__device__ __forceinline__ void transpose8(const uint2 (&r)[8], v8bf (&out)[8]) {
    uint32_t w[8][4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t a[2] = {r[2 * p].x, r[2 * p].y}, b[2] = {r[2 * p + 1].x, r[2 * p + 1].y};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t lo = __builtin_amdgcn_perm(b[c], a[c], 0x05010400u);
            const uint32_t hi = __builtin_amdgcn_perm(b[c], a[c], 0x07030602u);
            w[4 * c][p] = codes_bf16<false>(lo);
            w[4 * c + 1][p] = codes_bf16<true>(lo);
            w[4 * c + 2][p] = codes_bf16<false>(hi);
            w[4 * c + 3][p] = codes_bf16<true>(hi);
        }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) out[t] = as_bf(make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]));
}

// Inclusive sums over the lanes before.
__device__ __forceinline__ uint32_t lanes_scan(uint32_t v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast 15, 31
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
    return v;
}

// Part w of the batch: its sequence (-1: there are fewer parts), the number inside it and the
// parts it has, the sequence's length and a part's.  Every wave finds it.
struct Part {
    int seq, index, count, len, part_len;
};
__device__ __forceinline__ Part find_part(const DecodeArgs& a, int w, int target) {
    const int lane = threadIdx.x & 63, most = a.max_pages, size = a.cache.page_size;
    if (a.seqs == 1) {
        const int len = paged_len(scalar_load(a.lens, 0), most, size);
        const int per = decode_part_len(decode_units(len), target), count = decode_count(len, per);
        return Part{w < count ? 0 : -1, w, count, len, per};
    }
    auto length = [&](int s) { return s < a.seqs ? paged_len(a.lens[s], most, size) : 0; };
    const int len0 = length(lane);
    uint64_t units = 0;
    for (int s0 = 0; s0 < a.seqs; s0 += 64)
        units += uint32_t(__builtin_amdgcn_readlane(int(lanes_scan(decode_units(s0 ? length(s0 + lane) : len0))), 63));
    const int per = decode_part_len(units, target);
    uint32_t before = 0;
    for (int s0 = 0; s0 < a.seqs; s0 += 64) {
        const int len = s0 ? length(s0 + lane) : len0;
        const uint32_t n = s0 + lane < a.seqs ? decode_count(len, per) : 0, upto = before + lanes_scan(n);
        const uint64_t past = __ballot(upto > uint32_t(w));
        if (past) {
            const int at = __builtin_ctzll(past);
            return Part{s0 + at, w - __builtin_amdgcn_readlane(int(upto - n), at), __builtin_amdgcn_readlane(int(n), at),
                        __builtin_amdgcn_readlane(len, at), per};
        }
        before = uint32_t(__builtin_amdgcn_readlane(int(upto), 63));
    }
    return Part{-1, 0, 0, 0, per};
}

// DP: head_dim rounded up to a size with code of its own.  A lane's pieces past
// head_dim read the row's first piece: the query's zeros meet them in the first product, and
// the outputs of the second are not stored.
template <int DP, bool FP8>
__global__ __launch_bounds__(256) void attn_decode_kernel(DecodeArgs a, uint64_t magic, int target, int head_tiles) {
    constexpr int ES = FP8 ? 1 : 2;                       // bytes of a value
    constexpr int KL = FP8 ? (DP + 63) / 64 : DP / 32;    // loads of 16 bytes of a lane's key
    constexpr int KM = FP8 ? 2 * KL : KL;                 // products of a unit
    constexpr int HV = (DP + 127) / 128;                  // pieces of 8 d of a lane's value
    constexpr int LD = DP + 4;                            // (floats; a head's row in LDS starts on another bank)
    using vpiece = std::conditional_t<FP8, uint2, uint4>;
    __shared__ __attribute__((aligned(16))) float slab[kDecodeWaves][kDecodeHeads][LD];
    __shared__ float ml[2][kDecodeWaves][kDecodeHeads];

    const KvCache& kc = a.cache;
    const int D = kc.head_dim, lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // tile of heads, key head, part
    int id = blockIdx.x;
    const int ht = id % head_tiles;
    id /= head_tiles;
    const int kvh = id % kc.kv_heads, w = id / kc.kv_heads;
    const int group = a.q_heads / kc.kv_heads;
    const int heads = group - ht * kDecodeHeads < kDecodeHeads ? group - ht * kDecodeHeads : kDecodeHeads;
    const int head0 = kvh * group + ht * kDecodeHeads;

    const Part part = find_part(a, w, target);
    if (part.seq < 0) return;
    const int seq = part.seq, len = part.len;
    if (part.index == 0 && kvh == 0 && ht == 0 && threadIdx.x == 0) a.plan[seq] = make_int2(w, part.count);
    const int begin = part.index * part.part_len, end = min(begin + part.part_len, len);
    const int32_t* const table = a.page_table + int64_t(seq) * a.max_pages;

    // the query's operand
    v8bf q[KM];
    {
        const uint16_t* const qp = a.q + seq * a.q_token + (head0 + (col < heads ? col : 0)) * a.q_head;
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            const int d = FP8 ? 64 * (j / 2) + 16 * g + 8 * (j % 2) : 32 * j + 8 * g;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (col < heads && d < D) v = *reinterpret_cast<const uint4*>(qp + d);
            q[j] = as_bf(v);
        }
    }
    const float c = a.scale * kLog2e;

    // a lane's offsets inside a unit, in bytes
    const int row_bytes = D * ES;
    int koff[KL], voff[HV];
#pragma unroll
    for (int i = 0; i < KL; ++i) {
        const int at = 16 * (4 * i + g);
        koff[i] = col * row_bytes + (at < row_bytes ? at : 0);
    }
#pragma unroll
    for (int i = 0; i < HV; ++i) {
        const int d = 128 * i + 8 * col;
        voff[i] = 4 * g * row_bytes + (d < D ? d * ES : 0);
    }

    uint4 kf[2][KL];
    vpiece vf[HV][8];
    float4 ks[2], vs[2];
    v4f acc[HV][8];
#pragma unroll
    for (int i = 0; i < HV; ++i)
#pragma unroll
        for (int t = 0; t < 8; ++t) acc[i][t] = v4f{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.0f;

    PagedUnit u[2];
    auto find = [&](int t) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int ti = t + kDecodeUnit * i, entry = paged_entry(ti, len, magic);
            u[i] = paged_unit(scalar_load(table, entry), entry, ti, len, kc.pages, kc.page_size);
        }
    };
    auto load_k = [&] {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t row = paged_row(u[i].page, u[i].first, kvh, kc.kv_heads, kc.page_size);
            const uint8_t* const p = static_cast<const uint8_t*>(kc.k) + row * row_bytes;
#pragma unroll
            for (int j = 0; j < KL; ++j) kf[i][j] = *reinterpret_cast<const uint4*>(p + koff[j]);
            if constexpr (FP8) {
                ks[i] = *reinterpret_cast<const float4*>(kc.k_scale + row + 4 * g);
                vs[i] = *reinterpret_cast<const float4*>(kc.v_scale + row + 4 * g);
            }
        }
    };
    auto load_v = [&] {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t row = paged_row(u[i].page, u[i].first, kvh, kc.kv_heads, kc.page_size);
            const uint8_t* const p = static_cast<const uint8_t*>(kc.v) + row * row_bytes;
#pragma unroll
            for (int hv = 0; hv < HV; ++hv)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    vf[hv][4 * i + j] = *reinterpret_cast<const vpiece*>(p + voff[hv] + j * row_bytes);
        }
    };

    int t = begin + kDecodeTile * wave;
    if (t < end) {
        find(t);
        load_k();
        load_v();
    }
    for (; t < end; t += kDecodeTile * kDecodeWaves) {
        const int valid[2] = {u[0].valid, u[1].valid};
        const bool more = t + kDecodeTile * kDecodeWaves < end;
        if (more) find(t + kDecodeTile * kDecodeWaves);
        // scores
        v4f s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            s[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < KL; ++j) {
                if constexpr (FP8) {
                    const uint4 w = kf[i][j];
                    s[i] = mfma_bf16_16(as_bf(make_uint4(codes_bf16<false>(w.x), codes_bf16<true>(w.x),
                                                         codes_bf16<false>(w.y), codes_bf16<true>(w.y))), q[2 * j], s[i]);
                    s[i] = mfma_bf16_16(as_bf(make_uint4(codes_bf16<false>(w.z), codes_bf16<true>(w.z),
                                                         codes_bf16<false>(w.w), codes_bf16<true>(w.w))), q[2 * j + 1], s[i]);
                } else {
                    s[i] = mfma_bf16_16(as_bf(kf[i][j]), q[j], s[i]);
                }
            }
        }
        float x[8], w[8];
        const bool all = valid[0] == kDecodeUnit && valid[1] == kDecodeUnit;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4& kq = ks[i / 4];
            const float4& vq = vs[i / 4];
            const float kk = i % 4 == 0 ? kq.x : i % 4 == 1 ? kq.y : i % 4 == 2 ? kq.z : kq.w;
            const float vv = i % 4 == 0 ? vq.x : i % 4 == 1 ? vq.y : i % 4 == 2 ? vq.z : vq.w;
            x[i] = s[i / 4][i % 4] * (FP8 ? kk * c : c);
            w[i] = FP8 ? vv : 1.0f;
        }
        if (!all) {  // (what the cache holds there may be anything)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool seen = 4 * g + i % 4 < valid[i / 4];
                x[i] = seen ? x[i] : -INFINITY;
                w[i] = seen ? w[i] : 0.0f;
#pragma unroll
                for (int hv = 0; hv < HV; ++hv)
                    if (!seen) vf[hv][i] = vpiece{};
            }
        }
        if (more) load_k();
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
        const v8bf p = as_bf(make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                        pack_bf16x2(x[6], x[7])));
#pragma unroll
        for (int hv = 0; hv < HV; ++hv) {
            v8bf vt[8];
            transpose8(vf[hv], vt);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[hv][k] = mfma_bf16_16(vt[k], p, acc[hv][k]);
        }
        if (more) load_v();
    }

    // the waves' parts: each scaled to the common maximum
    l = sum_over_rows(l);
    if (g == 0) {
        ml[0][wave][col] = m;
        ml[1][wave][col] = l;
    }
    __syncthreads();
    {
        float top = ml[0][0][col];
#pragma unroll
        for (int i = 1; i < kDecodeWaves; ++i) top = fmaxf(top, ml[0][i][col]);
        const float f = top == -INFINITY ? 0.0f : exp2_fast(m - top);
        // register r of product k: d = 128 hv + 32 g + 8 r + k
#pragma unroll
        for (int hv = 0; hv < HV; ++hv)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = 128 * hv + 32 * g + 8 * r;
                if (d >= DP) continue;
                float* const out = &slab[wave][col][d];
                *reinterpret_cast<float4*>(out) =
                    make_float4(acc[hv][0][r] * f, acc[hv][1][r] * f, acc[hv][2][r] * f, acc[hv][3][r] * f);
                *reinterpret_cast<float4*>(out + 4) =
                    make_float4(acc[hv][4][r] * f, acc[hv][5][r] * f, acc[hv][6][r] * f, acc[hv][7][r] * f);
            }
    }
    __syncthreads();
    const int quads = D / 4;
    const bool whole = part.count == 1;
    for (int i = threadIdx.x; i < heads * quads; i += 64 * kDecodeWaves) {
        const int h = i / quads, d = 4 * (i - h * quads);
        float top = ml[0][0][h], sum = 0.0f;
#pragma unroll
        for (int w = 1; w < kDecodeWaves; ++w) top = fmaxf(top, ml[0][w][h]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kDecodeWaves; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(&slab[w][h][d]);
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            sum += ml[1][w][h] * (top == -INFINITY ? 0.0f : exp2_fast(ml[0][w][h] - top));
        }
        if (whole) {
            const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;  // (no token seen: zeros)
            *reinterpret_cast<uint2*>(a.o + seq * a.o_token + (head0 + h) * a.o_head + d) =
                make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
        } else {
            const int64_t row = int64_t(w) * a.q_heads + head0 + h;
            *reinterpret_cast<float4*>(a.sums + row * D + d) = v;
            if (d == 0) a.stats[row] = make_float2(top, sum);
        }
    }
}

// The parts of one query head.  A thread takes four d of every (256 / quads)-th part, eight
// parts' loads at once, with a running maximum of its own; the threads meet in LDS.
__global__ __launch_bounds__(256) void attn_join_kernel(DecodeArgs a) {
    __shared__ __attribute__((aligned(16))) float4 sums[256];
    __shared__ float2 stats[64];
    const int D = a.cache.head_dim, seq = blockIdx.x / a.q_heads, head = blockIdx.x - seq * a.q_heads;
    const int t = threadIdx.x, quads = D / 4, lines = 256 / quads, line = t / quads, d = 4 * (t - line * quads);
    const int2 plan = a.plan[seq];
    const int count = plan.y;
    if (count <= 1) return;
    const int64_t row0 = int64_t(plan.x) * a.q_heads + head;
    constexpr int UN = 8;
    float m = -INFINITY, l = 0.0f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (line < lines) {
        for (int i = line; i < count; i += UN * lines) {
            float4 x[UN];
            float2 st[UN];
#pragma unroll
            for (int k = 0; k < UN; ++k) {
                const int part = min(i + k * lines, count - 1);  // (past the last: loaded again, of no weight)
                const int64_t row = row0 + int64_t(part) * a.q_heads;
                x[k] = *reinterpret_cast<const float4*>(a.sums + row * D + d);
                st[k] = a.stats[row];
                if (i + k * lines >= count) st[k] = make_float2(-INFINITY, 0.0f);
            }
            float top = m;
#pragma unroll
            for (int k = 0; k < UN; ++k) top = fmaxf(top, st[k].x);
            const float base = top == -INFINITY ? 0.0f : top, f = exp2_fast(m - base);
            v.x *= f, v.y *= f, v.z *= f, v.w *= f, l *= f;
#pragma unroll
            for (int k = 0; k < UN; ++k) {
                const float w = exp2_fast(st[k].x - base);
                v.x += w * x[k].x, v.y += w * x[k].y, v.z += w * x[k].z, v.w += w * x[k].w;
                l += w * st[k].y;
            }
            m = top;
        }
        sums[t] = v;
        if (d == 0) stats[line] = make_float2(m, l);
    }
    __syncthreads();
    if (t >= quads) return;
    float top = -INFINITY;
    for (int i = 0; i < lines; ++i) top = fmaxf(top, stats[i].x);
    const float base = top == -INFINITY ? 0.0f : top;
    v = make_float4(0.f, 0.f, 0.f, 0.f);
    l = 0.0f;
    for (int i = 0; i < lines; ++i) {
        const float w = exp2_fast(stats[i].x - base);
        const float4 x = sums[i * quads + t];
        v.x += w * x.x, v.y += w * x.y, v.z += w * x.z, v.w += w * x.w;
        l += w * stats[i].y;
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    *reinterpret_cast<uint2*>(a.o + seq * a.o_token + head * a.o_head + d) =
        make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
}

template <int DP>
void launch_bits(const DecodeArgs& a, hipStream_t st) {
    const int tiles = decode_head_tiles(a.q_heads, a.cache.kv_heads), target = decode_target(a.cache.kv_heads, tiles);
    const dim3 grid(uint32_t(int64_t(a.parts) * a.cache.kv_heads * tiles));
    const uint64_t magic = paged_magic(a.cache.page_size);
    if (a.cache.k_scale)
        hipLaunchKernelGGL((attn_decode_kernel<DP, true>), grid, dim3(64 * kDecodeWaves), 0, st, a, magic, target, tiles);
    else
        hipLaunchKernelGGL((attn_decode_kernel<DP, false>), grid, dim3(64 * kDecodeWaves), 0, st, a, magic, target, tiles);
}

}  // namespace

hipError_t launch_attn_decode(const DecodeArgs& a, hipStream_t stream) {
    const int D = a.cache.head_dim;
    if (D <= 64)
        launch_bits<64>(a, stream);
    else if (D <= 96)
        launch_bits<96>(a, stream);
    else if (D <= 128)
        launch_bits<128>(a, stream);
    else if (D <= 192)
        launch_bits<192>(a, stream);
    else
        launch_bits<256>(a, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == a.seqs) return e;  // (no sequence can have more than one part)
    hipLaunchKernelGGL(attn_join_kernel, dim3(uint32_t(a.seqs * a.q_heads)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace fq
