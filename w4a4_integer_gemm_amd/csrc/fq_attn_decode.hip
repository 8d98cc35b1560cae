// Attention of one new token of each sequence over the paged cache (gfx950, wave64).
//
//   o[s][h] = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - max),  s_j = scale log2(e) <q[s][h], k_j>
//
// Bound by reading the visible keys and values once.  A workgroup takes up to 16
// query heads of one key head, so that they share the reading, and one part of a
// sequence; its four waves take tiles of 32 tokens in turn, each with its own
// running maximum, sum and output, and join at the end.  All parts of a batch have
// one length, found from its lengths by every workgroup (those of many sequences by a launch
// before), so that sequences of any lengths keep the chip equally busy.  Parts of a sequence
// meet in the workspace and are joined by a launch behind.
// (The products, and how a tile's operands are laid out, are in fq_attn_columns.h.)
//
// One sequence of 131071 tokens, 8 key heads of 128, bf16: 94 us and 5 to join its parts, 537 MB at 5.7 TB/s.  64
// sequences of 0 to 8191 tokens, 4 key heads of 128, e4m3: 19.8 us and 5 for 88 MB, 4.5 TB/s.  1024 of 500 tokens, 2 key
// heads, e4m3: 4.6 us for their plan and 54 for 275 MB, 5.1 TB/s.  One of 1024 tokens: 5.0 us and 3.6, latencies in a
// chain (lengths, page, keys, values, the meeting of the waves, and the parts again).
#include <hip/hip_runtime.h>

#include "fq_attn.h"
#include "fq_attn_columns.h"
#include "fq_device.h"
#include "fq_internal.h"
#include "fq_paged.h"
#include "fq_token.h"

namespace fq {
namespace {

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

// Sequences up to which every workgroup goes through all lengths; more of them are gone through once, by a launch of
// its own, since the workgroups grow with the sequences too.  (Graph-replayed us without / with that launch, 8 query heads of
// 128, e4m3.  8 key heads: 192 sequences of 64 tokens 14.1 / 15.8, 256 18.9 / 19.4, 384 28.5 / 24.4, 1024 107 / 58;
// 256 of 300 tokens 44.4 / 43.7, 384 67.6 / 59.4.  One key head: 256 of 300 17.4 / 19.1, 384 25.4 / 24.8, 768 43.9 / 34.1.)
constexpr int kScanned = 256;

// Part w of the batch: its sequence (-1: there are fewer parts), the number inside it and the
// parts it has, the sequence's length and a part's.  Every wave finds it.
struct Part {
    int seq, index, count, len, part_len;
};
__device__ __forceinline__ Part find_part(const DecodeArgs& a, int w, int target) {
    const int lane = threadIdx.x & 63, most = a.max_pages, size = a.cache.page_size;
    if (a.seqs > kScanned) {
        const int32_t* const plan = reinterpret_cast<const int32_t*>(a.plan);
        const int seq = find_sequence(a.seqs, w, [&](int s) { return a.plan[s].x; });
        const int first = scalar_load(plan, 2 * int64_t(seq)), count = scalar_load(plan, 2 * int64_t(seq) + 1);
        return Part{w - first < count ? seq : -1, w - first, count, paged_len(scalar_load(a.lens, seq), most, size),
                    scalar_load(plan, 2 * int64_t(a.seqs) + 1)};
    }
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

// The plan of a batch, by one workgroup.
constexpr int kPlanWaves = 16;
__global__ __launch_bounds__(64 * kPlanWaves) void attn_plan_kernel(DecodeArgs a, int target) {
    __shared__ uint64_t wave_units[kPlanWaves];
    __shared__ uint32_t wave_parts[kPlanWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    auto length = [&](int s) { return paged_len(a.lens[s], a.max_pages, a.cache.page_size); };
    unsigned long long units = 0;
    for (int s = threadIdx.x; s < a.seqs; s += 64 * kPlanWaves) units += decode_units(length(s));
    for (int d = 32; d; d >>= 1) units += __shfl_xor(units, d);
    if (lane == 0) wave_units[wave] = units;
    __syncthreads();
    units = 0;
    for (int i = 0; i < kPlanWaves; ++i) units += wave_units[i];
    const int per = decode_part_len(units, target);
    uint32_t before = 0;
    for (int s0 = 0; s0 < a.seqs; s0 += 64 * kPlanWaves) {
        const int s = s0 + threadIdx.x;
        const uint32_t n = s < a.seqs ? decode_count(length(s), per) : 0, upto = lanes_scan(n);
        if (lane == 63) wave_parts[wave] = upto;
        __syncthreads();
        uint32_t first = before + upto - n;
        for (int i = 0; i < kPlanWaves; ++i) {
            first += i < wave ? wave_parts[i] : 0;
            before += wave_parts[i];
        }
        if (s < a.seqs) a.plan[s] = make_int2(first, n);
        __syncthreads();
    }
    if (threadIdx.x == 0) a.plan[a.seqs] = make_int2(before, per);
}

template <int DP, bool FP8>
__global__ __launch_bounds__(256, 2) void attn_decode_kernel(DecodeArgs a, uint64_t magic, int target, int head_tiles) {
    using Cols = Columns<DP, FP8, true>;
    using Unit = typename Cols::Unit;
    __shared__ __attribute__((aligned(16))) typename Cols::template Shared<kDecodeWaves> lds;

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
    if (a.seqs <= kScanned && part.index == 0 && kvh == 0 && ht == 0 && threadIdx.x == 0) a.plan[seq] = make_int2(w, part.count);
    const int begin = part.index * part.part_len, end = min(begin + part.part_len, len);
    const int32_t* const table = a.page_table + int64_t(seq) * a.max_pages;
    const uint32_t row_bytes = uint32_t(D * Cols::ES);

    Cols x;
    x.load_query(col < heads ? a.q + seq * a.q_token + (head0 + col) * a.q_head : nullptr, D, lds);
    const float c = a.scale * kLog2e;

    Unit u[2];
    int valid[2];
    auto find = [&](int t) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int ti = t + kDecodeUnit * i, entry = paged_entry(ti, len, magic);
            const PagedUnit p = paged_unit(scalar_load(table, entry), entry, ti, len, kc.pages, kc.page_size);
            const int64_t row = paged_row(p.page, p.first, kvh, kc.kv_heads, kc.page_size);
            u[i] = Unit{static_cast<const uint8_t*>(kc.k) + row * row_bytes, static_cast<const uint8_t*>(kc.v) + row * row_bytes,
                        kc.k_scale + row, kc.v_scale + row, 15};
            valid[i] = p.valid;
        }
    };
    int t = begin + kDecodeTile * wave;
    // (Two copies of the loop's body: with the next tile's loads behind a branch, the waits for this one's
    // values would have to count on either and so wait for the next keys.)
    auto tile = [&](auto more) {
        const int seen[2] = {valid[0], valid[1]};
        if constexpr (decltype(more)::value) find(t + kDecodeStep);
        float s[8], scale[8];
        x.scores(lds, wave, c, s, scale);
        if (seen[0] != kDecodeUnit || seen[1] != kDecodeUnit) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (4 * g + i % 4 >= seen[i / 4]) x.drop(i, s, scale);
        }
        // (the next keys are on their way before the values are waited for, and older than the next values)
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (decltype(more)::value) x.load_k(u, D, row_bytes);
        __builtin_amdgcn_sched_barrier(0);
        x.add(s, scale);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (decltype(more)::value) x.load_v(u, D, row_bytes);
        __builtin_amdgcn_sched_barrier(0);
    };
    if constexpr (Cols::QL) __syncthreads();
    if (t < end) {
        find(t);
        x.load_k(u, D, row_bytes);
        __builtin_amdgcn_sched_barrier(0);
        x.load_v(u, D, row_bytes);
        __builtin_amdgcn_sched_barrier(0);
        for (; t + kDecodeStep < end; t += kDecodeStep) tile(std::true_type{});
        tile(std::false_type{});
    }
    x.meet(lds, wave);

    const int quads = D / 4;
    const bool whole = part.count == 1;
    for (int i = threadIdx.x; i < heads * quads; i += 64 * kDecodeWaves) {
        const int h = i / quads, d = 4 * (i - h * quads);
        float top, sum;
        const float4 v = Cols::joined(lds, h, d, top, sum);
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
    if (a.seqs > kScanned) hipLaunchKernelGGL(attn_plan_kernel, dim3(1), dim3(64 * kPlanWaves), 0, st, a, target);
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
