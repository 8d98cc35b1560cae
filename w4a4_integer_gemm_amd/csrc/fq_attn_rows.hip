// Attention of prompts of few rows (gfx950, wave64).
//
// The operator of fq_attn_prefill.hip where its blocks of rows would leave most of the chip
// idle.  A workgroup takes 16 columns of one key head, consecutive rows' query heads of
// its group, and its waves take tiles of 32 keys in turn and join at the end: a row's keys are
// shared out over the waves instead of passing one wave (fq_attn_columns.h).
//
// Bound by what a CU is given of the keys and values (about 90 GB/s: a tile is requested
// while the one before is worked on, and more do not fit the registers).  50 rows of 8 heads of 256 on one key head,
// 866 keys: 25 groups of columns, 13.2 us.  More workgroups along the keys would need a workspace for their
// parts, which the call does not have; along the values (PARTS) they only read all keys each.
#include <hip/hip_runtime.h>

#include "fq_attn.h"
#include "fq_attn_columns.h"
#include "fq_device.h"
#include "fq_internal.h"

namespace fq {
namespace {

constexpr int kColumns = kDecodeHeads;
constexpr int kWaves = 8;  // (a wave of the larger ones takes more than half of a SIMD's registers)

template <int DP, int WAVES, int PARTS>
__global__ __launch_bounds__(64 * WAVES) void attn_rows_kernel(PrefillArgs a, int64_t blocks) {
    using Cols = Columns<DP, false, false, PARTS>;
    using Unit = typename Cols::Unit;
    __shared__ __attribute__((aligned(16))) typename Cols::template Shared<WAVES> lds;
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kvh = int(blockIdx.x / PARTS) % a.kv_heads, group = a.q_heads / a.kv_heads;
    const int64_t b = blocks - 1 - int64_t(blockIdx.x / PARTS / a.kv_heads);  // (of a sequence, those that see most keys first)
    const int d0 = PARTS == 1 ? 0 : 128 * int(blockIdx.x % PARTS);             // the workgroup's first value,
    const int Dv = PARTS == 1 ? a.head_dim : min(a.head_dim - d0, 128);        // and how many it takes
    auto first = [&](int s) { return int64_t(max(0, min(a.cu_q[s], a.M))) * group / kColumns + s; };
    const int seq = find_sequence(a.seqs, b, first);
    if (seq < 0) return;
    const Rows qr = sequence_rows(a.cu_q, seq, a.M), kr = sequence_rows(a.cu_k, seq, a.M_k);
    const int q0 = qr.begin, Lq = qr.count, k0 = kr.begin, Lk = kr.count;
    const int64_t column0 = (b - (int64_t(q0) * group / kColumns + seq)) * kColumns;
    if (column0 < 0 || column0 >= int64_t(Lq) * group) return;
    const int D = a.head_dim, shift = Lk - Lq;  // row i sees the keys up to i + shift
    auto row_of = [&](int c) { return int((column0 + c) / group); };
    const int row = row_of(col), row_first = row_of(0), row_last = min(row_of(kColumns - 1), Lq - 1);
    const int head = kvh * group + int((column0 + col) % group);
    const int limit = row >= Lq ? -1 : a.causal ? min(row + shift, Lk - 1) : Lk - 1;  // the column's last key
    const int all = row_of(kColumns - 1) >= Lq ? -1 : a.causal ? min(row_first + shift, Lk - 1) : Lk - 1;  // every column's
    const int end = a.causal ? min(row_last + shift + 1, Lk) : Lk;

    Cols x;
    x.load_query(row < Lq ? a.q + (q0 + row) * a.q_token + head * a.q_head : nullptr, D, lds);
    const float c = a.scale * kLog2e;
    const uint8_t* const kbase = reinterpret_cast<const uint8_t*>(a.k + k0 * a.k_token + kvh * a.k_head);
    const uint8_t* const vbase = reinterpret_cast<const uint8_t*>(a.v + k0 * a.v_token + kvh * a.v_head + d0);
    const uint32_t kstride = uint32_t(2 * a.k_token), vstride = uint32_t(2 * a.v_token);
    Unit u[2];
    auto find = [&](int t) {  // (rows behind the sequence's last are read as that one)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = min(t + kDecodeUnit * i, Lk - 1);
            u[i] = Unit{kbase + 2 * (j * a.k_token), vbase + 2 * (j * a.v_token), nullptr, nullptr,
                        t + kDecodeUnit * i < Lk ? min(15, Lk - 1 - j) : 0};
        }
    };
    int t = kDecodeTile * wave;
    auto tile = [&](auto more) {  // (two copies of it: see fq_attn_decode.hip)
        float s[8], scale[8];
        x.scores(lds, wave, c, s, scale);
        if (t + kDecodeTile - 1 > all) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (t + kDecodeUnit * (i / 4) + 4 * g + i % 4 > limit) s[i] = -INFINITY;
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (decltype(more)::value) {
            find(t + kDecodeTile * WAVES);
            x.load_k(u, D, kstride);
        }
        __builtin_amdgcn_sched_barrier(0);
        x.add(s, scale);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (decltype(more)::value) x.load_v(u, Dv, vstride);
        __builtin_amdgcn_sched_barrier(0);
    };
    if constexpr (Cols::QL) __syncthreads();
    if (t < end) {
        find(t);
        x.load_k(u, D, kstride);
        __builtin_amdgcn_sched_barrier(0);
        x.load_v(u, Dv, vstride);
        __builtin_amdgcn_sched_barrier(0);
        for (; t + kDecodeTile * WAVES < end; t += kDecodeTile * WAVES) tile(std::true_type{});
        tile(std::false_type{});
    }
    x.meet(lds, wave);

    const int quads = Dv / 4;
    for (int i = threadIdx.x; i < kColumns * quads; i += 64 * WAVES) {
        const int column = i / quads, d = 4 * (i - column * quads), r = row_of(column);
        if (r >= Lq) continue;
        float top, sum;
        const float4 v = Cols::joined(lds, column, d, top, sum);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;  // (a row that sees no key: zeros)
        *reinterpret_cast<uint2*>(a.o + (q0 + r) * a.o_token + (kvh * group + int((column0 + column) % group)) * a.o_head + d0 + d) =
            make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
    }
}

}  // namespace

// Workgroups of a call.
int64_t attn_rows_groups(const PrefillArgs& a) {
    return (int64_t(a.M) * (a.q_heads / a.kv_heads) / kColumns + a.seqs) * a.kv_heads;
}
// (Two workgroups to a group are launched for few of them only.)
int64_t attn_rows_threads(const PrefillArgs& a) { return attn_rows_groups(a) * 64 * kWaves; }

namespace {

template <int DP, int PARTS>
void launch_parts(const PrefillArgs& a, hipStream_t st) {
    const int64_t groups = attn_rows_groups(a);
    hipLaunchKernelGGL((attn_rows_kernel<DP, kWaves, PARTS>), dim3(uint32_t(groups) * PARTS), dim3(64 * kWaves), 0, st, a,
                       groups / a.kv_heads);
}

template <int DP>
void launch_waves(const PrefillArgs& a, const DeviceInfo& dev, hipStream_t st) {
    // Two workgroups for a group of columns, each with half of the values, where both get a CU of their own (8
    // heads on 1 of 256, graph-replayed, us, one / two: 1 row on 817 keys 15.3 / 12.6, 50 on 866 16.8 / 13.6, 50 on
    // 3050 40.2 / 33.3, 200 rows 9.9 / 8.3).
    if constexpr (DP > 128) {
        if (2 * attn_rows_groups(a) <= dev.cus) return launch_parts<DP, 2>(a, st);
    }
    launch_parts<DP, 1>(a, st);
}

}  // namespace

hipError_t launch_attn_rows(const PrefillArgs& a, const DeviceInfo& dev, hipStream_t stream) {
    if (a.head_dim <= 64)
        launch_waves<64>(a, dev, stream);
    else if (a.head_dim <= 96)
        launch_waves<96>(a, dev, stream);
    else if (a.head_dim <= 128)
        launch_waves<128>(a, dev, stream);
    else if (a.head_dim <= 192)
        launch_waves<192>(a, dev, stream);
    else
        launch_waves<256>(a, dev, stream);
    return hipGetLastError();
}

}  // namespace fq
