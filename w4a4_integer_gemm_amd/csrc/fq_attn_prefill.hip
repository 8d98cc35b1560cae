// Attention of whole prompts, packed one behind another (gfx950, wave64).
//
//   o[i] = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(s_ij - max_j),  s_ij = scale log2(e) <q_i, k_j>
//
// Bound by its two products.  A workgroup takes a block of query rows of one head
// and passes over the keys that they see in tiles, with a running maximum, sum and
// output; a wave holds 32 of the rows.  Both products are transposed, so that the
// weights never leave their lane:
//   S^T[key][row] = K Q^T   the query is the operand that stays in registers
//   O^T[d][row]   = V^T P^T lane l holds column l % 32 of S^T and of O^T: one row
// A lane has its row's scores of keys 8 n + 4 (l / 32) + 0 .. 3; pairs of n make the 8
// keys that it presents to the second product, and the transposing LDS read gives
// the other operand the same keys.
//
// Tiles go from global memory straight into LDS, the next one while the products of
// the current one run; 16-byte pieces are swizzled, so that neither the first
// operand's rows nor the transposing reads meet in a bank.  Rows behind a sequence's
// last key are read as that key and masked, whatever lies there.
#include <hip/hip_runtime.h>

#include <climits>

#include "fq_attn.h"
#include "fq_device.h"
#include "fq_internal.h"
#include "fq_ring.h"
#include "fq_token.h"

namespace fq {
namespace {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) const v4i lds_v4i;
typedef __attribute__((address_space(3))) v4s lds_v4s;

__device__ __forceinline__ v8bf lds_read16(uint32_t addr) {
    return __builtin_bit_cast(v8bf, *reinterpret_cast<lds_v4i*>(uintptr_t(addr)));
}
// 4 keys of one d: the 16 lanes of a row read a block of 4 keys x 16 d, 8 bytes each,
// and lane i gets column i of it.
__device__ __forceinline__ v4s lds_read_tr(uint32_t addr) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_v4s*>(uintptr_t(addr)));
}

template <int DP_, int WAVES_>
struct Shape {
    static constexpr int DP = DP_, WAVES = WAVES_;
    static constexpr int BQ = 32 * WAVES;            // query rows of a workgroup
    static constexpr int BK = DP <= 128 ? 64 : 32;   // keys of a tile
    static constexpr int CH = DP <= 64 ? 8 : DP <= 128 ? 16 : 32;  // 16-byte pieces of a row in LDS
    static constexpr int ROW = 16 * CH;              // its bytes
    static constexpr int TILE = BK * ROW;
    static constexpr int COPIES = TILE / 1024 / WAVES;  // of a wave, for the keys (the values) of a tile
    static constexpr int KT = BK / 32, DT = DP / 32, DS = DP / 16;
};

// Slot of piece c of row r.
template <int CH>
__device__ __forceinline__ int key_slot(int r, int c) { return c ^ (r & 7); }
template <int CH>
__device__ __forceinline__ int value_slot(int r, int c) { return c ^ (CH == 8 ? ((r >> 1) & 1) << 2 : (r & 3) << 2); }

// The sequence that block b of the launch belongs to and its first row: blocks of
// sequence s are cu[s] / BQ + s and the ones behind it, of which those of sequence s + 1
// leave at least as many as s has.
struct Block {
    int seq, row;  // the row inside the sequence
};
template <int BQ>
__device__ __forceinline__ Block find_block(const int32_t* cu, int seqs, int M, int b) {
    const int lane = threadIdx.x & 63;
    auto first = [&](int s) { return max(0, min(cu[s], M)) / BQ + s; };
    int n = 0;
    for (int s0 = 0; s0 < seqs; s0 += 64) {
        const int s = s0 + lane;
        n += __popcll(__ballot(s < seqs && first(s) <= b));
    }
    const int seq = __builtin_amdgcn_readfirstlane(max(n - 1, 0));
    return Block{seq, __builtin_amdgcn_readfirstlane((b - first(seq)) * BQ)};
}

template <class SH>
__global__ __launch_bounds__(64 * SH::WAVES) void attn_prefill_kernel(PrefillArgs a, int blocks) {
    constexpr int BQ = SH::BQ, BK = SH::BK, CH = SH::CH, ROW = SH::ROW, KT = SH::KT, DT = SH::DT, DS = SH::DS;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * 2 * SH::TILE];
    const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // heads in turn, the blocks that see most keys first
    const int head = blockIdx.x % a.q_heads, b = blocks - 1 - int(blockIdx.x / a.q_heads);
    const Block at = find_block<BQ>(a.cu_q, a.seqs, a.M, b);
    auto range = [](const int32_t* cu, int s, int M, int& begin, int& count) {
        begin = __builtin_amdgcn_readfirstlane(max(0, min(cu[s], M)));
        count = __builtin_amdgcn_readfirstlane(max(0, min(cu[s + 1], M) - begin));
    };
    int q0, Lq, k0, Lk;
    range(a.cu_q, at.seq, a.M, q0, Lq);
    if (at.row < 0 || at.row >= Lq) return;
    range(a.cu_k, at.seq, a.M_k, k0, Lk);
    const int D = a.head_dim, kvh = head / (a.q_heads / a.kv_heads);
    const int shift = Lk - Lq;  // row i sees the keys up to i + shift
    const int rows = min(BQ, Lq - at.row);
    const int seen = a.causal ? min(Lk, at.row + rows + shift) : Lk;  // by any of the block's rows
    const int tiles = seen > 0 ? (seen + BK - 1) / BK : 0;
    const int row = at.row + 32 * wave + col;  // this lane's
    const int limit = a.causal ? min(row + shift, Lk - 1) : Lk - 1;  // its last key
    // keys that every row of the wave sees, and that any sees
    const int wave_all = a.causal ? min(at.row + 32 * wave + shift, Lk - 1) : Lk - 1;
    const int wave_any = at.row + 32 * wave >= Lq ? -1 : a.causal ? min(min(at.row + 32 * wave + 31, Lq - 1) + shift, Lk - 1) : Lk - 1;

    // the query's operand
    v8bf q[DS];
    {
        const uint16_t* const p = a.q + (q0 + min(row, Lq - 1)) * a.q_token + head * a.q_head;
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
        for (int i = 0; i < DS; ++i) {
            const int d = 16 * i + 8 * half;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (d < D) v = *reinterpret_cast<const uint4*>(p + d);
            q[i] = as_bf(make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip));
        }
    }
    const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);  // (0 times a masked score would be no number)

    // copies
    const uint32_t lds0 = lds_address(lds);
    const uint8_t* const kbase = reinterpret_cast<const uint8_t*>(a.k + k0 * a.k_token + kvh * a.k_head);
    const uint8_t* const vbase = reinterpret_cast<const uint8_t*>(a.v + k0 * a.v_token + kvh * a.v_head);
    constexpr int PER = 64 / CH;  // rows of a copy
    int crow[SH::COPIES];
    uint32_t kpiece[SH::COPIES], vpiece[SH::COPIES];
#pragma unroll
    for (int i = 0; i < SH::COPIES; ++i) {
        const int r = (wave * SH::COPIES + i) * PER + lane / CH, slot = lane % CH;
        const int kc = key_slot<CH>(r, slot), vc = value_slot<CH>(r, slot);
        crow[i] = r;
        kpiece[i] = kc * 8 < D ? 16 * kc : 0;  // (pieces past head_dim: any that exists)
        vpiece[i] = vc * 8 < D ? 16 * vc : 0;
    }
    auto copy = [&](int t) {
        const uint32_t dst = lds0 + (t & 1) * 2 * SH::TILE + wave * SH::COPIES * 1024;
        const int j0 = t * BK, last = min(BK, Lk - j0) - 1;
        const uint8_t* const kp = kbase + 2 * (j0 * a.k_token);
        const uint8_t* const vp = vbase + 2 * (j0 * a.v_token);
#pragma unroll
        for (int i = 0; i < SH::COPIES; ++i) {
            const uint32_t r = uint32_t(min(crow[i], last));
            copy16_base(kp, r * uint32_t(2 * a.k_token) + kpiece[i], dst + 1024 * i);
            copy16_base(vp, r * uint32_t(2 * a.v_token) + vpiece[i], dst + SH::TILE + 1024 * i);
        }
    };

    // addresses of the operands' reads in a stage
    uint32_t ka[4], va[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ka[i] = lds0 + col * ROW + 16 * key_slot<CH>(col, 2 * i + half);
        const int r = 4 * half + (lane & 15) / 4, sub = (lane >> 4) & 1;
        va[i] = lds0 + SH::TILE + r * ROW + 16 * value_slot<CH>(r, (CH == 8 ? 4 * (i & 1) : 4 * i) + 2 * sub + ((lane & 3) >> 1)) +
                8 * (lane & 1);
    }

    v16f o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
    float m = -INFINITY, l = 0.0f;

    if (tiles > 0) copy(0);
    for (int t = 0; t < tiles; ++t) {
        wait_vmcnt<0>();
        barrier_lds();
        if (t + 1 < tiles) copy(t + 1);
        const int j0 = t * BK;
        if (j0 > wave_any) continue;
        const uint32_t stage = (t & 1) * 2 * SH::TILE;
        v16f s[KT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[kt][r] = 0.0f;
#pragma unroll
        for (int i = 0; i < DS; ++i)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
                s[kt] = mfma_bf16_32(lds_read16(ka[i & 3] + stage + kt * 32 * ROW + (i >> 2) * 128), q[i], s[kt]);
        if (j0 + BK - 1 > wave_all) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (j0 + 32 * kt + 8 * (r / 4) + 4 * half + r % 4 > limit) s[kt][r] = -INFINITY;
        }
        float top = s[0][0];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[kt][r]);
        top = fmaxf(m, max_over_halves(top));
        // A maximum that grew by less than 2^8 stays where it was: the weights reach 256 at most.
        if (__any((top - m) * c > 8.0f)) {
            const float f = top == -INFINITY ? 1.0f : exp2_fast((m - top) * c);
            l *= f;
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[i][r] *= f;
            m = top;
        }
        const float base = m == -INFINITY ? 0.0f : m * c;
        v8bf p[KT][2];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[kt][r] = exp2_fast(__builtin_fmaf(s[kt][r], c, -base));
                l += s[kt][r];
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
                p[kt][u] = as_bf(make_uint4(pack_bf16x2(s[kt][8 * u], s[kt][8 * u + 1]), pack_bf16x2(s[kt][8 * u + 2], s[kt][8 * u + 3]),
                                            pack_bf16x2(s[kt][8 * u + 4], s[kt][8 * u + 5]),
                                            pack_bf16x2(s[kt][8 * u + 6], s[kt][8 * u + 7])));
        }
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) {
                    const uint32_t ad = va[dt & 3] + stage + (32 * kt + 16 * u) * ROW + (dt >> 2) * 256;
                    const v4s lo = lds_read_tr(ad), hi = lds_read_tr(ad + 8 * ROW);
                    const v8bf v = __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                    o[dt] = mfma_bf16_32(v, p[kt][u], o[dt]);
                }
    }

    if (row >= Lq) return;
    l = sum_over_halves(l);
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;  // (a row that sees no key: zeros)
    uint16_t* const op = a.o + (q0 + row) * a.o_token + head * a.o_head;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int d = 32 * dt + 8 * n + 4 * half;
            if (d < D)
                *reinterpret_cast<uint2*>(op + d) = make_uint2(pack_bf16x2(o[dt][4 * n] * inv, o[dt][4 * n + 1] * inv),
                                                               pack_bf16x2(o[dt][4 * n + 2] * inv, o[dt][4 * n + 3] * inv));
        }
}

template <class SH>
void launch_shape(const PrefillArgs& a, hipStream_t st) {
    const int blocks = a.M / SH::BQ + a.seqs;
    hipLaunchKernelGGL((attn_prefill_kernel<SH>), dim3(uint32_t(blocks) * uint32_t(a.q_heads)), dim3(64 * SH::WAVES), 0, st, a,
                       blocks);
}

}  // namespace

hipError_t launch_attn_prefill(const PrefillArgs& a, hipStream_t stream) {
    if (a.head_dim <= 64)
        launch_shape<Shape<64, 4>>(a, stream);
    else if (a.head_dim <= 96)
        launch_shape<Shape<96, 4>>(a, stream);
    else if (a.head_dim <= 128)
        launch_shape<Shape<128, 4>>(a, stream);
    else if (a.head_dim <= 192)
        launch_shape<Shape<192, 4>>(a, stream);
    else
        launch_shape<Shape<256, 4>>(a, stream);
    return hipGetLastError();
}

}  // namespace fq
