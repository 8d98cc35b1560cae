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
// Tiles go from global memory straight into LDS, two stages of them, each copy issued
// between two products; 16-byte pieces are swizzled, so that neither the first operand's rows
// nor the transposing reads meet in a bank.  Rows behind a sequence's last key are read as that
// key and masked, whatever lies there.
//
// A wave's loop is a software pipeline, so that the matrix unit has work while the vector unit makes
// weights: the products of the next tile's scores are issued with this tile's scalings, powers and
// packings between them, and those of the output with the next tile's maximum.  Operands are
// read four products ahead.
//
// Rounded: the output, and before it the weights, to bf16, as the product's operand (2^-8 of each at most; the
// sum takes them as rounded, so that they still add up to one).  Multiplying what the rounding leaves of them
// too, as decode and the kernel of few rows do, is half as many products again where products are the bound: without / with
// it, 28 heads on 4 of 128, 1024 rows 22.2 / 25.4 us, 4096 rows 134 / 196, 16384 rows 1757 / 2729; 16 heads of 64,
// 8192 rows 175 / 234; 8 on 1 of 256, 16384 rows 1103 / 1464.
//
// 16384 rows, 28 heads on 4 of 128, causal: 1.70 to 1.77 ms, 1.09 to 1.13 PFLOP/s, where a bf16 product of 8192^3 by
// the library runs at 1.26 and the matrix unit alone, on random operands in registers, at 1.69 to 1.75; the products keep
// it busy for 65 % of the cycles, at the 1.65 to 1.8 GHz that the power limit leaves it.  4580 rows of eight
// sequences: 59.7 us, 44 % busy: the last blocks, and a block's first loads and its epilogue (about 5 us).  1024 rows:
// 19.2 us, 24 % busy: two blocks to a CU, whose 16 tiles follow one another.
#include <hip/hip_runtime.h>

#include <atomic>
#include <type_traits>

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

// WQ x WK waves: WQ of them share a tile and have 32 query rows each; WK such groups take
// the tiles in turn and join at the end.
template <int DP_, int WQ_, int WK_, int BK_>
struct Shape {
    static constexpr int DP = DP_, WQ = WQ_, WK = WK_, THREADS = 64 * WQ * WK;
    static constexpr int BQ = 32 * WQ;  // query rows of a workgroup
    static constexpr int BK = BK_;      // keys of a tile
    static constexpr int CH = DP <= 64 ? 8 : DP <= 128 ? 16 : 32;  // 16-byte pieces of a row in LDS
    static constexpr int ROW = 16 * CH;              // its bytes
    static constexpr int TILE = BK * ROW;            // of keys, or of values
    static constexpr int RING = 2 * 2 * TILE;        // of a group: two stages
    static constexpr int COPIES = TILE / 1024 / WQ;  // of a wave, for the keys (the values) of a tile
    static constexpr int KT = BK / 32, DT = DP / 32, DS = DP / 16;
    static constexpr int SLAB = 1024 * 4 * DT + 512;  // a wave's output, maxima and sums
    static constexpr int JOIN = (WK - 1) * WQ * SLAB, LDS = WK * RING > JOIN ? WK * RING : JOIN;
    static_assert(COPIES * WQ * 1024 == TILE && LDS <= 160 * 1024, "LDS");
};

// Slot of piece c of row r.
template <int CH>
__device__ __forceinline__ int key_slot(int r, int c) { return c ^ (r & (CH == 8 ? 7 : 15)); }
template <int CH>
__device__ __forceinline__ int value_slot(int r, int c) { return c ^ (CH == 8 ? ((r >> 1) & 1) << 2 : (r & 3) << 2); }

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
// l plus the two packed weights: the sum is that of the weights as they are multiplied.
__device__ __forceinline__ float add_weights(uint32_t w, float l) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2bf, w), __builtin_bit_cast(v2bf, 0x3F803F80u), l, false);
}

template <class SH>
__global__ __launch_bounds__(SH::THREADS) void attn_prefill_kernel(PrefillArgs a, int blocks) {
    constexpr int BQ = SH::BQ, BK = SH::BK, CH = SH::CH, ROW = SH::ROW, KT = SH::KT, DT = SH::DT, DS = SH::DS, WK = SH::WK;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[SH::LDS];
    const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wq = wave % SH::WQ, wk = wave / SH::WQ;
    // heads in turn, from the last sequence to the first, and of a sequence the blocks that see most keys first (that
    // a long sequence in front has its blocks behind those of short ones is not looked at)
    const int head = blockIdx.x % a.q_heads, b = blocks - 1 - int(blockIdx.x / a.q_heads);
    // (those of sequence s are cu[s] / BQ + s and on, which leaves at least as many as it has)
    auto first = [&](int s) { return max(0, min(a.cu_q[s], a.M)) / BQ + s; };
    const int seq = find_sequence(a.seqs, b, first);
    if (seq < 0) return;
    const Rows qr = sequence_rows(a.cu_q, seq, a.M), kr = sequence_rows(a.cu_k, seq, a.M_k);
    const int q0 = qr.begin, Lq = qr.count, k0 = kr.begin, Lk = kr.count;
    const int at_row = (b - (q0 / BQ + seq)) * BQ;
    if (at_row < 0 || at_row >= Lq) return;
    const int D = a.head_dim, kvh = head / (a.q_heads / a.kv_heads);
    const int shift = Lk - Lq;  // row i sees the keys up to i + shift
    const int rows = min(BQ, Lq - at_row);
    const int seen = a.causal ? min(Lk, at_row + rows + shift) : Lk;  // by any of the block's rows
    const int tiles = seen > 0 ? (seen + BK - 1) / BK : 0;
    const int row0 = at_row + 32 * wq, row = row0 + col;  // the wave's first, this lane's
    const int limit = a.causal ? min(row + shift, Lk - 1) : Lk - 1;  // its last key
    // the last key that every row of the wave sees, and that any sees
    const int wave_all = a.causal ? min(row0 + shift, Lk - 1) : Lk - 1;
    const int wave_any = row0 >= Lq ? -1 : a.causal ? min(min(row0 + 31, Lq - 1) + shift, Lk - 1) : Lk - 1;

    // copies: of the rows of a whole tile, or of its first ones
    const uint32_t lds0 = lds_address(lds) + wk * SH::RING;
    const uint8_t* const kbase = reinterpret_cast<const uint8_t*>(a.k + k0 * a.k_token + kvh * a.k_head);
    const uint8_t* const vbase = reinterpret_cast<const uint8_t*>(a.v + k0 * a.v_token + kvh * a.v_head);
    const uint32_t kstride = uint32_t(2 * a.k_token), vstride = uint32_t(2 * a.v_token);
    constexpr int PER = 64 / CH;  // rows of a copy
    auto offset = [&](int i, int most, bool value) {
        const int r = (wq * SH::COPIES + i) * PER + lane / CH, slot = lane % CH;
        const int piece = value ? value_slot<CH>(r, slot) : key_slot<CH>(r, slot);
        // (pieces past head_dim: any that exists; rows behind the sequence: its last)
        return uint32_t(min(r, most)) * (value ? vstride : kstride) + (piece * 8 < D ? 16 * piece : 0);
    };
    uint32_t koff[SH::COPIES], voff[SH::COPIES];
#pragma unroll
    for (int i = 0; i < SH::COPIES; ++i) {
        koff[i] = offset(i, BK, false);
        voff[i] = offset(i, BK, true);
    }
    const uint32_t cdst = lds0 + wq * SH::COPIES * 1024;
    // Copies of the group's tile t, rows (t * WK + wk) * BK and on; behind the last tile they
    // read it again, so that no branch lies between the products.
    struct Source {
        const uint8_t *k, *v;
        uint32_t kdst, vdst;
    };
    auto source = [&](int tk, int tv) {
        const int jk = min(tk * WK + wk, tiles - 1) * BK, jv = min(tv * WK + wk, tiles - 1) * BK;
        if (jk + BK > Lk) {
#pragma unroll
            for (int i = 0; i < SH::COPIES; ++i) koff[i] = offset(i, Lk - jk - 1, false);
        }
        if (jv + BK > Lk) {
#pragma unroll
            for (int i = 0; i < SH::COPIES; ++i) voff[i] = offset(i, Lk - jv - 1, true);
        }
        return Source{kbase + 2 * (jk * a.k_token), vbase + 2 * (jv * a.v_token), cdst + (tk & 1) * 2 * SH::TILE,
                      cdst + (tv & 1) * 2 * SH::TILE + SH::TILE};
    };
    auto copy_k = [&](const Source& from, int i) { copy16_base(from.k, koff[i], from.kdst + 1024 * i); };
    auto copy_v = [&](const Source& from, int i) { copy16_base(from.v, voff[i], from.vdst + 1024 * i); };
    const int rounds = (tiles + WK - 1) / WK;  // tiles of the first group,
    const int wave_tiles = wave_any < wk * BK ? 0 : (wave_any / BK - wk) / WK + 1;  // and those that the wave's rows see
    if (tiles > 0) {
        const Source first = source(0, 0);
#pragma unroll
        for (int i = 0; i < SH::COPIES; ++i) copy_k(first, i);
#pragma unroll
        for (int i = 0; i < SH::COPIES; ++i) copy_v(first, i);
        const Source second = source(1, 1);
#pragma unroll
        for (int i = 0; i < SH::COPIES; ++i) copy_k(second, i);
    }

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
    // (0 times a masked score would be no number; no score of float32 gets past 2^-21 times this one)
    const float c = fmaxf(fabsf(a.scale) * kLog2e, 0x1p-149f);

    // addresses of the operands' reads in a stage
    constexpr int KA = CH == 8 ? 4 : 8;
    uint32_t ka[KA], va[4];
#pragma unroll
    for (int i = 0; i < KA; ++i) ka[i] = lds0 + col * ROW + 16 * key_slot<CH>(col, 2 * i + half);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
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

    // One product of the scores, or of the output, at a time, its operand read AHEAD
    // products before.
    constexpr int NS = DS * KT, NO = 2 * DT * KT, AHEAD = 4;
    auto key_frag = [&](int stage, int n) {
        const int i = n / KT, kt = n % KT;
        return lds_read16(ka[i % KA] + (stage + kt * 32 * ROW + (i / KA) * 32 * KA));
    };
    auto value_frag = [&](int stage, int n) {
        const int dt = n % DT, ku = n / DT;
        const uint32_t x = va[dt & 3] + (stage + 16 * ku * ROW + (dt >> 2) * 256);
        const v4s lo = lds_read_tr(x), hi = lds_read_tr(x + 8 * ROW);
        return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    // Scores of the tile in a stage; `between(n)` is put behind product n.
    auto scores = [&](int stage, v16f (&s)[KT], auto between) {
        v8bf f[AHEAD];
#pragma unroll
        for (int n = 0; n < AHEAD; ++n) f[n] = key_frag(stage, n);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[kt][r] = 0.0f;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            s[n % KT] = mfma_bf16_32(f[n % AHEAD], q[n / KT], s[n % KT]);
            if (n + AHEAD < NS) f[n % AHEAD] = key_frag(stage, n + AHEAD);
            between(n);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto mask = [&](int t, v16f (&s)[KT]) {
        const int j0 = (t * WK + wk) * BK;
        if (j0 + BK - 1 <= wave_all) return;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (j0 + 32 * kt + 8 * (r / 4) + 4 * half + r % 4 > limit) s[kt][r] = -INFINITY;
    };
    // A maximum that grew by less than 2^8 stays where it was: the weights reach 256 at most.
    auto raise = [&](float top) {
        top = fmaxf(m, max_over_halves(top));
        if (!__any((top - m) * c > 8.0f)) return;
        const float f = top == -INFINITY ? 1.0f : exp2_fast((m - top) * c);
        l *= f;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[i][r] *= f;
        m = top;
    };

    // Software pipeline: the scores of the next tile are computed between the weights of
    // this one, and their maximum between the products of this one's weights.
    v16f s0[KT], s1[KT];
    wait_vmcnt<0>();
    barrier_lds();
    if (wave_tiles > 0) {
        scores(0, s0, [](int) {});
        mask(0, s0);
        float top = -INFINITY;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s0[kt][r]);
        raise(top);
    }
    // Tile t, in stage STAGE, from its scores s; those of tile t + 1 go to next.
    auto tile = [&](int t, auto stage_tag, v16f (&s)[KT], v16f (&next)[KT]) {
        constexpr int HERE = decltype(stage_tag)::value * 2 * SH::TILE, THERE = 2 * SH::TILE - HERE;
        wait_vmcnt<0>();
        barrier_lds();
        const Source from = source(t + 2, t + 1);
        auto copy = [&](int n) {
            if (n < SH::COPIES)
                copy_k(from, n);
            else
                copy_v(from, n - SH::COPIES);
        };
        if (t >= wave_tiles) {
#pragma unroll
            for (int n = 0; n < 2 * SH::COPIES; ++n) copy(n);
            return;
        }
        const float base = m == -INFINITY ? 0.0f : m * c;
        uint32_t w[KT][8];
        // Pairs of weights, spread over the products: scaled one product ahead, raised, and packed one behind,
        // so that no instruction waits for the one before it.
        constexpr int PAIRS = 8 * KT;
        auto pairs = [&](int n, auto what) {
            if (n < 0 || n >= NS) return;
#pragma unroll
            for (int e = PAIRS * n / NS; e < PAIRS * (n + 1) / NS; ++e) what(e / 8, e % 8);
        };
        auto scaled = [&](int kt, int i) {
#pragma unroll
            for (int r = 2 * i; r < 2 * i + 2; ++r) s[kt][r] = __builtin_fmaf(s[kt][r], c, -base);
        };
        auto raised = [&](int kt, int i) {
#pragma unroll
            for (int r = 2 * i; r < 2 * i + 2; ++r) s[kt][r] = exp2_fast(s[kt][r]);
        };
        auto packed = [&](int kt, int i) {
            w[kt][i] = pack_bf16x2(s[kt][2 * i], s[kt][2 * i + 1]);
            l = add_weights(w[kt][i], l);
            asm volatile("" : "+v"(w[kt][i]), "+v"(l));  // (here, not behind the branch below)
        };
        pairs(0, scaled);
        // (behind the last tile: scores of whatever the stage holds, not used)
        scores(THERE, next, [&](int n) {
#pragma unroll
            for (int i = 2 * SH::COPIES * n / NS; i < 2 * SH::COPIES * (n + 1) / NS; ++i) copy(i);
            pairs(n + 1, scaled);
            pairs(n, raised);
            pairs(n - 1, packed);
        });
        pairs(NS - 1, packed);
        v8bf f[AHEAD];
#pragma unroll
        for (int n = 0; n < AHEAD; ++n) f[n] = value_frag(HERE, n);
        if (t + 1 < wave_tiles) mask(t + 1, next);
        float top = -INFINITY;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < NO; ++n) {
            const int dt = n % DT, ku = n / DT, kt = ku / 2, u = ku % 2;
            const v8bf p = as_bf(make_uint4(w[kt][4 * u], w[kt][4 * u + 1], w[kt][4 * u + 2], w[kt][4 * u + 3]));
            o[dt] = mfma_bf16_32(f[n % AHEAD], p, o[dt]);
            if (n + AHEAD < NO) f[n % AHEAD] = value_frag(HERE, n + AHEAD);
            constexpr int EACH = (16 * KT + NO - 1) / NO;
#pragma unroll
            for (int e = EACH * n; e < EACH * (n + 1) && e < 16 * KT; ++e) top = fmaxf(top, next[e / 16][e % 16]);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (t + 1 < wave_tiles) raise(top);
    };
    for (int t = 0; t < rounds; t += 2) {
        tile(t, std::integral_constant<int, 0>{}, s0, s1);
        if (t + 1 < rounds) tile(t + 1, std::integral_constant<int, 1>{}, s1, s0);
    }
    wait_vmcnt<0>();  // (the copies behind the last tile)
    l = sum_over_halves(l);

    barrier_lds();  // (every wave's copies have landed, and its reads are done)
    if constexpr (WK > 1) {
        // the groups' parts, scaled to the common maximum, are added in the groups' order
        uint8_t* const slab = lds + ((wk - 1) * SH::WQ + wq) * SH::SLAB;  // (not of group 0)
        if (wk > 0) {
#pragma unroll
            for (int i = 0; i < 4 * DT; ++i)
                reinterpret_cast<float4*>(slab)[64 * i + lane] = make_float4(o[i / 4][4 * (i % 4)], o[i / 4][4 * (i % 4) + 1],
                                                                             o[i / 4][4 * (i % 4) + 2], o[i / 4][4 * (i % 4) + 3]);
            reinterpret_cast<float2*>(slab + 4096 * DT)[lane] = make_float2(m, l);
        }
        barrier_lds();
        if (wk == 0) {
            float2 st[WK - 1];
            float top = m;
#pragma unroll
            for (int k = 0; k < WK - 1; ++k) {
                st[k] = reinterpret_cast<const float2*>(lds + (k * SH::WQ + wq) * SH::SLAB + 4096 * DT)[lane];
                top = fmaxf(top, st[k].x);
            }
            const float base = top == -INFINITY ? 0.0f : top, f = exp2_fast((m - base) * c);
            l *= f;
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[i][r] *= f;
#pragma unroll
            for (int k = 0; k < WK - 1; ++k) {
                const float fk = exp2_fast((st[k].x - base) * c);
                l += st[k].y * fk;
                const float4* const other = reinterpret_cast<const float4*>(lds + (k * SH::WQ + wq) * SH::SLAB);
#pragma unroll
                for (int i = 0; i < 4 * DT; ++i) {
                    const float4 x = other[64 * i + lane];
                    o[i / 4][4 * (i % 4)] += x.x * fk, o[i / 4][4 * (i % 4) + 1] += x.y * fk;
                    o[i / 4][4 * (i % 4) + 2] += x.z * fk, o[i / 4][4 * (i % 4) + 3] += x.w * fk;
                    if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // (few of them in registers at a time)
                }
            }
        }
        barrier_lds();
        if (wk > 0) return;
    }

    // A lane holds one row's output in pieces of 4 d; through LDS it leaves in whole rows
    // (each wave in a part of its own, so that only its own writes are waited for).
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;  // (a row that sees no key: zeros)
    uint8_t* const mine = lds + wq * 32 * ROW;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int n = 0; n < 4; ++n)
            *reinterpret_cast<uint2*>(mine + col * ROW + 16 * key_slot<CH>(col, 4 * dt + n) + 8 * half) =
                make_uint2(pack_bf16x2(o[dt][4 * n] * inv, o[dt][4 * n + 1] * inv),
                           pack_bf16x2(o[dt][4 * n + 2] * inv, o[dt][4 * n + 3] * inv));
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32 / PER; ++i) {
        const int r = i * PER + lane / CH, piece = lane % CH;
        const uint4 x = *reinterpret_cast<const uint4*>(mine + r * ROW + 16 * key_slot<CH>(r, piece));
        if (row0 + r < Lq && 8 * piece < D)
            *reinterpret_cast<uint4*>(a.o + (q0 + row0 + r) * a.o_token + head * a.o_head + 8 * piece) = x;
    }
}

// Blocks of query rows that a launch has for each head.
template <class SH>
int shape_blocks(const PrefillArgs& a) { return a.M / SH::BQ + a.seqs; }

enum class Blocks { few, large, small, wide };
// f(the shape) of a call's heads and blocks.
template <int DP, class F>
auto with_blocks(Blocks blocks, F f) {
    if (blocks == Blocks::few) return f(Shape<DP, 2, 2, DP <= 64 ? 64 : 32>{});
    if (blocks == Blocks::wide) return f(Shape<DP, 2, DP <= 128 ? 4 : 2, DP <= 64 ? 64 : 32>{});  // (larger ones do not fit LDS)
    if (blocks == Blocks::small) return f(Shape<DP, 2, 1, 32>{});
    return f(Shape<DP, 4, 1, DP <= 128 ? 64 : 32>{});
}
template <class F>
auto with_shape(int head_dim, Blocks blocks, F f) {
    if (head_dim <= 64) return with_blocks<64>(blocks, f);
    if (head_dim <= 96) return with_blocks<96>(blocks, f);
    if (head_dim <= 128) return with_blocks<128>(blocks, f);
    if (head_dim <= 192) return with_blocks<192>(blocks, f);
    return with_blocks<256>(blocks, f);
}

}  // namespace

hipError_t launch_attn_prefill(const PrefillArgs& a, const DeviceInfo& dev, hipStream_t stream) {
    const int forced = hooks().attn_prefill.load(std::memory_order_relaxed);
    // Few rows: as long as its workgroups are about one to a CU (graph-replayed, us, rows / blocks of 64 / of 128:
    // 28 heads on 4 of 128, 128 rows 6.6 / 8.2 / 8.4, 256 rows 11.1 / 9.7 / 10.5; 16 heads of 64, 256 rows 6.4 /
    // 7.1 / 7.9, 384 rows 9.3 / 7.9 / 9.4; 8 heads on 1 of 256, 512 rows 13.6 / 18.1 / 23.4, 1024 rows 28.0 / 26.6 /
    // 38.4; 16 heads on 2 of 256 with 8 sequences of 64 rows 16.8 / 11.6 at two to a CU).  Blocks of 64 rows with the
    // keys shared by two groups of waves: where blocks of 128 would be fewer than three to two CUs (28 on 4 of
    // 128, 1024 rows 20.2 / 23.2, 2048 rows 46.3 / 46.2, 4096 rows 149 / 129; 40 on 8 of 128, 1024 rows 24.2 / 25.0;
    // 16 heads of 64, 2048 rows 21.7 / 29.5, 8192 rows 177 / 175; 8 on 1 of 256, 4096 rows 92 / 128, 8192 rows 324 /
    // 289).
    // Long keys move both bounds, since a block then passes over them in as many more steps: few rows up to seven
    // workgroups to four CUs (one head of 128, 6466 rows 43 / 78; 4 on 2 of 64, 1700 rows 15.1 / 16.0, but 2000 rows, just
    // past that, 18.5 / 17.8), and four groups of waves instead of two where a CU has one block of 64 rows at
    // most, or two of the longest (four / two groups: 7 heads on 1 of 80, 1500 rows 17.1 / 19.3; 2 heads of 128, 8000
    // rows 71.7 / 94.5; 7 on 1 of 96, 3500 rows 34.1 / 44.0; 8 on 1 of 128, 4000 rows 50.7 / 54.9, 10000 rows 257 / 241;
    // but 28 on 4 of 128, 512 rows 14.0 / 12.9, 1024 rows 27.7 / 21.7).
    const int64_t groups = attn_rows_groups(a), blocks = (int64_t(a.M) / kPrefillRows + a.seqs) * a.q_heads;
    const int64_t blocks_64 = (int64_t(a.M) / 64 + a.seqs) * a.q_heads, cus = dev.cus;
    const bool long_keys = a.M_k >= 1024 && a.M_k >= 512 * int64_t(a.seqs), longest = a.M_k >= 2048 * int64_t(a.seqs);
    if (forced < 0 ? 8 * groups <= 9 * cus || (long_keys && 4 * groups <= 7 * cus) : forced == 0)
        return launch_attn_rows(a, dev, stream);
    // Blocks of 64 rows and two waves, four of which share a CU: where the sequences have few keys, so that a
    // block's first loads and its output are most of its time (small / 128, 28 heads on 4 of 128: 64 sequences of 16
    // rows 12.7 / 22.0, 64 of 64 24.7 / 29.3, 16 of 256 26.0 / 28.2, 12 of 384 33.6 / 35.5, 8 of 512 36.5 / 36.2, 16 of
    // 64 on 1064 keys 47.0 / 42.0; 16 of 384, 8 heads on 1 of 256 34.1 / 39.8, 16 heads of 64 17.3 / 22.6, 32 on 8 of
    // 80 37.9 / 37.1).
    const bool short_keys = a.M_k <= 384 * int64_t(a.seqs);
    const bool wide = long_keys && blocks_64 <= (longest ? 2 : 1) * cus;
    const Blocks shape = forced > 0               ? Blocks(forced - 1)
                         : wide                   ? Blocks::wide
                         : 2 * blocks < 3 * cus   ? Blocks::few
                         : short_keys             ? Blocks::small
                                                  : Blocks::large;
    with_shape(a.head_dim, shape, [&](auto of) {
        using SH = decltype(of);
        const int blocks = shape_blocks<SH>(a);
        hipLaunchKernelGGL((attn_prefill_kernel<SH>), dim3(uint32_t(blocks) * uint32_t(a.q_heads)), dim3(SH::THREADS), 0, stream,
                           a, blocks);
    });
    return hipGetLastError();
}

int64_t attn_prefill_threads(const PrefillArgs& a, int kernel) {
    if (kernel == 0) return attn_rows_threads(a);
    return with_shape(a.head_dim, Blocks(kernel - 1), [&](auto of) {
        using SH = decltype(of);
        return int64_t(shape_blocks<SH>(a)) * a.q_heads * SH::THREADS;
    });
}

}  // namespace fq
