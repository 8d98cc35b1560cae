// FP8 GEMM with block scales on gfx950:
//   y[m][n] = bf16_rne(sum_g sa[g][m] sw[n / 128][g] sum_{k in g} qa[m][k] qw[n][k] [+ bias[n]] [+ residual[m][n]])
// g running over the groups of 128 consecutive k, e4m3 codes on
// v_mfma_f32_16x16x128_f8f6f4.
//
// One instruction covers one scale group exactly: it multiplies 16 weight
// rows by 16 tokens over 128 k from a zero accumulator, and the four results a
// lane holds (four rows of one 128-row block, one token) are added to the
// float32 sums with one fma each, scaled by sa * sw.
//
// A k stage is the 128 codes of the tile's BM tokens and BN weight rows, the
// tokens' BM scales and the scales of the weight rows' blocks; NS stages live in
// LDS, copied there without passing through registers.  A stage's 16-byte chunk
// c of row rho sits at slot 8 rho + (c ^ ((rho / 2) % 8)), so the 16 lanes of an
// LDS read phase (16 consecutive rows, one chunk) take 16 distinct groups of
// four banks.
//
// A multiplying wave holds its TW weight fragments of a stage in registers and
// runs through its TF token fragments, reading each one step ahead; the sums of
// a step are scaled and added between the next step's products.  Before the
// products of a stage's last step its LDS reads have returned: the barrier there
// frees the stage's slot and publishes the next stage, whose first fragments
// are read behind the last step's products.  Copies run NS - 1 stages ahead,
// from four waves that do nothing else, or, on the largest tile, from the first
// four of the eight multiplying waves (one per SIMD: while one waits to issue a
// copy the other wave of its SIMD multiplies).
//
// Workgroups are persistent: as many as fit the chip, each running through its
// tiles with the copies going on into the next tile, so that only a tile's
// epilogue interrupts the products.
//
// Measured (4096 x 3584 x 37888, 256 x 256 tiles): 530 to 570 us by card, 2000 to
// 2100 TFLOP/s, against 890 us for the first version, whose stages waited for their scales from
// global memory.  What bounds it is power and the copies: without copies the same
// loop takes 430 us, and the clock falls to 1.6 GHz from 2.4 with both.  A
// prefetch of later stages into L2 (one dword of each line) made it slower
// (594 us; shared among the workgroups of an XCD 563).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

#include "fq_device.h"
#include "fq_fp8_tile.h"
#include "fq_internal.h"
#include "fq_ring.h"

namespace fq {
namespace {

template <int BM_, int BN_, int WM_, int WN_, int LW_, int OCC_, int NS_>
struct Fp8Cfg {
    static constexpr int BM = BM_, BN = BN_;  // tokens and weight rows of a tile
    static constexpr int WM = WM_, WN = WN_;  // waves along each
    static constexpr int OCC = OCC_;          // waves of a SIMD that share the registers
    static constexpr int NS = NS_;            // stages in LDS
    static constexpr int LW = LW_;            // waves that only copy (0: the multiplying waves copy)
    static constexpr int MW = WM * WN, WAVES = MW + LW, THREADS = 64 * WAVES;
    static constexpr int WGS = OCC * 4 / WAVES;                 // workgroups per CU
    static constexpr int TF = BM / WM / 16, TW = BN / WN / 16;  // fragments of a wave
    static constexpr int COPIES = (BM + BN) / 8;                // 1 KB copies of 8 rows
    static constexpr int CW = LW ? LW : MW == 8 ? 4 : MW;       // waves that copy: one per SIMD
    static constexpr int NC = (COPIES + CW - 1) / CW;           // per copying wave
    static constexpr bool EVEN = (BM / 8) % CW == 0 && COPIES % CW == 0;  // every copying wave's first BM / 8 / CW are tokens
    static constexpr int SA_OFF = (BM + BN) * 128;              // the tokens' scales (one 1 KB copy)
    static constexpr int SW_OFF = SA_OFF + 1024;                // the row blocks' scales (one 256-byte copy)
    static constexpr int STAGE = SW_OFF + 256;
    static constexpr int LDS = NS * STAGE;
    static constexpr bool ALIGNED = BN % 128 == 0 && 128 % (16 * TW) == 0;  // a wave's rows share one scale block
    static constexpr int UNITS = (TF - 1) * TW;                 // products before a stage's last step
    static constexpr int SPREAD = UNITS / 4 > 0 ? UNITS / 4 : 1;  // those with copies behind them
    static constexpr int NP = ALIGNED ? 1 : TW;                            // scale products per token fragment
    static_assert(BM % (16 * WM) == 0 && BN % (16 * WN) == 0, "whole fragments per wave");
    static_assert(BM <= 256, "one copy holds the tokens' scales");
    static_assert(TF % 2 == 0, "the two token registers alternate from stage to stage");
    static_assert(CW >= 2 && CW % 2 == 0 && WGS >= 1, "two waves copy the scales; a wave's rows share their swizzle");
    static_assert(LDS * WGS <= 160 * 1024, "LDS of a CU");
    // With copying waves and four stages a barrier publishes the stage after the
    // next, so that the next one's first fragments are read without waiting for it.
    static constexpr bool EARLY = LW > 0 && NS >= 4;
    static constexpr int FLIGHT = EARLY ? NS - 3 : NS - 2;  // newest stages that may be in flight at a barrier
    static_assert(FLIGHT >= 0 && FLIGHT * (NC + 1) < 64, "slots of the ring; vmcnt range");
};

// Copies global -> LDS, lane l's bytes landing at lds_dst + 16 l or + 4 l, in
// inline asm for the reason given at copy16_to_lds (no VGPR result).  The five
// wait states cover scalar operands that a vector instruction has just written
// (v_readfirstlane, or v_readlane of a spilled register), which the compiler
// does not see being read by a memory instruction here, and the M0 write.
//
// 16 bytes from a buffer descriptor at voff + soff; a lane whose voff lies past
// the descriptor's end reads zero (soff need not be part of that check).
__device__ __forceinline__ void copy16_buffer(const v4i& rsrc, uint32_t voff, uint32_t soff, uint32_t lds_dst) {
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds_dst)
                 : "memory");
}
// 16 or 4 bytes from base + voff.
__device__ __forceinline__ void copy16_base(const uint8_t* base, uint32_t voff, uint32_t lds_dst) {
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(voff), "s"(base), "{m0}"(lds_dst) : "memory");
}
__device__ __forceinline__ void copy4_base(const uint8_t* base, uint32_t voff, uint32_t lds_dst) {
    asm volatile("s_nop 4\n\tglobal_load_lds_dword %0, %1" : : "v"(voff), "s"(base), "{m0}"(lds_dst) : "memory");
}

// Descriptor of `bytes` bytes at p (wave uniform): base, no stride, size, raw 32-bit data.
__device__ __forceinline__ v4i buffer_of(const uint8_t* p, uint32_t bytes) {
    const uint64_t u = reinterpret_cast<uintptr_t>(p);
    return v4i{__builtin_amdgcn_readfirstlane(int(u)), __builtin_amdgcn_readfirstlane(int(u >> 32)),
               __builtin_amdgcn_readfirstlane(int(bytes)), 0x00020000};
}

typedef __attribute__((address_space(3))) const float lds_cfloat;
__device__ __forceinline__ float lds_float(uint32_t addr) { return *reinterpret_cast<lds_cfloat*>(uintptr_t(addr)); }

// SPLIT: each of `splits` parts of K (a divisor of its units) makes tiles of its
// own, whose float32 sums go to part[split][M][N] instead of the epilogue.
template <class CF, bool SPLIT>
__global__ __launch_bounds__(CF::THREADS) __attribute__((amdgpu_waves_per_eu(CF::OCC, CF::OCC))) void fp8_gemm_kernel(
    Fp8Args g, int tiles_m, int tiles_n, int group_m, int splits, float* part) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[CF::LDS];
    constexpr int TF = CF::TF, TW = CF::TW, NC = CF::NC, NS = CF::NS, NP = CF::NP;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cw = CF::LW ? wave - CF::MW : wave;  // copying wave (0 .. CW - 1), or none
    const int q = lane >> 4;
    const int nu = g.K / 128, nk = SPLIT ? nu / splits : nu;
    const int lda = fp8_scale_ld(g.M);
    const uint32_t lds0 = lds_address(lds);

    // This workgroup's tiles: dispatch b runs on XCD b % 8, each XCD takes a
    // contiguous range of tiles, and its workgroups go through that range side
    // by side.
    const int tiles = tiles_m * tiles_n, ntiles = SPLIT ? tiles * splits : tiles;
    const int x = blockIdx.x % 8, rem = ntiles % 8;
    const int on_xcd = (int(gridDim.x) - x + 7) / 8;  // workgroups of this XCD
    const int first = x * (ntiles / 8) + (x < rem ? x : rem), count = ntiles / 8 + (x < rem ? 1 : 0);
    const int j0 = blockIdx.x / 8;
    const int mine = j0 < count ? (count - j0 + on_xcd - 1) / on_xcd : 0;
    // Tiles are ordered in groups of group_m tiles of tokens, m fastest, so that
    // those in flight on an XCD share operand rows in its L2.
    auto origin = [&](int i, int& m0, int& n0) {  // returns the part of K
        const int item = first + j0 + i * on_xcd;
        const int split = SPLIT ? item / tiles : 0, t = SPLIT ? item - split * tiles : item;
        const int gsize = group_m * tiles_n;
        const int gi = t / gsize, r = t - gi * gsize;
        const int left = tiles_m - gi * group_m;
        const int gm = left < group_m ? left : group_m;
        m0 = (gi * group_m + r % gm) * CF::BM;
        n0 = (r / gm) * CF::BN;
        return split;
    };

    // The copy side, up to NS stages ahead of the products: copy i of a wave is
    // rows 8 c .. 8 c + 7 of the stage (tokens first), c = cw + CW i; lane l
    // fills the slot of row 8 c + l / 8, chunk (l % 8) ^ swizzle (the same for
    // every c: the swizzle has period 16 rows, a wave's copies are 8 CW apart).
    // Rows past M or N read as zeros (their results are not stored).
    const uint32_t copy_lane = fp8_copy_lane(lane, cw & 1, g.K);
    uint32_t sc_off = 0;
    v4i ra{}, rw{};
    const uint8_t* psc = nullptr;
    const int64_t sc_step = cw == 0 ? 4 * int64_t(lda) : 4;  // bytes from one stage's scales to the next's
    int copy_tile = 0, copy_s = 0, copy_u0 = 0;  // (u0: the part's first unit)
    uint32_t copy_dst = lds0;
    auto chunk = [&](int i) {
        const int c = cw + CF::CW * i;
        return CF::EVEN || c < CF::COPIES ? c : c - CF::CW;  // (past the end: the wave's copy before, again)
    };
    auto aim = [&](int tile) {
        int m0, n0;
        copy_u0 = origin(tile, m0, n0) * nk;
        const int rows_a = g.M - m0 < CF::BM ? g.M - m0 : CF::BM, rows_w = g.N - n0 < CF::BN ? g.N - n0 : CF::BN;
        ra = buffer_of(g.act + int64_t(m0) * g.K, uint32_t(rows_a) * uint32_t(g.K));
        rw = buffer_of(g.w + int64_t(n0) * g.K, uint32_t(rows_w) * uint32_t(g.K));
        if (cw == 0) {  // four tokens' scales per lane; the last whole four past the end
            int m = m0 + 4 * (lane < CF::BM / 4 ? lane : 0);
            m = m < lda - 4 ? m : lda - 4;
            sc_off = uint32_t(4 * (m - m0));
            psc = reinterpret_cast<const uint8_t*>(g.act_scale + int64_t(copy_u0) * lda + m0);
        } else if (cw == 1) {  // one row block's scale per lane
            const int blk0 = n0 / 128, blk_last = (g.N - 1) / 128;
            const int blk = blk0 + lane < blk_last ? blk0 + lane : blk_last;
            sc_off = uint32_t(4 * (blk - blk0) * nu);
            psc = reinterpret_cast<const uint8_t*>(g.wscale + int64_t(blk0) * nu + copy_u0);
        }
    };
    auto copy_part = [&](int i) {
        const int c = chunk(i);
        const bool act = CF::EVEN ? i < CF::BM / 8 / CF::CW : 8 * c < CF::BM;
        const Fp8CopyOffset at = fp8_copy_at(copy_lane, 8 * c - (act ? 0 : CF::BM), (SPLIT ? copy_u0 : 0) + copy_s, g.K);
        copy16_buffer(act ? ra : rw, at.lane, at.common, copy_dst + c * 1024);
    };
    auto copy_scales = [&]() {
        if (cw == 0)
            copy16_base(psc, sc_off, copy_dst + CF::SA_OFF);
        else if (cw == 1)
            copy4_base(psc, sc_off, copy_dst + CF::SW_OFF);
    };
    // To the next stage.  Past the last one the copies go on with descriptors of
    // no bytes and the last scales, into slots that nobody reads any more: every
    // stage has the same copies, without a branch between its products (a branch
    // around each copy cost 20 % of a stage's time even where no copy was made).
    auto copy_advance = [&]() {
        copy_dst = copy_dst + CF::STAGE == lds0 + CF::LDS ? lds0 : copy_dst + CF::STAGE;
        if (copy_tile == mine) return;
        if (++copy_s < nk) {
            psc += sc_step;
            return;
        }
        copy_s = 0;
        if (++copy_tile < mine) {
            aim(copy_tile);
        } else {
            ra[2] = 0;
            rw[2] = 0;
            copy_u0 = 0;  // (the wave's offset is zero too: no lane is in range of no bytes)
        }
    };
    // Waits until all but the newest k stages of this wave's copies have landed
    // (they return in order).
    auto wait_but = [&](auto k_tag) {
        constexpr int k = decltype(k_tag)::value;
        if (cw < 0) return;
        if (k == 0 || cw < 2)
            wait_vmcnt<k * (NC + 1)>();
        else if (cw < CF::CW)
            wait_vmcnt<k * NC>();
    };
    if (mine == 0) return;
    if (cw >= 0 && cw < CF::CW) aim(0);
    auto copy_stage = [&]() {
        if (cw < 0 || cw >= CF::CW) return;
        copy_scales();
#pragma unroll
        for (int i = 0; i < NC; ++i) copy_part(i);
        copy_advance();
    };
    for (int s = 0; s < NS - 1; ++s) copy_stage();
    wait_but(std::integral_constant<int, CF::FLIGHT>{});
    barrier_nofence();
    if (CF::LW && cw >= 0) {
        for (int i = mine * nk; i > 0; --i) {
            copy_stage();
            wait_but(std::integral_constant<int, CF::FLIGHT>{});
            barrier_nofence();
        }
        wait_vmcnt<0>();  // no copy outlives its workgroup's LDS
        return;
    }

    const int wm = wave % CF::WM, wn = wave / CF::WM;
    const int arow = wm * 16 * TF, wrow = wn * 16 * TW;
    // fragment j of an operand is 2048 j bytes further (the swizzle has period 16)
    const uint32_t oa = fp8_slot(arow + (lane & 15), q), ow = fp8_slot(CF::BM + wrow + (lane & 15), q);
    uint32_t ra0 = lds0 + oa, ra1 = lds0 + (oa ^ 64u), rw0 = lds0 + ow, rw1 = lds0 + (ow ^ 64u);
    const uint32_t osa = CF::SA_OFF + 4 * (arow + (lane & 15));

    v4f acc[TW][TF];
    v8i fa[2], fw[TW];
    v4f d[2][TW];
    float sa[TF], sw[NP], p[2][NP];
    uint32_t osw[NP];  // each weight fragment's scale block, from the tile's first
    auto add = [&](int f, int n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][f][i] = __builtin_fmaf(d[f & 1][n][i], p[f & 1][NP == 1 ? 0 : n], acc[n][f][i]);
        // (pinned here: left alone the compiler sinks the adds behind the stage's
        // branches, with every product of the stage live until then)
        asm volatile("" : "+v"(acc[n][f]));
    };
    auto products = [&](int f) {
#pragma unroll
        for (int n = 0; n < NP; ++n) p[f & 1][n] = sa[f] * sw[n];
    };
    auto read_scales = [&](uint32_t base) {
#pragma unroll
        for (int f = 0; f < TF; ++f) sa[f] = lds_float(base + osa + 64 * f);
#pragma unroll
        for (int n = 0; n < NP; ++n) sw[n] = lds_float(base + osw[n]);
    };

    uint32_t cur = lds0, nxt = lds0 + CF::STAGE;
    // One stage; COPY: with the copies of the stage NS - 1 further, one by one
    // behind the first products.
    auto stage = [&](auto copy_tag) {
        constexpr bool COPY = decltype(copy_tag)::value;
        if constexpr (COPY) copy_scales();
        // One product and the four adds of an earlier one in turn: the adds
        // then fit between the products' issue slots (clustered by the
        // scheduler, products and adds took 82 % of this order's rate).  The
        // copies of stage s + NS - 1, whose slot the last barrier freed, go
        // out one by one between the first products.
#pragma unroll
        for (int f = 0; f < TF - 1; ++f) {
            fa[(f + 1) & 1] = fp8_read_frag(ra0 + 2048 * (f + 1), ra1 + 2048 * (f + 1));
            products(f);
#pragma unroll
            for (int n = 0; n < TW; ++n) {
                d[f & 1][n] = mfma_e4m3(fw[n], fa[f & 1], v4f{0.f, 0.f, 0.f, 0.f});
                __builtin_amdgcn_sched_barrier(0);
                add((f + TF - 1) % TF, n);
                const int unit = f * TW + n;
                if constexpr (COPY) {
#pragma unroll
                    for (int i = 0; i < NC; ++i)
                        if (i * CF::SPREAD / NC == unit) copy_part(i);
                }
                __builtin_amdgcn_sched_barrier(0);
                if (COPY && unit == CF::SPREAD - 1) copy_advance();
            }
        }
        constexpr int L = TF - 1;
        products(L);
        if constexpr (!CF::EARLY) {
            // this wave's reads of stage s (and copies of stage s + 1) are done
            __builtin_amdgcn_s_waitcnt(0xC07F);
            if constexpr (CF::LW == 0) wait_but(std::integral_constant<int, CF::FLIGHT>{});
            barrier_nofence();
        }
        ra0 += nxt - cur;
        ra1 += nxt - cur;
        rw0 += nxt - cur;
        rw1 += nxt - cur;
        read_scales(nxt);
        fa[0] = fp8_read_frag(ra0, ra1);  // (past the last stage: a slot's stale bytes, never used)
#pragma unroll
        for (int n = 0; n < TW; ++n) {
            d[L & 1][n] = mfma_e4m3(fw[n], fa[L & 1], v4f{0.f, 0.f, 0.f, 0.f});
            fw[n] = fp8_read_frag(rw0 + 2048 * n, rw1 + 2048 * n);
            __builtin_amdgcn_sched_barrier(0);
            add(L - 1, n);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (CF::EARLY) barrier_nofence();  // (the products above have waited for every read of stage s)
        cur = nxt;
        nxt = nxt + CF::STAGE == lds0 + CF::LDS ? lds0 : nxt + CF::STAGE;
    };

    auto run = [&](auto copy_tag) {
        for (int tile = 0; tile < mine; ++tile) {
            int m0, n0;
            const int split = origin(tile, m0, n0);
#pragma unroll
            for (int n = 0; n < NP; ++n)
                osw[n] = CF::SW_OFF + 4 * (CF::ALIGNED ? wrow / 128 : (n0 + wrow + 16 * n) / 128 - n0 / 128);
            if (CF::ALIGNED ? tile == 0 : true) read_scales(cur);
            if (tile == 0) {
                fa[0] = fp8_read_frag(ra0, ra1);
#pragma unroll
                for (int n = 0; n < TW; ++n) fw[n] = fp8_read_frag(rw0 + 2048 * n, rw1 + 2048 * n);
            }
#pragma unroll
            for (int n = 0; n < TW; ++n) {
#pragma unroll
                for (int f = 0; f < TF; ++f) acc[n][f] = v4f{0.f, 0.f, 0.f, 0.f};
                d[1][n] = v4f{0.f, 0.f, 0.f, 0.f};  // no pending sums
            }
#pragma unroll
            for (int n = 0; n < NP; ++n) p[1][n] = 0.0f;

            for (int s = 0; s < nk; ++s) stage(copy_tag);
#pragma unroll
            for (int n = 0; n < TW; ++n) add(TF - 1, n);
            if constexpr (SPLIT)
                fp8_store_part<TW, TF>(acc, m0 + arow, n0 + wrow, lane, g, part + int64_t(split) * g.M * g.N);
            else
                fp8_store_tile<TW, TF>(acc, m0 + arow, n0 + wrow, lane, g);
        }
    };
    if (CF::LW == 0 && (CF::CW == CF::MW || wave < CF::CW))
        run(std::true_type{});
    else
        run(std::false_type{});
    wait_vmcnt<0>();  // no copy outlives its workgroup's LDS
}

template <class CF>
hipError_t launch_cfg(const Fp8Args& g, const DeviceInfo& dev, hipStream_t st) {
    const int tiles_m = (g.M + CF::BM - 1) / CF::BM;
    const int tiles_n = (g.N + CF::BN - 1) / CF::BN;
    const int slots = dev.cus * CF::WGS, tiles = tiles_m * tiles_n;
    hipLaunchKernelGGL((fp8_gemm_kernel<CF, false>), dim3(tiles < slots ? tiles : slots), dim3(CF::THREADS), 0, st, g,
                       tiles_m, tiles_n, 8, 1, nullptr);
    return hipGetLastError();
}

// Joins the parts of K in their order and runs the epilogue: a thread for 4
// features of one token, A parts requested at once (eight parts of 23 x 2048
// outputs: 3.1 us; one after the other 3.9).
template <int A>
__global__ __launch_bounds__(256) void fp8_join_kernel(Fp8Args g, int splits, const float* part) {
    const int per_row = g.N / 4, i = blockIdx.x * 256 + threadIdx.x;
    if (i >= g.M * per_row) return;
    const int m = i / per_row, n = 4 * (i - m * per_row);
    const float* const p = part + int64_t(m) * g.N + n;
    const int64_t step = int64_t(g.M) * g.N;
    float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
    uint2 res = make_uint2(0, 0);
    if (g.bias) bias = *reinterpret_cast<const float4*>(g.bias + n);
    if (g.residual) res = *reinterpret_cast<const uint2*>(g.residual + int64_t(m) * g.ldr + n);
    v4f s = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < splits; k0 += A) {
        v4f v[A];
#pragma unroll
        for (int k = 0; k < A; ++k) {  // (past the last part: the last again, not added)
            const int at = k0 + k < splits ? k0 + k : splits - 1;
            v[k] = *reinterpret_cast<const v4f*>(p + at * step);
        }
#pragma unroll
        for (int k = 0; k < A; ++k)
            if (k0 + k < splits) s = k0 + k == 0 ? v[0] : s + v[k];
    }
    if (g.bias) s += v4f{bias.x, bias.y, bias.z, bias.w};
    if (g.residual) s += v4f{bf16_lo(res.x), bf16_hi(res.x), bf16_lo(res.y), bf16_hi(res.y)};
    *reinterpret_cast<uint2*>(fp8_out_ptr(g, m, n)) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
}

struct Tile {
    const char* name;
    int bm, bn;
    float stage_us;  // one stage of one tile alone on a CU
    hipError_t (*launch)(const Fp8Args&, const DeviceInfo&, hipStream_t);
};
template <int BM, int BN, int WM, int WN, int LW, int NS>
constexpr Tile tile(const char* name, float stage_us) {
    return {name, BM, BN, stage_us, launch_cfg<Fp8Cfg<BM, BN, WM, WN, LW, 2, NS>>};
}
constexpr float kStage64 = 0.25f, kStage128 = 0.37f;
// The largest tile copies the fewest bytes per product and multiplies on eight
// waves, half of which copy between their products: with two waves of 256
// registers on a SIMD there is no room for waves that only copy.  The others
// multiply on four waves and copy on four more (128 x 128 this way: 0.38 us a
// stage, 0.61 with its multiplying waves copying).
const Tile kTiles[] = {
    tile<256, 256, 2, 4, 0, 2>("256x256", 1.15f), tile<256, 128, 2, 2, 4, 3>("256x128", 0.59f),
    tile<128, 192, 2, 2, 4, 3>("128x192", 0.52f), tile<128, 160, 2, 2, 4, 4>("128x160", 0.46f),
    tile<128, 128, 2, 2, 4, 4>("128x128", kStage128), tile<128, 96, 2, 2, 4, 5>("128x96", 0.35f),
    tile<128, 64, 2, 2, 4, 6>("128x64", 0.29f),   tile<64, 128, 2, 2, 4, 6>("64x128", 0.32f),
    tile<64, 64, 2, 2, 4, 8>("64x64", kStage64),
};
constexpr int kTileCount = int(sizeof kTiles / sizeof kTiles[0]);
constexpr float kTileUs = 2.0f;  // a tile's epilogue and first loads

// The tile with the least time by rounds of tiles over the CUs, and that time.
// Measured (us, the chosen one first): 1024 x 3584 x 4608: 128x160 22.7, 128x192
// 23.9, 256x128 27.2, 128x128 30.3; 811 x 16384 x 2048: 128x64 45.7, 64x128 46.1,
// 128x96 50.7, 256x256 165; 4096 x 3584 x 37888: 256x256 530, 256x128 538, 128x128
// 740.  Tiles of 32 tokens were no faster than those of 64 at 32 tokens.
//
// The stage times are of a tile alone: with every CU copying a 128 x 128 stage takes
// 0.5 us, and the estimate of a large product is mostly 15 to 40 % below its time
// (1024 x 3584 x 4608: 17.7, measured 22.3; 200 x 3584 x 37888: 32.6, measured 48).
// The order among the tiles holds; against the other paths' estimates below, taken
// from whole calls, it leans to the product in one piece.
struct Pick {
    int tile;
    float us;
};
Pick pick_tile(const Fp8Args& g, int cus) {
    Pick best{0, 0.0f};
    for (int i = 0; i < kTileCount; ++i) {
        const Tile& t = kTiles[i];
        const int64_t tiles = int64_t((g.M + t.bm - 1) / t.bm) * ((g.N + t.bn - 1) / t.bn);
        const float us = float((tiles + cus - 1) / cus) * (float(g.K / 128) * t.stage_us + kTileUs);
        if (i == 0 || us < best.us) best = Pick{i, us};
    }
    return best;
}

}  // namespace

int fp8_tile_id(const char* name) {
    for (int i = 0; i < kTileCount; ++i)
        if (!std::strcmp(kTiles[i].name, name)) return i;
    return -1;
}

// Estimates (us) that choose between the GEMV, the GEMM and the GEMM with K in
// parts.  All stream the weights, at 5.1 TB/s; the GEMV reads the codes again from
// L2 for every 16 weight rows (8 TB/s in all, less where workgroups are fewer than
// CUs); the GEMM takes its rounds of tiles; parts of K are written, read and joined by a launch more.
namespace {
constexpr float kCopyRate = 5.1f, kReadRate = 8.0f;  // MB per us

float weights_us(const Fp8Args& g) { return float(g.N) * float(g.K) * 1e-6f / kCopyRate; }
float larger(float a, float b) { return a > b ? a : b; }

float gemv_us(const Fp8Args& g, const DeviceInfo& dev) {  // (of a call that it takes)
    const int tokens = fp8_gemv_tokens(g.M, g.N, dev.cus);
    const int groups = (g.N + 15) / 16 * ((g.M + tokens - 1) / tokens), read = g.M < tokens ? g.M : tokens;
    const float fill = groups < dev.cus ? float(groups) / float(dev.cus) : 1.0f;
    const float bytes = float(groups) * float(16 + read) * float(g.K) * 1e-6f;
    return 2.5f + larger(bytes / (kReadRate * fill), weights_us(g));
}
float gemm_us(const Fp8Args& g, const DeviceInfo& dev) {
    return 2.8f + larger(pick_tile(g, dev.cus).us, weights_us(g));
}
// K in parts on tiles of `edge` squared: as many parts as the CUs take at once,
// each of at least 8 units, all alike, so that every workgroup has as many stages.
// (A number of units with few divisors gets fewer parts than would fit: 64 tokens of
// N = 2048 take 15.7 us at K = 16384, in 8 parts, 20.8 at 11008, in 2, 25.4 at 13696,
// whole.  Tiles for more than half of the CUs are not cut: 811 x 18944 x 3584 77 us.)
int parts_of(const Fp8Args& g, const DeviceInfo& dev, int edge) {
    const int cus = dev.cus < kSplitTiles ? dev.cus : kSplitTiles, nu = g.K / 128;
    const int64_t tiles = int64_t((g.M + edge - 1) / edge) * ((g.N + edge - 1) / edge);
    if (2 * tiles > cus) return 1;
    int splits = int(cus / tiles) < nu / 8 ? int(cus / tiles) : nu / 8;
    while (splits > 1 && nu % splits) --splits;
    return splits;
}
float split_us(const Fp8Args& g, int splits, int edge) {
    const float stage_us = edge == 64 ? kStage64 : kStage128, fixed = edge == 64 ? 6.5f : 9.0f;
    const float parts = 8e-6f * float(splits) * float(g.M) * float(g.N);  // (written and read)
    return fixed + larger(float(g.K / 128 / splits) * stage_us, weights_us(g)) + parts / kCopyRate;
}
}  // namespace

// Measured (us, GEMV / GEMM):
//   K = 3584, N = 37888: 26.9 / 28.0 with 4 tokens, 36.9 / 28.0 with 16, 50.5 / 28.1 with 32
//   K = 3584, N = 4608: 8.8 / 11.0 with 16, 12.0 / 11.1 with 32
//   K = 8192, N = 8192: 18.7 / 22.0 with 16, 25.7 / 23.9 with 32
//   K = 16384, N = 2048: 16.8 / 35.2 with 16, 16.7 / 35.4 with 32
//   K = 1024, N = 16384: 5.6 / 6.5 with 8, 8.4 / 6.8 with 32
//   K = 3584, N = 1024: 5.4 / 10.9 with 64, 7.1 / 10.9 with 128
bool fp8_gemv_takes(const Fp8Args& g, const DeviceInfo& dev) {
    if (!fp8_gemv_tokens(g.M, g.N, dev.cus) || hooks().fp8_tile.load(std::memory_order_relaxed) >= 0) return false;
    return gemv_us(g, dev) <= gemm_us(g, dev);
}

// Measured (us of fq_fp8_linear, in parts / whole): K = 16384, N = 2048: 13.5 / 16.7
// with 8 tokens, 15.3 / 40.3 with 64, 23.4 / 42.1 with 256; K = 18944, N = 3584: 21.2
// / 25.3 with 16, 26.8 / 55.0 with 64, 41.5 / 56.4 with 256; K = 32768, N = 1024: 60.4
// / 86.8 with 811; K = 4096, N = 1024: 11.3 / 14.3 with 64, 14.9 / 16.1 with 256, and
// whole 8.1 with 16, where parts took 11.
Fp8Split fp8_split(const Fp8Args& g, const DeviceInfo& dev) {
    if (hooks().fp8_tile.load(std::memory_order_relaxed) >= 0 || !fp8_may_split(g.M, g.K)) return Fp8Split{1, 0};
    Fp8Split best{1, 0};
    float least = gemm_us(g, dev);
    if (fp8_gemv_tokens(g.M, g.N, dev.cus) && gemv_us(g, dev) < least) least = gemv_us(g, dev);
    for (int edge = 64; edge <= 128; edge += 64) {
        const int splits = parts_of(g, dev, edge);
        const float us = split_us(g, splits, edge);
        if (splits > 1 && us < least) best = Fp8Split{splits, edge}, least = us;
    }
    return best;
}

namespace {
template <class CF>
hipError_t launch_parts(const Fp8Args& g, int splits, float* part, hipStream_t st) {
    const int tiles_m = (g.M + CF::BM - 1) / CF::BM, tiles_n = (g.N + CF::BN - 1) / CF::BN;
    hipLaunchKernelGGL((fp8_gemm_kernel<CF, true>), dim3(tiles_m * tiles_n * splits), dim3(CF::THREADS), 0, st, g,
                       tiles_m, tiles_n, 8, splits, part);
    return hipGetLastError();
}
}  // namespace

hipError_t launch_fp8_split(const Fp8Args& g, Fp8Split how, float* part, hipStream_t stream) {
    const hipError_t e = how.edge == 64 ? launch_parts<Fp8Cfg<64, 64, 2, 2, 4, 2, 8>>(g, how.splits, part, stream)
                                        : launch_parts<Fp8Cfg<128, 128, 2, 2, 4, 2, 4>>(g, how.splits, part, stream);
    if (e != hipSuccess) return e;
    const dim3 grid((g.M * (g.N / 4) + 255) / 256), block(256);
    if (how.splits <= 2)
        hipLaunchKernelGGL(fp8_join_kernel<2>, grid, block, 0, stream, g, how.splits, part);
    else if (how.splits <= 4)
        hipLaunchKernelGGL(fp8_join_kernel<4>, grid, block, 0, stream, g, how.splits, part);
    else
        hipLaunchKernelGGL(fp8_join_kernel<8>, grid, block, 0, stream, g, how.splits, part);
    return hipGetLastError();
}

hipError_t launch_fp8_gemm(const Fp8Args& g, const DeviceInfo& dev, hipStream_t stream) {
    const int forced = hooks().fp8_tile.load(std::memory_order_relaxed);
    return kTiles[forced >= 0 ? forced : pick_tile(g, dev.cus).tile].launch(g, dev, stream);
}

}  // namespace fq
