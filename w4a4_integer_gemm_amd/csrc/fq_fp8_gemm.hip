// FP8 GEMM with block scales on gfx950:
//   y[m][n] = bf16_rne(sum_g sa[g][m] sw[n / 128][g] sum_{k in g} qa[m][k] qw[n][k] [+ bias[n]] [+ residual[m][n]])
// g running over the groups of 128 consecutive k, e4m3 codes on
// v_mfma_f32_16x16x128_f8f6f4.
//
// One instruction covers one scale group exactly: it multiplies 16 weight
// rows by 16 tokens over 128 k from a zero accumulator, and the four results a
// lane holds (four rows of one 128-row block, one token) are added to the
// float32 sums with one fma each, scaled by sa * sw (one product per lane,
// token fragment and stage).
//
// Tile BM tokens x BN weight rows, one k stage = 128 codes of every row.  Four
// load waves copy a stage into an LDS ring slot with global_load_lds_dwordx4;
// four MFMA waves split the tile 2 x 2.  A row's 16-byte chunk c sits at slot
// 8 row + (c ^ ((row / 2) % 8)), so the 16 lanes of an LDS read phase (16
// consecutive rows, one chunk) take 16 distinct groups of four banks.
//
// Ring protocol (barrier B(s) ends MFMA iteration s; B(-1) precedes it):
//   - an MFMA wave reads stage 0 after B(-1) and stage s + 1 during iteration
//     s, and waits for those reads before B(s): after B(s) the slots of
//     stages <= s + 1 are free;
//   - the load waves first fill the slots of stages 0 .. NS-2; at iteration s
//     a load wave refills slot (s - 1) mod NS (free since B(s - 1); at s = 0
//     the slot still empty) with stage s + NS - 1, waits until stage s + 2 has
//     landed, and reaches B(s), which publishes it for iteration s + 1's reads.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "fq_device.h"
#include "fq_fp8_tile.h"
#include "fq_internal.h"
#include "fq_ring.h"

namespace fq {
namespace {

constexpr int kThreads = 512;  // 4 load waves + 4 MFMA waves
constexpr int kLdsMax = 160 * 1024;

template <int BM_, int BN_>
struct Fp8Cfg {
    static constexpr int BM = BM_, BN = BN_;
    static constexpr int STAGE = (BM + BN) * 128;
    static constexpr int COPIES = STAGE / 1024;  // 1 KB copies of 8 rows
    static constexpr int NHI = COPIES / 4;       // per load wave
    static constexpr int NS = kLdsMax / STAGE > 8 ? 8 : kLdsMax / STAGE;
    static constexpr int LDS = NS * STAGE;
    static constexpr int TF = BM / 32;  // token fragments per MFMA wave
    static constexpr int TW = BN / 32;  // weight fragments per MFMA wave
    static_assert(BM % 32 == 0 && BN % 32 == 0, "whole fragments per wave");
    static_assert(COPIES % 4 == 0, "the load waves' shares are equal");
    static_assert(BN / 2 <= 128 && 128 % (BN / 2) == 0, "a wave's rows stay in one scale block");
    static_assert(NS >= 4, "the ring needs four stages");
    static_assert((NS - 2) * NHI < 64, "vmcnt range");
};

template <class CF>
__global__ __launch_bounds__(kThreads) void fp8_gemm_kernel(Fp8Args g, int tiles_m, int tiles_n) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[CF::LDS];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // XCD-aware tile order: dispatch b runs on XCD b % 8, which takes the tile
    // range [x per, (x + 1) per), m fastest
    const int ntiles = tiles_m * tiles_n;
    int t = blockIdx.x;
    if (ntiles % 8 == 0) t = (blockIdx.x % 8) * (ntiles / 8) + blockIdx.x / 8;
    const int m0 = (t % tiles_m) * CF::BM, n0 = (t / tiles_m) * CF::BN;
    const int64_t ld = g.K;
    const int nk = g.K / 128;

    if (wave >= 4) {
        // copy q = p + 4 i of a stage is rows 8 q .. 8 q + 7 (tokens first):
        // lane l fills the slot of row 8 q + l / 8 and chunk (l % 8) ^ swizzle
        const int p = wave - 4;
        uint32_t voff[CF::NHI];
#pragma unroll
        for (int i = 0; i < CF::NHI; ++i) {
            const int q = p + 4 * i;
            const int rho = 8 * q + (lane >> 3);
            const int c = (lane & 7) ^ fp8_swizzle(rho);
            const bool act = 8 * q < CF::BM;
            int row = act ? m0 + rho : n0 + rho - CF::BM;
            const int last = act ? g.M - 1 : g.N - 1;
            row = row < last ? row : last;
            voff[i] = uint32_t(int64_t(row - (act ? m0 : n0)) * ld + 16 * c);
        }
        const uint8_t* const abase = g.act + int64_t(m0) * ld;
        const uint8_t* const wbase = g.w + int64_t(n0) * ld;
        const uint32_t lds0 = lds_address(lds);
        auto load_stage = [&](int j) {
            const int src = j < nk ? j : nk - 1;  // stages past K repeat the last one (never read)
            const uint32_t dst = lds0 + uint32_t((j % CF::NS) * CF::STAGE);
#pragma unroll
            for (int i = 0; i < CF::NHI; ++i) {
                const int q = p + 4 * i;
                copy16_to_lds((8 * q < CF::BM ? abase : wbase) + int64_t(src) * 128, voff[i], dst + q * 1024);
            }
        };
        for (int j = 0; j < CF::NS - 1; ++j) load_stage(j);
        int issued = CF::NS - 1;
        wait_vmcnt<(CF::NS - 3) * CF::NHI>();  // stages 0 and 1 landed
        barrier_nofence();                      // B(-1)
        for (int s = 0; s < nk; ++s) {
            if (s + CF::NS - 1 < nk) {
                load_stage(s + CF::NS - 1);
                ++issued;
            }
            const int younger = issued - (s + 3);  // copies issued after stage s + 2
            wait_stages_in_flight<CF::NHI>(younger > 0 ? younger : 0);
            barrier_nofence();  // B(s)
        }
        return;
    }

    constexpr int TF = CF::TF, TW = CF::TW;
    const int wm = wave & 1, wn = wave >> 1;
    const int q = lane >> 4;
    uint32_t oa[TF], ow[TW];
#pragma unroll
    for (int f = 0; f < TF; ++f) oa[f] = fp8_slot(wm * (CF::BM / 2) + 16 * f + (lane & 15), q);
#pragma unroll
    for (int n = 0; n < TW; ++n) ow[n] = fp8_slot(CF::BM + wn * (CF::BN / 2) + 16 * n + (lane & 15), q);
    v4f acc[TW][TF];
#pragma unroll
    for (int n = 0; n < TW; ++n)
#pragma unroll
        for (int f = 0; f < TF; ++f) acc[n][f] = v4f{0.f, 0.f, 0.f, 0.f};
    v8i fa[2][TF], fw[2][TW];
    float sa[2][TF], sw[2];
    const uint32_t lds0 = lds_address(lds);
    // scales of stage s: this lane's tokens, and the wave's block of 128 rows
    const int lda = fp8_scale_ld(g.M);
    int mrow[TF];
#pragma unroll
    for (int f = 0; f < TF; ++f) {
        const int m = m0 + wm * (CF::BM / 2) + 16 * f + (lane & 15);
        mrow[f] = m < g.M ? m : g.M - 1;
    }
    const int nrow = n0 + wn * (CF::BN / 2);
    const float* const swp = g.wscale + int64_t((nrow < g.N ? nrow : g.N - 1) / 128) * nk;
    auto read_stage = [&](int s, int b) {
        const uint32_t base = lds0 + uint32_t((s % CF::NS) * CF::STAGE);
        const int sc = s < nk ? s : nk - 1;
#pragma unroll
        for (int f = 0; f < TF; ++f) sa[b][f] = g.act_scale[int64_t(sc) * lda + mrow[f]];
        sw[b] = swp[sc];
#pragma unroll
        for (int f = 0; f < TF; ++f) fa[b][f] = fp8_read_frag(base + oa[f]);
#pragma unroll
        for (int n = 0; n < TW; ++n) fw[b][n] = fp8_read_frag(base + ow[n]);
    };
    auto iteration = [&](int s, auto b_tag) {
        constexpr int B = decltype(b_tag)::value;
        read_stage(s + 1, B ^ 1);  // (past K: a slot's stale bytes, never used)
        float p[TF];
#pragma unroll
        for (int f = 0; f < TF; ++f) p[f] = sa[B][f] * sw[B];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < TW; ++n)
#pragma unroll
            for (int f = 0; f < TF; ++f) {
                const v4f d = mfma_e4m3(fw[B][n], fa[B][f], v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][f][i] = __builtin_fmaf(d[i], p[f], acc[n][f][i]);
            }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): stage s + 1 is in registers
        barrier_nofence();                   // B(s)
    };
    barrier_nofence();  // B(-1): stages 0 and 1 published
    read_stage(0, 0);
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_sched_barrier(0);
    int s = 0;
    for (; s + 1 < nk; s += 2) {  // stages in pairs, so that the register set of each is fixed
        iteration(s, std::integral_constant<int, 0>{});
        iteration(s + 1, std::integral_constant<int, 1>{});
    }
    if (s < nk) iteration(s, std::integral_constant<int, 0>{});

    int mm[TF], nn[TW];
#pragma unroll
    for (int f = 0; f < TF; ++f) mm[f] = m0 + wm * (CF::BM / 2) + 16 * f + (lane & 15);
#pragma unroll
    for (int n = 0; n < TW; ++n) nn[n] = n0 + wn * (CF::BN / 2) + 16 * n + 4 * q;
    fp8_store_tiles<TW, TF>(acc, mm, nn, g);
}

template <class CF>
hipError_t launch_cfg(const Fp8Args& g, hipStream_t st) {
    const int tiles_m = (g.M + CF::BM - 1) / CF::BM;
    const int tiles_n = (g.N + CF::BN - 1) / CF::BN;
    hipLaunchKernelGGL((fp8_gemm_kernel<CF>), dim3(tiles_m * tiles_n), dim3(kThreads), 0, st, g, tiles_m, tiles_n);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8Args& g, hipStream_t stream) { return launch_cfg<Fp8Cfg<128, 128>>(g, stream); }

}  // namespace fq
