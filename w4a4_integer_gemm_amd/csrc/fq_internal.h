// Internal interfaces between the C ABI layer (fq_api.cpp) and the kernel
// translation units.  Not installed; the public surface is include/fq.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <string>

namespace fq {

// Thread-local error message shared by every entry point.
void set_error(const std::string& msg);
void clear_error();

struct PrologueArgs {
    const uint16_t* x;
    int32_t M, K;
    int64_t ldx;
    const float* gamma;   // nullptr: no RMSNorm
    float eps;
    const float* ascale;  // nullptr: no explicit smoothing
    int32_t fold_after;
    int32_t hblock;
    int32_t abits;
    uint8_t* codes;
    float* act_scale;
};

struct GemmArgs {
    const uint8_t* act;   // [M][K*abits/8]
    const float* act_scale;
    int32_t M, abits;
    const uint8_t* w;     // [N][K*wbits/8]
    const float* wscale;
    int32_t N, K, wbits;
    const float* bias;        // nullptr: none
    const uint16_t* residual; // nullptr: none
    int64_t ldr;
    uint16_t* y;
    int64_t ldy;
    int32_t* acc;             // nullptr: not written
    int32_t head_dim;         // 0: y is [M][ldy]; else y is [N/head_dim][M][head_dim]
};

// Address of output (m, n) (n a multiple of 4 inside one head when head_dim > 0).
__host__ __device__ inline uint16_t* out_ptr(const GemmArgs& g, int m, int n) {
    if (g.head_dim > 0) {
        const int h = n / g.head_dim;
        return g.y + (int64_t(h) * g.M + m) * g.head_dim + (n - h * g.head_dim);
    }
    return g.y + int64_t(m) * g.ldy + n;
}

// Forced kernel choices for the tests (fq_test_hook, or the FQ_TEST_HOOK
// environment variable read once, at the first use).  The launch paths read
// these with relaxed atomic loads; nothing on them calls getenv.
struct Hooks {
    std::atomic<int> gemm_tile{-1};  // -1: the cost model picks; else a tile id of fq_gemm.hip
    std::atomic<int> gemm_mfma{16};  // 16: v_mfma_i32_16x16x64_i8 where it applies; 32: 32x32x32 only
    std::atomic<int> gemv_split{0};  // 1: decode-sized M always takes the split-K GEMV
    std::atomic<int> fp8_tile{-1};   // -1: the rule of fq_fp8_gemm.hip picks; else one of its tile ids
    std::atomic<int> attn_prefill{-1};  // -1: by size; 0: few rows; 1: blocks of 64 rows, 2: of 128, 3: of 64 rows of short sequences, 4: of 64 with more waves
    std::atomic<int> decode1_off{0}; // 1: one-token fq_linear as two launches, never the fused kernel
};
Hooks& hooks();
// Tile id of a tile name ("128x144", ...), or -1 (fq_gemm.hip).
int gemm_tile_id(const char* name);
// The same for the FP8 GEMM (fq_fp8_gemm.hip).
int fp8_tile_id(const char* name);

// What a device's launches need to know, gathered once per device and process
// by prepare_device (fq_api.cpp): the compute-unit count, the LDS of a CU and,
// per streaming-GEMV kernel (bit mix x token tiles), how many of its
// workgroups the register file lets a CU hold.  The same set-up raises those
// kernels' dynamic-LDS limit, so no launch makes a HIP call other than the
// launch itself.
constexpr int kMaxDevices = 64;
struct DeviceInfo {
    int device;
    int cus;
    int lds_per_cu;
    int stream_regs_wg[4][2];  // [bit mix: 8/8, 4/4, 8/4, 4/8][token tiles - 1]
    void* scratch;             // this device's copy of the allocation-free workspace
};

// Size of the device array that fq_linear_noalloc uses as its workspace (the
// activation codes and scales, laid out as fq_linear's workspace).
constexpr size_t kNoallocScratchBytes = size_t(24) << 20;
// Set-up of the current device (once); *info points at its record.
hipError_t prepare_device(const DeviceInfo** info);
// The streaming GEMV's part of that set-up (fq_gemv.hip).
hipError_t init_gemv_device(DeviceInfo& d);
// The address of this device's scratch array (fq_noalloc.hip).
hipError_t init_scratch_device(DeviceInfo& d);

// Enqueue the kernels; they return hipGetLastError() of the launch.  Shapes
// are validated by the caller; a launch makes no other HIP call.
hipError_t launch_prologue(const PrologueArgs& a, hipStream_t stream);
hipError_t launch_gemm(const GemmArgs& a, hipStream_t stream);
// The FP6 kernel for E2M3 codes (abits = wbits = 6), every M.
hipError_t launch_gemm_e2m3(const GemmArgs& g, hipStream_t stream);
hipError_t launch_gemv(const GemmArgs& a, const DeviceInfo& dev, hipStream_t stream);
// One-token fq_linear in one launch (fq_decode1.hip): whether the shape takes
// it, and the launch (prologue arguments and GEMM arguments of the same call).
bool decode1_eligible(const PrologueArgs& p, const GemmArgs& g);
hipError_t launch_decode1(const PrologueArgs& p, const GemmArgs& g, hipStream_t stream);
// Rows of the block norms and of the FP8 prologue (fq_block_norm.hip):
//   r' = r + res_scale * gate * norm(x; post_gamma)   (only with x)
//   h  = norm(r'; pre_gamma) * (1 + mod_scale) + mod_shift
// h leaves as bf16 rows, as e4m3 codes with their scales, or both.
struct NormArgs {
    int32_t M, K;
    const uint16_t* x;  // nullptr: the stream is taken as it is
    int64_t ldx;
    const float* post_gamma;  // nullptr: x is added without a norm
    float post_eps;
    const uint16_t* gate;  // nullptr: 1
    int64_t ld_gate;
    float res_scale;
    const void* r_in;  // bf16, or float32 with stream_f32
    int64_t ld_rin;
    void* r_out;  // nullptr: not written
    int64_t ld_rout;
    int32_t stream_f32;
    int32_t pre_norm;        // 0: h = r_in (the FP8 prologue of a quant-only site: no x, modulation or h)
    const float* pre_gamma;  // nullptr: unit gain
    float pre_eps;
    const uint16_t* mod_scale;  // nullptr: 0
    const uint16_t* mod_shift;  // nullptr: 0
    int64_t ld_mod;
    int32_t rows_per_cond;
    uint16_t* h;  // nullptr: not written
    int64_t ld_h;
    uint8_t* codes;    // nullptr: not written
    float* act_scale;  // [K / 128][fp8_scale_ld(M)]
};
// Pieces of 8 values per lane (1, 2, 4 or 8) and threads of a row's workgroup.  Many
// rows are bound by the instructions of their waves, half of which are the row's
// sums and scales, once per wave: two pieces per lane halve those (us, two / one:
// 4096 x 3584 to codes 13.0 / 15.3, with post norm and stream 24.5 / 26.6, 4096 x
// 8192 29.2 / 35.0; 1024 x 3584 and 1024 x 2048 within 0.2 of each other).  Rows
// of a float32 stream wait for memory instead (12800 x 2048 gated: 64.4 / 60.6).
inline int block_norm_pieces(int32_t K, int32_t M, bool f32) {
    if (K > 8192) return K <= 16384 ? 2 : K <= 32768 ? 4 : 8;
    return !f32 && K >= 1024 && int64_t(M) * K >= 1 << 22 ? 2 : 1;
}
inline int block_norm_threads(int32_t K, int32_t M, bool f32) {
    const int P = block_norm_pieces(K, M, f32);
    return ((K / 8 + P - 1) / P + 63) / 64 * 64;
}
hipError_t launch_block_norm(const NormArgs& a, hipStream_t stream);

// FP8 sites: row stride of an activation scale matrix [K / 128][ld] in floats
// (16-byte aligned rows), and the GEMM's arguments.
__host__ __device__ inline int32_t fp8_scale_ld(int32_t M) { return (M + 3) / 4 * 4; }
struct Fp8Args {
    const uint8_t* act;      // e4m3 [M][K]
    const float* act_scale;  // [K / 128][fp8_scale_ld(M)]
    int32_t M;
    const uint8_t* w;     // e4m3 [N][K]
    const float* wscale;  // [ceil(N / 128)][K / 128]
    int32_t N, K;
    const float* bias;         // nullptr: none
    const uint16_t* residual;  // nullptr: none
    int64_t ldr;
    uint16_t* y;
    int64_t ldy;
    int32_t head_dim;  // 0: y is [M][ldy]; else y is [N/head_dim][M][head_dim]
};
hipError_t launch_fp8_gemm(const Fp8Args& g, const DeviceInfo& dev, hipStream_t stream);
// K in parts (fq_fp8_linear's workspace has room for kSplitTiles partial tiles of
// 128 x 128 floats where fp8_may_split): how many and on which tiles (1: whole), and
// the two launches.
constexpr int kSplitTiles = 256, kSplitEdge = 128;
struct Fp8Split {
    int splits, edge;
};
// (shorter K gained nothing: K = N = 3584 with 64 tokens 13.9 us in parts, 14.0 whole)
inline bool fp8_may_split(int32_t M, int32_t K) { return M > 1 && K >= 4096; }
Fp8Split fp8_split(const Fp8Args& g, const DeviceInfo& dev);
hipError_t launch_fp8_split(const Fp8Args& g, Fp8Split how, float* part, hipStream_t stream);
// Tokens of a GEMV workgroup: 16, or 32, which share its weights; 0 where it takes no
// call.  More than 32 tokens need workgroups for all of them at once.
inline int fp8_gemv_tokens(int32_t M, int32_t N, int cus) {
    const int64_t groups = (int64_t(N) + 15) / 16;
    if (M <= 16 || groups * ((M + 15) / 16) <= cus) return 16;
    return M <= 32 || groups * ((M + 31) / 32) <= cus ? 32 : 0;
}
bool fp8_gemv_takes(const Fp8Args& g, const DeviceInfo& dev);
hipError_t launch_fp8_gemv(const Fp8Args& g, const DeviceInfo& dev, hipStream_t stream);
// A few tokens with their prologue in one launch (fq_fp8_decode.hip), and whether it takes a call.
bool fp8_decode_takes(const NormArgs& p, const Fp8Args& g);
hipError_t launch_fp8_decode(const NormArgs& p, const Fp8Args& g, const DeviceInfo& dev, hipStream_t stream);
// The same from codes.
bool fp8_decode_codes_takes(const Fp8Args& g);
hipError_t launch_fp8_decode_codes(const Fp8Args& g, hipStream_t stream);

// Rotary positions (fq_rope.hip).
struct RopeArgs {
    const uint16_t* x;
    int64_t x_token, x_head;
    int32_t M, heads, rot_heads, head_dim, rot_dim, interleaved;
    const uint64_t* freq;  // [rot_dim / 2] turns per position, fraction of a turn in 2^-64
    float attn_scale;
    const int32_t* positions;  // nullptr: pos0 + m
    int32_t pos0;
    int32_t inverse;
    uint16_t* y;
    int64_t y_token, y_head;
};
hipError_t launch_rope(const RopeArgs& a, hipStream_t stream);

// Norm of query and key heads with their rotation (fq_qk_norm.hip).
struct QkNormArgs {
    const uint16_t* x;
    int64_t x_token, x_head;
    int32_t M, heads, q_heads, k_heads, head_dim;
    const float *q_gamma, *k_gamma;  // nullptr: unit gain
    float eps;
    int32_t rot_dim, interleaved;  // rot_dim 0: no rotation
    const uint64_t* freq;
    float attn_scale;
    const int32_t* positions;  // nullptr: pos0 + m
    int32_t pos0;
    uint16_t* y;
    int64_t y_token, y_head;
};
hipError_t launch_qk_norm(const QkNormArgs& a, hipStream_t stream);

// The paged cache, and the tokens written to it or read from it (fq_kv_cache.hip).
struct KvCache {
    void *k, *v;                // bf16 or e4m3 [pages][kv_heads][page_size][head_dim]
    float *k_scale, *v_scale;   // [pages][kv_heads][page_size]; nullptr: bf16
    int32_t pages, page_size, kv_heads, head_dim;
};
struct KvRows {
    uint16_t* p;  // (read only by a write into the cache)
    int64_t token, head;
};
hipError_t launch_kv_write(const KvCache& c, const KvRows& k, const KvRows& v, const int32_t* slots, int32_t M,
                           hipStream_t stream);
hipError_t launch_kv_read(const KvCache& c, const KvRows& k, const KvRows& v, const int32_t* slots, int32_t M,
                          hipStream_t stream);

// Attention of packed prompts (fq_attn_prefill.hip).
struct PrefillArgs {
    const uint16_t* q;
    int64_t q_token, q_head;
    const uint16_t* k;
    int64_t k_token, k_head;
    const uint16_t* v;
    int64_t v_token, v_head;
    int32_t M, M_k;
    const int32_t *cu_q, *cu_k;
    int32_t seqs, q_heads, kv_heads, head_dim;
    float scale;
    int32_t causal;
    uint16_t* o;
    int64_t o_token, o_head;
};
// Query rows of the largest block.  A call has fewer than 2^23 blocks of them (the entry point's check), hence
// fewer than 2^24 of 64 rows: of the kernels that the rule picks whatever the size, the one of 128 rows has 256
// threads to a block and the one of 64 for short sequences 128, fewer than 2^31 in all; the others are picked
// where there are a few workgroups to a CU at most.  A forced kernel's launch is checked by itself.
constexpr int kPrefillRows = 128;
hipError_t launch_attn_prefill(const PrefillArgs& a, const DeviceInfo& dev, hipStream_t stream);
// Threads of a launch on one of its kernels (numbered as in Hooks::attn_prefill).
int64_t attn_prefill_threads(const PrefillArgs& a, int kernel);
// The same for few rows (fq_attn_rows.hip), its workgroups and its threads.
int64_t attn_rows_groups(const PrefillArgs& a);
int64_t attn_rows_threads(const PrefillArgs& a);
hipError_t launch_attn_rows(const PrefillArgs& a, const DeviceInfo& dev, hipStream_t stream);

// Attention of one token per sequence over the paged cache (fq_attn_decode.hip).
struct DecodeArgs {
    const uint16_t* q;
    int64_t q_token, q_head;
    int32_t seqs, q_heads;
    float scale;
    KvCache cache;
    const int32_t* page_table;
    int32_t max_pages;
    const int32_t* lens;
    uint16_t* o;
    int64_t o_token, o_head;
    int2* plan;    // [seqs] first part and parts of each; [seqs]: parts of the batch, tokens of one
    float2* stats; // [parts][q_heads] maximum and sum of weights
    float* sums;   // [parts][q_heads][head_dim]
    int32_t parts; // (at most)
};
hipError_t launch_attn_decode(const DecodeArgs& a, hipStream_t stream);

hipError_t launch_geglu(const uint16_t* gu, int32_t M, int32_t F, int64_t ld_in, uint16_t* h, int64_t ld_out,
                        hipStream_t stream);

// Largest M that the GEMV kernel takes.
constexpr int32_t kGemvMaxM = 32;

}  // namespace fq
