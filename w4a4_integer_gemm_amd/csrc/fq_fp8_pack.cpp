// Host side of the FP8 sites: weight rows to e4m3 codes with one float32 scale
// for every block of 128 x 128, and back.
//
//   s = (float)(max|w| / 448) over the block, q = e4m3(w / s)
// computed in float64, codes rounded to nearest (ties to even) against the
// stored float32 scale and clamped to +-448; a block whose scale is zero has
// zero codes.  E4M3: sign, 4 exponent bits with bias 7, 3 mantissa bits,
// exponent 0 subnormal (multiples of 2^-9), no infinities, 0x7F / 0xFF NaN.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/fq.h"
#include "fq_check.h"
#include "fq_host_rows.h"
#include "fq_internal.h"

namespace {

constexpr int32_t kBlock = 128;

uint8_t e4m3_pattern(double v) {
    const uint8_t sign = std::signbit(v) ? 0x80 : 0;
    double a = std::fabs(v);
    if (a > 448.0) a = 448.0;
    int e = -6;  // exponent of the smallest normal number
    if (a >= 0x1p-6) e = std::ilogb(a);
    const long m = std::lrint(std::ldexp(a, 3 - e));  // 8ths of 2^e; ties to even
    // m < 8: subnormal.  8 <= m <= 15: normal; 16 carries into the exponent field.
    const int field = m < 8 ? int(m) : ((e + 7) << 3) + int(m) - 8;
    return uint8_t(sign | field);
}

double e4m3_number(uint8_t p) {
    const int e = (p >> 3) & 15, m = p & 7;
    if (e == 15 && m == 7) return std::nan("");
    const double a = e == 0 ? std::ldexp(double(m), -9) : std::ldexp(double(8 + m), e - 10);
    return (p & 0x80) ? -a : a;
}

fq_status check_site(const char* fn, int32_t N, int32_t K) {
    if (N < 1) return fail(FQ_ERR_SHAPE, fmt("%s: N=%d must be >= 1", fn, N));
    return check_k(fn, K, kGemmK);
}

int32_t blocks_of(int32_t N) { return N / kBlock + (N % kBlock != 0); }

}  // namespace

extern "C" {

size_t fq_fp8_wscale_count(int32_t N, int32_t K) {
    if (N < 1 || K < kBlock || K > kMaxK || K % kBlock) return 0;
    return size_t(blocks_of(N)) * size_t(K / kBlock);
}

fq_status fq_fp8_pack_weights(const float* W, int32_t N, int32_t K, void* codes_out, float* wscale_out) {
    fq::clear_error();
    const char* fn = "fq_fp8_pack_weights";
    if (!W || !codes_out || !wscale_out)
        return fail(FQ_ERR_ARG, "fq_fp8_pack_weights: W, codes_out or wscale_out is NULL");
    FQ_TRY(check_site(fn, N, K));
    std::atomic<int64_t> bad{-1};
    parallel_rows(N, [&](int32_t n0, int32_t n1) {
        for (int64_t i = int64_t(n0) * K; i < int64_t(n1) * K; ++i)
            if (!std::isfinite(W[i])) {
                bad.store(i);
                return;
            }
    });
    if (bad.load() >= 0)
        return fail(FQ_ERR_ARG, fmt("%s: W[%lld][%lld] is not finite", fn, (long long)(bad.load() / K),
                                    (long long)(bad.load() % K)));
    uint8_t* const codes = static_cast<uint8_t*>(codes_out);
    const int32_t nk = K / kBlock;
    parallel_rows(blocks_of(N), [&](int32_t b0, int32_t b1) {
        for (int32_t b = b0; b < b1; ++b) {
            const int64_t r0 = int64_t(b) * kBlock, r1 = r0 + kBlock < N ? r0 + kBlock : N;
            for (int32_t g = 0; g < nk; ++g) {
                float amax = 0.0f;
                for (int64_t n = r0; n < r1; ++n)
                    for (int32_t k = 0; k < kBlock; ++k)
                        amax = std::max(amax, std::fabs(W[n * K + int64_t(g) * kBlock + k]));
                const float s = static_cast<float>(double(amax) / 448.0);
                wscale_out[size_t(b) * nk + g] = s;
                for (int64_t n = r0; n < r1; ++n)
                    for (int32_t k = 0; k < kBlock; ++k) {
                        const int64_t i = n * K + int64_t(g) * kBlock + k;
                        codes[i] = s > 0.0f ? e4m3_pattern(double(W[i]) / double(s)) : 0;
                    }
            }
        }
    });
    return FQ_OK;
}

fq_status fq_fp8_dequant_rows(const void* codes, const float* wscale, int32_t N, int32_t K, float* W_out) {
    fq::clear_error();
    if (!codes || !wscale || !W_out)
        return fail(FQ_ERR_ARG, "fq_fp8_dequant_rows: codes, wscale or W_out is NULL");
    FQ_TRY(check_site("fq_fp8_dequant_rows", N, K));
    const uint8_t* const c = static_cast<const uint8_t*>(codes);
    const int32_t nk = K / kBlock;
    parallel_rows(N, [&](int32_t n0, int32_t n1) {
        double value[256];
        for (int i = 0; i < 256; ++i) value[i] = e4m3_number(uint8_t(i));
        for (int64_t n = n0; n < n1; ++n)
            for (int32_t k = 0; k < K; ++k)
                W_out[n * K + k] =
                    static_cast<float>(double(wscale[(n / kBlock) * nk + k / kBlock]) * value[c[n * K + k]]);
    });
    return FQ_OK;
}

}  // extern "C"
