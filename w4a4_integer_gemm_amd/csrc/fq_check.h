// Argument checks shared by the entry points' translation units: messages,
// status returns and the rules every call has in common.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>

#include "../../include/fq.h"
#include "fq_internal.h"

namespace {

inline std::string fmt(const char* f, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, f);
    vsnprintf(buf, sizeof(buf), f, ap);
    va_end(ap);
    return std::string(buf);
}

inline fq_status fail(fq_status s, const std::string& msg) {
    fq::set_error(msg);
    return s;
}

inline bool is_pow2(int64_t v) { return v >= 1 && (v & (v - 1)) == 0; }
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

constexpr int32_t kMaxK = 65536;
constexpr int32_t kProloguePack = 32;  // 32 bf16 values per prologue lane
constexpr int32_t kGemmK = 128;        // one k stage of the GEMM

// Checks shared by the prologue, the GEMM and the packer.  Returns FQ_OK or the failure.
inline fq_status check_bits(const char* fn, const char* name, int32_t bits) {
    if (bits != 8 && bits != 4 && bits != FQ_CODES_E2M3)
        return fail(FQ_ERR_UNSUPPORTED,
                    fmt("%s: %s=%d is not a supported code width (4, 8, or 6 for E2M3)", fn, name, bits));
    return FQ_OK;
}

// K bounds; `mult` is the granularity the entry point needs (32 for the
// prologue, whose lanes hold up to 32 values each below K = 32768; 128 for the
// GEMM's k stages and the groups of the FP8 codes; 8 for the block norms).
inline fq_status check_k(const char* fn, int32_t K, int32_t mult) {
    if (K < mult || K > kMaxK)
        return fail(FQ_ERR_SHAPE, fmt("%s: K=%d outside [%d, %d]", fn, K, mult, kMaxK));
    if (K % mult)
        return fail(FQ_ERR_SHAPE, fmt("%s: K=%d is not a multiple of %d (%d/%d = %.2f)", fn, K, mult, K, mult,
                                      double(K) / mult));
    return FQ_OK;
}

inline fq_status check_hblock(const char* fn, int32_t K, int32_t hblock) {
    if (!is_pow2(hblock) || hblock > 256)
        return fail(FQ_ERR_SHAPE, fmt("%s: hblock=%d must be a power of two in [1, 256]", fn, hblock));
    if (K % hblock)
        return fail(FQ_ERR_SHAPE, fmt("%s: K=%d not divisible by hblock=%d (%d/%d = %.2f)", fn, K, hblock,
                                      K, hblock, double(K) / hblock));
    return FQ_OK;
}

inline fq_status device_status(const char* fn, hipError_t e) {
    if (e != hipSuccess) return fail(FQ_ERR_DEVICE, fmt("%s: %s", fn, hipGetErrorString(e)));
    return FQ_OK;
}

// The device set-up every device entry point runs before it queues anything.
inline fq_status prepare(const char* fn, const fq::DeviceInfo** info) {
    return device_status(fn, fq::prepare_device(info));
}

}  // namespace

#define FQ_TRY(expr)                     \
    do {                                 \
        fq_status _s = (expr);           \
        if (_s != FQ_OK) return _s;      \
    } while (0)
