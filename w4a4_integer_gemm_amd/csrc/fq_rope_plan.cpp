// Host plan of the rotary positions: turns per position of every pair, under
// the rules that stretch the positions of a longer context.
//
// Pair i of rot_dim / 2 turns by theta_i = base^(-2 i / rot_dim) radians per
// position.  A table entry is theta_i / (2 pi) turns as a 64-bit fraction (a
// whole turn = 2^64), from long double arithmetic (64-bit mantissa): off by
// a few 2^-64 turns, so an angle at position p is off by a few p 2^-64 turns.
#include <cmath>
#include <cstdint>

#include "../../include/fq.h"
#include "fq_check.h"
#include "fq_internal.h"

namespace {

constexpr long double kTwoPi = 6.283185307179586476925286766559005768L;

uint64_t fraction_of_turn(long double turns) {
    turns -= std::floor(turns);
    const long double v = std::floor(turns * 18446744073709551616.0L + 0.5L);
    return v >= 18446744073709551616.0L ? 0 : static_cast<uint64_t>(v);
}

}  // namespace

extern "C" fq_status fq_rope_freqs(int32_t rot_dim, double base, int32_t kind, double factor, int32_t trained_len,
                                   double low, double high, const float* pair_factors, uint64_t* freq_out,
                                   float* attn_scale_out) {
    fq::clear_error();
    const char* fn = "fq_rope_freqs";
    if (!freq_out || !attn_scale_out) return fail(FQ_ERR_ARG, "fq_rope_freqs: freq_out or attn_scale_out is NULL");
    if (rot_dim < 2 || rot_dim > 65536 || rot_dim % 2)
        return fail(FQ_ERR_SHAPE, fmt("%s: rot_dim=%d must be even and in [2, 65536]", fn, rot_dim));
    if (!(base > 1.0) || !std::isfinite(base)) return fail(FQ_ERR_ARG, fmt("%s: base=%g must be finite and > 1", fn, base));
    if (kind < FQ_ROPE_PLAIN || kind > FQ_ROPE_PAIRS)
        return fail(FQ_ERR_UNSUPPORTED, fmt("%s: kind=%d is not a scaling rule (0 .. %d)", fn, kind, FQ_ROPE_PAIRS));
    const bool scaled = kind == FQ_ROPE_LINEAR || kind == FQ_ROPE_BASE || kind == FQ_ROPE_BANDS || kind == FQ_ROPE_RAMP;
    if (scaled && !(factor >= 1.0 && std::isfinite(factor)))
        return fail(FQ_ERR_ARG, fmt("%s: factor=%g must be finite and >= 1", fn, factor));
    if (kind == FQ_ROPE_BASE && rot_dim < 4)
        return fail(FQ_ERR_SHAPE, fmt("%s: rot_dim=%d must be at least 4 for a changed base", fn, rot_dim));
    if (kind == FQ_ROPE_BANDS || kind == FQ_ROPE_RAMP) {
        if (trained_len < 1) return fail(FQ_ERR_ARG, fmt("%s: trained_len=%d must be >= 1", fn, trained_len));
        if (!(low > 0.0 && high > low && std::isfinite(high)))
            return fail(FQ_ERR_ARG, fmt("%s: low=%g and high=%g must satisfy 0 < low < high", fn, low, high));
    }
    const int32_t pairs = rot_dim / 2;
    if (kind == FQ_ROPE_PAIRS) {
        if (!pair_factors) return fail(FQ_ERR_ARG, "fq_rope_freqs: pair_factors is NULL");
        for (int32_t i = 0; i < pairs; ++i)
            if (!(pair_factors[i] > 0.0f) || !std::isfinite(pair_factors[i]))
                return fail(FQ_ERR_ARG, fmt("%s: pair_factors[%d]=%g must be finite and > 0", fn, i,
                                            double(pair_factors[i])));
    }

    long double b = base;
    if (kind == FQ_ROPE_BASE) b *= std::pow((long double)factor, (long double)rot_dim / (rot_dim - 2));
    double lo = 0.0, hi = 0.0;
    if (kind == FQ_ROPE_RAMP) {
        // the pair index at which a pair makes n turns over the trained length
        auto at = [&](double n) { return rot_dim * std::log(trained_len / (n * double(kTwoPi))) / (2.0 * std::log(base)); };
        lo = std::fmax(std::floor(at(high)), 0.0);
        hi = std::fmin(std::ceil(at(low)), rot_dim - 1.0);
    }
    for (int32_t i = 0; i < pairs; ++i) {
        long double th = std::pow(b, -2.0L * i / rot_dim);
        if (kind == FQ_ROPE_LINEAR) {
            th /= factor;
        } else if (kind == FQ_ROPE_BANDS) {
            const long double turns = trained_len * th / kTwoPi;  // over the trained length
            long double keep = (turns - low) / ((long double)high - low);
            keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
            th *= keep + (1 - keep) / factor;
        } else if (kind == FQ_ROPE_RAMP) {
            const double span = std::fmax(hi - lo, 0.001);
            const double ramp = std::fmin(std::fmax((i - lo) / span, 0.0), 1.0);
            th = th * (1 - (long double)ramp) + th / factor * ramp;
        } else if (kind == FQ_ROPE_PAIRS) {
            th /= pair_factors[i];
        }
        freq_out[i] = fraction_of_turn(th / kTwoPi);
    }
    *attn_scale_out = kind == FQ_ROPE_RAMP ? float(0.1 * std::log(factor) + 1.0) : 1.0f;
    return FQ_OK;
}
