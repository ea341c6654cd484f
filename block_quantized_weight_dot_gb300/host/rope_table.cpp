// rope_table.cpp -- rotary frequencies and their whole-number form
// (lean_rope_frequencies, lean_rope_turns).  Host code.
#include <algorithm>
#include <cmath>

#include "../../include/lean_step.h"

namespace {
const double kTwoPi = 6.28318530717958647692;
}

extern "C" lean_status lean_rope_turns(const double *freq, int64_t n, uint64_t *turns) {
    if (!freq || !turns) return LEAN_ERR_NULL;
    if (n <= 0) return LEAN_ERR_SHAPE;
    for (int64_t i = 0; i < n; ++i) {
        if (!std::isfinite(freq[i]) || freq[i] < 0) return LEAN_ERR_SHAPE;
        const double t = freq[i] / kTwoPi, part = t - std::floor(t);  // whole turns per position drop out
        // part < 1 has 53 bits, so the product is exact and below 2^64
        turns[i] = (uint64_t)std::ldexp(part, 64);
    }
    return LEAN_OK;
}

extern "C" lean_status lean_rope_frequencies(int kind, int64_t rot_dim, double base, double factor,
                                             double trained_len, double slow, double fast, double *freq) {
    if (kind < LEAN_ROPE_PLAIN || kind > LEAN_ROPE_BANDS) return LEAN_ERR_FORMAT;
    if (!freq) return LEAN_ERR_NULL;
    if (rot_dim <= 0 || rot_dim % 2 || rot_dim > 65536 || !std::isfinite(base) || !(base > 1) ||
        !std::isfinite(factor) || !(factor >= 1) || (kind == LEAN_ROPE_BASE && rot_dim <= 2))
        return LEAN_ERR_SHAPE;
    if ((kind == LEAN_ROPE_RAMP || kind == LEAN_ROPE_BANDS) &&
        (!std::isfinite(trained_len) || !(trained_len > 0) || !(slow > 0) || !std::isfinite(fast) || !(fast > slow)))
        return LEAN_ERR_SHAPE;
    const double d = (double)rot_dim;
    if (kind == LEAN_ROPE_BASE) base *= std::pow(factor, d / (d - 2));
    // index (not whole) of the pair that makes t turns within trained_len
    auto pair_of = [&](double t) { return d * std::log(trained_len / (kTwoPi * t)) / (2 * std::log(base)); };
    double lo = 0, hi = 0;
    if (kind == LEAN_ROPE_RAMP) {
        lo = std::max(0.0, std::floor(pair_of(fast)));
        hi = std::min(d - 1, std::ceil(pair_of(slow)));
    }
    for (int64_t i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * (double)i / d);
        double r = 0;  // share of the frequency that is divided by the factor
        if (kind == LEAN_ROPE_LINEAR) r = 1;
        if (kind == LEAN_ROPE_RAMP) r = std::min(1.0, std::max(0.0, ((double)i - lo) / std::max(hi - lo, 0.001)));
        if (kind == LEAN_ROPE_BANDS) {
            const double t = trained_len * f / kTwoPi;
            r = 1 - std::min(1.0, std::max(0.0, (t - slow) / (fast - slow)));
        }
        freq[i] = f * (1 - r + r / factor);
    }
    return LEAN_OK;
}
