// rotary_plan.cpp -- the host side of rotary positions: a head's frequencies,
// scaled for long contexts, and their fixed-point form (gbattn_rotary.h).
#include <math.h>
#include <algorithm>

#include "../../include/gbattn_rotary.h"

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

}  // namespace

extern "C" {

gbattn_status attn_rotary_frequencies(int rot_dim, double base, gbattn_rotary_scaling scaling, double factor, double low,
                                      double high, double length, double* inv_freq, double* gain) {
    if (!inv_freq || !gain || rot_dim < 2 || rot_dim % 2 != 0) return GBATTN_ERR_INVALID_ARG;
    if (!isfinite(base) || base <= 1.0) return GBATTN_ERR_INVALID_ARG;
    if (scaling < GBATTN_ROTARY_PLAIN || scaling > GBATTN_ROTARY_YARN) return GBATTN_ERR_UNSUPPORTED;
    const bool parts = scaling == GBATTN_ROTARY_BY_PARTS || scaling == GBATTN_ROTARY_YARN;
    if (scaling != GBATTN_ROTARY_PLAIN && (!isfinite(factor) || factor < 1.0)) return GBATTN_ERR_INVALID_ARG;
    if (parts && !(isfinite(low) && isfinite(high) && isfinite(length) && low > 0.0 && high > low && length > 0.0))
        return GBATTN_ERR_INVALID_ARG;
    if (scaling == GBATTN_ROTARY_NTK) {
        if (rot_dim == 2) return GBATTN_ERR_INVALID_ARG;
        base *= pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
        if (!isfinite(base)) return GBATTN_ERR_INVALID_ARG;
    }
    // YARN: the pairs between which g falls
    double from = 0.0, to = 0.0;
    if (scaling == GBATTN_ROTARY_YARN) {
        auto pair_of = [&](double turns) { return rot_dim * log(length / (kTwoPi * turns)) / (2.0 * log(base)); };
        from = std::min(std::max(floor(pair_of(high)), 0.0), rot_dim - 1.0);
        to = std::min(std::max(ceil(pair_of(low)), 0.0), rot_dim - 1.0);
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = pow(base, -2.0 * i / rot_dim);
        double g = scaling == GBATTN_ROTARY_LINEAR ? 0.0 : 1.0;
        if (scaling == GBATTN_ROTARY_BY_PARTS) g = (length * f / kTwoPi - low) / (high - low);
        if (scaling == GBATTN_ROTARY_YARN) g = 1.0 - (i - from) / std::max(to - from, 0.001);
        g = std::min(std::max(g, 0.0), 1.0);
        inv_freq[i] = g < 1.0 ? g * f + (1.0 - g) * f / factor : f;
    }
    *gain = scaling == GBATTN_ROTARY_YARN ? 0.1 * log(factor) + 1.0 : 1.0;
    return GBATTN_OK;
}

gbattn_status attn_rotary_steps(const double* inv_freq, int n, uint64_t* steps) {
    if (n < 0 || (n > 0 && (!inv_freq || !steps))) return GBATTN_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (!isfinite(inv_freq[i])) return GBATTN_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        // |turns| < 1 with the frequency's sign; scaled by 2^64 it is an integer or rounded to one.  A negative
        // one is its magnitude's negation modulo 2^64.
        const double turns = fabs(inv_freq[i]) / kTwoPi;
        const double part = nearbyint(ldexp(turns - floor(turns), 64));
        const uint64_t s = part >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(part);
        steps[i] = inv_freq[i] < 0.0 ? 0 - s : s;
    }
    return GBATTN_OK;
}

}  // extern "C"
