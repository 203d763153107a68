// rope_table.h -- the frequencies of a rope description as 64-bit fractions of a turn per
// position (host code).
//
// A position multiplies the entry's error, and 2^31 of them turn one double's 2^-53 into an
// angle that fp32 can see (2.8e-7 radians).  So frequencies are sums of two doubles, some 100 bits, and an
// entry is off by its own rounding alone, half a unit of 2^-64 turns.
#pragma once

#include <math.h>
#include <stdint.h>

#include "splash.h"

namespace splash {

// hi + lo, |lo| at most half a unit in hi's last place.
struct TwoDoubles {
    double hi, lo;
};

inline TwoDoubles two_sum(double a, double b) {
    const double s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
inline TwoDoubles mul(TwoDoubles a, TwoDoubles b) {
    const double p = a.hi * b.hi;
    return two_sum(p, fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
inline TwoDoubles add(TwoDoubles a, TwoDoubles b) {
    const TwoDoubles s = two_sum(a.hi, b.hi);
    return two_sum(s.hi, s.lo + (a.lo + b.lo));
}
inline TwoDoubles div(TwoDoubles a, double b) {
    const double q = a.hi / b;
    return two_sum(q, (fma(-q, b, a.hi) + a.lo) / b);
}

// base^(-1 / n): pow, and one Newton step on base * y^n = 1.
inline TwoDoubles inverse_root(double base, int n) {
    const double y = pow(base, -1.0 / n);
    TwoDoubles one = {base, 0};
    for (int i = 0; i < n; ++i) one = mul(one, {y, 0});
    return two_sum(y, y * ((1 - one.hi) - one.lo) / n);
}

// A frequency of at most 1 radian as a fraction of a turn in units of 2^-64 (below 2^62), rounded.
inline uint64_t to_turns(TwoDoubles f) {
    const TwoDoubles t = mul(f, {0.15915494309189535, -9.839338337591243e-18});   // 1 / (2 pi)
    const double h = ldexp(t.hi, 64), whole = floor(h);
    return static_cast<uint64_t>(whole) + static_cast<uint64_t>(static_cast<int64_t>(floor((h - whole) + ldexp(t.lo, 64) + 0.5)));
}

// The d->dims / 2 entries of a valid description.
inline void rope_table(const splash_rope_desc& d, uint64_t* turns) {
    double lo = 0, hi = 0;
    if (d.scaling == SPLASH_ROPE_YARN) {
        const double two_pi = 6.283185307179586476925;
        lo = floor(d.dims * log(d.orig_ctx / (two_pi * d.beta_fast)) / (2 * log(d.base)));
        hi = ceil(d.dims * log(d.orig_ctx / (two_pi * d.beta_slow)) / (2 * log(d.base)));
        lo = lo > 0 ? lo : 0;
        hi = hi < d.dims - 1 ? hi : d.dims - 1;
    }
    const TwoDoubles step = inverse_root(d.base, d.dims / 2);
    TwoDoubles power = {1, 0};                    // base^(-2 i / dims)
    for (int i = 0; i < d.dims / 2; ++i, power = mul(power, step)) {
        TwoDoubles f = power;
        if (d.scaling == SPLASH_ROPE_LINEAR) f = div(f, d.factor);
        if (d.scaling == SPLASH_ROPE_YARN) {
            const double w = hi - lo > 0.001 ? hi - lo : 0.001;
            TwoDoubles g = i >= lo + w ? TwoDoubles{1, 0} : (i <= lo ? TwoDoubles{0, 0} : div({i - lo, 0}, w));
            const TwoDoubles kept = add({1, 0}, {-g.hi, -g.lo});
            f = mul(f, add(kept, div(g, d.factor)));
        }
        turns[i] = to_turns(f);
    }
}

}  // namespace splash
