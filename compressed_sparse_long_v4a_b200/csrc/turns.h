// turns.h -- angles of rotary positions: sines and cosines that stay exact to fp32 for positions up to 2^40.
#pragma once

#include <math.h>

#include "common.cuh"

namespace v4a {

constexpr int kMaxPairs = 256;

// turns (not radians) per position of every pair, each as a sum of two
struct Turns {
    double hi[kMaxPairs];
    float lo[kMaxPairs];
};

// cos and sin of p f, f = hi + lo turns per position: the product as an exact sum of two doubles, so
// the fraction of a turn keeps more than 24 bits for |p| up to 2^40.  It is rounded to fp32, up to 2^-24 pi radians, for
// sincospif: fp32 outputs are off by 6e-8 relative where 64-bit sines give 4.6e-8.
__device__ __forceinline__ float2 turn(double p, double f_hi, float f_lo) {
    const double hi = p * f_hi;
    const double lo = fma(p, f_hi, -hi) + p * (double)f_lo;
    const double frac = (hi - rint(hi)) + lo;
    float s, c;
    sincospif((float)(2.0 * frac), &s, &c);
    return make_float2(c, s);
}

// base^(-2k/R) radians per position, k < R / 2, extended by `factor` (1: not): divided by it, or, with an original
// length orig_ctx, those pairs only that turn less than beta_slow times over it, blended up to beta_fast
inline void make_turns(int rope_dims, double base, Turns* t, double factor = 1, long long orig_ctx = 0, double beta_fast = 0,
                       double beta_slow = 0) {
    const long double two_pi = 6.283185307179586476925286766559005768L;
    const long double step = powl((long double)base, -2.0L / rope_dims), inv_factor = 1.0L / (long double)factor;
    const long double span = 1.0L / ((long double)beta_fast - (long double)beta_slow);  // used with orig_ctx only
    long double f = 1.0L / two_pi;  // turns
    for (int k = 0; k < rope_dims / 2; ++k, f *= step) {
        long double g = f * inv_factor;
        if (orig_ctx > 0) {
            long double w = ((long double)orig_ctx * f - (long double)beta_slow) * span;
            w = w < 0 ? 0 : w > 1 ? 1 : w;
            g = f * w + g * (1 - w);
        }
        t->hi[k] = (double)g;
        t->lo[k] = (float)(g - (long double)t->hi[k]);
    }
}

}  // namespace v4a
