// The table of a rotation: theta_i / (2 pi) as 64-bit fractions of a turn (host code).
//
// A position of 31 bits multiplies an entry's error by 2^31, so an entry is wanted to its last
// bit, 2^-65 of a turn: 64-bit floating point leaves 2^-55 (at position 2^31 - 1 an angle off by
// 3e-7, as much as everything else in the rotation). The values are therefore carried as
// unevaluated sums of two doubles (Dekker 1971; sums by Knuth's exact addition, products by a
// fused multiply-add), some 2^-104 of themselves off an operation. Products are never contracted
// by the compiler (-ffp-contract=off), so every machine makes the same table.

#include <cmath>

#include "host.h"

namespace {

// (hi + lo) 2^e with |lo| at most half a step of hi; hi in [1/2, 1) (or 0).
struct Wide {
    double hi, lo;
    int e;
};

// a + b with |a| >= |b|, or a = 0: the rounded sum and its error.
Wide scaled(double a, double b, int e) {
    const double s = a + b;
    const double r = b - (s - a);
    int k = 0;
    const double m = std::frexp(s, &k);
    return {m, std::ldexp(r, -k), e + k};
}

Wide wide(double a) { return scaled(a, 0.0, 0); }

Wide mul(const Wide& a, const Wide& b) {
    const double p = a.hi * b.hi;
    return scaled(p, std::fma(a.hi, b.lo, std::fma(a.lo, b.hi, std::fma(a.hi, b.hi, -p))), a.e + b.e);
}

Wide div(const Wide& a, double d) {
    const double q = a.hi / d;
    return scaled(q, (std::fma(-q, d, a.hi) + a.lo) / d, a.e);
}

Wide add(const Wide& a, const Wide& b) {
    const int e = a.e > b.e ? a.e : b.e;  // what falls below the range of the larger counts for nothing
    const double x = std::ldexp(a.hi, a.e - e), y = std::ldexp(b.hi, b.e - e);
    const double s = x + y, t = s - x;
    const double r = (x - (s - t)) + (y - t);
    return scaled(s, r + (std::ldexp(a.lo, a.e - e) + std::ldexp(b.lo, b.e - e)), e);
}

Wide negative(const Wide& a) { return {-a.hi, -a.lo, a.e}; }

// base^(-1 / n): two Newton steps r -= r (r^n base - 1) / n from the rounded value.
Wide root(double base, uint32_t n) {
    Wide r = wide(std::pow(base, -1.0 / n));
    for (int step = 0; step < 2; ++step) {
        Wide p = wide(1.0), x = r;
        for (uint32_t k = n; k; k >>= 1, x = mul(x, x))
            if (k & 1) p = mul(p, x);
        const Wide off = div(add(mul(p, wide(base)), wide(-1.0)), n);
        r = add(r, negative(mul(r, off)));
    }
    return r;
}

}  // namespace

extern "C" int ds_rows_rope_turns(uint32_t rot_dim, double base, double factor, uint32_t original_len, double beta_fast,
                                  double beta_slow, uint64_t* turns) {
    using dsrows::fail;
    if (!turns) return fail(DS_EINVAL, "turns is NULL");
    if (rot_dim < 2 || rot_dim > DS_DIM || rot_dim % 2)
        return fail(DS_EINVAL, "rot_dim must be even, 2..=%d, got %u", DS_DIM, rot_dim);
    if (!(base > 1.0) || !std::isfinite(base)) return fail(DS_EINVAL, "base must be finite and above 1");
    if (!(factor >= 1.0) || !std::isfinite(factor)) return fail(DS_EINVAL, "factor must be finite and at least 1");
    if (original_len && (!(beta_slow > 0.0) || !(beta_fast >= beta_slow) || !std::isfinite(beta_fast)))
        return fail(DS_EINVAL, "beta_fast >= beta_slow > 0 must be finite");
    double low = 0.0, high = 0.0;
    if (original_len) {
        const double two_pi = 6.283185307179586476925;
        auto turns_at = [&](double beta) {
            return rot_dim * std::log(original_len / (two_pi * beta)) / (2.0 * std::log(base));
        };
        low = std::fmax(std::floor(turns_at(beta_fast)), 0.0);
        high = std::fmin(std::ceil(turns_at(beta_slow)), (double)rot_dim - 1.0);
    }
    const double width = std::fmax(high - low, 0.001);
    const Wide step = root(base, rot_dim / 2);
    Wide turn = scaled(0.15915494309189535, -9.839338337591243e-18, 0);  // theta_0 / (2 pi) = 1 / (2 pi)
    for (uint32_t i = 0; i < rot_dim / 2; ++i, turn = mul(turn, step)) {
        Wide t = turn;
        if (factor != 1.0) {
            // How far the pair is interpolated: fully without YaRN's ramp.
            const double at = original_len ? i - low : width;
            if (at >= width) {
                t = div(t, factor);
            } else if (at > 0.0) {
                const Wide r = div(wide(at), width);
                t = mul(t, add(add(wide(1.0), negative(r)), div(r, factor)));
            }
        }
        // At most 2^62 (theta <= 1): the whole part and what is left of both halves.
        const double x = std::ldexp(t.hi, t.e + 64), whole = std::nearbyint(x);
        turns[i] = (uint64_t)((int64_t)whole + (int64_t)std::llrint((x - whole) + std::ldexp(t.lo, t.e + 64)));
    }
    return DS_OK;
}
