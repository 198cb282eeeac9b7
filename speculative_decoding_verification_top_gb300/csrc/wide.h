// wide.h -- numbers held as the sum of two doubles, some 2^-104 of themselves off
// after an operation (Dekker 1971, Knuth's two-sum; products by a fused operation),
// for constants that the host computes.  Not a public header.
#pragma once

#include <cmath>
#include <cstdint>

namespace specv {

struct Wide {
    double hi, lo;  // |lo| is at most half a step of hi
};

inline Wide wide(double x) { return {x, 0.0}; }

// a + b where |a| >= |b|, and in any order: exact.
inline Wide sum_ordered(double a, double b) {
    const double s = a + b;
    return {s, b - (s - a)};
}

inline Wide sum_exact(double a, double b) {
    const double s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}

inline Wide operator+(Wide a, Wide b) {
    const Wide s = sum_exact(a.hi, b.hi), t = sum_exact(a.lo, b.lo);
    const Wide u = sum_ordered(s.hi, s.lo + t.hi);
    return sum_ordered(u.hi, u.lo + t.lo);
}

inline Wide operator-(Wide a, Wide b) { return a + Wide{-b.hi, -b.lo}; }

inline Wide operator*(Wide a, Wide b) {
    // volatile: a compiler may fuse a product with the sum it goes to, and the
    // rounded product is meant here.
    volatile double p = a.hi * b.hi;
    const double hi = p;
    return sum_ordered(hi, std::fma(a.lo, b.hi, std::fma(a.hi, b.lo, std::fma(a.hi, b.hi, -hi))));
}

inline Wide operator/(Wide a, Wide b) {
    const double q0 = a.hi / b.hi;
    const Wide r = a - b * wide(q0);
    const double q1 = r.hi / b.hi;
    const Wide s = r - b * wide(q1);
    return sum_ordered(q0, q1) + wide(s.hi / b.hi);
}

// a / b clamped to [0, 1], for b > 0 of any size.
inline Wide share(Wide a, Wide b) {
    if (a.hi <= 0.0) return wide(0.0);
    return (a - b).hi >= 0.0 ? wide(1.0) : a / b;
}

// x^(1/n) for x > 0: Newton's steps r (1 + (x / r^n - 1) / n) from the double's root.
inline Wide root(double x, int n) {
    Wide r = wide(std::pow(x, 1.0 / n));
    for (int i = 0; i < 2; ++i) {
        Wide power = wide(1.0);
        for (int k = 0; k < n; ++k) power = power * r;
        r = r + r * ((wide(x) / power - wide(1.0)) / wide(n));
    }
    return r;
}

// The integer nearest to 0 <= x < 2^63.
inline uint64_t nearest(Wide x) {
    const double whole = std::floor(x.hi);
    return static_cast<uint64_t>(static_cast<int64_t>(whole) + static_cast<int64_t>(std::nearbyint(x.hi - whole + x.lo)));
}

}  // namespace specv
