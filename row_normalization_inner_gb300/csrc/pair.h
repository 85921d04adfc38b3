// Host arithmetic on pairs of doubles: a number is hi + lo, |lo| at most half a
// step of hi, some 104 bits.  For what is computed once and kept in 64 bits (the
// rates of a rotation), where doubles alone lose the last eleven.
//
// Sums and products without error as in T. J. Dekker, "A floating-point technique
// for extending the available precision" (1971) and D. E. Knuth, "The Art of
// Computer Programming", vol. 2, 4.2.2.
#pragma once

#include <cmath>

namespace nf {

struct Pair {
    double hi, lo;
    Pair(double h = 0.0, double l = 0.0) : hi(h), lo(l) {}
};

// A product rounded by itself: a compiler may join it with a sum (gcc does on Arm),
// and the same call would then give another machine other bits.
inline double rounded(double a, double b) {
    volatile double p = a * b;
    return p;
}

// a + b, |a| >= |b| or a = 0.
inline Pair joined(double a, double b) {
    const double s = a + b;
    return {s, b - (s - a)};
}
inline Pair exact_sum(double a, double b) {
    const double s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}

inline Pair operator+(Pair a, Pair b) {
    const Pair s = exact_sum(a.hi, b.hi), t = exact_sum(a.lo, b.lo);
    const Pair u = joined(s.hi, s.lo + t.hi);
    return joined(u.hi, u.lo + t.lo);
}
inline Pair operator-(Pair a) { return {-a.hi, -a.lo}; }
inline Pair operator-(Pair a, Pair b) { return a + -b; }
inline Pair operator*(Pair a, Pair b) {
    const double p = rounded(a.hi, b.hi);
    const double e = std::fma(a.hi, b.hi, -p) + (rounded(a.hi, b.lo) + rounded(a.lo, b.hi));
    return joined(p, e);
}
inline Pair operator/(Pair a, Pair b) {
    const double q = a.hi / b.hi;
    const Pair r = a - b * q;
    const double q2 = r.hi / b.hi, q3 = (r - b * q2).hi / b.hi;
    return joined(q, q2) + q3;
}
inline Pair scaled(Pair a, int exponent) { return {std::ldexp(a.hi, exponent), std::ldexp(a.lo, exponent)}; }

inline Pair two_pi() { return {0x1.921fb54442d18p+2, 0x1.1a62633145c07p-52}; }

// e^x, |x| below 1400: x = k ln 2 + r, then e^(r / 2^9) - 1 by its Taylor series (what
// is left out is below 2^-112) and (1 + s)^2 - 1 = 2s + s^2 nine times.
inline Pair exponential(Pair x) {
    const Pair ln2(0x1.62e42fefa39efp-1, 0x1.abc9e3b39803fp-56);
    const double k = std::nearbyint(x.hi / ln2.hi);
    const Pair r = scaled(x - ln2 * k, -9);
    Pair s, term(1.0);
    for (int n = 1; n <= 9; ++n) {
        term = term * r / static_cast<double>(n);
        s = s + term;
    }
    for (int n = 0; n < 9; ++n) s = scaled(s, 1) + s * s;
    return scaled(s + 1.0, static_cast<int>(k));
}

// ln x of a positive finite x, by Newton's steps from the double's.
inline Pair logarithm(double x) {
    Pair y(std::log(x));
    for (int n = 0; n < 2; ++n) {
        int e;
        const double m = std::frexp(x, &e);  // x e^-y as m 2^e e^-y: neither factor leaves the range
        const Pair ln2(0x1.62e42fefa39efp-1, 0x1.abc9e3b39803fp-56);
        y = y + (Pair(m) * exponential(ln2 * static_cast<double>(e) - y) - 1.0);
    }
    return y;
}

}  // namespace nf
