// The frequencies of the position rotation as fractions of a turn (host only).
#pragma once

#include <cmath>

namespace pe {

// Turns per position of pair i, theta^(-2i/hd) / 2 pi, as the nearest whole
// number of 2^-64, for the hd/2 pairs of a head (a power of two of them). A
// position below 2^31 is then off by 2^-34 of a turn; from a power in double,
// whose 53 bits end at 2^-55 of a turn, it was 2^-24.
//
// Sums of two doubles, hi + lo, carry 2^-100 or so: theta^(-2/hd) is one over
// repeated square roots of theta, each with a Newton step on the remainder that
// fma gives exactly, and the powers follow one from the last.
inline void rotation_turns(float theta, int hd, unsigned long long* freq) {
    struct Two {
        double hi, lo;
    };
    auto sum = [](double a, double b) {   // |b| is not above |a|
        const double s = a + b;
        return Two{s, b - (s - a)};
    };
    auto product = [&](const Two& a, const Two& b) {
        const double p = a.hi * b.hi;
        return sum(p, std::fma(a.hi, b.hi, -p) + std::fma(a.hi, b.lo, a.lo * b.hi));
    };
    Two root{static_cast<double>(theta), 0.0};
    for (int n = hd / 2; n > 1; n /= 2) {
        const double x = std::sqrt(root.hi);
        root = sum(x, (std::fma(-x, x, root.hi) + root.lo) / (2 * x));
    }
    const double inv = 1 / root.hi;
    const Two step = sum(inv, (std::fma(-inv, root.hi, 1.0) - inv * root.lo) * inv);
    Two turns{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};   // 1 / 2 pi
    for (int i = 0; i < hd / 2; ++i) {
        const double high = std::ldexp(turns.hi, 64), whole = std::floor(high);
        freq[i] = static_cast<unsigned long long>(whole) +
                  static_cast<unsigned long long>(std::llrint((high - whole) + std::ldexp(turns.lo, 64)));
        turns = product(turns, step);
    }
}

}  // namespace pe
