// rope_step.h -- a rotary frequency as the kernels take it, for the entry points and for checks on the
// host.  Plain C++.
#pragma once

#include <cmath>
#include <cstdint>

namespace fvattn {

constexpr double kMostRopeFreq = 18446744073709551616.0;  // 2^64: neighbouring doubles lie 2^12 radians apart

// Revolutions per unit of position, freq / (2 pi), modulo 1 and rounded to the nearest 2^-64, for
// |freq| < 2^64.  In whole numbers: freq = n 2^(e - 53), 1 / (2 pi) = W 2^-192 (less than 2^-192 off, which
// n 2^(e - 53) makes 2^-128 at most), and of n W the 64 bits below the point are wanted.  (A quotient in
// floating point loses the bits that the whole revolutions take: at 1e9 radians a unit and position 2^31, up to 0.1 radians.)
inline uint64_t rope_step(double freq) {
    constexpr uint64_t W[3] = {0x36d8a5664f10e410u, 0x7f09d5f47d4d3770u, 0x28be60db9391054au};  // low word first
    int e;
    const uint64_t n = static_cast<uint64_t>(std::ldexp(std::frexp(std::fabs(freq), &e), 53));
    uint64_t p[5] = {0, 0, 0, 0, 0}, carry = 0;  // n W, and a word of zeros above it
    for (int i = 0; i < 3; ++i) {
        const unsigned __int128 x = static_cast<unsigned __int128>(n) * W[i] + carry;
        p[i] = static_cast<uint64_t>(x);
        carry = static_cast<uint64_t>(x >> 64);
    }
    p[3] = carry;
    const int shift = 181 - e;  // of the step's last bit in n W: at least 117
    if (shift > 256) return 0;  // (n W has 256 bits at most)
    auto bit = [&](int i) { return i < 256 ? (p[i >> 6] >> (i & 63)) & 1u : 0u; };
    const int word = shift >> 6, low = shift & 63;
    const uint64_t here = word < 4 ? p[word] : 0, above = word < 4 ? p[word + 1] : 0;
    const uint64_t step = (low ? here >> low | above << (64 - low) : here) + bit(shift - 1);
    return freq < 0 ? 0 - step : step;  // (backwards: what is missing to a whole revolution)
}

}  // namespace fvattn
