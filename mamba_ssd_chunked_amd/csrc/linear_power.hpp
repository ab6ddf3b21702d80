// Powers of a head's constant decay, for every part of linear attention.
#pragma once

#include "ssd_device.hpp"

namespace ssd {

// Below this a log decay counts as this: its powers but the zeroth are zero in fp32, and 0 * -inf
// does not come up.
constexpr double kMinDecay = -1.0e4;

// Base-2 logarithm of a head's decay.
__device__ __forceinline__ double log2_decay(float log_decay) {
    return (log_decay < kMinDecay ? kMinDecay : static_cast<double>(log_decay)) * kLog2e;
}

// a^n for the base-2 logarithm of a, by the hardware's exponential (about 1 ulp) of the product e rounded to fp32 and
// the first order of what that leaves: 2^rest = 1 + rest ln 2 to 24 bits, as |rest| < 2^-16 wherever the power is
// neither 0 nor infinite.  (Without it e costs |e| 2^-24 ln 2 of the power: 22 half steps at n = 32 and a = 1 / e.)
// Below the fp32 range it is 0.
__device__ __forceinline__ float power(double log2a, int n) {
    const float hi = static_cast<float>(log2a), lo = static_cast<float>(log2a - hi), m = static_cast<float>(n);
    const float e = hi * m, rest = fmaf(hi, m, -e) + lo * m;
    return __builtin_amdgcn_exp2f(e) * fmaf(rest, 0.693147182f, 1.0f);
}

}  // namespace ssd
