// Cosine and sine of rotary angles, shared by the appends (sm_103a).
#pragma once

#include <cuda_runtime.h>

namespace tts {

// The angle a = s * theta is formed in double (the same product the
// definition takes) and reduced modulo 2 pi in double (Cody and Waite's
// reduction with 2 pi split into two doubles); the reduced angle r,
// |r| <= pi, is split into floats r_hi + r_lo, and cos/sin come from
// sincosf(r_hi) with the first-order correction for r_lo: an error of a few
// 2^-24 for a handful of double operations per angle (double throughput is
// low on this part).
constexpr double kTwoPiHi = 6.283185307179586;       // 2 pi rounded to double
constexpr double kTwoPiLo = 2.4492935982947064e-16;  // 2 pi - kTwoPiHi
constexpr double kInvTwoPi = 0.15915494309189535;    // 1 / (2 pi)

__device__ __forceinline__ float2 rope_cos_sin(int s, double theta) {
    const double a = static_cast<double>(s) * theta;
    const double k = rint(a * kInvTwoPi);
    const double r = fma(-k, kTwoPiLo, fma(-k, kTwoPiHi, a));
    const float rh = static_cast<float>(r);
    const float rl = static_cast<float>(r - static_cast<double>(rh));
    float sh, ch;
    sincosf(rh, &sh, &ch);
    return make_float2(fmaf(-sh, rl, ch), fmaf(ch, rl, sh));
}

}  // namespace tts
