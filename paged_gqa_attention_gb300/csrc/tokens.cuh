// tokens.cuh -- what the kernels over new tokens share: which sequence a token belongs to, and
// the angle of a rotation at its position.
#pragma once

#include "common.cuh"

namespace pa {

// Largest s in [0, n) with cu[s] <= t (cu non-decreasing, cu[0] <= t): each round the
// 32 lanes probe 32 evenly spaced entries, narrowing the range 32-fold.
__device__ __forceinline__ int warp_find_sequence(const int32_t *cu, int n, int t, int lane) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int idx = lo + lane * step;
        const bool le = idx < hi && __ldg(cu + idx) <= t;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int last = m ? 31 - __clz(m) : 0;
        lo = lo + last * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// 2 pi in three fp32 parts (hi + mid + lo, each the rounding of what remains) and 1 / (2 pi)
constexpr double kTwoPiD = 6.28318530717958647692528676655900577;
constexpr float kTwoPiHi = (float)kTwoPiD;
constexpr float kTwoPiMid = (float)(kTwoPiD - (double)kTwoPiHi);
constexpr float kTwoPiLo = (float)(kTwoPiD - (double)kTwoPiHi - (double)kTwoPiMid);
constexpr float kInvTwoPi = (float)(1.0 / kTwoPiD);

// cos and sin of the rotation angle at position pf (an integer below 2^24, exact in fp32) for
// the frequency fh + fl (pair i's: rope_cos_sin).  p * freq is formed as hi + lo (the product's rounding error recovered with an fma),
// the multiple of 2 pi nearest hi is taken off in three parts (Cody and Waite), lo is added
// back, and the reduced angle (|r| < 4) goes to the fast sine/cosine.
__device__ __forceinline__ void angle_cos_sin(float pf, float fh, float fl, float &c, float &s) {
    const float ah = __fmul_rn(pf, fh);
    const float al = fmaf(pf, fl, fmaf(pf, fh, -ah));
    const float k = rintf(__fmul_rn(ah, kInvTwoPi));
    float r = fmaf(-k, kTwoPiHi, ah);
    r = fmaf(-k, kTwoPiMid, r);
    r = fmaf(-k, kTwoPiLo, r);
    __sincosf(__fadd_rn(r, al), &s, &c);
}

}  // namespace pa
