// turn.cuh -- cos and sin of a rotary angle.
//
// Pair (x_0, x_1) of a token at position t turns by t * inv_freq[i]. The angle is formed in half
// turns as an unevaluated sum of two floats (error-free product by fused multiply-add, after
// Dekker): t * f in one float is off by up to 2^-25 of its size, 0.03 rad at t = 10^6. Whole turns
// are removed exactly before the sum is rounded, so cos and sin are good to 2^-22 up to positions of 2^24; beyond,
// the low part's own roundings (2^-46 of the angle) show: 2^-21 at 2^26, 2^-17.5 at 2^29.
#pragma once

namespace mha {

// (cos, sin) of pos * f
__device__ __forceinline__ float2 turn_of(int pos, float f) {
    constexpr float kInvPi = 0.318309873342514038f;        // 1 / pi rounded to fp32 ...
    constexpr float kInvPiLow = 1.28412766334e-8f;         // ... and the rest
    const float ph = f * kInvPi;
    const float pl = fmaf(f, kInvPiLow, fmaf(f, kInvPi, -ph));
    const float th = static_cast<float>(pos);
    const float tl = static_cast<float>(static_cast<long long>(pos) - static_cast<long long>(th));
    const float ah = th * ph;
    float al = fmaf(th, ph, -ah);
    al = fmaf(th, pl, al);
    al = fmaf(tl, ph, al);
    const float r = (ah - 2.0f * rintf(0.5f * ah)) + al;   // the difference is exact
    float2 cs;
    sincospif(r, &cs.y, &cs.x);
    return cs;
}

}  // namespace mha
