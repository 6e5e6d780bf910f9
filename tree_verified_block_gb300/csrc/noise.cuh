// The sampling noise, shared by the LM head's sampling mode and by the sampler
// over rows of logits: both give a token the same noise.
#pragma once

#include <stdint.h>

namespace glance_dev {

// Philox4x32-10: ten rounds of two 32x32 -> 64-bit products; the key advances
// by the Weyl increments (2^32 / golden ratio, 2^32 (sqrt 3 - 1)) per round.
__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint32_t k0, uint32_t k1) {
  constexpr uint32_t kM0 = 0xD2511F53u, kM1 = 0xCD9E8D57u;
  constexpr uint32_t kW0 = 0x9E3779B9u, kW1 = 0xBB67AE85u;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    if (r) {
      k0 += kW0;
      k1 += kW1;
    }
    // each 32 x 32 -> 64-bit product as one wide multiply
    const unsigned long long p0 = static_cast<unsigned long long>(c.x) * kM0;
    const unsigned long long p1 = static_cast<unsigned long long>(c.z) * kM1;
    const uint32_t lo0 = static_cast<uint32_t>(p0), hi0 = static_cast<uint32_t>(p0 >> 32);
    const uint32_t lo1 = static_cast<uint32_t>(p1), hi1 = static_cast<uint32_t>(p1 >> 32);
    c = make_uint4(hi1 ^ c.y ^ k0, lo1, hi0 ^ c.w ^ k1, lo0);
  }
  return c;
}

// Gumbel noise from one 32-bit word: u = (k + 1/2) / 2^23 in (0, 1), k = the
// top 23 bits. The inner log needs relative accuracy near u = 1, where -ln u
// is tiny and decides the largest noise values; the outer one only absolute
// accuracy. With t = 1 - u = (2^23 - 1/2 - k) / 2^23 (exact in fp32): for
// t < 1/32 the Taylor series -ln(1 - t) = t + t^2/2 + t^3/3 + t^4/4 + t^5/5
// (relative error below t^5 / 6 < 6e-9); elsewhere -ln u > 1/32 and the
// hardware logarithm's absolute error (~1e-7) is below 4e-6 relative.
__device__ __forceinline__ float gumbel_of(uint32_t w) {
  const float k = static_cast<float>(w >> 9);
  const float u = (k + 0.5f) * (1.0f / 8388608.0f);
  const float t = (8388607.5f - k) * (1.0f / 8388608.0f);
  const float series = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 0.2f, 0.25f), 1.0f / 3.0f), 0.5f), 1.0f);
  const float nl = t < 0.03125f ? series : -__logf(u);
  return -__logf(nl);
}

}  // namespace glance_dev
