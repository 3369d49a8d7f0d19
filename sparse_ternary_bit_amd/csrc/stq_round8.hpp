// The rounding of scaled values to 8-bit integers, the same bits for every
// operator that writes 8-bit rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace stq {

// The nearest integer to v / scale for N values (a multiple of 4), packed; inv
// is 1 / scale.  In fp32, adding 1.5 * 2^23 to v * (1 / scale) in one fused
// step rounds it to an integer, halves to even, whose two's complement is the
// sum's low byte.  The quotient is within 127 * 2^-23 of the exact one, so
// this decides wherever it is farther than 2^-15 from a half; one lane in a
// thousand has a value that close and redoes its N in fp64, where the
// remainder v - q scale is exact.  (No value exceeds 127 there: |v| / scale <=
// 127 (1 + 2^-24).)  fast: the scale is far above where the reciprocal or the
// products leave the normal range.
template <int N>
__device__ __forceinline__ void quantize(const float (&v)[N], float scale, float inv, bool fast, uint32_t (&o)[N / 4]) {
  constexpr float kMagic = 12582912.0f;
  float far = 0.0f;
  uint32_t b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float s = fmaf(v[i], inv, kMagic);
    far = fmaxf(far, fabsf(fmaf(v[i], inv, kMagic - s)));
    b[i] = __builtin_bit_cast(uint32_t, s);
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x04000C0Cu);
    o[i] = lo | hi;
  }
  if (fast && far < 0.5f - 0x1p-15f) return;
  const double sd = static_cast<double>(scale), invd = 1.0 / sd, half = 0.5 * sd;
#pragma unroll
  for (int i = 0; i < N / 4; ++i) o[i] = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const double x = static_cast<double>(v[i]);
    double q = rint(x * invd);
    const double rem = fma(-q, sd, x);
    // the product can land on the wrong side only next to a half
    const double other = q + (rem > 0.0 ? 1.0 : -1.0);
    if (fabs(rem) > half || (fabs(rem) == half && (static_cast<int>(q) & 1))) q = other;
    const int qi = max(-127, min(127, static_cast<int>(q)));
    o[i >> 2] |= (static_cast<uint32_t>(qi) & 0xFFu) << (8 * (i & 3));
  }
}

}  // namespace stq
