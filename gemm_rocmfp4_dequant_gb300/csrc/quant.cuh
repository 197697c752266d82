// The scale rule of the quantisers (dense weights, cache rows): the scale byte
// of a group of values and its exact value.
#pragma once
#include "common.cuh"

namespace rocmfp4 {

// E4M3 value of a scale byte (bit 7 clear), exact.
RF4_DEV float ue4m3_f32(uint32_t e) {
  const uint32_t E = (e >> 3) & 15u, M = e & 7u;
  return E ? __uint_as_float(((E + 120u) << 23) | (M << 20)) : (float)M * (1.0f / 512.0f);
}

// The scale byte of a group: E4M3 values increase with the byte, so this is
// the smallest e with 5 * E4M3(e) >= amax.  A candidate comes from the fp32
// bits of amax * 0.2 (E4M3 rounded up: within one step of the answer, as the
// estimate is within a few ulp of amax / 5); one exact check each way (5 *
// E4M3(e) is exact in fp32) then fixes it.
RF4_DEV uint32_t quant_scale(float amax) {
  if (!(amax > 0.f)) return 0u;
  if (5.f * ue4m3_f32(0x7Eu) < amax) return 0x7Eu;
  const float t = amax * 0.2f;
  uint32_t e;
  if (t >= 0.015625f) {  // 2^-6 and up: E4M3 exponent field E >= 1
    const uint32_t b = __float_as_uint(t);
    uint32_t E = (b >> 23) - 120u, M = (b >> 20) & 7u;
    if (b & 0xFFFFFu) ++M;  // round the 3-bit mantissa up
    if (M == 8u) {
      M = 0u;
      ++E;
    }
    e = E > 15u ? 0x7Eu : (E << 3) | M;
  } else {  // subnormal E4M3: value M / 512
    e = (uint32_t)ceilf(t * 512.f);  // at most 8, which is 2^-6 (E = 1, M = 0)
  }
  e = e > 0x7Eu ? 0x7Eu : (e == 0u ? 1u : e);
  if (e > 1u && 5.f * ue4m3_f32(e - 1u) >= amax) --e;
  else if (5.f * ue4m3_f32(e) < amax) ++e;
  return e;
}

}  // namespace rocmfp4
