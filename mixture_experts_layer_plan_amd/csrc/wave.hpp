// Reductions over a wavefront without LDS.
#pragma once

#include "common.hpp"

namespace moe {

// Wavefront reductions: row shifts by 1, 2, 4, 8 leave the result of each row of 16 lanes
// in its last lane (lanes without a source add the identity), and the four rows' results
// are joined as scalars.  Every lane gets the same value, by additions in a fixed order.
// A shuffle would be a round trip through LDS a step.
template <int CTRL>
MOE_DEV uint32_t row_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
MOE_DEV uint32_t lane_u(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
MOE_DEV uint32_t max_u(uint32_t a, uint32_t b) { return a > b ? a : b; }
// of two scalars, by the scalar unit (the compiler would move them to the vector unit)
MOE_DEV uint32_t max_s(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("s_max_u32 %0, %1, %2" : "=s"(m) : "s"(a), "s"(b) : "scc");
  return m;
}
MOE_DEV uint32_t wave_max_u32(uint32_t v) {
  v = max_u(row_u32<0x111>(v), v);
  v = max_u(row_u32<0x112>(v), v);
  v = max_u(row_u32<0x114>(v), v);
  v = max_u(row_u32<0x118>(v), v);
  return max_s(max_s(lane_u(v, 15), lane_u(v, 31)), max_s(lane_u(v, 47), lane_u(v, 63)));
}
// Order-preserving map of fp32 to 32 bits, above 0 for numbers and infinities
MOE_DEV uint32_t ordered_u32(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
MOE_DEV float from_ordered_u32(uint32_t o) {
  return __uint_as_float(o ^ ((uint32_t)((int32_t)~o >> 31) | 0x80000000u));
}
MOE_DEV float wave_max_f32(float v) { return from_ordered_u32(wave_max_u32(ordered_u32(v))); }
template <int CTRL>
MOE_DEV float row_f32(float v) {
  return __uint_as_float(row_u32<CTRL>(__float_as_uint(v)));
}
MOE_DEV float dpp_sum_f32(float v) {
  v += row_f32<0x111>(v);
  v += row_f32<0x112>(v);
  v += row_f32<0x114>(v);
  v += row_f32<0x118>(v);
  const uint32_t u = __float_as_uint(v);
  return (__uint_as_float(lane_u(u, 15)) + __uint_as_float(lane_u(u, 31))) +
         (__uint_as_float(lane_u(u, 47)) + __uint_as_float(lane_u(u, 63)));
}

template <int CTRL, int ROWS>
MOE_DEV double dpp_f64(double old, double v) {
  const int hi =
      __builtin_amdgcn_update_dpp(__double2hiint(old), __double2hiint(v), CTRL, ROWS, 0xf, false);
  const int lo =
      __builtin_amdgcn_update_dpp(__double2loint(old), __double2loint(v), CTRL, ROWS, 0xf, false);
  return __hiloint2double(hi, lo);
}
MOE_DEV double wave_sum_f64(double v) {
  v += dpp_f64<0x111, 0xf>(0.0, v);
  v += dpp_f64<0x112, 0xf>(0.0, v);
  v += dpp_f64<0x114, 0xf>(0.0, v);
  v += dpp_f64<0x118, 0xf>(0.0, v);
  v += dpp_f64<0x142, 0xa>(0.0, v);
  v += dpp_f64<0x143, 0xc>(0.0, v);
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), 63),
                          __builtin_amdgcn_readlane(__double2loint(v), 63));
}

}  // namespace moe
