// One AdamW step over many tensors in one launch.  For every element, with g the gradient
// times grad_scale:
//   m' = beta1 m + (1 - beta1) g            each product and sum rounded to fp32
//   v' = beta2 v + ((1 - beta2) g) g
//   p' = p - lr ((m' corr1) / (sqrt(v' corr2) + eps) + weight_decay p)
// with corr = 1 / (1 - beta^step).  The states' sums are not contracted, so that their 8-bit
// codes are the same wherever the formula is evaluated in fp32.
//
// States of 8 bits: blocks of 32 neighbouring elements of a tensor share a power of two, an
// E8M0 byte.  m is E4M3; v, which is never negative, has 5 exponent and 3 mantissa bits
// (code c > 0 stands for (1 + c%8 / 8) 2^(c/8 - 31), 0 for 0), as its range is that of g
// squared.  Both are rounded to one of their two neighbours at random, in proportion to the
// distances, so that the average over steps is the state: rounded to nearest, a v would
// stay where it is while a step moves it by less than half a code (6 %), and with beta2 =
// 0.999 a step moves it by 0.1 %.  A power-of-two scale keeps codes on the grid from step to
// step, so that the variance that a step adds is |v' - v| times the distance of two codes,
// not its square.  v > 0 never becomes 0: the smallest code is its floor, as a denominator
// that vanishes would throw the weight far off.
//
// bf16 parameters without a master are rounded at random as well: to nearest, a weight would
// stay where it is while lr is below 2^-9 of it.
//
// 32 random bits per element come from the step's seed, the tensor's place in the table and
// the element's place in the tensor through mix32 below: m takes the low half, v the high
// half, p their difference by xor (pairwise independent).
#include "common.hpp"
#include "internal.hpp"
#include "step.hpp"

namespace moe {
namespace {

// Mixes the bits of x: two multiplications by the fractions of the square roots of 19 and 3
// between shifts (every bit of x turns every bit of the result with probability 0.49 to 0.51).
MOE_DEV uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x5BE0CD19u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

MOE_DEV uint32_t max_of_four_lanes(uint32_t v) {
  const uint32_t a = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true);
  v = v > a ? v : a;
  const uint32_t b = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true);
  return v > b ? v : b;
}

// The scale byte of a block whose largest magnitude has the bits `top` (as whole numbers
// they order magnitudes, with inf and NaN above): the smallest 2^(e - 127) with top <= the
// largest code * scale; CARRY is what carries into the exponent past that code's mantissa,
// SHIFT its exponent.  255 (NaN) where the state is not finite or from 2^126 on.
template <uint32_t CARRY, int SHIFT>
MOE_DEV uint32_t scale_byte(uint32_t top) {
  const int e = (int)((top + CARRY) >> 23) - SHIFT;
  return top >= 0x7E800000u ? 255u : e < 1 ? 1u : (uint32_t)e;
}
// 2^(127 - e), e in [1, 253]
MOE_DEV float inverse_scale(uint32_t e) { return __uint_as_float((254u - e) << 23); }
// 2^(e - 127); +0 for e = 0 (a buffer of zeros: codes of zero), inf for 255
MOE_DEV float scale_of(uint32_t e) { return __uint_as_float(e << 23); }

constexpr uint32_t M_CARRY = 0x1FFFFFu, V_CARRY = 0x0FFFFFu;  // past 1.75 (448), past 1.875
constexpr int M_SHIFT = 8, V_SHIFT = 0;

// Codes from 16 random bits r16, which stand for the middle of their interval: the upper
// neighbour where (distance from the lower one in steps) + (r16 + 1/2) / 2^16 >= 1.  The
// conversion instruction does just that with its upper 20 random bits.
template <int BYTE>
MOE_DEV uint32_t encode_m(float m, float inv, uint32_t r, uint32_t word) {
  return (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(m * inv, (int)(r << 16 | 0x8000u), (int)word, BYTE);
}
// v's code, plus 768: bits 20 and up of an fp32 of exponent -31 .. 0 are 768 + code
MOE_DEV uint32_t encode_v(float v, float inv, uint32_t r) {
  const uint32_t c = (__float_as_uint(v * inv) + ((r >> 12 & 0xffff0u) | 8u)) >> 20;
  const uint32_t least = v > 0.0f ? 769u : 768u;
  return c > least ? c : least;
}
MOE_DEV uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
  return lo | hi;
}
MOE_DEV float decode_v(uint32_t c) { return c ? __uint_as_float(c << 20 | 0x30000000u) : 0.0f; }
// four E4M3 codes of one word
MOE_DEV void decode_m4(uint32_t w, float* f) {
  const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  f[0] = lo.x; f[1] = lo.y; f[2] = hi.x; f[3] = hi.y;
}

typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
// 8 or 16 bytes past the caches: nothing of a step is read again in it (200 million fp32
// elements: 1098 -> 1030 us, with bf16 copies of masters 1130 -> 1040).
template <typename V>
MOE_DEV void store_past(void* p, V v) {
  __builtin_nontemporal_store(v, (V*)p);
}

MOE_DEV float round_bf16_at_random(float p, uint32_t r) {
  const uint32_t u = __float_as_uint(p);
  if ((u & 0x7f800000u) == 0x7f800000u) return p;  // inf and NaN as they are
  return __uint_as_float((u + (r & 0xffffu)) & 0xffff0000u);
}
MOE_DEV void update_state(float& m, float& v, float& g, const AdamwHyper& h) {
#pragma clang fp contract(off)
  g = g * h.grad_scale;
  m = m * h.beta1 + g * h.one_minus_beta1;
  v = v * h.beta2 + (g * h.one_minus_beta2) * g;
}

// Eight elements of a thread: a tile's eight neighbours (states of 8 bits, whose blocks of 32
// are then four lanes), or four of each of its halves, so that the lanes of a 16-byte access
// of fp32 are neighbours (SPLIT; 5.2 million elements with fp32 states: 25.0 -> 23.4 us).
constexpr int HALF = ADAMW_TILE / 2;
template <bool SPLIT>
MOE_DEV constexpr int place(int j) {
  return SPLIT ? (j >> 2) * HALF + (j & 3) : j;
}
// V neighbours; zeros from the end n on
template <bool F32, int V>
MOE_DEV void load_some(const void* p, int i, int n, float* f) {
  if (i + V <= n) {
    if constexpr (F32) {
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const float4 a = *(const float4*)((const float*)p + i + j);
        f[j] = a.x; f[j + 1] = a.y; f[j + 2] = a.z; f[j + 3] = a.w;
      }
    } else if constexpr (V == 8) {
      unpack8(*(const uint4*)((const bf16_t*)p + i), f);
    } else {
      const uint2 a = *(const uint2*)((const bf16_t*)p + i);
      f[0] = __uint_as_float(a.x << 16); f[1] = __uint_as_float(a.x & 0xffff0000u);
      f[2] = __uint_as_float(a.y << 16); f[3] = __uint_as_float(a.y & 0xffff0000u);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    f[j] = 0.0f;
    if (i + j < n) f[j] = F32 ? ((const float*)p)[i + j] : bf16_to_f32(((const bf16_t*)p)[i + j]);
  }
}
// EXACT: the values lie on bf16's grid
template <bool F32, bool EXACT, int V>
MOE_DEV void store_some(void* p, int i, int n, const float* f) {
  uint32_t w[V / 2];
#pragma unroll
  for (int j = 0; j < V / 2; ++j)
    w[j] = EXACT ? __builtin_amdgcn_perm(__float_as_uint(f[2 * j + 1]), __float_as_uint(f[2 * j]), 0x07060302u)
                 : cvt_bf16x2(f[2 * j], f[2 * j + 1]);
  if (i + V <= n) {
    if constexpr (F32) {
#pragma unroll
      for (int j = 0; j < V; j += 4)
        store_past((float*)p + i + j, f32x4_t{f[j], f[j + 1], f[j + 2], f[j + 3]});
    } else if constexpr (V == 8) {
      store_past((bf16_t*)p + i, u32x4_t{w[0], w[1], w[2], w[3]});
    } else {
      store_past((bf16_t*)p + i, u32x2_t{w[0], w[1]});
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (i + j < n) {
      if (F32) ((float*)p)[i + j] = f[j];
      else ((bf16_t*)p)[i + j] = (bf16_t)(w[j >> 1] >> (16 * (j & 1)));
    }
  }
}
template <bool F32, bool SPLIT>
MOE_DEV void load8(const void* p, int i, int n, float* f) {
  if constexpr (SPLIT) {
    load_some<F32, 4>(p, i, n, f);
    load_some<F32, 4>(p, i + HALF, n, f + 4);
  } else {
    load_some<F32, 8>(p, i, n, f);
  }
}
template <bool F32, bool EXACT, bool SPLIT>
MOE_DEV void store8(void* p, int i, int n, const float* f) {
  if constexpr (SPLIT) {
    store_some<F32, EXACT, 4>(p, i, n, f);
    store_some<F32, EXACT, 4>(p, i + HALF, n, f + 4);
  } else {
    store_some<F32, EXACT, 8>(p, i, n, f);
  }
}
// eight codes; zeros from the end n on
MOE_DEV uint2 load_codes(const void* p, int i, int n) {
  if (i + 8 <= n) return *(const uint2*)((const uint8_t*)p + i);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < n) w[j >> 2] |= (uint32_t)((const uint8_t*)p)[i + j] << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}
MOE_DEV void store_codes(void* p, int i, int n, uint2 v) {
  if (i + 8 <= n) {
    *(uint2*)((uint8_t*)p + i) = v;
    return;
  }
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < n) ((uint8_t*)p)[i + j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
}

// The tensor of a tile: the last i in [0, n) with first[i] <= tile (first ascends; a tensor
// without elements has no tiles, and the last of equal entries is the one that has).  64
// entries a step.
MOE_DEV int tensor_of(const int32_t* first, int n, int tile) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo - 1 + 63) / 64;
    const int i = lo + ((int)(threadIdx.x & 63) + 1) * step;
    const int ones = __popcll(ballot64(i < hi && first[i] <= tile));
    const int nhi = lo + (ones + 1) * step;
    hi = nhi < hi ? nhi : hi;
    lo += ones * step;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// 2048 elements a workgroup, eight a thread: larger tiles leave CUs without work in sets of
// small tensors (8192: 789 thousand elements 9.1 us, now 5.4).  fp32 states are bound by memory
// (222 million elements with masters: 6.22 GB, the least, in 1140 us, 5.45 TB/s), states of 8
// bits by vector issue (87 % of it: 490 instructions for eight elements, 70 of them the random
// bits, 60 the codes) at 5.7 TB/s.  Places are 32-bit offsets over scalar bases (64-bit places:
// 17 instructions more, 410 -> 391 us).
template <bool P32, bool G32, bool MASTER, bool EIGHT>
__global__ __launch_bounds__(256) void adamw_kernel(AdamwArgs a) {
  const int tile = blockIdx.x;
  const int id = tensor_of(a.first, a.n_tensors, tile);
  const AdamwDesc d = a.desc[id];
  const AdamwHyper h = a.hyper_dev ? *a.hyper_dev : a.hyper;
  const int64_t tile0 = (int64_t)(tile - a.first[id]) * ADAMW_TILE;
  if (tile0 >= d.n) return;  // the grid is an upper bound
  // (a tile starts at a multiple of 2^11, so the high word of the place is the tile's)
  const uint32_t key = mix32(mix32((uint32_t)id + 1u) + h.seed) + (uint32_t)(tile0 >> 32) * 0x3C6EF373u;
  const uint32_t place0 = (uint32_t)tile0;
  // from here on places in the tile, of which the tensor has n: bases are scalars, offsets 32 bits
  constexpr bool SPLIT = !EIGHT;
  const int n = d.n - tile0 < ADAMW_TILE ? (int)(d.n - tile0) : ADAMW_TILE;
  const int i = (int)threadIdx.x * (SPLIT ? 4 : 8);
  constexpr int SB = EIGHT ? 1 : 4, PB = P32 ? 4 : 2;
  const auto at = [&](const void* base, int bytes) { return (const char*)base + tile0 * bytes; };
  const auto to = [&](void* base, int bytes) { return (char*)base + tile0 * bytes; };
  float g[8], p[8], m[8], v[8];
  uint32_t r[8];
  load8<G32, SPLIT>(at(d.grad, G32 ? 4 : 2), i, n, g);
  if (MASTER) load8<true, SPLIT>(at(d.master, 4), i, n, p);
  else load8<P32, SPLIT>(at(d.param, PB), i, n, p);
  if (EIGHT) {
    const uint2 mc = load_codes(at(d.m, SB), i, n), vc = load_codes(at(d.v, SB), i, n);
    const uint8_t *ms = d.m_scale + (tile0 >> 5), *vs = d.v_scale + (tile0 >> 5);
    const uint32_t me = i < n ? ms[i >> 5] : 0u, ve = i < n ? vs[i >> 5] : 0u;
    decode_m4(mc.x, m);
    decode_m4(mc.y, m + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] *= scale_of(me);
      v[j] = decode_v(((j < 4 ? vc.x : vc.y) >> (8 * (j & 3))) & 255u) * scale_of(ve);
    }
  } else {
    load8<true, SPLIT>(at(d.m, SB), i, n, m);
    load8<true, SPLIT>(at(d.v, SB), i, n, v);
  }
  // The root instruction takes a subnormal number for 0: 2^-63 off at most, which matters beside
  // an eps below 2^-39 alone.  There it gets 2^24 times the number (inf from 2^104 on); a test of
  // each number would cost the step of 8-bit states 2 %.
  const bool small = h.eps < 0x1p-39f;
  const float corr2 = small ? h.corr2 * 0x1p24f : h.corr2, unscale = small ? 0x1p-12f : 1.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    update_state(m[j], v[j], g[j], h);
    // reciprocal and root of one unit: the quotient is far below the weight it is added to
    const float root = __builtin_amdgcn_sqrtf(v[j] * corr2);
    const float u = m[j] * h.corr1 * __builtin_amdgcn_rcpf(fmaf(root, unscale, h.eps));
    p[j] = fmaf(-h.lr, fmaf(d.weight_decay, p[j], u), p[j]);
    if (EIGHT || (!P32 && !MASTER)) r[j] = mix32((place0 + (uint32_t)(i + place<SPLIT>(j))) ^ key);
  }
  if (MASTER) store8<true, false, SPLIT>(to(d.master_out, 4), i, n, p);
  if (!P32 && !MASTER) {
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = round_bf16_at_random(p[j], r[j] ^ (r[j] >> 16));
  }
  store8<P32, !P32 && !MASTER, SPLIT>(to(d.param_out, PB), i, n, p);
  if (EIGHT) {
    uint32_t mt = 0, vt = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t mu = __float_as_uint(m[j]) & 0x7fffffffu, vu = __float_as_uint(v[j]);
      mt = mt > mu ? mt : mu;
      vt = vt > vu ? vt : vu;
    }
    mt = max_of_four_lanes(mt);
    vt = max_of_four_lanes(vt);
    const uint32_t me = scale_byte<M_CARRY, M_SHIFT>(mt), ve = scale_byte<V_CARRY, V_SHIFT>(vt);
    const float mi = inverse_scale(me), vi = inverse_scale(ve);
    uint32_t mw[2] = {0, 0}, c[8];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      mw[w] = encode_m<0>(m[4 * w], mi, r[4 * w], mw[w]);
      mw[w] = encode_m<1>(m[4 * w + 1], mi, r[4 * w + 1], mw[w]);
      mw[w] = encode_m<2>(m[4 * w + 2], mi, r[4 * w + 2], mw[w]);
      mw[w] = encode_m<3>(m[4 * w + 3], mi, r[4 * w + 3], mw[w]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = encode_v(v[j], vi, r[j]);
    const uint32_t vw[2] = {low_bytes(c[0], c[1], c[2], c[3]), low_bytes(c[4], c[5], c[6], c[7])};
    // a block that is not finite: codes of zero under a scale of inf, which is NaN
    store_codes(to(d.m_out, SB), i, n, me == 255u ? make_uint2(0, 0) : make_uint2(mw[0], mw[1]));
    store_codes(to(d.v_out, SB), i, n, ve == 255u ? make_uint2(0, 0) : make_uint2(vw[0], vw[1]));
    if (i < n && (threadIdx.x & 3) == 0) {
      (d.m_scale_out + (tile0 >> 5))[i >> 5] = (uint8_t)me;
      (d.v_scale_out + (tile0 >> 5))[i >> 5] = (uint8_t)ve;
    }
  } else {
    store8<true, false, SPLIT>(to(d.m_out, SB), i, n, m);
    store8<true, false, SPLIT>(to(d.v_out, SB), i, n, v);
  }
}

__global__ __launch_bounds__(64) void adamw_table_kernel(AdamwChunk c, AdamwDesc* desc, int32_t* first) {
  const int i = threadIdx.x;
  if (i < c.count) {
    desc[c.base + i] = c.d[i];
    first[c.base + i] = c.first[i];
  }
}

// The values that codes stand for, as bf16 (exact: at most 4 significant bits, down to the
// type's smallest normal number).
template <bool V>
__global__ __launch_bounds__(256) void adamw_values_kernel(int64_t n, const uint8_t* codes,
                                                           const uint8_t* scales, bf16_t* out) {
  for (int64_t t = (int64_t)blockIdx.x * 2048; t < n; t += (int64_t)gridDim.x * 2048) {
    const int left = n - t < 2048 ? (int)(n - t) : 2048, i = (int)threadIdx.x * 8;
    const uint2 c = load_codes(codes + t, i, left);
    const float s = i < left ? scale_of((scales + (t >> 5))[i >> 5]) : 0.0f;
    float f[8];
    if (V) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = decode_v(((j < 4 ? c.x : c.y) >> (8 * (j & 3))) & 255u) * s;
    } else {
      decode_m4(c.x, f);
      decode_m4(c.y, f + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= s;
    }
    store8<false, true, false>(out + t, i, left, f);
  }
}

template <bool P32, bool G32, bool MASTER>
hipError_t adamw_as(const AdamwArgs& p, bool eight, hipStream_t s) {
  if (eight)
    return MOE_LAUNCH("adamw", s, adamw_kernel<P32, G32, MASTER, true><<<p.tiles, 256, 0, s>>>(p));
  return MOE_LAUNCH("adamw", s, adamw_kernel<P32, G32, MASTER, false><<<p.tiles, 256, 0, s>>>(p));
}

}  // namespace

hipError_t launch_adamw_table(const AdamwChunk& c, AdamwDesc* desc, int32_t* first, hipStream_t s) {
  return MOE_LAUNCH("adamw_table", s, adamw_table_kernel<<<1, 64, 0, s>>>(c, desc, first));
}

hipError_t launch_adamw(const AdamwArgs& p, bool f32, bool g32, bool master, bool eight,
                        hipStream_t s) {
  if (p.tiles == 0) return hipSuccess;
  if (f32) return g32 ? adamw_as<true, true, false>(p, eight, s) : adamw_as<true, false, false>(p, eight, s);
  if (master) return g32 ? adamw_as<false, true, true>(p, eight, s) : adamw_as<false, false, true>(p, eight, s);
  return g32 ? adamw_as<false, true, false>(p, eight, s) : adamw_as<false, false, false>(p, eight, s);
}

hipError_t launch_adamw_values(bool v, int64_t n, const uint8_t* codes, const uint8_t* scales,
                               void* out, hipStream_t s) {
  if (n == 0) return hipSuccess;
  const int64_t want = (n + 2047) / 2048;
  const int grid = want < 65536 ? (int)want : 65536;
  if (v)
    return MOE_LAUNCH("adamw_values", s,
                      adamw_values_kernel<true><<<grid, 256, 0, s>>>(n, codes, scales, (bf16_t*)out));
  return MOE_LAUNCH("adamw_values", s,
                    adamw_values_kernel<false><<<grid, 256, 0, s>>>(n, codes, scales, (bf16_t*)out));
}

}  // namespace moe
