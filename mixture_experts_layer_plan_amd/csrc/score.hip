// Scored routing: the choice of k experts per token from softmax or sigmoid scores of
// the router's logits, with a selection bias, expert groups and renormalised weights,
// and the gradient of the logits.
//
// With l the logits of one token, s_e = sigmoid(l_e) or softmax(l)_e and the choice value
// c_e = s_e + bias_e: the experts are taken in groups of E / n_groups neighbours, a
// group's score is the sum of its group_top largest c, the topk_groups best groups stay,
// and the k largest c of their experts are chosen (ties: lowest id).  The weights come
// from s alone: w_j = scale s_j, over sum_i s_i if renormalised.
//
// One 64-lane wavefront per token; lane i holds the NPL neighbouring experts
// i NPL .. i NPL + NPL - 1, so that the lowest lane of a tie is the lowest id.
#include <math.h>

#include "common.hpp"
#include "internal.hpp"
#include "wave.hpp"

namespace moe {
namespace {

// exp(x) for x <= 0 in double, of N values at once (the constants are loaded once):
// x = n ln 2 + r with |r| <= ln 2 / 2, the Taylor series of exp(r) to r^13 / 13! (the rest
// is below 2^-57), scaled by 2^n (down to the subnormals).  Below -746, past the smallest
// double, 0.
template <int N>
MOE_DEV void exp_neg(double (&x)[N]) {
  constexpr double C[14] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040,
                            1.0 / 40320, 1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800,
                            1.0 / 479001600, 1.0 / 6227020800.0};
  double n[N], r[N], p[N];
#pragma unroll
  for (int i = 0; i < N; ++i) n[i] = rint(x[i] * 1.4426950408889634074);
#pragma unroll
  for (int i = 0; i < N; ++i)
    r[i] = fma(n[i], -1.9082149292705877e-10, fma(n[i], -6.93147180369123816490e-01, x[i]));
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = C[13];
#pragma unroll
  for (int c = 12; c >= 0; --c)
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = fma(p[i], r[i], C[c]);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const double e = ldexp(p[i], (int)n[i]);
    x[i] = x[i] < -746.0 ? 0.0 : e;
  }
}

// 1 / d for d in [1, 2]: the reciprocal instruction and two Newton steps.
MOE_DEV double recip(double d) {
  double y = __builtin_amdgcn_rcp(d);
  y = fma(fma(-d, y, 1.0), y, y);
  return fma(fma(-d, y, 1.0), y, y);
}

MOE_DEV int lane_i(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
MOE_DEV float lane_f(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// An expert is present if its logit is a number above -inf.
MOE_DEV bool present(float l) { return l > -INFINITY; }

// Order-preserving map of a double to 64 bits; 0 is kept for "absent or taken" (no
// number maps to it).  -0.0 is turned into +0.0 first.
MOE_DEV unsigned long long ordered_f64(double v) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(v + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
MOE_DEV unsigned long long ordered_f32(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (unsigned long long)((u >> 31) ? ~u : (u | 0x80000000u)) << 32;
}

// The two largest of two pairs (b1 >= b2), the other pair from a lane that CTRL names.
template <int CTRL>
MOE_DEV void merge2(double& b1, double& b2) {
  const double o1 = dpp_f64<CTRL, 0xf>(b1, b1), o2 = dpp_f64<CTRL, 0xf>(b2, b2);
  b2 = fmax(fmin(b1, o1), fmax(b2, o2));
  b1 = fmax(b1, o1);
}

// The NPL logits of this lane; experts past E read as -inf.
template <int NPL>
MOE_DEV void load_row(const float* __restrict__ L, int E, int lane, bool vec, float (&l)[NPL]) {
  const int e0 = lane * NPL;
  if (vec) {  // E and the row are multiples of min(NPL, 4) values
    constexpr int V = NPL < 4 ? NPL : 4;
#pragma unroll
    for (int i = 0; i < NPL; i += V) {
      const bool in = e0 + i < E;
      if constexpr (V == 4) {
        const float4 v = in ? *(const float4*)(L + e0 + i)
                            : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        l[i] = v.x; l[i + 1] = v.y; l[i + 2] = v.z; l[i + 3] = v.w;
      } else if constexpr (V == 2) {
        const float2 v = in ? *(const float2*)(L + e0 + i) : make_float2(-INFINITY, -INFINITY);
        l[i] = v.x; l[i + 1] = v.y;
      } else {
        l[i] = in ? L[e0 + i] : -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) l[i] = e0 + i < E ? L[e0 + i] : -INFINITY;
  }
}

// sigmoid(l) = exp(-a) q with a = max(-l, 0), q = 1 / (1 + exp(-|l|)) in (1/2, 1]:
// neither factor overflows, and a ratio of two sigmoids needs only the difference of
// their a, so renormalised weights survive where exp(l) itself would underflow.
MOE_DEV void sigmoid_parts(float l, float& a, float& q) {
  a = fmaxf(-l, 0.0f);
  q = 1.0f / (1.0f + expf(-fabsf(l)));
}

// Normalised scores p of the k chosen logits, one per lane (p = 0 where !mine): the
// scores over their sum if renormalised, else the scores themselves.
// row_max, row_sum: of exp over all experts (softmax without renormalisation only).
MOE_DEV float chosen_score(int score, bool renorm, bool mine, float l, float row_max,
                           float row_sum) {
  if (score == 1) {
    float a, q;
    sigmoid_parts(l, a, q);
    if (!renorm) return mine ? expf(-a) * q : 0.0f;
    const float a_min = -wave_max_f32(mine ? -a : -INFINITY);
    const float z = mine ? expf(a_min - a) * q : 0.0f;
    const float sum = dpp_sum_f32(z);
    return mine ? z / sum : 0.0f;
  }
  if (renorm) {
    const float top = wave_max_f32(mine ? l : -INFINITY);
    const float z = mine ? expf(l - top) : 0.0f;
    const float sum = dpp_sum_f32(z);
    return mine ? z / sum : 0.0f;
  }
  return mine ? expf(l - row_max) / row_sum : 0.0f;
}

template <int NPL>
MOE_DEV void row_softmax_stats(const float (&l)[NPL], float& top, float& sum) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    if (present(l[i])) m = l[i] > m ? l[i] : m;
  top = wave_max_f32(m);
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) z += present(l[i]) ? expf(l[i] - top) : 0.0f;
  sum = dpp_sum_f32(z);
}

// MODE 0: the logits decide; 1, 2: choice values of sigmoid, softmax scores, in double.  A
// choice that rounds is a choice that may differ: near the border of the top k two fp32
// scores are often equal where the scores are not.  Without bias and groups both score
// functions keep the order of the logits, which then decide, exactly, without forming a
// score.
// Bound by the vector unit, not by memory: 8192 tokens of 256 experts in 8 groups, k = 8,
// take 12 us for 8.9 MB and 707 vector instructions a token, 150 of them in 64 bits at half
// rate, whose issue alone is about 11 us (8 wavefronts a SIMD).  One token: 4.5 us, of which the launch is half and the rest a
// chain (row, exp, group scores, k maxima of 64 lanes).  Row shifts for the maxima instead
// of a round trip through LDS a step, lanes sorted once so that a round looks at one key of
// each, and the vectorised exp took it there from 20 us (and 7.6 us); scalar maxima across
// the rows and a shift for a lane's group saved 60 instructions of 766.
template <int NPL, int MODE>
__global__ __launch_bounds__(256) void route_scored_kernel(const float* __restrict__ logits,
                                                           const float* __restrict__ bias, int T,
                                                           int E, int k, ScoreArgs sc, bool vec,
                                                           int32_t* __restrict__ topk_idx,
                                                           float* __restrict__ topk_w) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wv;
  constexpr bool BY_VALUE = MODE != 0;
  __shared__ double lds_c[BY_VALUE ? 4 : 1][BY_VALUE ? 64 * NPL : 1];
  if (t >= T) return;  // no workgroup barrier below
  const float* L = logits + (size_t)t * E;
  float l[NPL];
  load_row<NPL>(L, E, lane, vec, l);
  unsigned long long key[NPL];
  if constexpr (BY_VALUE) {
    float b[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) b[i] = 0.0f;
    if (bias) load_row<NPL>(bias, E, lane, vec, b);
    double c[NPL];
    if constexpr (MODE == 1) {  // e / (1 + e) or 1 / (1 + e), e = exp(-|l|)
      double e[NPL];
#pragma unroll
      for (int i = 0; i < NPL; ++i) e[i] = -fabs((double)l[i]);
      exp_neg<NPL>(e);
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const double q = recip(1.0 + e[i]), eq = e[i] * q;
        c[i] = l[i] < 0.0f ? eq : q;
      }
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < NPL; ++i) m = max_u(m, present(l[i]) ? ordered_u32(l[i]) : 0u);
      const double top = (double)from_ordered_u32(wave_max_u32(m));
#pragma unroll
      for (int i = 0; i < NPL; ++i) c[i] = present(l[i]) ? (double)l[i] - top : -1e9;
      exp_neg<NPL>(c);
      double z = 0.0;
#pragma unroll
      for (int i = 0; i < NPL; ++i) z += c[i];
      z = wave_sum_f64(z);
#pragma unroll
      for (int i = 0; i < NPL; ++i) c[i] /= z;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      c[i] += (double)b[i];
      if (!present(l[i])) c[i] = -INFINITY;
    }
    bool kept_all[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) kept_all[i] = true;
    if (sc.n_groups > 1) {
      const int per = E / sc.n_groups;
      double b1 = -INFINITY, b2 = -INFINITY;  // the two largest of this lane's group
      if (sc.lanes) {
        // a group is a power of two of neighbouring lanes, at most a row of 16: merge the
        // lanes' best two with their mirror images (after the steps before, equal to xor)
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          b2 = fmax(b2, fmin(b1, c[i]));
          b1 = fmax(b1, c[i]);
        }
        if (sc.lanes > 1) merge2<0xb1>(b1, b2);    // lane ^ 1
        if (sc.lanes > 2) merge2<0x4e>(b1, b2);    // lane ^ 2
        if (sc.lanes > 4) merge2<0x141>(b1, b2);   // mirror in 8
        if (sc.lanes > 8) merge2<0x140>(b1, b2);   // mirror in 16
      } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) lds_c[wv][lane * NPL + i] = c[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (lane < sc.n_groups) {
#pragma unroll 4
          for (int i = 0; i < per; ++i) {
            const double v = lds_c[wv][lane * per + i];
            b2 = fmax(b2, fmin(b1, v));
            b1 = fmax(b1, v);
          }
        }
      }
      const double gs = (sc.group_top == 2 && b2 > -INFINITY) ? b1 + b2 : b1;
      // lane g * step scores group g; step is a power of two
      const int step = sc.lanes ? sc.lanes : 1, me = lane >> __builtin_ctz(step);
      int better = 0;
      for (int g = 0; g < sc.n_groups; ++g) {
        const double o = __hiloint2double(lane_i(__double2hiint(gs), g * step),
                                          lane_i(__double2loint(gs), g * step));
        better += o > gs ? 1 : 0;
        better += o == gs && g < me ? 1 : 0;
      }
      const bool keep = better < sc.topk_groups;
      if (sc.lanes) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) kept_all[i] = keep;
      } else {
        const unsigned long long kept = ballot64(lane < sc.n_groups && keep);
#pragma unroll
        for (int i = 0; i < NPL; ++i) kept_all[i] = (kept >> (((lane * NPL + i) / per) & 63)) & 1ull;
      }
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const bool in = lane * NPL + i < E && present(l[i]) && kept_all[i];
      key[i] = in ? ordered_f64(c[i]) : 0ull;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) key[i] = present(l[i]) ? ordered_f32(l[i]) : 0ull;
  }

  // Up to 4 a lane: sorted once, by neighbours only, so that equal keys keep their order.
  // The heads' high words then take part in the choice; a lane's order is 4 bits an entry of
  // `order`, and its low words stay where they are (they are read where high words tie).
  constexpr bool SORTED = NPL <= 4;
  uint32_t order = 0x3210u, head[NPL];
  if constexpr (SORTED) {
    uint32_t at[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) at[i] = i;
#pragma unroll
    for (int r = 0; r < NPL; ++r)
#pragma unroll
      for (int i = r & 1; i + 1 < NPL; i += 2) {
        const bool sw = key[i] < key[i + 1];
        const unsigned long long ka = key[i], kb = key[i + 1];
        const uint32_t ia = at[i], ib = at[i + 1];
        key[i] = sw ? kb : ka;
        key[i + 1] = sw ? ka : kb;
        at[i] = sw ? ib : ia;
        at[i + 1] = sw ? ia : ib;
      }
    order = 0u;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      order |= at[i] << (4 * i);
      head[i] = (uint32_t)(key[i] >> 32);
    }
  }
  // k times the largest key: its high word by a wavefront maximum, its low word only
  // among the lanes that tie there, then the lowest lane
  int my_e = -1;
  uint32_t popped = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t hi, lo = 0, bi = order & 15u;
    if constexpr (SORTED) {
      hi = head[0];
    } else {
      unsigned long long best = key[0];
      bi = 0;
#pragma unroll
      for (int i = 1; i < NPL; ++i)
        if (key[i] > best) {
          best = key[i];
          bi = i;
        }
      hi = (uint32_t)(best >> 32);
      lo = (uint32_t)best;
    }
    const uint32_t m = wave_max_u32(hi);
    if (m == 0u) break;  // nothing left to choose
    unsigned long long tie = ballot64(hi == m);
    if (BY_VALUE && (tie & (tie - 1ull))) {
      if constexpr (SORTED) {
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          if (popped == (uint32_t)i) lo = (uint32_t)key[i];
      }
      lo = hi == m ? lo : 0u;
      const uint32_t ml = wave_max_u32(lo);
      tie = ballot64(hi == m && lo == ml);
    }
    const int win = __builtin_ctzll(tie);
    const int wi = lane_i((int)bi, win);
    if (lane == j) my_e = win * NPL + wi;
    if (lane == win) {
      if constexpr (SORTED) {
#pragma unroll
        for (int i = 0; i + 1 < NPL; ++i) head[i] = head[i + 1];
        head[NPL - 1] = 0u;
        order >>= 4;
        ++popped;
      } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          if (i == wi) key[i] = 0ull;
      }
    }
  }
  const float my_l = my_e >= 0 ? L[my_e] : 0.0f;

  float row_max = 0.0f, row_sum = 1.0f;
  if (sc.score == 0 && !sc.renormalise) row_softmax_stats<NPL>(l, row_max, row_sum);
  const float p = chosen_score(sc.score, sc.renormalise != 0, my_e >= 0, my_l, row_max, row_sum);
  if (lane < k) {
    topk_idx[(size_t)t * k + lane] = my_e;
    topk_w[(size_t)t * k + lane] = sc.scale * p;
  }
}

// d_logits from the gradient of the weights, with p the normalised scores and g_j =
// scale dw_j:
//   renormalised           p_j (g_j - sum_i p_i g_i) for chosen experts, times 1 - s_j for
//                          sigmoid scores; 0 elsewhere
//   sigmoid                g_j s_j (1 - s_j); 0 elsewhere
//   softmax                s_e (g_e - sum_i s_i g_i) for every expert, g = 0 off the choice
// The row is put together in LDS and written once.  8192 x 256, k = 8: 6.8 us for 8.9 MB (a
// chain as above: the choice, its logits, the sums, the row).
template <int NPL>
__global__ __launch_bounds__(256) void route_scored_backward_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
    const float* __restrict__ d_topk_w, int T, int E, int k, ScoreArgs sc, bool vec,
    float* __restrict__ d_logits) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wv;
  __shared__ __attribute__((aligned(16))) float row[4][64 * NPL];
  if (t >= T) return;  // no workgroup barrier below
  const float* L = logits + (size_t)t * E;
  const bool dense = sc.score == 0 && !sc.renormalise;
  int e = -1;
  float g = 0.0f, l = 0.0f;
  if (lane < k) {
    e = topk_idx[(size_t)t * k + lane];
    if ((uint32_t)e >= (uint32_t)E) e = -1;  // a slot without an expert
    if (e >= 0) {
      g = sc.scale * d_topk_w[(size_t)t * k + lane];
      l = L[e];
    }
  }
  const bool mine = e >= 0 && present(l);
  float lr[NPL], top = 0.0f, sum = 1.0f;
  if (dense) {
    load_row<NPL>(L, E, lane, vec, lr);
    row_softmax_stats<NPL>(lr, top, sum);
  }
  const float p = chosen_score(sc.score, sc.renormalise != 0, mine, l, top, sum);
  const float pg = mine ? p * g : 0.0f;
  const float dot = (dense || sc.renormalise) ? dpp_sum_f32(pg) : 0.0f;
  float v = mine ? (dense ? pg : p * (g - dot)) : 0.0f;
  if (sc.score == 1 && mine) {
    float a, q;
    sigmoid_parts(-l, a, q);
    v *= expf(-a) * q;  // 1 - sigmoid(l)
  }
  // an id that a row holds twice gets the sum of its slots, written by the first
  float tot = 0.0f;
  bool first = mine;
  for (int j = 0; j < k; ++j) {
    const int ej = lane_i(e, j);
    const float vj = lane_f(v, j);
    if (ej == e) {
      tot += vj;
      if (j < lane) first = false;
    }
  }
  float* out = row[wv];
#pragma unroll
  for (int i = 0; i < NPL; ++i) out[lane * NPL + i] = 0.0f;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (first) out[e] = tot;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  float* dst = d_logits + (size_t)t * E;
  float o[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    o[i] = out[lane * NPL + i];
    if (dense && present(lr[i])) o[i] -= expf(lr[i] - top) / sum * dot;
  }
  const int e0 = lane * NPL;
  if (vec) {
    constexpr int V = NPL < 4 ? NPL : 4;
#pragma unroll
    for (int i = 0; i < NPL; i += V) {
      if (e0 + i >= E) break;
      if constexpr (V == 4) *(float4*)(dst + e0 + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
      else if constexpr (V == 2) *(float2*)(dst + e0 + i) = make_float2(o[i], o[i + 1]);
      else dst[e0 + i] = o[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (e0 + i < E) dst[e0 + i] = o[i];
  }
}

// experts per lane: the smallest power of two that covers E
int experts_per_lane(int E) {
  int n = 1;
  while (64 * n < E) n *= 2;
  return n;
}

}  // namespace

template <int NPL>
static hipError_t route_scored_n(const float* logits, const float* bias, int T, int E, int k,
                                 ScoreArgs sc, int32_t* idx, float* w, hipStream_t s) {
  const bool vec = E % (NPL < 4 ? NPL : 4) == 0;
  // lanes of a group, where a group is 1, 2, 4, 8 or 16 whole lanes (0: it is not)
  const int per = E / sc.n_groups, lanes = per / NPL;
  sc.lanes = per % NPL == 0 && lanes <= 16 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  const unsigned grid = (unsigned)((T + 3) / 4);
#define MOE_ROUTE_SCORED(MODE) \
  MOE_LAUNCH("route_scored", s, route_scored_kernel<NPL, MODE><<<grid, 256, 0, s>>>(logits, bias, T, E, k, sc, vec, idx, w))
  if (!bias && sc.n_groups == 1) return MOE_ROUTE_SCORED(0);
  if (sc.score == 1) return MOE_ROUTE_SCORED(1);
  return MOE_ROUTE_SCORED(2);
#undef MOE_ROUTE_SCORED
}

hipError_t launch_route_scored(const float* logits, const float* bias, int T, int E, int k,
                               const ScoreArgs& sc, int32_t* idx, float* w, hipStream_t s) {
  if (T == 0) return hipSuccess;
  switch (experts_per_lane(E)) {
    case 1: return route_scored_n<1>(logits, bias, T, E, k, sc, idx, w, s);
    case 2: return route_scored_n<2>(logits, bias, T, E, k, sc, idx, w, s);
    case 4: return route_scored_n<4>(logits, bias, T, E, k, sc, idx, w, s);
    case 8: return route_scored_n<8>(logits, bias, T, E, k, sc, idx, w, s);
    default: return route_scored_n<16>(logits, bias, T, E, k, sc, idx, w, s);
  }
}

template <int NPL>
static hipError_t route_scored_backward_n(const float* logits, const int32_t* idx, const float* dw,
                                          int T, int E, int k, const ScoreArgs& sc, float* dL,
                                          hipStream_t s) {
  const bool vec = E % (NPL < 4 ? NPL : 4) == 0;
  return MOE_LAUNCH("route_scored_backward", s,
                    route_scored_backward_kernel<NPL><<<(unsigned)((T + 3) / 4), 256, 0, s>>>(
                        logits, idx, dw, T, E, k, sc, vec, dL));
}

hipError_t launch_route_scored_backward(const float* logits, const int32_t* idx, const float* dw,
                                        int T, int E, int k, const ScoreArgs& sc, float* dL,
                                        hipStream_t s) {
  if (T == 0) return hipSuccess;
  switch (experts_per_lane(E)) {
    case 1: return route_scored_backward_n<1>(logits, idx, dw, T, E, k, sc, dL, s);
    case 2: return route_scored_backward_n<2>(logits, idx, dw, T, E, k, sc, dL, s);
    case 4: return route_scored_backward_n<4>(logits, idx, dw, T, E, k, sc, dL, s);
    case 8: return route_scored_backward_n<8>(logits, idx, dw, T, E, k, sc, dL, s);
    default: return route_scored_backward_n<16>(logits, idx, dw, T, E, k, sc, dL, s);
  }
}

}  // namespace moe
