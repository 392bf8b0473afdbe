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

namespace moe {
namespace {

template <int CTRL, int ROWS>
MOE_DEV uint32_t dpp_max_step(uint32_t v) {
  // lanes without a source keep their own value
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, ROWS, 0xf, false);
  return o > v ? o : v;
}

// Largest value of the wavefront, in every lane: row shifts by 1, 2, 4, 8 leave each
// 16-lane row's maximum in its last lane, two broadcasts carry it to lane 63.
MOE_DEV uint32_t wave_max_u32(uint32_t v) {
  v = dpp_max_step<0x111, 0xf>(v);
  v = dpp_max_step<0x112, 0xf>(v);
  v = dpp_max_step<0x114, 0xf>(v);
  v = dpp_max_step<0x118, 0xf>(v);
  v = dpp_max_step<0x142, 0xa>(v);
  v = dpp_max_step<0x143, 0xc>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

MOE_DEV float wave_max_f32(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

MOE_DEV double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
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
    const float sum = wave_sum_f32(z);
    return mine ? z / sum : 0.0f;
  }
  if (renorm) {
    const float top = wave_max_f32(mine ? l : -INFINITY);
    const float z = mine ? expf(l - top) : 0.0f;
    const float sum = wave_sum_f32(z);
    return mine ? z / sum : 0.0f;
  }
  return mine ? expf(l - row_max) / row_sum : 0.0f;
}

template <int NPL>
MOE_DEV void row_softmax_stats(const float (&l)[NPL], float& top, float& sum) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    if (present(l[i])) m = fmaxf(m, l[i]);
  top = wave_max_f32(m);
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    if (present(l[i])) z += expf(l[i] - top);
  sum = wave_sum_f32(z);
}

// BY_VALUE: choice values are formed in double.  A choice that rounds is a choice that
// may differ: near the border of the top k two fp32 scores are often equal where the
// scores are not.  Without bias and groups both score functions keep the order of the
// logits, which then decide, exactly, without forming a score.
template <int NPL, bool BY_VALUE>
__global__ __launch_bounds__(256) void route_scored_kernel(const float* __restrict__ logits,
                                                           const float* __restrict__ bias, int T,
                                                           int E, int k, ScoreArgs sc, bool vec,
                                                           int32_t* __restrict__ topk_idx,
                                                           float* __restrict__ topk_w) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wv;
  __shared__ double lds_c[BY_VALUE ? 4 : 1][BY_VALUE ? 64 * NPL : 1];
  if (t >= T) return;  // no workgroup barrier below
  const float* L = logits + (size_t)t * E;
  float l[NPL];
  load_row<NPL>(L, E, lane, vec, l);
  unsigned long long key[NPL];
  if constexpr (BY_VALUE) {
    double c[NPL];
    if (sc.score == 1) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) c[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    } else {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (present(l[i])) m = fmaxf(m, l[i]);
      m = wave_max_f32(m);
      double z = 0.0;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        c[i] = present(l[i]) ? exp((double)l[i] - (double)m) : 0.0;
        z += c[i];
      }
      z = wave_sum_f64(z);
#pragma unroll
      for (int i = 0; i < NPL; ++i) c[i] /= z;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane * NPL + i;
      if (bias && e < E) c[i] += (double)bias[e];
      if (!present(l[i])) c[i] = -INFINITY;
    }
    unsigned long long kept = ~0ull;
    const int per = E / sc.n_groups;
    if (sc.n_groups > 1) {
      // lane g scores group g
#pragma unroll
      for (int i = 0; i < NPL; ++i) lds_c[wv][lane * NPL + i] = c[i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      double b1 = -INFINITY, b2 = -INFINITY;
      if (lane < sc.n_groups) {
        for (int i = 0; i < per; ++i) {
          const double v = lds_c[wv][lane * per + i];
          if (v > b1) {
            b2 = b1;
            b1 = v;
          } else if (v > b2) {
            b2 = v;
          }
        }
      }
      const double gs = (sc.group_top == 2 && b2 > -INFINITY) ? b1 + b2 : b1;
      const unsigned long long gk = ordered_f64(gs);
      int better = 0;
      for (int g = 0; g < sc.n_groups; ++g) {
        const unsigned long long o =
            ((unsigned long long)(uint32_t)lane_i((int)(uint32_t)(gk >> 32), g) << 32) |
            (uint32_t)lane_i((int)(uint32_t)gk, g);
        better += (o > gk || (o == gk && g < lane)) ? 1 : 0;
      }
      kept = ballot64(lane < sc.n_groups && better < sc.topk_groups);
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane * NPL + i;
      const int g = sc.n_groups > 1 ? e / per : 0;
      const bool in = e < E && present(l[i]) && ((kept >> (g & 63)) & 1ull);
      key[i] = in ? ordered_f64(c[i]) : 0ull;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) key[i] = present(l[i]) ? ordered_f32(l[i]) : 0ull;
  }

  // k times the largest key: its high word by a wavefront maximum, its low word only
  // among the lanes that tie there, then the lowest lane
  int my_e = -1;
  float my_l = 0.0f;
  for (int j = 0; j < k; ++j) {
    unsigned long long best = key[0];
    int bi = 0;
    float bl = l[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i)
      if (key[i] > best) {
        best = key[i];
        bi = i;
        bl = l[i];
      }
    const uint32_t hi = (uint32_t)(best >> 32);
    const uint32_t m = wave_max_u32(hi);
    if (m == 0u) break;  // nothing left to choose
    unsigned long long tie = ballot64(hi == m);
    if (BY_VALUE && (tie & (tie - 1ull))) {
      const uint32_t lo = hi == m ? (uint32_t)best : 0u;
      const uint32_t ml = wave_max_u32(lo);
      tie = ballot64(hi == m && lo == ml);
    }
    const int win = __ffsll((long long)tie) - 1;
    const int wi = lane_i(bi, win);
    const float wl = lane_f(bl, win);
    if (lane == j) {
      my_e = win * NPL + wi;
      my_l = wl;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (lane == win && i == wi) key[i] = 0ull;
  }

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
// The row is put together in LDS and written once.
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
  const float dot = (dense || sc.renormalise) ? wave_sum_f32(pg) : 0.0f;
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
                                 const ScoreArgs& sc, int32_t* idx, float* w, hipStream_t s) {
  const bool vec = E % (NPL < 4 ? NPL : 4) == 0;
  const unsigned grid = (unsigned)((T + 3) / 4);
  if (bias || sc.n_groups > 1)
    return MOE_LAUNCH("route_scored", s,
                      route_scored_kernel<NPL, true><<<grid, 256, 0, s>>>(logits, bias, T, E, k, sc,
                                                                          vec, idx, w));
  return MOE_LAUNCH("route_scored", s,
                    route_scored_kernel<NPL, false><<<grid, 256, 0, s>>>(logits, bias, T, E, k, sc,
                                                                         vec, idx, w));
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
