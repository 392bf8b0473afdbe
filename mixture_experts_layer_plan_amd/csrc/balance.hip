// The balance loss of the router's scores and the experts' counts, per sequence, and the
// gradient of the logits.
//
// For a token t of sequence i with at least one expert, p_te = softmax(l_t)_e or
// sigmoid(l_te) / sum_j sigmoid(l_tj); with N_i such tokens and c_ie pairs of expert e,
//   loss = coef / n sum_i E / (k N_i^2) sum_e c_ie sum_t p_te,  n = sequences with tokens
//   d l_te = s_i p_te (c_ie - sum_j p_tj c_ij) (1 - sigmoid(l_te) for sigmoid scores),
//   s_i = coef E / (k N_i^2 n)
// An expert whose logit is -inf or NaN has p = 0 and no gradient.
//
// One wavefront per token, lane l holding the experts l, l + 64, ...  Workgroups sum the
// tokens of one chunk, segment by segment; a second launch adds a sequence's segments in
// their order, its last workgroup joining the sequences.
#include <math.h>

#include "common.hpp"
#include "internal.hpp"
#include "step.hpp"
#include "wave.hpp"

namespace moe {
namespace {

// The last i in [0, n] with start[i] <= t (entries ascend), n for a token behind the last
// sequence, -1 for one before the first.  64 entries a step; every lane gets the result,
// which lies in [-1, n] whatever the entries hold.
MOE_DEV int sequence_of(const int32_t* start, int n, int t) {
  if (!start) return t < 0 ? -1 : 0;
  int lo = -1, hi = n + 1;  // start[lo] <= t < start[hi], with -inf and inf at the ends
  while (hi - lo > 1) {
    const int step = (hi - lo - 1 + 63) / 64;
    const int i = lo + (lane_id() + 1) * step;
    const bool le = i < hi && start[i] <= t;
    const int ones = __popcll(ballot64(le));
    const int nlo = lo + ones * step;
    const int nhi = lo + (ones + 1) * step;
    hi = nhi < hi ? nhi : hi;
    lo = nlo;
  }
  return lo;
}

// Scores of one token: p (normalised) and, for sigmoid, q = 1 - sigmoid.  An expert out of
// play has p = 0.  The largest exponent is 0, so that neither overflows or all vanish.
template <int NPL, bool SIGMOID>
MOE_DEV void scores(const float* l, float* p, float* q) {
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < NPL; ++j) top = fmaxf(top, l[j]);  // fmaxf leaves NaN out
  top = wave_max_f32(top);
  if (SIGMOID) top = fminf(top, 0.0f);
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < NPL; ++j) {
    const bool in = l[j] > -INFINITY;
    if (SIGMOID) {
      // e^(l - top) / (1 + e^l) where l <= 0, else 1 / (1 + e^-l) e^-top with top = 0
      const float e = expf(-fabsf(l[j]));
      const float r = 1.0f / (1.0f + e);
      p[j] = in ? (l[j] > 0.0f ? r : expf(l[j] - top) * r) : 0.0f;
      q[j] = l[j] > 0.0f ? e * r : r;
    } else {
      p[j] = in ? expf(l[j] - top) : 0.0f;
    }
    sum += p[j];
  }
  sum = dpp_sum_f32(sum);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int j = 0; j < NPL; ++j) p[j] *= inv;
}

template <int NPL>
MOE_DEV void load_row(const float* row, int E, float* l) {
#pragma unroll
  for (int j = 0; j < NPL; ++j) {
    const int e = j * 64 + lane_id();
    l[j] = e < E ? row[e] : -INFINITY;
  }
}

template <int NPL, bool SIGMOID>
__global__ __launch_bounds__(256) void balance_part_kernel(BalanceArgs a, int chunk) {
  extern __shared__ float s_mem[];
  float* s_p = s_mem;                       // [4][E]
  int32_t* s_c = (int32_t*)(s_mem + 4 * a.E);  // [E]
  __shared__ int s_n[4];
  const int wave = threadIdx.x >> 6, lane = lane_id();
  if (blockIdx.x == 0 && threadIdx.x == 0) a.ticket[0] = 0;  // for the launch that follows
  const int t0 = blockIdx.x * chunk;
  const int t1 = t0 + chunk < a.T ? t0 + chunk : a.T;
  int t = t0;
  while (t < t1) {
    // the tokens [t, end) of the chunk that are in t's sequence
    const int seq = sequence_of(a.start, a.n_seq, t);
    if (seq >= a.n_seq) break;  // behind the last one
    int end = t1;
    if (a.start) {
      const int next = a.start[seq + 1];
      end = next < t1 ? next : t1;
      if (end <= t) end = t1;  // entries that do not ascend: no endless loop
    }
    if (seq < 0) {  // before the first sequence
      t = end;
      continue;
    }
    for (int e = threadIdx.x; e < a.E; e += 256) s_c[e] = 0;
    __syncthreads();
    float acc[NPL];
#pragma unroll
    for (int j = 0; j < NPL; ++j) acc[j] = 0.0f;
    int used = 0;
    for (int u = t + wave; u < end; u += 4) {
      const int id = lane < a.k ? a.idx[(size_t)u * a.k + lane] : -1;
      const bool ok = (unsigned)id < (unsigned)a.E;
      float l[NPL], p[NPL], q[NPL];
      load_row<NPL>(a.logits + (size_t)u * a.E, a.E, l);
      if (ok) atomicAdd(&s_c[id], 1);
      if (!ballot64(ok)) continue;
      ++used;
      scores<NPL, SIGMOID>(l, p, q);
#pragma unroll
      for (int j = 0; j < NPL; ++j) acc[j] += p[j];
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      const int e = j * 64 + lane;
      if (e < a.E) s_p[wave * a.E + e] = acc[j];
    }
    if (lane == 0) s_n[wave] = used;
    __syncthreads();
    const size_t seg = (size_t)blockIdx.x + seq;
    for (int e = threadIdx.x; e < a.E; e += 256) {
      a.seg_p[seg * a.E + e] = (s_p[e] + s_p[a.E + e]) + (s_p[2 * a.E + e] + s_p[3 * a.E + e]);
      a.seg_c[seg * a.E + e] = s_c[e];
    }
    if (threadIdx.x == 0) a.seg_n[seg] = s_n[0] + s_n[1] + s_n[2] + s_n[3];
    __syncthreads();
    t = end;
  }
}

// Adds the segments of sequence blockIdx.x / blocks for 64 experts: 16 wavefronts take
// every 16th chunk each.  The last workgroup to finish joins the sequences.
__global__ __launch_bounds__(1024) void balance_join_kernel(BalanceArgs a, int chunk, int blocks) {
  __shared__ float s_p[16][64];
  __shared__ int s_c[16][64], s_n[16];
  __shared__ int s_last;
  const int seq = blockIdx.x / blocks, blk = blockIdx.x - seq * blocks;
  const int wave = threadIdx.x >> 6, lane = lane_id();
  const int e = blk * 64 + lane;
  int b = a.start ? a.start[seq] : 0, end = a.start ? a.start[seq + 1] : a.T;
  b = b > 0 ? b : 0;
  end = end < a.T ? end : a.T;
  float p = 0.0f;
  int c = 0, n = 0;
  if (b < end) {
    const int c1 = (end - 1) / chunk;
    for (int i = b / chunk + wave; i <= c1; i += 16) {
      const size_t seg = (size_t)i + seq;
      if (e < a.E) {
        p += a.seg_p[seg * a.E + e];
        c += a.seg_c[seg * a.E + e];
      }
      n += a.seg_n[seg];
    }
  }
  s_p[wave][lane] = p;
  s_c[wave][lane] = c;
  if (lane == 0) s_n[wave] = n;
  __syncthreads();
  if (wave == 0) {
    for (int w = 1; w < 16; ++w) {
      p += s_p[w][lane];
      c += s_c[w][lane];
      n += s_n[w];
    }
    if (e < a.E) a.counts[(size_t)seq * a.E + e] = c;
    const float x = dpp_sum_f32(e < a.E ? p * (float)c : 0.0f);
    if (lane == 0) {
      a.part[(size_t)seq * blocks + blk] = x;
      if (blk == 0) a.tokens[seq] = n;
      __threadfence();
      s_last = atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // n and the loss, in 64 bits; a thread takes every 1024th sequence
  __shared__ double s_loss[16];
  __shared__ int s_seq[16];
  int have = 0;
  double loss = 0.0;
  const double per = (double)a.coef * a.E / a.k;
  for (int i = threadIdx.x; i < a.n_seq; i += 1024) {
    const int N = a.tokens[i];
    if (N > 0) {
      ++have;
      double x = 0.0;
      for (int k = 0; k < blocks; ++k) x += (double)a.part[(size_t)i * blocks + k];
      loss += per / ((double)N * N) * x;
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    loss += __shfl_xor(loss, o, 64);
    have += __shfl_xor(have, o, 64);
  }
  if (lane == 0) {
    s_loss[wave] = loss;
    s_seq[wave] = have;
  }
  __syncthreads();
  loss = 0.0;
  have = 0;
  for (int w = 0; w < 16; ++w) {
    loss += s_loss[w];
    have += s_seq[w];
  }
  const double each = have ? 1.0 / have : 0.0;
  if (threadIdx.x == 0) a.loss[0] = (float)(loss * each);
  for (int i = threadIdx.x; i < a.n_seq; i += 1024) {
    const int N = a.tokens[i];
    a.scales[i] = N > 0 ? (float)(per * each / ((double)N * N)) : 0.0f;
  }
}

template <int NPL, bool SIGMOID>
__global__ __launch_bounds__(256) void balance_backward_kernel(BalanceArgs a) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const int lane = lane_id();
  const int seq = sequence_of(a.start, a.n_seq, t);
  const int id = lane < a.k ? a.idx[(size_t)t * a.k + lane] : -1;
  const bool used = ballot64((unsigned)id < (unsigned)a.E) && seq >= 0 && seq < a.n_seq;
  float d[NPL];
#pragma unroll
  for (int j = 0; j < NPL; ++j) {
    const int e = j * 64 + lane;
    d[j] = a.d_in && e < a.E ? a.d_in[(size_t)t * a.E + e] : 0.0f;
  }
  if (used) {
    float l[NPL], p[NPL], q[NPL], c[NPL];
    load_row<NPL>(a.logits + (size_t)t * a.E, a.E, l);
    float dot = 0.0f;
    scores<NPL, SIGMOID>(l, p, q);
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      const int e = j * 64 + lane;
      c[j] = e < a.E ? (float)a.counts[(size_t)seq * a.E + e] : 0.0f;
      dot = fmaf(p[j], c[j], dot);
    }
    dot = dpp_sum_f32(dot);
    const float scale = a.scales[seq] * (a.d_loss ? a.d_loss[0] : 1.0f);
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      const float g = p[j] * (c[j] - dot) * (SIGMOID ? q[j] : 1.0f);
      d[j] = l[j] > -INFINITY ? fmaf(scale, g, d[j]) : d[j];
    }
  }
#pragma unroll
  for (int j = 0; j < NPL; ++j) {
    const int e = j * 64 + lane;
    if (e < a.E) a.d_logits[(size_t)t * a.E + e] = d[j];
  }
}

template <int NPL>
hipError_t part_as(const BalanceArgs& a, int chunk, int grid, hipStream_t s) {
  const size_t lds = (size_t)a.E * 5 * 4;
  if (a.sigmoid)
    return MOE_LAUNCH("balance_part", s,
                      balance_part_kernel<NPL, true><<<grid, 256, lds, s>>>(a, chunk));
  return MOE_LAUNCH("balance_part", s,
                    balance_part_kernel<NPL, false><<<grid, 256, lds, s>>>(a, chunk));
}
template <int NPL>
hipError_t back_as(const BalanceArgs& a, hipStream_t s) {
  const int grid = (a.T + 3) / 4;
  if (a.sigmoid)
    return MOE_LAUNCH("balance_backward", s,
                      balance_backward_kernel<NPL, true><<<grid, 256, 0, s>>>(a));
  return MOE_LAUNCH("balance_backward", s,
                    balance_backward_kernel<NPL, false><<<grid, 256, 0, s>>>(a));
}

}  // namespace

int balance_chunk(int T) {
  const int c = (T + 511) / 512;
  return c < 16 ? 16 : (c + 15) / 16 * 16;
}

hipError_t launch_balance(const BalanceArgs& a, hipStream_t s) {
  const int chunk = balance_chunk(a.T);
  // one workgroup at least: the second launch needs the ticket that the first one clears
  const int grid = a.T > chunk ? (a.T + chunk - 1) / chunk : 1;
  hipError_t e;
  if (a.E <= 64) e = part_as<1>(a, chunk, grid, s);
  else if (a.E <= 128) e = part_as<2>(a, chunk, grid, s);
  else if (a.E <= 256) e = part_as<4>(a, chunk, grid, s);
  else if (a.E <= 512) e = part_as<8>(a, chunk, grid, s);
  else e = part_as<16>(a, chunk, grid, s);
  if (e != hipSuccess) return e;
  const int blocks = (a.E + 63) / 64;
  return MOE_LAUNCH("balance_join", s,
                    balance_join_kernel<<<a.n_seq * blocks, 1024, 0, s>>>(a, chunk, blocks));
}

hipError_t launch_balance_backward(const BalanceArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  if (a.E <= 64) return back_as<1>(a, s);
  if (a.E <= 128) return back_as<2>(a, s);
  if (a.E <= 256) return back_as<4>(a, s);
  if (a.E <= 512) return back_as<8>(a, s);
  return back_as<16>(a, s);
}

}  // namespace moe
