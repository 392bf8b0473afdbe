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
// A wavefront takes a token's row, U tokens at a time.  Workgroups sum the tokens of one
// chunk, segment by segment; a second launch adds a sequence's segments in their order, its
// last workgroup joining the sequences.  A small batch takes one launch of one workgroup.
#include <math.h>

#include <algorithm>

#include "common.hpp"
#include "internal.hpp"
#include "step.hpp"
#include "wave.hpp"

namespace moe {
namespace {

constexpr int PART_W = 8;  // wavefronts of a chunk's workgroup

// A barrier for what lies in LDS alone: stores to memory stay under way (__syncthreads waits
// for them too, a microsecond a sequence here).
MOE_DEV void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The last i in [0, n] with start[i] <= t (entries ascend), n for a token behind the last
// sequence, -1 for one before the first; next: start[i + 1] (for i < n).  64 entries a step;
// every lane gets the result, which lies in [-1, n] whatever the entries hold.
MOE_DEV int sequence_of(const int32_t* start, int n, int t, int* next) {
  int lo = -1, hi = n + 1;  // start[lo] <= t < start[hi], with -inf and inf at the ends
  while (hi - lo > 1) {
    const int step = (hi - lo - 1 + 63) / 64;
    const int i = lo + (lane_id() + 1) * step;
    const int v = start[i < hi ? i : hi - 1];
    const int ones = __popcll(ballot64(i < hi && v <= t));
    const int nhi = lo + (ones + 1) * step;
    // the first entry above t, if this step read it
    *next = __builtin_amdgcn_readlane(v, ones < 63 ? ones : 63);
    if (ones > 63 || nhi >= hi) *next = hi <= n ? start[hi] : 0;
    hi = nhi < hi ? nhi : hi;
    lo += ones * step;
  }
  return lo;
}

// Looks up sequences; fewer than 64 have their starts read once, an entry a lane.
struct Sequences {
  const int32_t* start;
  int n, v;
  MOE_DEV Sequences(const BalanceArgs& a) : start(a.start), n(a.n_seq), v(INT_MAX) {
    if (start && n < 64 && lane_id() <= n) v = start[lane_id()];
  }
  // as sequence_of; without starts one sequence takes every token
  MOE_DEV int of(int t, int* next) const {
    *next = INT_MAX;
    if (!start) return 0;
    if (n >= 64) return sequence_of(start, n, t, next);
    const int ones = __popcll(ballot64(lane_id() <= n && v <= t));
    if (ones <= n) *next = __builtin_amdgcn_readlane(v, ones);
    return ones - 1;
  }
};

// How a row of E experts lies in the lanes of a wavefront: N values a lane, four
// neighbours a load (E a multiple of 4) or one; U rows at a time.
template <int N_, int U_, bool FOUR_>
struct Row {
  static constexpr int N = N_, U = U_;
  static constexpr bool FOUR = FOUR_;
  MOE_DEV static int expert(int j) {
    return FOUR ? ((j >> 2) * 64 + lane_id()) * 4 + (j & 3) : j * 64 + lane_id();
  }
  template <typename T>
  MOE_DEV static void load(const T* row, int E, T none, T* v) {
#pragma unroll
    for (int j = 0; j < N; j += FOUR ? 4 : 1) {
      const int e = expert(j);
      if constexpr (FOUR) {
        typedef T T4 __attribute__((ext_vector_type(4)));
        T4 x = {none, none, none, none};
        if (e < E) x = *(const T4*)(row + e);
        v[j] = x.x; v[j + 1] = x.y; v[j + 2] = x.z; v[j + 3] = x.w;
      } else {
        v[j] = e < E ? row[e] : none;
      }
    }
  }
  MOE_DEV static void store(float* row, int E, const float* v) {
#pragma unroll
    for (int j = 0; j < N; j += FOUR ? 4 : 1) {
      const int e = expert(j);
      if (e < E) {
        if constexpr (FOUR) *(float4*)(row + e) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        else row[e] = v[j];
      }
    }
  }
};

// e^x for |x| <= 200 or so: 2^(x log2 e) with the product's rounding carried along.
MOE_DEV float exp_near(float x) {
  const float h = x * 1.44269502f;
  const float lo = fmaf(x, 1.92596299e-8f, fmaf(x, 1.44269502f, -h));
  const float e = __builtin_amdgcn_exp2f(h);
  return fmaf(e, lo * 0.693147181f, e);
}

// Shares of one token whose logits are far from zero: exponents relative to the largest, so
// that they neither overflow nor all vanish.
template <int N, bool SIGMOID>
MOE_DEV void shares_far(const float (&l)[N], float (&p)[N]) {
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < N; ++j) top = fmaxf(top, l[j]);  // fmaxf leaves NaN out
  top = wave_max_f32(top);
  if (SIGMOID) top = fminf(top, 0.0f);
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float z = exp_near(fmaxf(l[j] - top, -200.0f));
    if (SIGMOID) {
      // e^(l - top) / (1 + e^l) where l <= 0, else 1 / (1 + e^-l) with top = 0
      const float r = __builtin_amdgcn_rcpf(1.0f + exp_near(fmaxf(-fabsf(l[j]), -200.0f)));
      z = l[j] > 0.0f ? r : z * r;
    }
    p[j] = l[j] > -INFINITY ? z : 0.0f;
    sum += p[j];
  }
  sum = dpp_sum_f32(sum);
  const float inv = sum > 0.0f ? __builtin_amdgcn_rcpf(sum) : 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) p[j] *= inv;
}

// Shares p of U tokens and, for sigmoid scores, q = 1 - sigmoid.  An expert out of play has
// p = 0.  Scores as they are, without the search for the largest, serve wherever their sum
// is far from the ends of fp32: the others are done again by shares_far.
template <typename R, bool SIGMOID>
MOE_DEV void shares(const float (&l)[R::U][R::N], float (&p)[R::U][R::N], float (&q)[R::U][R::N]) {
  float sum[R::U];
#pragma unroll
  for (int u = 0; u < R::U; ++u) {
    sum[u] = 0.0f;
#pragma unroll
    for (int j = 0; j < R::N; ++j) {
      const float v = l[u][j];
      float z;
      if (SIGMOID) {
        const float e = exp_near(fmaxf(-fabsf(v), -200.0f));
        const float r = __builtin_amdgcn_rcpf(1.0f + e), s = e * r;
        z = v > 0.0f ? r : s;
        q[u][j] = v > 0.0f ? s : r;
      } else {
        z = exp_near(fmaxf(v, -200.0f));
      }
      p[u][j] = v > -INFINITY ? z : 0.0f;
      sum[u] += p[u][j];
    }
  }
#pragma unroll
  for (int u = 0; u < R::U; ++u) sum[u] = dpp_sum_f32(sum[u]);
#pragma unroll
  for (int u = 0; u < R::U; ++u) {
    if (sum[u] > 0x1p-60f && sum[u] < 0x1p100f) {
      const float inv = __builtin_amdgcn_rcpf(sum[u]);
#pragma unroll
      for (int j = 0; j < R::N; ++j) p[u][j] *= inv;
    } else {
      shares_far<R::N, SIGMOID>(l[u], p[u]);
    }
  }
}

// The tokens [t0, t1) of a workgroup of W wavefronts, W * U at a time: their shares, summed
// sequence by sequence.  done(seq, n) is called for each sequence with its sums in LDS (s_p:
// one row of E per wavefront, s_c) and n, the number of its tokens that count, in every thread.
template <typename R, bool SIGMOID, int W, typename Done>
MOE_DEV void walk(const BalanceArgs& a, int t0, int t1, float* s_p, int32_t* s_c, int* s_n, Done done) {
  const int wave = threadIdx.x >> 6, lane = lane_id();
  const Sequences seqs(a);
  float acc[R::N];
  int used = 0, seq = -1, end = t0;  // the tokens [.., end) are in seq
  const auto close = [&]() {
    if (seq < 0) return;
    R::store(s_p + wave * a.E, a.E, acc);
    if (lane == 0) s_n[wave] = used;
    lds_barrier();
    int n = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) n += s_n[w];
    done(seq, n);
    lds_barrier();
  };
  for (int r0 = t0; r0 < t1; r0 += W * R::U) {
    const int r1 = r0 + W * R::U < t1 ? r0 + W * R::U : t1, w0 = r0 + wave * R::U;
    float l[R::U][R::N], p[R::U][R::N], q[R::U][R::N];
    int id[R::U];
#pragma unroll
    for (int u = 0; u < R::U; ++u) {
      const int v = w0 + u < r1 ? w0 + u : r1 - 1;
      id[u] = lane < a.k ? a.idx[(size_t)v * a.k + lane] : -1;
      R::load(a.logits + (size_t)v * a.E, a.E, -INFINITY, l[u]);
    }
    shares<R, SIGMOID>(l, p, q);
    for (int t = r0; t < r1;) {
      if (t >= end) {
        close();
        seq = seqs.of(t, &end);
        if (seq >= a.n_seq) return;          // behind the last one
        if (end <= t || end > t1) end = t1;  // (entries that do not ascend: no endless loop)
        if (seq >= 0) {
          for (int e = threadIdx.x; e < a.E; e += 64 * W) s_c[e] = 0;
          lds_barrier();
        }
        used = 0;
#pragma unroll
        for (int j = 0; j < R::N; ++j) acc[j] = 0.0f;
      }
      const int stop = end < r1 ? end : r1;
      if (seq >= 0) {  // (tokens before the first sequence are left out)
#pragma unroll
        for (int u = 0; u < R::U; ++u) {
          const bool ok = w0 + u >= t && w0 + u < stop && (unsigned)id[u] < (unsigned)a.E;
          if (ok) atomicAdd(&s_c[id[u]], 1);  // whole numbers: any order gives the same
          if (ballot64(ok)) {
            ++used;
#pragma unroll
            for (int j = 0; j < R::N; ++j) acc[j] += p[u][j];
          }
        }
      }
      t = stop;
    }
  }
  close();
}

template <int W>
MOE_DEV float rows_sum(const float* s_p, int E, int e) {
  float v = s_p[e];
#pragma unroll
  for (int w = 1; w < W; ++w) v += s_p[w * E + e];
  return v;
}

// The sums of one chunk, segment by segment.  32768 x 256 sigmoid: 12.6 us, 54 % of vector
// issue (529 instructions for a wavefront's four rows, 40 of them for each sigmoid) at 2.8 TB/s.
// Eight wavefronts: 32 tokens a chunk, whose sums are a sixteenth of the logits.
template <typename R, bool SIGMOID>
__global__ __launch_bounds__(64 * PART_W) void balance_part_kernel(BalanceArgs a, int chunk) {
  extern __shared__ float s_mem[];
  float* s_p = s_mem;                               // [PART_W][E]
  int32_t* s_c = (int32_t*)(s_mem + PART_W * a.E);  // [E]
  __shared__ int s_n[PART_W];
  if (blockIdx.x == 0 && threadIdx.x == 0) a.ticket[0] = 0;  // for the launch that follows
  const int t0 = blockIdx.x * chunk;
  const int t1 = t0 + chunk < a.T ? t0 + chunk : a.T;
  if (t0 >= t1) return;  // no tokens at all
  walk<R, SIGMOID, PART_W>(a, t0, t1, s_p, s_c, s_n, [&](int seq, int n) {
    const size_t seg = (size_t)blockIdx.x + seq;
    for (int e = threadIdx.x; e < a.E; e += 64 * PART_W) {
      a.seg_p[seg * a.E + e] = rows_sum<PART_W>(s_p, a.E, e);
      a.seg_c[seg * a.E + e] = s_c[e];
    }
    if (threadIdx.x == 0) a.seg_n[seg] = n;
  });
}

// Sum over W wavefronts in 64 bits, in every thread.
template <int W>
MOE_DEV double sum_f64(double v) {
  v = wave_sum_f64(v);
  if constexpr (W == 1) return v;
  __shared__ double slot[W];
  __syncthreads();
  if (lane_id() == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  v = slot[0];
#pragma unroll
  for (int w = 1; w < W; ++w) v += slot[w];
  return v;
}

// The loss and the scales from the sequences' tokens and sums of counts * p over `blocks`
// groups of experts, in 64 bits, by W wavefronts; a thread takes every (64 W)th sequence.
template <int W>
MOE_DEV void finish(const BalanceArgs& a, const int32_t* tokens, const float* part, int blocks) {
  double loss = 0.0, have = 0.0;
  const double per = (double)a.coef * a.E / a.k;
  for (int i = threadIdx.x; i < a.n_seq; i += 64 * W) {
    const int N = tokens[i];
    double x = 0.0;
#pragma unroll 4
    for (int k = 0; k < blocks; ++k) x += (double)part[(size_t)i * blocks + k];
    if (N > 0) {
      have += 1.0;
      loss += per / ((double)N * N) * x;
    }
  }
  loss = sum_f64<W>(loss);
  have = sum_f64<W>(have);
  const double each = have > 0.0 ? 1.0 / have : 0.0;
  if (threadIdx.x == 0) a.loss[0] = (float)(loss * each);
  for (int i = threadIdx.x; i < a.n_seq; i += 64 * W) {
    const int N = tokens[i];
    a.scales[i] = N > 0 ? (float)(per * each / ((double)N * N)) : 0.0f;
  }
}

// A batch of few tokens, whole, in one workgroup of 16 wavefronts: the tokens' shares and the
// sequences' counts in LDS, then a thread for each (sequence, expert).  One CU's vector issue
// sets its limits: 128 tokens of 64 experts take 7.9 us (two launches 8.4), 64 of 256 7.4 (9.2),
// and 128 of 256 would take 12.
constexpr int SMALL_T = 128, SMALL_E = 256, SMALL_SEQ = 64, SMALL_COUNTS = 4096;
constexpr int SMALL_SHARES = SMALL_T / 2 * SMALL_E;  // 64 KB; a row for each token, or for each wavefront
static_assert(SMALL_T * 64 <= SMALL_SHARES && 16 * SMALL_E <= SMALL_SHARES, "what is_small lets in");
bool is_small(const BalanceArgs& a) {
  return a.T <= (a.E <= 64 ? SMALL_T : SMALL_T / 2) && a.E <= SMALL_E && a.n_seq <= SMALL_SEQ && a.n_seq * a.E <= SMALL_COUNTS;
}
template <typename R, bool SIGMOID>
__global__ __launch_bounds__(1024) void balance_small_kernel(BalanceArgs a) {
  __shared__ float s_p[SMALL_SHARES];
  __shared__ int32_t s_c[SMALL_COUNTS];
  __shared__ float s_part[SMALL_SEQ];
  __shared__ int32_t s_seq[SMALL_T], s_tokens[SMALL_SEQ], s_start[SMALL_SEQ + 1];
  const int wave = threadIdx.x >> 6, lane = lane_id(), w0 = wave * R::U;
  float l[R::U][R::N], p[R::U][R::N], q[R::U][R::N];
  int id[R::U], seq[R::U];
  if (w0 < a.T) {
#pragma unroll
    for (int u = 0; u < R::U; ++u) {
      const int v = w0 + u < a.T ? w0 + u : a.T - 1;
      id[u] = lane < a.k && w0 + u < a.T ? a.idx[(size_t)v * a.k + lane] : -1;
      R::load(a.logits + (size_t)v * a.E, a.E, -INFINITY, l[u]);
    }
  }
  const Sequences seqs(a);
  const bool one = a.n_seq == 1;
  if ((int)threadIdx.x <= a.n_seq) {
    const int v = a.start ? a.start[threadIdx.x] : threadIdx.x ? a.T : 0;
    s_start[threadIdx.x] = v < 0 ? 0 : v < a.T ? v : a.T;
  }
  for (int i = threadIdx.x; i < a.n_seq * a.E; i += 1024) s_c[i] = 0;
  if (w0 < a.T) {
    shares<R, SIGMOID>(l, p, q);
#pragma unroll
    for (int u = 0; u < R::U; ++u) {
      if (w0 + u >= a.T) break;
      int end;
      seq[u] = seqs.of(w0 + u, &end);
      const bool used = ballot64((unsigned)id[u] < (unsigned)a.E) && seq[u] >= 0 && seq[u] < a.n_seq;
      if (!used) {
        seq[u] = -1;
#pragma unroll
        for (int j = 0; j < R::N; ++j) p[u][j] = 0.0f;
      }
      if (!one) R::store(s_p + (w0 + u) * a.E, a.E, p[u]);
      if (lane == 0) s_seq[w0 + u] = seq[u];
    }
  }
  if (one) {  // one row of sums for each wavefront
    float acc[R::N];
#pragma unroll
    for (int j = 0; j < R::N; ++j) acc[j] = 0.0f;
#pragma unroll
    for (int u = 0; u < R::U; ++u) {
      if (w0 + u >= a.T) break;
#pragma unroll
      for (int j = 0; j < R::N; ++j) acc[j] += p[u][j];
    }
    R::store(s_p + wave * a.E, a.E, acc);
  }
  lds_barrier();
  if (w0 < a.T) {
#pragma unroll
    for (int u = 0; u < R::U; ++u)  // whole numbers: any order gives the same
      if (w0 + u < a.T && seq[u] >= 0 && (unsigned)id[u] < (unsigned)a.E)
        atomicAdd(&s_c[seq[u] * a.E + id[u]], 1);
  }
  lds_barrier();
  for (int i = threadIdx.x; i < a.n_seq * a.E; i += 1024) {
    const int sq = i / a.E, e = i - sq * a.E;
    const int b = one ? 0 : s_start[sq], end = one ? 16 : s_start[sq + 1];
    float v = 0.0f;
    for (int t = b; t < end; t += 16) {
      float x[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = s_p[(t + k < end ? t + k : t) * a.E + e];
#pragma unroll
      for (int k = 0; k < 16; ++k) v += t + k < end ? x[k] : 0.0f;
    }
    a.counts[i] = s_c[i];
    s_c[i] = __float_as_int(v * (float)s_c[i]);  // from here on the products
  }
  lds_barrier();
  for (int i = wave; i < a.n_seq; i += 16) {
    const int b = s_start[i], end = s_start[i + 1];
    float x = 0.0f;
    int n = 0;
    for (int e = lane; e < a.E; e += 64) x += __int_as_float(s_c[i * a.E + e]);
    x = dpp_sum_f32(x);
    for (int t = b; t < end; t += 64) n += __popcll(ballot64(t + lane < end && s_seq[t + lane < end ? t + lane : b] == i));
    if (lane == 0) {
      s_part[i] = x;
      s_tokens[i] = n;
    }
  }
  lds_barrier();
  if (wave == 0) finish<1>(a, s_tokens, s_part, 1);
}

// Adds the segments of sequence x / blocks for JOIN_E experts, for each x < n: 16 lanes an
// expert each, W * 4 rows of lanes every (W * 4)th chunk each.  With TICKET the grid is n, and
// the last workgroup to finish joins the sequences; else balance_finish_kernel does.  Bound by
// waits: for sums that other dies wrote, for the count of finished workgroups, for the
// sequences' sums (5 to 8 us; a launch of its own for the last step takes as long, and 4 us of
// the host).
constexpr int JOIN_E = 16;
template <int W, bool TICKET>
__global__ __launch_bounds__(64 * W) void balance_join_kernel(BalanceArgs a, int chunk, int blocks,
                                                              int n_all) {
  constexpr int G = 4 * W, AT = W == 16 ? 8 : 4;  // chunks a thread reads at a time
  __shared__ float s_p[G][JOIN_E];
  __shared__ int s_c[G][JOIN_E], s_n[G];
  const int lane = threadIdx.x & (JOIN_E - 1), g = threadIdx.x / JOIN_E;
  for (int x = blockIdx.x; x < n_all; x += gridDim.x) {
    const int seq = x / blocks, blk = x - seq * blocks;
    const int e = blk * JOIN_E + lane;
    int b = a.start ? a.start[seq] : 0, end = a.start ? a.start[seq + 1] : a.T;
    b = b > 0 ? b : 0;
    end = end < a.T ? end : a.T;
    float p = 0.0f;
    int c = 0, n = 0;
    if (b < end) {
      const int c1 = (end - 1) / chunk;
      const int col = e < a.E ? e : a.E - 1;  // (lanes past the last expert are left out below)
      for (int i0 = b / chunk + g; i0 <= c1; i0 += AT * G) {
        float pv[AT];
        int cv[AT], nv[AT];
#pragma unroll
        for (int k = 0; k < AT; ++k) {  // all on their way before the first is added
          const int i = i0 + k * G <= c1 ? i0 + k * G : i0;
          const size_t seg = (size_t)i + seq;
          pv[k] = a.seg_p[seg * a.E + col];
          cv[k] = a.seg_c[seg * a.E + col];
          nv[k] = a.seg_n[seg];
        }
#pragma unroll
        for (int k = 0; k < AT; ++k) {
          if (i0 + k * G <= c1) {
            p += pv[k];
            c += cv[k];
            n += nv[k];
          }
        }
      }
    }
    s_p[g][lane] = p;
    s_c[g][lane] = c;
    if (lane == 0) s_n[g] = n;
    lds_barrier();
    if (threadIdx.x < 64) {
      // every fourth row in each 16 lanes, then the four
      const int q = threadIdx.x / JOIN_E;
      p = s_p[q][lane];
      c = s_c[q][lane];
      n = s_n[q];
#pragma unroll
      for (int k = 4; k < G; k += 4) {
        p += s_p[k + q][lane];
        c += s_c[k + q][lane];
        n += s_n[k + q];
      }
#pragma unroll
      for (int o = 16; o <= 32; o <<= 1) {
        p += __shfl_xor(p, o, 64);
        c += __shfl_xor(c, o, 64);
        n += __shfl_xor(n, o, 64);
      }
      const bool own = e < a.E && q == 0;
      if (own) a.counts[(size_t)seq * a.E + e] = c;
      const float sum = dpp_sum_f32(own ? p * (float)c : 0.0f);
      if (threadIdx.x == 0) {
        a.part[(size_t)seq * blocks + blk] = sum;
        if (blk == 0) a.tokens[seq] = n;
      }
      if constexpr (TICKET) {
        int last = 0;
        if (threadIdx.x == 0) {
          // the sums are out before the count, and read after the last one is in
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
          last = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                 (int)gridDim.x - 1;
        }
        if (!__builtin_amdgcn_readfirstlane(last)) return;
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        finish<1>(a, a.tokens, a.part, blocks);
      }
    }
    if constexpr (TICKET) return;
    lds_barrier();
  }
}

__global__ __launch_bounds__(1024) void balance_finish_kernel(BalanceArgs a, int blocks) {
  finish<16>(a, a.tokens, a.part, blocks);
}

// U tokens a wavefront, nothing shared: the shares again (cheaper than 4 bytes a logit each
// way), the counts of the sequence from cache.  32768 x 256 sigmoid: 14.3 us, 62 % of vector
// issue, 4.6 TB/s of logits and gradients.
template <typename R, bool SIGMOID>
__global__ __launch_bounds__(256) void balance_backward_kernel(BalanceArgs a) {
  const int t0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * R::U;
  if (t0 >= a.T) return;
  const int lane = lane_id();
  float l[R::U][R::N], d[R::U][R::N], p[R::U][R::N], q[R::U][R::N];
  int id[R::U];
#pragma unroll
  for (int u = 0; u < R::U; ++u) {
    const int t = t0 + u < a.T ? t0 + u : t0;
    id[u] = lane < a.k ? a.idx[(size_t)t * a.k + lane] : -1;
    R::load(a.logits + (size_t)t * a.E, a.E, -INFINITY, l[u]);
#pragma unroll
    for (int j = 0; j < R::N; ++j) d[u][j] = 0.0f;
    if (a.d_in) R::load(a.d_in + (size_t)t * a.E, a.E, 0.0f, d[u]);
  }
  const Sequences seqs(a);
  const float up = a.d_loss ? a.d_loss[0] : 1.0f;
  int seq = -2, end = 0, have = -2;
  int c[R::N];
  float scale = 0.0f;
  shares<R, SIGMOID>(l, p, q);
#pragma unroll
  for (int u = 0; u < R::U; ++u) {
    const int t = t0 + u;
    if (t >= a.T) break;
    if (u == 0 || t >= end) {
      seq = seqs.of(t, &end);
      if (seq >= a.n_seq) end = a.T;
    }
    if (ballot64((unsigned)id[u] < (unsigned)a.E) && seq >= 0 && seq < a.n_seq) {
      if (have != seq) {
        R::load(a.counts + (size_t)seq * a.E, a.E, 0, c);
        scale = a.scales[seq] * up;
        have = seq;
      }
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < R::N; ++j) dot = fmaf(p[u][j], (float)c[j], dot);
      dot = dpp_sum_f32(dot);
#pragma unroll
      for (int j = 0; j < R::N; ++j) {
        const float g = p[u][j] * ((float)c[j] - dot) * (SIGMOID ? q[u][j] : 1.0f);
        d[u][j] = l[u][j] > -INFINITY ? fmaf(scale, g, d[u][j]) : d[u][j];
      }
    }
    R::store(a.d_logits + (size_t)t * a.E, a.E, d[u]);
  }
}

// Calls f with the Row that fits E: past 128 experts four neighbours a lane where rows
// start at 16 bytes, so that a row is one load or few.  U1, U2, U4: rows at a time of up to 64,
// 128 and 256 experts.
template <int U1, int U2, int U4, typename F>
hipError_t with_row(int E, F f) {
  if (E <= 64) return f(Row<1, U1, false>());
  if (E <= 128) return f(Row<2, U2, false>());
  const bool four = E % 4 == 0;
  if (E <= 256) return four ? f(Row<4, U4, true>()) : f(Row<4, U4, false>());
  if (E <= 512) return four ? f(Row<8, 2, true>()) : f(Row<8, 2, false>());
  return four ? f(Row<16, 1, true>()) : f(Row<16, 1, false>());
}

}  // namespace

// As many tokens as the wavefronts hold at once, or more, so that there are at most 1024
// chunks to join (the loss of 262144 x 128: 77 -> 50 us).
int balance_chunk(int T, int E) {
  const int once = PART_W * (E <= 256 ? 4 : E <= 512 ? 2 : 1);
  return once * (int)std::max<int64_t>(1, ((int64_t)T + once * 1024 - 1) / (once * 1024));
}
int balance_blocks(int E) { return (E + JOIN_E - 1) / JOIN_E; }

hipError_t launch_balance(const BalanceArgs& a, hipStream_t s) {
  if (is_small(a)) {
    return with_row<SMALL_T / 16, SMALL_T / 32, SMALL_T / 32>(a.E, [&](auto row) {
      using R = decltype(row);
      if constexpr (R::N > 4) return hipErrorInvalidValue;  // E is at most 256
      else if (a.sigmoid)
        return MOE_LAUNCH("balance_small", s, balance_small_kernel<R, true><<<1, 1024, 0, s>>>(a));
      else
        return MOE_LAUNCH("balance_small", s, balance_small_kernel<R, false><<<1, 1024, 0, s>>>(a));
    });
  }
  const int chunk = balance_chunk(a.T, a.E);
  // one workgroup at least: the second launch needs the ticket that the first one clears
  const int grid = a.T > chunk ? (a.T - 1) / chunk + 1 : 1;
  const size_t lds = (size_t)a.E * (PART_W + 1) * 4;
  hipError_t e = with_row<4, 4, 4>(a.E, [&](auto row) {
    using R = decltype(row);
    if (a.sigmoid)
      return MOE_LAUNCH("balance_part", s,
                        balance_part_kernel<R, true><<<grid, 64 * PART_W, lds, s>>>(a, chunk));
    return MOE_LAUNCH("balance_part", s,
                      balance_part_kernel<R, false><<<grid, 64 * PART_W, lds, s>>>(a, chunk));
  });
  if (e != hipSuccess) return e;
  const int blocks = balance_blocks(a.E), n = a.n_seq * blocks;
  // few sequences have many chunks each, and few workgroups count themselves out
  if (n <= 256)
    return MOE_LAUNCH("balance_join", s,
                      balance_join_kernel<16, true><<<n, 1024, 0, s>>>(a, chunk, blocks, n));
  const int most = 1 << 20, groups = n < most ? n : most;
  e = MOE_LAUNCH("balance_join", s,
                 balance_join_kernel<4, false><<<groups, 256, 0, s>>>(a, chunk, blocks, n));
  if (e != hipSuccess) return e;
  return MOE_LAUNCH("balance_finish", s, balance_finish_kernel<<<1, 1024, 0, s>>>(a, blocks));
}

hipError_t launch_balance_backward(const BalanceArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  // two rows of 256 leave registers for more wavefronts (32768 x 256: 17.1 -> 14.3 us), four of
  // 128 fit (262144 x 128 behind the loss, which leaves logits in the cache: 65 -> 58)
  return with_row<4, 4, 2>(a.E, [&](auto row) {
    using R = decltype(row);
    const int grid = (a.T + 4 * R::U - 1) / (4 * R::U);
    if (a.sigmoid)
      return MOE_LAUNCH("balance_backward", s,
                        balance_backward_kernel<R, true><<<grid, 256, 0, s>>>(a));
    return MOE_LAUNCH("balance_backward", s,
                      balance_backward_kernel<R, false><<<grid, 256, 0, s>>>(a));
  });
}

}  // namespace moe
