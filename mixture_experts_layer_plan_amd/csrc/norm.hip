// The norm in front of the layer, joined with the residual stream, and its gradient.
//
// With h = round(x + res) the row that is normalised, mu its mean (0 without centring)
// and s = 1 / sqrt(mean((h - mu)^2) + eps):
//   y = round((h - mu) s w + b)
// and with xh = (h - mu) s, g = dy w:
//   dx = round(dh + s (g - mean(g) - xh mean(g xh)))   (mean(g) only with centring)
//   dw = sum_t dy xh,  db = sum_t dy
//
// A row stays in registers: the sums of squares are of the differences from the mean, not
// differences of sums.  All sums are in fp32, in an order that depends on the sizes alone.
// Rows past 512 elements take a workgroup each, shorter ones 2^i lanes each.
#include <type_traits>

#include "common.hpp"
#include "internal.hpp"
#include "step.hpp"
#include "wave.hpp"

namespace moe {
namespace {

// Eight elements of a row of `chunks` such eights that starts at eight `at`, in 16-byte
// accesses whose lanes are neighbours: in bf16 the i-th eight, in fp32 the i-th four of each
// half of the row (eight neighbours would be halves of 32 bytes: forward and backward of 4096 x
// 7168 with a residual take 74 + 103 us so, 68 + 97 by halves).  column() is the column of
// element j.  keep() is no instruction: the compiler takes the values as new ones, so that it
// unpacks them again behind it and does not hold them unpacked over a barrier.
// Stores of rows go past the caches.  The norm by itself takes the same up to 64 rows of 7168
// and less from there on (bf16, us, past the caches / not: 256 rows 4.1 / 4.5, 1024 8.5 / 11.5,
// 8192 69 / 86); with the router projection that reads y behind it, the same up to 16 rows and
// around 256 to 4096 (27.5 / 27.8 at 1024), 14.6 / 13.7 at 64, 123 / 139 at 8192.
template <typename E>
struct Vec8;
template <>
struct Vec8<bf16_t> {
  uint4 a;
  MOE_DEV static int column(int i, int j, int) { return 8 * i + j; }
  MOE_DEV void load(const void* p, size_t at, int i, int) { a = ((const uint4*)p)[at + i]; }
  MOE_DEV void store(void* p, size_t at, int i, int) const {
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, a), (u32x4_t*)p + at + i);
  }
  MOE_DEV void get(float* f) const { unpack8(a, f); }
  MOE_DEV void keep() { asm volatile("" : "+v"(a.x), "+v"(a.y), "+v"(a.z), "+v"(a.w)); }
  MOE_DEV void set(const float* f) { a = cvt8(f); }
};
template <>
struct Vec8<float> {
  float4 a, b;
  MOE_DEV static int column(int i, int j, int chunks) {
    return 4 * (j < 4 ? i : chunks + i) + (j & 3);
  }
  MOE_DEV void load(const void* p, size_t at, int i, int chunks) {
    a = ((const float4*)p)[2 * at + i];
    b = ((const float4*)p)[2 * at + chunks + i];
  }
  MOE_DEV void store(void* p, size_t at, int i, int chunks) const {
    __builtin_nontemporal_store(__builtin_bit_cast(f32x4_t, a), (f32x4_t*)p + 2 * at + i);
    __builtin_nontemporal_store(__builtin_bit_cast(f32x4_t, b), (f32x4_t*)p + 2 * at + chunks + i);
  }
  MOE_DEV void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  MOE_DEV void keep() {
    asm volatile("" : "+v"(a.x), "+v"(a.y), "+v"(a.z), "+v"(a.w), "+v"(b.x), "+v"(b.y), "+v"(b.z), "+v"(b.w));
  }
  MOE_DEV void set(const float* f) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};
// Eight sums of a thread's columns, to a row of sums that a second launch reads.
template <typename E>
MOE_DEV void store_sums(float* row, int i, int chunks, const float* f) {
  const float4 a = make_float4(f[0], f[1], f[2], f[3]), b = make_float4(f[4], f[5], f[6], f[7]);
  *(float4*)(row + Vec8<E>::column(i, 0, chunks)) = a;
  *(float4*)(row + Vec8<E>::column(i, 4, chunks)) = b;
}

// The sum of v over the workgroup, in every thread; `slot` is W floats of LDS that no
// wavefront reads any more (two calls on one slot have another call between them).
template <int W>
MOE_DEV float group_sum(float v, float* slot) {
  v = dpp_sum_f32(v);
  if (W == 1) return v;
  if (lane_id() == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = slot[0];
#pragma unroll
  for (int w = 1; w < W; ++w) t += slot[w];
  return t;
}

// dw and db of eight chunks of columns over all rows, by one workgroup of W wavefronts: a lane
// takes a chunk of every (8 W)th row.  They need h, dy and the forward's stats alone, so that
// workgroups of this kind run beside those of the rows, in one launch.
constexpr int COLS = 8;
template <typename E, int W, bool CENTRE>
MOE_DEV void column_sums(const NormBackArgs& p, int block) {
  constexpr int ROWS = 64 * W / COLS, AT = 4;
  __shared__ float s_sum[W][16][COLS];
  const int chunks = p.H / 8, lane = threadIdx.x & (COLS - 1), i = block * COLS + lane;
  const int col = i < chunks ? i : chunks - 1;
  float sum[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) sum[j] = 0.0f;
  for (int64_t r0 = threadIdx.x / COLS; r0 < p.T; r0 += AT * ROWS) {
    Vec8<E> h[AT], dy[AT];
    float2 st[AT];
#pragma unroll
    for (int k = 0; k < AT; ++k) {  // all on their way before the first is used
      const int64_t row = r0 + k * ROWS < p.T ? r0 + k * ROWS : r0;
      h[k].load(p.h, (size_t)row * chunks, col, chunks);
      dy[k].load(p.dy, (size_t)row * chunks, col, chunks);
      st[k] = *(const float2*)(p.stats + 2 * row);
    }
#pragma unroll
    for (int k = 0; k < AT; ++k) {
      if (r0 + k * ROWS < p.T) {
        float x[8], g[8];
        h[k].get(x);
        dy[k].get(g);
        const float mu = CENTRE ? st[k].x : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sum[j] = fmaf(g[j], (x[j] - mu) * st[k].y, sum[j]);
          sum[8 + j] += g[j];
        }
      }
    }
  }
#pragma unroll
  for (int o = COLS; o < 64; o <<= 1) {
#pragma unroll
    for (int j = 0; j < 16; ++j) sum[j] += __shfl_xor(sum[j], o, 64);
  }
  if (lane_id() < COLS) {
#pragma unroll
    for (int j = 0; j < 16; ++j) s_sum[threadIdx.x >> 6][j][lane] = sum[j];
  }
  __syncthreads();
  if (threadIdx.x >= COLS || i >= chunks) return;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
#pragma unroll
    for (int w = 1; w < W; ++w) sum[j] += s_sum[w][j][lane];
  }
  Vec8<E> v;
  if (p.dw) v.set(sum), v.store(p.dw, 0, i, chunks);
  if (p.db) v.set(sum + 8), v.store(p.db, 0, i, chunks);
}

// The sum of v over L neighbouring lanes, in each of them.
template <int L>
MOE_DEV float lanes_sum(float v) {
  if constexpr (L == 64) return dpp_sum_f32(v);
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Rows of at most L chunks, L lanes each, one chunk a lane: no LDS and no barrier.  Bound by
// memory where there are enough rows (32768 x 512 bf16 with a residual, 21.4 us, 6.3 TB/s), by
// the launch below (8192 x 256: 6 us).
template <typename E, int L, bool CENTRE>
__global__ __launch_bounds__(256) void norm_short_kernel(NormArgs p) {
  constexpr int ROWS = 256 / L;
  const int chunks = p.H / 8, i = threadIdx.x & (L - 1), slot = threadIdx.x / L;
  const float inv = 1.0f / (float)p.H;
  const bool on = i < chunks;
  float wf[8], bf[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    wf[j] = 1.0f;
    bf[j] = 0.0f;
  }
  Vec8<E> v;
  if (on && p.w) v.load(p.w, 0, i, chunks), v.get(wf);
  if (on && p.b) v.load(p.b, 0, i, chunks), v.get(bf);
  for (int64_t row = (int64_t)blockIdx.x * ROWS + slot; row < p.T; row += (int64_t)gridDim.x * ROWS) {
    const size_t at = (size_t)row * chunks;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    if (on) {
      v.load(p.x, at, i, chunks);
      v.get(f);
      if (p.res) {
        float r[8];
        v.load(p.res, at, i, chunks);
        v.get(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += r[j];
        v.set(f);
        v.store(p.h, at, i, chunks);
        v.get(f);  // the norm is that of h as it is kept: the backward reads it
      }
    }
    float sum = 0.0f, sq = 0.0f;
    if (CENTRE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += f[j];
      sum = lanes_sum<L>(sum);
    }
    const float mu = sum * inv;
    if (on) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[j] -= mu;
        sq = fmaf(f[j], f[j], sq);
      }
    }
    const float rstd = 1.0f / sqrtf(lanes_sum<L>(sq) * inv + p.eps);
    if (i == 0) *(float2*)(p.stats + 2 * row) = make_float2(mu, rstd);
    if (on) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * wf[j] + bf[j];
      v.set(f);
      v.store(p.y, at, i, chunks);
    }
  }
}

template <typename E, int L, bool CENTRE>
__global__ __launch_bounds__(256) void norm_short_backward_kernel(NormBackArgs p) {
  if ((int)blockIdx.x >= p.groups) return column_sums<E, 4, CENTRE>(p, blockIdx.x - p.groups);
  constexpr int ROWS = 256 / L;
  __shared__ float s_sum[4][2][8 * L];
  const int chunks = p.H / 8, i = threadIdx.x & (L - 1), slot = threadIdx.x / L;
  const float inv = 1.0f / (float)p.H;
  const bool on = i < chunks;
  float wf[8], dw[8], db[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    wf[j] = 1.0f;
    dw[j] = db[j] = 0.0f;
  }
  Vec8<E> v;
  if (on && p.w) v.load(p.w, 0, i, chunks), v.get(wf);
  for (int64_t row = (int64_t)blockIdx.x * ROWS + slot; row < p.T; row += (int64_t)p.groups * ROWS) {
    const size_t at = (size_t)row * chunks;
    const float2 st = *(const float2*)(p.stats + 2 * row);
    const float mu = CENTRE ? st.x : 0.0f, rstd = st.y;
    float x[8], g[8], d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = g[j] = d[j] = 0.0f;
    float sg = 0.0f, sgx = 0.0f;
    if (on) {
      Vec8<E> vg, vd;
      v.load(p.h, at, i, chunks);
      vg.load(p.dy, at, i, chunks);
      if (p.dh) vd.load(p.dh, at, i, chunks);
      v.get(x);
      vg.get(g);
      if (p.dh) vd.get(d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = (x[j] - mu) * rstd;
        dw[j] = fmaf(g[j], x[j], dw[j]);
        db[j] += g[j];
        g[j] *= wf[j];
        sg += g[j];
        sgx = fmaf(g[j], x[j], sgx);
      }
    }
    const float mg = CENTRE ? lanes_sum<L>(sg) * inv : 0.0f;
    const float mgx = lanes_sum<L>(sgx) * inv;
    if (on) {
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] += rstd * (g[j] - mg - x[j] * mgx);
      v.set(d);
      v.store(p.dx, at, i, chunks);
    }
  }
  if (!p.sums) return;
  // the rows of a wavefront, then the wavefronts
#pragma unroll
  for (int o = L; o < 64; o <<= 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dw[j] += __shfl_xor(dw[j], o, 64);
      db[j] += __shfl_xor(db[j], o, 64);
    }
  }
  const int wave = threadIdx.x >> 6;
  if (lane_id() < L) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s_sum[wave][0][j * L + i] = dw[j];
      s_sum[wave][1][j * L + i] = db[j];
    }
  }
  __syncthreads();
  float* out = p.parts + (size_t)blockIdx.x * 2 * p.H;
  for (int c = threadIdx.x; c < 2 * p.H; c += 256) {
    const int k = c >= p.H, x = c - k * p.H, j = x / chunks, col = x - j * chunks, at = j * L + col;
    const int e = Vec8<E>::column(col, j, chunks);
    out[k * p.H + e] = (s_sum[0][k][at] + s_sum[1][k][at]) + (s_sum[2][k][at] + s_sum[3][k][at]);
  }
}

// One row at a time in W wavefronts, C chunks a thread, with w and b in registers for all of
// them.  Bound by memory: x, residual, h and y once (8192 x 7168 bf16: 470 MB in 82 us, 5.7
// TB/s).  The two sums are joined through LDS, a barrier each; while a workgroup waits there
// the others of its CU load.
template <typename E, int W, int C, bool CENTRE>
__global__ __launch_bounds__(64 * W) void norm_kernel(NormArgs p) {
  __shared__ float s_mean[2][W], s_var[2][W];
  const int chunks = p.H / 8;
  const float inv = 1.0f / (float)p.H;
  Vec8<E> w[C], b[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * 64 * W + (int)threadIdx.x;
    if (i < chunks && p.w) w[c].load(p.w, 0, i, chunks);
    if (i < chunks && p.b) b[c].load(p.b, 0, i, chunks);
  }
  int parity = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, parity ^= 1) {
    const size_t at = (size_t)row * chunks;
    float f[C][8];
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * 64 * W + (int)threadIdx.x;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[c][j] = 0.0f;
      if (i < chunks) {
        Vec8<E> x;
        x.load(p.x, at, i, chunks);
        x.get(f[c]);
        if (p.res) {
          float r[8];
          Vec8<E> v;
          v.load(p.res, at, i, chunks);
          v.get(r);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[c][j] += r[j];
          v.set(f[c]);
          v.store(p.h, at, i, chunks);
          v.get(f[c]);  // the norm is that of h as it is kept: the backward reads it
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += f[c][j];
    }
    const float mu = CENTRE ? group_sum<W>(sum, s_mean[parity]) * inv : 0.0f;
    float sq = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * 64 * W + (int)threadIdx.x;
      if (i < chunks) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[c][j] -= mu;
          sq = fmaf(f[c][j], f[c][j], sq);
        }
      }
    }
    const float rstd = 1.0f / sqrtf(group_sum<W>(sq, s_var[parity]) * inv + p.eps);
    if (threadIdx.x == 0) {
      p.stats[2 * row] = mu;
      p.stats[2 * row + 1] = rstd;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * 64 * W + (int)threadIdx.x;
      if (i < chunks) {
        float wf[8], bf[8];
        if (p.w) w[c].get(wf);
        if (p.b) b[c].get(bf);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[c][j] *= rstd;
          if (p.w) f[c][j] *= wf[j];
          if (p.b) f[c][j] += bf[j];
        }
        Vec8<E> y;
        y.set(f[c]);
        y.store(p.y, at, i, chunks);
      }
    }
  }
}

// As norm_kernel, over every p.groups-th row, with the sums of dw and db of a thread's columns
// beside it.  Bound by memory: h, dy, dh and dx once (8192 x 7168 bf16: 500 MB with the sums in
// 90 us, 5.5 TB/s); rows stay packed over the barrier, so that two workgroups of 512 threads
// fit a CU (126 registers; unpacked 129, and 121 us).
template <typename E, int W, int C, bool CENTRE>
__global__ __launch_bounds__(64 * W) void norm_backward_kernel(NormBackArgs p) {
  if ((int)blockIdx.x >= p.groups) return column_sums<E, W, CENTRE>(p, blockIdx.x - p.groups);
  // Two chunks of fp32 leave no registers for the sums of dw and db (1024 threads have 128
  // each): they lie in LDS, each thread's own, with lanes side by side.
  constexpr bool IN_LDS = sizeof(E) == 4 && C > 1;
  constexpr int NT = 64 * W, SUMS = IN_LDS ? 2 * C * 8 * NT : 1;
  __shared__ float s_g[2][W], s_gx[2][W], s_acc[SUMS];
  const int chunks = p.H / 8;
  const float inv = 1.0f / (float)p.H;
  Vec8<E> w[C];
  float dw[C][8], db[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * NT + (int)threadIdx.x;
    if (!IN_LDS && i < chunks && p.w) w[c].load(p.w, 0, i, chunks);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (IN_LDS) {
        s_acc[(c * 8 + j) * NT + threadIdx.x] = 0.0f;
        s_acc[((C + c) * 8 + j) * NT + threadIdx.x] = 0.0f;
      } else {
        dw[c][j] = db[c][j] = 0.0f;
      }
    }
  }
  int parity = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += p.groups, parity ^= 1) {
    const size_t at = (size_t)row * chunks;
    const float mu = CENTRE ? p.stats[2 * row] : 0.0f;
    const float rstd = p.stats[2 * row + 1];
    Vec8<E> vh[C], vdy[C], vdh[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * NT + (int)threadIdx.x;
      if (i < chunks) {
        vh[c].load(p.h, at, i, chunks);
        vdy[c].load(p.dy, at, i, chunks);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * NT + (int)threadIdx.x;
      if (!IN_LDS && i < chunks && p.dh) vdh[c].load(p.dh, at, i, chunks);
    }
    float sg = 0.0f, sgx = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * NT + (int)threadIdx.x;
      if (i < chunks) {
        float x[8], g[8], wf[8];
        vh[c].get(x);
        vdy[c].get(g);
        if (IN_LDS && p.w) w[c].load(p.w, 0, i, chunks);
        if (p.w) w[c].get(wf);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = (x[j] - mu) * rstd;
          if (IN_LDS) {
            float* acc = s_acc + (c * 8 + j) * NT + threadIdx.x;
            acc[0] = fmaf(g[j], x[j], acc[0]);
            acc[C * 8 * NT] += g[j];
          } else {
            dw[c][j] = fmaf(g[j], x[j], dw[c][j]);
            db[c][j] += g[j];
          }
          if (p.w) g[j] *= wf[j];
          sg += g[j];
          sgx = fmaf(g[j], x[j], sgx);
        }
        vh[c].keep();
        vdy[c].keep();
      }
    }
    const float mg = CENTRE ? group_sum<W>(sg, s_g[parity]) * inv : 0.0f;
    const float mgx = group_sum<W>(sgx, s_gx[parity]) * inv;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * NT + (int)threadIdx.x;
      if (i < chunks) {
        float x[8], g[8], wf[8], d[8];
        vh[c].get(x);
        vdy[c].get(g);
        if (IN_LDS && p.w) w[c].load(p.w, 0, i, chunks);
        if (IN_LDS && p.dh) vdh[c].load(p.dh, at, i, chunks);
        if (p.w) w[c].get(wf);
        if (p.dh) vdh[c].get(d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = (x[j] - mu) * rstd;
          if (p.w) g[j] *= wf[j];
          const float t = rstd * (g[j] - mg - x[j] * mgx);
          d[j] = p.dh ? d[j] + t : t;
        }
        Vec8<E> v;
        v.set(d);
        v.store(p.dx, at, i, chunks);
      }
    }
  }
  if (!p.sums) return;
  float* out = p.parts + (size_t)blockIdx.x * 2 * p.H;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * NT + (int)threadIdx.x;
    if (i < chunks) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (IN_LDS) {
          dw[c][j] = s_acc[(c * 8 + j) * NT + threadIdx.x];
          db[c][j] = s_acc[((C + c) * 8 + j) * NT + threadIdx.x];
        }
      }
      store_sums<E>(out, i, chunks, dw[c]);
      store_sums<E>(out + p.H, i, chunks, db[c]);
    }
  }
}

// dw and db from the workgroups' sums, added up in their order: L lanes take 4 L
// neighbouring columns, 256 / L such rows of lanes every (256 / L)th workgroup each, joined
// through LDS.  Few columns take 4 lanes, so that there are more parts and workgroups
// (the backward of 1003 x 2040 in fp32: 13.9 -> 12.9 us); many take 16, whose reads are longer.
template <typename E, int L>
__global__ __launch_bounds__(256) void norm_wgrad_kernel(NormBackArgs p, int groups) {
  constexpr int PARTS = 256 / L;
  __shared__ float4 s_sum[PARTS][L];
  const int lane = threadIdx.x & (L - 1), part = threadIdx.x / L;
  const int col = blockIdx.x * 4 * L + lane * 4;  // of the 2 H columns (dw | db)
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < 2 * p.H) {
#pragma unroll 8
    for (int g = part; g < groups; g += PARTS) {
      const float4 v = *(const float4*)(p.parts + (size_t)g * 2 * p.H + col);
      t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
    }
  }
  s_sum[part][lane] = t;
#pragma unroll
  for (int half = PARTS / 2; half >= 1; half >>= 1) {
    __syncthreads();
    if (part < half) {
      const float4 v = s_sum[part + half][lane];
      t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
      s_sum[part][lane] = t;
    }
  }
  if (part || col >= 2 * p.H) return;
  void* out = col < p.H ? p.dw : p.db;
  const int at = col < p.H ? col : col - p.H;
  if (!out) return;
  if constexpr (sizeof(E) == 2) {
    *(uint2*)((bf16_t*)out + at) = make_uint2(cvt_bf16x2(t.x, t.y), cvt_bf16x2(t.z, t.w));
  } else {
    *(float4*)((float*)out + at) = t;
  }
}

// Wavefronts of a row: as many as it has 64 chunks of 8 elements, so that a thread holds
// one chunk, up to 8; then two chunks, and 16 wavefronts past 1024 chunks.
int waves_of(int H) {
  const int chunks = H / 8;
  int w = 1;
  while (w < 8 && 64 * w < chunks) w *= 2;
  return chunks > 1024 ? 16 : w;
}
int chunks_of(int H) { return H / 8 > 64 * waves_of(H) ? 2 : 1; }

constexpr int SHORT_H = 512;
// Lanes of a short row.
int lanes_of(int H) {
  int l = 1;
  while (8 * l < H) l *= 2;
  return l;
}

template <int N>
using Int = std::integral_constant<int, N>;
// Calls f with the lanes of short rows.
template <typename F>
hipError_t with_lanes(int H, F f) {
  switch (lanes_of(H)) {
    case 1: return f(Int<1>());
    case 2: return f(Int<2>());
    case 4: return f(Int<4>());
    case 8: return f(Int<8>());
    case 16: return f(Int<16>());
    case 32: return f(Int<32>());
  }
  return f(Int<64>());
}
// Calls f with the wavefronts and the chunks of long rows.
template <typename F>
hipError_t with_waves(int H, F f) {
  switch (waves_of(H) * chunks_of(H)) {
    case 2: return f(Int<2>(), Int<1>());
    case 4: return f(Int<4>(), Int<1>());
    case 8: return f(Int<8>(), Int<1>());
    case 16: return f(Int<8>(), Int<2>());
  }
  return f(Int<16>(), Int<2>());
}

// Whether the sums of dw and db are taken by workgroups of their own beside the rows', which
// read h and dy again but need no second launch: up to 1 KB of a column (256 x 7168: bf16 14.5
// -> 6.8 us, fp32 18.3 -> 9.2; 512 x 4096: 11.5 -> 8.0 and, left as it is, 12.0 -> 14.3).  A dx
// over dy takes two launches all the same, the columns first (kernels alone, 256 x 7168 bf16:
// 13.2 us against 8.0), so that its sums are those of a dx elsewhere.
bool norm_columns_beside(const NormBackArgs& p, int esize) {
  return (p.dw || p.db) && p.T > 0 && (int64_t)p.T * esize <= 1024;
}
// Their workgroups where they leave no sums.
int norm_rows_alone(int T, int H) {
  return H <= SHORT_H ? (T + 256 / lanes_of(H) - 1) / (256 / lanes_of(H)) : T;
}

template <typename E, bool CENTRE>
hipError_t norm_of(const NormArgs& p, hipStream_t s) {
  if (p.H <= SHORT_H)
    return with_lanes(p.H, [&](auto l) {
      constexpr int L = decltype(l)::value;
      const int64_t passes = ((int64_t)p.T + 256 / L - 1) / (256 / L);
      const int grid = passes < 4096 ? (int)passes : 4096;
      return MOE_LAUNCH("norm", s, norm_short_kernel<E, L, CENTRE><<<grid, 256, 0, s>>>(p));
    });
  const auto launch = [&](auto w, auto c) {
    constexpr int W = decltype(w)::value, C = decltype(c)::value;
    const int grid = p.T < 16384 / W ? p.T : 16384 / W;
    return MOE_LAUNCH("norm", s, norm_kernel<E, W, C, CENTRE><<<grid, 64 * W, 0, s>>>(p));
  };
  // the forward has the registers for 16 wavefronts of one chunk, if most of them have one
  // (8192 x 7168: 86.5 -> 82.4 us; the backward, one workgroup of them a CU: 90 -> 111)
  if (p.H / 8 > 768 && p.H / 8 <= 1024) return launch(Int<16>(), Int<1>());
  return with_waves(p.H, launch);
}
template <typename E, bool CENTRE>
hipError_t norm_back_launch(const NormBackArgs& p, int grid, hipStream_t s) {
  if (p.H <= SHORT_H)
    return with_lanes(p.H, [&](auto l) {
      constexpr int L = decltype(l)::value;
      return MOE_LAUNCH("norm_backward", s,
                        norm_short_backward_kernel<E, L, CENTRE><<<grid, 256, 0, s>>>(p));
    });
  return with_waves(p.H, [&](auto w, auto c) {
    constexpr int W = decltype(w)::value, C = decltype(c)::value;
    return MOE_LAUNCH("norm_backward", s,
                      norm_backward_kernel<E, W, C, CENTRE><<<grid, 64 * W, 0, s>>>(p));
  });
}
template <typename E, bool CENTRE>
hipError_t norm_back_of(NormBackArgs p, hipStream_t s) {
  const bool beside = norm_columns_beside(p, sizeof(E));
  const int groups = beside ? norm_rows_alone(p.T, p.H) : norm_groups(p.T, p.H);
  int columns = beside ? (p.H / 8 + COLS - 1) / COLS : 0;
  p.sums = (p.dw || p.db) && !beside;
  if (columns && p.dx == p.dy) {  // dy is overwritten: the columns first, with the same sums
    p.groups = 0;
    const hipError_t e = norm_back_launch<E, CENTRE>(p, columns, s);
    if (e != hipSuccess) return e;
    columns = 0;
  }
  p.groups = groups;
  if (p.T > 0) {
    const hipError_t e = norm_back_launch<E, CENTRE>(p, groups + columns, s);
    if (e != hipSuccess) return e;
  }
  if (!p.sums) return hipSuccess;
  if (2 * p.H < 4096)
    return MOE_LAUNCH("norm_wgrad", s,
                      norm_wgrad_kernel<E, 4><<<(2 * p.H + 15) / 16, 256, 0, s>>>(p, p.groups));
  return MOE_LAUNCH("norm_wgrad", s,
                    norm_wgrad_kernel<E, 16><<<(2 * p.H + 63) / 64, 256, 0, s>>>(p, p.groups));
}

}  // namespace

// Workgroups of the backward's rows: each leaves a row of sums, so that there are no more
// than fill the card, and four rows for each (1003 x 2040 in fp32: 12.7 us; two 15.1, eight
// 14.7).
int norm_groups(int T, int H) {
  const int most = H <= SHORT_H ? 1024 : 4096 / waves_of(H);
  const int rows = H <= SHORT_H ? 2 * 256 / lanes_of(H) : 4;
  const int64_t want = ((int64_t)T + rows - 1) / rows;
  return want < most ? (int)want : most;
}

hipError_t launch_norm(const NormArgs& p, bool f32, bool centre, hipStream_t s) {
  if (f32) return centre ? norm_of<float, true>(p, s) : norm_of<float, false>(p, s);
  return centre ? norm_of<bf16_t, true>(p, s) : norm_of<bf16_t, false>(p, s);
}

hipError_t launch_norm_backward(const NormBackArgs& p, bool f32, bool centre, hipStream_t s) {
  if (f32) return centre ? norm_back_of<float, true>(p, s) : norm_back_of<float, false>(p, s);
  return centre ? norm_back_of<bf16_t, true>(p, s) : norm_back_of<bf16_t, false>(p, s);
}

}  // namespace moe
