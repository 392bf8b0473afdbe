// The norm in front of the layer, joined with the residual stream, and its gradient.
//
// With h = round(x + res) the row that is normalised, mu its mean (0 without centring)
// and s = 1 / sqrt(mean((h - mu)^2) + eps):
//   y = round((h - mu) s w + b)
// and with xh = (h - mu) s, g = dy w:
//   dx = round(dh + s (g - mean(g) - xh mean(g xh)))   (mean(g) only with centring)
//   dw = sum_t dy xh,  db = sum_t dy
//
// A workgroup takes one row at a time and keeps it in registers: the sums of squares are
// of the differences from the mean, not differences of sums.  All sums are in fp32, in an
// order that depends on the sizes alone.
#include "common.hpp"
#include "internal.hpp"
#include "step.hpp"
#include "wave.hpp"

namespace moe {
namespace {

// Eight neighbouring elements of a row: one 16-byte access in bf16, two in fp32.
template <typename E>
struct Vec8;
template <>
struct Vec8<bf16_t> {
  uint4 a;
  MOE_DEV void load(const void* p, size_t i) { a = ((const uint4*)p)[i]; }
  MOE_DEV void store(void* p, size_t i) const { ((uint4*)p)[i] = a; }
  MOE_DEV void get(float* f) const { unpack8(a, f); }
  MOE_DEV void set(const float* f) { a = pack8(f); }
};
template <>
struct Vec8<float> {
  float4 a, b;
  MOE_DEV void load(const void* p, size_t i) {
    a = ((const float4*)p)[2 * i];
    b = ((const float4*)p)[2 * i + 1];
  }
  MOE_DEV void store(void* p, size_t i) const {
    ((float4*)p)[2 * i] = a;
    ((float4*)p)[2 * i + 1] = b;
  }
  MOE_DEV void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  MOE_DEV void set(const float* f) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

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

template <typename E, int W, int C, bool CENTRE>
__global__ __launch_bounds__(64 * W) void norm_kernel(NormArgs p) {
  __shared__ float s_mean[2][W], s_var[2][W];
  const int chunks = p.H / 8;
  const float inv = 1.0f / (float)p.H;
  Vec8<E> w[C], b[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * 64 * W + (int)threadIdx.x;
    if (i < chunks && p.w) w[c].load(p.w, i);
    if (i < chunks && p.b) b[c].load(p.b, i);
  }
  int parity = 0;
  for (int row = blockIdx.x; row < p.T; row += gridDim.x, parity ^= 1) {
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
        x.load(p.x, at + i);
        x.get(f[c]);
        if (p.res) {
          float r[8];
          Vec8<E> v;
          v.load(p.res, at + i);
          v.get(r);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[c][j] += r[j];
          v.set(f[c]);
          v.store(p.h, at + i);
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
      p.stats[2 * (size_t)row] = mu;
      p.stats[2 * (size_t)row + 1] = rstd;
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
        y.store(p.y, at + i);
      }
    }
  }
}

template <typename E, int W, int C, bool CENTRE>
__global__ __launch_bounds__(64 * W) void norm_backward_kernel(NormBackArgs p) {
  __shared__ float s_g[2][W], s_gx[2][W];
  const int chunks = p.H / 8;
  const float inv = 1.0f / (float)p.H;
  Vec8<E> w[C];
  float dw[C][8], db[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * 64 * W + (int)threadIdx.x;
    if (i < chunks && p.w) w[c].load(p.w, i);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[c][j] = db[c][j] = 0.0f;
  }
  int parity = 0;
  for (int row = blockIdx.x; row < p.T; row += gridDim.x, parity ^= 1) {
    const size_t at = (size_t)row * chunks;
    const float mu = CENTRE ? p.stats[2 * (size_t)row] : 0.0f;
    const float rstd = p.stats[2 * (size_t)row + 1];
    float xh[C][8], g[C][8];
    float sg = 0.0f, sgx = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * 64 * W + (int)threadIdx.x;
      if (i < chunks) {
        float wf[8];
        Vec8<E> v;
        v.load(p.h, at + i);
        v.get(xh[c]);
        v.load(p.dy, at + i);
        v.get(g[c]);
        if (p.w) w[c].get(wf);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          xh[c][j] = (xh[c][j] - mu) * rstd;
          dw[c][j] = fmaf(g[c][j], xh[c][j], dw[c][j]);
          db[c][j] += g[c][j];
          if (p.w) g[c][j] *= wf[j];
          sg += g[c][j];
          sgx = fmaf(g[c][j], xh[c][j], sgx);
        }
      }
    }
    const float mg = CENTRE ? group_sum<W>(sg, s_g[parity]) * inv : 0.0f;
    const float mgx = group_sum<W>(sgx, s_gx[parity]) * inv;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * 64 * W + (int)threadIdx.x;
      if (i < chunks) {
        float d[8];
        Vec8<E> v;
        if (p.dh) {
          v.load(p.dh, at + i);
          v.get(d);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float t = rstd * (g[c][j] - mg - xh[c][j] * mgx);
          d[j] = p.dh ? d[j] + t : t;
        }
        v.set(d);
        v.store(p.dx, at + i);
      }
    }
  }
  if (!p.dw && !p.db) return;
  float* out = p.parts + (size_t)blockIdx.x * 2 * p.H;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * 64 * W + (int)threadIdx.x;
    if (i < chunks) {
      Vec8<float> v;
      v.set(dw[c]);
      v.store(out, i);
      v.set(db[c]);
      v.store(out + p.H, i);
    }
  }
}

// dw and db from the workgroups' sums, added up in their order.  16 lanes take 64
// neighbouring columns, 16 such rows of lanes every 16th part each, joined through LDS.
template <typename E>
__global__ __launch_bounds__(256) void norm_wgrad_kernel(NormBackArgs p, int groups) {
  __shared__ float4 s_sum[16][16];
  const int lane = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int col = blockIdx.x * 64 + lane * 4;  // of the 2 H columns (dw | db)
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < 2 * p.H) {
    for (int g = part; g < groups; g += 16) {
      const float4 v = *(const float4*)(p.parts + (size_t)g * 2 * p.H + col);
      t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
    }
  }
  s_sum[part][lane] = t;
  __syncthreads();
  if (part || col >= 2 * p.H) return;
  for (int k = 1; k < 16; ++k) {
    const float4 v = s_sum[k][lane];
    t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
  }
  void* out = col < p.H ? p.dw : p.db;
  const int at = col < p.H ? col : col - p.H;
  if (!out) return;
  if constexpr (sizeof(E) == 2) {
    *(uint2*)((bf16_t*)out + at) = make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
  } else {
    *(float4*)((float*)out + at) = t;
  }
}

// Wavefronts of a row and 16-byte chunks of a thread: the fewest wavefronts whose threads
// hold at most two chunks each.
int waves_of(int H) {
  const int chunks = H / 8;
  int w = 1;
  while (w < 16 && 64 * w * 2 < chunks) w *= 2;
  return w;
}

template <typename E, int W, int C>
hipError_t norm_as(const NormArgs& p, bool centre, int grid, hipStream_t s) {
  if (centre)
    return MOE_LAUNCH("norm", s, norm_kernel<E, W, C, true><<<grid, 64 * W, 0, s>>>(p));
  return MOE_LAUNCH("norm", s, norm_kernel<E, W, C, false><<<grid, 64 * W, 0, s>>>(p));
}
template <typename E, int W, int C>
hipError_t norm_back_as(const NormBackArgs& p, bool centre, int grid, hipStream_t s) {
  if (centre)
    return MOE_LAUNCH("norm_backward", s,
                      norm_backward_kernel<E, W, C, true><<<grid, 64 * W, 0, s>>>(p));
  return MOE_LAUNCH("norm_backward", s,
                    norm_backward_kernel<E, W, C, false><<<grid, 64 * W, 0, s>>>(p));
}

template <typename E>
hipError_t norm_of(const NormArgs& p, bool centre, hipStream_t s) {
  const int w = waves_of(p.H);
  const int grid = p.T < 16384 / w ? p.T : 16384 / w;
  if (w == 1 && p.H <= 512) return norm_as<E, 1, 1>(p, centre, grid, s);
  switch (w) {
    case 1: return norm_as<E, 1, 2>(p, centre, grid, s);
    case 2: return norm_as<E, 2, 2>(p, centre, grid, s);
    case 4: return norm_as<E, 4, 2>(p, centre, grid, s);
    case 8: return norm_as<E, 8, 2>(p, centre, grid, s);
  }
  return norm_as<E, 16, 2>(p, centre, grid, s);
}
template <typename E>
hipError_t norm_back_of(const NormBackArgs& p, bool centre, hipStream_t s) {
  const int w = waves_of(p.H), grid = norm_groups(p.T, p.H);
  if (p.T > 0) {
    hipError_t e;
    if (w == 1 && p.H <= 512) e = norm_back_as<E, 1, 1>(p, centre, grid, s);
    else if (w == 1) e = norm_back_as<E, 1, 2>(p, centre, grid, s);
    else if (w == 2) e = norm_back_as<E, 2, 2>(p, centre, grid, s);
    else if (w == 4) e = norm_back_as<E, 4, 2>(p, centre, grid, s);
    else if (w == 8) e = norm_back_as<E, 8, 2>(p, centre, grid, s);
    else e = norm_back_as<E, 16, 2>(p, centre, grid, s);
    if (e != hipSuccess) return e;
  }
  if (!p.dw && !p.db) return hipSuccess;
  const int blocks = (2 * p.H + 63) / 64;
  return MOE_LAUNCH("norm_wgrad", s, norm_wgrad_kernel<E><<<blocks, 256, 0, s>>>(p, grid));
}

}  // namespace

int norm_groups(int T, int H) {
  const int most = 4096 / waves_of(H);
  const int rows = (T + 3) / 4;
  return rows < most ? rows : most;
}

hipError_t launch_norm(const NormArgs& p, bool f32, bool centre, hipStream_t s) {
  return f32 ? norm_of<float>(p, centre, s) : norm_of<bf16_t>(p, centre, s);
}

hipError_t launch_norm_backward(const NormBackArgs& p, bool f32, bool centre, hipStream_t s) {
  return f32 ? norm_back_of<float>(p, centre, s) : norm_back_of<bf16_t>(p, centre, s);
}

}  // namespace moe
