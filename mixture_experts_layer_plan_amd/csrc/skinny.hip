// Products with one short side: the bf16 router projection (N = E experts) and the
// low-rank adapters (N or K = rank), forward and backward.
//
//   dot      out[m, j] = sum_k a[m, k] b[j, k]          logits = x W^T, u = x A^T, v = dy B
//   expand   y[m, o] = base[m, o] + sum_j u[m, j] w[o, j]   y += u B^T, dx += v A, dx += dL W
//   wgrad    g[j, h] = sum_m u[m, j] x[m, h]             dA = v^T x, dB = dy^T u, dW = dL^T x
//
// "Grouped" launches take the rows of a plan (the tokens of each adapter one after the
// other, as the plan orders the pairs of each expert) and group a's own weights; the
// others take all T tokens and one set of weights.
//
// x, dy and the weights are bf16.  u, v and dL are fp32 and enter the second product as
// two bf16 halves (hi = round(v), lo = round(v - hi): 16 bits of the 24-bit mantissa, an
// error of 2^-17 against the 2^-9 of the bf16 result), so that it costs two matrix
// instructions and no accuracy.
#include "gemm_common.hpp"
#include "skinny.hpp"

namespace moe {
namespace {

typedef float f32x4v __attribute__((ext_vector_type(4)));

MOE_DEV f32x4v mfma16(bf16x8_t a, bf16x8_t b, f32x4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
MOE_DEV f32x16_t mfma32(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
MOE_DEV bf16x8_t as_frag(const uint4& v) { return __builtin_bit_cast(bf16x8_t, v); }

// Inclusive sum over the lanes of a wavefront.
template <int CTRL, int ROWS>
MOE_DEV int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, true);
}
MOE_DEV int wave_scan(int v) {
  v = dpp_add<0x111, 0xf>(v);
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);
  v = dpp_add<0x143, 0xc>(v);
  return v;
}

// Where unit `want` lies when group a has units(counts[a]) units, the groups in id order:
// its group, its index inside the group, and the sums of rows and of 16-row tiles of the
// groups before.  Every wavefront finds its own (one pass over the counts).
struct GroupPos {
  int a, unit, count, row0, t16;
};
template <class F>
MOE_DEV bool find_group(const int32_t* __restrict__ counts, int n, int want, const F& units,
                        GroupPos& g) {
  const int lane = threadIdx.x & 63;
  int u0 = 0, r0 = 0, t0 = 0;
  for (int b = 0; b < n; b += 64) {
    const int c = b + lane < n ? counts[b + lane] : 0;
    const int u = b + lane < n ? units(c) : 0;
    const int tt = (c + 15) >> 4;
    const int us = wave_scan(u), rs = wave_scan(c), ts = wave_scan(tt);
    const unsigned long long m = ballot64(u0 + us > want);
    if (m) {
      const int w = __ffsll((long long)m) - 1;
      g.a = b + w;
      g.count = __builtin_amdgcn_readlane(c, w);
      g.unit = want - u0 - __builtin_amdgcn_readlane(us - u, w);
      g.row0 = r0 + __builtin_amdgcn_readlane(rs - c, w);
      g.t16 = t0 + __builtin_amdgcn_readlane(ts - tt, w);
      return true;
    }
    u0 += __builtin_amdgcn_readlane(us, 63);
    r0 += __builtin_amdgcn_readlane(rs, 63);
    t0 += __builtin_amdgcn_readlane(ts, 63);
  }
  return false;
}

// Row tile `tile` of bm rows: its group, first row (of the plan's row order), valid rows
// and first 16-row tile.
struct SkinnyTile {
  int a, row0, rows, t16;
};
template <bool GR>
MOE_DEV bool skinny_tile(const int32_t* counts, int n, int T, int bm, int tile, SkinnyTile& t) {
  if (GR) {
    GroupPos g;
    if (!find_group(counts, n, tile, [bm](int c) { return (c + bm - 1) / bm; }, g)) return false;
    t.a = g.a;
    t.row0 = g.row0 + g.unit * bm;
    t.rows = min(bm, g.count - g.unit * bm);
    t.t16 = g.t16 + g.unit * (bm >> 4);
    return true;
  }
  t.a = 0;
  t.row0 = tile * bm;
  t.rows = min(bm, T - t.row0);
  t.t16 = t.row0 >> 4;
  return t.rows > 0;
}

// ------------------------------------------------------------------------- dot
// A workgroup of NW wavefronts forms 16 MB rows x 16 NB columns over one of S parts of K.
// The wavefronts take 64-deep K steps in turn, each with the whole tile, and load their
// fragments straight into registers: a row element is used by one wavefront only, so LDS
// would add a copy and barriers, and no reuse.  The tiles are joined in LDS, pair by pair.
template <int MB, int NB, int NW, bool GR>
__global__ __launch_bounds__(NW * 64) void dot_kernel(DotArgs p) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int nblk = (p.N + 16 * NB - 1) / (16 * NB);
  const int s = blockIdx.x % p.S, rest = blockIdx.x / p.S;
  const int n0 = (rest % nblk) * 16 * NB;
  SkinnyTile t;
  if (!skinny_tile<GR>(p.counts, p.n, p.T, 16 * MB, rest / nblk, t)) return;
  const int K = p.K, kg = 8 * (lane >> 4);
  const bf16_t* ap[MB];
  const bf16_t* bp[NB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {  // rows past the tile repeat its last row, columns the last
    const int r = t.row0 + min(16 * i + (lane & 15), t.rows - 1);
    ap[i] = p.a + (size_t)(GR ? p.src_token[r] : r) * K + kg;
  }
#pragma unroll
  for (int i = 0; i < NB; ++i)
    bp[i] = p.b + ((size_t)t.a * p.N + min(n0 + 16 * i + (lane & 15), p.N - 1)) * K + kg;
  f32x4v acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = (f32x4v){0.f, 0.f, 0.f, 0.f};

  const int steps = (K + 63) / 64, per = (steps + p.S - 1) / p.S;
  const int end = min(steps, (s + 1) * per);
  const auto load = [&](int st, uint4 (&fa)[2][MB], uint4 (&fb)[2][NB]) {
    const int k0 = st * 64;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + 32 * h;
      if (k + 32 <= K) {
#pragma unroll
        for (int i = 0; i < MB; ++i) fa[h][i] = *(const uint4*)(ap[i] + k);
#pragma unroll
        for (int j = 0; j < NB; ++j) fb[h][j] = *(const uint4*)(bp[j] + k);
      } else {  // K is a multiple of 8: each lane's 8 values are in or out together
        const bool in = k + kg < K;
#pragma unroll
        for (int i = 0; i < MB; ++i) fa[h][i] = in ? *(const uint4*)(ap[i] + k) : zero4();
#pragma unroll
        for (int j = 0; j < NB; ++j) fb[h][j] = in ? *(const uint4*)(bp[j] + k) : zero4();
      }
    }
  };
  const auto mul = [&](const uint4 (&fa)[2][MB], const uint4 (&fb)[2][NB]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)  // columns as the M side: a lane gets 4 neighbours
          acc[i][j] = mfma16(as_frag(fb[h][j]), as_frag(fa[h][i]), acc[i][j]);
  };
  uint4 fa0[2][MB], fb0[2][NB], fa1[2][MB], fb1[2][NB];
  int st = s * per + wv;
  if (st < end) load(st, fa0, fb0);
  while (st < end) {
    if (st + NW < end) load(st + NW, fa1, fb1);
    mul(fa0, fb0);
    st += NW;
    if (st >= end) break;
    if (st + NW < end) load(st + NW, fa0, fb0);
    mul(fa1, fb1);
    st += NW;
  }

  __shared__ f32x4v part[NW / 2][MB * NB][64];
#pragma unroll
  for (int h = NW / 2; h >= 1; h /= 2) {
    if (wv >= h && wv < 2 * h)
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) part[wv - h][i * NB + j][lane] = acc[i][j];
    __syncthreads();
    if (wv < h)
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] += part[wv][i * NB + j][lane];
    __syncthreads();
  }
  if (wv) return;
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int m = 16 * i + (lane & 15);
    if (m >= t.rows) continue;
    float* o = p.out + ((size_t)s * p.R + t.row0 + m) * p.N;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int c = n0 + 16 * j + 4 * (lane >> 4);
      if ((p.N & 3) == 0) {
        if (c < p.N) *(f32x4v*)(o + c) = acc[i][j];
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (c + v < p.N) o[c + v] = acc[i][j][v];
      }
    }
  }
}

// out[i] = sum over the S parts, in order
__global__ __launch_bounds__(256) void sum_parts_kernel(const float* __restrict__ parts, int S,
                                                        size_t n, float* __restrict__ out) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = 0.0f;
  for (int s = 0; s < S; ++s) v += parts[(size_t)s * n + i];
  out[i] = v;
}

// ---------------------------------------------------------------------- expand
// byte offset of 16-byte chunk c of row m in the LDS copy of u (kp values a row)
MOE_DEV int u_chunk(int m, int c, int kp) { return m * kp * 2 + ((c ^ (m & 3)) << 4); }

// A workgroup takes 16 MB rows and one of `osplit` parts of the output columns; each
// wavefront 32 columns at a time.  The rows' u (summed over its S parts, scaled, split)
// lies in LDS, in registers where KS (K steps of 32) is known; the weights come straight
// from memory in the order of the fragments.  As the M side of the product, weight row i
// of block b stands for column 8 (i / 4) + 4 b + i % 4, so that a lane ends with 8
// neighbouring outputs: base and y move 16 bytes at a time, 64 bytes of a row per lane
// group, without another trip through LDS.
template <int MB, int KS, bool GR>
__global__ __launch_bounds__(256) void expand_kernel(ExpandArgs p) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int tile = blockIdx.x / p.osplit, oz = blockIdx.x % p.osplit;
  if (GR && tile >= p.max_tiles) {
    // rows without a group: the base alone, 16 tokens per workgroup
    const int b = blockIdx.x - p.max_tiles * p.osplit;
    for (int i = wv; i < 16; i += 4) {
      const int tok = b * 16 + i;
      if (tok >= p.T || p.pos[tok] >= 0) continue;
      const size_t o = (size_t)tok * p.nout;
      for (int c = lane * 8; c < p.nout; c += 512)
        *(uint4*)(p.y + o + c) = p.base ? *(const uint4*)(p.base + o + c) : zero4();
    }
    return;
  }
  SkinnyTile t;
  if (!skinny_tile<GR>(p.counts, p.n, p.T, 16 * MB, tile, t)) return;
  const int ksteps = KS ? KS : (p.K + 31) / 32, kp = 32 * ksteps;
  const int lo_off = 16 * MB * kp * 2;
  {
    const float sc = p.scale ? p.scale[t.a] : 1.0f;
    const int ch = kp / 8;
    for (int i = threadIdx.x; i < 16 * MB * ch; i += 256) {
      const int m = i / ch, c = i % ch;
      float f[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) f[v] = 0.0f;
      if (m < t.rows) {
        for (int s = 0; s < p.S; ++s) {
          const float* u = p.u + ((size_t)s * p.R + t.row0 + m) * p.K;
          if ((p.K & 3) == 0) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
              if (8 * c + 4 * q < p.K) {
                const float4 v = *(const float4*)(u + 8 * c + 4 * q);
                f[4 * q] += v.x; f[4 * q + 1] += v.y; f[4 * q + 2] += v.z; f[4 * q + 3] += v.w;
              }
          } else {
#pragma unroll
            for (int v = 0; v < 8; ++v)
              if (8 * c + v < p.K) f[v] += u[8 * c + v];
          }
        }
      }
      float lo[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        f[v] *= sc;
        const float hi = bf16_to_f32(f32_to_bf16(f[v]));
        lo[v] = fabsf(hi) < INFINITY ? f[v] - hi : 0.0f;  // inf stays inf, not NaN
      }
      *(uint4*)(lds + u_chunk(m, c, kp)) = pack8(f);
      *(uint4*)(lds + lo_off + u_chunk(m, c, kp)) = pack8(lo);
    }
  }
  __syncthreads();
  if (p.ut && oz == 0) {
    // the halves along the rows, for the weight gradients: [16-row tile][j][16 hi, 16 lo]
    const int nt = (t.rows + 15) / 16;
    for (int i = threadIdx.x; i < nt * p.K; i += 256) {
      const int q = i / p.K, j = i % p.K;
      uint32_t w[16];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
          const char* b = lds + h * lo_off + (j & 7) * 2;
          const uint32_t v0 = *(const uint16_t*)(b + u_chunk(16 * q + r, j >> 3, kp));
          const uint32_t v1 = *(const uint16_t*)(b + u_chunk(16 * q + r + 1, j >> 3, kp));
          w[8 * h + r / 2] = v0 | (v1 << 16);
        }
      uint4* d = (uint4*)(p.ut + ((size_t)(t.t16 + q) * p.K + j) * 32);
#pragma unroll
      for (int v = 0; v < 4; ++v) d[v] = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
    }
  }
  const auto frag_u = [&](int i, int ks, int half) {
    return as_frag(*(const uint4*)(lds + half * lo_off + u_chunk(16 * i + (lane & 15), 4 * ks + (lane >> 4), kp)));
  };
  size_t rowo[MB];
  bool ok[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int m = 16 * i + (lane & 15);
    ok[i] = m < t.rows;
    const int r = t.row0 + (ok[i] ? m : 0);
    rowo[i] = (size_t)(GR ? p.src_token[r] : r) * p.nout + 8 * (lane >> 4);
  }
  bf16x8_t uh[KS ? MB : 1][KS ? KS : 1], ul[KS ? MB : 1][KS ? KS : 1];
  if constexpr (KS > 0) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uh[i][ks] = frag_u(i, ks, 0);
        ul[i][ks] = frag_u(i, ks, 1);
      }
  }
  const bf16_t* W = p.w + (size_t)t.a * p.nout * p.wld;
  const int chunks = (p.nout + 31) / 32, cper = (chunks + p.osplit - 1) / p.osplit;
  const int c1 = min(chunks, (oz + 1) * cper);
  const int rho = lane & 15, wrow = 8 * (rho >> 2) + (rho & 3);
  for (int c = oz * cper + wv; c < c1; c += 4) {
    const int o0 = c * 32;
    const bool in = o0 + 8 * (lane >> 4) < p.nout;
    uint4 bs[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
      bs[i] = p.base && ok[i] && in ? *(const uint4*)(p.base + rowo[i] + o0) : zero4();
    f32x4v acc[MB][2];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b) acc[i][b] = (f32x4v){0.f, 0.f, 0.f, 0.f};
    const bf16_t* wp[2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
      wp[b] = W + (size_t)min(o0 + wrow + 4 * b, p.nout - 1) * p.wld + 8 * (lane >> 4);
    if constexpr (KS > 0) {
      uint4 wf[KS][2];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int b = 0; b < 2; ++b)
          wf[ks][b] = 32 * ks + 8 * (lane >> 4) < p.wld ? *(const uint4*)(wp[b] + 32 * ks) : zero4();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            acc[i][b] = mfma16(as_frag(wf[ks][b]), ul[i][ks], acc[i][b]);
            acc[i][b] = mfma16(as_frag(wf[ks][b]), uh[i][ks], acc[i][b]);
          }
    } else {
#pragma unroll 2
      for (int ks = 0; ks < ksteps; ++ks) {
        uint4 wf[2];
#pragma unroll
        for (int b = 0; b < 2; ++b)
          wf[b] = 32 * ks + 8 * (lane >> 4) < p.wld ? *(const uint4*)(wp[b] + 32 * ks) : zero4();
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          const bf16x8_t h = frag_u(i, ks, 0), l = frag_u(i, ks, 1);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            acc[i][b] = mfma16(as_frag(wf[b]), l, acc[i][b]);
            acc[i][b] = mfma16(as_frag(wf[b]), h, acc[i][b]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      if (!ok[i] || !in) continue;
      float f[8];
      unpack8(bs[i], f);
#pragma unroll
      for (int v = 0; v < 8; ++v) f[v] += acc[i][v >> 2][v & 3];
      *(uint4*)(p.y + rowo[i] + o0) = pack8(f);
    }
  }
}

// ----------------------------------------------------------------------- wgrad
// A workgroup of 4 wavefronts forms 32 JB WJ rows (j) x 128 columns (h) of one group's
// gradient over one chunk of its rows.  The wide operand x passes through LDS, where the
// transposing reads turn its rows into K-major fragments; the short one comes as the
// halves that `expand` left along the rows, straight into registers.  WJ wavefronts share
// out j, the others h.
template <int JB, int WJ, bool GR>
__global__ __launch_bounds__(256) void wgrad_kernel(WgradArgs p) {
  constexpr int WH = 4 / WJ, HB = 4 / WH;  // wavefronts along h, 32-column blocks of each
  __shared__ __attribute__((aligned(16))) char lds[2][64 * 256];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const WgradSide d = p.side[blockIdx.z];
  const int h0 = blockIdx.x * 128, ch = blockIdx.y / p.jblk;
  const int j0 = (blockIdx.y % p.jblk) * 32 * JB * WJ + (wv % WJ) * 32 * JB;
  const int hw = (wv / WJ) * 32 * HB;
  if (h0 >= d.H) return;
  GroupPos g;
  const int crows = p.chunk_rows;
  int nch;
  if (GR) {
    const auto units = [crows](int c) { return max(1, (c + crows - 1) / crows); };
    if (!find_group(p.counts, p.n, ch, units, g)) return;
    nch = units(g.count);
  } else {
    nch = max(1, (p.T + crows - 1) / crows);
    g.a = 0;
    g.unit = ch;
    g.count = p.T;
    g.row0 = g.t16 = 0;
  }
  const int r0 = g.unit * crows, rows = max(0, min(crows, g.count - r0));
  const int row0 = g.row0 + r0, t16 = g.t16 + (r0 >> 4);
  f32x16_t acc[JB][HB];
#pragma unroll
  for (int i = 0; i < JB; ++i)
#pragma unroll
    for (int j = 0; j < HB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  const int kb = threadIdx.x >> 4, ib = threadIdx.x & 15;  // rows 4 kb .. + 3, columns 8 ib .. + 7
  const bool cin = h0 + 8 * ib < d.H;
  const auto load = [&](int st, uint4 (&r)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int m = st * 64 + 4 * kb + q;
      r[q] = zero4();
      if (m < rows && cin) {
        const int tok = GR ? p.src_token[row0 + m] : row0 + m;
        r[q] = *(const uint4*)(d.x + (size_t)tok * d.H + h0 + 8 * ib);
      }
    }
  };
  const auto store = [&](char* t, const uint4 (&r)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int k = 4 * kb + q;
      *(uint4*)(t + k * 256 + ((ib ^ mn_swz(k)) << 4)) = r[q];
    }
  };
  const int stages = (rows + 63) / 64, nt = (rows + 15) / 16;
  uint4 r[4];
  if (stages) {
    load(0, r);
    store(lds[0], r);
  }
  __syncthreads();
  for (int st = 0; st < stages; ++st) {
    if (st + 1 < stages) load(st + 1, r);
    const char* cur = lds[st & 1];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const int tt = st * 4 + ks;
      if (tt < nt) {  // past the last tile there are no halves
        bf16x8_t uh[JB], ul[JB];
#pragma unroll
        for (int i = 0; i < JB; ++i) {
          const int j = min(j0 + 32 * i + (lane & 31), p.J - 1);
          const bf16_t* u = d.ut + ((size_t)(t16 + tt) * p.J + j) * 32 + 8 * (lane >> 5);
          uh[i] = as_frag(*(const uint4*)u);
          ul[i] = as_frag(*(const uint4*)(u + 16));
        }
#pragma unroll
        for (int c = 0; c < HB; ++c) {
          const bf16x8_t x = frag16<false>(cur, hw + 32 * c, ks, lane);
#pragma unroll
          for (int i = 0; i < JB; ++i) {
            if (d.transposed) {  // j along a lane's registers
              acc[i][c] = mfma32(ul[i], x, acc[i][c]);
              acc[i][c] = mfma32(uh[i], x, acc[i][c]);
            } else {             // h along a lane's registers
              acc[i][c] = mfma32(x, ul[i], acc[i][c]);
              acc[i][c] = mfma32(x, uh[i], acc[i][c]);
            }
          }
        }
      }
    }
    if (st + 1 < stages) store(lds[(st + 1) & 1], r);
    __syncthreads();
  }
  const size_t per = (size_t)p.J * d.H;
  float* part = d.parts + (size_t)ch * per;
  bf16_t* out = d.out + (size_t)g.a * per;
#pragma unroll
  for (int i = 0; i < JB; ++i)
#pragma unroll
    for (int c = 0; c < HB; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int one = lane & 31, four = 8 * q + 4 * (lane >> 5);
        const int j = j0 + 32 * i + (d.transposed ? four : one);
        const int h = h0 + hw + 32 * c + (d.transposed ? one : four);
        if (j >= p.J || h >= d.H) continue;
        const f32x4v v = {acc[i][c][4 * q], acc[i][c][4 * q + 1], acc[i][c][4 * q + 2],
                          acc[i][c][4 * q + 3]};
        const size_t at = d.transposed ? (size_t)h * p.J + j : (size_t)j * d.H + h;
        if (nch > 1) {
          *(f32x4v*)(part + at) = v;
        } else {
          *(uint2*)(out + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        }
      }
}

// Gradients of the groups with several chunks: the sum of the chunks' parts, in order.
template <bool GR>
__global__ __launch_bounds__(256) void wgrad_sum_kernel(WgradArgs p) {
  const WgradSide d = p.side[blockIdx.z];
  const size_t per = (size_t)p.J * d.H;
  const int a = blockIdx.y, lane = threadIdx.x & 63;
  const int crows = p.chunk_rows;
  int first = 0, nch;
  if (GR) {
    int before = 0;
    for (int b = 0; b < a; b += 64)
      before += b + lane < a ? max(1, (p.counts[b + lane] + crows - 1) / crows) : 0;
    first = __builtin_amdgcn_readlane(wave_scan(before), 63);
    nch = max(1, (p.counts[a] + crows - 1) / crows);
  } else {
    nch = max(1, (p.T + crows - 1) / crows);
  }
  if (nch < 2) return;
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= per) return;
  f32x4v v = {0.f, 0.f, 0.f, 0.f};
  for (int c = 0; c < nch; ++c) v += *(const f32x4v*)(d.parts + (size_t)(first + c) * per + i);
  *(uint2*)(d.out + (size_t)a * per + i) =
      make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// ------------------------------------------------------------------- transpose
// dst [n][C][ldd] = src [n][R][C] transposed, zero for rows R .. ldd - 1; 64 x 64 tiles.
__global__ __launch_bounds__(256) void transpose_kernel(TransposeArgs a0, TransposeArgs a1) {
  const TransposeArgs a = blockIdx.z ? a1 : a0;
  __shared__ bf16_t t[64][66];
  const int rt = (a.ldd + 63) / 64, ct = (a.C + 63) / 64;
  const int g = blockIdx.y;
  if ((int)blockIdx.x >= rt * ct) return;
  const int r0 = (blockIdx.x % rt) * 64, c0 = (blockIdx.x / rt) * 64;
  const bf16_t* src = a.src + (size_t)g * a.R * a.C;
  bf16_t* dst = a.dst + (size_t)g * a.C * a.ldd;
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int r = r0 + i / 64, c = c0 + i % 64;
    t[i / 64][i % 64] = r < a.R && c < a.C ? src[(size_t)r * a.C + c] : (bf16_t)0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int c = c0 + i / 64, r = r0 + i % 64;
    if (c < a.C && r < a.ldd) dst[(size_t)c * a.ldd + r] = t[i % 64][i / 64];
  }
}

template <int MB, int NB, int NW>
hipError_t dot_go(const char* name, const DotArgs& p, int tiles, hipStream_t s) {
  const long g = (long)tiles * ((p.N + 16 * NB - 1) / (16 * NB)) * p.S;
  if (p.counts)
    return MOE_LAUNCH(name, s, dot_kernel<MB, NB, NW, true><<<(unsigned)g, NW * 64, 0, s>>>(p));
  return MOE_LAUNCH(name, s, dot_kernel<MB, NB, NW, false><<<(unsigned)g, NW * 64, 0, s>>>(p));
}

template <int MB, int KS>
hipError_t expand_go(const char* name, const ExpandArgs& p, hipStream_t s) {
  const int ksteps = KS ? KS : (p.K + 31) / 32;
  const unsigned lds = 16u * MB * 32 * ksteps * 4;
  const long extra = p.counts && p.base != p.y ? (p.T + 15) / 16 : 0;
  const unsigned g = (unsigned)((long)p.max_tiles * p.osplit + extra);
  if (p.counts) {
    auto* k = expand_kernel<MB, KS, true>;
    return MOE_LAUNCH(name, s, k<<<g, 256, lds, s>>>(p));
  }
  auto* k = expand_kernel<MB, KS, false>;
  return MOE_LAUNCH(name, s, k<<<g, 256, lds, s>>>(p));
}

int div_up(int a, int b) { return (a + b - 1) / b; }

}  // namespace

SkinnyPlan skinny_plan(int T, int n, bool grouped, int K, int N) {
  SkinnyPlan c;
  const int groups = !grouped ? 1 : (n < T ? n : T);
  c.mb = T >= 32 * groups ? 4 : 1;
  c.tiles = skinny_tiles(T, n, grouped, c.mb);
  const int nblk = div_up(N, N > 32 ? 64 : (N > 16 ? 32 : 16));
  const int nw = c.mb == 4 ? 4 : 8, steps = div_up(K, 64);
  const int most = div_up(steps, c.mb == 4 ? 2 * nw : nw);
  const int want = c.tiles > 0 ? div_up(512, c.tiles * nblk) : 1;
  c.S = want < most ? want : most;
  return c;
}

int skinny_tiles(int T, int n, bool grouped, int mb) {
  return div_up(T, 16 * mb) + (grouped ? (n < T ? n : T) : 0);
}

int expand_osplit(int tiles, int nout) {
  const int most = div_up(div_up(nout, 32), 4);
  int w = div_up(1024, tiles > 0 ? tiles : 1);
  return w < most ? w : most;
}

hipError_t launch_dot(const char* name, const DotArgs& p, int mb, int tiles, hipStream_t s) {
  if (tiles == 0) return hipSuccess;
  if (mb == 4) {
    if (p.N <= 16) return dot_go<4, 1, 4>(name, p, tiles, s);
    if (p.N <= 32) return dot_go<4, 2, 4>(name, p, tiles, s);
    return dot_go<4, 4, 4>(name, p, tiles, s);
  }
  if (p.N <= 16) return dot_go<1, 1, 8>(name, p, tiles, s);
  if (p.N <= 32) return dot_go<1, 2, 8>(name, p, tiles, s);
  return dot_go<1, 4, 8>(name, p, tiles, s);
}

hipError_t launch_sum_parts(const char* name, const float* parts, int S, size_t n, float* out,
                            hipStream_t s) {
  if (n == 0) return hipSuccess;
  return MOE_LAUNCH(name, s, sum_parts_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(parts, S, n, out));
}

hipError_t launch_expand(const char* name, const ExpandArgs& p, int mb, hipStream_t s) {
  if (p.T == 0) return hipSuccess;
  const int ks = div_up(p.K, 32);
  if (mb == 4) {
    if (ks == 1) return expand_go<4, 1>(name, p, s);
    if (ks == 2) return expand_go<4, 2>(name, p, s);
    return expand_go<4, 0>(name, p, s);
  }
  if (ks == 1) return expand_go<1, 1>(name, p, s);
  if (ks == 2) return expand_go<1, 2>(name, p, s);
  return expand_go<1, 0>(name, p, s);
}

int wgrad_chunk_slots(int T, int n, int chunk_rows) {
  return n > 0 ? T / chunk_rows + n : (T > 0 ? div_up(T, chunk_rows) : 1);
}

hipError_t launch_wgrad(const char* name, WgradArgs p, int sides, hipStream_t s) {
  const int hmax = sides > 1 && p.side[1].H > p.side[0].H ? p.side[1].H : p.side[0].H;
  const int slots = wgrad_chunk_slots(p.T, p.counts ? p.n : 0, p.chunk_rows);
  const int jt = p.J <= 32 ? 32 : (p.J <= 64 ? 64 : (p.J <= 128 ? 128 : 256));
  p.jblk = div_up(p.J, jt);
  const dim3 g((unsigned)div_up(hmax, 128), (unsigned)(slots * p.jblk), (unsigned)sides);
  hipError_t e;
#define MOE_WGRAD_GO(JB, WJ)                                                                  \
  e = p.counts ? MOE_LAUNCH(name, s, wgrad_kernel<JB, WJ, true><<<g, 256, 0, s>>>(p))         \
               : MOE_LAUNCH(name, s, wgrad_kernel<JB, WJ, false><<<g, 256, 0, s>>>(p))
  if (jt == 32) MOE_WGRAD_GO(1, 1);
  else if (jt == 64) MOE_WGRAD_GO(2, 1);
  else if (jt == 128) MOE_WGRAD_GO(2, 2);
  else MOE_WGRAD_GO(2, 4);
#undef MOE_WGRAD_GO
  if (e != hipSuccess || p.T <= p.chunk_rows) return e;
  const size_t per = (size_t)p.J * hmax;
  const dim3 gs((unsigned)((per + 1023) / 1024), (unsigned)(p.counts ? p.n : 1), (unsigned)sides);
  if (p.counts) return MOE_LAUNCH("wgrad_sum", s, wgrad_sum_kernel<true><<<gs, 256, 0, s>>>(p));
  return MOE_LAUNCH("wgrad_sum", s, wgrad_sum_kernel<false><<<gs, 256, 0, s>>>(p));
}

hipError_t launch_transpose(const char* name, int n, const TransposeArgs& a, const TransposeArgs* b,
                            hipStream_t s) {
  int blocks = div_up(a.ldd, 64) * div_up(a.C, 64);
  if (b) {
    const int o = div_up(b->ldd, 64) * div_up(b->C, 64);
    if (o > blocks) blocks = o;
  }
  return MOE_LAUNCH(name, s,
                    transpose_kernel<<<dim3((unsigned)blocks, (unsigned)n, b ? 2u : 1u), 256, 0, s>>>(
                        a, b ? *b : a));
}

}  // namespace moe
