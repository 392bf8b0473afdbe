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
// error of 2^-17 against the 2^-8 of the bf16 result), so that it costs two matrix
// instructions and no accuracy.
#include <algorithm>
#include <type_traits>

#include "gemm_common.hpp"
#include "skinny.hpp"

namespace moe {
namespace {

typedef float f32x4v __attribute__((ext_vector_type(4)));

typedef __bf16 bf16x4v __attribute__((ext_vector_type(4)));
MOE_DEV uint2 cvt4(const f32x4v& v) {
  return __builtin_bit_cast(uint2, __builtin_convertvector(v, bf16x4v));
}

MOE_DEV f32x4v mfma16(bf16x8_t a, bf16x8_t b, f32x4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
MOE_DEV bf16x8_t as_frag(const uint4& v) { return __builtin_bit_cast(bf16x8_t, v); }

// 8 floats -> 8 bf16 by the conversion instruction (two values each, to nearest even); the
// integer form of pack8 is six instructions a value, more than the matrix work beside it.
typedef float f32x8v __attribute__((ext_vector_type(8)));
MOE_DEV uint4 cvt8(const float* f) {
  const f32x8v v = {f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]};
  return __builtin_bit_cast(uint4, __builtin_convertvector(v, bf16x8_t));
}

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
// its group, its index inside the group, and the sums of rows and of 32-row tiles of the
// groups before.  Every wavefront finds its own (one pass over the counts).
struct GroupPos {
  int a, unit, count, row0, t32;
};
template <class F>
MOE_DEV bool find_group(const int32_t* __restrict__ counts, int n, int want, const F& units,
                        GroupPos& g) {
  const int lane = threadIdx.x & 63;
  int u0 = 0, r0 = 0, t0 = 0;
  for (int b = 0; b < n; b += 64) {
    const int c = b + lane < n ? counts[b + lane] : 0;
    const int u = b + lane < n ? units(c) : 0;
    const int tt = (c + 31) >> 5;
    const int us = wave_scan(u), rs = wave_scan(c), ts = wave_scan(tt);
    const unsigned long long m = ballot64(u0 + us > want);
    if (m) {
      const int w = __ffsll((long long)m) - 1;
      g.a = b + w;
      g.count = __builtin_amdgcn_readlane(c, w);
      g.unit = want - u0 - __builtin_amdgcn_readlane(us - u, w);
      g.row0 = r0 + __builtin_amdgcn_readlane(rs - c, w);
      g.t32 = t0 + __builtin_amdgcn_readlane(ts - tt, w);
      return true;
    }
    u0 += __builtin_amdgcn_readlane(us, 63);
    r0 += __builtin_amdgcn_readlane(rs, 63);
    t0 += __builtin_amdgcn_readlane(ts, 63);
  }
  return false;
}

// Row tile `tile` of bm rows: its group, first row (of the plan's row order) and valid
// rows; its first row inside the group, the group's rows and first 32-row tile.
struct SkinnyTile {
  int a, row0, rows, off, count, t32;
};
template <bool GR>
MOE_DEV bool skinny_tile(const int32_t* counts, int n, int T, int bm, int tile, SkinnyTile& t) {
  if (GR) {
    GroupPos g;
    if (!find_group(counts, n, tile, [bm](int c) { return (c + bm - 1) / bm; }, g)) return false;
    t.a = g.a;
    t.off = g.unit * bm;
    t.row0 = g.row0 + t.off;
    t.count = g.count;
    t.t32 = g.t32;
  } else {
    t.a = 0;
    t.off = t.row0 = tile * bm;
    t.count = T;
    t.t32 = 0;
  }
  t.rows = min(bm, t.count - t.off);
  return t.rows > 0;
}

// Workgroup i runs on XCD i mod 8: give each XCD a contiguous run of the work, so that the
// column blocks and K parts of a row tile share that XCD's L2 (for work of one size; tiles
// that turn out empty would leave the last XCD idle).
MOE_DEV int xcd_order(int id, int total) {
  const int per = total / N_XCD, rem = total % N_XCD, x = id % N_XCD, local = id / N_XCD;
  return x < rem ? x * (per + 1) + local : rem * (per + 1) + (x - rem) * per + local;
}

// 4 neighbouring values of a row of N
MOE_DEV void put4(float* o, int c, int N, const f32x4v& v) {
  if ((N & 3) == 0) {
    if (c < N) *(f32x4v*)(o + c) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < N) o[c + i] = v[i];
  }
}

// ------------------------------------------------------------------------- dot
// Few rows (a tile of 16): a workgroup of 8 wavefronts forms 16 rows x 16 NB columns over
// one of S parts of K.  The wavefronts take 64-deep K blocks in turn and load their
// fragments straight into registers; the tiles are joined in LDS, pair by pair.  (A
// fragment's 16 lanes lie in 16 rows, which costs the address unit four times the cycles
// of 256 neighbouring bytes: of no weight here, where latency counts, see dot_tile_kernel.)
template <int NB, bool GR>
__global__ __launch_bounds__(512) void dot_kernel(DotArgs p) {
  constexpr int NW = 8;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int nblk = (p.N + 16 * NB - 1) / (16 * NB);
  const int id = xcd_order(blockIdx.x, gridDim.x);
  const int n0 = (id % nblk) * 16 * NB, s = (id / nblk) % p.S;
  SkinnyTile t;
  if (!skinny_tile<GR>(p.counts, p.n, p.T, 16, id / (nblk * p.S), t)) return;
  const int K = p.K, kg = 8 * (lane >> 4);
  // rows past the tile repeat its last row, columns the last
  const int r = t.row0 + min(lane & 15, t.rows - 1);
  const bf16_t* ap = p.a + (size_t)(GR ? p.src_token[r] : r) * K + kg;
  const bf16_t* bp[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
    bp[i] = p.b + ((size_t)t.a * p.N + min(n0 + 16 * i + (lane & 15), p.N - 1)) * K + kg;
  f32x4v acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = (f32x4v){0.f, 0.f, 0.f, 0.f};
  const int blocks = (K + 63) / 64, per = (blocks + p.S - 1) / p.S;
  const int end = min(blocks, (s + 1) * per);
  const auto load = [&](int b, uint4 (&fa)[2], uint4 (&fb)[2][NB]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = b * 64 + 32 * h;
      const bool in = k + kg < K;  // K is a multiple of 8: a lane's 8 values go together
      fa[h] = in ? *(const uint4*)(ap + k) : zero4();
#pragma unroll
      for (int j = 0; j < NB; ++j) fb[h][j] = in ? *(const uint4*)(bp[j] + k) : zero4();
    }
  };
  const auto mul = [&](const uint4 (&fa)[2], const uint4 (&fb)[2][NB]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NB; ++j)  // columns as the M side: a lane gets 4 neighbours
        acc[j] = mfma16(as_frag(fb[h][j]), as_frag(fa[h]), acc[j]);
  };
  uint4 fa0[2], fb0[2][NB], fa1[2], fb1[2][NB];
  int b = s * per + wv;
  if (b < end) load(b, fa0, fb0);
  for (; b < end; b += 2 * NW) {
    if (b + NW < end) load(b + NW, fa1, fb1);
    mul(fa0, fb0);
    if (b + NW >= end) break;
    if (b + 2 * NW < end) load(b + 2 * NW, fa0, fb0);
    mul(fa1, fb1);
  }
  __shared__ f32x4v part[NW / 2][NB][64];
#pragma unroll
  for (int h = NW / 2; h >= 1; h /= 2) {
    if (wv >= h && wv < 2 * h)
#pragma unroll
      for (int j = 0; j < NB; ++j) part[wv - h][j][lane] = acc[j];
    __syncthreads();
    if (wv < h)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[j] += part[wv][j][lane];
    __syncthreads();
  }
  const int m = lane & 15;
  if (wv || m >= t.rows) return;
  float* o = p.out + ((size_t)s * p.R + t.row0 + m) * p.N;
#pragma unroll
  for (int j = 0; j < NB; ++j) put4(o, n0 + 16 * j + 4 * (lane >> 4), p.N, acc[j]);
}

// Many rows: a workgroup forms BM rows x BN columns over one of S parts of K, S chosen to
// fill the chip.  Both operands reach LDS by direct loads of K2-byte row pieces, 16 bytes a
// lane, into a ring of NS stages; the product of a stage runs while NS - 1 more are in
// flight.  Row r's 16-byte chunk c lies at r * K2 + 16 (c ^ swz(r)): the 16 rows of a
// fragment read hit all 64 banks.
// Measured: fragments loaded from memory without LDS took 121 us for the 8192 x 256 x 7168
// router product (16 lanes in 16 rows keep the address unit busy for 64 cycles a KiB), 64 x
// 128 tiles 53 us, 128 x 128 tiles with two sets of wavefronts 45 us and 6.5 us for the sum
// of the two parts.  Of those 45 us the direct loads alone, without a product or a store, take
// 39: 470 MB out of L2 (10 TB/s, where direct loads from L2 reach 29), 147 MB of them from
// memory (3.2 TB/s).  x alone takes 23 us and the weights, which come from L2, 12: the two add
// up instead of overlapping (each 64 rows x 128 columns less of tile costs 235 MB more and 13
// us).  Nothing is full, the matrix units are 26 % busy; that a CU's L1 answers in order, so
// that the weights wait behind x, would explain it and has not been shown.  Fragments read one
// step ahead of their products, 3 or 5 stages, and K from another start in each tile change
// nothing.  128 x 256 tiles with 4 parts would save 4 us of loads and cost 4 us of parts.
// Rank 64 over 8192 rows of 7168 (117 MB, 8 adapters): 31 to 33 us against 20 to 31 us for the
// plain read, as much as the writes of the kernel before still have to leave the Infinity
// Cache; the rest is the start of the workgroups.  S = 3 there: with 2 or 4 parts the tiles do
// not spread evenly (38, 40 us), and each further part costs the second product 1 to 2 us.
template <int BM, int BN>
struct DotTile {
  static constexpr int WN = BN >= 64 ? 2 : 1, WM = 4 / WN;  // wavefronts along columns, rows
  // 128 columns: a second set of wavefronts takes half of each stage's K
  static constexpr int KG = BN == 128 ? 2 : 1, BK = BM == 64 ? 64 * KG : 64, K2 = 2 * BK, CH = K2 / 16;
  static constexpr int NWV = 4 * KG, NT = 64 * NWV, HS = BK / 32 / KG;  // K steps of a wavefront
  static constexpr int MB = BM / 16 / WM, NB = BN / 16 / WN;
  static constexpr int STAGE = (BM + BN) * K2;
  // BM x 32, 64, 128: 36, 48, 144 KiB for 64 rows, -, 72, 128 for 128: 4, 3, 1, -, 2, 1 a CU
  static constexpr int NS = BM == 128 && BN == 128 ? 4 : 3;
  static constexpr int LOADS = STAGE / (1024 * NWV), ALOADS = BM * K2 / (1024 * NWV);  // a wavefront
  static MOE_DEV int swz(int r) { return CH == 8 ? (r >> 1) & 7 : r & 15; }
};

// Wait until at most `ahead` (0 to 3) stages of L loads are in flight, then meet the
// workgroup.  vmcnt's two high bits are bits 14 and 15 of the operand.
template <int L>
MOE_DEV void ring_wait_for(int ahead) {
  static_assert(3 * L < 64, "vmcnt has 6 bits");
  constexpr auto vm = [](int n) { return (n & 15) | ((n >> 4) << 14) | 0x70; };
  if (ahead >= 3) __builtin_amdgcn_s_waitcnt(vm(3 * L));
  else if (ahead == 2) __builtin_amdgcn_s_waitcnt(vm(2 * L));
  else if (ahead == 1) __builtin_amdgcn_s_waitcnt(vm(L));
  else __builtin_amdgcn_s_waitcnt(vm(0));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");  // no LDS read of the stage moves above the barrier
}

// NR fragments (16 x 32) from LDS, waited for in the same block: the compiler would wait
// for every direct load in flight before a read of its own.
MOE_DEV uint32_t lds_at(const char* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}
MOE_DEV void lds_read3(const uint32_t (&a)[3], s16x8_t (&f)[3]) {
  asm volatile(
      "ds_read_b128 %0, %3\n\tds_read_b128 %1, %4\n\tds_read_b128 %2, %5\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2])
      : "v"(a[0]), "v"(a[1]), "v"(a[2])
      : "memory");
}
MOE_DEV void lds_read4(const uint32_t (&a)[4], s16x8_t (&f)[4]) {
  asm volatile(
      "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %6\n\t"
      "ds_read_b128 %3, %7\n\ts_waitcnt lgkmcnt(0)"
      : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3])
      : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3])
      : "memory");
}
MOE_DEV void lds_read6(const uint32_t (&a)[6], s16x8_t (&f)[6]) {
  asm volatile(
      "ds_read_b128 %0, %6\n\tds_read_b128 %1, %7\n\tds_read_b128 %2, %8\n\t"
      "ds_read_b128 %3, %9\n\tds_read_b128 %4, %10\n\tds_read_b128 %5, %11\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3]), "=&v"(f[4]), "=&v"(f[5])
      : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(a[4]), "v"(a[5])
      : "memory");
}

MOE_DEV void lds_read8(const uint32_t (&a)[8], s16x8_t (&f)[8]) {
  asm volatile(
      "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\tds_read_b128 %2, %10\n\t"
      "ds_read_b128 %3, %11\n\tds_read_b128 %4, %12\n\tds_read_b128 %5, %13\n\t"
      "ds_read_b128 %6, %14\n\tds_read_b128 %7, %15\n\ts_waitcnt lgkmcnt(0)"
      : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3]), "=&v"(f[4]), "=&v"(f[5]),
        "=&v"(f[6]), "=&v"(f[7])
      : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(a[4]), "v"(a[5]), "v"(a[6]), "v"(a[7])
      : "memory");
}

template <int BM, int BN, bool GR>
__global__ __launch_bounds__((DotTile<BM, BN>::NT)) void dot_tile_kernel(DotArgs p) {
  using C = DotTile<BM, BN>;
  constexpr int NR = C::MB + C::NB, NWV = C::NWV;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int nblk = (p.N + BN - 1) / BN;
  // a row tile's column blocks on one XCD (grouped: one block; empty tiles spread evenly)
  const int id = GR ? (int)blockIdx.x : xcd_order(blockIdx.x, gridDim.x);
  const int n0 = (id % nblk) * BN, s = (id / nblk) % p.S;
  SkinnyTile t;
  if (!skinny_tile<GR>(p.counts, p.n, p.T, BM, id / (nblk * p.S), t)) return;
  const uint32_t K2 = (uint32_t)p.K * 2;
  const rsrc_t ra = make_rsrc(p.a, (uint32_t)p.T * K2);  // below 4 GiB, checked on the host
  const rsrc_t rb = make_rsrc(p.b + (size_t)t.a * p.N * p.K, (uint32_t)p.N * K2);
  // load q of a wavefront brings the RP rows from RP (NWV q + wv) on of the stage (the BM
  // rows of a, then the BN of b): lane L row L / CH, chunk L % CH of LDS; out of range: zeros
  constexpr uint32_t OUT = 0xffffffffu;
  constexpr int RP = 64 / C::CH;
  uint32_t off[C::LOADS];  // of the row's first byte
  int cq[C::LOADS];        // byte of its chunk in the piece
#pragma unroll
  for (int q = 0; q < C::LOADS; ++q) {
    const int r = RP * (NWV * q + wv) + lane / C::CH;
    cq[q] = ((lane & (C::CH - 1)) ^ C::swz(r)) * 16;
    if (q < C::ALOADS) {
      const int row = t.row0 + min(r, t.rows - 1);
      off[q] = (uint32_t)(GR ? p.src_token[row] : row) * K2;
      if (r >= t.rows) off[q] = OUT;
    } else {
      // row 16 f + i of a wavefront's columns holds column NB i + f: a lane ends with NB
      // neighbours, 16 lanes with a run of 16 NB
      const int l = r - BM, i = l & 15, f = (l >> 4) % C::NB, w = l / (16 * C::NB);
      const int n = n0 + (16 * w + i) * C::NB + f;
      off[q] = n < p.N ? (uint32_t)n * K2 : OUT;
    }
  }
  const int blocks = (p.K + C::BK - 1) / C::BK, per = (blocks + p.S - 1) / p.S;
  const int b0 = s * per, nk = min(blocks, b0 + per) - b0;
  const auto issue = [&](int i) {
    char* st = lds + (i % C::NS) * C::STAGE;
#pragma unroll
    for (int q = 0; q < C::LOADS; ++q) {
      const uint32_t k2 = (uint32_t)(b0 + i) * C::K2 + cq[q];  // past K in the last stage
      dma16_buf(q < C::ALOADS ? ra : rb, k2 < K2 && off[q] != OUT ? off[q] + k2 : OUT, 0u,
                st + (NWV * q + wv) * 1024);
    }
  };
  f32x4v acc[C::MB][C::NB];
#pragma unroll
  for (int i = 0; i < C::MB; ++i)
#pragma unroll
    for (int j = 0; j < C::NB; ++j) acc[i][j] = (f32x4v){0.f, 0.f, 0.f, 0.f};
  const int kg = wv / 4, wm = (wv % 4) / C::WN, wn = wv % C::WN;
  const int g = lane >> 4, rho = lane & 15;
  for (int i = 0; i < C::NS - 1 && i < nk; ++i) issue(i);
  for (int i = 0; i < nk; ++i) {
    // stage i is in (each later one has LOADS instructions), stage i - 1 no longer read
    ring_wait_for<C::LOADS>(min(C::NS - 2, nk - 1 - i));
    if (i + C::NS - 1 < nk) issue(i + C::NS - 1);
    const char* st = lds + (i % C::NS) * C::STAGE;
#pragma unroll
    for (int h = 0; h < C::HS; ++h) {
      uint32_t ad[NR];
      s16x8_t f[NR];
      const int cx = ((4 * (C::HS * kg + h) + g) ^ C::swz(rho)) << 4;
#pragma unroll
      for (int m = 0; m < C::MB; ++m)
        ad[m] = lds_at(st + (16 * (C::MB * wm + m) + rho) * C::K2 + cx);
#pragma unroll
      for (int n = 0; n < C::NB; ++n)
        ad[C::MB + n] = lds_at(st + (BM + 16 * (C::NB * wn + n) + rho) * C::K2 + cx);
      if constexpr (NR == 3) lds_read3(ad, f);
      else if constexpr (NR == 4) lds_read4(ad, f);
      else if constexpr (NR == 6) lds_read6(ad, f);
      else lds_read8(ad, f);
#pragma unroll
      for (int m = 0; m < C::MB; ++m)
#pragma unroll
        for (int n = 0; n < C::NB; ++n)
          acc[m][n] = mfma16(__builtin_bit_cast(bf16x8_t, f[m]),
                             __builtin_bit_cast(bf16x8_t, f[C::MB + n]), acc[m][n]);
    }
  }
  if constexpr (C::KG == 2) {  // join the halves of K
    __syncthreads();           // every wavefront is done with the ring
    f32x4v(*part)[C::NB][64] = (f32x4v(*)[C::NB][64])(lds + (wv % 4) * C::MB * C::NB * 1024);
    if (kg)
#pragma unroll
      for (int m = 0; m < C::MB; ++m)
#pragma unroll
        for (int n = 0; n < C::NB; ++n) part[m][n][lane] = acc[m][n];
    __syncthreads();
    if (kg) return;
#pragma unroll
    for (int m = 0; m < C::MB; ++m)
#pragma unroll
      for (int n = 0; n < C::NB; ++n) acc[m][n] += part[m][n][lane];
  }
  const int c0 = n0 + (16 * wn + rho) * C::NB;
#pragma unroll
  for (int m = 0; m < C::MB; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * (C::MB * wm + m) + 4 * g + i;
      if (r >= t.rows || c0 >= p.N) continue;
      float* o = p.out + ((size_t)s * p.R + t.row0 + r) * p.N + c0;
      if (p.N % C::NB == 0) {  // the row and this run of it are aligned to the run
        typedef float run_t __attribute__((ext_vector_type(C::NB)));
        run_t v;
#pragma unroll
        for (int n = 0; n < C::NB; ++n) v[n] = acc[m][n][i];
        *(run_t*)o = v;
      } else {
#pragma unroll
        for (int n = 0; n < C::NB; ++n)
          if (c0 + n < p.N) o[n] = acc[m][n][i];
      }
    }
}

// out[i] = sum over the S parts, in order.  Bound by memory: 25 MB in 6.5 us (8192 x 256, two
// parts), 21 MB in 5.2 us.
__global__ __launch_bounds__(256) void sum_parts_kernel(const float* __restrict__ parts, int S,
                                                        size_t n, float* __restrict__ out) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = 0.0f;
#pragma unroll 4
  for (int s = 0; s < S; ++s) v += parts[(size_t)s * n + i];
  out[i] = v;
}

// The dot of a few tokens (at most TB): a workgroup per column, its row of b read once and
// multiplied with every token's, without matrix instructions (which would leave 16 - T of 16
// rows idle and need a second launch to join the parts of K).  One token, 256 x 7168: 2.8 us
// against 5.3 + 4.0 us; 3.7 MB, so the launch and one round trip to memory are all of it.
template <int TB>
__global__ __launch_bounds__(256) void dot_few_kernel(DotArgs p) {
  __shared__ float part[4][TB];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const bf16_t* b = p.b + (size_t)blockIdx.x * p.K;
  float acc[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) acc[t] = 0.0f;
#pragma unroll 2
  for (int k = threadIdx.x * 8; k < p.K; k += 2048) {
    float fb[8];
    unpack8(*(const uint4*)(b + k), fb);
    uint4 xa[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t)  // tokens past the last repeat it
      xa[t] = *(const uint4*)(p.a + (size_t)min(t, p.T - 1) * p.K + k);
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      float fx[8];
      unpack8(xa[t], fx);
#pragma unroll
      for (int v = 0; v < 8; ++v) acc[t] = fmaf(fx[v], fb[v], acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const float v = wave_sum_f32(acc[t]);
    if (lane == 0) part[wv][t] = v;
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t < TB && t < p.T)
    p.out[(size_t)t * p.N + blockIdx.x] = (part[0][t] + part[1][t]) + (part[2][t] + part[3][t]);
}

// ---------------------------------------------------------------------- expand
// byte offset of 16-byte chunk c of row m in the LDS copy of u (kp values a row)
MOE_DEV int u_chunk(int m, int c, int kp) { return m * kp * 2 + ((c ^ (m & 3)) << 4); }

// 8 rows of 8 bf16 (one uint4 each) -> the 8 columns, 8 values each: every output word
// takes one half of two input words.
MOE_DEV void transpose8(const uint4 (&r)[8], uint4 (&c)[8]) {
#pragma unroll
  for (int h = 0; h < 8; ++h) {
    const uint32_t sel = h & 1 ? 0x07060302u : 0x05040100u;
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[q] = __builtin_amdgcn_perm(u4_word(r[2 * q + 1], h >> 1), u4_word(r[2 * q], h >> 1), sel);
    c[h] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The halves of u along the rows, in the order of wgrad's fragments (K = 32 rows):
// [32-row tile][16 values of j][hi, lo][lane: j = lane % 16, rows 8 (lane / 16) .. + 7][8].
// Rows past the group's last, up to its last tile's end, are zero.
template <int MB, int NT = 256>
MOE_DEV void store_halves(const char* lds, int lo_off, int kp, int K, const SkinnyTile& t,
                          int part, int parts, bf16_t* __restrict__ ut) {
  const int jb = (K + 15) / 16;
  const bool pad = t.off + 16 * MB >= t.count;  // the last tile: zeros up to a multiple of 32
  const int groups = pad ? (((t.off + t.rows + 31) >> 5 << 5) - t.off) / 8 : 2 * MB;
  for (int i = (threadIdx.x >> 4) + NT / 16 * part; i < groups * jb; i += NT / 16 * parts) {
    const int q = i / jb, j = (i - q * jb) * 16 + (threadIdx.x & 15), g8 = (t.off >> 3) + q;
    uint32_t w[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        uint32_t v0 = 0, v1 = 0;
        if (q < 2 * MB) {
          const char* b = lds + h * lo_off + (j & 7) * 2;
          v0 = *(const uint16_t*)(b + u_chunk(8 * q + 2 * r, j >> 3, kp));
          v1 = *(const uint16_t*)(b + u_chunk(8 * q + 2 * r + 1, j >> 3, kp));
        }
        w[h][r] = v0 | (v1 << 16);
      }
    bf16_t* d = ut + (((size_t)(t.t32 + (g8 >> 2)) * jb + (j >> 4)) * 2) * 512 +
                ((g8 & 3) * 16 + (j & 15)) * 8;
    *(uint4*)d = make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]);
    *(uint4*)(d + 512) = make_uint4(w[1][0], w[1][1], w[1][2], w[1][3]);
  }
}

// u of a row tile into LDS: its S parts summed, scaled and split, zeros past K and past
// the tile's rows; kp = K rounded up to 32.
// Q pieces of 8 and U parts are in flight at a time: one wait for memory, not one a part.
template <int ROWS, int Q, int U>
MOE_DEV void fill_u(const ExpandArgs& p, const SkinnyTile& t, int kp, char* lds) {
  const float sc = p.scale ? p.scale[t.a] : 1.0f;
  const int ch = kp / 8, lo_off = ROWS * kp * 2, items = ROWS * ch;
  const size_t part = p.R * p.K;
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < items; i0 += Q * 256) {
    float f[Q][8];
    const float* u[Q];
    bool in[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int i = min(i0 + q * 256, items - 1), m = i / ch, cc = i - m * ch;
      in[q] = m < t.rows && 8 * cc < p.K;
      u[q] = p.u + ((size_t)t.row0 + (in[q] ? m : 0)) * p.K + (in[q] ? 8 * cc : 0);
#pragma unroll
      for (int v = 0; v < 8; ++v) f[q][v] = 0.0f;
    }
    if ((p.K & 7) == 0) {
#pragma unroll 1
      for (int s = 0; s < p.S; s += U) {
        float4 a[U][Q], b[U][Q];
#pragma unroll
        for (int w = 0; w < U; ++w)
#pragma unroll
          for (int q = 0; q < Q; ++q) {  // parts past the last repeat it and are not added
            const float* x = u[q] + min(s + w, p.S - 1) * part;
            a[w][q] = *(const float4*)x;
            b[w][q] = *(const float4*)(x + 4);
          }
#pragma unroll
        for (int w = 0; w < U; ++w) {
          if (w && s + w >= p.S) break;
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            f[q][0] += a[w][q].x; f[q][1] += a[w][q].y; f[q][2] += a[w][q].z; f[q][3] += a[w][q].w;
            f[q][4] += b[w][q].x; f[q][5] += b[w][q].y; f[q][6] += b[w][q].z; f[q][7] += b[w][q].w;
          }
        }
      }
    } else if ((p.K & 3) == 0) {  // the router's dL: one part, a last piece of 4
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int i = min(i0 + q * 256, items - 1);
        const bool two = 8 * (i % ch) + 4 < p.K;
        const float4 a = *(const float4*)u[q];
        const float4 b = *(const float4*)(u[q] + (in[q] && two ? 4 : 0));
        f[q][0] = a.x; f[q][1] = a.y; f[q][2] = a.z; f[q][3] = a.w;
        f[q][4] = two ? b.x : 0.0f; f[q][5] = two ? b.y : 0.0f;
        f[q][6] = two ? b.z : 0.0f; f[q][7] = two ? b.w : 0.0f;
      }
    } else {  // rows of any length
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int i = min(i0 + q * 256, items - 1), left = p.K - 8 * (i % ch);
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const float x = u[q][in[q] && v < left ? v : 0];
          f[q][v] = v < left ? x : 0.0f;
        }
      }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int i = i0 + q * 256, m = i / ch, cc = i - m * ch;
      float hi[8], lo[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) f[q][v] = in[q] ? f[q][v] * sc : 0.0f;
      const uint4 h8 = cvt8(f[q]);
      unpack8(h8, hi);
#pragma unroll
      for (int v = 0; v < 8; ++v) lo[v] = fabsf(hi[v]) < INFINITY ? f[q][v] - hi[v] : 0.0f;
      if (i < items) {
        *(uint4*)(lds + u_chunk(m, cc, kp)) = h8;
        *(uint4*)(lds + lo_off + u_chunk(m, cc, kp)) = cvt8(lo);
      }
    }
  }
}

// Rows without a group: the base alone, a token per wavefront and 8 KiB in flight, by the
// workgroups behind the tiles' (at most COPY_GROUPS, which then take several tokens).
constexpr int COPY_GROUPS = 1 << 22;
MOE_DEV void copy_ungrouped(const ExpandArgs& p) {
  const int lane = threadIdx.x & 63, waves = (int)(blockDim.x >> 6);
  const int first = p.max_tiles * p.osplit, step = ((int)gridDim.x - first) * waves;
  for (int tok = ((int)blockIdx.x - first) * waves + (int)(threadIdx.x >> 6); tok < p.T; tok += step) {
    if (p.pos[tok] >= 0) continue;
    const size_t o = (size_t)tok * p.nout;
#pragma unroll 1
    for (int c = lane * 8; c < p.nout; c += 8 * 512) {
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = p.base && c + i * 512 < p.nout ? *(const uint4*)(p.base + o + c + i * 512) : zero4();
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i * 512 < p.nout) *(uint4*)(p.y + o + c + i * 512) = v[i];
    }
  }
}

// In both forms below u's rows are the M side of the product and fragment f's column i
// stands for output column 8 i + f of a 128-column block: a lane ends with 8 neighbouring
// outputs of 4 rows, and 16 lanes with 256 bytes of one row, so that base and y move in
// whole lines without a trip through LDS.  (With the weights as the M side a store's 16
// lanes lie in 16 rows: 92 us against 57 us for 8192 rows of 7168 at rank 64.)

// Few rows (16 MB a tile): each wavefront takes 128-column blocks of one of `osplit` parts
// of the columns; the weights come straight from memory, one K step of 32 ahead.  Bound by
// its chain of dependent loads (the group, its tokens and parts of u, base): both products of
// 96 tokens of 32 adapters take 14 us (rank 32, 7168 to 2048 columns), half of it here.
// `fill` puts u's halves into LDS (as fill_u) by way of all NW wavefronts.
template <int MB, bool NN, bool GR, int NW, class F>
MOE_DEV void expand_columns(const ExpandArgs& p, const SkinnyTile& t, int oz, char* lds, const F& fill) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int ksteps = (p.K + 31) / 32, kp = 32 * ksteps, lo_off = 16 * MB * kp * 2;
  const int g = lane >> 4, rho = lane & 15;
  size_t rowo[MB][4];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = t.row0 + min(16 * m + 4 * g + i, t.rows - 1);
      rowo[m][i] = (size_t)(GR ? p.src_token[r] : r) * p.nout + 8 * rho;
    }
  const bf16_t* W = p.w + (size_t)t.a * p.nout * p.K;
  const int blocks = (p.nout + 127) / 128, bper = (blocks + p.osplit - 1) / p.osplit;
  const int c1 = min(blocks, (oz + 1) * bper);
  const auto load_base = [&](int c, uint4 (&bs)[MB][4]) {
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        bs[m][i] = p.base && c * 128 + 8 * rho < p.nout
                       ? *(const uint4*)(p.base + rowo[m][i] + c * 128) : zero4();
  };
  const auto load_w = [&](int c, int ks, uint4 (&wf)[8]) {
    if constexpr (NN) {
      const int col = min(c * 128 + 8 * rho, p.nout - 8);
#pragma unroll
      for (int i = 0; i < 8; ++i)  // rows past K meet zeros of u
        wf[i] = *(const uint4*)(W + (size_t)min(32 * ks + 8 * g + i, p.K - 1) * p.nout + col);
    } else {
      const int k = 32 * ks + 8 * g;
#pragma unroll
      for (int f = 0; f < 8; ++f)
        wf[f] = k < p.K ? *(const uint4*)(W + (size_t)min(c * 128 + 8 * rho + f, p.nout - 1) * p.K + k)
                        : zero4();
    }
  };
  // the first block's loads go out before u is put together
  int c = oz * bper + wv;
  uint4 bs[MB][4], wf0[8], wf1[8];
  if (c < c1) {
    load_w(c, 0, wf0);
    load_base(c, bs);  // later blocks': at their start, after the stores before them
  }
  bool first = true;
  fill(kp);
  __syncthreads();
  if (p.ut) store_halves<MB, 64 * NW>(lds, lo_off, kp, p.K, t, oz, p.osplit, p.ut);
  for (; c < c1; c += NW) {
    if (!first) load_base(c, bs);
    first = false;
    f32x4v acc[MB][8];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int f = 0; f < 8; ++f) acc[m][f] = (f32x4v){0.f, 0.f, 0.f, 0.f};
    const auto step = [&](int ks, const uint4 (&wf)[8]) {
      bf16x8_t h[MB], l[MB];
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const char* a = lds + u_chunk(16 * m + rho, 4 * ks + g, kp);
        h[m] = as_frag(*(const uint4*)a);
        l[m] = as_frag(*(const uint4*)(a + lo_off));
      }
      uint4 w[8];
      if constexpr (NN) {
        transpose8(wf, w);
      } else {
#pragma unroll
        for (int f = 0; f < 8; ++f) w[f] = wf[f];
      }
#pragma unroll
      for (int f = 0; f < 8; ++f) {
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[m][f] = mfma16(l[m], as_frag(w[f]), acc[m][f]);
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[m][f] = mfma16(h[m], as_frag(w[f]), acc[m][f]);
      }
    };
    const bool more = c + NW < c1;
    for (int ks = 0; ks < ksteps; ks += 2) {
      if (ks + 1 < ksteps) load_w(c, ks + 1, wf1);
      else if (more) load_w(c + NW, 0, wf1);
      step(ks, wf0);
      if (ks + 1 < ksteps) {
        if (ks + 2 < ksteps) load_w(c, ks + 2, wf0);
        else if (more) load_w(c + NW, 0, wf0);
        step(ks + 1, wf1);
      } else {
#pragma unroll
        for (int f = 0; f < 8; ++f) wf0[f] = wf1[f];
      }
    }
    if (c * 128 + 8 * rho < p.nout) {
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (16 * m + 4 * g + i >= t.rows) continue;
          float f[8];
          unpack8(bs[m][i], f);
#pragma unroll
          for (int v = 0; v < 8; ++v) f[v] += acc[m][v][i];
          *(uint4*)(p.y + rowo[m][i] + c * 128) = cvt8(f);
        }
    }
  }
}

template <int MB, bool NN, bool GR>
__global__ __launch_bounds__(256, 2) void expand_kernel(ExpandArgs p) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  if (GR && (int)blockIdx.x >= p.max_tiles * p.osplit) {
    copy_ungrouped(p);
    return;
  }
  const int tile = blockIdx.x / p.osplit, oz = blockIdx.x % p.osplit;
  SkinnyTile t;
  if (!skinny_tile<GR>(p.counts, p.n, p.T, 16 * MB, tile, t)) return;
  expand_columns<MB, NN, GR, 4>(p, t, oz, lds, [&](int kp) {
    fill_u<16 * MB, GR ? 1 : 2, GR ? 8 : 1>(p, t, kp, lds);
  });
}

// Both products of few grouped rows in one launch (rank <= 16): every workgroup of a 16-row
// tile forms the tile's u anew and then its part of the columns.  The tile's rows of a and the
// group's of b come as whole KiB by direct loads into a ring of 512-deep stages, of which each
// of the 8 wavefronts takes two K steps (fragments straight from memory keep the address unit
// busy: 13 us for one token).  Bound by the chain of its stages, 14 of about 0.4 us for 7168
// (a ring of 7 is no faster).  Against the two launches, in a captured graph, 7168 columns in:
// one token 9.4 and 9.1 us (2048: 6.5 and 7.7), 96 tokens of 32 adapters 10.6 and 11.7 us, 256
// of 64 18.9 and 24.6, 1000 of 100 (4096) 18.6 and 24.5; called one by one it also saves the
// host's second launch.  It loses at rank 32 for few tiles (one token 11.6 and 10.8 us) and
// where K is long and few tiles fill the chip (16384 values, 96 tokens of 32 adapters 24.6 and
// 16.3 us; 512 of 128 29.6 and 37.1).
constexpr int DOT_EXPAND_STAGE = 32768, DOT_EXPAND_STAGES = 4, DOT_EXPAND_U = 2048;
template <bool NN>
__global__ __launch_bounds__(512) void dot_expand_kernel(DotArgs d, ExpandArgs p) {
  constexpr int NW = 8, NS = DOT_EXPAND_STAGES;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if ((int)blockIdx.x >= p.max_tiles * p.osplit) {
    copy_ungrouped(p);
    return;
  }
  const int tile = blockIdx.x / p.osplit, oz = blockIdx.x % p.osplit;
  SkinnyTile t;
  if (!skinny_tile<true>(p.counts, p.n, p.T, 16, tile, t)) return;
  char* ring = lds + DOT_EXPAND_U;  // behind u's halves
  expand_columns<1, NN, true, NW>(p, t, oz, lds, [&](int kp) {
    const uint32_t K2 = (uint32_t)d.K * 2;
    const rsrc_t ra = make_rsrc(d.a, (uint32_t)d.T * K2);  // below 4 GiB
    const rsrc_t rb = make_rsrc(d.b + (size_t)t.a * d.N * d.K, (uint32_t)d.N * K2);
    // this wavefront's rows, wv and wv + 8: nx of a's are the tile's.  A stage: 16 rows of a
    // (those past the tile are not loaded), 16 of b; chunk c of row r lies at c ^ r.
    const int nx = (wv < t.rows) + (wv + 8 < t.rows);
    uint32_t xo[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
      xo[q] = (uint32_t)d.src_token[t.row0 + min(wv + 8 * q, t.rows - 1)] * K2;
    const int stages = (d.K + 511) / 512;
    const auto issue = [&](int i) {
      char* st = ring + (i % NS) * DOT_EXPAND_STAGE;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int r = wv + 8 * q;
        const uint32_t k2 = (uint32_t)i * 1024 + ((lane ^ r) << 4);
        if (q < nx) dma16_buf(ra, k2 < K2 ? xo[q] + k2 : 0xffffffffu, 0u, st + r * 1024);
        dma16_buf(rb, k2 < K2 && r < d.N ? (uint32_t)r * K2 + k2 : 0xffffffffu, 0u,
                  st + 16384 + r * 1024);
      }
    };
    const auto wait = [&](int ahead) {  // 2 + nx loads a stage
      if (nx == 0) ring_wait_for<2>(ahead);
      else if (nx == 1) ring_wait_for<3>(ahead);
      else ring_wait_for<4>(ahead);
    };
    const int g = lane >> 4, m = lane & 15, mr = min(m, t.rows - 1);  // past the tile: its last row
    f32x4v acc = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < NS - 1 && i < stages; ++i) issue(i);
    for (int i = 0; i < stages; ++i) {
      wait(min(NS - 2, stages - 1 - i));
      if (i + NS - 1 < stages) issue(i + NS - 1);
      const char* st = ring + (i % NS) * DOT_EXPAND_STAGE;
      uint32_t ad[4];
      s16x8_t f[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int ch = 4 * (2 * wv + h) + g;
        ad[2 * h] = lds_at(st + mr * 1024 + ((ch ^ mr) << 4));
        ad[2 * h + 1] = lds_at(st + 16384 + m * 1024 + ((ch ^ m) << 4));
      }
      lds_read4(ad, f);
#pragma unroll
      for (int h = 0; h < 2; ++h)  // columns as the M side: a lane gets 4 neighbours
        acc = mfma16(__builtin_bit_cast(bf16x8_t, f[2 * h + 1]),
                     __builtin_bit_cast(bf16x8_t, f[2 * h]), acc);
    }
    __syncthreads();  // every wavefront is done with the ring
    f32x4v(*part)[64] = (f32x4v(*)[64])ring;
    part[wv][lane] = acc;
    __syncthreads();
    if (wv < kp / 16) {  // 4 columns of a row a lane, zeros from 16 on
      const float sc = p.scale ? p.scale[t.a] : 1.0f;
      f32x4v v = {0.f, 0.f, 0.f, 0.f};
      if (wv == 0)
#pragma unroll
        for (int q = 0; q < NW; ++q) v += part[q][lane];
      v *= sc;
      if (m >= t.rows) v = (f32x4v){0.f, 0.f, 0.f, 0.f};
      const int c = 16 * wv + 4 * g;
      const uint2 hi = cvt4(v);
      f32x4v lo;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = i < 2 ? hi.x : hi.y;
        const float f = __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
        lo[i] = fabsf(f) < INFINITY ? v[i] - f : 0.0f;
      }
      char* o = lds + u_chunk(m, c >> 3, kp) + (c & 7) * 2;
      *(uint2*)o = hi;
      *(uint2*)(o + 16 * kp * 2) = cvt4(lo);
    }
  });
}

// Many rows (64 MB a tile, 16 MB a wavefront): u stays in registers (KS K steps of 32) and
// the weights of SB column blocks pass through LDS in fragment order, shared by the four
// wavefronts, double-buffered: loaded from memory in whole lines while the blocks before
// are multiplied, turned in registers (NN) or by where they are written (NT).  K over 128
// (the router's dx) passes in halves of 128 with 64-row tiles, so that two workgroups fit a
// CU (58 us with all of K in LDS and one, 45 us with two; T = 4096, H = 7168, E = 256).
// Every load and store of the loop is a buffer access whose range does the masking: with
// branches around them the compiler waits for all that is in flight, stores included, which
// took a plain copy of this pattern from 48 to 73 us (8192 x 7168).
// 8192 rows of 7168 at rank 64: 56 to 57 us for 235 MB, against 45 to 48 us for that copy;
// the router's dx (46 us) spends 15 us on the start of its workgroups, which put 64 rows of
// d_logits in LDS first; after that nothing is full (matrix units 26 % busy, vector issue 23 %,
// 160 MB to and from memory), a wavefront reads its fragments, multiplies and stores in a row.
template <int MB, int KS, bool NN, bool GR>
__global__ __launch_bounds__(256, MB * KS <= 8 ? 2 : 1) void expand_tile_kernel(ExpandArgs p) {
  constexpr int SB = KS >= 4 ? 1 : 4 / KS;  // column blocks of a stage
  constexpr int KC = KS > 4 ? 4 : KS;       // K steps of a stage
  constexpr int STAGE = SB * KC * 8192;     // 32 KiB: a fragment group (8 KiB) a wavefront
  constexpr int ROWS = 64 * MB, KP = 32 * KS;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (GR && (int)blockIdx.x >= p.max_tiles * p.osplit) {
    copy_ungrouped(p);
    return;
  }
  const int tile = blockIdx.x / p.osplit, oz = blockIdx.x % p.osplit;
  SkinnyTile t;
  if (!skinny_tile<GR>(p.counts, p.n, p.T, ROWS, tile, t)) return;
  const int g = lane >> 4, rho = lane & 15;
  const bf16_t* W = p.w + (size_t)t.a * p.nout * p.K;
  const int blocks = (p.nout + 128 * SB - 1) / (128 * SB), bper = (blocks + p.osplit - 1) / p.osplit;
  const int s0 = oz * bper, s1 = min(blocks, s0 + bper);
  // a group's weights: past its K rows (NN) or columns (NT) zeros, without branches
  const rsrc_t rw = make_rsrc(W, (uint32_t)p.K * (uint32_t)p.nout * 2);
  u32x4_t wr[KS / KC][8];  // a stage ahead, two where a block has two stages
  const auto load_w = [&](int sb, int half, u32x4_t (&w)[8]) {
    if constexpr (NN) {  // K step ks of column block cb
      const int ks = wv % KC + half * KC, cb = wv / KC;
      const int col = min((sb * SB + cb) * 128 + 8 * rho, p.nout - 8);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = __builtin_amdgcn_raw_buffer_load_b128(
            rw, ((uint32_t)(32 * ks + 8 * g + i) * (uint32_t)p.nout + col) * 2, 0, 0);
    } else {  // the stage's rows of K values lie one after the other: 16-byte pieces in turn
      const uint32_t at = (uint32_t)(sb * SB * 128) * (uint32_t)p.K * 2;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = __builtin_amdgcn_raw_buffer_load_b128(rw, at + (i * 256 + threadIdx.x) * 16, 0, 0);
    }
  };
  const auto store_w = [&](char* st, const u32x4_t (&wr)[8]) {
    if constexpr (NN) {
      uint4 w[8], f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __builtin_bit_cast(uint4, wr[i]);
      transpose8(w, f);
      char* d = st + wv * 8192 + lane * 16;
#pragma unroll
      for (int i = 0; i < 8; ++i) *(uint4*)(d + i * 1024) = f[i];
    } else {
      // q / cpr for q < 2048, cpr <= 16: exact, as 2048 / 65536 < 1 / 16
      const int cpr = p.K >> 3, magic = (65535 + cpr) / cpr;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int q = i * 256 + (int)threadIdx.x, row = (q * magic) >> 16, c = q - row * cpr;
        if (q < SB * 128 * cpr)  // row 8 rho + f of block cb, chunk 4 ks + g
          *(uint4*)(st + (((row >> 7) * KS + (c >> 2)) * 8 + (row & 7)) * 1024 +
                    ((c & 3) * 16 + ((row >> 3) & 15)) * 16) = __builtin_bit_cast(uint4, wr[i]);
      }
    }
  };
  // byte offsets of this lane's rows; past the tile's rows or the columns: out of range,
  // where loads give zeros and stores nothing (as all of a null base), without branches
  constexpr uint32_t OUT = 0xffffffffu;
  const uint32_t nbytes = (uint32_t)p.T * (uint32_t)p.nout * 2;  // below 4 GiB
  const rsrc_t rb = make_rsrc(p.base, p.base ? nbytes : 0), ry = make_rsrc(p.y, nbytes);
  // what only the tile decides goes out first: weights, tokens, u
  if (s0 < s1) {
#pragma unroll
    for (int h = 0; h < KS / KC; ++h) load_w(s0, h, wr[h]);
  }
  uint32_t rowo[MB][4];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = t.row0 + min(16 * (MB * wv + m) + 4 * g + i, t.rows - 1);
      rowo[m][i] = (uint32_t)(GR ? p.src_token[row] : row);
    }
  constexpr int Q = ROWS * KP / 2048 < 8 ? ROWS * KP / 2048 : 8;
  fill_u<ROWS, Q, GR ? 8 / Q : 1>(p, t, KP, lds);
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      rowo[m][i] = 16 * (MB * wv + m) + 4 * g + i < t.rows
                       ? (rowo[m][i] * (uint32_t)p.nout + 8 * rho) * 2 : OUT;
  // base is read a block ahead where that fits the registers (small K: few blocks a
  // workgroup, each of which would wait for its own)
  constexpr bool AHEAD = MB * KS <= 2;
  u32x4_t bs[MB][4], bn[MB][4];
  const auto load_base = [&](int c, u32x4_t (&b)[MB][4]) {
    const bool in = c < s1 * SB && c * 128 + 8 * rho < p.nout;
    const auto get = [&](auto aux) {
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          b[m][i] = __builtin_amdgcn_raw_buffer_load_b128(
              rb, in && rowo[m][i] != OUT ? rowo[m][i] + (uint32_t)c * 256 : OUT, 0,
              decltype(aux)::value);
    };
    if (p.stream) get(std::integral_constant<int, 2>{});  // non-temporal
    else get(std::integral_constant<int, 0>{});
  };
  if (AHEAD) load_base(s0 * SB, bs);
  __syncthreads();
  if (p.ut) store_halves<4 * MB>(lds, ROWS * KP * 2, KP, p.K, t, oz, p.osplit, p.ut);
  bf16x8_t uh[MB][KS], ul[MB][KS];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const char* a = lds + u_chunk(16 * (MB * wv + m) + rho, 4 * ks + g, KP);
      uh[m][ks] = as_frag(*(const uint4*)a);
      ul[m][ks] = as_frag(*(const uint4*)(a + ROWS * KP * 2));
    }
  __syncthreads();
  // K values that no store below writes (of K = 96 a whole step): u is zero there, and zero
  // times what an earlier workgroup left in LDS may be NaN
  if (!NN && p.K < KP) {
    for (int i = threadIdx.x; i < 2 * STAGE / 16; i += 256) *(uint4*)(lds + i * 16) = zero4();
    __syncthreads();
  }
  if (s0 < s1) store_w(lds, wr[0]);
  __syncthreads();
  for (int sb = s0; sb < s1; ++sb) {
#pragma unroll 1  // short code: a workgroup that runs once pays for every line it fetches
    for (int cb = 0; cb < SB; ++cb) {
      const int c = sb * SB + cb;
      const bool in = c * 128 + 8 * rho < p.nout;
      if constexpr (AHEAD) load_base(c + 1, bn);
      else load_base(c, bs);
      f32x4v acc[MB][8];
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int f = 0; f < 8; ++f) acc[m][f] = (f32x4v){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int half = 0; half < KS / KC; ++half) {
        const int st = (sb - s0) * (KS / KC) + half;
        const char* cur = lds + (st & 1) * STAGE;
        const bool last_half = half + 1 == KS / KC;
        if (cb == 0) load_w(sb + 1, half, wr[half]);  // this half of the next block
#pragma unroll
        for (int kc = 0; kc < KC; ++kc)
#pragma unroll
          for (int f4 = 0; f4 < 8; f4 += 4) {
            const int ks = half * KC + kc;
            bf16x8_t w[4];
#pragma unroll
            for (int f = 0; f < 4; ++f)
              w[f] = as_frag(*(const uint4*)(cur + ((cb * KC + kc) * 8 + f4 + f) * 1024 + lane * 16));
#pragma unroll
            for (int f = 0; f < 4; ++f)
#pragma unroll
              for (int m = 0; m < MB; ++m) acc[m][f4 + f] = mfma16(ul[m][ks], w[f], acc[m][f4 + f]);
#pragma unroll
            for (int f = 0; f < 4; ++f)
#pragma unroll
              for (int m = 0; m < MB; ++m) acc[m][f4 + f] = mfma16(uh[m][ks], w[f], acc[m][f4 + f]);
          }
        if (!last_half) {  // SB is 1 here
          store_w(lds + ((st + 1) & 1) * STAGE, wr[(half + 1) % (KS / KC)]);
          __syncthreads();
        }
      }
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[8];
          unpack8(__builtin_bit_cast(uint4, bs[m][i]), f);
#pragma unroll
          for (int v = 0; v < 8; ++v) f[v] += acc[m][v][i];
          bs[m][i] = __builtin_bit_cast(u32x4_t, cvt8(f));
        }
      const auto put = [&](auto aux) {
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            __builtin_amdgcn_raw_buffer_store_b128(
                bs[m][i], ry, in && rowo[m][i] != OUT ? rowo[m][i] + (uint32_t)c * 256 : OUT, 0,
                decltype(aux)::value);
      };
      if (p.stream) put(std::integral_constant<int, 2>{});  // non-temporal
      else put(std::integral_constant<int, 0>{});
      if constexpr (AHEAD) {
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) bs[m][i] = bn[m][i];
      }
    }
    // the next stage's weights (past the last: not used)
    store_w(lds + ((sb + 1 - s0) * (KS / KC) & 1) * STAGE, wr[0]);
    __syncthreads();
  }
}

// ----------------------------------------------------------------------- wgrad
// A workgroup of 4 wavefronts forms 16 JT WJ rows (j) x 128 columns (h) of one group's
// gradient over one chunk of its rows; WJ wavefronts share out j, the others the chunk's
// 32-row tiles, whose sums are joined in LDS at the end.  Both operands reach LDS by direct
// loads into a ring of 32-row tiles, x as whole 256-byte pieces of its rows, the short one
// as the halves that `expand` left in fragment order, so that enough is in flight without
// registers (8192 rows of 7168 at rank 64, x and dy: 235 MB in 58 us; with both in registers
// one tile ahead 88 us).  The router's (256 x 7168 over 4096 rows) takes 37 us, in which
// nothing is full (matrix units 32 % busy, vector issue 24 %, 352 MB out of L2, 124 MB to and
// from memory): each wavefront waits for its reads, turns them and multiplies in a row, two
// wavefronts a SIMD, and eight repeat the turning for 32 rows of j each; 64 rows each leave
// one wavefront a SIMD and take 46 us.  A lane reads 8 rows of 8 columns and turns them in
// registers into 8 fragments along the rows; row i of fragment f stands for column 8 i + f.
// With the halves as the M side a lane ends with 4 neighbouring j of 8 neighbouring h: it
// stores 8 h of a row (16 lanes: 128 of them) for [J][H], 4 j for [H][J] (TR).
template <int JT, int WJ>
struct WgradTile {
  static constexpr int WK = 4 / WJ, JB = JT * WJ;       // 16-row blocks of j
  static constexpr int UB = JB < 2 ? 4096 : JB * 2048;  // bytes of halves a tile
  static constexpr int STAGE = WK * (8192 + UB);        // a tile for each wavefront along K
  static constexpr int NS = STAGE <= 16384 ? 4 : 3;  // 76, 68, 76 KiB with the tokens: 2 a CU
  static constexpr int LOADS = WK * (2 + UB / 4096);    // per wavefront and stage
  static constexpr int TOK = 4 * WGRAD_MAX_CHUNK;
  static constexpr int LDS = NS * STAGE + TOK;
};

// 8 x 16 bytes of x (256 apart) and 2 JT x 16 bytes of halves (1024 apart)
MOE_DEV void lds_read_x(uint32_t a, s16x8_t (&x)[8]) {
  asm volatile(
      "ds_read_b128 %0, %8\n\tds_read_b128 %1, %8 offset:256\n\t"
      "ds_read_b128 %2, %8 offset:512\n\tds_read_b128 %3, %8 offset:768\n\t"
      "ds_read_b128 %4, %8 offset:1024\n\tds_read_b128 %5, %8 offset:1280\n\t"
      "ds_read_b128 %6, %8 offset:1536\n\tds_read_b128 %7, %8 offset:1792\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]),
        "=&v"(x[6]), "=&v"(x[7])
      : "v"(a)
      : "memory");
}
MOE_DEV void lds_read_u(uint32_t a, s16x8_t (&u)[2][2]) {
  asm volatile(
      "ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:1024\n\t"
      "ds_read_b128 %2, %4 offset:2048\n\tds_read_b128 %3, %4 offset:3072\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(u[0][0]), "=&v"(u[0][1]), "=&v"(u[1][0]), "=&v"(u[1][1])
      : "v"(a)
      : "memory");
}
MOE_DEV void lds_read_u(uint32_t a, s16x8_t (&u)[1][2]) {
  asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:1024\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(u[0][0]), "=&v"(u[0][1])
               : "v"(a)
               : "memory");
}
MOE_DEV int lds_read_int(uint32_t a) {
  int v;
  asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(v) : "v"(a) : "memory");
  return v;
}

template <int JT, int WJ, bool GR, bool TR>
MOE_DEV void wgrad_body(const WgradArgs& p, const WgradSide& d, int hb, int cj, char* lds) {
  using C = WgradTile<JT, WJ>;
  constexpr int WK = C::WK;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int h0 = hb * 128, ch = cj / p.jblk;
  const int jb0 = (cj % p.jblk) * C::JB, wj = wv % WJ, wk = wv / WJ;
  const int crows = p.chunk_rows;
  GroupPos gp;
  int nch;
  if (GR) {
    const auto units = [crows](int c) { return max(1, (c + crows - 1) / crows); };
    if (!find_group(p.counts, p.n, ch, units, gp)) return;
    nch = units(gp.count);
  } else {
    nch = max(1, (p.T + crows - 1) / crows);
    gp.a = 0;
    gp.unit = ch;
    gp.count = p.T;
    gp.row0 = gp.t32 = 0;
  }
  const int r0 = gp.unit * crows, rows = max(0, min(crows, gp.count - r0));
  const int row0 = gp.row0 + r0;
  char* tok = lds + C::NS * C::STAGE;  // the chunk's tokens
  if (GR) {
    int32_t v[WGRAD_MAX_CHUNK / 256];
#pragma unroll
    for (int q = 0; q < WGRAD_MAX_CHUNK / 256; ++q)  // rows past the last repeat it
      v[q] = rows > 0 ? p.src_token[row0 + min((int)threadIdx.x + 256 * q, rows - 1)] : 0;
#pragma unroll
    for (int q = 0; q < WGRAD_MAX_CHUNK / 256; ++q) ((int32_t*)tok)[threadIdx.x + 256 * q] = v[q];
    __syncthreads();
  }
  const int g = lane >> 4, rho = lane & 15;
  const int jb = (p.J + 15) / 16;
  constexpr uint32_t OUT = 0xffffffffu;
  const rsrc_t rx = make_rsrc(d.x, (uint32_t)p.T * (uint32_t)d.H * 2);  // below 4 GiB
  const bool cin = h0 + 8 * rho < d.H;
  // the chunk's halves, jb * 2048 bytes a tile, from block jb0 on
  const int tiles = (rows + 31) / 32;
  const rsrc_t ru = make_rsrc(d.ut + (size_t)(gp.t32 + (r0 >> 5)) * jb * 1024,
                              (uint32_t)tiles * (uint32_t)jb * 2048);
  f32x4v acc[JT][8];
#pragma unroll
  for (int i = 0; i < JT; ++i)
#pragma unroll
    for (int f = 0; f < 8; ++f) acc[i][f] = (f32x4v){0.f, 0.f, 0.f, 0.f};
  const int stages = (tiles + WK - 1) / WK;
  const auto issue = [&](int st) {
    char* dst = lds + (st % C::NS) * C::STAGE;
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      const int tt = st * WK + w;
#pragma unroll
      for (int q = 0; q < 2; ++q) {  // rows 4 (2 wv + q) .. + 3: lane L row L / 16, 16 (L % 16)
        const int m = 32 * tt + 4 * (2 * wv + q) + g;
        uint32_t off = OUT;
        if (GR) {
          const int tk = lds_read_int(lds_at(tok) + 4 * min(m, WGRAD_MAX_CHUNK - 1));
          if (m < rows && cin) off = ((uint32_t)tk * (uint32_t)d.H + h0 + 8 * rho) * 2;
        } else {
          if (m < rows && cin) off = ((uint32_t)(row0 + m) * (uint32_t)d.H + h0 + 8 * rho) * 2;
        }
        dma16_buf(rx, off, 0u, dst + w * 8192 + (2 * wv + q) * 1024);
      }
#pragma unroll
      for (int q = 0; q < C::UB / 4096; ++q) {  // 1 KiB pieces; of blocks past the last: zeros
        const int piece = q * 4 + wv;
        const bool in = tt < tiles && jb0 * 2 + piece < jb * 2;
        dma16_buf(ru, in ? (uint32_t)(tt * jb + jb0) * 2048 + piece * 1024 + lane * 16 : OUT, 0u,
                  dst + WK * 8192 + w * C::UB + piece * 1024);
      }
    }
  };
  for (int st = 0; st < C::NS - 1 && st < stages; ++st) issue(st);
  for (int st = 0; st < stages; ++st) {
    ring_wait_for<C::LOADS>(min(C::NS - 2, stages - 1 - st));
    if (st + C::NS - 1 < stages) issue(st + C::NS - 1);
    const char* cur = lds + (st % C::NS) * C::STAGE;
    s16x8_t x[8], u[JT][2];
    lds_read_x(lds_at(cur + wk * 8192) + 8 * g * 256 + rho * 16, x);
    lds_read_u(lds_at(cur + WK * 8192 + wk * C::UB) + wj * JT * 2048 + lane * 16, u);
    uint4 xr[8], f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) xr[i] = __builtin_bit_cast(uint4, x[i]);
    transpose8(xr, f);
#pragma unroll
    for (int v = 0; v < 8; ++v)
#pragma unroll
      for (int h = 1; h >= 0; --h)
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          const bf16x8_t uf = __builtin_bit_cast(bf16x8_t, u[j][h]);
          acc[j][v] = mfma16(uf, as_frag(f[v]), acc[j][v]);
        }
  }
  __syncthreads();  // every wavefront is done with the ring
  if constexpr (WK > 1) {
    f32x4v(*part)[8][64] = (f32x4v(*)[8][64])lds;
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int h = WK / 2; h >= 1; h /= 2) {
        __syncthreads();
        if (wk >= h && wk < 2 * h)
#pragma unroll
          for (int v = 0; v < 8; ++v) part[(wk - h) * WJ + wj][v][lane] = acc[j][v];
        __syncthreads();
        if (wk < h)
#pragma unroll
          for (int v = 0; v < 8; ++v) acc[j][v] += part[wk * WJ + wj][v][lane];
      }
    if (wk) return;
  }
  const size_t per = (size_t)p.J * d.H;
  float* part = d.parts + (size_t)ch * per;
  bf16_t* out = d.out + (size_t)gp.a * per;
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    if constexpr (TR) {
      const int jj = (jb0 + wj * JT + j) * 16 + 4 * g;
      if (jj >= p.J) continue;  // J is a multiple of 8 here
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const int h = h0 + 8 * rho + v;
        if (h >= d.H) continue;
        const f32x4v a = acc[j][v];
        const size_t at = (size_t)h * p.J + jj;
        if (nch > 1) *(f32x4v*)(part + at) = a;
        else *(uint2*)(out + at) = cvt4(a);
      }
    } else {
      const int h = h0 + 8 * rho;
      if (h >= d.H) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int jj = (jb0 + wj * JT + j) * 16 + 4 * g + i;
        if (jj >= p.J) continue;
        float f[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) f[v] = acc[j][v][i];
        const size_t at = (size_t)jj * d.H + h;
        if (nch > 1) {
          *(float4*)(part + at) = make_float4(f[0], f[1], f[2], f[3]);
          *(float4*)(part + at + 4) = make_float4(f[4], f[5], f[6], f[7]);
        } else {
          *(uint4*)(out + at) = cvt8(f);
        }
      }
    }
  }
}

template <int JT, int WJ, bool GR>
__global__ __launch_bounds__(256) void wgrad_kernel(WgradArgs p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int hb = blockIdx.x % p.hblk, rest = blockIdx.x / p.hblk;
  const bool second = hb >= p.hblk0;
  const WgradSide d = p.side[second ? 1 : 0];
  if (GR && d.transposed) wgrad_body<JT, WJ, GR, true>(p, d, hb - (second ? p.hblk0 : 0), rest, lds);
  else wgrad_body<JT, WJ, GR, false>(p, d, hb, rest, lds);
}

// Gradients of the groups with several chunks: the sum of the chunks' parts, in order.
// Bound by memory: 256 x 7168, 4 parts, 33 MB in 6.3 us.
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
#pragma unroll 4
  for (int c = 0; c < nch; ++c) v += *(const f32x4v*)(d.parts + (size_t)(first + c) * per + i);
  *(uint2*)(d.out + (size_t)a * per + i) =
      cvt4(v);
}

// ------------------------------------------------------------------- transpose
// dst [n][C][R] = src [n][R][C] transposed (R and C multiples of 8); 64 x 64 tiles, rows of
// 66 values in LDS so that a column's reads spread over the banks.  8 x 7168 x 64: 4.7 us,
// half of it the launch.
__global__ __launch_bounds__(256) void transpose_kernel(const bf16_t* __restrict__ src_all,
                                                        bf16_t* __restrict__ dst_all, int R, int C) {
  __shared__ bf16_t t[64][66];
  const int rt = (R + 63) / 64;
  const int r0 = (blockIdx.x % rt) * 64, c0 = (blockIdx.x / rt) * 64;
  const bf16_t* src = src_all + (size_t)blockIdx.y * R * C;
  bf16_t* dst = dst_all + (size_t)blockIdx.y * R * C;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = threadIdx.x + 256 * q, r = i >> 3, c = (i & 7) * 8;
    uint4 v = zero4();
    if (r0 + r < R && c0 + c < C) v = *(const uint4*)(src + (size_t)(r0 + r) * C + c0 + c);
#pragma unroll
    for (int w = 0; w < 4; ++w) *(uint32_t*)&t[r][c + 2 * w] = u4_word(v, w);
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = threadIdx.x + 256 * q, c = i >> 3, r = (i & 7) * 8;
    if (c0 + c >= C || r0 + r >= R) continue;
    uint32_t w[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) w[v] = t[r + 2 * v][c] | ((uint32_t)t[r + 2 * v + 1][c] << 16);
    *(uint4*)(dst + (size_t)(c0 + c) * R + r0 + r) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

int div_up(int a, int b) { return (a + b - 1) / b; }

template <int NB>
hipError_t dot_small(const char* name, const DotArgs& p, int tiles, hipStream_t s) {
  const unsigned g = (unsigned)((long)tiles * div_up(p.N, 16 * NB) * p.S);
  if (p.counts) return MOE_LAUNCH(name, s, dot_kernel<NB, true><<<g, 512, 0, s>>>(p));
  return MOE_LAUNCH(name, s, dot_kernel<NB, false><<<g, 512, 0, s>>>(p));
}

template <int BM, int BN>
hipError_t dot_tiles(const char* name, const DotArgs& p, int tiles, hipStream_t s) {
  const unsigned g = (unsigned)((long)tiles * div_up(p.N, BN) * p.S);
  using C = DotTile<BM, BN>;
  constexpr unsigned lds = C::NS * C::STAGE;
  if constexpr (BM == 64 || BN == 64)
    if (p.counts)
      return MOE_LAUNCH(name, s, dot_tile_kernel<BM, BN, true><<<g, C::NT, lds, s>>>(p));
  return MOE_LAUNCH(name, s, dot_tile_kernel<BM, BN, false><<<g, C::NT, lds, s>>>(p));
}

// below 2^32 threads: 4 T of the tiles (T < 2^26) and 2^30 or 2^31 of the copies
unsigned expand_grid(const ExpandArgs& p, int waves = 4) {
  const long extra =  // copy_ungrouped
      p.counts && p.base != p.y ? std::min(div_up(p.T, waves), COPY_GROUPS) : 0;
  return (unsigned)((long)p.max_tiles * p.osplit + extra);
}

template <int MB, bool NN, bool GR>
hipError_t expand_small(const char* name, const ExpandArgs& p, hipStream_t s) {
  const unsigned lds = 16u * MB * 32 * div_up(p.K, 32) * 4;
  auto* k = expand_kernel<MB, NN, GR>;
  return MOE_LAUNCH(name, s, k<<<expand_grid(p), 256, lds, s>>>(p));
}

// Outputs of this size and more leave with non-temporal stores, and their base comes with
// non-temporal loads: the Infinity Cache (256 MB) would hold them, the outputs dirty, to be
// written back under the kernels that follow, in the place of the dy that the weight
// gradients read next.  8192 x 7168 at rank 64, forward and backward: 289 -> 268 us.
constexpr size_t STREAM_BYTES = 32u << 20;

template <int MB, int KS, bool NN, bool GR>
hipError_t expand_tiles(const char* name, const ExpandArgs& p, hipStream_t s) {
  const unsigned w = 2u * 32768, u = 64u * MB * 32 * KS * 4;
  auto* k = expand_tile_kernel<MB, KS, NN, GR>;
  return MOE_LAUNCH(name, s, k<<<expand_grid(p), 256, w > u ? w : u, s>>>(p));
}

template <bool NN, bool GR>
hipError_t expand_ks(const char* name, const ExpandArgs& p, const ExpandPlan& c, hipStream_t s) {
  if (c.ks == 0) {
    if constexpr (!GR)  // rank <= 128: grouped tiles of 64 rows and more have their K steps
      if (c.mb == 2) return expand_small<2, NN, GR>(name, p, s);
    return expand_small<1, NN, GR>(name, p, s);
  }
  if (c.ks == 8) {
    if constexpr (!GR) return expand_tiles<1, 8, NN, GR>(name, p, s);  // rank <= 128
    return hipErrorNotSupported;
  }
  if (c.mb == 1) {
    if (c.ks == 1) return expand_tiles<1, 1, NN, GR>(name, p, s);
    if (c.ks == 2) return expand_tiles<1, 2, NN, GR>(name, p, s);
    return expand_tiles<1, 4, NN, GR>(name, p, s);
  }
  if (c.ks == 1) return expand_tiles<2, 1, NN, GR>(name, p, s);
  if (c.ks == 2) return expand_tiles<2, 2, NN, GR>(name, p, s);
  return expand_tiles<2, 4, NN, GR>(name, p, s);
}

int row_tiles(int T, int n, bool grouped, int rows) {
  return div_up(T, rows) + (grouped ? (n < T ? n : T) : 0);
}

}  // namespace

SkinnyPlan skinny_plan(int T, int n, bool grouped, int K, int N) {
  SkinnyPlan c;
  const int groups = !grouped ? 1 : (n < T ? n : T);
  c.few = !grouped && T <= DOT_FEW;
  c.tile = T >= 32 * groups;
  // dot_expand_kernel: one workgroup's stages along K against parts of K on many
  const int tiles16 = row_tiles(T, n, grouped, 16);
  c.fused = grouped && !c.tile && N <= 16 && tiles16 <= FUSED_TILES && (K <= 8192 || tiles16 >= 128);
  c.bn = !c.tile ? (N <= 16 ? 16 : (N <= 32 ? 32 : 64)) : (N <= 32 ? 32 : (N <= 64 ? 64 : 128));
  // 128 rows halve the weights' way through a CU's L1: at 64 columns where that outweighs the
  // longer start (8192 rows of 7168: rank 64 of 8 adapters 35 -> 32 us, E = 64 29 -> 25; 4096
  // rows the same; 8192 rows of 2048 12 -> 13, 1024 of 7168 11 -> 12), not at 32, where x is
  // most of it (rank 16: 92 -> 95 us with the second product), nor at 128 for groups, whose
  // ragged tiles then leave CUs idle (rank 128: 66 -> 74 us)
  const bool tall = c.bn == 64 ? (int64_t)T * K >= 1 << 25 && T >= 128 * groups
                               : c.bn == 128 && !grouped && T >= 1024;
  c.bm = !c.tile ? 16 : (tall ? 128 : 64);
  c.tiles = row_tiles(T, n, grouped, c.bm);
  const int wg = c.tiles * div_up(N, c.bn);
  // at least two steps of each of 8 wavefronts, or a ring's stages
  const int most = div_up(K, c.tile ? 512 : 1024);
  int want = 1;  // at most 8: every part is read again by the second product
  if (c.bm == 128) {
    // One workgroup a CU: whole rounds of 256, against the sum of the parts, which takes
    // about 1/64 of a round for each part of 64 tiles (4096 x 384 x 7168: 59 -> 49 us).
    float least = 0.0f;
    for (int S = 1; S <= 8; ++S) {
      const float cost = (float)div_up(wg * S, 256) / S + (float)wg * S / 4096;
      if (S == 1 || cost < least) least = cost, want = S;
    }
  } else {
    const int target = c.tile ? (c.bn == 128 ? 256 : 384) : 512;
    want = wg > 0 ? div_up(target, wg) : 1;
    if (want > 8) want = 8;
  }
  c.S = c.few || c.fused ? 1 : (want < most ? want : most);
  return c;
}

hipError_t launch_dot(const char* name, const DotArgs& p, const SkinnyPlan& c, hipStream_t s) {
  if (p.T == 0) return hipSuccess;
  if (c.few) {
    if (p.T <= 1) return MOE_LAUNCH(name, s, dot_few_kernel<1><<<(unsigned)p.N, 256, 0, s>>>(p));
    if (p.T <= 4) return MOE_LAUNCH(name, s, dot_few_kernel<4><<<(unsigned)p.N, 256, 0, s>>>(p));
    if (p.T <= 8) return MOE_LAUNCH(name, s, dot_few_kernel<8><<<(unsigned)p.N, 256, 0, s>>>(p));
    return MOE_LAUNCH(name, s, dot_few_kernel<DOT_FEW><<<(unsigned)p.N, 256, 0, s>>>(p));
  }
  if (!c.tile) {
    if (c.bn == 16) return dot_small<1>(name, p, c.tiles, s);
    if (c.bn == 32) return dot_small<2>(name, p, c.tiles, s);
    return dot_small<4>(name, p, c.tiles, s);
  }
  if (c.bm == 64) {
    if (c.bn == 32) return dot_tiles<64, 32>(name, p, c.tiles, s);
    if (c.bn == 64) return dot_tiles<64, 64>(name, p, c.tiles, s);
    return dot_tiles<64, 128>(name, p, c.tiles, s);
  }
  if (c.bn == 64) return dot_tiles<128, 64>(name, p, c.tiles, s);
  return dot_tiles<128, 128>(name, p, c.tiles, s);
}

hipError_t launch_sum_parts(const char* name, const float* parts, int S, size_t n, float* out,
                            hipStream_t s) {
  if (n == 0) return hipSuccess;
  return MOE_LAUNCH(name, s, sum_parts_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(parts, S, n, out));
}

ExpandPlan expand_plan(int T, int n, bool grouped, int K, int nout) {
  ExpandPlan c;
  const int groups = !grouped ? 1 : (n < T ? n : T);
  if (T < 32 * groups || K > 256) {
    c.ks = 0;
    c.mb = T >= 32 * groups && K <= 512 ? 2 : 1;  // the rows' halves take at most 64 KiB of LDS
    c.tiles = row_tiles(T, n, grouped, 16 * c.mb);
    const int most = div_up(div_up(nout, 128), 4), w = c.tiles > 0 ? div_up(1024, c.tiles) : 1;
    c.osplit = w < most ? w : most;
  } else {
    c.ks = K <= 32 ? 1 : (K <= 64 ? 2 : (K <= 128 ? 4 : 8));
    const int stages = div_up(nout, c.ks >= 4 ? 128 : 512 / c.ks);
    // 128 rows a tile halve the weights' way through LDS; 64 where that leaves CUs idle
    c.mb = c.ks < 8 && T >= 128 * groups && row_tiles(T, n, grouped, 128) * stages >= 512 ? 2 : 1;
    c.tiles = row_tiles(T, n, grouped, 64 * c.mb);
    const int w = c.tiles > 0 ? 512 / c.tiles : 1;  // one round of workgroups, 2 a CU
    c.osplit = w < 1 ? 1 : (w < stages ? w : stages);
  }
  return c;
}

hipError_t launch_expand(const char* name, ExpandArgs p, const ExpandPlan& c, bool nn,
                         hipStream_t s) {
  if (p.T == 0) return hipSuccess;
  p.stream = (size_t)p.T * p.nout * 2 >= STREAM_BYTES;
  if (!p.counts) return expand_ks<true, false>(name, p, c, s);
  return nn ? expand_ks<true, true>(name, p, c, s) : expand_ks<false, true>(name, p, c, s);
}

hipError_t launch_dot_expand(const char* name, const DotArgs& d, ExpandArgs p, bool nn, hipStream_t s) {
  if (p.T == 0) return hipSuccess;
  p.stream = 0;
  p.max_tiles = row_tiles(p.T, p.n, true, 16);
  const int most = div_up(div_up(p.nout, 128), 8), w = p.max_tiles < 256 ? 256 / p.max_tiles : 1;
  p.osplit = w < most ? w : most;
  const unsigned g = expand_grid(p, 8), lds = DOT_EXPAND_U + DOT_EXPAND_STAGES * DOT_EXPAND_STAGE;
  if (nn) return MOE_LAUNCH(name, s, dot_expand_kernel<true><<<g, 512, lds, s>>>(d, p));
  return MOE_LAUNCH(name, s, dot_expand_kernel<false><<<g, 512, lds, s>>>(d, p));
}

int wgrad_chunk(int T, int hblocks, int J) {
  const int wg = hblocks * div_up(J, 128);
  const int chunks = wg < 512 ? 512 / wg : 1;
  const int r = div_up(div_up(T > 0 ? T : 1, chunks), 128) * 128;
  return r > WGRAD_MAX_CHUNK ? WGRAD_MAX_CHUNK : r;
}

int wgrad_chunk_slots(int T, int n, bool grouped, int chunk_rows) {
  return grouped ? T / chunk_rows + n : (T > 0 ? div_up(T, chunk_rows) : 1);
}

hipError_t launch_wgrad(const char* name, WgradArgs p, int sides, hipStream_t s) {
  const int hmax = sides > 1 && p.side[1].H > p.side[0].H ? p.side[1].H : p.side[0].H;
  const int slots = wgrad_chunk_slots(p.T, p.n, p.counts != nullptr, p.chunk_rows);
  p.jblk = div_up(p.J, 128);
  p.hblk0 = div_up(p.side[0].H, 128);
  p.hblk = p.hblk0 + (sides > 1 ? div_up(p.side[1].H, 128) : 0);
  const unsigned g = (unsigned)((long)p.hblk * slots * p.jblk);
  hipError_t e;
#define MOE_WGRAD_GO(JT, WJ)                                                                     \
  e = p.counts ? MOE_LAUNCH(name, s,                                                             \
                            wgrad_kernel<JT, WJ, true><<<g, 256, WgradTile<JT, WJ>::LDS, s>>>(p)) \
               : MOE_LAUNCH(name, s,                                                             \
                            wgrad_kernel<JT, WJ, false><<<g, 256, WgradTile<JT, WJ>::LDS, s>>>(p))
  if (p.J <= 32) MOE_WGRAD_GO(1, 2);
  else if (p.J <= 64) MOE_WGRAD_GO(1, 4);
  else MOE_WGRAD_GO(2, 4);
#undef MOE_WGRAD_GO
  if (e != hipSuccess || p.T <= p.chunk_rows) return e;
  const size_t per = (size_t)p.J * hmax;
  const dim3 gs((unsigned)((per + 1023) / 1024), (unsigned)(p.counts ? p.n : 1), (unsigned)sides);
  if (p.counts) return MOE_LAUNCH("wgrad_sum", s, wgrad_sum_kernel<true><<<gs, 256, 0, s>>>(p));
  return MOE_LAUNCH("wgrad_sum", s, wgrad_sum_kernel<false><<<gs, 256, 0, s>>>(p));
}

hipError_t launch_transpose(const char* name, int n, const bf16_t* src, bf16_t* dst, int R, int C,
                            hipStream_t s) {
  const dim3 g((unsigned)(div_up(R, 64) * div_up(C, 64)), (unsigned)n);
  return MOE_LAUNCH(name, s, transpose_kernel<<<g, 256, 0, s>>>(src, dst, R, C));
}

}  // namespace moe
