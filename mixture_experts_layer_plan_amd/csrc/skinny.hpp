// Launch functions of the products with one short side (skinny.hip).
#pragma once

#include "common.hpp"
#include "internal.hpp"

namespace moe {

// Grouped launches (counts != nullptr): group a has counts[a] rows, the groups' rows one
// after the other; row r is token src_token[r].  Others: T rows, one set of weights.

// out [S][R][N] (fp32): part s of K of out[m, j] = sum_k a[m, k] b[j, k]
struct DotArgs {
  const bf16_t* a;  // rows of K values, by token
  const bf16_t* b;  // [n][N][K]
  float* out;
  const int32_t* counts;
  const int32_t* src_token;
  int n, T, K, N, S;
  size_t R;  // rows of one part
};

// y[m, :] = base[m, :] + (scale_a sum over parts of u[m, :]) w^T, rounded once
struct ExpandArgs {
  const float* u;  // [S][R][K]
  const bf16_t* w;  // [n][nout][K], or nn: [n][K][nout]
  const bf16_t* base;  // by token, or null (zero); may be y
  bf16_t* y;
  const float* scale;  // [n] or null
  bf16_t* ut;          // halves of the scaled u along the rows, or null
  const int32_t* counts;
  const int32_t* src_token;
  const int32_t* pos;  // row of each token, < 0: none (its y is its base)
  int n, T, K, S, nout, max_tiles, osplit;
  int stream;  // set by launch_expand
  size_t R;
};
// bytes of the halves of `rows` rows in n groups, K values each
inline size_t halves_bytes(size_t rows, int n, int K) {
  return (rows / 32 + n) * (size_t)((K + 15) / 16) * 2048;
}

// out[a] = sum over group a's rows of u (x) x: [J][H], or [H][J] if transposed
struct WgradSide {
  const bf16_t* ut;
  const bf16_t* x;  // by token
  bf16_t* out;
  float* parts;     // [chunk slots][J * H]
  int H, transposed;
};
struct WgradArgs {
  WgradSide side[2];
  const int32_t* counts;
  const int32_t* src_token;
  int n, T, J, chunk_rows;
  int jblk, hblk, hblk0;  // set by launch_wgrad
};

constexpr int WGRAD_MAX_CHUNK = 1024;  // rows of one chunk (their tokens lie in LDS)
constexpr int DOT_FEW = 16;            // tokens of the dot without matrix instructions
constexpr int FUSED_TILES = 256;       // 16-row tiles of both products in one launch

// How a dot or an expand of T rows in n groups (one if not grouped) is cut up: from the
// sizes alone, so that the order of every sum is too.  tiles: row tiles, an upper bound.
struct SkinnyPlan {
  bool few, tile;  // dot_few_kernel; dot_tile_kernel (else dot_kernel)
  bool fused;      // launch_dot_expand for both products
  int bm, bn, tiles, S;
};
SkinnyPlan skinny_plan(int T, int n, bool grouped, int K, int N);
struct ExpandPlan {
  int ks;  // K steps of expand_tile_kernel, 0: expand_kernel
  int mb, tiles, osplit;
};
ExpandPlan expand_plan(int T, int n, bool grouped, int K, int nout);
int wgrad_chunk(int T, int hblocks, int J);      // rows of a chunk; 128-column blocks of all sides
int wgrad_chunk_slots(int T, int n, bool grouped, int chunk_rows);

hipError_t launch_dot(const char* name, const DotArgs& p, const SkinnyPlan& c, hipStream_t s);
hipError_t launch_sum_parts(const char* name, const float* parts, int S, size_t n, float* out,
                            hipStream_t s);
hipError_t launch_expand(const char* name, ExpandArgs p, const ExpandPlan& c, bool nn,
                         hipStream_t s);
// Both products of few grouped rows (SkinnyPlan::fused); p.u and p.S are not used.
hipError_t launch_dot_expand(const char* name, const DotArgs& d, ExpandArgs p, bool nn, hipStream_t s);
hipError_t launch_wgrad(const char* name, WgradArgs p, int sides, hipStream_t s);
// dst [n][C][R] from src [n][R][C]
hipError_t launch_transpose(const char* name, int n, const bf16_t* src, bf16_t* dst, int R, int C,
                            hipStream_t s);

}  // namespace moe
