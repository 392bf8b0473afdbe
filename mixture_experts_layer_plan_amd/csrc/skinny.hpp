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
  const bf16_t* w; // [n][nout][wld], wld >= K, zeros past K
  const bf16_t* base;  // by token, or null (zero); may be y
  bf16_t* y;
  const float* scale;  // [n] or null
  bf16_t* ut;          // halves of the scaled u along the rows, or null
  const int32_t* counts;
  const int32_t* src_token;
  const int32_t* pos;  // row of each token, < 0: none (its y is its base)
  int n, T, K, S, wld, nout, max_tiles, osplit;
  size_t R;
};
// bytes of the halves of `rows` rows in n groups, K values each
inline size_t halves_bytes(size_t rows, int n, int K) { return (rows / 16 + n) * (size_t)K * 64; }

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
  int n, T, J, chunk_rows, jblk;
};

struct TransposeArgs {
  const bf16_t* src;
  bf16_t* dst;
  int R, C, ldd;
};

// Row tile, row tiles (an upper bound) and K parts of a dot over T rows in n groups
// (one if not grouped): from the sizes alone, so that the order of every sum is too.
struct SkinnyPlan {
  int mb, tiles, S;
};
SkinnyPlan skinny_plan(int T, int n, bool grouped, int K, int N);
int skinny_tiles(int T, int n, bool grouped, int mb);  // row tiles of 16 mb rows, at most
int expand_osplit(int tiles, int nout);
int wgrad_chunk_slots(int T, int n, int chunk_rows);

hipError_t launch_dot(const char* name, const DotArgs& p, int mb, int tiles, hipStream_t s);
hipError_t launch_sum_parts(const char* name, const float* parts, int S, size_t n, float* out,
                            hipStream_t s);
hipError_t launch_expand(const char* name, const ExpandArgs& p, int mb, hipStream_t s);
hipError_t launch_wgrad(const char* name, WgradArgs p, int sides, hipStream_t s);
hipError_t launch_transpose(const char* name, int n, const TransposeArgs& a, const TransposeArgs* b,
                            hipStream_t s);

}  // namespace moe
