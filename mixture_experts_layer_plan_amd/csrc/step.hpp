// Launch functions of the training step's operators around the layer: the norm in front
// of it (norm.hip), the balance loss (balance.hip) and the AdamW step (adamw.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// ------------------------------------------------------------------------- norm
struct NormArgs {
  const void *x, *res;  // [T, H]; res may be null
  const void *w, *b;    // [H] or null (1, 0)
  void *h, *y;          // [T, H]; h only with res
  float* stats;         // [T, 2]: mean, 1 / sqrt(variance + eps)
  int T, H;
  float eps;
};
struct NormBackArgs {
  const void *h, *w, *dy, *dh;  // w, dh may be null
  const float* stats;
  void *dx, *dw, *db;  // dw, db may be null
  float* parts;        // [groups][2][H]: sums of dw and db over each workgroup's rows
  int T, H;
  // set by the launch: workgroups of rows (those behind them take columns), and whether they
  // leave sums of dw and db
  int groups;
  bool sums;
};
constexpr int NORM_MAX_H = 16384;
int norm_groups(int T, int H);  // workgroups of the backward: from the sizes alone
// f32: fp32 elements, else bf16; centre: the mean is taken off
hipError_t launch_norm(const NormArgs& p, bool f32, bool centre, hipStream_t s);
hipError_t launch_norm_backward(const NormBackArgs& p, bool f32, bool centre, hipStream_t s);

// ---------------------------------------------------------------------- balance
// Segment c + i holds the sums of chunk c's tokens of sequence i: as a walk along the
// tokens never goes back in c or i, no two (c, i) that hold tokens share a sum c + i.
struct BalanceArgs {
  const float* logits;
  const int32_t* idx;
  const int32_t* start;  // [n_seq + 1] or null (one sequence of all tokens)
  int T, E, k, n_seq;
  bool sigmoid;
  float coef;
  float* loss;
  int32_t* counts;  // [n_seq, E]
  float* scales;    // [n_seq]
  // workspace
  float* seg_p;       // [n_chunks + n_seq, E]
  int32_t* seg_c;     // the same
  int32_t* seg_n;     // [n_chunks + n_seq]
  float* part;        // [n_seq, blocks]: sum of counts * p over a block's experts
  int32_t* tokens;    // [n_seq]
  int32_t* ticket;    // [1]
  // backward
  const float* d_loss;  // [1] or null (1)
  const float* d_in;    // [T, E] or null
  float* d_logits;
};
int balance_chunk(int T, int E);  // tokens of a chunk
int balance_blocks(int E);        // workgroups that add up one sequence
hipError_t launch_balance(const BalanceArgs& p, hipStream_t s);
hipError_t launch_balance_backward(const BalanceArgs& p, hipStream_t s);

// ------------------------------------------------------------------------ AdamW
// One tensor of the step's table.  In and out pointers may be the same.
struct AdamwDesc {
  const void *grad, *param, *m, *v;
  const float* master;
  const uint8_t *m_scale, *v_scale;
  void *param_out, *m_out, *v_out;
  float* master_out;
  uint8_t *m_scale_out, *v_scale_out;
  int64_t n;
  float weight_decay;
  int32_t pad;
};
constexpr int ADAMW_TILE = 2048;       // elements of a workgroup
constexpr int ADAMW_TABLE_CHUNK = 24;  // tensors that one launch writes into the table
struct AdamwChunk {
  AdamwDesc d[ADAMW_TABLE_CHUNK];
  int32_t first[ADAMW_TABLE_CHUNK];  // first tile of each
  int32_t base, count;
};
struct AdamwHyper {  // = moe_adamw_hyper
  float lr, beta1, one_minus_beta1, beta2, one_minus_beta2, eps, corr1, corr2, grad_scale;
  uint32_t seed;
};
struct AdamwArgs {
  const AdamwDesc* desc;
  const int32_t* first;  // [n_tensors]: first tile of each
  int n_tensors;
  int tiles;  // an upper bound
  AdamwHyper hyper;
  const AdamwHyper* hyper_dev;  // or null: hyper
};
hipError_t launch_adamw_table(const AdamwChunk& c, AdamwDesc* desc, int32_t* first, hipStream_t s);
// f32: fp32 parameters; g32: fp32 gradients; eight: states in 8 bits
hipError_t launch_adamw(const AdamwArgs& p, bool f32, bool g32, bool master, bool eight,
                        hipStream_t s);
hipError_t launch_adamw_values(bool v, int64_t n, const uint8_t* codes, const uint8_t* scales,
                               void* out, hipStream_t s);

}  // namespace moe
