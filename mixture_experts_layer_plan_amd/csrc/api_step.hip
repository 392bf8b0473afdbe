// C-ABI of the training step's operators around the layer (include/moe.h): argument
// checks and enqueues of the norm, the balance loss and the AdamW step.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>

#include "api_common.hpp"
#include "step.hpp"

using namespace moe;

namespace {

// ------------------------------------------------------------------------- norm
moe_status check_norm(const moe_norm_shape* s) {
  if (!s) return MOE_E_NULL;
  if (s->T < 0 || s->H < 8 || s->H % 8 || s->H > NORM_MAX_H) return MOE_E_SHAPE;
  if (s->kind != MOE_NORM_LAYER && s->kind != MOE_NORM_RMS) return MOE_E_SHAPE;
  // squares of a row below fp32's normal numbers are off by 2^-150: beside a smaller eps the
  // root would be too (values of 1e-21 with eps = 1e-42: by 1e-4, of 2^-75 with 2^-149: by 13 %)
  if (!(s->eps >= 0x1p-126f) || !(s->eps <= 1.0f)) return MOE_E_SHAPE;
  return MOE_OK;
}

size_t norm_ws_bytes(const moe_norm_shape* s) {
  return up((size_t)norm_groups(s->T, s->H) * 2 * s->H * sizeof(float));
}

moe_status norm_impl(bool f32, const moe_norm_shape* s, const void* x, const void* res,
                     const void* w, const void* b, void* h, void* y, float* stats,
                     hipStream_t st) {
  const moe_status rc = check_norm(s);
  if (rc != MOE_OK) return rc;
  if (s->T > 0 && any_null({x, y, stats})) return MOE_E_NULL;
  if (s->T > 0 && (res != nullptr) != (h != nullptr)) return MOE_E_NULL;
  if (!all_aligned({x, res, w, b, h, y, stats})) return MOE_E_ALIGN;
  const uint64_t row = (uint64_t)s->H * (f32 ? 4 : 2), n = s->T * row;
  // a workgroup reads a row before it writes it: the same pointer is fine
  if (overlap_base(y, x, n) || overlap_base(y, res, n) || overlap_base(h, x, n) ||
      overlap_base(h, res, n) || overlap(y, n, h, n))
    return MOE_E_UNSUPPORTED;
  // w and b are read, and rows of stats written, while other workgroups write theirs
  if (overlaps_any({y, n}, {{w, row}, {b, row}}) || overlaps_any({h, n}, {{w, row}, {b, row}}) ||
      overlaps_any({stats, (uint64_t)s->T * 8}, {{x, n}, {res, n}, {w, row}, {b, row}, {h, n}, {y, n}}))
    return MOE_E_UNSUPPORTED;
  if (s->T == 0) return MOE_OK;
  NormArgs a;
  a.x = x;
  a.res = res;
  a.w = w;
  a.b = b;
  a.h = h;
  a.y = y;
  a.stats = stats;
  a.T = s->T;
  a.H = s->H;
  a.eps = s->eps;
  return hip_status(launch_norm(a, f32, s->kind == MOE_NORM_LAYER, st));
}

moe_status norm_backward_impl(bool f32, const moe_norm_shape* s, const void* h, const void* w,
                              const float* stats, const void* dy, const void* dh_in, void* dx,
                              void* dw, void* db, void* ws, size_t ws_bytes, hipStream_t st) {
  const moe_status rc = check_norm(s);
  if (rc != MOE_OK) return rc;
  if (s->T > 0 && (any_null({h, stats, dy, dx}) || ((dw || db) && !ws))) return MOE_E_NULL;
  if (!all_aligned({h, w, stats, dy, dh_in, dx, dw, db, ws})) return MOE_E_ALIGN;
  if ((dw || db) && ws_bytes < norm_ws_bytes(s)) return MOE_E_WORKSPACE;
  const uint64_t row = (uint64_t)s->H * (f32 ? 4 : 2), n = s->T * row;
  const Span out = {dx, n}, read = {stats, (uint64_t)s->T * 8};
  if (overlap_base(dx, dy, n) || overlap_base(dx, dh_in, n) || overlap(dw, row, db, row) ||
      overlaps_any(out, {{h, n}, {w, row}, read}))
    return MOE_E_UNSUPPORTED;
  // dw, db and the sums in ws are written while rows are still read and written
  const Span sums = {dw || db ? ws : nullptr, norm_ws_bytes(s)};
  for (const Span& d : {Span{dw, row}, Span{db, row}, sums})
    if (overlaps_any(d, {{h, n}, {w, row}, read, {dy, n}, {dh_in, n}, out})) return MOE_E_UNSUPPORTED;
  if (overlaps_any(sums, {{dw, row}, {db, row}})) return MOE_E_UNSUPPORTED;
  NormBackArgs a;
  a.h = h;
  a.w = w;
  a.dy = dy;
  a.dh = dh_in;
  a.stats = stats;
  a.dx = dx;
  a.dw = dw;
  a.db = db;
  a.parts = (float*)ws;
  a.T = s->T;
  a.H = s->H;
  return hip_status(launch_norm_backward(a, f32, s->kind == MOE_NORM_LAYER, st));
}

// ---------------------------------------------------------------------- balance
constexpr int MAX_BALANCED = (1 << 26) - 4, MAX_SEQUENCES = 1 << 20;

moe_status check_balance(const moe_shape* s, const moe_balance* b) {
  if (!s || !b) return MOE_E_NULL;
  // the loss has no use for the other sizes and flags
  moe_shape own = *s;
  own.H = own.I = 128;
  own.flags = 0;
  const moe_status rc = check_shape(&own, false);
  if (rc != MOE_OK) return rc;
  if (b->score != MOE_SCORE_SOFTMAX && b->score != MOE_SCORE_SIGMOID) return MOE_E_SHAPE;
  if (b->n_seq < 1 || b->n_seq > MAX_SEQUENCES) return MOE_E_SHAPE;
  if (!(b->coef - b->coef == 0.0f)) return MOE_E_SHAPE;
  // a wavefront a token in the backward, four a workgroup: below 2^32 threads
  return s->T <= MAX_BALANCED ? MOE_OK : MOE_E_UNSUPPORTED;
}

// the chunks' sums by segment, the sequences' sums, and the count of finished workgroups
struct BalanceWs {
  size_t seg_p, seg_c, seg_n, part, tokens, ticket, total;
};
BalanceWs balance_ws(const moe_shape* s, const moe_balance* b) {
  const int chunk = balance_chunk(s->T, s->E);
  const size_t segs = ((size_t)s->T + chunk - 1) / chunk + b->n_seq;
  Carve c;
  BalanceWs L;
  L.seg_p = c.take(segs * s->E * sizeof(float));
  L.seg_c = c.take(segs * s->E * sizeof(int32_t));
  L.seg_n = c.take(segs * sizeof(int32_t));
  L.part = c.take((size_t)b->n_seq * balance_blocks(s->E) * sizeof(float));
  L.tokens = c.take((size_t)b->n_seq * sizeof(int32_t));
  L.ticket = c.take(sizeof(int32_t));
  L.total = c.off;
  return L;
}

BalanceArgs balance_args(const moe_shape* s, const moe_balance* b, const float* logits,
                         const int32_t* idx, const int32_t* start) {
  BalanceArgs a;
  memset(&a, 0, sizeof(a));
  a.logits = logits;
  a.idx = idx;
  a.start = start;
  a.T = s->T;
  a.E = s->E;
  a.k = s->k;
  a.n_seq = b->n_seq;
  a.sigmoid = b->score == MOE_SCORE_SIGMOID;
  a.coef = b->coef;
  return a;
}

// ------------------------------------------------------------------------ AdamW
static_assert(sizeof(AdamwHyper) == sizeof(moe_adamw_hyper), "one layout");

int64_t adamw_tiles(int64_t n) { return (n + ADAMW_TILE - 1) / ADAMW_TILE; }

moe_status check_adamw(const moe_adamw_shape* s) {
  if (!s) return MOE_E_NULL;
  if (s->elements < 0 || s->n_tensors < 1 || s->n_tensors > MOE_ADAMW_MAX_TENSORS) return MOE_E_SHAPE;
  for (const int32_t t : {s->p_type, s->g_type})
    if (t != MOE_F32 && t != MOE_BF16) return MOE_E_SHAPE;
  if (s->master != 0 && s->master != 1) return MOE_E_SHAPE;
  if (s->master && s->p_type != MOE_BF16) return MOE_E_SHAPE;
  if (s->state_bits != 32 && s->state_bits != 8) return MOE_E_SHAPE;
  // a workgroup of 256 threads a tile: below 2^32 threads
  if (s->elements / ADAMW_TILE + s->n_tensors >= (int64_t)1 << 24) return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

struct AdamwTable {
  size_t desc, first, total;
};
AdamwTable adamw_table(const moe_adamw_shape* s) {
  Carve c;
  AdamwTable L;
  L.desc = c.take((size_t)s->n_tensors * sizeof(AdamwDesc));
  L.first = c.take((size_t)s->n_tensors * sizeof(int32_t));
  L.total = c.off;
  return L;
}

// The byte ranges of one tensor: inputs that the step does not write, and outputs.
struct Range {
  uintptr_t begin, end;
  bool out;
};
struct Pair {
  const void* in;
  void* out;
  uint64_t bytes;
};
int pairs_of(const moe_adamw_shape* s, const moe_adamw_tensor& t, Pair* p) {
  const uint64_t n = (uint64_t)t.n, ps = s->p_type == MOE_F32 ? 4 : 2;
  const uint64_t ss = s->state_bits == 32 ? 4 : 1, blocks = (n + 31) / 32;
  int k = 0;
  p[k++] = {s->master ? nullptr : t.param, t.param_out, n * ps};  // with a master only written
  p[k++] = {t.m, t.m_out, n * ss};
  p[k++] = {t.v, t.v_out, n * ss};
  if (s->master) p[k++] = {t.master, t.master_out, n * 4};
  if (s->state_bits == 8) {
    p[k++] = {t.m_scale, t.m_scale_out, blocks};
    p[k++] = {t.v_scale, t.v_scale_out, blocks};
  }
  return k;
}

// Outputs may be their own inputs; otherwise no output shares bytes with an input or
// with another output, of whatever tensor, nor does the table, which every step reads.
moe_status check_ranges(const moe_adamw_shape* s, const moe_adamw_tensor* t, const void* table) {
  const size_t most = (size_t)s->n_tensors * 13 + 1;
  Range* r = new (std::nothrow) Range[most];
  if (!r) return MOE_E_WORKSPACE;
  size_t k = 0;
  const auto add = [&](const void* p, uint64_t bytes, bool out) {
    if (bytes) r[k++] = {(uintptr_t)p, (uintptr_t)p + bytes, out};
  };
  add(table, adamw_table(s).total, true);
  for (int i = 0; i < s->n_tensors; ++i) {
    Pair p[6];
    const int np = pairs_of(s, t[i], p);
    add(t[i].grad, (uint64_t)t[i].n * (s->g_type == MOE_F32 ? 4 : 2), false);
    for (int j = 0; j < np; ++j) {
      if (p[j].in && p[j].in != p[j].out) add(p[j].in, p[j].bytes, false);
      add(p[j].out, p[j].bytes, true);
    }
  }
  std::sort(r, r + k, [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uintptr_t any = 0, out = 0;
  bool clash = false;
  for (size_t i = 0; i < k && !clash; ++i) {
    clash = r[i].begin < (r[i].out ? any : out);
    any = std::max(any, r[i].end);
    if (r[i].out) out = std::max(out, r[i].end);
  }
  delete[] r;
  return clash ? MOE_E_UNSUPPORTED : MOE_OK;
}

moe_status check_tensors(const moe_adamw_shape* s, const moe_adamw_tensor* t, const void* table) {
  int64_t sum = 0;
  for (int i = 0; i < s->n_tensors; ++i) {
    if (t[i].n < 0 || t[i].n > s->elements) return MOE_E_SHAPE;
    if (!(t[i].weight_decay - t[i].weight_decay == 0.0f)) return MOE_E_SHAPE;
    sum += t[i].n;  // at most 65536 terms of at most 2^37
    if (t[i].n == 0) continue;
    Pair p[6];
    const int np = pairs_of(s, t[i], p);
    if (!t[i].grad) return MOE_E_NULL;
    if (!aligned16(t[i].grad)) return MOE_E_ALIGN;
    for (int j = 0; j < np; ++j) {
      const bool no_input = s->master && j == 0;
      if (!p[j].out || (!p[j].in && !no_input)) return MOE_E_NULL;
      if (!aligned16(p[j].out) || !aligned16(p[j].in)) return MOE_E_ALIGN;
    }
  }
  return sum == s->elements ? check_ranges(s, t, table) : MOE_E_SHAPE;
}

}  // namespace

extern "C" {

size_t moe_norm_workspace_bytes(const moe_norm_shape* s) {
  return check_norm(s) == MOE_OK ? norm_ws_bytes(s) : 0;
}

moe_status moe_norm_bf16(const moe_norm_shape* s, const void* x, const void* residual,
                         const void* w, const void* b, void* h, void* y, float* stats,
                         hipStream_t st) {
  return norm_impl(false, s, x, residual, w, b, h, y, stats, st);
}
moe_status moe_norm_f32(const moe_norm_shape* s, const float* x, const float* residual,
                        const float* w, const float* b, float* h, float* y, float* stats,
                        hipStream_t st) {
  return norm_impl(true, s, x, residual, w, b, h, y, stats, st);
}
moe_status moe_norm_backward_bf16(const moe_norm_shape* s, const void* h, const void* w,
                                  const float* stats, const void* dy, const void* dh_in, void* dx,
                                  void* dw, void* db, void* ws, size_t ws_bytes, hipStream_t st) {
  return norm_backward_impl(false, s, h, w, stats, dy, dh_in, dx, dw, db, ws, ws_bytes, st);
}
moe_status moe_norm_backward_f32(const moe_norm_shape* s, const float* h, const float* w,
                                 const float* stats, const float* dy, const float* dh_in,
                                 float* dx, float* dw, float* db, void* ws, size_t ws_bytes,
                                 hipStream_t st) {
  return norm_backward_impl(true, s, h, w, stats, dy, dh_in, dx, dw, db, ws, ws_bytes, st);
}

size_t moe_balance_workspace_bytes(const moe_shape* s, const moe_balance* b) {
  return check_balance(s, b) == MOE_OK ? balance_ws(s, b).total : 0;
}

moe_status moe_balance_loss(const moe_shape* s, const moe_balance* b, const float* logits,
                            const int32_t* topk_idx, const int32_t* seq_start, float* loss,
                            int32_t* counts, float* scales, void* ws, size_t ws_bytes,
                            hipStream_t st) {
  const moe_status rc = check_balance(s, b);
  if (rc != MOE_OK) return rc;
  if (any_null({loss, counts, scales, ws}) || any_null_rows(s, {logits, topk_idx})) return MOE_E_NULL;
  if (b->n_seq > 1 && !seq_start) return MOE_E_NULL;
  if (!all_aligned({logits, topk_idx, seq_start, loss, counts, scales, ws})) return MOE_E_ALIGN;
  const BalanceWs W = balance_ws(s, b);
  if (ws_bytes < W.total) return MOE_E_WORKSPACE;
  // all of them are written while others of the call are still read
  const uint64_t T = s->T, n = b->n_seq;
  const Span in[3] = {{logits, T * s->E * 4}, {topk_idx, T * s->k * 4}, {seq_start, (n + 1) * 4}};
  const Span out[4] = {{loss, 4}, {counts, n * s->E * 4}, {scales, n * 4}, {ws, W.total}};
  for (int i = 0; i < 4; ++i) {
    if (overlaps_any(out[i], {in[0], in[1], in[2]})) return MOE_E_UNSUPPORTED;
    for (int j = 0; j < i; ++j)
      if (overlaps_any(out[i], {out[j]})) return MOE_E_UNSUPPORTED;
  }
  BalanceArgs a = balance_args(s, b, logits, topk_idx, seq_start);
  a.loss = loss;
  a.counts = counts;
  a.scales = scales;
  a.seg_p = at<float>(ws, W.seg_p);
  a.seg_c = at<int32_t>(ws, W.seg_c);
  a.seg_n = at<int32_t>(ws, W.seg_n);
  a.part = at<float>(ws, W.part);
  a.tokens = at<int32_t>(ws, W.tokens);
  a.ticket = at<int32_t>(ws, W.ticket);
  return hip_status(launch_balance(a, st));
}

moe_status moe_balance_loss_backward(const moe_shape* s, const moe_balance* b, const float* logits,
                                     const int32_t* topk_idx, const int32_t* seq_start,
                                     const int32_t* counts, const float* scales,
                                     const float* d_loss, const float* d_in, float* d_logits,
                                     hipStream_t st) {
  const moe_status rc = check_balance(s, b);
  if (rc != MOE_OK) return rc;
  if (any_null({counts, scales}) || any_null_rows(s, {logits, topk_idx, d_logits})) return MOE_E_NULL;
  if (b->n_seq > 1 && !seq_start) return MOE_E_NULL;
  if (!all_aligned({logits, topk_idx, seq_start, counts, scales, d_loss, d_in, d_logits}))
    return MOE_E_ALIGN;
  const uint64_t T = s->T, seqs = b->n_seq, n = T * s->E * 4;
  if (overlap_base(d_logits, logits, n) || overlap_base(d_logits, d_in, n)) return MOE_E_UNSUPPORTED;
  // read by every workgroup, at any time
  if (overlaps_any({d_logits, n}, {{topk_idx, T * s->k * 4}, {seq_start, (seqs + 1) * 4},
                                   {counts, seqs * s->E * 4}, {scales, seqs * 4}, {d_loss, 4}}))
    return MOE_E_UNSUPPORTED;
  BalanceArgs a = balance_args(s, b, logits, topk_idx, seq_start);
  a.counts = const_cast<int32_t*>(counts);
  a.scales = const_cast<float*>(scales);
  a.d_loss = d_loss;
  a.d_in = d_in;
  a.d_logits = d_logits;
  return hip_status(launch_balance_backward(a, st));
}

size_t moe_adamw_table_bytes(const moe_adamw_shape* s) {
  return check_adamw(s) == MOE_OK ? adamw_table(s).total : 0;
}

moe_status moe_adamw_table(const moe_adamw_shape* s, const moe_adamw_tensor* tensors, void* table,
                           hipStream_t st) {
  moe_status rc = check_adamw(s);
  if (rc != MOE_OK) return rc;
  if (any_null({tensors, table})) return MOE_E_NULL;
  if (!aligned16(table)) return MOE_E_ALIGN;
  rc = check_tensors(s, tensors, table);
  if (rc != MOE_OK) return rc;
  const AdamwTable L = adamw_table(s);
  int32_t tiles = 0;
  for (int base = 0; base < s->n_tensors; base += ADAMW_TABLE_CHUNK) {
    AdamwChunk c;
    memset(&c, 0, sizeof(c));
    c.base = base;
    c.count = std::min(ADAMW_TABLE_CHUNK, s->n_tensors - base);
    for (int i = 0; i < c.count; ++i) {
      const moe_adamw_tensor& t = tensors[base + i];
      c.d[i] = {t.grad, t.param, t.m, t.v, t.master, t.m_scale, t.v_scale, t.param_out, t.m_out,
                t.v_out, t.master_out, t.m_scale_out, t.v_scale_out, t.n, t.weight_decay, 0};
      c.first[i] = tiles;
      tiles += (int32_t)adamw_tiles(t.n);
    }
    MOE_TRY(launch_adamw_table(c, at<AdamwDesc>(table, L.desc), at<int32_t>(table, L.first), st));
  }
  return MOE_OK;
}

moe_status moe_adamw_hyper_of(double lr, double beta1, double beta2, double eps, int64_t step,
                              double grad_scale, uint32_t seed, moe_adamw_hyper* out) {
  if (!out) return MOE_E_NULL;
  const float lr32 = (float)lr, scale32 = (float)grad_scale;  // (1e39 is finite in double alone)
  if (!(lr32 - lr32 == 0.0f) || !(scale32 - scale32 == 0.0f) || step < 1) return MOE_E_SHAPE;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) return MOE_E_SHAPE;
  if (!(eps >= 1e-30 && eps <= 1.0)) return MOE_E_SHAPE;
  out->lr = lr32;
  out->beta1 = (float)beta1;
  out->one_minus_beta1 = (float)(1.0 - beta1);
  out->beta2 = (float)beta2;
  out->one_minus_beta2 = (float)(1.0 - beta2);
  out->eps = (float)eps;
  out->corr1 = (float)(1.0 / (1.0 - pow(beta1, (double)step)));
  out->corr2 = (float)(1.0 / (1.0 - pow(beta2, (double)step)));
  out->grad_scale = scale32;
  out->seed = seed;
  return MOE_OK;
}

moe_status moe_adamw_step(const moe_adamw_shape* s, const void* table, const moe_adamw_hyper* hyper,
                          const moe_adamw_hyper* hyper_dev, hipStream_t st) {
  const moe_status rc = check_adamw(s);
  if (rc != MOE_OK) return rc;
  if (!table || (hyper != nullptr) == (hyper_dev != nullptr)) return MOE_E_NULL;
  if (!all_aligned({table, hyper_dev})) return MOE_E_ALIGN;
  const AdamwTable L = adamw_table(s);
  AdamwArgs a;
  memset(&a, 0, sizeof(a));
  a.desc = at<AdamwDesc>(table, L.desc);
  a.first = at<int32_t>(table, L.first);
  a.n_tensors = s->n_tensors;
  a.tiles = s->elements ? (int)(s->elements / ADAMW_TILE + s->n_tensors) : 0;
  if (hyper) memcpy(&a.hyper, hyper, sizeof(a.hyper));
  a.hyper_dev = (const AdamwHyper*)hyper_dev;
  return hip_status(launch_adamw(a, s->p_type == MOE_F32, s->g_type == MOE_F32, s->master != 0,
                                 s->state_bits == 8, st));
}

moe_status moe_adamw_values(int32_t which, int64_t n, const uint8_t* codes, const uint8_t* scales,
                            void* out, hipStream_t st) {
  if (which != MOE_ADAMW_M && which != MOE_ADAMW_V) return MOE_E_SHAPE;
  if (n < 0) return MOE_E_SHAPE;
  if (n > 0 && any_null({codes, scales, out})) return MOE_E_NULL;
  if (!all_aligned({codes, scales, out})) return MOE_E_ALIGN;
  const uint64_t un = (uint64_t)n;
  if (overlap(out, 2 * un, codes, un) || overlap(out, 2 * un, scales, (un + 31) / 32))
    return MOE_E_UNSUPPORTED;
  return hip_status(launch_adamw_values(which == MOE_ADAMW_V, n, codes, scales, out, st));
}

}  // extern "C"
