// Argument checks, buffer layouts and small helpers shared by the C-ABI's sources.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/moe.h"
#include "internal.hpp"

namespace moe {

constexpr size_t ALIGN = 256;

inline size_t up(size_t v) { return (v + ALIGN - 1) / ALIGN * ALIGN; }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Carves consecutive 256-byte-aligned regions out of one buffer.
struct Carve {
  size_t off = 0;
  size_t take(size_t bytes) {
    const size_t o = off;
    off += up(bytes);
    return o;
  }
};

inline moe_status check_shape(const moe_shape* s, bool need_gemm_dims) {
  if (!s) return MOE_E_NULL;
  if (s->T < 0 || s->E < 1 || s->E > MOE_MAX_E || s->k < 1 || s->k > s->E || s->k > MOE_MAX_K)
    return MOE_E_SHAPE;
  if ((int64_t)s->T * s->k >= (int64_t)1 << 31) return MOE_E_SHAPE;
  if (s->H < 128 || s->H % 128) return MOE_E_SHAPE;
  if (s->flags & ~(MOE_REPLAY | MOE_FUSED_FORWARD)) return MOE_E_SHAPE;
  if (need_gemm_dims) {
    if (s->I < 128 || s->I % 128) return MOE_E_SHAPE;
    if (s->I_shared < 0 || s->I_shared % 128) return MOE_E_SHAPE;
    if (s->T_minibatch < 0) return MOE_E_SHAPE;
  }
  return MOE_OK;
}

template <typename P>
P* at(void* base, size_t off) {
  return (P*)((char*)base + off);
}
template <typename P>
const P* at(const void* base, size_t off) {
  return (const P*)((const char*)base + off);
}

inline moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_E_HIP; }

#define MOE_TRY(expr)                         \
  do {                                        \
    const hipError_t e_ = (expr);             \
    if (e_ != hipSuccess) return MOE_E_HIP;   \
  } while (0)

inline bool all_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p && !aligned16(p)) return false;
  return true;
}

inline bool any_null(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p) return true;
  return false;
}

// Arrays whose size is a multiple of T may be NULL when T == 0.
inline bool any_null_rows(const moe_shape* s, std::initializer_list<const void*> ps) {
  return s->T > 0 && any_null(ps);
}

// Whether an output shares bytes with an input that is still read while it is written (an
// output over its own base is read and written row by row: the same pointer is fine).
inline bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t p = (uintptr_t)a, q = (uintptr_t)b;
  return a && b && na && nb && p < q + nb && q < p + na;
}
inline bool overlap_base(const void* y, const void* base, uint64_t n) {
  return y != base && overlap(y, n, base, n);
}
// A buffer of a call, and whether it shares bytes with one of `others`.
struct Span {
  const void* p;
  uint64_t n;
};
inline bool overlaps_any(Span a, std::initializer_list<Span> others) {
  for (const Span& o : others)
    if (overlap(a.p, a.n, o.p, o.n)) return true;
  return false;
}

}  // namespace moe
