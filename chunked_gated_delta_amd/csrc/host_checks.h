// Checks of arguments that the C entries over strided views share (all before any HIP call): alignment, reach,
// overlap, and the error code of a launch.
#pragma once

#include <initializer_list>
#include <utility>

#include "gdr_internal.h"

namespace kda {

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// the bytes a tensor reaches, [lo, hi); empty for null or no elements
struct Span {
  uintptr_t lo = 0, hi = 0;
};

inline Span dense(const void* p, double bytes) {
  if (!p || bytes <= 0) return Span{};
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Span{lo, lo + (uintptr_t)bytes};
}

constexpr int64_t kMaxExtent = (int64_t)1 << 46;        // bytes
constexpr int64_t kMaxTokenStride = (int64_t)1 << 25;   // bytes: the 64 rows of a chunk within 32 bits

constexpr int64_t kMaxStride = 4 * kMaxExtent;          // bytes: no limit of its own

// the span of a [B, H, T, D] view, D contiguous (strides already checked)
inline Span view(const void* p, kda_stride_t s, int64_t B, int64_t H, int64_t T, int64_t D, int64_t esz) {
  if (!p || B < 1 || H < 1 || T < 1) return Span{};
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Span{lo, lo + (uintptr_t)(((B - 1) * s.b + (H - 1) * s.h + (T - 1) * s.t + D) * esz)};
}

inline bool meet(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

// strides of an input: not negative, in reach, each row `align` bytes apart from an aligned place, tokens at most
// `most` bytes apart (the rule's kernels; the norms address every row in 64 bits)
inline int check_strides(const void* p, kda_stride_t s, int64_t B, int64_t H, int64_t T, int64_t D, int64_t esz, int64_t align,
                  int64_t most = kMaxTokenStride) {
  if (!p) return KDA_OK;
  if (!aligned(p, (unsigned)align)) return KDA_ERR_ARG;
  const int64_t st[3] = {s.b, s.h, s.t}, n[3] = {B, H, T};
  double reach = (double)D;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;      // never stepped by
    if (st[i] < 0 || st[i] > kMaxExtent || (st[i] * esz) % align != 0) return KDA_ERR_ARG;
    reach += (double)(n[i] - 1) * (double)st[i];
  }
  if (T > 1 && s.t * esz > most) return KDA_ERR_ARG;
  return reach * esz > (double)kMaxExtent ? KDA_ERR_SHAPE : KDA_OK;
}

// an output also may not hold one place twice: by stride, each step passes everything below it
inline int check_out(const void* p, kda_stride_t s, int64_t B, int64_t H, int64_t T, int64_t D, int64_t esz, int64_t align,
              int64_t most = kMaxTokenStride) {
  if (!p) return KDA_OK;
  const int rc = check_strides(p, s, B, H, T, D, esz, align, most);
  if (rc != KDA_OK) return rc;
  int64_t st[3] = {s.b, s.h, s.t}, n[3] = {B, H, T};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[j] < st[i]) {
        std::swap(st[i], st[j]);
        std::swap(n[i], n[j]);
      }
  int64_t reach = D;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (st[i] < reach) return KDA_ERR_ARG;
    reach += (n[i] - 1) * st[i];
  }
  return KDA_OK;
}

// no output meets an input or another output
inline int check_apart(std::initializer_list<Span> ins, std::initializer_list<Span> outs) {
  for (const Span* a = outs.begin(); a != outs.end(); ++a) {
    for (const Span& b : ins)
      if (meet(*a, b)) return KDA_ERR_ARG;
    for (const Span* b = a + 1; b != outs.end(); ++b)
      if (meet(*a, *b)) return KDA_ERR_ARG;
  }
  return KDA_OK;
}

inline bool head_dim(int64_t d) { return d == 32 || d == 64 || d == 128; }
inline int64_t elem(int32_t dtype) { return dtype == KDA_DTYPE_BF16 ? 2 : 4; }
inline int done(hipError_t e) { return e == hipSuccess ? KDA_OK : record_hip_error(e); }

}  // namespace kda
