// abi_rows.h -- what the C entry points with strided [N,H,T,d] tensors check their arguments
// with: element sizes, strides, spans of memory and whether two tensors share an element.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <utility>

#include "lizard_internal.h"

namespace lz {
namespace abi {

inline size_t elem_size(lizard_dtype t) { return t == LIZARD_F32 ? 4 : 2; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool ptr_ok(const void* p, bool optional) { return p ? aligned16(p) : optional; }
inline bool dtype_ok(lizard_dtype t) { return t == LIZARD_F32 || t == LIZARD_BF16; }
constexpr int64_t kMaxExtent = 1ll << 46;  // elements a strided tensor may span

// A strided [N,H,T,d] tensor: its strides and the bytes from its first to past its last
// element.
struct Rows {
  Strides s{};
  size_t bytes = 0;
  bool ok = false;
};

inline Rows rows_of(const lizard_strides* s, int64_t N, int64_t H, int64_t T, int64_t d, lizard_dtype dt,
             bool output) {
  Rows r;
  if (!s) {
    r.s = {H * T * d, T * d, d};
  } else {
    r.s = {s->n, s->h, s->t};
    const int64_t dim[3] = {N, H, T}, st[3] = {s->n, s->h, s->t};
    const int64_t unit = 16 / (int64_t)elem_size(dt);
    for (int i = 0; i < 3; ++i) {
      if (dim[i] <= 1) continue;  // never stepped over
      if (st[i] < 0 || st[i] % unit || st[i] > kMaxExtent) return r;
      if (output && st[i] < d) return r;
    }
    if (output) {
      // distinct elements: sorted by stride, each axis steps past all of the smaller ones
      std::pair<int64_t, int64_t> axes[3];
      int k = 0;
      for (int i = 0; i < 3; ++i)
        if (dim[i] > 1) axes[k++] = {st[i], dim[i]};
      std::sort(axes, axes + k);
      int64_t span = d;
      for (int i = 0; i < k; ++i) {
        if (axes[i].first < span || axes[i].second > kMaxExtent / axes[i].first) return r;
        span += axes[i].first * (axes[i].second - 1);
      }
    }
  }
  const __int128 span = (__int128)(N > 1 ? (N - 1) * (__int128)r.s.n : 0) +
                        (H > 1 ? (H - 1) * (__int128)r.s.h : 0) +
                        (T > 1 ? (T - 1) * (__int128)r.s.t : 0) + d;
  if (span > kMaxExtent) return r;
  r.bytes = N && H && T ? (size_t)span * elem_size(dt) : 0;
  r.ok = true;
  return r;
}

struct Span {
  const void* p;
  size_t n;
};
inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}
inline bool any_overlap(const Span* outs, int no, const Span* ins, int ni) {
  for (int i = 0; i < no; ++i) {
    for (int j = 0; j < ni; ++j)
      if (overlap(outs[i], ins[j])) return true;
    for (int j = i + 1; j < no; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

// Two strided tensors share no element: their spans are apart, or, counted modulo the stride of
// some axis of either, what each covers lies beside the other (slices of one packed projection:
// of its heads, whichever axis is outermost).
struct Tensor {
  const void* p;
  const Rows* r;
  int64_t N, H, T, d, es;
};
inline bool apart(const Tensor& a, const Tensor& b) {
  if (!overlap(Span{a.p, a.r->bytes}, Span{b.p, b.r->bytes})) return true;
  const int64_t off = static_cast<const char*>(b.p) - static_cast<const char*>(a.p);
  for (const Tensor* x : {&a, &b}) {
    const int64_t dim[3] = {x->N, x->H, x->T}, stride[3] = {x->r->s.n, x->r->s.h, x->r->s.t};
    for (int i = 0; i < 3; ++i) {
      if (dim[i] <= 1 || stride[i] <= 0) continue;
      // bytes from the first element on, steps of a multiple of the stride left out
      auto width = [&](const Tensor& t) {
        const int64_t td[3] = {t.N, t.H, t.T}, ts[3] = {t.r->s.n, t.r->s.h, t.r->s.t};
        int64_t w = t.d;
        for (int k = 0; k < 3; ++k)
          if (td[k] > 1 && ts[k] % stride[i]) w += (td[k] - 1) * ts[k];
        return w * t.es;
      };
      const int64_t step = stride[i] * a.es, at = (off % step + step) % step;
      if (width(a) <= at && at + width(b) <= step) return true;
    }
  }
  return false;
}

inline bool same(const Strides& a, const Strides& b) { return a.n == b.n && a.h == b.h && a.t == b.t; }

inline lizard_status finish(cudaError_t e, int launches) {
  set_last_launches(launches);
  return e == cudaSuccess ? LIZARD_OK : LIZARD_ERR_CUDA;
}

}  // namespace abi
}  // namespace lz
