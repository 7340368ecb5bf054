// Host-side argument checks shared by the C entries of the operators around the
// token mixer.
#pragma once
#include <exception>
#include <initializer_list>
#include <utility>

#include "host.hpp"
#include "layer.hpp"

namespace rewy {

// No exception leaves the C ABI.
template <typename F>
int guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    return fail(REWY_EHIP, "host error: %s", e.what());
  }
}

inline int64_t up64(int64_t v) { return (v + CH - 1) / CH * CH; }
inline size_t esize(int dtype) { return dtype == REWY_F32 ? 4 : 2; }

inline int check_dtype(const char* what, int v) {
  if (v != REWY_BF16 && v != REWY_F32) return fail(REWY_EINVAL, "bad %s %d", what, v);
  return REWY_OK;
}

// A given pointer has its elements' alignment.
inline int check_ptr(const char* name, const void* p, size_t align, bool need) {
  if (!p) return need ? fail(REWY_EINVAL, "%s is NULL", name) : (int)REWY_OK;
  if (!aligned(p, align)) return fail(REWY_EINVAL, "%s is not %zu-byte aligned", name, align);
  return REWY_OK;
}
#define REWY_TRY(expr)                \
  do {                                \
    const int rc_ = (expr);           \
    if (rc_ != REWY_OK) return rc_;   \
  } while (0)

inline int check_stride(const char* name, int64_t given, int64_t len, int64_t& out) {
  if (given != 0 && given < len)
    return fail(REWY_EINVAL, "%s %lld is shorter than the row's %lld elements", name, (long long)given, (long long)len);
  if (given > (int64_t)1 << 31) return fail(REWY_EINVAL, "%s %lld is too large", name, (long long)given);
  out = given ? given : len;
  return REWY_OK;
}

inline int check_workspace(const void* ws, size_t have, size_t need) {
  if (need && (!ws || !aligned(ws, ALIGN) || have < need))
    return fail(REWY_EWORKSPACE, "workspace needs %zu bytes, 256-byte aligned (got %zu)", need, have);
  return REWY_OK;
}

// ---- places ----------------------------------------------------------------------
// Bytes of a tensor: `rows` rows of `row` bytes, `stride` bytes from one to the next.
struct Place {
  const char* name;
  const void* p;
  int64_t rows, row, stride;
};
inline Place whole(const char* name, const void* p, int64_t bytes) { return {name, p, 1, bytes, bytes}; }

// Two tensors have a byte in common.  Rows may lie between each other's (slices of one
// longer row), so what counts is the rows and not the ranges from first to last byte.
inline bool meet(Place a, Place b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.row <= 0 || b.row <= 0) return false;
  for (Place* t : {&a, &b})
    if (t->rows == 1 || t->row == t->stride) *t = whole(t->name, t->p, (t->rows - 1) * t->stride + t->row);
  if (a.rows > b.rows) std::swap(a, b);
  const int64_t d = (int64_t)((uintptr_t)a.p - (uintptr_t)b.p), s = b.stride;  // a's first byte from b's
  if (d >= (b.rows - 1) * s + b.row || -d >= (a.rows - 1) * a.stride + a.row) return false;
  // first row of b that ends behind x
  auto first = [&](int64_t x) {
    const int64_t y = x - b.row, q = y / s - (y % s < 0);
    return q + 1;
  };
  if (a.rows > 1 && a.stride == s) {
    // row i of a meets row i + k of b for the same k everywhere
    for (int64_t k = first(d); k * s < d + a.row; ++k)
      if (std::max<int64_t>(0, -k) < std::min(a.rows, b.rows - k)) return true;
    return false;
  }
  for (int64_t i = 0; i < a.rows; ++i) {
    const int64_t x = d + i * a.stride, j = std::max<int64_t>(0, first(x));
    if (j < b.rows && j * s < x + a.row) return true;
  }
  return false;
}
// No output shares a byte with an input or another output.
inline int check_apart(std::initializer_list<Place> outs, std::initializer_list<Place> ins) {
  for (const Place* o = outs.begin(); o != outs.end(); ++o) {
    for (const Place& i : ins)
      if (meet(*o, i)) return fail(REWY_EINVAL, "%s overlaps %s", o->name, i.name);
    for (const Place* p = outs.begin(); p != o; ++p)
      if (meet(*o, *p)) return fail(REWY_EINVAL, "%s overlaps %s", o->name, p->name);
  }
  return REWY_OK;
}

// ---- sequences ------------------------------------------------------------------
inline int seq_args(int B, int T, int N, const int32_t* cu, const int32_t* host, SeqArgs& q) {
  if (B <= 0 || T < 0) return fail(REWY_EINVAL, "bad shape B=%d T=%d", B, T);
  const int64_t total = (int64_t)B * T;
  if (total > INT32_MAX - 65536) return fail(REWY_EINVAL, "B*T=%lld is too large", (long long)total);
  q.cu = cu; q.T = T; q.total = (int)total;
  if (cu) {
    if (B != 1) return fail(REWY_EINVAL, "cu_seqlens requires B == 1 (got B=%d)", B);
    if (N <= 0) return fail(REWY_EINVAL, "cu_seqlens requires N >= 1 (got N=%d)", N);
    if (!aligned(cu, 4)) return fail(REWY_EINVAL, "cu_seqlens is not 4-byte aligned");
    if (N > (1 << 24)) return fail(REWY_EINVAL, "N=%d is too large", N);
    if (host) {
      if (host[0] != 0 || host[N] > T) return fail(REWY_EINVAL, "cu_seqlens must start at 0 and end at T=%d at most", T);
      for (int i = 0; i < N; ++i)
        if (host[i + 1] < host[i]) return fail(REWY_EINVAL, "cu_seqlens not ascending at %d", i);
    }
    q.N = N;
  } else {
    if (N != 0 && N != B) return fail(REWY_EINVAL, "N=%d must equal B=%d without cu_seqlens", N, B);
    q.N = B;
  }
  return REWY_OK;
}

}  // namespace rewy
