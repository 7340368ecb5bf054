// Host-side argument checks shared by the C entries of the operators around the
// token mixer.
#pragma once
#include <exception>

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
