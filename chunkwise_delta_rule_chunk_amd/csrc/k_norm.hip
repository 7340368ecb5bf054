// RMS norm of s = x + res, with the sum written back for the residual stream
// and an 8-bit output with scales:
//   rstd = (mean_j s_j^2 + eps)^-1/2,  y_j = s_j rstd w_j,
//   scale_g = max_{j in g} |y_j| / qmax,  q_j = round(y_j / scale_g),
// qmax = 448 (e4m3) or 127 (int8), one scale per row or per group of columns.
// Everything is formed from the unrounded fp32 sum; y, sum and q are each
// rounded once, to nearest even.  Backward, with s the sum as it was stored
// and u = dy w:
//   dx = rstd (u - s rstd^2 mean(u s)) + ds,   dw_j = sum_rows dy_j s_j rstd.
//
// Memory is all it costs: each input is read once and each output written
// once.  A row is held by TPR threads in registers (NC vectors of 16 bytes a
// thread), so nothing is read twice and sum may overwrite x or res.  (A square over
// 3e38 makes the sum of squares infinite and the row zero, as in any fp32 norm.)
#include "row.hpp"

namespace rewy {

namespace {

// One row a group of TPR threads: all loads first, one join for the mean, one for the
// scale (a group of columns lies in neighbouring lanes: no LDS).  Bound by HBM:
// 8192 x 4096 bf16 with the sum, e4m3 in groups of 128: 304 MB in 55 us (5.5 TB/s);
// without the 8-bit output but with y 49 us (5.5 TB/s); 10007 x 1537 fp32 to int8 33
// us; 16 rows of 4096: 6 us, a launch and two trips to memory.
template <typename T, typename W, int TPR, int NC>
__global__ __launch_bounds__(TPR > NORM_BLOCK ? TPR : NORM_BLOCK) void k_norm_fwd(NormArgs a) {
  constexpr int VE = Vec<T>::VE, BLOCK = TPR > NORM_BLOCK ? TPR : NORM_BLOCK, RPB = BLOCK / TPR;
  __shared__ float sbuf[BLOCK / 64];
  __shared__ uint32_t mbuf[BLOCK / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = (blockIdx.y * (int64_t)gridDim.x + blockIdx.x) * RPB + threadIdx.x / TPR;
  const bool on = row < a.M;
  const int D = on ? a.D : 0;  // threads past the last row hold nothing and write nothing
  const int64_t m = on ? row : 0;
  const T* x = reinterpret_cast<const T*>(a.x) + m * a.xs;
  const T* r = a.res ? reinterpret_cast<const T*>(a.res) + m * a.rs : nullptr;
  const W* w = reinterpret_cast<const W*>(a.w);

  float s[NC][VE], ssq = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int j = (c * TPR + t) * VE;
    ldv<T, VE>(s[c], x + j, D - j);
  }
  if (r) {
    float rv[NC][VE];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int j = (c * TPR + t) * VE;
      ldv<T, VE>(rv[c], r + j, D - j);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < VE; ++e) s[c][e] += rv[c][e];
  }
  if (a.sum) {
    T* o = reinterpret_cast<T*>(a.sum) + m * a.ss;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int j = (c * TPR + t) * VE;
      stv<T, VE>(o + j, s[c], D - j);
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < VE; ++e) ssq += s[c][e] * s[c][e];
  const float rstd = 1.f / sqrtf(row_sum<TPR>(ssq, sbuf) / (float)a.D + a.eps);
  if (a.rstd && on && t == 0) a.rstd[row] = rstd;

#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int j = (c * TPR + t) * VE;
    float wv[VE];
    if (w) ldv<W, VE>(wv, w + j, D - j);
#pragma unroll
    for (int e = 0; e < VE; ++e) s[c][e] = s[c][e] * rstd * (w ? wv[e] : 1.f);
  }
  if (a.y) {
    T* o = reinterpret_cast<T*>(a.y) + m * a.ys;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int j = (c * TPR + t) * VE;
      stv<T, VE>(o + j, s[c], D - j);
    }
  }
  if (!a.quant) return;
  const float qmax = a.quant == REWY_QUANT_E4M3 ? 448.f : 127.f;
  uint32_t mx[NC], all = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    mx[c] = 0;
#pragma unroll
    for (int e = 0; e < VE; ++e) mx[c] = max(mx[c], mag(s[c][e]));
    all = max(all, mx[c]);
  }
  if (!a.group) all = row_max<TPR>(all, mbuf);
  const int lanes = a.group ? min(a.group / VE, TPR) : 0;  // lanes that share a scale
  uint8_t* q = reinterpret_cast<uint8_t*>(a.q) + m * a.D;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int j = (c * TPR + t) * VE;
    const float scale = make_scale(a.group ? lanes_max_n(mx[c], lanes) : all, qmax);
    if (a.group) {
      if (j < D && j % a.group == 0) a.scale[m * a.ng + j / a.group] = scale;
    } else if (c == 0 && t == 0 && on) {
      a.scale[m] = scale;
    }
    store_codes<VE>(q + j, s[c], scale, a.quant == REWY_QUANT_E4M3, D - j);
  }
}

// Each block takes rows blockIdx, + gridDim, ... and keeps dw of its columns in
// registers; one partial row per block goes to the workspace (no atomics: the
// same sums every time).  Bound by HBM: 8192 x 4096 bf16 with the sum's adjoint, 286 MB
// with the partial rows in 56.4 us (5.1 TB/s).
template <typename T, typename W, int TPR, int NC>
__global__ __launch_bounds__(TPR > NORM_BLOCK ? TPR : NORM_BLOCK) void k_norm_bwd(NormArgs a) {
  constexpr int VE = Vec<T>::VE, BLOCK = TPR > NORM_BLOCK ? TPR : NORM_BLOCK, RPB = BLOCK / TPR;
  __shared__ float sbuf[2][BLOCK / 64];
  __shared__ float wbuf[RPB > 1 ? BLOCK * NC * VE : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR, D = a.D;
  const W* w = reinterpret_cast<const W*>(a.w);
  float wv[NC][VE], dw[NC][VE];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int j = (c * TPR + t) * VE;
    if (w) ldv<W, VE>(wv[c], w + j, D - j);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      if (!w) wv[c][e] = 1.f;
      dw[c][e] = 0.f;
    }
  }
  int flip = 0;
  for (int64_t r0 = blockIdx.x * (int64_t)RPB; r0 < a.M; r0 += (int64_t)gridDim.x * RPB, flip ^= 1) {
    const bool on = r0 + sub < a.M;
    const int64_t m = on ? r0 + sub : 0;
    const int n = on ? D : 0;
    const T* sp = reinterpret_cast<const T*>(a.x) + m * a.xs;
    const T* dp = reinterpret_cast<const T*>(a.dy) + m * a.ys;
    float s[NC][VE], dy[NC][VE];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int j = (c * TPR + t) * VE;
      ldv<T, VE>(s[c], sp + j, n - j);
      ldv<T, VE>(dy[c], dp + j, n - j);
    }
    const float rstd = a.rstd[m];
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        dw[c][e] += dy[c][e] * (s[c][e] * rstd);  // rows past the end are zeros
        dy[c][e] *= wv[c][e];
        dot += dy[c][e] * s[c][e];
      }
    // the two buffers alternate, so a row's sums are read before they are overwritten
    const float k = row_sum<TPR>(dot, sbuf[flip]) / (float)D * rstd * rstd;
    if (a.res) {
      const T* gp = reinterpret_cast<const T*>(a.res) + m * a.rs;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int j = (c * TPR + t) * VE;
        float ds[VE];
        ldv<T, VE>(ds, gp + j, n - j);
#pragma unroll
        for (int e = 0; e < VE; ++e) dy[c][e] = rstd * (dy[c][e] - s[c][e] * k) + ds[e];
      }
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < VE; ++e) dy[c][e] = rstd * (dy[c][e] - s[c][e] * k);
    }
    T* o = reinterpret_cast<T*>(a.sum) + m * a.ss;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int j = (c * TPR + t) * VE;
      stv<T, VE>(o + j, dy[c], n - j);
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * D;
  if constexpr (RPB > 1) {  // the block's row groups, joined in their order
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < VE; ++e) wbuf[(sub * NC * VE + c * VE + e) * TPR + t] = dw[c][e];
    __syncthreads();
    for (int i = threadIdx.x; i < TPR * NC * VE; i += BLOCK) {
      // entry i is element e of vector c of thread tt
      const int tt = i % TPR, ce = i / TPR, j = ((ce / VE) * TPR + tt) * VE + ce % VE;
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < RPB; ++k) v += wbuf[(k * NC * VE + ce) * TPR + tt];
      if (j < D) part[j] = v;
    }
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int j = (c * TPR + t) * VE;
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (j + e < D) part[j + e] = dw[c][e];
    }
  }
}

// Column sums: 16 columns a block, 64 groups of partial rows, joined in LDS (1024
// rows of 4096: 7.3 us, most of it latency; the rows lie in the last-level cache).
template <typename O>
__global__ __launch_bounds__(1024) void k_colsum(const float* part, int np, int64_t ld, int64_t n, O* out, O* out2, int64_t split) {
  __shared__ float buf[64][17];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int64_t j = blockIdx.x * (int64_t)16 + c;
  float v = 0.f;
  if (j < n) {
#pragma unroll 8
    for (int p = g; p < np; p += 64) v += part[p * ld + j];
  }
  buf[g][c] = v;
  __syncthreads();
  if (g == 0 && j < n) {
    float s = 0.f;
#pragma unroll 16
    for (int i = 0; i < 64; ++i) s += buf[i][c];
    O* o = j < split ? out + j : out2 + (j - split);
    if (j < split ? out != nullptr : out2 != nullptr) *o = (O)s;
  }
}

// The row shape of a length: the fewest threads that hold it in at most
// 16 (TPR <= 64) or 32 elements each, so that long rows keep many loads in
// flight and short ones share a block.
template <typename T, typename F>
hipError_t norm_shape(int D, F&& f) {
  constexpr int VE = Vec<T>::VE;
  const int v = (D + VE - 1) / VE;  // vectors of a row
#define REWY_NORM_SHAPE(TPR, NC) \
  if (v <= (TPR) * (NC)) return f(std::integral_constant<int, TPR>{}, std::integral_constant<int, NC>{})
  REWY_NORM_SHAPE(16, 1);
  REWY_NORM_SHAPE(64, 1);
  REWY_NORM_SHAPE(64, 2);
  REWY_NORM_SHAPE(256, 1);
  REWY_NORM_SHAPE(256, 2);
  REWY_NORM_SHAPE(256, 4);
  REWY_NORM_SHAPE(1024, 2);
  if constexpr (VE == 4) REWY_NORM_SHAPE(1024, 4);
#undef REWY_NORM_SHAPE
  return hipErrorInvalidValue;
}

template <typename T, typename W>
hipError_t norm_fwd_t(const NormArgs& a, hipStream_t s) {
  return norm_shape<T>(a.D, [&](auto tpr, auto nc) {
    constexpr int TPR = decltype(tpr)::value, NC = decltype(nc)::value;
    constexpr int BLOCK = TPR > NORM_BLOCK ? TPR : NORM_BLOCK, RPB = BLOCK / TPR;
    // (a launch takes fewer than 2^32 threads along x)
    const int64_t n = (a.M + RPB - 1) / RPB, gx = std::min<int64_t>(n, 1 << 20);
    REWY_LAUNCH((k_norm_fwd<T, W, TPR, NC>), dim3((unsigned)gx, (unsigned)((n + gx - 1) / gx)), dim3(BLOCK), s, a);
    return hipGetLastError();
  });
}
template <typename T, typename W>
hipError_t norm_bwd_t(const NormArgs& a, hipStream_t s) {
  return norm_shape<T>(a.D, [&](auto tpr, auto nc) {
    constexpr int TPR = decltype(tpr)::value, NC = decltype(nc)::value;
    constexpr int BLOCK = TPR > NORM_BLOCK ? TPR : NORM_BLOCK;
    REWY_LAUNCH((k_norm_bwd<T, W, TPR, NC>), dim3(a.nblk), dim3(BLOCK), s, a);
    return hipGetLastError();
  });
}

}  // namespace

int norm_bwd_blocks(int64_t M, int D, bool f32) {
  int rpb = 1;
  auto take = [&](auto tpr, auto) {
    rpb = std::max(1, NORM_BLOCK / decltype(tpr)::value);
    return hipSuccess;
  };
  (void)(f32 ? norm_shape<float>(D, take) : norm_shape<bf16>(D, take));
  // four blocks a CU (8192 x 4096 bf16: 58 + 9 us with 1024, 84 + 7 us with 512 blocks)
  return (int)std::min<int64_t>((M + rpb - 1) / rpb, 1024);
}

hipError_t launch_norm_fwd(const NormArgs& a, bool f32, bool wf32, hipStream_t s) {
  if (f32) return wf32 ? norm_fwd_t<float, float>(a, s) : norm_fwd_t<float, bf16>(a, s);
  return wf32 ? norm_fwd_t<bf16, float>(a, s) : norm_fwd_t<bf16, bf16>(a, s);
}
hipError_t launch_norm_bwd(const NormArgs& a, bool f32, bool wf32, hipStream_t s) {
  if (f32) return wf32 ? norm_bwd_t<float, float>(a, s) : norm_bwd_t<float, bf16>(a, s);
  return wf32 ? norm_bwd_t<bf16, float>(a, s) : norm_bwd_t<bf16, bf16>(a, s);
}
hipError_t launch_colsum(const float* part, int np, int64_t ld, int64_t n, void* out, bool out_f32,
                         hipStream_t s, void* out2, int64_t split) {
  const dim3 grid((unsigned)((n + 15) / 16)), block(1024);
  if (split < 0) split = n;
  if (out_f32)
    REWY_LAUNCH((k_colsum<float>), grid, block, s, part, np, ld, n, reinterpret_cast<float*>(out),
                reinterpret_cast<float*>(out2), split);
  else
    REWY_LAUNCH((k_colsum<bf16>), grid, block, s, part, np, ld, n, reinterpret_cast<bf16*>(out),
                reinterpret_cast<bf16*>(out2), split);
  return hipGetLastError();
}

}  // namespace rewy
