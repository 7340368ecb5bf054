// Group norm over a token's channels, with a gate or an activation behind it and an
// 8-bit output.  Row by row, for each of G groups of L channels,
//   mean = avg x (or 0),  rstd = (avg (x - mean)^2 + eps)^-1/2,
//   n = (x - mean) rstd w + b,   y = n act(z)  or  y = act(n)  without a gate z,
// and scales and codes of y as the RMS norm's.  Everything is formed from the
// unrounded fp32 values; y and q are rounded once each.  Backward, with xh = (x -
// mean) rstd, dn = dy act(z) or dy act'(n), u = dn w:
//   dx = rstd (u - avg u - xh avg(u xh)),  dz = dy n act'(z),
//   dw = sum_rows dn xh,  db = sum_rows dn
// (avg u only with a mean).
//
// Memory is all it costs: each input is read once and each output written once.  A
// row is held by TPR threads in registers (NC vectors of 16 bytes a thread).  Where a
// group is a power of two of whole vectors, at most a wave, its lanes are neighbours
// and its statistics a few lane moves.  Any other group length takes them from the row's
// copy in LDS, and the backward its two means from the row's u and u xh there.
#include "gnorm.hpp"

namespace rewy {

namespace {

// Sum over aligned groups of `lanes` lanes (a power of two up to 64), in every lane.
__device__ __forceinline__ float group_sum(float x, int lanes) {
  if (lanes > 1) x += dpp_mov<0xB1>(x);   // quad_perm [1,0,3,2]
  if (lanes > 2) x += dpp_mov<0x4E>(x);   // quad_perm [2,3,0,1]
  if (lanes > 4) x += dpp_mov<0x141>(x);  // row_half_mirror
  if (lanes > 8) x += dpp_mov<0x140>(x);  // row_mirror
  if (lanes > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if (lanes > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return x;
}

// the same for the maximum of magnitudes (as bits)
__device__ __forceinline__ uint32_t group_max(uint32_t x, int lanes) {
  if (lanes > 1) x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xf, 0xf, true));
  if (lanes > 2) x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xf, 0xf, true));
  if (lanes > 4) x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x141, 0xf, 0xf, true));
  if (lanes > 8) x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x140, 0xf, 0xf, true));
  if (lanes > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = max((uint32_t)r[0], (uint32_t)r[1]);
  }
  if (lanes > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = max((uint32_t)r[0], (uint32_t)r[1]);
  }
  return x;
}

// the activation's value, and its derivative.  The sigmoid is the hardware's exponential and
// reciprocal: within (2 |t| + 8) 2^-24 of itself, for 32-bit tensors too.
template <int ACT>
__device__ __forceinline__ float act_value(float t) {
  return ACT == REWY_ACT_NONE ? t : ACT == REWY_ACT_SILU ? t * sigmoid_f(t) : sigmoid_f(t);
}
template <int ACT>
__device__ __forceinline__ float act_both(float t, float& d) {
  if constexpr (ACT == REWY_ACT_NONE) {
    d = 1.f;
    return t;
  } else {
    const float s = sigmoid_f(t);
    d = ACT == REWY_ACT_SILU ? s * (1.f + t * (1.f - s)) : s * (1.f - s);
    return ACT == REWY_ACT_SILU ? t * s : s;
  }
}
// f with the activation as a constant (the choice is the same in the whole launch and made
// outside the loops over elements)
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  if (act == REWY_ACT_SILU) f(std::integral_constant<int, REWY_ACT_SILU>{});
  else if (act == REWY_ACT_SIGMOID) f(std::integral_constant<int, REWY_ACT_SIGMOID>{});
  else f(std::integral_constant<int, REWY_ACT_NONE>{});
}

// The groups' statistics of a vector of a row, from memory: element e of columns j ..
template <int VE>
struct GroupOf {
  int g[VE];
  __device__ __forceinline__ GroupOf(int j, int L, int G) {
    int k = j / L, r = j - k * L;
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      g[e] = min(k, G - 1);
      if (++r == L) {
        r = 0;
        ++k;
      }
    }
  }
};

// Statistics of a row's groups from its copy q in LDS, by TPR threads, to memory: P lanes a
// group (a power of two: about four channels a lane, or vectors where groups are whole
// ones), or several waves where there are two for each group (8192 rows of one group of 4096
// bf16: 49 us, with a wave 69).  m < 0: no row.
template <typename T, int TPR>
__device__ __forceinline__ void row_stats(const GnormArgs& a, const T* q, int t, int64_t m) {
  constexpr int VE = Vec<T>::VE, LIM = TPR < 64 ? TPR : 64, NW = TPR / LIM;
  __shared__ float parts[TPR < NORM_BLOCK ? NORM_BLOCK / TPR : 1][2][NW];  // (of each row of the block)
  float(&part)[2][NW] = parts[threadIdx.x / TPR];
  const bool vec = a.L % VE == 0;
  // f of a lane's share of x, lane p of n
  auto all = [&](const T* x, int p, int n, auto&& f) {
    if (vec) {
      for (int j = p * VE; j < a.L; j += n * VE) {
        const auto v = *reinterpret_cast<const typename VecN<T, VE>::raw*>(x + j);
#pragma unroll
        for (int e = 0; e < VE; ++e) f((float)v[e]);
      }
    } else {
      for (int j = p; j < a.L; j += n) f((float)x[j]);
    }
  };
  auto put = [&](int i, float mean, float rstd) {
    if (m < 0 || i >= a.G) return;
    if (a.center) a.mean[m * a.G + i] = mean;
    a.rstd[m * a.G + i] = rstd;
  };
  if (NW > 1 && 2 * a.G <= NW) {
    const int S = 1 << (31 - __builtin_clz(NW / a.G)), w = t / LIM, p = t - w * LIM, i = w / S;
    const int at = (w & (S - 1)) * LIM + p;
    const T* x = q + min(i, a.G - 1) * a.L;
    auto join = [&](float (&buf)[NW], float s) {
      s = group_sum(s, LIM);
      if (p == 0) buf[w] = s;
      __syncthreads();
      s = 0.f;
      for (int k = 0; k < S; ++k) s += buf[(w & -S) + k];
      return s;
    };
    float s = 0.f, mean = 0.f;
    if (a.center) {
      all(x, at, S * LIM, [&](float v) { s += v; });
      mean = join(part[0], s) / (float)a.L;
      s = 0.f;
    }
    all(x, at, S * LIM, [&](float v) { s += (v - mean) * (v - mean); });
    s = join(part[1], s);
    if (at == 0) put(i, mean, rsqrtf(s / (float)a.L + a.eps));
    return;
  }
  int P = 1;
  while (P < LIM && 4 * P < a.L) P *= 2;
  const int p = t & (P - 1), sh = __builtin_ctz(P), per = TPR >> sh;
  for (int i0 = 0; i0 < a.G; i0 += per) {
    const int i = i0 + (t >> sh);  // (whole waves stay together for the lane moves)
    const T* x = q + min(i, a.G - 1) * a.L;
    float s = 0.f, mean = 0.f;
    if (a.center) {
      all(x, p, P, [&](float v) { s += v; });
      mean = group_sum(s, P) / (float)a.L;
      s = 0.f;
    }
    all(x, p, P, [&](float v) { s += (v - mean) * (v - mean); });
    const float rstd = rsqrtf(group_sum(s, P) / (float)a.L + a.eps);
    if (p == 0) put(i, mean, rstd);
  }
}

// The means of u and v over a row's groups, from LDS and to each group's first place there
// (shared out as in row_stats; a barrier before and after).
template <int TPR>
__device__ __forceinline__ void row_means(const GnormArgs& a, float* u, float* v, int t) {
  constexpr int LIM = TPR < 64 ? TPR : 64, NW = TPR / LIM;
  __shared__ float parts[TPR < NORM_BLOCK ? NORM_BLOCK / TPR : 1][2][NW];  // (of each row of the block)
  float(&part)[2][NW] = parts[threadIdx.x / TPR];
  const bool vec = a.L % 4 == 0;
  auto sum = [&](int at, int p, int n, float& s1, float& s2) {
    s1 = s2 = 0.f;
    if (vec) {
      for (int j = at + 4 * p; j < at + a.L; j += 4 * n) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(u + j), y = *reinterpret_cast<const f32x4*>(v + j);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s1 += x[e];
          s2 += y[e];
        }
      }
    } else {
      for (int j = at + p; j < at + a.L; j += n) {
        s1 += u[j];
        s2 += v[j];
      }
    }
  };
  float s1, s2;
  if (NW > 1 && 2 * a.G <= NW) {
    const int S = 1 << (31 - __builtin_clz(NW / a.G)), w = t / LIM, p = t - w * LIM, i = w / S;
    sum(min(i, a.G - 1) * a.L, (w & (S - 1)) * LIM + p, S * LIM, s1, s2);
    s1 = group_sum(s1, LIM);
    s2 = group_sum(s2, LIM);
    if (p == 0) {
      part[0][w] = s1;
      part[1][w] = s2;
    }
    __syncthreads();
    if (t < a.G) {
      s1 = s2 = 0.f;
      for (int k = 0; k < S; ++k) {
        s1 += part[0][t * S + k];
        s2 += part[1][t * S + k];
      }
      u[t * a.L] = s1 / (float)a.L;
      v[t * a.L] = s2 / (float)a.L;
    }
    return;
  }
  int P = 1;
  while (P < LIM && 4 * P < a.L) P *= 2;
  const int p = t & (P - 1), sh = __builtin_ctz(P), per = TPR >> sh;
  for (int i0 = 0; i0 < a.G; i0 += per) {
    // (whole waves stay together for the lane moves; a lane that has no group takes part
    // with the last one's and keeps nothing)
    const int i = i0 + (t >> sh), at = min(i, a.G - 1) * a.L;
    sum(at, p, P, s1, s2);
    s1 = group_sum(s1, P);
    s2 = group_sum(s2, P);
    if (p == 0 && i < a.G) {
      u[at] = s1 / (float)a.L;
      v[at] = s2 / (float)a.L;
    }
  }
}

// A thread's NC vectors of a row as they lie in memory (columns past n: zeros).
template <typename T, int NC>
struct RawRow {
  static constexpr int VE = Vec<T>::VE;
  typename VecN<T, VE>::raw v[NC];
  __device__ __forceinline__ void load(const T* p, int t, int tpr, int n) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int j = (c * tpr + t) * VE;
      if (n - j >= VE) {
        v[c] = *reinterpret_cast<const typename VecN<T, VE>::type*>(p + j);
      } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) v[c][e] = j + e < n ? p[j + e] : (T)0.f;
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[NC][VE]) const {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < VE; ++e) f[c][e] = (float)v[c][e];
  }
};

// One row a TPR threads, and a block's rows are all it does: the blocks that wait for
// memory and those that count lie over each other (a block that walks rows with the next
// one sent for ahead: 55.7 us where this takes 47.8).  All loads go out before the first
// use; group and scale indices are shifts and a group's mean a product with an exact
// 1 / L, for the row's arithmetic costs nearly what its bytes do (with divisions 51.7 us
// where this takes 45).  8192 rows of 32 groups of 128 bf16 with a gate: 47.8 us
// (4.2 TB/s) to bf16, 45.7 us (3.7 TB/s) to e4m3 with a scale for each 128; 16 rows 4.1.
// 2003 rows of 29 groups of 53 fp32 to int8: 18.9 us (12.2 behind a launch of 9.2 that took
// the statistics from memory; 8192 x 32 x 100 bf16 to bf16: 55 and 76 us a call).
template <typename T, typename W, int TPR, int NC, bool ODD>
__global__ __launch_bounds__(TPR > NORM_BLOCK ? TPR : NORM_BLOCK) void k_gnorm_fwd(GnormArgs a) {
  constexpr int VE = Vec<T>::VE, BLOCK = TPR > NORM_BLOCK ? TPR : NORM_BLOCK, RPB = BLOCK / TPR;
  __shared__ uint32_t mbuf[BLOCK / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = (blockIdx.y * (int64_t)gridDim.x + blockIdx.x) * RPB + threadIdx.x / TPR;
  const bool on = row < a.M;
  const int D = on ? a.D : 0;  // threads past the last row hold nothing and write nothing
  const int64_t m = on ? row : 0;
  const T* x = reinterpret_cast<const T*>(a.x) + m * a.xs;
  const T* z = a.z ? reinterpret_cast<const T*>(a.z) + m * a.zs : nullptr;
  const W* w = reinterpret_cast<const W*>(a.w);
  const W* b = reinterpret_cast<const W*>(a.b);

  const int lsh = ODD ? 0 : __builtin_ctz(a.lanes);  // (a power of two)
  float s[NC][VE], zv[NC][VE], wv[NC][VE], bv[NC][VE];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int j = (c * TPR + t) * VE;
    ldv<T, VE>(s[c], x + j, D - j);
  }
  if (z) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int j = (c * TPR + t) * VE;
      ldv<T, VE>(zv[c], z + j, D - j);
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int j = (c * TPR + t) * VE;
    if (w) ldv<W, VE>(wv[c], w + j, D - j);
    if (b) ldv<W, VE>(bv[c], b + j, D - j);
  }
  if constexpr (ODD) {
    constexpr int ROW = TPR * NC * VE;
    __shared__ __align__(16) T copy[RPB * ROW];
    T* q = copy + threadIdx.x / TPR * ROW;
#pragma unroll
    for (int c = 0; c < NC; ++c) stv<T, VE>(q + (c * TPR + t) * VE, s[c], VE);  // (exact: as they were read)
    __syncthreads();
    row_stats<T, TPR>(a, q, t, on ? row : -1);
    __syncthreads();  // (statistics of the block's own rows, read below)
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int j = (c * TPR + t) * VE;
    if constexpr (ODD) {
      const GroupOf<VE> of(j, a.L, a.G);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int64_t i = m * a.G + of.g[e];
        s[c][e] = (s[c][e] - (a.center ? a.mean[i] : 0.f)) * a.rstd[i];
      }
    } else {
      // (a vector lies in one group, and a group's lanes in one wave)
      float mean = 0.f, ss = 0.f;
      if (a.center) {
#pragma unroll
        for (int e = 0; e < VE; ++e) mean += s[c][e];
        mean = group_sum(mean, a.lanes) * a.rL;
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        s[c][e] -= mean;
        ss += s[c][e] * s[c][e];
      }
      const float rstd = rsqrtf(group_sum(ss, a.lanes) * a.rL + a.eps);
#pragma unroll
      for (int e = 0; e < VE; ++e) s[c][e] *= rstd;
      if (j < D && (t & (a.lanes - 1)) == 0) {
        const int64_t i = m * a.G + ((c * TPR + t) >> lsh);
        if (a.center) a.mean[i] = mean;
        a.rstd[i] = rstd;
      }
    }
    if (w) {
#pragma unroll
      for (int e = 0; e < VE; ++e) s[c][e] *= wv[c][e];
    }
    if (b) {
#pragma unroll
      for (int e = 0; e < VE; ++e) s[c][e] += bv[c][e];
    }
  }
  with_act(a.act, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    if (z) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < VE; ++e) s[c][e] *= act_value<ACT>(zv[c][e]);
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < VE; ++e) s[c][e] = act_value<ACT>(s[c][e]);
    }
  });
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
    const int j = (c * TPR + t) * VE;
    mx[c] = 0;
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (j + e < D) mx[c] = max(mx[c], mag(s[c][e]));
    all = max(all, mx[c]);
  }
  if (!a.group) all = row_max<TPR>(all, mbuf);
  const int lanes = a.group ? min(a.group / VE, TPR) : 0;  // lanes that share a scale
  const int gsh = a.group ? __builtin_ctz(a.group) : 0;          // (a power of two)
  uint8_t* q = reinterpret_cast<uint8_t*>(a.q) + m * a.D;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int j = (c * TPR + t) * VE;
    const float scale = make_scale(a.group ? group_max(mx[c], lanes) : all, qmax);
    if (a.group) {
      if (j < D && (j & (a.group - 1)) == 0) a.scale[m * a.ng + (j >> gsh)] = scale;
    } else if (c == 0 && t == 0 && on) {
      a.scale[m] = scale;
    }
    const bool e4m3 = a.quant == REWY_QUANT_E4M3;
    if (ScaleDiv::holds(scale)) store_codes_by<VE>(q + j, s[c], ScaleDiv(scale), e4m3, D - j);
    else store_codes<VE>(q + j, s[c], scale, e4m3, D - j);
  }
}

// Each block takes rows blockIdx, + gridDim, ... and keeps dw and db of its columns in
// registers; one partial row of each per block goes to the workspace (no atomics: the
// same sums every time).  With one vector a thread the next row is sent for before this
// one is counted.  8192 rows of 32 groups of 128 bf16 with a gate: 74.5 us (4.5 TB/s),
// and 7.4 for the two column sums, whose floor is a launch's latency.  Other group lengths
// pay for their means in LDS: 65536 x 19 x 53 bf16 351 us a call (with the means by a
// launch of its own 478), 65536 x 8 x 128 80.
template <typename T, typename W, int TPR, int NC, bool ODD>
__global__ __launch_bounds__(TPR > NORM_BLOCK ? TPR : NORM_BLOCK) void k_gnorm_bwd(GnormArgs a) {
  constexpr int VE = Vec<T>::VE, BLOCK = TPR > NORM_BLOCK ? TPR : NORM_BLOCK, RPB = BLOCK / TPR;
  constexpr int ROW = TPR * NC * VE;
  __shared__ float wbuf[RPB > 1 ? BLOCK * NC * VE : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR, D = a.D;
  const W* w = reinterpret_cast<const W*>(a.w);
  const W* b = reinterpret_cast<const W*>(a.b);
  float wv[NC][VE], bv[NC][VE], dw[NC][VE], db[NC][VE];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int j = (c * TPR + t) * VE;
    if (w) ldv<W, VE>(wv[c], w + j, D - j);
    if (b) ldv<W, VE>(bv[c], b + j, D - j);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      if (!w) wv[c][e] = 1.f;
      if (!b) bv[c][e] = 0.f;
      dw[c][e] = db[c][e] = 0.f;
    }
  }
  const int lsh = ODD ? 0 : __builtin_ctz(a.lanes);
  // rows as they lie in memory, one ahead of its use
  RawRow<T, NC> nx, nd, nz;
  auto fetch = [&](int64_t r0) {
    const bool on = r0 + sub < a.M;
    const int64_t m = on ? r0 + sub : 0;
    const int n = on ? D : 0;
    nx.load(reinterpret_cast<const T*>(a.x) + m * a.xs, t, TPR, n);
    nd.load(reinterpret_cast<const T*>(a.dy) + m * a.ys, t, TPR, n);
    if (a.z) nz.load(reinterpret_cast<const T*>(a.z) + m * a.zs, t, TPR, n);
  };
  if constexpr (NC == 1) fetch(blockIdx.x * (int64_t)RPB);
  for (int64_t r0 = blockIdx.x * (int64_t)RPB; r0 < a.M; r0 += (int64_t)gridDim.x * RPB) {
    const bool on = r0 + sub < a.M, zp = a.z != nullptr;
    const int64_t m = on ? r0 + sub : 0;
    const int n = on ? D : 0;
    float x[NC][VE], dy[NC][VE], zv[NC][VE];
    if constexpr (NC > 1) fetch(r0);  // (no registers to hold a second row)
    nx.get(x);
    nd.get(dy);
    if (zp) nz.get(zv);
    if constexpr (NC == 1) fetch(r0 + (int64_t)gridDim.x * RPB);
    float rs[NC][VE];  // (one value a vector unless ODD)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int j = (c * TPR + t) * VE;
      if constexpr (ODD) {
        const GroupOf<VE> of(j, a.L, a.G);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const int64_t i = m * a.G + of.g[e];
          rs[c][e] = a.rstd[i];
          x[c][e] = j + e < n ? (x[c][e] - (a.center ? a.mean[i] : 0.f)) * rs[c][e] : 0.f;
        }
      } else {
        const int64_t i = m * a.G + (j < n ? (c * TPR + t) >> lsh : 0);
        const float r = a.rstd[i], mean = a.center ? a.mean[i] : 0.f;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          rs[c][e] = r;
          x[c][e] = j < n ? (x[c][e] - mean) * r : 0.f;
        }
      }
      // dn (rows and columns past the end: zero), and dz
      with_act(a.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        if (zp) {
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            float d;
            const float v = act_both<ACT>(zv[c][e], d);
            zv[c][e] = dy[c][e] * (x[c][e] * wv[c][e] + bv[c][e]) * d;
            dy[c][e] *= v;
          }
        } else {
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            float d;
            act_both<ACT>(x[c][e] * wv[c][e] + bv[c][e], d);
            dy[c][e] *= d;
          }
        }
      });
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        dw[c][e] += dy[c][e] * x[c][e];
        db[c][e] += dy[c][e];
        dy[c][e] *= wv[c][e];
      }
    }
    float *mu = nullptr, *mv = nullptr;
    if constexpr (ODD) {
      __shared__ __align__(16) float us[RPB * ROW], vs[RPB * ROW];
      mu = us + sub * ROW;
      mv = vs + sub * ROW;
      __syncthreads();  // (the row before has been read)
#pragma unroll
      for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          mu[(c * TPR + t) * VE + e] = dy[c][e];
          mv[(c * TPR + t) * VE + e] = dy[c][e] * x[c][e];
        }
      }
      __syncthreads();
      row_means<TPR>(a, mu, mv, t);
      __syncthreads();
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int j = (c * TPR + t) * VE;
      if constexpr (ODD) {
        const GroupOf<VE> of(j, a.L, a.G);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const int at = of.g[e] * a.L;
          dy[c][e] = rs[c][e] * (dy[c][e] - (a.center ? mu[at] : 0.f) - x[c][e] * mv[at]);
        }
      } else {
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          s1 += dy[c][e];
          s2 += dy[c][e] * x[c][e];
        }
        s1 = a.center ? group_sum(s1, a.lanes) * a.rL : 0.f;
        s2 = group_sum(s2, a.lanes) * a.rL;
#pragma unroll
        for (int e = 0; e < VE; ++e) dy[c][e] = rs[c][e] * (dy[c][e] - s1 - x[c][e] * s2);
      }
      stv<T, VE>(reinterpret_cast<T*>(a.dx) + m * a.dxs + j, dy[c], n - j);
      if (zp) stv<T, VE>(reinterpret_cast<T*>(a.dz) + m * a.dzs + j, zv[c], n - j);
    }
  }
  if (!a.part) return;
  // dw, then db
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float* part = a.part + ((int64_t)blockIdx.x * 2 + k) * D;
    float(&d)[NC][VE] = k ? db : dw;
    if constexpr (RPB > 1) {  // the block's row groups, joined in their order
      __syncthreads();
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < VE; ++e) wbuf[(sub * NC * VE + c * VE + e) * TPR + t] = d[c][e];
      __syncthreads();
      for (int i = threadIdx.x; i < TPR * NC * VE; i += BLOCK) {
        // entry i is element e of vector c of thread tt
        const int tt = i % TPR, ce = i / TPR, j = ((ce / VE) * TPR + tt) * VE + ce % VE;
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < RPB; ++q) v += wbuf[(q * NC * VE + ce) * TPR + tt];
        if (j < D) part[j] = v;
      }
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int j = (c * TPR + t) * VE;
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (j + e < D) part[j + e] = d[c][e];
      }
    }
  }
}

// The row shape of a length: one vector a thread as far as a block reaches, which leaves
// registers for the next row (8192 x 4096 bf16 with a gate, backward: 76 us; with two
// vectors and no row ahead 132), and as many threads as vectors to the next power of two:
// threads without a vector cost what the others do (262144 x 256 bf16 by 32 threads a row 53
// us, by 64 87; 1048576 x 32 by 4 threads 25, by 16 75).
// The backward of the longest rows asks for more than the 128 registers that 1024 threads leave
// and spills: with two vectors of bf16 or four of fp32 (past 8192 channels) about 200 bytes a
// thread with groups in lanes and 650 with others, 60 to 150 with others from 4097 channels.  With
// a gate, weight and bias, 2048 rows of 16384 bf16 take 158 us with groups in lanes (128 of 128;
// 68.6 at copy rate) and 440 with others (8 of 2048), 1024 rows of 16384 fp32 133 and 308; the
// forward does not spill (47, 66, 43 and 52 us; 41.2).
template <typename T, typename F>
hipError_t gnorm_shape(int D, F&& f) {
  constexpr int VE = Vec<T>::VE;
  const int v = (D + VE - 1) / VE;  // vectors of a row
#define REWY_GNORM_SHAPE(TPR, NC) \
  if (v <= (TPR) * (NC)) return f(std::integral_constant<int, TPR>{}, std::integral_constant<int, NC>{})
  REWY_GNORM_SHAPE(4, 1);
  REWY_GNORM_SHAPE(8, 1);
  REWY_GNORM_SHAPE(16, 1);
  REWY_GNORM_SHAPE(32, 1);
  REWY_GNORM_SHAPE(64, 1);
  REWY_GNORM_SHAPE(128, 1);
  REWY_GNORM_SHAPE(256, 1);
  REWY_GNORM_SHAPE(512, 1);
  REWY_GNORM_SHAPE(1024, 1);
  REWY_GNORM_SHAPE(1024, 2);
  if constexpr (VE == 4) REWY_GNORM_SHAPE(1024, 4);
#undef REWY_GNORM_SHAPE
  return hipErrorInvalidValue;
}
// rows side by side in a block, and its threads
template <typename T>
void gnorm_block(int D, int& rows, int& threads) {
  (void)gnorm_shape<T>(D, [&](auto tpr, auto) {
    rows = std::max(1, NORM_BLOCK / decltype(tpr)::value);
    threads = std::max(NORM_BLOCK, decltype(tpr)::value);
    return hipSuccess;
  });
}

template <typename T, typename W, bool ODD>
hipError_t gnorm_fwd_t(const GnormArgs& a, hipStream_t s) {
  return gnorm_shape<T>(a.D, [&](auto tpr, auto nc) {
    constexpr int TPR = decltype(tpr)::value, NC = decltype(nc)::value;
    constexpr int BLOCK = TPR > NORM_BLOCK ? TPR : NORM_BLOCK, RPB = BLOCK / TPR;
    // (a launch takes fewer than 2^32 threads along x)
    const int64_t n = (a.M + RPB - 1) / RPB, gx = std::min<int64_t>(n, 1 << 20);
    REWY_LAUNCH((k_gnorm_fwd<T, W, TPR, NC, ODD>), dim3((unsigned)gx, (unsigned)((n + gx - 1) / gx)), dim3(BLOCK), s, a);
    return hipGetLastError();
  });
}
template <typename T, typename W, bool ODD>
hipError_t gnorm_bwd_t(const GnormArgs& a, hipStream_t s) {
  return gnorm_shape<T>(a.D, [&](auto tpr, auto nc) {
    constexpr int TPR = decltype(tpr)::value, NC = decltype(nc)::value;
    REWY_LAUNCH((k_gnorm_bwd<T, W, TPR, NC, ODD>), dim3(a.nblk), dim3(TPR > NORM_BLOCK ? TPR : NORM_BLOCK), s, a);
    return hipGetLastError();
  });
}
// the (T, W) variants
template <typename F>
hipError_t gnorm_types(bool f32, bool wf32, F&& f) {
  if (f32) return wf32 ? f(float{}, float{}) : f(float{}, bf16{});
  return wf32 ? f(bf16{}, float{}) : f(bf16{}, bf16{});
}

}  // namespace

int gnorm_lanes(int L, bool f32) {
  const int ve = f32 ? 4 : 8, n = L / ve;
  return L % ve == 0 && n <= 64 && (n & (n - 1)) == 0 ? n : 0;
}
int gnorm_bwd_blocks(int64_t M, int D, bool f32) {
  int rpb = 1, block = NORM_BLOCK;
  if (f32) gnorm_block<float>(D, rpb, block);
  else gnorm_block<bf16>(D, rpb, block);
  // as many as are at work at once, 1024 threads a CU (8192 x 4096 bf16: 76 us with 512
  // blocks of 512 threads, 106 with half and 87 with twice as many)
  return (int)std::min<int64_t>((M + rpb - 1) / rpb, 256 * 1024 / block);
}

hipError_t launch_gnorm_fwd(const GnormArgs& a, bool f32, bool wf32, hipStream_t s) {
  return gnorm_types(f32, wf32, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    return a.lanes ? gnorm_fwd_t<T, W, false>(a, s) : gnorm_fwd_t<T, W, true>(a, s);
  });
}
hipError_t launch_gnorm_bwd(const GnormArgs& a, bool f32, bool wf32, hipStream_t s) {
  return gnorm_types(f32, wf32, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    return a.lanes ? gnorm_bwd_t<T, W, false>(a, s) : gnorm_bwd_t<T, W, true>(a, s);
  });
}

}  // namespace rewy
