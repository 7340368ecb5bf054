// Short causal convolution along the tokens, channel by channel, with an
// optional bias and SiLU:
//   pre_t = bias + sum_{j < W} w_j x_{t - (W-1) + j},   y_t = act(pre_t),
// where the W - 1 rows before a sequence's first token are its initial state
// (zeros without one) and the final state is the last W - 1 rows of
// [initial state ; x].  Backward, with dpre_t = dy_t act'(pre_t):
//   dx_t = sum_{o < W} w_{W-1-o} dpre_{t+o} (+ the final state's adjoint on the
//   last W - 1 rows),   dw_j = sum_t dpre_t x_{t-(W-1)+j},   dbias = sum_t dpre_t.
//
// Memory is all it costs.  A lane owns VE channels (16 bytes) and walks a run
// of tokens with the last W - 1 rows in registers, so each row is read once
// per run plus W - 1 rows at its start.  Tokens are packed; a run that meets
// the end of a sequence takes up the next one's state.
#include "layer.hpp"

namespace rewy {

namespace {

constexpr int CONV_WAVES = 4;  // runs (waves) of one block, side by side along the tokens

__device__ __forceinline__ float silu(float z) { return z * sigmoid_f(z); }

// The sequence that token t < total belongs to: the largest n with start(n) <= t.
__device__ __forceinline__ int seq_of(const SeqArgs& q, int t) {
  if (!q.cu) return t / q.T;
  int lo = 0, hi = q.N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq_start(q, mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Row p of sequence n counted from its first token; p < 0 reads the initial state.
template <typename T, int W>
__device__ __forceinline__ void conv_row(float (&f)[Vec<T>::VE], const ConvArgs& a, int n, int bos, int p, int c, int nv) {
  constexpr int VE = Vec<T>::VE;
  if (p >= 0) {
    ldv<T>(f, reinterpret_cast<const T*>(a.x) + (int64_t)(bos + p) * a.xs + c, nv);
  } else if (a.h0) {
    ldv<T>(f, reinterpret_cast<const T*>(a.h0) + ((int64_t)n * (W - 1) + (W - 1) + p) * a.D + c, nv);
  } else {
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = 0.f;
  }
}

// taps as wt[j][e] for channels c .. c + VE - 1
template <typename WT, int VE, int W>
__device__ __forceinline__ void conv_taps(float (&wt)[W][VE], float (&b)[VE], const ConvArgs& a, int c, int nv) {
  const WT* w = reinterpret_cast<const WT*>(a.w) + (int64_t)c * W;
#pragma unroll
  for (int e = 0; e < VE; ++e)
#pragma unroll
    for (int j = 0; j < W; ++j) wt[j][e] = e < nv ? (float)w[e * W + j] : 0.f;
#pragma unroll
  for (int e = 0; e < VE; ++e) b[e] = 0.f;
  if (a.bias) ldw<VE, WT>(b, reinterpret_cast<const WT*>(a.bias) + c, nv);
}

// Final state of sequence n (grid rows past the token tiles).
template <typename T, int W>
__device__ __forceinline__ void conv_final(const ConvArgs& a, int n, int c, int nv) {
  constexpr int VE = Vec<T>::VE;
  int bos, eos;
  seq_range(a.seq, n, bos, eos);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    float f[VE];
    conv_row<T, W>(f, a, n, bos, eos - bos - (W - 1) + k, c, nv);
    stv<T>(reinterpret_cast<T*>(a.ht) + ((int64_t)n * (W - 1) + k) * a.D + c, f, nv);
  }
}

template <typename T, typename WT, int W>
__global__ __launch_bounds__(64 * CONV_WAVES) void k_conv_fwd(ConvArgs a) {
  constexpr int VE = Vec<T>::VE;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = (blockIdx.y * 64 + lane) * VE, nv = a.D - c;
  if (nv <= 0) return;
  if ((int)blockIdx.x >= a.tiles) {  // one sequence's final state per wave
    const int n = (blockIdx.x - a.tiles) * CONV_WAVES + wave;
    if (n < a.seq.N) conv_final<T, W>(a, n, c, nv);
    return;
  }
  const int64_t first = (blockIdx.x * (int64_t)CONV_WAVES + wave) * a.run;
  const int total = seq_start(a.seq, a.seq.N);  // rows behind the last sequence stay as they are
  if (first >= total) return;
  int t = (int)first;
  const int end = min(t + a.run, total);
  float wt[W][VE], b[VE], h[W - 1][VE];  // h[k]: row t - (W-1) + k
  conv_taps<WT, VE, W>(wt, b, a, c, nv);
  int n = seq_of(a.seq, t), bos, eos;
  seq_range(a.seq, n, bos, eos);
  const T* x = reinterpret_cast<const T*>(a.x) + c;
  T* y = reinterpret_cast<T*>(a.y) + c;
  while (t < end) {
    while (eos <= t && n + 1 < a.seq.N) seq_range(a.seq, ++n, bos, eos);  // (skips empty ones)
    const int stop = eos > t ? min(end, eos) : end;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) conv_row<T, W>(h[k], a, n, bos, t - bos - (W - 1) + k, c, nv);
    constexpr int U = 4;  // rows requested together
    for (; t < stop; t += U) {
      float xv[U][VE];
#pragma unroll
      for (int u = 0; u < U; ++u) ldv<T>(xv[u], x + (int64_t)min(t + u, stop - 1) * a.xs, nv);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float o[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          float p = b[e];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) p += wt[j][e] * h[j][e];
          p += wt[W - 1][e] * xv[u][e];
          o[e] = a.act == REWY_ACT_SILU ? silu(p) : p;
#pragma unroll
          for (int j = 0; j + 1 < W - 1; ++j) h[j][e] = h[j + 1][e];
          h[W - 2][e] = xv[u][e];
        }
        if (t + u < stop) stv<T>(y + (int64_t)(t + u) * a.ys, o, nv);
      }
    }
    t = stop;
  }
}

// One token per sequence; every state row is read before any is written, by
// the same lane, so the state may be updated in place.
template <typename T, typename WT, int W>
__global__ __launch_bounds__(64) void k_conv_step(ConvArgs a) {
  constexpr int VE = Vec<T>::VE;
  const int c = (blockIdx.y * 64 + threadIdx.x) * VE, nv = a.D - c, n = blockIdx.x;
  if (nv <= 0) return;
  float h[W][VE], wt[W][VE], b[VE];
#pragma unroll
  for (int k = 0; k < W; ++k) conv_row<T, W>(h[k], a, n, n, k - (W - 1), c, nv);
  conv_taps<WT, VE, W>(wt, b, a, c, nv);
  float o[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    float p = b[e];
#pragma unroll
    for (int j = 0; j < W; ++j) p += wt[j][e] * h[j][e];
    o[e] = a.act == REWY_ACT_SILU ? silu(p) : p;
  }
  stv<T>(reinterpret_cast<T*>(a.y) + (int64_t)n * a.ys + c, o, nv);
  if (a.ht) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      stv<T>(reinterpret_cast<T*>(a.ht) + ((int64_t)n * (W - 1) + k) * a.D + c, h[k + 1], nv);
  }
}

// dpre = dy act'(pre) of one row, h[j] = the row's taps
template <typename T, int W>
__device__ __forceinline__ void conv_dpre(float (&dp)[Vec<T>::VE], const float (&h)[W][Vec<T>::VE],
                                          const float (&wt)[W][Vec<T>::VE], const float (&b)[Vec<T>::VE], int act) {
  if (act != REWY_ACT_SILU) return;
#pragma unroll
  for (int e = 0; e < Vec<T>::VE; ++e) {
    float p = b[e];
#pragma unroll
    for (int j = 0; j < W; ++j) p += wt[j][e] * h[j][e];
    const float s = sigmoid_f(p);
    dp[e] *= s * (1.f + p * (1.f - s));
  }
}

// Initial state's adjoint of sequence n: row k takes dpre_t of the tokens
// t <= k through tap k - t, and the final state's adjoint where the sequence
// is shorter than the state.
template <typename T, typename WT, int W>
__device__ __forceinline__ void conv_dh0(const ConvArgs& a, int n, int c, int nv) {
  constexpr int VE = Vec<T>::VE;
  int bos, eos;
  seq_range(a.seq, n, bos, eos);
  const int L = eos - bos;
  float wt[W][VE], b[VE], g[W - 1][VE];
  conv_taps<WT, VE, W>(wt, b, a, c, nv);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
#pragma unroll
    for (int e = 0; e < VE; ++e) g[k][e] = 0.f;
    const int f = k - L;  // row of the final state that this row is
    if (a.dht && f >= 0) ldv<T>(g[k], reinterpret_cast<const T*>(a.dht) + ((int64_t)n * (W - 1) + f) * a.D + c, nv);
  }
#pragma unroll
  for (int t = 0; t < W - 1; ++t) {
    if (t >= L) break;
    float h[W][VE], dp[VE];
#pragma unroll
    for (int j = 0; j < W; ++j) conv_row<T, W>(h[j], a, n, bos, t - (W - 1) + j, c, nv);
    ldv<T>(dp, reinterpret_cast<const T*>(a.dy) + (int64_t)(bos + t) * a.ys + c, nv);
    conv_dpre<T, W>(dp, h, wt, b, a.act);
#pragma unroll
    for (int k = t; k < W - 1; ++k)
#pragma unroll
      for (int e = 0; e < VE; ++e) g[k][e] += wt[k - t][e] * dp[e];
  }
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    stv<T>(reinterpret_cast<T*>(a.dh0) + ((int64_t)n * (W - 1) + k) * a.D + c, g[k], nv);
}

template <typename T, typename WT, int W>
__global__ __launch_bounds__(64 * CONV_WAVES) void k_conv_bwd(ConvArgs a) {
  constexpr int VE = Vec<T>::VE;
  __shared__ float red[CONV_WAVES - 1][VE][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = (blockIdx.y * 64 + lane) * VE, nv = a.D - c;
  if ((int)blockIdx.x >= a.tiles) {
    const int n = (blockIdx.x - a.tiles) * CONV_WAVES + wave;
    if (n < a.seq.N && nv > 0) conv_dh0<T, WT, W>(a, n, c, nv);
    return;
  }
  float wt[W][VE], b[VE], dw[W][VE], db[VE];
  conv_taps<WT, VE, W>(wt, b, a, c, nv);
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
  }
  const int64_t first = (blockIdx.x * (int64_t)CONV_WAVES + wave) * a.run;
  const int total = seq_start(a.seq, a.seq.N);  // rows behind the last sequence stay as they are
  if (first < total && nv > 0) {
    int t0 = (int)first;
    const int end = min(t0 + a.run, total);
    int n = seq_of(a.seq, t0), bos, eos;
    seq_range(a.seq, n, bos, eos);
    const T* dy = reinterpret_cast<const T*>(a.dy) + c;
    T* dx = reinterpret_cast<T*>(a.dx) + c;
    while (t0 < end) {
      while (eos <= t0 && n + 1 < a.seq.N) seq_range(a.seq, ++n, bos, eos);
      // this run's tokens of the sequence: [t0, stop)
      const int stop = eos > t0 ? min(end, eos) : end, last = max(eos, stop);
      float h[W][VE], d[W][VE];  // h[j]: row t - (W-1) + j;  d[j]: dpre of the same row
#pragma unroll
      for (int j = 1; j < W; ++j) conv_row<T, W>(h[j], a, n, bos, t0 - bos - W + j, c, nv);
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int e = 0; e < VE; ++e) d[j][e] = 0.f;
      // token t enters; the row t - (W-1) has met all its taps and leaves
      for (int t = t0; t < stop + W - 1; ++t) {
#pragma unroll
        for (int j = 0; j + 1 < W; ++j)
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            h[j][e] = h[j + 1][e];
            d[j][e] = d[j + 1][e];
          }
        float dp[VE];
        if (t < last) {
          conv_row<T, W>(h[W - 1], a, n, bos, t - bos, c, nv);
          ldv<T>(dp, dy + (int64_t)t * a.ys, nv);
          conv_dpre<T, W>(dp, h, wt, b, a.act);
        } else {
#pragma unroll
          for (int e = 0; e < VE; ++e) dp[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) d[W - 1][e] = dp[e];
        if (t < stop) {
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            db[e] += dp[e];
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][e] += dp[e] * h[j][e];
          }
        }
        const int o = t - (W - 1);
        if (o >= t0) {
          float g[VE];
          const int f = o - (last - (W - 1));  // its row of the final state
          if (a.dht && f >= 0) {
            ldv<T>(g, reinterpret_cast<const T*>(a.dht) + ((int64_t)n * (W - 1) + f) * a.D + c, nv);
          } else {
#pragma unroll
            for (int e = 0; e < VE; ++e) g[e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < VE; ++e)
#pragma unroll
            for (int j = 0; j < W; ++j) g[e] += wt[W - 1 - j][e] * d[j][e];
          stv<T>(dx + (int64_t)o * a.dxs, g, nv);
        }
      }
      t0 = stop;
    }
  }
  // the block's runs, joined in their order
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    float v[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) v[e] = j < W ? dw[j < W ? j : 0][e] : db[e];
    __syncthreads();
    if (wave > 0) {
#pragma unroll
      for (int e = 0; e < VE; ++e) red[wave - 1][e][lane] = v[e];
    }
    __syncthreads();
    if (wave == 0 && nv > 0) {
#pragma unroll
      for (int k = 0; k < CONV_WAVES - 1; ++k)
#pragma unroll
        for (int e = 0; e < VE; ++e) v[e] += red[k][e][lane];
      stv<float>(a.part + ((int64_t)blockIdx.x * (W + 1) + j) * a.D + c, *reinterpret_cast<float(*)[4]>(v), min(nv, 4));
      if constexpr (VE == 8)
        stv<float>(a.part + ((int64_t)blockIdx.x * (W + 1) + j) * a.D + c + 4, *reinterpret_cast<float(*)[4]>(v + 4),
                   min(nv - 4, 4));
    }
  }
}

// dw [D, W] and dbias [D] from the partial sums [tiles, W + 1, D]: 16
// channels a block, 16 groups of tiles, joined in LDS.
template <typename WT, int W>
__global__ __launch_bounds__(256) void k_conv_reduce(ConvArgs a) {
  __shared__ float buf[16][17];
  const int e = threadIdx.x & 15, g = threadIdx.x >> 4, j = blockIdx.y;
  const int c = blockIdx.x * 16 + e;
  float v = 0.f;
  if (c < a.D) {
#pragma unroll 4
    for (int p = g; p < a.tiles; p += 16) v += a.part[((int64_t)p * (W + 1) + j) * a.D + c];
  }
  buf[g][e] = v;
  __syncthreads();
  if (g == 0 && c < a.D) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += buf[i][e];
    if (j < W) reinterpret_cast<WT*>(a.dw)[(int64_t)c * W + j] = (WT)s;
    else if (a.dbias) reinterpret_cast<WT*>(a.dbias)[c] = (WT)s;
  }
}

template <typename F>
hipError_t conv_taps_of(int W, F&& f) {
  switch (W) {
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    case 4: return f(std::integral_constant<int, 4>{});
    default: return hipErrorInvalidValue;
  }
}
int conv_cblocks(int D, bool f32) { return (D + 64 * (f32 ? 4 : 8) - 1) / (64 * (f32 ? 4 : 8)); }

template <typename T, typename WT>
hipError_t conv_fwd_t(const ConvArgs& a, int cb, hipStream_t s) {
  return conv_taps_of(a.W, [&](auto w) {
    const int fin = a.ht ? (a.seq.N + CONV_WAVES - 1) / CONV_WAVES : 0;
    REWY_LAUNCH((k_conv_fwd<T, WT, decltype(w)::value>), dim3(a.tiles + fin, cb), dim3(64 * CONV_WAVES), s, a);
    return hipGetLastError();
  });
}
template <typename T, typename WT>
hipError_t conv_step_t(const ConvArgs& a, int cb, hipStream_t s) {
  return conv_taps_of(a.W, [&](auto w) {
    REWY_LAUNCH((k_conv_step<T, WT, decltype(w)::value>), dim3(a.seq.N, cb), dim3(64), s, a);
    return hipGetLastError();
  });
}
template <typename T, typename WT>
hipError_t conv_bwd_t(const ConvArgs& a, int cb, hipStream_t s) {
  return conv_taps_of(a.W, [&](auto w) {
    constexpr int W = decltype(w)::value;
    const int fin = a.dh0 ? (a.seq.N + CONV_WAVES - 1) / CONV_WAVES : 0;
    if (a.tiles + fin > 0)
      REWY_LAUNCH((k_conv_bwd<T, WT, W>), dim3(a.tiles + fin, cb), dim3(64 * CONV_WAVES), s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    REWY_LAUNCH((k_conv_reduce<WT, W>), dim3((a.D + 15) / 16, W + 1), dim3(256), s, a);
    return hipGetLastError();
  });
}

// Tokens of a run: the longest of 4 .. most whose runs still give each SIMD two
// waves or so; a longer run reads fewer rows twice.
int conv_run(int total, int cb, int most) {
  int run = most;
  while (run > 4 && (int64_t)((total + run - 1) / run) * cb < 2048) run /= 2;
  return run;
}
int conv_tiles(int total, int run) { return (int)(((int64_t)total + (int64_t)run * CONV_WAVES - 1) / ((int64_t)run * CONV_WAVES)); }

}  // namespace

void conv_bwd_shape(int total, int D, bool f32, int& run, int& tiles) {
  run = conv_run(total, conv_cblocks(D, f32), 64);
  tiles = conv_tiles(total, run);
}

hipError_t launch_conv_fwd(ConvArgs a, bool f32, bool wf32, hipStream_t s) {
  const int cb = conv_cblocks(a.D, f32);
  a.run = conv_run(a.seq.total, cb, 32);
  a.tiles = conv_tiles(a.seq.total, a.run);
  if (f32) return wf32 ? conv_fwd_t<float, float>(a, cb, s) : conv_fwd_t<float, bf16>(a, cb, s);
  return wf32 ? conv_fwd_t<bf16, float>(a, cb, s) : conv_fwd_t<bf16, bf16>(a, cb, s);
}
hipError_t launch_conv_step(const ConvArgs& a, bool f32, bool wf32, hipStream_t s) {
  const int cb = conv_cblocks(a.D, f32);
  if (f32) return wf32 ? conv_step_t<float, float>(a, cb, s) : conv_step_t<float, bf16>(a, cb, s);
  return wf32 ? conv_step_t<bf16, float>(a, cb, s) : conv_step_t<bf16, bf16>(a, cb, s);
}
hipError_t launch_conv_bwd(const ConvArgs& a, bool f32, bool wf32, hipStream_t s) {
  const int cb = conv_cblocks(a.D, f32);
  if (f32) return wf32 ? conv_bwd_t<float, float>(a, cb, s) : conv_bwd_t<float, bf16>(a, cb, s);
  return wf32 ? conv_bwd_t<bf16, float>(a, cb, s) : conv_bwd_t<bf16, bf16>(a, cb, s);
}

}  // namespace rewy
