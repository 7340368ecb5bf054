// Short causal convolution along the tokens, channel by channel, with an
// optional bias and SiLU:
//   pre_t = bias + sum_{j < W} w_j x_{t - (W-1) + j},   y_t = act(pre_t),
// where the W - 1 rows before a sequence's first token are its initial state
// (zeros without one) and the final state is the last W - 1 rows of
// [initial state ; x].  Backward, with dpre_t = dy_t act'(pre_t):
//   dx_t = sum_{o < W} w_{W-1-o} dpre_{t+o} (+ the final state's adjoint on the
//   last W - 1 rows),   dw_j = sum_t dpre_t x_{t-(W-1)+j},   dbias = sum_t dpre_t.
//
// Memory is all it costs.  A lane owns four channels and walks a run
// of tokens with the last W - 1 rows in registers, so each row is read once
// per run plus W - 1 rows at its start.  Workgroups that follow each other share
// their tokens, so whole rows are streamed.  Tokens are packed; a run that meets
// the end of a sequence takes up the next one's state.
#include "layer.hpp"

namespace rewy {

namespace {

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

// Channels of a lane: four, in either type.  With 16 bytes of bf16 (eight) fewer waves
// fit and fewer rows are in flight: 34 instead of 30 us for 8192 x 4352.
constexpr int VE = 4;

// Row p of sequence n counted from its first token; p < 0 reads the initial state.
template <typename T, int W>
__device__ __forceinline__ void conv_row(float (&f)[VE], const ConvArgs& a, int n, int bos, int p, int c, int nv) {
  if (p >= 0) {
    ldv<T, VE>(f, reinterpret_cast<const T*>(a.x) + (int64_t)(bos + p) * a.xs + c, nv);
  } else if (a.h0) {
    ldv<T, VE>(f, reinterpret_cast<const T*>(a.h0) + ((int64_t)n * (W - 1) + (W - 1) + p) * a.D + c, nv);
  } else {
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = 0.f;
  }
}

// taps as wt[j][e] for channels c .. c + VE - 1
template <typename WT, int W>
__device__ __forceinline__ void conv_taps(float (&wt)[W][VE], float (&b)[VE], const ConvArgs& a, int c, int nv) {
  const WT* w = reinterpret_cast<const WT*>(a.w) + (int64_t)c * W;
  float f[VE * W];
#pragma unroll
  for (int k = 0; k < VE * W; k += 4) {
    float g[4];
    ldv<WT, 4>(g, w + k, nv * W - k);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[k + e] = g[e];
  }
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    b[e] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) wt[j][e] = f[e * W + j];
  }
  if (a.bias) ldv<WT, VE>(b, reinterpret_cast<const WT*>(a.bias) + c, nv);
}

// Final state of sequence n (grid rows past the token tiles).
template <typename T, int W>
__device__ __forceinline__ void conv_final(const ConvArgs& a, int n, int c, int nv) {
  int bos, eos;
  seq_range(a.seq, n, bos, eos);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    float f[VE];
    conv_row<T, W>(f, a, n, bos, eos - bos - (W - 1) + k, c, nv);
    stv<T, VE>(reinterpret_cast<T*>(a.ht) + ((int64_t)n * (W - 1) + k) * a.D + c, f, nv);
  }
}

// A row's VE channels on their way from memory.  FULL (every lane's channels exist
// and rows keep 4-byte alignment): one unconditional load, kept in the operand type,
// and stores through a buffer resource, whose range check drops the rows past the
// run.  The compiler can then count the requests in flight (one counter serves
// loads and stores) and a row's use waits for that row alone; with loads and stores
// in branches, as other channel numbers and alignments take them, it waits for all of
// them (8192 x 4352: 28 us, x 4354: 46, x 4351, whose vectors are also unaligned: 60;
// backward of 32768 x 2304: 111 us, x 2306: 243).
template <typename T, bool FULL>
struct Row {
  typename VecN<T, VE>::raw v;
  float f[FULL ? 1 : VE];
  __device__ __forceinline__ void load(const T* p, int nv) {
    if constexpr (FULL) v = *reinterpret_cast<const typename VecN<T, VE>::type*>(p);
    else ldv<T, VE>(f, p, nv);
  }
  __device__ __forceinline__ void get(float (&o)[VE]) const {
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      if constexpr (FULL) o[e] = (float)v[e];
      else o[e] = f[e];
    }
  }
};
template <typename T, bool FULL>
__device__ __forceinline__ void put_row(const GBuf& g, T* p, int row, int64_t stride, int c, bool on,
                                        const float (&o)[VE], int nv) {
  if constexpr (FULL) {
    typename VecN<T, VE>::raw v;
#pragma unroll
    for (int e = 0; e < VE; ++e) v[e] = (T)o[e];
    const uint32_t off = on ? (uint32_t)(row * (int)stride + c) * (uint32_t)sizeof(T) : OOB;
    if constexpr (sizeof(T) == 4) gst16(g, off, __builtin_bit_cast(uint4, v));
    else gst8(g, off, __builtin_bit_cast(uint2, v));
  } else {
    if (on) stv<T, VE>(p + row * stride + c, o, nv);
  }
}
// values loaded in front of a loop: waited for here, so that the loop's uses need not
__device__ __forceinline__ void settle(float (&f)[VE]) {
#pragma unroll
  for (int e = 0; e < VE; ++e) asm volatile("" : "+v"(f[e]));
}
// tokens worked on side by side: a multiple of W, so that the ring of the last W rows
// turns at compile time
constexpr int conv_group(int W) { return W == 3 ? 6 : 8; }

// The rows of the next U tokens are in flight while one is worked on.  Bound by HBM:
// 8192 x 4352 bf16, W = 4: 143 MB in 28.2 us (5.1 TB/s); runs of 32 tokens, so that 3
// of 35 rows are read twice, out of a cache.
template <typename T, typename WT, int W, bool FULL>
__global__ __launch_bounds__(64) void k_conv_fwd(ConvArgs a) {
  constexpr int U = conv_group(W);
  const int cb = blockIdx.x % a.cblocks, tile = blockIdx.x / a.cblocks;
  const int c = (cb * 64 + threadIdx.x) * VE, nv = a.D - c;
  if (nv <= 0) return;
  if (tile >= a.tiles) {  // a sequence's final state
    conv_final<T, W>(a, tile - a.tiles, c, nv);
    return;
  }
  const int64_t first = (int64_t)tile * a.run;
  const int total = seq_start(a.seq, a.seq.N);  // rows behind the last sequence stay as they are
  if (first >= total) return;
  int t0 = (int)first;
  const int end = min(t0 + a.run, total);
  int n = seq_of(a.seq, t0), bos, eos;
  seq_range(a.seq, n, bos, eos);
  float wt[W][VE], b[VE];
  conv_taps<WT, W>(wt, b, a, c, nv);
  const T* x = reinterpret_cast<const T*>(a.x) + c;
  T* y = reinterpret_cast<T*>(a.y) + first * a.ys;
  const GBuf gy = gbuf(y, tile_bytes<T>(end - (int)first, a.ys, a.D));
  while (t0 < end) {
    while (eos <= t0 && n + 1 < a.seq.N) seq_range(a.seq, ++n, bos, eos);  // (passes over empty ones)
    const int stop = eos > t0 ? min(end, eos) : end;
    Row<T, FULL> in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) in[u].load(x + (int64_t)min(t0 + u, stop - 1) * a.xs, nv);
    float h[W][VE];  // token t0 + u is in h[u % W]
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      conv_row<T, W>(h[k + 1], a, n, bos, t0 - bos - (W - 1) + k, c, nv);
      settle(h[k + 1]);
    }
    for (int t = t0; t < stop; t += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        in[u].get(h[u % W]);
        in[u].load(x + (int64_t)min(t + u + U, stop - 1) * a.xs, nv);
        float o[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          float p = b[e];
#pragma unroll
          for (int j = 0; j < W; ++j) p += wt[j][e] * h[(u + 1 + j) % W][e];
          o[e] = a.act == REWY_ACT_SILU ? silu(p) : p;
        }
        put_row<T, FULL>(gy, y, t + u - (int)first, a.ys, c, t + u < stop, o, nv);
      }
    }
    t0 = stop;
  }
}

// One token per sequence; every state row is read before any is written, by
// the same lane, so the state may be updated in place.  64 x 4352: 4.4 us, one trip to
// memory and back.
template <typename T, typename WT, int W>
__global__ __launch_bounds__(64) void k_conv_step(ConvArgs a) {
  const int c = (blockIdx.y * 64 + threadIdx.x) * VE, nv = a.D - c, n = blockIdx.x;
  if (nv <= 0) return;
  float h[W][VE], wt[W][VE], b[VE];
#pragma unroll
  for (int k = 0; k < W; ++k) conv_row<T, W>(h[k], a, n, n, k - (W - 1), c, nv);
  conv_taps<WT, W>(wt, b, a, c, nv);
  float o[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    float p = b[e];
#pragma unroll
    for (int j = 0; j < W; ++j) p += wt[j][e] * h[j][e];
    o[e] = a.act == REWY_ACT_SILU ? silu(p) : p;
  }
  stv<T, VE>(reinterpret_cast<T*>(a.y) + (int64_t)n * a.ys + c, o, nv);
  if (a.ht) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      stv<T, VE>(reinterpret_cast<T*>(a.ht) + ((int64_t)n * (W - 1) + k) * a.D + c, h[k + 1], nv);
  }
}

// dp (dy of a row) becomes dy act'(pre); pre = the row before the activation
__device__ __forceinline__ void conv_dpre(float (&dp)[VE], const float (&pre)[VE], int act) {
  if (act != REWY_ACT_SILU) return;
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    const float s = sigmoid_f(pre[e]);
    dp[e] *= s * (1.f + pre[e] * (1.f - s));
  }
}

// Initial state's adjoint of sequence n: row k takes dpre_t of the tokens
// t <= k through tap k - t, and the final state's adjoint where the sequence
// is shorter than the state.
template <typename T, typename WT, int W>
__device__ __forceinline__ void conv_dh0(const ConvArgs& a, int n, int c, int nv) {
  int bos, eos;
  seq_range(a.seq, n, bos, eos);
  const int L = eos - bos;
  float wt[W][VE], b[VE], g[W - 1][VE];
  conv_taps<WT, W>(wt, b, a, c, nv);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
#pragma unroll
    for (int e = 0; e < VE; ++e) g[k][e] = 0.f;
    const int f = k - L;  // row of the final state that this row is
    if (a.dht && f >= 0) ldv<T, VE>(g[k], reinterpret_cast<const T*>(a.dht) + ((int64_t)n * (W - 1) + f) * a.D + c, nv);
  }
#pragma unroll
  for (int t = 0; t < W - 1; ++t) {
    if (t >= L) break;
    float pre[VE], dp[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) pre[e] = b[e];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float h[VE];
      conv_row<T, W>(h, a, n, bos, t - (W - 1) + j, c, nv);
#pragma unroll
      for (int e = 0; e < VE; ++e) pre[e] += wt[j][e] * h[e];
    }
    ldv<T, VE>(dp, reinterpret_cast<const T*>(a.dy) + (int64_t)(bos + t) * a.ys + c, nv);
    conv_dpre(dp, pre, a.act);
#pragma unroll
    for (int k = t; k < W - 1; ++k)
#pragma unroll
      for (int e = 0; e < VE; ++e) g[k][e] += wt[k - t][e] * dp[e];
  }
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    stv<T, VE>(reinterpret_cast<T*>(a.dh0) + ((int64_t)n * (W - 1) + k) * a.D + c, g[k], nv);
}

// A run's part of each sequence it meets: tokens enter one by one (the rows of the next
// U in flight); a token's dpre meets the W rows that it reached, and a row leaves
// when the W - 1 tokens behind it have entered.  One pass: the convolution is formed
// again from x, so x, dy and dx pass memory once.  32768 x 2304 bf16 in 16 sequences:
// 453 MB, 500 with the partial sums and the runs' shared rows, in 113 us (4.4 TB/s;
// the forward of the same rows 62 us, 5.1 TB/s).
template <typename T, typename WT, int W, bool FULL>
__global__ __launch_bounds__(64) void k_conv_bwd(ConvArgs a) {
  constexpr int U = W == 3 ? 3 : 4;  // (more do not fit beside the windows and sums)
  const int cb = blockIdx.x % a.cblocks, tile = blockIdx.x / a.cblocks;
  const int c = (cb * 64 + threadIdx.x) * VE, nv = a.D - c;
  if (nv <= 0) return;
  if (tile >= a.tiles) {  // a sequence's initial state
    conv_dh0<T, WT, W>(a, tile - a.tiles, c, nv);
    return;
  }
  float wt[W][VE], b[VE], dw[W][VE], db[VE];
  conv_taps<WT, W>(wt, b, a, c, nv);
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
  }
  const int64_t first = (int64_t)tile * a.run;
  const int total = seq_start(a.seq, a.seq.N);  // rows behind the last sequence stay as they are
  if (first < total) {
    int t0 = (int)first;
    const int end = min(t0 + a.run, total);
    int n = seq_of(a.seq, t0), bos, eos;
    seq_range(a.seq, n, bos, eos);
    const T* x = reinterpret_cast<const T*>(a.x) + c;
    const T* dy = reinterpret_cast<const T*>(a.dy) + c;
    T* dx = reinterpret_cast<T*>(a.dx) + first * a.dxs;
    const GBuf gx = gbuf(dx, tile_bytes<T>(end - (int)first, a.dxs, a.D));
    while (t0 < end) {
      while (eos <= t0 && n + 1 < a.seq.N) seq_range(a.seq, ++n, bos, eos);
      // this run's tokens of the sequence: [t0, stop); the tokens that reach them: [t0, last)
      const int stop = eos > t0 ? min(end, eos) : end, eoq = max(eos, stop), last = min(stop + W - 1, eoq);
      Row<T, FULL> xin[U], din[U];
      auto fetch = [&](int u, int t) {
        const int64_t tt = min(t, last - 1);
        xin[u].load(x + tt * a.xs, nv);
        din[u].load(dy + tt * a.ys, nv);
      };
#pragma unroll
      for (int u = 0; u < U; ++u) fetch(u, t0 + u);
      float h[W][VE], d[W][VE];  // token t0 + u and its dpre are in h[u % W], d[u % W]
#pragma unroll
      for (int k = 0; k < W - 1; ++k) {
        conv_row<T, W>(h[k + 1], a, n, bos, t0 - bos - (W - 1) + k, c, nv);
        settle(h[k + 1]);
#pragma unroll
        for (int e = 0; e < VE; ++e) d[k + 1][e] = 0.f;
      }
      for (int t = t0; t < stop + W - 1; t += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float(&hn)[VE] = h[u % W];
          float(&dn)[VE] = d[u % W];
          xin[u].get(hn);
          din[u].get(dn);
          fetch(u, t + u + U);
          float pre[VE];
          const float live = t + u < last ? 1.f : 0.f, own = t + u < stop ? 1.f : 0.f;
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            pre[e] = b[e];
#pragma unroll
            for (int j = 0; j < W; ++j) pre[e] += wt[j][e] * h[(u + 1 + j) % W][e];
          }
          conv_dpre(dn, pre, a.act);
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            dn[e] = live != 0.f ? dn[e] : 0.f;
            const float m = own != 0.f ? dn[e] : 0.f;
            db[e] += m;
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][e] += m * h[(u + 1 + j) % W][e];
          }
          const int o = t + u - (W - 1);  // the row that leaves
          float g[VE];
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            g[e] = 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) g[e] += wt[W - 1 - j][e] * d[(u + 1 + j) % W][e];
          }
          const int f = o - (eoq - (W - 1));  // its row of the final state
          if (a.dht && f >= 0 && o < stop && o >= t0) {
            float q[VE];
            ldv<T, VE>(q, reinterpret_cast<const T*>(a.dht) + ((int64_t)n * (W - 1) + f) * a.D + c, nv);
            settle(q);
#pragma unroll
            for (int e = 0; e < VE; ++e) g[e] += q[e];
          }
          put_row<T, FULL>(gx, dx, o - (int)first, a.dxs, c, o >= t0 && o < stop, g, nv);
        }
      }
      t0 = stop;
    }
  }
#pragma unroll
  for (int j = 0; j <= W; ++j)
    stv<float, VE>(a.part + ((int64_t)tile * (W + 1) + j) * a.D + c, j < W ? dw[j < W ? j : 0] : db, nv);
}

// dw [D, W] and dbias [D] from the partial sums [tiles, W + 1, D]: 16
// channels a block, 16 groups of tiles, joined in LDS (512 tiles of 2304: 8.6 us).
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

template <typename T, typename WT>
hipError_t conv_fwd_t(const ConvArgs& a, hipStream_t s) {
  return conv_taps_of(a.W, [&](auto w) {
    const int fin = a.ht ? a.seq.N : 0;
    const dim3 grid((a.tiles + fin) * a.cblocks), block(64);
    if (a.full) REWY_LAUNCH((k_conv_fwd<T, WT, decltype(w)::value, true>), grid, block, s, a);
    else REWY_LAUNCH((k_conv_fwd<T, WT, decltype(w)::value, false>), grid, block, s, a);
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
hipError_t conv_bwd_t(const ConvArgs& a, hipStream_t s) {
  return conv_taps_of(a.W, [&](auto w) {
    constexpr int W = decltype(w)::value;
    const int fin = a.dh0 ? a.seq.N : 0;
    const dim3 grid((a.tiles + fin) * a.cblocks), block(64);
    if (a.full) REWY_LAUNCH((k_conv_bwd<T, WT, W, true>), grid, block, s, a);
    else REWY_LAUNCH((k_conv_bwd<T, WT, W, false>), grid, block, s, a);
    return hipGetLastError();
  });
}
template <typename WT>
hipError_t conv_reduce_t(const ConvArgs& a, hipStream_t s) {
  return conv_taps_of(a.W, [&](auto w) {
    constexpr int W = decltype(w)::value;
    REWY_LAUNCH((k_conv_reduce<WT, W>), dim3((a.D + 15) / 16, W + 1), dim3(256), s, a);
    return hipGetLastError();
  });
}

// Tokens of a run: the longest of 4 .. most whose runs still give each SIMD two
// waves or so; a longer run reads fewer rows twice.
int conv_run(int total, int cw, int most) {
  int run = most;
  while (run > 4 && (int64_t)((total + run - 1) / run) * cw < 2048) run /= 2;
  return run;
}
int conv_tiles(int total, int run) { return (int)(((int64_t)total + run - 1) / run); }

}  // namespace

// waves (workgroups) along the channels
int conv_cblocks(int D) { return (D + 64 * VE - 1) / (64 * VE); }

void conv_bwd_shape(int total, int D, int& run, int& tiles) {
  run = conv_run(total, conv_cblocks(D), 64);
  tiles = conv_tiles(total, run);
}

namespace {
// whether every lane's channels exist and the rows that are written keep 4-byte alignment
// (and their offsets within a run 32 bits)
bool conv_full(const ConvArgs& a, size_t e, const void* out, int64_t stride) {
  return a.D % VE == 0 && (uintptr_t)out % 4 == 0 && stride * e % 4 == 0 && stride <= (1 << 22);
}
}  // namespace

hipError_t launch_conv_fwd(ConvArgs a, bool f32, bool wf32, hipStream_t s) {
  const int cw = conv_cblocks(a.D);
  a.run = conv_run(a.seq.total, cw, 32);
  a.tiles = conv_tiles(a.seq.total, a.run);
  a.cblocks = cw;
  a.full = conv_full(a, f32 ? 4 : 2, a.y, a.ys);
  if (f32) return wf32 ? conv_fwd_t<float, float>(a, s) : conv_fwd_t<float, bf16>(a, s);
  return wf32 ? conv_fwd_t<bf16, float>(a, s) : conv_fwd_t<bf16, bf16>(a, s);
}
hipError_t launch_conv_step(const ConvArgs& a, bool f32, bool wf32, hipStream_t s) {
  const int cb = conv_cblocks(a.D);
  if (f32) return wf32 ? conv_step_t<float, float>(a, cb, s) : conv_step_t<float, bf16>(a, cb, s);
  return wf32 ? conv_step_t<bf16, float>(a, cb, s) : conv_step_t<bf16, bf16>(a, cb, s);
}
hipError_t launch_conv_bwd(ConvArgs a, bool f32, bool wf32, hipStream_t s) {
  a.cblocks = conv_cblocks(a.D);
  a.full = conv_full(a, f32 ? 4 : 2, a.dx, a.dxs);
  if (f32) return wf32 ? conv_bwd_t<float, float>(a, s) : conv_bwd_t<float, bf16>(a, s);
  return wf32 ? conv_bwd_t<bf16, float>(a, s) : conv_bwd_t<bf16, bf16>(a, s);
}
hipError_t launch_conv_reduce(const ConvArgs& a, bool wf32, hipStream_t s) {
  return wf32 ? conv_reduce_t<float>(a, s) : conv_reduce_t<bf16>(a, s);
}

}  // namespace rewy
