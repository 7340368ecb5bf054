// The operators around the token mixer (RMS norm with the residual's addition,
// short causal convolution, selective state space scan): argument records,
// launchers and device helpers shared by their kernels.
#pragma once
#include <algorithm>

#include "kernels.hpp"
#include "rewy.h"

namespace rewy {

// ---- vectors at any element alignment ---------------------------------------
// Global memory takes 16-byte accesses at any address aligned to the element
// (gfx950 in its unaligned access mode, the mode of HSA queues), so rows of an
// odd length or stride take the same wide accesses as aligned ones and only a
// row's last, partial vector is read element by element.
template <typename T, int N>
struct VecN {
  typedef T raw __attribute__((ext_vector_type(N)));
  typedef raw type __attribute__((aligned(sizeof(T))));
};
template <typename T>
struct Vec {
  static constexpr int VE = 16 / (int)sizeof(T);
};

// p[0 .. VE) as fp32, of which the first n exist (the others are zero), in loads of at
// most 16 bytes
template <typename T, int VE>
__device__ __forceinline__ void ldv(float (&f)[VE], const T* p, int n) {
  constexpr int N = VE < Vec<T>::VE ? VE : Vec<T>::VE;
  if (n >= VE) {
#pragma unroll
    for (int j = 0; j < VE; j += N) {
      const typename VecN<T, N>::raw v = *reinterpret_cast<const typename VecN<T, N>::type*>(p + j);
#pragma unroll
      for (int e = 0; e < N; ++e) f[j + e] = (float)v[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < VE; ++e) f[e] = e < n ? (float)p[e] : 0.f;
  }
}
template <typename T, int VE>
__device__ __forceinline__ void stv(T* p, const float (&f)[VE], int n) {
  constexpr int N = VE < Vec<T>::VE ? VE : Vec<T>::VE;
  if (n >= VE) {
#pragma unroll
    for (int j = 0; j < VE; j += N) {
      typename VecN<T, N>::raw v;
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = (T)f[j + e];
      *reinterpret_cast<typename VecN<T, N>::type*>(p + j) = v;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (e < n) p[e] = (T)f[e];
  }
}

// Sum over groups of LANES lanes (a power of two up to 64), in every lane.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
  static_assert(LANES == 16 || LANES == 64, "");
  x = row16_sum(x);
  return LANES == 64 ? rows_sum(x) : x;
}

// Workgroup b of n in an order that gives each XCD (workgroups go to the 8 XCDs
// in turn) one contiguous range, so that neighbours, which share operands, share an L2.
__device__ __forceinline__ int xcd_range(int b, int n) {
  const int x = b & 7, per = n >> 3, rem = n & 7;
  return x * per + min(x, rem) + (b >> 3);
}

// ---- RMS norm -----------------------------------------------------------------
struct NormArgs {
  int64_t M;
  int D;
  int quant, group;
  float eps;
  int64_t xs, rs, ss, ys;  // row strides of x, res, sum, y (backward: s, ds, dx, dy)
  const void* x;           // backward: s
  const void* res;         // backward: ds
  const void* w;
  const void* dy;
  void* sum;               // backward: dx
  void* y;
  void* q;
  float* scale;
  float* rstd;             // written by the forward, read by the backward
  void* dw;
  float* part;             // [nblk, D] partial sums of dw
  int nblk;
  int ng;                  // scales per row
};
// blocks of the backward, and so rows of its partial sums
int norm_bwd_blocks(int64_t M, int D, bool f32);
hipError_t launch_norm_fwd(const NormArgs& a, bool f32, bool wf32, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, bool f32, bool wf32, hipStream_t s);
// out[j] (bf16 or fp32) = sum over p < np of part[p * ld + j], j < n, in a fixed order; with
// a split, columns from there on go to out2 (either may be nullptr: not written)
hipError_t launch_colsum(const float* part, int np, int64_t ld, int64_t n, void* out, bool out_f32,
                         hipStream_t s, void* out2 = nullptr, int64_t split = -1);

// ---- sequences ------------------------------------------------------------------
// First token of sequence n (n = N: the end of the last one): from the device
// cu_seqlens, clamped to the packed token axis, or n T.  The first sequence
// starts at 0.  Rows at or behind start(N) belong to no sequence.
struct SeqArgs {
  const int* cu;
  int N, T;    // T tokens per sequence without cu
  int total;   // packed tokens
};
__device__ __forceinline__ int seq_start(const SeqArgs& q, int n) {
  return q.cu ? (n == 0 ? 0 : min(max(q.cu[n], 0), q.total)) : n * q.T;
}
// [bos, eos) of sequence n; a decreasing cu_seqlens gives an empty sequence
__device__ __forceinline__ void seq_range(const SeqArgs& q, int n, int& bos, int& eos) {
  bos = seq_start(q, n);
  eos = max(seq_start(q, n + 1), bos);
}

// ---- short convolution ------------------------------------------------------------
struct ConvArgs {
  SeqArgs seq;
  int D, W, act;
  int64_t xs, ys, dxs;  // token strides of x, y (backward: dy) and dx
  const void* x;
  const void* w;        // [D, W]
  const void* bias;     // [D] or nullptr
  const void* h0;       // [N, W-1, D] or nullptr
  void* y;
  void* ht;
  const void* dy;
  const void* dht;
  void* dx;
  void* dh0;
  float* part;          // [tiles, W + 1, D] partial sums of dw (tap by tap) and dbias
  void* dw;
  void* dbias;
  int run;              // tokens of one wave's run
  int tiles;            // runs
  int cblocks;          // waves along the channels
  int full;             // no lane has a partial vector (k_conv.hip)
};
// waves along the channels; tokens of one wave's run, and runs, of the backward
int conv_cblocks(int D);
void conv_bwd_shape(int total, int D, int& run, int& tiles);
hipError_t launch_conv_fwd(ConvArgs a, bool f32, bool wf32, hipStream_t s);
hipError_t launch_conv_step(const ConvArgs& a, bool f32, bool wf32, hipStream_t s);
hipError_t launch_conv_bwd(ConvArgs a, bool f32, bool wf32, hipStream_t s);
hipError_t launch_conv_reduce(const ConvArgs& a, bool wf32, hipStream_t s);

}  // namespace rewy
