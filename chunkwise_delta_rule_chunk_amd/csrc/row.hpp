// Rows held by a group of threads (the norms): joins over the threads of a row and
// the 8-bit outputs with their scales.
#pragma once
#include "layer.hpp"

namespace rewy {

constexpr int NORM_BLOCK = 256;

// Largest magnitude by its bits: NaN > infinity > every number, so a row that
// holds one keeps it in its scale.
__device__ __forceinline__ uint32_t mag(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
#pragma unroll
  for (int m = 1; m < LANES; m *= 2) x = max(x, (uint32_t)__shfl_xor((int)x, m, 64));
  return x;
}
__device__ __forceinline__ uint32_t lanes_max_n(uint32_t x, int lanes) {
  for (int m = 1; m < lanes; m *= 2) x = max(x, (uint32_t)__shfl_xor((int)x, m, 64));
  return x;
}

// first wave of the thread's row, where a block holds several rows of several waves
template <int TPR>
__device__ __forceinline__ int row_wave() { return TPR < NORM_BLOCK ? threadIdx.x / TPR * (TPR / 64) : 0; }

// Sum (and maximum) over the TPR threads of a row; `buf` holds one word per
// wave of the block and is used once per call site.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* buf) {
  if constexpr (TPR <= 64) {
    return lanes_sum<TPR>(x);
  } else {
    x = lanes_sum<64>(x);
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = x;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) t += buf[row_wave<TPR>() + i];
    return t;
  }
}
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t x, uint32_t* buf) {
  if constexpr (TPR <= 64) {
    return lanes_max<TPR>(x);
  } else {
    x = lanes_max<64>(x);
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = x;
    __syncthreads();
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) t = max(t, buf[row_wave<TPR>() + i]);
    return t;
  }
}

// scale from the largest magnitude's bits: 1 where there is nothing to scale (all zeros,
// or magnitudes so small that a step of the scale would be lost)
__device__ __forceinline__ float make_scale(uint32_t bits, float qmax) {
  const float m = __uint_as_float(bits);
  return m < 0x1p-100f ? 1.f : m / qmax;
}
// four values to four bytes
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  // (a value that rounding left just above the largest stays the largest; NaN stays NaN)
  auto lim = [](float v) { return v > 448.f ? 448.f : v < -448.f ? -448.f : v; };
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(lim(a), lim(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(lim(c), lim(d), r, true);
}
__device__ __forceinline__ uint32_t pack_int8(float a, float b, float c, float d) {
  // NaN (a row whose scale says so) becomes 0
  auto cv = [](float v) { return (uint32_t)(int)fminf(fmaxf(v != v ? 0.f : rintf(v), -127.f), 127.f) & 255u; };
  return cv(a) | cv(b) << 8 | cv(c) << 16 | cv(d) << 24;
}
// v / scale as the product with the scale's inverse and one correction, in three operations
// instead of a division's nine, for scales from 2^-90.  The inverse is rounded correctly, so
// the first guess q is within 1.5 steps and its remainder exact but for half a unit of its
// last place: what is rounded last lies within 2^-22.7 steps of the quotient, which can round
// apart only where v S' - T' S = +-1 .. 4 for the 24 bits S' of the scale and the 25 bits T'
// of the middle between two floats.  Beside the borders between codes, whose T' are
// one of 8 bits +- 1, none of these does: the codes are the division's.  Under 2^-90 the remainder
// falls below the smallest float (and an infinite or NaN scale has no such inverse).
struct ScaleDiv {
  float inv, s;
  __device__ __forceinline__ explicit ScaleDiv(float scale) : inv(1.f / scale), s(scale) {}
  static __device__ __forceinline__ bool holds(float scale) { return scale >= 0x1p-90f && scale <= 3.4028235e38f; }
  __device__ __forceinline__ float operator()(float v) const {
    const float q = v * inv;
    return fmaf(fmaf(-q, s, v), inv, q);
  }
};

// One vector's codes of v / scale, of which the first n exist.
template <int VE, typename DIV>
__device__ __forceinline__ void store_codes_by(uint8_t* q, const float (&s)[VE], DIV&& div, bool e4m3, int n) {
  uint32_t b[VE / 4];
#pragma unroll
  for (int k = 0; k < VE / 4; ++k) {
    const float v[4] = {div(s[4 * k]), div(s[4 * k + 1]), div(s[4 * k + 2]), div(s[4 * k + 3])};
    b[k] = e4m3 ? pack_e4m3(v[0], v[1], v[2], v[3]) : pack_int8(v[0], v[1], v[2], v[3]);
  }
  if (n >= VE) {
    typedef uint32_t words __attribute__((ext_vector_type(VE / 4)));
    typedef words words_u __attribute__((aligned(1)));
    if constexpr (VE == 8) {
      *reinterpret_cast<words_u*>(q) = words{b[0], b[1]};
    } else {
      typedef uint32_t word_u __attribute__((aligned(1)));
      *reinterpret_cast<word_u*>(q) = b[0];
    }
  } else {
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (e < n) q[e] = (uint8_t)(b[e / 4] >> (8 * (e & 3)));
  }
}

// (divided: a product with a rounded inverse alone takes the neighbouring code beside a
// tie; no slower for 8192 x 4096 bf16, 33 instead of 30.5 us for 10007 x 1537 fp32)
template <int VE>
__device__ __forceinline__ void store_codes(uint8_t* q, const float (&s)[VE], float scale, bool e4m3, int n) {
  store_codes_by<VE>(q, s, [scale](float v) { return v / scale; }, e4m3, n);
}

}  // namespace rewy
