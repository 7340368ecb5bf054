// y[m, n] = sum_b sa[m, b] sw[n, b] (sum_{k in b} a[m, k] w[n, k]) + bias[n], with a and w
// in e4m3, blocks b of 128 along k and sw given for 128 rows of w or for each.
//
// Products of two codes are exact, a block's sum starts from zero and meets the two scales
// in fp32 once: acc += p (sa sw).  w is the first operand, so a lane holds four
// neighbouring columns of one row of y.
//
// A block is as long as one v_mfma_f32_16x16x128_f8f6f4.  The 8-bit matrix instructions
// line up neighbouring products before they are added and drop what lies 13 bits under
// the largest: for normally distributed codes a block's sum is off by 1.5e-5 in norm (5e-5
// where all codes are equally frequent), the same for the 32-long instruction.  A 16-bit y
// does not show that (its rounding is 1.7e-3), a 32-bit y would: it takes bf16 matrix
// instructions on the widened codes (exact; 1e-8), at half the rate.  Where w is read
// once for few rows nothing is bound by the matrix unit, and both take the wide form.
#include "mm8.hpp"

namespace rewy {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// 16 x 16 x 128: rows of w, columns (rows of a); lane l gives row l & 15, and any
// assignment of k to the lanes' bytes serves that is the same for both
__device__ __forceinline__ f32x4 mma8(i32x8 w, i32x8 a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, zero4(), 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ i32x8 join16(uint4 x, uint4 y) {
  return i32x8{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
}
// eight codes as bf16
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// a lane's 32 codes of a block
struct Wide32 {
  bf16x8 v[4];
  __device__ __forceinline__ Wide32(uint4 x, uint4 y) : v{widen8(x.x, x.y), widen8(x.z, x.w), widen8(y.x, y.y), widen8(y.z, y.w)} {}
};
__device__ __forceinline__ f32x4 mma_wide(const Wide32& w, const Wide32& a) {
  f32x4 p = zero4();
#pragma unroll
  for (int q = 0; q < 4; ++q) p = mma(w.v[q], a.v[q], p);
  return p;
}
__device__ __forceinline__ float ld_bias(const Mm8Args& a, int n) { return a.bias ? ld_beta(a.bias, a.bias_f32, n) : 0.f; }

// four neighbouring columns n .. of a row, as far as they exist
template <typename O>
__device__ __forceinline__ void store4(const Mm8Args& a, int m, int n, const f32x4& v) {
  O* p = reinterpret_cast<O*>(a.y) + m * a.ys + n;
  if (n + 4 <= a.N) {
    typename VecN<O, 4>::raw o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (O)v[i];
    *reinterpret_cast<typename VecN<O, 4>::type*>(p) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.N) p[i] = (O)v[i];
  }
}

// Few rows: w is read once, straight into the operands' registers.  A workgroup takes
// 16 rows of w and 16 MT rows of a, its eight waves every eighth block, joined
// through LDS in their order.
template <typename O, int MT>
__global__ __launch_bounds__(512) void k_mm8_rows(Mm8Args a) {
  __shared__ float part[8][MT][4][64];
  const int w = wave_id(), l = lane_id(), r = l & 15, g = l >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MT;
  const GBuf gw = gbuf(a.w + n0 * a.ws, (uint32_t)((min(16, a.N - n0) - 1) * a.ws + a.K));
  const GBuf ga = gbuf(a.a + m0 * a.as, (uint32_t)((min(16 * MT, a.M - m0) - 1) * a.as + a.K));
  const uint32_t wo = (uint32_t)(r * a.ws) + 32 * g, ao = (uint32_t)(r * a.as) + 32 * g;
  const float* swp[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = min(n0 + 4 * g + i, a.N - 1);
    swp[i] = a.sw + (int64_t)(a.wrow ? n : n / 128) * a.nb;
  }
  const float* sap[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) sap[t] = a.sa + (int64_t)min(m0 + 16 * t + r, a.M - 1) * (a.ablk ? a.nb : 1);
  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = zero4();
#pragma unroll 2
  for (int kb = w; kb < a.nb; kb += 8) {
    const int k = kb * 128 + 32 * g;
    auto at = [&](uint32_t o, int h) { return k + h < a.K ? o + kb * 128 + h : OOB; };  // (past a row's end: zeros)
    const Wide32 wf(gld16(gw, at(wo, 0)), gld16(gw, at(wo, 16)));
    f32x4 sw;
#pragma unroll
    for (int i = 0; i < 4; ++i) sw[i] = swp[i][kb];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint32_t o = ao + (uint32_t)(16 * t * a.as);
      const Wide32 af(gld16(ga, at(o, 0)), gld16(ga, at(o, 16)));
      const float sa = sap[t][a.ablk ? kb : 0];
      const f32x4 p = mma_wide(wf, af);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] += p[i] * (sa * sw[i]);
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[w][t][i][l] = acc[t][i];
  __syncthreads();
  // wave t joins tile t
#pragma unroll
  for (int t0 = 0; t0 < MT; t0 += 8) {
    const int t = t0 + w, m = m0 + 16 * t + r, n = n0 + 4 * g;
    if (t >= MT || m >= a.M) continue;
    f32x4 s = zero4();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int q = 0; q < 8; ++q) s[i] += part[q][t][i][l];
      if (n + i < a.N) s[i] += ld_bias(a, n + i);
    }
    store4<O>(a, m, n, s);
  }
}

// Wait until at most N of the wave's vector memory operations are in flight.
template <int N>
__device__ __forceinline__ void wait_vm() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

// 64 lanes' 16 bytes straight to LDS, lane l's at address dst + 16 l (dst the same in the
// whole wave); bytes outside the buffer arrive as zeros.  The compiler does not count these:
// wait_vm before the barrier behind which they are read.
__device__ __forceinline__ void load_lds16(u32x4 b, uint32_t off, uint32_t dst) {
  dst = __builtin_amdgcn_readfirstlane(dst);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(dst), "v"(off), "s"(b) : "memory");
}
// gbuf's resource as its four words
__device__ __forceinline__ u32x4 buf_words(const void* base, uint32_t bytes) {
  const uint64_t p = (uint64_t)base;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(p >> 32) & 0xffffu)),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}

// A wave's tiles, from row m0 of a and row n0 of w, with the bias
template <typename O, int TM, int TN>
__device__ __forceinline__ void store_tile(const Mm8Args& a, const f32x4 (&acc)[TM][TN], int m0, int n0) {
  const int r = lane_id() & 15, g = lane_id() >> 4;
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int n = n0 + 16 * j + 4 * g;
    f32x4 b = zero4();
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < a.N) b[e] = ld_bias(a, n + e);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int m = m0 + 16 * i + r;
      if (m < a.M && n < a.N) store4<O>(a, m, n, acc[i][j] + b);
    }
  }
}

// First rows of a workgroup's tile: the workgroups go to the XCDs in turn, each of which
// takes a contiguous range, eight tiles of rows by as many of columns as are at work at
// once.
template <int BM, int BN>
__device__ __forceinline__ void tile_origin(const Mm8Args& a, int& m0, int& n0) {
  const int nm = (a.M + BM - 1) / BM, nn = (a.N + BN - 1) / BN, id = xcd_range(blockIdx.x, nm * nn);
  const int grp = id / (8 * nn), gm = min(8, nm - 8 * grp), in = id - grp * 8 * nn;
  m0 = (8 * grp + in % gm) * BM;
  n0 = in / gm * BN;
}
// Thread t's scales of each block: row t of [a's rows ; w's rows] of a tile
template <int BM, int BN, int NTH, bool WROW>
struct TileScales {
  static constexpr int N = (BM + BN + NTH - 1) / NTH;
  const float* p[N];
  int step[N];
  float v[N];
  __device__ __forceinline__ TileScales(const Mm8Args& a, int m0, int n0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = threadIdx.x + i * NTH, n = min(n0 + max(t - BM, 0), a.N - 1);
      p[i] = t < BM ? a.sa + (int64_t)min(m0 + t, a.M - 1) * (a.ablk ? a.nb : 1) : a.sw + (int64_t)(WROW ? n : n / 128) * a.nb;
      step[i] = t < BM ? a.ablk : 1;
    }
  }
  __device__ __forceinline__ void load(int kb) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = p[i][kb * step[i]];
  }
  __device__ __forceinline__ void store(float* s) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = threadIdx.x + i * NTH;
      if (N * NTH == BM + BN || t < BM + BN) s[t] = v[i];
    }
  }
};

// Tiles of BM rows of a by BN rows of w, WM x WN waves; two blocks of 128 in LDS, the
// next one on its way while one is used.  A row's eight pieces of 16 bytes lie in LDS at
// their place xor the row's last three bits, so that sixteen lanes that read one piece
// of sixteen rows meet the banks evenly.
template <typename O, int BM, int BN, int WM, int WN, bool WROW>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_mm8_tile(Mm8Args a) {
  constexpr int NTH = 64 * WM * WN, NW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16, P = (BM + BN) / 8 / NW;
  static_assert((BM + BN) % (8 * NW) == 0 && BM % (8 * P) == 0, "a wave's pieces are rows of one operand");
  static_assert(WROW || BN / WN <= 128, "a wave's columns share a scale");
  __shared__ __align__(16) uint8_t tile[2][(BM + BN) * 128];
  __shared__ __align__(16) float sc[2][BM + BN];
  const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), r = l & 15, g = l >> 4, wm = w / WN, wn = w - wm * WN;
  int m0, n0;
  tile_origin<BM, BN>(a, m0, n0);

  // the wave's pieces: eight rows of 128 bytes each, of a for the first waves, of w for the others
  const int row0 = w * P * 8;
  const bool is_a = row0 < BM;
  const int64_t st = is_a ? a.as : a.ws;
  const int rows = is_a ? min(BM, a.M - m0) : min(BN, a.N - n0), rbase = is_a ? row0 : row0 - BM;
  const u32x4 gb = buf_words(is_a ? a.a + m0 * a.as : a.w + n0 * a.ws, (uint32_t)((rows - 1) * st + a.K));
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)tile) + row0 * 128;
  const int kc = 16 * ((l & 7) ^ (l >> 3));
  const uint32_t off = (uint32_t)((rbase + (l >> 3)) * st) + kc;
  TileScales<BM, BN, NTH, WROW> sv(a, m0, n0);
  auto fetch = [&](int kb) {
    const uint32_t o = (kb * 128 + kc < a.K ? off : OOB) + kb * 128;  // (past a row's end: zeros)
#pragma unroll
    for (int p = 0; p < P; ++p)
      load_lds16(gb, o + (uint32_t)(8 * p * st), lds0 + (kb & 1) * (BM + BN) * 128 + 8 * p * 128);
    sv.load(kb);
  };
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = zero4();
  const int ra = (wm * TM * 16 + r) * 128 + 16 * (g ^ (r & 7)), rw = (BM + wn * TN * 16 + r) * 128 + 16 * (g ^ (r & 7));
  fetch(0);
  sv.store(sc[0]);
  wait_vm<0>();
  lds_barrier();
  auto block = [&](int kb) {
    const uint8_t* t = tile[kb & 1];
    const float* s = sc[kb & 1];
    auto frag = [&](int at) {
      return join16(*reinterpret_cast<const uint4*>(t + at), *reinterpret_cast<const uint4*>(t + (at ^ 64)));
    };
    i32x8 wf[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) wf[j] = frag(rw + j * 16 * 128);
    f32x4 sw[WROW ? TN : 1];
    if constexpr (WROW) {
#pragma unroll
      for (int j = 0; j < TN; ++j) sw[j] = *reinterpret_cast<const f32x4*>(s + BM + (wn * TN + j) * 16 + 4 * g);
    } else {
      sw[0][0] = s[BM + wn * TN * 16];
    }
    // a row of tiles ahead its operand is read, and two tiles behind a product meets its
    // scales, while the matrix unit works
    constexpr int LAG = 2;
    f32x4 p[LAG + 1];
    static_assert(LAG <= TN, "a row's scale is kept for one row more");
    float sa[3];
    i32x8 af[2];
    af[0] = frag(ra);
    sa[0] = s[wm * TM * 16 + r] * (WROW ? 1.f : sw[0][0]);
    static_for<0, TM * TN + LAG>([&](auto T) {
      constexpr int t = decltype(T)::value, i = t / TN, j = t % TN, u = t - LAG;
      if constexpr (t < TM * TN) {
        if constexpr (j == 0 && i + 1 < TM) {
          af[(i + 1) & 1] = frag(ra + (i + 1) * 16 * 128);
          sa[(i + 1) % 3] = s[(wm * TM + i + 1) * 16 + r] * (WROW ? 1.f : sw[0][0]);
        }
        p[t % (LAG + 1)] = mma8(wf[j], af[i & 1]);
      }
      if constexpr (u >= 0) {
        constexpr int ui = u / TN, uj = u % TN;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[ui][uj][e] += p[u % (LAG + 1)][e] * (WROW ? sa[ui % 3] * sw[WROW ? uj : 0][e] : sa[ui % 3]);
      }
      __builtin_amdgcn_sched_barrier(0);  // (as written: the scheduler would gather the products first)
    });
  };
  for (int kb = 0; kb + 1 < a.nb; ++kb) {
    fetch(kb + 1);
    block(kb);
    sv.store(sc[(kb + 1) & 1]);
    wait_vm<0>();
    lds_barrier();
  }
  block(a.nb - 1);
  // (all sums here: sunk into the stores' branches, they would keep every product alive)
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) asm volatile("" : "+v"(acc[i][j]));
  store_tile<O>(a, acc, m0 + wm * TM * 16, n0 + wn * TN * 16);
}

// The same with the codes widened to bf16 on their way through registers into LDS, half
// a block (64 columns) at a time, for a 32-bit y.  128 x 128, four waves, two
// workgroups a CU.
template <typename O, bool WROW>
__global__ __launch_bounds__(256, 2) void k_mm8_wide(Mm8Args a) {
  constexpr int BM = 128, BN = 128, NTH = 256, TM = 4, TN = 4, P = (BM + BN) * 4 / NTH;
  __shared__ __align__(16) uint8_t tile[2][(BM + BN) * 128];
  __shared__ __align__(16) float sc[2][BM + BN];
  const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), r = l & 15, g = l >> 4, wm = w >> 1, wn = w & 1;
  int m0, n0;
  tile_origin<BM, BN>(a, m0, n0);
  const GBuf ga = gbuf(a.a + m0 * a.as, (uint32_t)((min(BM, a.M - m0) - 1) * a.as + a.K));
  const GBuf gw = gbuf(a.w + n0 * a.ws, (uint32_t)((min(BN, a.N - n0) - 1) * a.ws + a.K));
  TileScales<BM, BN, NTH, WROW> sv(a, m0, n0);
  const int pr = threadIdx.x >> 2, pk = 16 * (threadIdx.x & 3);  // a thread's rows pr + 64 j, columns pk .. + 15
  uint4 st[P];
  auto fetch = [&](int h) {  // half block h
    const int k = 64 * h + pk;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const bool is_a = j < P / 2;
      const int row = pr + 64 * (is_a ? j : j - P / 2);
      st[j] = gld16(is_a ? ga : gw, k < a.K ? (uint32_t)(row * (is_a ? a.as : a.ws)) + k : OOB);
    }
  };
  auto put = [&](int b) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      uint8_t* row = tile[b] + (pr + 64 * j) * 128;
      const int c = pk / 8;  // 16-byte pieces c and c + 1 of the row
      *reinterpret_cast<bf16x8*>(row + 16 * (c ^ (pr & 7))) = widen8(st[j].x, st[j].y);
      *reinterpret_cast<bf16x8*>(row + 16 * ((c + 1) ^ (pr & 7))) = widen8(st[j].z, st[j].w);
    }
  };
  f32x4 acc[TM][TN], p[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = zero4();
  const int ra = (wm * 64 + r) * 128, rw = (BM + wn * 64 + r) * 128;
  auto half = [&](int b, bool first) {
    const uint8_t* t = tile[b];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int c = 16 * ((4 * q + g) ^ (r & 7));
      bf16x8 wf[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) wf[j] = *reinterpret_cast<const bf16x8*>(t + rw + j * 16 * 128 + c);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const bf16x8 af = *reinterpret_cast<const bf16x8*>(t + ra + i * 16 * 128 + c);
#pragma unroll
        for (int j = 0; j < TN; ++j) p[i][j] = mma(wf[j], af, first && q == 0 ? zero4() : p[i][j]);
      }
    }
  };
  fetch(0);
  sv.load(0);
  put(0);
  sv.store(sc[0]);
  lds_barrier();
  for (int kb = 0; kb < a.nb; ++kb) {
    fetch(2 * kb + 1);
    half(0, true);
    put(1);
    lds_barrier();
    // (behind the last block: columns past the rows' end, zeros that nobody reads)
    fetch(2 * kb + 2);
    sv.load(min(kb + 1, a.nb - 1));
    half(1, false);
    const float* s = sc[kb & 1];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const float sa = s[wm * 64 + 16 * i + r];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        f32x4 sw;
        if constexpr (WROW) sw = *reinterpret_cast<const f32x4*>(s + BM + wn * 64 + 16 * j + 4 * g);
        else sw = f32x4{1.f, 1.f, 1.f, 1.f} * s[BM + wn * 64];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] += p[i][j][e] * (sa * sw[e]);
      }
    }
    put(0);
    sv.store(sc[(kb + 1) & 1]);
    lds_barrier();
  }
  store_tile<O>(a, acc, m0 + wm * 64, n0 + wn * 64);
}

bool few_rows(const Mm8Args& a) { return a.M <= 64; }

template <typename O>
hipError_t mm8_t(const Mm8Args& a, hipStream_t s) {
  if (few_rows(a)) {
    const unsigned nt = (unsigned)((a.N + 15) / 16);
    const int mt = (a.M + 15) / 16;
    if (mt == 1) REWY_LAUNCH((k_mm8_rows<O, 1>), dim3(nt), dim3(512), s, a);
    else if (mt == 2) REWY_LAUNCH((k_mm8_rows<O, 2>), dim3(nt), dim3(512), s, a);
    else REWY_LAUNCH((k_mm8_rows<O, 4>), dim3(nt), dim3(512), s, a);
    return hipGetLastError();
  }
  if constexpr (std::is_same_v<O, float>) {
    const dim3 grid((unsigned)(((a.M + 127) / 128) * (int64_t)((a.N + 127) / 128)));
    if (a.wrow) REWY_LAUNCH((k_mm8_wide<O, true>), grid, dim3(256), s, a);
    else REWY_LAUNCH((k_mm8_wide<O, false>), grid, dim3(256), s, a);
    return hipGetLastError();
  } else {
    auto tile = [&](auto bm, auto bn, auto wm, auto wn) {
      constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value, WM = decltype(wm)::value, WN = decltype(wn)::value;
      const dim3 grid((unsigned)(((a.M + BM - 1) / BM) * (int64_t)((a.N + BN - 1) / BN)));
      if (a.wrow) REWY_LAUNCH((k_mm8_tile<O, BM, BN, WM, WN, true>), grid, dim3(64 * WM * WN), s, a);
      else REWY_LAUNCH((k_mm8_tile<O, BM, BN, WM, WN, false>), grid, dim3(64 * WM * WN), s, a);
      return hipGetLastError();
    };
    std::integral_constant<int, 128> c128;
    std::integral_constant<int, 256> c256;
    std::integral_constant<int, 2> c2;
    std::integral_constant<int, 4> c4;
    const int64_t big = ((a.M + 255) / 256) * (int64_t)((a.N + 255) / 256);
    if (big >= 256) return tile(c256, c256, c2, c4);
    return tile(c128, c128, c2, c2);
  }
}

}  // namespace

const char* mm8_kernel(const Mm8Args& a, bool f32) { return few_rows(a) ? "k_mm8_rows" : f32 ? "k_mm8_wide" : "k_mm8_tile"; }
hipError_t launch_mm8(const Mm8Args& a, bool f32, hipStream_t s) { return f32 ? mm8_t<float>(a, s) : mm8_t<bf16>(a, s); }

}  // namespace rewy
