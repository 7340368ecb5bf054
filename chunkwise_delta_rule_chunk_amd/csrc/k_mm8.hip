// y[m, n] = sum_b sa[m, b] sw[n, b] (sum_{k in b} a[m, k] w[n, k]) + bias[n], with a and w
// in e4m3, blocks b of 128 along k and sw given for 128 rows of w or for each.
//
// Products of two codes are exact, a block's sum starts from zero and meets the two scales
// in fp32 once: acc += p (sa sw).  w is the first operand, so a lane holds four
// neighbouring columns of one row of y.
//
// A block is as long as one v_mfma_f32_16x16x128_f8f6f4.  The 8-bit matrix instructions
// line up at most eight neighbouring products before they are added and drop what lies 13 bits
// under the largest: 2^-10 of the sum of magnitudes at most; for normally distributed codes
// a block's sum is off by 1.5e-5 in norm (5e-5 where all codes are equally frequent), the same
// for the 32-long instruction.  A 16-bit y does not show that in norm (its rounding is 1.7e-3),
// only where its terms cancel; a 32-bit y would everywhere: it takes bf16 matrix instructions on the
// widened codes (exact; 1e-8), at half the rate.  Where w is read once for few rows nothing
// is bound by the matrix unit, and both take the wide form.
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
// An operand of 16 rows and a block: as it is, or widened to bf16.
template <bool WIDE>
struct Oper {
  i32x8 v;
  __device__ __forceinline__ void set(uint4 x, uint4 y) { v = join16(x, y); }
};
template <>
struct Oper<true> {
  bf16x8 v[4];
  __device__ __forceinline__ void set(uint4 x, uint4 y) {
    v[0] = widen8(x.x, x.y); v[1] = widen8(x.z, x.w); v[2] = widen8(y.x, y.y); v[3] = widen8(y.z, y.w);
  }
};
__device__ __forceinline__ f32x4 mma_block(const Oper<false>& w, const Oper<false>& a) { return mma8(w.v, a.v); }
__device__ __forceinline__ f32x4 mma_block(const Oper<true>& w, const Oper<true>& a) {
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
// 16 rows of w and all of a (at most 16 MT rows), its eight waves every eighth block, joined
// through LDS in their order.  16 x 4096 x 4096: 7.5 us for 17 MB; a launch, one trip to
// memory for rows and scales together, and the join, no rate.
template <typename O, int MT>
__global__ __launch_bounds__(512) void k_mm8_rows(Mm8Args a) {
  __shared__ float part[8][MT][4][64];
  const int w = wave_id(), l = lane_id(), r = l & 15, g = l >> 4;
  const int n0 = blockIdx.x * 16;
  const GBuf gw = gbuf(a.w + n0 * a.ws, (uint32_t)((min(16, a.N - n0) - 1) * a.ws + a.K));
  const GBuf ga = gbuf(a.a, (uint32_t)((a.M - 1) * a.as + a.K));
  const uint32_t wo = (uint32_t)(r * a.ws) + 32 * g, ao = (uint32_t)(r * a.as) + 32 * g;
  const float* swp[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = min(n0 + 4 * g + i, a.N - 1);
    swp[i] = a.sw + (int64_t)(a.wrow ? n : n / 128) * a.nb;
  }
  const float* sap[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) sap[t] = a.sa + (int64_t)min(16 * t + r, a.M - 1) * (a.ablk ? a.nb : 1);
  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = zero4();
  // four blocks at a time, all their loads first (blocks past the last and bytes past a
  // row's end: zeros)
  constexpr int U = 4;
#pragma unroll 1
  for (int k0 = w; k0 < a.nb; k0 += 8 * U) {
    uint4 wx[U][2], ax[U][MT][2];
    float sw[U][4], sa[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = k0 + 8 * u, k = kb * 128 + 32 * g, ks = min(kb, a.nb - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = k + 16 * h < a.K;
        wx[u][h] = gld16(gw, in ? wo + kb * 128 + 16 * h : OOB);
#pragma unroll
        for (int t = 0; t < MT; ++t) ax[u][t][h] = gld16(ga, in ? ao + (uint32_t)(16 * t * a.as) + kb * 128 + 16 * h : OOB);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sw[u][i] = swp[i][ks];
#pragma unroll
      for (int t = 0; t < MT; ++t) sa[u][t] = sap[t][a.ablk ? ks : 0];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + 8 * u >= a.nb) break;  // (zeros, but not beside a scale that is no number)
      Oper<true> wf, af;
      wf.set(wx[u][0], wx[u][1]);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        af.set(ax[u][t][0], ax[u][t][1]);
        const f32x4 p = mma_block(wf, af);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] += p[i] * (sa[u][t] * sw[u][i]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[w][t][i][l] = acc[t][i];
  __syncthreads();
  // wave t joins tile t
  const int m = 16 * w + r, n = n0 + 4 * g;
  if (w >= MT || m >= a.M) return;
  f32x4 s = zero4();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int q = 0; q < 8; ++q) s[i] += part[q][w][i][l];
    if (n + i < a.N) s[i] += ld_bias(a, n + i);
  }
  store4<O>(a, m, n, s);
}

// Wait until at most N of the wave's vector memory operations are in flight.
template <int N>
__device__ __forceinline__ void wait_vm() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

// 64 lanes' 16 bytes straight to LDS, lane l's at address dst + 16 l (dst the same in the
// whole wave); bytes outside the buffer arrive as zeros.  The compiler does not count these:
// wait_vm before the barrier behind which they are read.
__device__ __forceinline__ void load_lds16(u32x4 b, uint32_t off, uint32_t dst) {
  dst = __builtin_amdgcn_readfirstlane(dst);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(dst), "v"(off), "s"(b) : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(u32x4 b, uint32_t off, uint32_t dst) {  // the same with 4 bytes a lane
  dst = __builtin_amdgcn_readfirstlane(dst);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(dst), "v"(off), "s"(b) : "memory", "m0");
}
// gbuf's resource as its four words
__device__ __forceinline__ u32x4 buf_words(const void* base, uint32_t bytes) {
  const uint64_t p = (uint64_t)base;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(p >> 32) & 0xffffu)),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}

// A wave's tiles, from row m0 of a and row n0 of w, with the bias (FULL: all of them
// exist, TM TN stores)
template <typename O, int TM, int TN, bool FULL>
__device__ __forceinline__ void store_tile(const Mm8Args& a, const f32x4 (&acc)[TM][TN], int m0, int n0) {
  const int r = lane_id() & 15, g = lane_id() >> 4;
  if constexpr (FULL && std::is_same_v<O, bf16> && TN % 2 == 0) {
    // two tiles' columns change places between neighbouring lane groups, so that a lane
    // stores eight of one tile: columns 8 (g >> 1) .. of tile j + (g & 1)
#pragma unroll
    for (int j = 0; j < TN; j += 2) {
      float b[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) b[k][e] = ld_bias(a, n0 + 16 * (j + k) + 4 * g + e);
      bf16* y = reinterpret_cast<bf16*>(a.y) + (m0 + r) * a.ys + n0 + 16 * (j + (g & 1)) + 8 * (g >> 1);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        uint32_t x[2][2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            x[k][h] = __builtin_bit_cast(uint32_t, bf16x2{(bf16)(acc[i][j + k][2 * h] + b[k][2 * h]),
                                                          (bf16)(acc[i][j + k][2 * h + 1] + b[k][2 * h + 1])});
        const auto p = __builtin_amdgcn_permlane16_swap(x[0][0], x[1][0], false, false);
        const auto q = __builtin_amdgcn_permlane16_swap(x[0][1], x[1][1], false, false);
        typedef u32x4 u32x4_u __attribute__((aligned(2)));
        *reinterpret_cast<u32x4_u*>(y + 16 * i * a.ys) = u32x4{p[0], q[0], p[1], q[1]};
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int n = n0 + 16 * j + 4 * g;
    f32x4 b = zero4();
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (FULL || n + e < a.N) b[e] = ld_bias(a, n + e);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int m = m0 + 16 * i + r;
      if constexpr (FULL) {
        typename VecN<O, 4>::raw o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = (O)(acc[i][j][e] + b[e]);
        *reinterpret_cast<typename VecN<O, 4>::type*>(reinterpret_cast<O*>(a.y) + m * a.ys + n) = o;
      } else if (m < a.M && n < a.N) {
        store4<O>(a, m, n, acc[i][j] + b);
      }
    }
  }
}

// First rows of tile b: the workgroups go to the XCDs in turn, each of which
// takes a contiguous range, eight tiles of rows by as many of columns as are at work at
// once.
template <int BM, int BN>
__device__ __forceinline__ void tile_origin(const Mm8Args& a, int b, int& m0, int& n0) {
  const int nm = (a.M + BM - 1) / BM, nn = (a.N + BN - 1) / BN, id = xcd_range(b, nm * nn);
  const int grp = id / (8 * nn), gm = min(8, nm - 8 * grp), in = id - grp * 8 * nn;
  m0 = (8 * grp + in % gm) * BM;
  n0 = in / gm * BN;
}
// Tiles of BM rows of a by BN rows of w, WM x WN waves; NS blocks of 128 and their scales
// in LDS, straight from memory, the later ones on their way while one is used.  A row's
// eight pieces of 16 bytes lie in LDS at their place xor the row's last three bits, so
// that sixteen lanes that read one piece of sixteen rows meet the banks evenly.  A
// workgroup takes tiles blockIdx, + gridDim, ... as one run of blocks: the only barrier of a
// block stands before the last row of its products, and behind it the next block's first
// operands are read, so that the matrix unit does not wait at a block's start, nor at a
// tile's.  8192 x 12288 x 4096 to bf16, tiles of 256: 398 us in a row of calls (2.07
// PFLOP/s; a library's product without blocks' scales 2.7 at 8192 cubed); 1000 x 4354 x
// 2320 with a scale for each row of w to fp32, tiles of 128: 45 us (450 TFLOP/s), where 24
// of the 280 tiles share a CU with another one (256 tiles: 32 us).  Bound by the matrix
// unit and the sums behind it (a scale's product and a sum for each of four columns a tile
// and block), in small products by the latency of a block's loads, reads and products.
template <typename O, int BM, int BN, int WM, int WN, int NS, bool WROW, bool WIDE>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_mm8_tile(Mm8Args a, int tiles) {
  constexpr int NW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16, P = (BM + BN) / 8 / NW;
  static_assert((BM + BN) % (8 * NW) == 0 && BM % (8 * P) == 0 && 8 * P <= 64, "a wave's pieces are rows of one operand");
  static_assert(WROW || BN / WN <= 128, "a wave's columns share a scale");
  __shared__ __align__(16) uint8_t tile[NS][(BM + BN) * 128];
  __shared__ __align__(16) float sc[NS][BM + BN];
  const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), r = l & 15, g = l >> 4, wm = w / WN, wn = w - wm * WN;
  // the wave's pieces: eight rows of 128 bytes each, of a for the first waves, of w for the others
  const int row0 = w * P * 8;
  const bool is_a = row0 < BM;
  const int64_t st = is_a ? a.as : a.ws;
  const int rbase = is_a ? row0 : row0 - BM;
  const auto lds_at = [](const void* p) {
    return (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p);
  };
  const uint32_t tile0 = lds_at(tile) + row0 * 128, sc0 = lds_at(sc) + row0 * 4;
  const int kc = 16 * ((l & 7) ^ (l >> 3));
  const uint32_t off = (uint32_t)((rbase + (l >> 3)) * st) + kc;
  // a scale's rows share it, and it serves the whole row or a block
  const int srows = is_a || WROW ? 1 : 128, sblocks = is_a && !a.ablk ? 1 : a.nb, sstep = sblocks == 1 ? 0 : 4;
  const int ra = (wm * TM * 16 + r) * 128 + 16 * (g ^ (r & 7)), rw = (BM + wn * TN * 16 + r) * 128 + 16 * (g ^ (r & 7));
  int buf = 0, to = 0;          // where the block in use lies, where the next loads go
  int fb = blockIdx.x, fk = 0;  // tile and block of the next loads
  u32x4 gb, gs;
  uint32_t soff;
  auto begin = [&] {
    int m0, n0;
    tile_origin<BM, BN>(a, fb, m0, n0);
    const int rows = is_a ? min(BM, a.M - m0) : min(BN, a.N - n0);
    gb = buf_words(is_a ? a.a + m0 * a.as : a.w + n0 * a.ws, (uint32_t)((rows - 1) * st + a.K));
    // (lane l's scale is that of row rbase + l)
    const int x0 = (is_a ? m0 : n0) / srows, xl = ((is_a ? m0 : n0) + rows - 1) / srows;
    gs = buf_words((is_a ? a.sa : a.sw) + (int64_t)x0 * sblocks, (uint32_t)(xl - x0 + 1) * 4 * sblocks);
    soff = (uint32_t)(((is_a ? m0 : n0) + rbase + l) / srows - x0) * 4 * sblocks;
  };
  // (behind the last tile fk stays at nb: loads of zeros that nobody reads)
  auto advance = [&] {
    to = to + 1 == NS ? 0 : to + 1;
    if (++fk >= a.nb) {
      fk = a.nb;
      fb += gridDim.x;
      if (fb < tiles) {
        fk = 0;
        begin();
      }
    }
  };
  // loads 0 .. P - 1 of a block: rows; load P: scales (bytes past a row's end, rows and
  // blocks past the last: zeros)
  auto piece = [&](int p) {
    const uint32_t o = (fk * 128 + kc < a.K ? off : OOB) + fk * 128;
    load_lds16(gb, o + (uint32_t)(8 * p * st), tile0 + to * (BM + BN) * 128 + 8 * p * 128);
  };
  auto piece_scales = [&] {
    if (8 * P == 64 || l < 8 * P) load_lds4(gs, fk < a.nb ? soff + fk * sstep : OOB, sc0 + to * (BM + BN) * 4);
  };
  f32x4 acc[TM][TN];
  Oper<WIDE> wf[TN], af[2];
  f32x4 sw[WROW ? TN : 1], swn[WROW ? TN : 1];
  float sa[3];
  auto frag = [&](Oper<WIDE>& f, int from, int at) {
    f.set(*reinterpret_cast<const uint4*>(tile[from] + at), *reinterpret_cast<const uint4*>(tile[from] + (at ^ 64)));
  };
  auto scale_w = [&](int from, int j) {
    if constexpr (WROW) return *reinterpret_cast<const f32x4*>(sc[from] + BM + (wn * TN + j) * 16 + 4 * g);
    else return f32x4{sc[from][BM + wn * TN * 16], 0.f, 0.f, 0.f};
  };
  auto scale_a = [&](int from, int i) { return sc[from][(wm * TM + i) * 16 + r]; };
  // The products of the block in `buf`.  A row of tiles ahead its operand is read, and two
  // tiles behind a product meets its scales, while the matrix unit works.  Before the
  // last row: the next block's loads, sent for NS - 1 blocks ago, have arrived (those of the
  // blocks behind it may be on their way), and all waves have read this one, whose place
  // the next loads take.
  auto block = [&] {
    constexpr int LAST = (TM - 1) * TN, PT = (P + TN) / TN;
    const int nxt = buf + 1 == NS ? 0 : buf + 1;
    auto add = [&](auto I, auto J, const f32x4& p) {
      constexpr int i = decltype(I)::value, j = decltype(J)::value;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] += p[e] * (sa[i % 3] * (WROW ? sw[WROW ? j : 0][e] : sw[0][0]));
    };
    // the next block's scales for column tile j, and a share of the loads
    auto next = [&](auto J) {
      constexpr int j = decltype(J)::value;
      if constexpr (WROW || j == 0) swn[WROW ? j : 0] = scale_w(nxt, j);
      if constexpr (j == TN - 1) sa[TM % 3] = scale_a(nxt, 0);
      static_for<0, PT>([&](auto k) {
        constexpr int q = j * PT + decltype(k)::value;
        if constexpr (q < P) piece(q);
        else if constexpr (q == P) piece_scales();
      });
    };
    constexpr int LAG = std::min(2, TN);
    f32x4 p[LAG + 1];
    static_for<0, TM * TN + LAG>([&](auto T) {
      constexpr int t = decltype(T)::value, i = t / TN, j = t % TN, u = t - LAG;
      if constexpr (t < TM * TN) {
        if constexpr (j == 0 && i + 1 < TM) {
          frag(af[(i + 1) & 1], buf, ra + (i + 1) * 16 * 128);
          sa[(i + 1) % 3] = scale_a(buf, i + 1);
        }
        if constexpr (t == LAST) {
          wait_vm<(NS - 2) * (P + 1)>();
          lds_barrier();
          frag(af[TM & 1], nxt, ra);
        }
        p[t % (LAG + 1)] = mma_block(wf[j], af[i & 1]);
        if constexpr (t >= LAST) {
          frag(wf[j], nxt, rw + j * 16 * 128);
          next(std::integral_constant<int, j>{});
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // (as written: the next product first, then the sums of one that is done)
      if constexpr (u >= 0) add(std::integral_constant<int, u / TN>{}, std::integral_constant<int, u % TN>{}, p[u % (LAG + 1)]);
      __builtin_amdgcn_sched_barrier(0);
    });
    // (all sums here: sunk behind a branch, they would keep every product alive)
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) asm volatile("" : "+v"(acc[i][j]));
#pragma unroll
    for (int j = 0; j < (WROW ? TN : 1); ++j) sw[j] = swn[j];
    af[0] = af[TM & 1];
    sa[0] = sa[TM % 3];
    buf = nxt;
    advance();
  };
  begin();
  for (int q = 0; q < NS; ++q) {
#pragma unroll
    for (int p = 0; p < P; ++p) piece(p);
    piece_scales();
    advance();
  }
  wait_vm<(NS - 1) * (P + 1)>();
  lds_barrier();
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    frag(wf[j], 0, rw + j * 16 * 128);
    if (WROW || j == 0) sw[WROW ? j : 0] = scale_w(0, j);
  }
  frag(af[0], 0, ra);
  sa[0] = scale_a(0, 0);
  for (int b = blockIdx.x; b < tiles; b += gridDim.x) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = zero4();
    for (int kb = 0; kb < a.nb; ++kb) block();
    int m0, n0;
    tile_origin<BM, BN>(a, b, m0, n0);
    m0 += wm * TM * 16;
    n0 += wn * TN * 16;
    if (m0 + TM * 16 <= a.M && n0 + TN * 16 <= a.N) store_tile<O, TM, TN, true>(a, acc, m0, n0);
    else store_tile<O, TM, TN, false>(a, acc, m0, n0);
  }
  wait_vm<0>();  // (nothing may arrive in LDS behind the workgroup's end)
}

// up to 32 rows w is read straight into registers (N = K = 4096: 10.5 us a call up to 32
// rows, 16.3 for 64; tiles of 64: 13.9 us for up to 128 rows)
bool few_rows(const Mm8Args& a) { return a.M <= 32; }

template <typename O>
hipError_t mm8_t(const Mm8Args& a, hipStream_t s) {
  if (few_rows(a)) {
    const unsigned nt = (unsigned)((a.N + 15) / 16);
    if (a.M <= 16) REWY_LAUNCH((k_mm8_rows<O, 1>), dim3(nt), dim3(512), s, a);
    else REWY_LAUNCH((k_mm8_rows<O, 2>), dim3(nt), dim3(512), s, a);
    return hipGetLastError();
  }
  constexpr bool WIDE = std::is_same_v<O, float>;
  // workgroups: as many as the chip holds at once
  auto tile = [&](auto bm, auto bn, auto wm, auto wn, auto ns, int held) {
    constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value, WM = decltype(wm)::value, WN = decltype(wn)::value,
                  NS = decltype(ns)::value;
    const int tiles = (int)(((a.M + BM - 1) / BM) * (int64_t)((a.N + BN - 1) / BN));
    const dim3 grid(std::min(tiles, held));
    if (a.wrow) REWY_LAUNCH((k_mm8_tile<O, BM, BN, WM, WN, NS, true, WIDE>), grid, dim3(64 * WM * WN), s, a, tiles);
    else REWY_LAUNCH((k_mm8_tile<O, BM, BN, WM, WN, NS, false, WIDE>), grid, dim3(64 * WM * WN), s, a, tiles);
    return hipGetLastError();
  };
  constexpr std::integral_constant<int, 2> c2;
  constexpr std::integral_constant<int, 4> c4;
  constexpr std::integral_constant<int, 64> c64;
  constexpr std::integral_constant<int, 128> c128;
  constexpr std::integral_constant<int, 256> c256;
  auto count = [&](int64_t e) { return ((a.M + e - 1) / e) * ((a.N + e - 1) / e); };
  // Tiles of 64 while they all run at once, two a CU (512 x 4096 x 4096: 19 us, tiles of 128
  // 26; twice the rows: 35 and 29); tiles of 256 as soon as they fill the CUs (4096 x 4096 x
  // 4096: 69 us, tiles of 128 80; half the rows: 58 and 42).  Between them tiles of 128: where
  // each has a CU to itself with twice the waves and blocks (1000 x 4096 x 2320: 19.6 us
  // instead of 22.5; 1000 x 6144, two a CU: 32 instead of 29.7).  Widened operands leave no
  // registers for tiles of 256, and gain nothing from more waves (32 and 31 us).
  if (count(64) <= 512) return tile(c64, c64, c2, c2, c4, 512);
  if constexpr (!WIDE) {
    if (count(256) >= 256) return tile(c256, c256, c2, c4, c2, 256);
    if (count(128) <= 256) return tile(c128, c128, c2, c4, c4, 256);
  }
  return tile(c128, c128, c2, c2, c2, 512);
}

}  // namespace

const char* mm8_kernel(const Mm8Args& a) { return few_rows(a) ? "k_mm8_rows" : "k_mm8_tile"; }
hipError_t launch_mm8(const Mm8Args& a, bool f32, hipStream_t s) { return f32 ? mm8_t<float>(a, s) : mm8_t<bf16>(a, s); }

}  // namespace rewy
