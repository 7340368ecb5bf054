// Linear attention with one constant decay for each head (decay.hpp): the
// segments' states, the pass that joins them, the walks, and the token-serial
// form.
#include "decay.hpp"

namespace rewy {

namespace {

// lam^n with n >= 0, formed in 64 bits (lam^0 is 1, also for lam = 0)
__device__ __forceinline__ double decay_pow(float g, int n) { return n == 0 ? 1.0 : exp((double)g * n); }
// the same as hi + lo: a factor that meets the same state once a chunk would
// otherwise carry its rounding along with the state's age
__device__ __forceinline__ void decay_pow2(float g, int n, float& hi, float& lo) {
  const double d = decay_pow(g, n);
  hi = (float)d;
  lo = (float)(d - (double)hi);
}
// lo S of such a factor: an infinite S counts as the largest number, so that hi S stays what
// it is (lo may be zero or negative)
__device__ __forceinline__ float decay_low(float lo, float S) { return lo * __builtin_amdgcn_fmed3f(S, -3.4028235e38f, 3.4028235e38f); }

// Row fragment (rows in slot order) of a tile with its columns as they are, for a
// contraction whose partner lies in acc order (store_acc_order)
template <typename T>
__device__ __forceinline__ uint4 frag_row_slot_acc(const T* p, int ld, int r0, int k0) {
  const int l = lane_id();
  if constexpr (std::is_same_v<T, bf16>) {
    const T* q = p + (r0 + slot_row<T>(l & 15)) * ld + k0 + 4 * (l >> 4);
    const uint2 x = *reinterpret_cast<const uint2*>(q), y = *reinterpret_cast<const uint2*>(q + 16);
    return uint4{x.x, x.y, y.x, y.y};
  } else {
    return frag_row_slot<T>(p, ld, r0, k0);
  }
}

// S = dec S + sum_t B_t (al_t C_t)^T for the wave's CT tiles of 16 columns (B from the
// tile sb; C's columns in cf, scaled and split into NS pieces; sal in slot order).  Two
// pieces: the products are added onto hi S, one rounding of the state's size for each
// matrix instruction, which the pieces' 2^-17 allow.  Else they are summed by themselves
// and lo S joins them.
template <typename T, int KA, int CT, int NS>
__device__ __forceinline__ void decay_update(f32x4 (&S)[CT][KA / 16], const T* sb, int ldb, const uint4 (&cf)[CT][CH / KG<T>],
                                             const float* sal, const float (&hi)[CT], float lo) {
  constexpr int NQ = CH / KG<T>, VE = VEC<T>;
  const int g = lane_id() >> 4;
  uint4 uf[CT][NQ][NS];
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      float f[VE];
      frag_get<T>(f, cf[ct][q]);
#pragma unroll
      for (int e = 0; e < VE; e += 4) {
        const f32x4 al = *reinterpret_cast<const f32x4*>(sal + q * KG<T> + VE * g + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[e + i] *= al[i];
      }
      frag_split<T, NS>(uf[ct][q], f);
    }
#pragma unroll
  for (int nt = 0; nt < KA / 16; ++nt) {
    f32x4 u[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i) u[ct][i] = NS == 2 ? hi[ct] * S[ct][nt][i] : 0.f;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const uint4 bf = frag_col<T>(sb, ldb, q * KG<T>, 16 * nt);
#pragma unroll
      for (int s = NS - 1; s >= 0; --s)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) mma16B<T>(u[ct], bf, uf[ct][q][s]);
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        S[ct][nt][i] = NS == 2 ? u[ct][i] : hi[ct] * S[ct][nt][i] + (decay_low(lo, S[ct][nt][i]) + u[ct][i]);
  }
}

// Local state of one segment and head: forward, from zero, the sum of its keys and
// values; reverse, the adjoint that its queries and output adjoints send to the state
// that enters it.  Where a sequence is one segment the state starts from h0 (dht) and is
// ht (dh0) itself.  Wave w holds 16 CT columns of the state.
// Three pieces of bf16 (24 bits) a chunk make 48 products where one would make 16, so
// the matrix unit and the pieces' arithmetic cost what the loads do: 8192 tokens of 32
// heads, K = V = 128, bf16: 48 us for 134 MB read and 34 written (3.5 TB/s), 45 with all
// heads on one key and value head, whose rows come from L2.  Two tiles of 16 columns a
// wave read the key tile half as often (49 us with one, and with spills).
// Two waves a SIMD: two workgroups of 256 threads a CU, four of 128 (V = 32).
// 16-column tiles of a wave, threads of a workgroup
template <typename T, int V>
constexpr int state_ct() { return V == 128 ? 2 : 1; }
template <typename T, int V>
constexpr int state_threads() { return 4 * V / state_ct<T, V>(); }
template <typename T, int K, int V>
__global__ __launch_bounds__((state_threads<T, V>()), 2) void k_decay_state(DecayArgs a, int dirs) {
  constexpr int CT = state_ct<T, V>(), NTH = state_threads<T, V>(), LK = pitch<T>(K), LV = pitch<T>(V), NQ = CH / KG<T>, NT = K / 16;
  __shared__ __align__(16) T sk[CH * LK];
  __shared__ __align__(16) T su[CH * LV];
  __shared__ float pw[CH + 1], pl[CH + 1];     // powers of the decay, and what their rounding left
  __shared__ __align__(16) float sal[CH];
  const int dir = dirs == 2 ? 1 : blockIdx.y;
  const int wk = xcd_range(blockIdx.x, a.nslot * a.H), slot = wk / a.H, h = wk - slot * a.H, grp = h / a.per;
  const Piece pc = find_piece(a.seq, slot, a.seg);
  if (!pc.on) return;
  const int t0 = pc.bos + pc.k * a.seg, t1 = min(t0 + a.seg, pc.eos);
  float* const end = dir ? a.dh0 : a.ht;       // the sequence's own end
  if (a.two && !end && (dir ? pc.k == 0 : t1 >= pc.eos)) return;  // nobody reads it
  const int nch = max(t1 - t0 + CH - 1, 0) / CH, w = wave_id(), l = lane_id();
  const float g = a.g[h];
  if (threadIdx.x <= CH) decay_pow2(g, threadIdx.x, pw[threadIdx.x], pl[threadIdx.x]);
  float hi = 1.f, lo = 0.f;

  const int64_t kv = (int64_t)K * V, seqhead = ((int64_t)pc.n * a.H + h) * kv;
  const int col = 16 * CT * w + (l & 15), row = 4 * (l >> 4);
  const float* init = a.two ? nullptr : dir ? a.dht : a.h0;
  f32x4 S[CT][NT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[ct][nt][i] = init ? init[seqhead + (16 * nt + row + i) * V + col + 16 * ct] : 0.f;
  TileRegs<T, CH, K, NTH> rk;
  TileRegs<T, CH, V, NTH> ru;
  auto fetch = [&](int c) {
    const int ci = dir ? nch - 1 - c : c, tok = t0 + ci * CH, len = min(CH, t1 - tok);
    load_tile<T, K, NTH>(rk, dir ? a.q : a.k, tok, dir ? a.qs : a.ks, (dir ? h : grp) * K, len, K);
    load_tile<T, V, NTH>(ru, dir ? a.dO : a.v, tok, dir ? a.os : a.vs, (dir ? h : grp) * V, len, V);
  };
  if (nch > 0) fetch(0);
  __syncthreads();
  int last = -1;  // tokens of the chunk before
  for (int c = 0; c < nch; ++c) {
    const int ci = dir ? nch - 1 - c : c, len = min(CH, t1 - t0 - ci * CH);
    rk.store(sk, LK, threadIdx.x);
    ru.store(su, LV, threadIdx.x);
    if (len != last) {  // (at most twice: the sequence's end)
      if (w == 0) sal[slot_of<T>(l)] = dir ? a.scale * pw[l + 1] : l < len ? pw[len - 1 - l] : 0.f;
      hi = pw[len];
      lo = pl[len];
      last = len;
    }
    lds_barrier();
    if (c + 1 < nch) fetch(c + 1);
    uint4 ut[CT][NQ];
    float dec[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      dec[ct] = hi;
#pragma unroll
      for (int q = 0; q < NQ; ++q) ut[ct][q] = frag_col<T>(su, LV, q * KG<T>, 16 * (CT * w + ct));
    }
    decay_update<T, K, CT, SPLIT<T>>(S, sk, LK, ut, sal, dec, lo);
    lds_barrier();
  }
  float* o = a.two ? (dir ? a.sr : a.sf) + ((int64_t)slot * a.H + h) * kv : end + seqhead;
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[(16 * nt + row + i) * V + col + 16 * ct] = S[ct][nt][i];
}

// In place: the local states of a sequence's segments become the states that enter
// them (forward; from h0) or the adjoints of the states that leave them (reverse; from
// dht); what is left at the end is ht or dh0.  Bound by memory: 16 segments of 32 heads
// of 128 x 128 in 12.3 us (5.5 TB/s read and written), 2 x 8 of 16 heads of 64 x 64 in 4.8
// (one segment's load at a time, behind the powers: 13.4 and 6.3).
__global__ __launch_bounds__(256) void k_decay_pass(DecayArgs a, int dirs) {
  const int kv = a.K * a.V, n = blockIdx.x / a.H, h = blockIdx.x - n * a.H, dir = dirs == 2 ? 1 : blockIdx.z;
  const int e = (blockIdx.y * 256 + threadIdx.x) * 4;
  if (e >= kv) return;
  int bos, eos;
  seq_range(a.seq, n, bos, eos);
  const int base = slot_base(a.seq, n, a.seg), ns = (eos - bos + a.seg - 1) / a.seg;
  const float* init = dir ? a.dht : a.h0;
  float* st = dir ? a.sr : a.sf;
  float* end = dir ? a.dh0 : a.ht;
  const int64_t at = ((int64_t)n * a.H + h) * kv + e;
  const float g = a.g[h];
  constexpr int U = 8;  // segments sent for at once
  auto place = [&](int i) {
    return reinterpret_cast<f32x4*>(st + ((int64_t)(base + (dir ? ns - 1 - i : i)) * a.H + h) * kv + e);
  };
  // (the last local state is there only if its end is handed out)
  const int nl = end ? ns : ns - 1;
  f32x4 loc[U];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < nl) loc[u] = *place(i0 + u);
  };
  fetch(0);
  f32x4 S = zero4();
  if (init) S = *reinterpret_cast<const f32x4*>(init + at);
  float hi, lo, hl, ll;  // a whole segment's decay, and the last one's
  decay_pow2(g, a.seg, hi, lo);
  decay_pow2(g, eos - bos - (ns - 1) * a.seg, hl, ll);
  for (int i0 = 0; i0 < ns; i0 += U) {
    f32x4 in[U];  // the states that enter
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;
      in[u] = S;
      if (i < nl) {
        const bool last = dir ? i == 0 : i + 1 == ns;
        const float dh = last ? hl : hi, dl = last ? ll : lo;
#pragma unroll
        for (int j = 0; j < 4; ++j) S[j] = dh * S[j] + (decay_low(dl, S[j]) + loc[u][j]);
      }
    }
    fetch(i0 + U);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < ns) *place(i0 + u) = in[u];
  }
  if (end) *reinterpret_cast<f32x4*>(end + at) = S;
}

// A walk's operands: rows A and B (KA long) and C (CV long) of one head.
struct WalkIo {
  const void *a, *b, *c;
  int64_t as, bs, cs;
  int acol, bcol, ccol;  // first columns
  void* out;             // in the operands' type, or
  float* outf;           // in fp32, before the sum over a group's heads
  int64_t outs;
  int ocol;
};

// The walk of one segment and head.  Wave w owns 16 CT columns of the output and of the
// state, whose rows are B's columns.  A chunk's coefficients (64 x 64, masked by the
// order and scaled by powers of the decay) are formed block by block by all waves and
// shared through LDS.  REV: tokens from the end, coefficients above the diagonal.  TS:
// the state's memory [K, V] holds the walk's state transposed.
// bf16: the coefficients and the entering state are rounded once each as operands,
// which the output's own rounding covers; the carried state is fp32, its update in two
// pieces (17 bits: only outputs of 16 bits read it, the states that are handed out come
// from k_decay_state in three).
// An infinity or NaN of C would reach rows on the other side of the diagonal through the
// coefficients' zeros: forward, it leaves the tile and comes back as NaN in its own and
// later rows (the backward's inputs are finite).
// What bounds it: with 246 registers a thread two workgroups fit a CU, two waves a SIMD,
// and a chunk's three barriers stand between a load, LDS, the products and the next tile;
// the matrix unit is at work 27% of the time, the vector unit 33%, LDS 46% (8192 tokens of 32
// heads, K = V = 128).
// Rows that come from L2 alone are 4% faster, so it is not HBM.  Registers for three waves
// a SIMD are not there (K = 64, V = 128 with spills: 86 us where this takes 57).
template <typename T, int KA, int CV, int CT, bool REV, bool TS, bool ODD>
__device__ __forceinline__ void decay_walk(const DecayArgs& a, const WalkIo& io, T* lds, float* tab, int* sodd,
                                           const Piece& pc, int slot, int h) {
  constexpr int NW = CV / 16 / CT, NTH = 64 * NW;
  constexpr int LA = pitch<T>(KA), LC = pitch<T>(CV), LM = pitch<T>(CH);
  constexpr int NQ = CH / KG<T>, NT = KA / 16, KQ = KA / KG<T>, NB = (10 + NW - 1) / NW;
  T* sa = lds;            // columns in the slot order of frag_acc
  T* sb = sa + CH * LA;
  T* sc = sb + CH * LA;
  T* sm = sc + CH * LC;   // coefficients, columns in slot order
  // the update's factors in slot order; the powers 0 .. 64 of the decay, and what their rounding left
  float *sal = tab, *pw = tab + CH, *pl = pw + CH + 1;
  const int t0 = pc.bos + pc.k * a.seg, t1 = min(t0 + a.seg, pc.eos), nch = max(t1 - t0 + CH - 1, 0) / CH;
  if (nch == 0) return;
  const int w = wave_id(), l = lane_id(), g4 = l >> 4, r = l & 15;
  const float g = a.g[h];
  TileRegs<T, CH, KA, NTH> ra, rb;
  TileRegs<T, CH, CV, NTH> rc;
  auto chunk = [&](int c) { return REV ? nch - 1 - c : c; };
  auto fetch = [&](int c) {
    const int tok = t0 + chunk(c) * CH, len = min(CH, t1 - tok);
    load_tile<T, KA, NTH>(ra, io.a, tok, io.as, io.acol, len, KA);
    load_tile<T, KA, NTH>(rb, io.b, tok, io.bs, io.bcol, len, KA);
    load_tile<T, CV, NTH>(rc, io.c, tok, io.cs, io.ccol, len, CV);
  };
  fetch(0);

  // the state that enters (REV: the adjoint of the state that leaves) the segment
  const int64_t kv = (int64_t)KA * CV;
  const float* init = a.two ? (REV ? a.sr : a.sf) + ((int64_t)slot * a.H + h) * kv
                            : (REV ? a.dht : a.h0) ? (REV ? a.dht : a.h0) + ((int64_t)pc.n * a.H + h) * kv : nullptr;
  f32x4 S[CT][NT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = 16 * nt + 4 * g4, col = 16 * (CT * w + ct) + r;
      S[ct][nt] = zero4();
      if (init) {
        if constexpr (TS) {
          S[ct][nt] = *reinterpret_cast<const f32x4*>(init + col * KA + row);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) S[ct][nt][i] = init[(row + i) * CV + col];
        }
      }
    }
  if (threadIdx.x <= CH) {
    const int i = threadIdx.x;
    decay_pow2(g, i, pw[i], pl[i]);
    const float p = pw[i];
    if (REV ? i > 0 : i < CH) sal[slot_of<T>(REV ? i - 1 : CH - 1 - i)] = REV ? a.scale * p : p;
  }
  // pairs of blocks right of the diagonal lie inside a contraction of 32: zeros, written once
  for (int i = threadIdx.x; i < CH * LM; i += NTH) sm[i] = (T)0.f;
  if (ODD && threadIdx.x == 0) *sodd = 0;
  lds_barrier();
  // of a chunk, and (REV) of the sequence's last one
  const int nl = min(CH, t1 - t0 - (nch - 1) * CH);
  const float hi = pw[CH], lo = pl[CH], hl = pw[nl], ll = pl[nl];
  // Coefficients of a lane: block (I, J) holds rows j = 16 J + slot_row(4 g4 + e), columns
  // i = 16 I + r; within a diagonal block lam^|i-j| or zero, 16 (n + 1) tokens away
  // lam^(16 n) lam^(16 +- (i-j)).
  float pd[4], po[4], p16[3];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int d = REV ? slot_row<T>(4 * g4 + e) - r : r - slot_row<T>(4 * g4 + e);
    pd[e] = d >= 0 ? a.scale * pw[max(d, 0)] : 0.f;
    po[e] = a.scale * pw[16 + d];
  }
#pragma unroll
  for (int e = 0; e < 3; ++e) p16[e] = pw[16 * e];
  auto put_tiles = [&](int c) {
    if (ODD && tile_not_finite<T, CV, NTH>(rc)) *sodd = c + 1;
    store_acc_order<T, KA, NTH>(ra, sa, LA);
    rb.store(sb, LA, threadIdx.x);
    rc.store(sc, LC, threadIdx.x);
  };
  put_tiles(0);
  for (int c = 0; c < nch; ++c) {
    const int tok = t0 + chunk(c) * CH, len = min(CH, t1 - tok);
    lds_barrier();  // tiles complete
    if (c + 1 < nch) fetch(c + 1);
    // coefficients
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int blk = b * NW + w;
      if (blk < 10) {
        int X, Y;
        tri_block(blk, X, Y);
        const int I = REV ? Y : X, J = REV ? X : Y, i = 16 * I + r;
        f32x4 acc = zero4();
#pragma unroll
        for (int q = 0; q < KQ; ++q)
          mma16B<T>(acc, frag_row_slot_acc<T>(sb, LA, 16 * J, q * KG<T>), frag_row<T>(sa, LA, 16 * I, q * KG<T>));
        f32x4 m;
        const float p = X - Y == 3 ? p16[2] : X - Y == 2 ? p16[1] : p16[0];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = REV ? slot_row<T>(4 * g4 + e) - r : r - slot_row<T>(4 * g4 + e);
          m[e] = X == Y ? (d >= 0 ? acc[e] * pd[e] : 0.f) : acc[e] * (po[e] * p);
        }
        st4<T>(sm + i * LM + slot_base4<T>(J, g4), m);
      }
    }
    const bool odd = ODD && __builtin_amdgcn_readfirstlane(*sodd) == c + 1;
    if (odd) {
#pragma unroll 1
      for (int ct = 0; ct < CT; ++ct) {
        const int col = 16 * (CT * w + ct) + r;
        int first = CH;
#pragma unroll 1
        for (int j = CH - 4 + g4; j >= 0; j -= 4)
          if (!(fabsf((float)sc[j * LC + col]) <= 3.4028235e38f)) {
            sc[j * LC + col] = (T)0.f;
            first = j;
          }
        first = min(first, __shfl_xor(first, 16, 64));
        sodd[1 + col] = min(first, __shfl_xor(first, 32, 64));
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // entering state: Y^T = S^T A^T, columns scaled by the decay since
    f32x4 Y[CT][4];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int I = 0; I < 4; ++I) Y[ct][I] = zero4();
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      uint4 sf[CT][1];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) frag_acc<T, 1>(sf[ct], S[ct], q);
#pragma unroll
      for (int I = 0; I < 4; ++I) {
        const uint4 af = frag_row<T>(sa, LA, 16 * I, q * KG<T>);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) mma16B<T>(Y[ct][I], sf[ct][0], af);
      }
    }
#pragma unroll
    for (int I = 0; I < 4; ++I) {
      const float e = REV ? pw[max(len - 1 - 16 * I - r, 0)] : a.scale * pw[16 * I + r + 1];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int i = 0; i < 4; ++i) Y[ct][I][i] *= e;
    }
    lds_barrier();  // coefficients complete
    uint4 xt[CT][NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) xt[ct][q] = frag_col<T>(sc, LC, q * KG<T>, 16 * (CT * w + ct));
#pragma unroll
      for (int I = 0; I < 4; ++I)
        if (REV ? (q + 1) * KG<T> > 16 * I : q * KG<T> <= 16 * I) {
          const uint4 mf = frag_row<T>(sm, LM, 16 * I, q * KG<T>);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) mma16B<T>(Y[ct][I], xt[ct][q], mf);
        }
    }
    if (io.outf) {
      const GBuf gy = gbuf(io.outf + tok * io.outs + io.ocol, tile_bytes<float>(len, io.outs, CV));
#pragma unroll
      for (int I = 0; I < 4; ++I)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
          gst16(gy, (uint32_t)(((16 * I + r) * io.outs + 16 * (CT * w + ct) + 4 * g4) * 4), __builtin_bit_cast(uint4, Y[ct][I]));
    } else {
      // (the wave's own columns of the C tile, read above and by no other wave)
      T* xw = sc + r * LC + 16 * CT * w + 4 * g4;
#pragma unroll
      for (int I = 0; I < 4; ++I)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) st4<T>(xw + 16 * I * LC + 16 * ct, Y[ct][I]);
    }
    if (c + 1 < nch) {
      constexpr int NS = std::is_same_v<T, bf16> ? 2 : 1;
      const float uh = REV && c == 0 ? hl : hi, ul = REV && c == 0 ? ll : lo;
      float dec[CT];
      // (a column that held an infinity or NaN: its state is NaN from here on)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) dec[ct] = ODD && odd && sodd[1 + 16 * (CT * w + ct) + r] < CH ? __builtin_nanf("") : uh;
      decay_update<T, KA, CT, NS>(S, sb, LA, xt, sal, dec, ul);
    }
    if (odd) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 1
      for (int ct = 0; ct < CT; ++ct) {
        const int col = 16 * (CT * w + ct) + r;
#pragma unroll 1
        for (int j = sodd[1 + col] + g4; j < CH; j += 4) sc[j * LC + col] = (T)__builtin_nanf("");
      }
    }
    lds_barrier();  // tiles and coefficients free, outputs complete
    if (!io.outf) {
      using TR = TileRegs<T, CH, CV, NTH>;
      const GBuf gy = gbuf(reinterpret_cast<T*>(io.out) + tok * io.outs + io.ocol, tile_bytes<T>(len, io.outs, CV));
#pragma unroll
      for (int j = 0; j < TR::N; ++j) {
        const int idx = threadIdx.x + j * NTH, row = idx / TR::PER, col = (idx - row * TR::PER) * TR::VEC;
        if (idx < TR::TOTAL)
          gst16(gy, (uint32_t)((row * io.outs + col) * (int64_t)sizeof(T)), *reinterpret_cast<const uint4*>(sc + row * LC + col));
      }
    }
    if (c + 1 < nch) put_tiles(c + 1);
  }
}

// LDS elements of a walk
template <typename T, int KA, int CV>
constexpr int walk_lds() { return 2 * CH * pitch<T>(KA) + CH * pitch<T>(CV) + CH * pitch<T>(CH); }
// 16-column tiles of a wave, threads of a workgroup
template <typename T, int CV>
constexpr int walk_ct() { return CV == 128 ? 2 : 1; }
template <typename T, int CV>
constexpr int walk_threads() { return 4 * CV / walk_ct<T, CV>(); }
// (fp32 tiles of 128 columns fill the LDS of a CU by themselves)
template <typename T, int KA, int CV>
constexpr int walk_waves() { return std::is_same_v<T, float> && KA + CV > 128 ? 1 : 2; }

template <typename T, int K, int V, int WHAT>
__device__ __forceinline__ void decay_one(const DecayArgs& a, T* lds, float* tab, int* sodd, int wk) {
  constexpr bool TS = WHAT & 1, REV = WHAT >= 2;  // (dq and dk)
  constexpr int KA = TS ? V : K, CV = TS ? K : V;
  const int slot = wk / a.H, h = wk - slot * a.H, grp = h / a.per;
  const Piece pc = find_piece(a.seq, slot, a.seg);
  if (!pc.on) return;
  WalkIo io = {};
  if constexpr (WHAT == DECAY_O)
    io = WalkIo{a.q, a.k, a.v, a.qs, a.ks, a.vs, h * K, grp * K, grp * V, a.o, nullptr, a.os, h * V};
  else if constexpr (WHAT == DECAY_DQ)
    io = WalkIo{a.dO, a.v, a.k, a.os, a.vs, a.ks, h * V, grp * V, grp * K, a.dq, nullptr, a.dqs, h * K};
  else if constexpr (WHAT == DECAY_DV)
    io = WalkIo{a.k, a.q, a.dO, a.ks, a.qs, a.os, grp * K, h * K, h * V, a.dv, a.vpart, a.vpart ? (int64_t)a.H * V : a.dvs, h * V};
  else
    io = WalkIo{a.v, a.dO, a.q, a.vs, a.os, a.qs, grp * V, h * V, h * K, a.dk, a.kpart, a.kpart ? (int64_t)a.H * K : a.dks, h * K};
  decay_walk<T, KA, CV, walk_ct<T, CV>(), REV, TS, WHAT == DECAY_O>(a, io, lds, tab, sodd, pc, slot, h);
}

// 8192 tokens of 32 heads, K = V = 128, bf16: 65 us (4.1 TB/s); 9000 tokens in 16
// sequences, 32 heads on 8, K = 64: 58 us; 2 x 1000 tokens of 16 heads, 64, fp32: 15.2 us;
// fp32, 8192 tokens of 32 heads, a call with its states: K = V = 64 114 us, 128 363 (one
// workgroup a CU beside 120 KB of LDS).
template <typename T, int K, int V>
__global__ __launch_bounds__((walk_threads<T, V>()), (walk_waves<T, K, V>())) void k_decay_fwd(DecayArgs a) {
  __shared__ __align__(16) T lds[walk_lds<T, K, V>()];
  __shared__ __align__(16) float tab[3 * CH + 2];
  __shared__ int sodd[1 + V];  // last chunk with an infinity or NaN, from 1; each column's first
  decay_one<T, K, V, DECAY_O>(a, lds, tab, sodd, xcd_range(blockIdx.x, a.nslot * a.H));
}

// The three walks of a segment and head are neighbours, so that the rows that they share
// come from an L2 while they are there: 171 us for 8192 tokens of 32 heads, K = V = 128,
// bf16 (151 in a row of calls), 805 MB past the CUs, 470 of them different (three launches
// one behind the other 201, when this took 186).  2 x 1000 tokens of 16 heads, 64, fp32: 32.
template <typename T, int K, int V>
__global__ __launch_bounds__((walk_threads<T, std::max(K, V)>()), (walk_waves<T, K, V>())) void k_decay_bwd(DecayArgs a) {
  __shared__ __align__(16) T lds[std::max(walk_lds<T, K, V>(), walk_lds<T, V, K>())];
  __shared__ __align__(16) float tab[3 * CH + 2];
  const int wk = xcd_range(blockIdx.x, 3 * a.nslot * a.H), at = wk / 3, what = wk - 3 * at;
  // (waves that a narrow output has no columns for leave; the barriers do without them)
  if (threadIdx.x >= (what == 0 ? walk_threads<T, V>() : walk_threads<T, K>())) return;
  if (what == 0) decay_one<T, K, V, DECAY_DV>(a, lds, tab, nullptr, at);
  else if (what == 1) decay_one<T, K, V, DECAY_DK>(a, lds, tab, nullptr, at);
  else decay_one<T, K, V, DECAY_DQ>(a, lds, tab, nullptr, at);
}

// dk and dv of a group: the sum over its heads, in order (rows behind the last sequence
// were not written and stay).  Bound by memory: 8192 tokens of 32 heads on 8, 128 wide: 54
// us for 302 MB (5.6 TB/s).  (A walk that took a group's heads one after the other would
// keep the sum in registers, and leave a quarter of the workgroups.)
template <typename T>
__global__ __launch_bounds__(256) void k_decay_sum(DecayArgs a) {
  const int d = blockIdx.y ? a.V : a.K, q = d / 4;
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x, tg = i / q;
  const int c = (int)(i - tg * q) * 4, grp = (int)(tg % a.G);
  const int64_t tok = tg / a.G;
  if (tok >= seq_start(a.seq, a.seq.N)) return;
  const float* p = (blockIdx.y ? a.vpart : a.kpart) + (tok * a.H + grp * a.per) * (int64_t)d + c;
  f32x4 s = *reinterpret_cast<const f32x4*>(p);
  for (int j = 1; j < a.per; ++j) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(p + (int64_t)j * d);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += x[e];
  }
  st4<T>(reinterpret_cast<T*>(blockIdx.y ? a.dv : a.dk) + tok * (blockIdx.y ? a.dvs : a.dks) + grp * d + c, s);
}

// Token by token: one workgroup per sequence and head, the state in registers, four
// neighbouring columns of K V / 1024 rows a thread.  For one new token it costs the
// state's bytes, read and written once: 64 sequences of 32 heads, K = V = 128: 53.6 us
// (5.0 TB/s).
template <typename T, int K, int V>
__global__ __launch_bounds__(256) void k_decay_recurrent(DecayArgs a) {
  constexpr int CQ = V / 4, RP = 256 / CQ, NR = (K + RP - 1) / RP;  // column quads, rows side by side, rows of a thread
  __shared__ __align__(16) float sk[2][K], sq[2][K];
  __shared__ float sy[2][4][V];
  const int n = blockIdx.x / a.H, h = blockIdx.x - n * a.H, grp = h / a.per;
  const int cq = threadIdx.x % CQ, r0 = threadIdx.x / CQ, w = wave_id(), l = lane_id();
  int bos, eos;
  seq_range(a.seq, n, bos, eos);
  float hi, lo;
  decay_pow2(a.g[h], 1, hi, lo);
  const int64_t st = ((int64_t)n * a.H + h) * K * V + 4 * cq;
  f32x4 S[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i)
    S[i] = a.h0 ? *reinterpret_cast<const f32x4*>(a.h0 + st + (int64_t)(r0 + RP * i) * V) : zero4();
  for (int t = bos; t < eos; ++t) {
    const int p = t & 1;  // (two sets: a token's sums are read before the next but one writes them)
    const T* kp = reinterpret_cast<const T*>(a.k) + (int64_t)t * a.ks + grp * K;
    const T* qp = reinterpret_cast<const T*>(a.q) + (int64_t)t * a.qs + h * K;
    const f32x4 v = ld4<T>(reinterpret_cast<const T*>(a.v) + (int64_t)t * a.vs + grp * V + 4 * cq);
    for (int i = threadIdx.x; i < 2 * K; i += 256) {
      if (i < K) sk[p][i] = (float)kp[i];
      else sq[p][i - K] = a.scale * (float)qp[i - K];
    }
    lds_barrier();
    f32x4 y = zero4();
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const float kx = sk[p][r0 + RP * i], qx = sq[p][r0 + RP * i];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        S[i][e] = hi * S[i][e] + (decay_low(lo, S[i][e]) + kx * v[e]);
        y[e] += qx * S[i][e];
      }
    }
    // join the rows: lanes of one column quad in a wave, then the waves
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int d = CQ; d < 64; d *= 2) y[e] += __shfl_xor(y[e], d, 64);
    }
    if (l < CQ) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sy[p][w][4 * cq + e] = y[e];
    }
    lds_barrier();
    if (threadIdx.x < CQ) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int x = 4 * cq + e;
        y[e] = (sy[p][0][x] + sy[p][1][x]) + (sy[p][2][x] + sy[p][3][x]);
      }
      st4<T>(reinterpret_cast<T*>(a.o) + (int64_t)t * a.os + h * V + 4 * cq, y);
    }
  }
  if (a.ht) {
#pragma unroll
    for (int i = 0; i < NR; ++i) *reinterpret_cast<f32x4*>(a.ht + st + (int64_t)(r0 + RP * i) * V) = S[i];
  }
}

// the (type, K, V) variants of a kernel
template <typename F>
hipError_t decay_kv(const DecayArgs& a, bool f32, F&& f) {
  auto dim = [](int d, auto&& g) -> hipError_t {
    if (d == 32) return g(std::integral_constant<int, 32>{});
    if (d == 64) return g(std::integral_constant<int, 64>{});
    if (d == 128) return g(std::integral_constant<int, 128>{});
    return hipErrorInvalidValue;
  };
  return dim(a.K, [&](auto k) { return dim(a.V, [&](auto v) { return f32 ? f(float{}, k, v) : f(bf16{}, k, v); }); });
}
}  // namespace

hipError_t launch_decay_state(const DecayArgs& a, bool f32, int dirs, hipStream_t s) {
  return decay_kv(a, f32, [&](auto t, auto k, auto v) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value, V = decltype(v)::value;
    REWY_LAUNCH((k_decay_state<T, K, V>), dim3(a.nslot * a.H, dirs == 3 ? 2 : 1), dim3((state_threads<T, V>())), s, a, dirs);
    return hipGetLastError();
  });
}
hipError_t launch_decay_pass(const DecayArgs& a, int dirs, hipStream_t s) {
  REWY_LAUNCH(k_decay_pass, dim3(a.seq.N * a.H, (a.K * a.V + 1023) / 1024, dirs == 3 ? 2 : 1), dim3(256), s, a, dirs);
  return hipGetLastError();
}
hipError_t launch_decay_fwd(const DecayArgs& a, bool f32, hipStream_t s) {
  return decay_kv(a, f32, [&](auto t, auto k, auto v) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value, V = decltype(v)::value;
    REWY_LAUNCH((k_decay_fwd<T, K, V>), dim3(a.nslot * a.H), dim3(walk_threads<T, V>()), s, a);
    return hipGetLastError();
  });
}
hipError_t launch_decay_bwd(const DecayArgs& a, bool f32, hipStream_t s) {
  return decay_kv(a, f32, [&](auto t, auto k, auto v) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value, V = decltype(v)::value;
    REWY_LAUNCH((k_decay_bwd<T, K, V>), dim3(3 * a.nslot * a.H), dim3(walk_threads<T, std::max(K, V)>()), s, a);
    return hipGetLastError();
  });
}
hipError_t launch_decay_sum(const DecayArgs& a, bool f32, hipStream_t s) {
  const int64_t n = (int64_t)a.seq.total * a.G * std::max(a.K, a.V) / 4;
  const dim3 grid((unsigned)((n + 255) / 256), 2);
  if (f32) REWY_LAUNCH((k_decay_sum<float>), grid, dim3(256), s, a);
  else REWY_LAUNCH((k_decay_sum<bf16>), grid, dim3(256), s, a);
  return hipGetLastError();
}
hipError_t launch_decay_recurrent(const DecayArgs& a, bool f32, hipStream_t s) {
  return decay_kv(a, f32, [&](auto t, auto k, auto v) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value, V = decltype(v)::value;
    REWY_LAUNCH((k_decay_recurrent<T, K, V>), dim3(a.seq.N * a.H), dim3(256), s, a);
    return hipGetLastError();
  });
}

}  // namespace rewy
