// Selective state space scan, forward: the local end states of the segments,
// the pass that joins them, and the walk that forms y; and the token-serial
// form.
#include "ssm.hpp"

namespace rewy {

namespace {

// What every walk of a call reads and no walk should form again.  Workgroups < nblk:
// C B^T of the chunks and groups, one wave for each of the lower triangle's ten 16 x 16
// blocks, as C fragments shared by the heads of the group; forward: rows j in slot
// order, columns i (what the coefficients' rows are made of); backward: rows i, columns
// j.  The others: the gates, one wave per chunk and head, lane t its token.  8192 x 32 heads,
// K = 128: 7 us, most of it latency.
template <typename T, int K>
__global__ __launch_bounds__(256) void k_ssm_prep(SsmArgs a, int nblk, int bwd) {
  const int t = lane_id(), w = wave_id();
  if ((int)blockIdx.x < nblk) {
    const int wb = blockIdx.x * 4 + w, wk = wb / 10, cslot = wk / a.G, grp = wk - cslot * a.G;
    if (cslot >= a.nchunk) return;
    const Piece pc = find_piece(a.seq, cslot, CH);
    const int tok = pc.bos + pc.k * CH, len = min(CH, pc.eos - tok);
    if (!pc.on || len <= 0) return;
    const T* bp = reinterpret_cast<const T*>(a.b) + (int64_t)tok * a.bs + grp * K;
    const T* cp = reinterpret_cast<const T*>(a.c) + (int64_t)tok * a.cs + grp * K;
    const GBuf gb = gbuf(bp, tile_bytes<T>(len, a.bs, K)), gc = gbuf(cp, tile_bytes<T>(len, a.cs, K));
    int I, J;
    tri_block(wb - wk * 10, I, J);
    const int r = t & 15, k0 = VEC<T> * (t >> 4);
    const int i = 16 * I + (bwd ? slot_row<T>(r) : r), j = 16 * J + (bwd ? r : slot_row<T>(r));
    f32x4 acc = zero4();
#pragma unroll
    for (int q = 0; q < K / KG<T>; ++q) {
      const uint4 bf = gld16(gb, (uint32_t)((j * a.bs + k0 + q * KG<T>) * (int64_t)sizeof(T)));
      const uint4 cf = gld16(gc, (uint32_t)((i * a.cs + k0 + q * KG<T>) * (int64_t)sizeof(T)));
      if (bwd) mma16B<T>(acc, cf, bf);
      else mma16B<T>(acc, bf, cf);
    }
    reinterpret_cast<f32x4*>(a.cb)[(int64_t)wb * 64 + t] = acc;
    return;
  }
  const int wk = (blockIdx.x - nblk) * 4 + w;
  if (wk >= a.nchunk * a.H) return;
  const int cslot = wk / a.H, h = wk - cslot * a.H;
  const Piece pc = find_piece(a.seq, cslot, CH);
  const int tok = pc.bos + pc.k * CH, len = min(CH, pc.eos - tok);
  if (!pc.on || len <= 0) return;
  Gate r;
  r.dt = 0.f;
  if (t < len) r.dt = softplus_full(ld_beta(a.dt, a.dt_f32, (int64_t)(tok + t) * a.H + h) + gate_bias(a, h));
  double p = -exp((double)a.a_log[h]) * 1.4426950408889634 * (double)r.dt;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double u = __shfl_up(p, d, 64);
    if (t >= d) p += u;
  }
  r.G = (float)p;
  r.Glo = (float)(p - (double)r.G);
  r.E = (float)(__shfl(p, 63, 64) - p);
  reinterpret_cast<f32x4*>(a.gates)[(int64_t)wk * CH + t] = f32x4{r.dt, r.G, r.Glo, r.E};
}

// Local state of one segment and HB heads: forward (dir 0), from zero, all but a
// sequence's last segment; reverse (dir 1), the adjoint that the segment's own
// tokens send to the state that enters it, all but the first.  Wave w holds 16 columns
// of one head's state.  8192 x 32 heads, K = V = 128 in segments of 512: x read and 31 MB
// of states written, 34 us (3.0 TB/s).  Both directions of K = 128, V = 64: 35 us.
template <typename T, int K, int V, int HB>
__global__ __launch_bounds__(4 * HB * V, 2) void k_ssm_state(SsmArgs a) {
  constexpr int CW = HB * V, CT = 1, NTH = 4 * CW, LK = pitch<T>(K), LV = pitch<T>(CW);
  constexpr int NQ = CH / KG<T>, NT = K / 16;
  __shared__ __align__(16) T sk[CH * LK];
  __shared__ __align__(16) T su[CH * LV];
  __shared__ __align__(16) float sal[HB][CH];
  __shared__ float sdec[HB];
  const int dir = blockIdx.y;
  const int nhb = head_blocks(a, HB), wk = xcd_range(blockIdx.x, a.nslot * nhb), slot = wk / nhb, hb = wk - slot * nhb;
  const Piece pc = find_piece(a.seq, slot, a.seg);
  if (!pc.on) return;
  const int t0 = pc.bos + pc.k * a.seg, t1 = min(t0 + a.seg, pc.eos);
  if (dir == 0 ? t1 >= pc.eos : pc.k == 0) return;
  const int gb = (a.per + HB - 1) / HB, grp = hb / gb, h0 = grp * a.per + (hb - grp * gb) * HB;
  const int nh = min(HB, (grp + 1) * a.per - h0);  // heads of this block
  const int nch = (t1 - t0 + CH - 1) / CH, w = wave_id(), l = lane_id(), hw = 16 * CT * w / V;
  const int cbase = slot_base(a.seq, pc.n, CH) + pc.k * (a.seg / CH);
  f32x4 S[CT][NT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int i = 0; i < NT; ++i) S[ct][i] = zero4();
  float gs = 0.f;
  TileRegs<T, CH, K, NTH> rk;
  TileRegs<T, CH, CW, NTH> ru;
  Gate gt = {};
  auto fetch = [&](int c) {
    const int ci = dir ? nch - 1 - c : c, tok = t0 + ci * CH, len = min(CH, t1 - tok);
    if (w < nh) gt = chunk_gates(a, cbase + ci, h0 + w)[l];
    load_tile<T, K, NTH>(rk, dir ? a.c : a.b, tok, dir ? a.cs : a.bs, grp * K, len, K);
    load_tile<T, CW, NTH>(ru, dir ? a.dy : a.x, tok, dir ? a.ys : a.xs, h0 * V, len, nh * V);
  };
  fetch(0);
  for (int c = 0; c < nch; ++c) {
    rk.store(sk, LK, threadIdx.x);
    ru.store(su, LV, threadIdx.x);
    if (w < nh) {
      sal[w][slot_of<T>(l)] = dir ? fexp2(gt.G) : fexp2(gt.E) * gt.dt;
      if (l == 63) sdec[w] = fexp2(gt.G);
      gs += gt.G;
    }
    lds_barrier();
    if (c + 1 < nch) fetch(c + 1);
    uint4 ut[CT][NQ];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int q = 0; q < NQ; ++q) ut[ct][q] = frag_col<T>(su, LV, q * KG<T>, 16 * (CT * w + ct));
    state_update<T, K, CT, SPLIT<T>>(S, sk, LK, ut, sal[hw], sdec[hw]);
    lds_barrier();
  }
  // (forward and reverse sum the same decays, each for the segments it takes)
  if (w < nh && l == 63) a.gsum[((int64_t)dir * a.nslot + slot) * a.H + h0 + w] = gs;
  if (hw >= nh) return;
  float* o = (dir ? a.sr : a.sf) + ((int64_t)slot * a.H + h0 + hw) * K * V + 16 * CT * w - hw * V + (l & 15);
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[(16 * nt + 4 * (l >> 4) + i) * V + 16 * ct] = S[ct][nt][i];
}

// In place: the local states of a sequence's segments become the states that
// enter them (forward; from h0) or the adjoints of the states that leave them
// (reverse; from dht).  Bound by HBM (the 15 states of 64 KB and 32 heads above:
// 11.7 us, 5.6 TB/s).
__global__ __launch_bounds__(256) void k_ssm_pass(SsmArgs a) {
  const int kv = a.K * a.V, n = blockIdx.x / a.H, h = blockIdx.x - n * a.H, dir = blockIdx.z;
  const int e = (blockIdx.y * 256 + threadIdx.x) * 4;
  if (e >= kv) return;
  int bos, eos;
  seq_range(a.seq, n, bos, eos);
  const int base = slot_base(a.seq, n, a.seg), ns = (eos - bos + a.seg - 1) / a.seg;
  const float* init = dir ? a.dht : a.h0;
  float* st = dir ? a.sr : a.sf;
  f32x4 S = zero4();
  if (init) S = *reinterpret_cast<const f32x4*>(init + ((int64_t)n * a.H + h) * kv + e);
  for (int i = 0; i < ns; ++i) {
    const int k = dir ? ns - 1 - i : i;
    const int64_t sl = (int64_t)(base + k) * a.H + h;
    f32x4* p = reinterpret_cast<f32x4*>(st + sl * kv + e);
    if (i + 1 < ns) {
      const f32x4 loc = *p;
      const float d = fexp2(a.gsum[(int64_t)dir * a.nslot * a.H + sl]);
      *p = S;
#pragma unroll
      for (int j = 0; j < 4; ++j) S[j] = d * S[j] + loc[j];
    } else {
      *p = S;
    }
  }
}

// The walk of one segment and HB heads.  Wave w owns 16 columns of y and of the
// state (with CT = 2, 32: a fragment read from LDS serves two products).  A chunk's
// coefficients M (one 64 x 64 matrix a head, from C B^T and the gates, which are a
// chunk ahead) are formed block by block by all waves and shared through LDS.  Two
// barriers a chunk: tiles and M complete; tiles and M free.  y leaves through
// the x tile, whole rows at a time.
// With bf16 operands M and the entering state are rounded to bf16 once each as operands of
// y's products, which y's own rounding covers (8192 x 32 heads, K = V = 128: y is off by
// 1.8e-3 in norm, by 1.7e-3 if it is formed in 32 bits and only rounded at the end); two
// pieces each would double those products.  The carried state meets no such rounding.
// The size above: 80 us, 225 MB (2.8 TB/s; 18 MB of it registers that do not fit) and 38
// GFLOP (470 TFLOP/s): two waves a SIMD, whose matrix instructions, coefficients and LDS
// traffic leave each other gaps (66 us if the state's updates come in two pieces,
// ssm.hpp).  V = 64: 46 us; fp32, 9000 x 16 heads, K = V = 64 in 16 sequences: 63 us,
// where the fp32 matrix instructions take half of the time.
template <typename T, int K, int V, int HB, int CT>
__global__ __launch_bounds__(4 * HB * V / CT, 2) void k_ssm_fwd(SsmArgs a) {
  constexpr int CW = HB * V, NTH = 4 * CW / CT, NW = NTH / 64;
  constexpr int LK = pitch<T>(K), LV = pitch<T>(CW), LM = pitch<T>(CH);
  constexpr int NQ = CH / KG<T>, NT = K / 16, KQ = K / KG<T>, NB = (10 + NW - 1) / NW;
  __shared__ __align__(16) T sb[CH * LK];
  __shared__ __align__(16) T sc[CH * LK];  // columns in the slot order of frag_acc
  __shared__ __align__(16) T sx[CH * LV];
  __shared__ __align__(16) T sm[HB][CH * LM];  // columns in slot order
  // gates of each head: by token, and (t) in slot order
  __shared__ __align__(16) float sG[2][HB][CH], sGl[2][HB][CH], tG[2][HB][CH], tGl[2][HB][CH], tdt[2][HB][CH];
  __shared__ __align__(16) float seq[2][HB][CH], sal[2][HB][CH];
  __shared__ float sdec[2][HB];
  __shared__ int sodd;  // the last chunk, counted from 1, whose x tile holds an infinity or NaN
  const int nhb = head_blocks(a, HB), wk = xcd_range(blockIdx.x, a.nslot * nhb), slot = wk / nhb, hb = wk - slot * nhb;
  const Piece pc = find_piece(a.seq, slot, a.seg);
  if (!pc.on) return;
  const int t0 = pc.bos + pc.k * a.seg, t1 = min(t0 + a.seg, pc.eos);
  const int gb = (a.per + HB - 1) / HB, grp = hb / gb, h0 = grp * a.per + (hb - grp * gb) * HB;
  const int nh = min(HB, (grp + 1) * a.per - h0);  // heads of this block
  const int nch = (t1 - t0 + CH - 1) / CH, w = wave_id(), l = lane_id(), g4 = l >> 4, r = l & 15;
  const int hw = 16 * CT * w / V, h = min(h0 + hw, h0 + nh - 1), pc0 = 16 * CT * w - hw * V;  // the wave's head, its columns
  const bool live = hw < nh;
  const int cbase = slot_base(a.seq, pc.n, CH) + pc.k * (a.seg / CH);
  const float D = a.d ? a.d[h] : 0.f;
  const int64_t head = ((int64_t)pc.n * a.H + h) * K * V + pc0 + r;
  // (an empty sequence has no segment of its own: its state is given through)
  const float* init = a.two && nch > 0 ? a.sf + ((int64_t)slot * a.H + h) * K * V + pc0 + r
                      : a.h0           ? a.h0 + head
                                       : nullptr;
  f32x4 S[CT][NT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[ct][nt][i] = init ? init[(16 * nt + 4 * g4 + i) * V + 16 * ct] : 0.f;

  TileRegs<T, CH, K, NTH> rb, rc;
  TileRegs<T, CH, CW, NTH> rx;
  f32x4 rcb[NB];
  auto fetch = [&](int c) {
    const int tok = t0 + c * CH, len = min(CH, t1 - tok);
    load_tile<T, K, NTH>(rb, a.b, tok, a.bs, grp * K, len, K);
    load_tile<T, K, NTH>(rc, a.c, tok, a.cs, grp * K, len, K);
    load_tile<T, CW, NTH>(rx, a.x, tok, a.xs, h0 * V, len, nh * V);
#pragma unroll
    for (int b = 0; b < NB; ++b)
      rcb[b] = reinterpret_cast<const f32x4*>(a.cb)[((int64_t)((cbase + c) * a.G + grp) * 10 + min(b * NW + w, 9)) * 64 + l];
  };
  auto put_tiles = [&](int c) {
    if (tile_not_finite<T, CW, NTH>(rx)) sodd = c + 1;
    rb.store(sb, LK, threadIdx.x);
    store_acc_order<T, K, NTH>(rc, sc, LK);
    rx.store(sx, LV, threadIdx.x);
  };
  auto put_gates = [&](const Gate& gt, int p) {
    const int sl = slot_of<T>(l);
    const float eG = fexp2(gt.G);
    sG[p][w][l] = tG[p][w][sl] = gt.G;
    sGl[p][w][l] = tGl[p][w][sl] = gt.Glo;
    tdt[p][w][sl] = gt.dt;
    seq[p][w][l] = eG;
    sal[p][w][sl] = fexp2(gt.E) * gt.dt;
    if (l == 63) sdec[p][w] = eG;
  };
  // coefficients of the chunk whose C B^T is in rcb, gates in set p: block (I, J) as its
  // transpose (rows j in slot order, columns i), so that a lane holds four neighbours
  // of a row of M
  auto put_coefficients = [&](int p) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int blk = b * NW + w;
      if (blk < 10) {
        int I, J;
        tri_block(blk, I, J);
        const int i = 16 * I + r, sl = slot_base4<T>(J, g4);
#pragma unroll
        for (int k = 0; k < HB; ++k) {
          const float Gi = sG[p][k][i], Gil = sGl[p][k][i];
          const f32x4 Gj = *reinterpret_cast<const f32x4*>(tG[p][k] + sl), Gjl = *reinterpret_cast<const f32x4*>(tGl[p][k] + sl);
          const f32x4 dj = *reinterpret_cast<const f32x4*>(tdt[p][k] + sl);
          f32x4 m;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m[e] = 16 * J + slot_row<T>(4 * g4 + e) <= i ? rcb[b][e] * fexp2((Gi - Gj[e]) + (Gil - Gjl[e])) * dj[e] : 0.f;
          st4<T>(sm[k] + i * LM + sl, m);
        }
      }
    }
  };
  const bool gater = w < nh;
  Gate gt = {};
  if (nch > 0) {
    fetch(0);
    if (gater) {
      put_gates(chunk_gates(a, cbase, h0 + w)[l], 0);
      if (nch > 1) put_gates(chunk_gates(a, cbase + 1, h0 + w)[l], 1);
    }
    // a pair of blocks above the diagonal lies inside a contraction of 32: zeros, written once
    for (int i = threadIdx.x; i < HB * CH * LM; i += NTH) sm[0][i] = (T)0.f;
    if (threadIdx.x == 0) sodd = 0;
    lds_barrier();
    put_coefficients(0);
    put_tiles(0);
  }
  for (int c = 0; c < nch; ++c) {
    const int tok = t0 + c * CH, len = min(CH, t1 - tok), p = c & 1;
    lds_barrier();  // tiles, coefficients and gates complete
    if (c + 1 < nch) fetch(c + 1);
    if (gater && c + 2 < nch) gt = chunk_gates(a, cbase + c + 2, h0 + w)[l];
    // An infinity or NaN of x would reach earlier tokens through the product's zeros
    // right of the diagonal: it leaves the tile (each wave its own columns), and y from
    // its token on and the column's state are set to NaN below.
    const bool odd = __builtin_amdgcn_readfirstlane(sodd) == c + 1;
    int first[CT];
    if (odd) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        T* xc = sx + 16 * (CT * w + ct) + r;
        first[ct] = CH;
#pragma unroll 1
        for (int j = CH - 4 + g4; j >= 0; j -= 4)
          if (!(fabsf((float)xc[j * LV]) <= 3.4028235e38f)) {
            xc[j * LV] = (T)0.f;
            first[ct] = j;
          }
        first[ct] = min(first[ct], __shfl_xor(first[ct], 16, 64));
        first[ct] = min(first[ct], __shfl_xor(first[ct], 32, 64));
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // entering state: Y^T = S^T C^T, columns scaled by exp(G)
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
        const uint4 cf = frag_row<T>(sc, LK, 16 * I, q * KG<T>);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) mma16B<T>(Y[ct][I], sf[ct][0], cf);
      }
    }
    T* xw = sx + r * LV + 16 * CT * w + 4 * g4;  // the wave's own columns of the x tile
#pragma unroll
    for (int I = 0; I < 4; ++I) {
      const float e = seq[p][hw][16 * I + r];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const f32x4 xv = ld4<T>(xw + 16 * I * LV + 16 * ct);
#pragma unroll
        for (int i = 0; i < 4; ++i) Y[ct][I][i] = Y[ct][I][i] * e + D * xv[i];
      }
    }
    uint4 xt[CT][NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) xt[ct][q] = frag_col<T>(sx, LV, q * KG<T>, 16 * (CT * w + ct));
#pragma unroll
      for (int I = 0; I < 4; ++I)
        if (q * KG<T> <= 16 * I) {
          const uint4 mf = frag_row<T>(sm[hw], LM, 16 * I, q * KG<T>);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) mma16B<T>(Y[ct][I], xt[ct][q], mf);
        }
    }
    // (read above, and by no other wave)
#pragma unroll
    for (int I = 0; I < 4; ++I)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) st4<T>(xw + 16 * I * LV + 16 * ct, Y[ct][I]);
    state_update<T, K, CT, SPLIT<T>>(S, sb, LK, xt, sal[p][hw], sdec[p][hw]);
    if (odd) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        T* yc = sx + 16 * (CT * w + ct) + r;
#pragma unroll 1
        for (int j = first[ct] + g4; j < CH; j += 4) yc[j * LV] = (T)__builtin_nanf("");
        if (first[ct] < CH) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[ct][nt][i] = __builtin_nanf("");
        }
      }
    }
    lds_barrier();  // tiles and coefficients free, y complete
    {
      // each thread takes y from where its pieces of the next x tile go
      using TR = TileRegs<T, CH, CW, NTH>;
      const GBuf gy = gbuf(reinterpret_cast<T*>(a.y) + (int64_t)tok * a.ys + h0 * V, tile_bytes<T>(len, a.ys, nh * V));
#pragma unroll
      for (int j = 0; j < TR::N; ++j) {
        const int idx = threadIdx.x + j * NTH, row = idx / TR::PER, col = (idx - row * TR::PER) * TR::VEC;
        if (idx < TR::TOTAL)
          gst16(gy, col < nh * V ? (uint32_t)((row * a.ys + col) * (int64_t)sizeof(T)) : OOB,
                *reinterpret_cast<const uint4*>(sx + row * LV + col));
      }
    }
    if (c + 1 < nch) {
      put_tiles(c + 1);
      put_coefficients(p ^ 1);
    }
    if (gater && c + 2 < nch) put_gates(gt, p);
  }
  if (a.ht && live && t1 >= pc.eos) {
    float* o = a.ht + head;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[(16 * nt + 4 * g4 + i) * V + 16 * ct] = S[ct][nt][i];
  }
}

// Token by token: one workgroup per sequence and head, the state in registers,
// four neighbouring columns of K V / 1024 rows a thread.  For one new token it
// costs the state's bytes, read and written once: 64 sequences of 32 heads, K = 128, V =
// 64: 134 MB in 23.6 us (5.7 TB/s).
template <typename T, int K, int V>
__global__ __launch_bounds__(256) void k_ssm_recurrent(SsmArgs a) {
  constexpr int CQ = V / 4, RP = 256 / CQ, NR = K / RP;  // column quads, rows side by side, rows of a thread
  __shared__ __align__(16) float sb[K], sc[K];
  __shared__ float sy[4][V];
  const int n = blockIdx.x / a.H, h = blockIdx.x - n * a.H, grp = h / a.per;
  const int cq = threadIdx.x % CQ, r0 = threadIdx.x / CQ, w = wave_id(), l = lane_id();
  int bos, eos;
  seq_range(a.seq, n, bos, eos);
  const float A2 = -expf(a.a_log[h]) * LOG2E, bias = gate_bias(a, h), D = a.d ? a.d[h] : 0.f;
  const int64_t st = ((int64_t)n * a.H + h) * K * V + 4 * cq;
  f32x4 S[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i)
    S[i] = a.h0 ? *reinterpret_cast<const f32x4*>(a.h0 + st + (int64_t)(r0 + RP * i) * V) : zero4();
  for (int t = bos; t < eos; ++t) {
    const T* bp = reinterpret_cast<const T*>(a.b) + (int64_t)t * a.bs + grp * K;
    const T* cp = reinterpret_cast<const T*>(a.c) + (int64_t)t * a.cs + grp * K;
    const f32x4 x = ld4<T>(reinterpret_cast<const T*>(a.x) + (int64_t)t * a.xs + h * V + 4 * cq);
    const float dt = softplus_full(ld_beta(a.dt, a.dt_f32, (int64_t)t * a.H + h) + bias), dec = fexp2(A2 * dt);
    for (int i = threadIdx.x; i < 2 * K; i += 256) {
      if (i < K) sb[i] = dt * (float)bp[i];
      else sc[i - K] = (float)cp[i - K];
    }
    lds_barrier();
    f32x4 y = zero4();
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const float bv = sb[r0 + RP * i], cv = sc[r0 + RP * i];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        S[i][e] = dec * S[i][e] + bv * x[e];
        y[e] += cv * S[i][e];
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
      for (int e = 0; e < 4; ++e) sy[w][4 * cq + e] = y[e];
    }
    lds_barrier();
    if (threadIdx.x < CQ) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = 4 * cq + e;
        y[e] = (sy[0][p] + sy[1][p]) + (sy[2][p] + sy[3][p]) + D * x[e];
      }
      st4<T>(reinterpret_cast<T*>(a.y) + (int64_t)t * a.ys + h * V + 4 * cq, y);
    }
  }
  if (a.ht) {
#pragma unroll
    for (int i = 0; i < NR; ++i) *reinterpret_cast<f32x4*>(a.ht + st + (int64_t)(r0 + RP * i) * V) = S[i];
  }
}

}  // namespace

hipError_t launch_ssm_prep(const SsmArgs& a, bool f32, bool bwd, hipStream_t s) {
  return ssm_kv(a.K, 32, f32, [&](auto t, auto k, auto) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value;
    const int nblk = (int)(((int64_t)a.nchunk * a.G * 10 + 3) / 4), ngate = (a.nchunk * a.H + 3) / 4;
    REWY_LAUNCH((k_ssm_prep<T, K>), dim3(nblk + ngate), dim3(256), s, a, nblk, (int)bwd);
    return hipGetLastError();
  });
}
int ssm_head_blocks(const SsmArgs& a, int hb) { return a.G * ((a.per + hb - 1) / hb); }

hipError_t launch_ssm_state(const SsmArgs& a, bool f32, bool both, hipStream_t s) {
  return ssm_kv_heads<128>(a, f32, [&](auto t, auto k, auto v, auto hb) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value, V = decltype(v)::value, HB = decltype(hb)::value;
    const dim3 grid(a.nslot * ssm_head_blocks(a, HB), both ? 2 : 1), block(4 * HB * V);
    REWY_LAUNCH((k_ssm_state<T, K, V, HB>), grid, block, s, a);
    return hipGetLastError();
  });
}
hipError_t launch_ssm_pass(const SsmArgs& a, bool both, hipStream_t s) {
  REWY_LAUNCH(k_ssm_pass, dim3(a.seq.N * a.H, (a.K * a.V + 1023) / 1024, both ? 2 : 1), dim3(256), s, a);
  return hipGetLastError();
}
hipError_t launch_ssm_fwd(const SsmArgs& a, bool f32, hipStream_t s) {
  return ssm_kv_heads<128>(a, f32, [&](auto t, auto k, auto v, auto hb) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value, V = decltype(v)::value, HB = decltype(hb)::value;
    constexpr int CT = V == 128 ? 2 : 1;
    const dim3 grid(a.nslot * ssm_head_blocks(a, HB)), block(4 * HB * V / CT);
    REWY_LAUNCH((k_ssm_fwd<T, K, V, HB, CT>), grid, block, s, a);
    return hipGetLastError();
  });
}
hipError_t launch_ssm_recurrent(const SsmArgs& a, bool f32, hipStream_t s) {
  return ssm_kv(a.K, a.V, f32, [&](auto t, auto k, auto v) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value, V = decltype(v)::value;
    REWY_LAUNCH((k_ssm_recurrent<T, K, V>), dim3(a.seq.N * a.H), dim3(256), s, a);
    return hipGetLastError();
  });
}

}  // namespace rewy
