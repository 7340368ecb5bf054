// Selective state space scan, backward.  With dS the adjoint of the state that
// leaves a chunk, v = dt x and M0_ij = exp(G_i - G_j) (C_i . B_j), i >= j:
//   dS_in = exp(G_L) dS + sum_i exp(G_i) C_i dy_i^T
//   dv_j  = sum_i M0_ij dy_i + exp(G_L - G_j) dS^T B_j,     dx = dt dv + D dy
//   W_ij  = exp(G_i - G_j) (dy_i . x_j) dt_j
//   dC_i  = sum_heads [ sum_j W_ij B_j + exp(G_i) S_in dy_i ]
//   dB_j  = sum_heads [ sum_i W_ij C_i + exp(G_L - G_j) dt_j dS x_j ]
// and the decay's gradient from r_i = dy_i . (y_i - D x_i) and c_j = x_j . dv_j,
//   dg_t = sum_{i >= t} (r_i - dt_i c_i) + <S, dS> behind the last i,
//   d raw_t = (c_t - exp(A_log) dg_t) sigmoid(raw_t + dt_bias),   dA_log = sum dg_t g_t.
// r and c split into parts inside the chunk (formed where W is) and parts through
// the states (formed by the walks, whose states are fp32); the states that the
// 16-bit outputs need are handed over in the operand type, and everything that
// sums into a parameter's gradient stays fp32.
#include "ssm.hpp"

namespace rewy {

namespace {

// Walks of one segment and HB heads, both directions (blockIdx.y).  Forward: the
// state that enters each chunk goes to hs, and rx_t = exp(G_t) dy_t . (S_in^T
// C_t); reverse: the adjoint that leaves each chunk goes to hd, and cx_t =
// exp(G_L - G_t) x_t . (dS^T B_t).  Wave w holds 16 columns of one head.  Heads of 64
// columns in workgroups of their own (two a CU, which fill each other's waits: 85 us in a row
// of calls, two heads in one workgroup 93).  8192 x 32 heads, K = 128, V = 64, alone: 97 us, 90 at
// least; 321 MB (134 of them the handed-over states; 3.3 TB/s) and 52 GFLOP, as the states
// meet the 16-bit operands in three pieces (540 TFLOP/s).
template <typename T, int K, int V, int HB>
__global__ __launch_bounds__(4 * HB * V, 2) void k_ssm_walk(SsmArgs a) {
  constexpr int CW = HB * V, CT = 1, NTH = 4 * CW, NW = NTH / 64;
  constexpr int LK = pitch<T>(K), LV = pitch<T>(CW), NQ = CH / KG<T>;
  constexpr int NT = K / 16, KQ = K / KG<T>, NS = SPLIT<T>, WH = V / (16 * CT);  // waves of a head
  __shared__ __align__(16) T sk[CH * LK];  // update: B (forward), C (reverse)
  __shared__ __align__(16) T sq[CH * LK];  // probe: C, B (columns in the slot order of frag_acc)
  __shared__ __align__(16) T su[CH * LV];  // update: x, dy
  __shared__ __align__(16) T sp[CH * LV];  // probe: dy, x
  __shared__ __align__(16) float sal[HB][CH], sdot[NW][CH];
  __shared__ float sdec[HB];
  __shared__ double sred[NW];
  const int dir = blockIdx.y;
  const int nhb = head_blocks(a, HB), wk = xcd_range(blockIdx.x, a.nslot * nhb), slot = wk / nhb, hb = wk - slot * nhb;
  const Piece pc = find_piece(a.seq, slot, a.seg);
  if (!pc.on) return;
  const int t0 = pc.bos + pc.k * a.seg, t1 = min(t0 + a.seg, pc.eos);
  const int gb = (a.per + HB - 1) / HB, grp = hb / gb, h0 = grp * a.per + (hb - grp * gb) * HB;
  const int nh = min(HB, (grp + 1) * a.per - h0);  // heads of this block
  const int nch = (t1 - t0 + CH - 1) / CH, w = wave_id(), l = lane_id(), g4 = l >> 4, r = l & 15;
  const int hw = w / WH, h = min(h0 + hw, h0 + nh - 1), pc0 = 16 * CT * w - hw * V;
  const bool live = hw < nh;
  const int cbase = slot_base(a.seq, pc.n, CH) + pc.k * (a.seg / CH);
  const int64_t seqst = ((int64_t)pc.n * a.H + h) * K * V + pc0 + r;
  const int64_t segst = ((int64_t)slot * a.H + h) * K * V + pc0 + r;
  const float* given = dir ? a.dht : a.h0;
  // (an empty sequence has no segment of its own: its state is given through)
  const float* init = a.two && nch > 0 ? (dir ? a.sr : a.sf) + segst : given ? given + seqst : nullptr;
  f32x4 S[CT][NT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[ct][nt][i] = init ? init[(16 * nt + 4 * g4 + i) * V + 16 * ct] : 0.f;
  TileRegs<T, CH, K, NTH> rk, rq;
  TileRegs<T, CH, CW, NTH> ru, rp;
  Gate gt = {};
  auto fetch = [&](int c) {
    const int ci = dir ? nch - 1 - c : c, tok = t0 + ci * CH, len = min(CH, t1 - tok);
    if (w < nh) gt = chunk_gates(a, cbase + ci, h0 + w)[l];
    load_tile<T, K, NTH>(rk, dir ? a.c : a.b, tok, dir ? a.cs : a.bs, grp * K, len, K);
    load_tile<T, K, NTH>(rq, dir ? a.b : a.c, tok, dir ? a.bs : a.cs, grp * K, len, K);
    load_tile<T, CW, NTH>(ru, dir ? a.dy : a.x, tok, dir ? a.ys : a.xs, h0 * V, len, nh * V);
    load_tile<T, CW, NTH>(rp, dir ? a.x : a.dy, tok, dir ? a.xs : a.ys, h0 * V, len, nh * V);
  };
  if (nch > 0) fetch(0);
  T* hand = reinterpret_cast<T*>(dir ? a.hd : a.hs);
  for (int c = 0; c < nch; ++c) {
    const int ci = dir ? nch - 1 - c : c, tok = t0 + ci * CH, len = min(CH, t1 - tok);
    rk.store(sk, LK, threadIdx.x);
    store_acc_order<T, K, NTH>(rq, sq, LK);
    ru.store(su, LV, threadIdx.x);
    rp.store(sp, LV, threadIdx.x);
    float be = 0.f;
    if (w < nh) {
      const float eG = fexp2(gt.G), eE = fexp2(gt.E);
      sal[w][slot_of<T>(l)] = dir ? eG : eE * gt.dt;
      be = dir ? eE : eG;
      if (l == 63) sdec[w] = eG;
    }
    lds_barrier();
    if (c + 1 < nch) fetch(c + 1);
    if (live) {
      T* hp = hand + (((int64_t)(cbase + ci) * a.H + h) * (V / 16) + pc0 / 16) * (K * 16) + l * 4;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) st4<T>(hp + ct * K * 16 + nt * 256, S[ct][nt]);
    }
    // The probe's sums decide the decay gradient's accuracy (its terms cancel), so
    // they are kept in two accumulators, which halves the roundings that meet the large
    // part: bf16: the leading piece of the state apart from the others; fp32: every
    // other step.
    f32x4 Y[2][4];
#pragma unroll
    for (int I = 0; I < 4; ++I) Y[0][I] = Y[1][I] = zero4();
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      uint4 sf[NS];
      frag_acc<T, NS>(sf, S[0], q);
#pragma unroll
      for (int I = 0; I < 4; ++I) {
        const uint4 qf = frag_row<T>(sq, LK, 16 * I, q * KG<T>);
#pragma unroll
        for (int s = NS - 1; s >= 0; --s) mma16B<T>(Y[NS > 1 ? s > 0 : q & 1][I], sf[s], qf);
      }
    }
    // Y[.][I] holds columns t = 16 I + r, rows (columns of the state) 4 g4 + i
#pragma unroll
    for (int I = 0; I < 4; ++I) {
      const f32x4 u = ld4<T>(sp + (16 * I + r) * LV + 16 * w + 4 * g4);
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = Y[0][I][i] * u[i] + Y[1][I][i] * u[i];
      const float d = rows_sum((v[0] + v[1]) + (v[2] + v[3]));
      if (g4 == I) sdot[w][16 * I + r] = d;
    }
    uint4 ut[CT][NQ];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int q = 0; q < NQ; ++q) ut[ct][q] = frag_col<T>(su, LV, q * KG<T>, 16 * (CT * w + ct));
    state_update<T, K, CT, NS>(S, sk, LK, ut, sal[hw], sdec[hw]);
    lds_barrier();  // dots complete, tiles free
    if (w < nh && l < len) {
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < WH; ++i) d += sdot[w * WH + i][l];
      ((dir ? a.cx : a.rx) + (int64_t)(h0 + w) * a.seq.total)[tok + l] = be * d;
    }
  }
  if (dir == 0) {
    if constexpr (!std::is_same_v<T, bf16>) return;  // (k_ssm_gate needs no E)
    // E = <S, dS> at the segment's end
    const float* adj = a.two && nch > 0 ? a.sr + segst : a.dht ? a.dht + seqst : nullptr;
    double d = 0.;
    if (adj) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) d += (double)S[ct][nt][i] * adj[(16 * nt + 4 * g4 + i) * V + 16 * ct];
    }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) d += __shfl_xor(d, m, 64);
    if (l == 0) sred[w] = d;
    lds_barrier();
    if (w < nh && l == 0) {
      d = 0.;
      for (int i = 0; i < WH; ++i) d += sred[w * WH + i];
      a.ends[(int64_t)slot * a.H + h0 + w] = d;
    }
  } else if (a.dh0 && live && pc.k == 0) {
    float* o = a.dh0 + seqst;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[(16 * nt + 4 * g4 + i) * V + 16 * ct] = S[ct][nt][i];
  }
}

// Waves of a chunk's workgroup: 16 where a wave's part fits in 128 registers (K = 64, V = 64
// and 128: 63 -> 59 and 92 -> 85 us for 8192 x 32 heads bf16, 149 -> 130 fp32), else 8 (K = 128
// spills with 16: 122 instead of 77 us; K or V = 32 has no 16 parts).
constexpr int cb_waves(int K, int V) { return K == 64 && V >= 64 ? 16 : 8; }

// One chunk, one group, a range of its heads: dx, the parts of r and c inside
// the chunk, and dB, dC summed over the heads in registers.  Wave w owns rows
// 16 (w & 3) .. + 15 of the chunk and share w >> 2 of the state rows (dB, dC) or
// of the columns (dx).  The size above, alone: 85 us, 79 at least (77 in a row of calls), 267
// MB (3.1 TB/s; the states half of them) and 16 GFLOP; one workgroup a CU, as its tiles take
// most of the LDS.
template <typename T, int K, int V>
__global__ __launch_bounds__(64 * cb_waves(K, V)) void k_ssm_chunk(SsmArgs a) {
  constexpr int NW = cb_waves(K, V), NTH = 64 * NW, LK = pitch<T>(K), LV = pitch<T>(V), LM = pitch<T>(CH), NQ = CH / KG<T>;
  constexpr int KQ = K / KG<T>, VQ = V / KG<T>, NTW = K / 4 / NW, PTW = V / 4 / NW;  // tiles of a wave
  __shared__ __align__(16) T sb[CH * LK];
  __shared__ __align__(16) T sc[CH * LK];
  __shared__ __align__(16) T sx[CH * LV];
  __shared__ __align__(16) T sy[CH * LV];  // dy
  __shared__ __align__(16) T ss[V * LK];   // S_in^T, rows placed for frag_col
  __shared__ __align__(16) T sd[V * LK];   // dS^T, the same
  __shared__ __align__(16) T sm[CH * LM];  // M0^T (columns in slot order), at the end W^T, then W
  __shared__ __align__(16) float sG[CH], sGl[CH], sdt[CH], seG[CH], seE[CH], tG[CH], tGl[CH];  // t: in slot order
  __shared__ float srp[4][CH], scp[4][CH], scd[CH], sdd[NW], shd[NW];
  const int nwork = a.nchunk * a.G * a.split;
  int wk = xcd_range(blockIdx.x, nwork);
  const int part = wk % a.split;
  wk /= a.split;
  const int grp = wk % a.G, cslot = wk / a.G;
  const Piece pc = find_piece(a.seq, cslot, CH);
  const int tok = pc.bos + pc.k * CH, len = min(CH, pc.eos - tok);
  if (!pc.on || len <= 0) return;
  const int h0 = grp * a.per + part * a.per / a.split, h1 = grp * a.per + (part + 1) * a.per / a.split;
  // (the wave's number in a scalar register: with 16 waves every one of the 128 others counts)
  const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), g4 = l >> 4, r = l & 15, tb = w & 3, sh = w >> 2;

  TileRegs<T, CH, V, NTH> rx, ry;
  TileRegs<T, V, K, NTH> rs, rd;  // pieces of the handed-over states, 16 bytes = two lanes' fragments
  Gate gt = {};
  auto fetch = [&](int h) {
    if (w == 0) gt = chunk_gates(a, cslot, h)[l];
    load_tile<T, V, NTH>(rx, a.x, tok, a.xs, h * V, len, V);
    load_tile<T, V, NTH>(ry, a.dy, tok, a.ys, h * V, len, V);
    const int64_t o = ((int64_t)cslot * a.H + h) * K * V;
    rs.load(gbuf(reinterpret_cast<const T*>(a.hs) + o, K * V * sizeof(T)), K, threadIdx.x);
    rd.load(gbuf(reinterpret_cast<const T*>(a.hd) + o, K * V * sizeof(T)), K, threadIdx.x);
  };
  // element 4 f of a handed-over state (fragment f: tile f / 64, lane f % 64) goes to
  // its place in [V][K] order
  auto put_state = [&](T* s, const TileRegs<T, V, K, NTH>& t) {
#pragma unroll
    for (int j = 0; j < TileRegs<T, V, K, NTH>::N; ++j) {
      const int idx = threadIdx.x + j * NTH;
      if (idx < TileRegs<T, V, K, NTH>::TOTAL) {
        constexpr int FP = VEC<T> / 4;  // fragments of a piece
#pragma unroll
        for (int k = 0; k < FP; ++k) {
          const int f = idx * FP + k, lane = f & 63, tile = f >> 6, nt = tile % (K / 16), pt = tile / (K / 16);
          T* p = s + slot_place<T>(16 * pt + (lane & 15)) * LK + 16 * nt + 4 * (lane >> 4);
          if constexpr (FP == 2) *reinterpret_cast<uint2*>(p) = k ? uint2{t.r[j].z, t.r[j].w} : uint2{t.r[j].x, t.r[j].y};
          else *reinterpret_cast<uint4*>(p) = t.r[j];
        }
      }
    }
  };

  {
    TileRegs<T, CH, K, NTH> rb, rc;
    load_tile<T, K, NTH>(rb, a.b, tok, a.bs, grp * K, len, K);
    load_tile<T, K, NTH>(rc, a.c, tok, a.cs, grp * K, len, K);
    rb.store(sb, LK, threadIdx.x);
    rc.store(sc, LK, threadIdx.x);
  }
  for (int i = threadIdx.x; i < CH * LM; i += NTH) sm[i] = (T)0.f;
  lds_barrier();
  // blocks (I, J) of the lower triangle: 10 over the waves.  C B^T and the sum of W over
  // the heads stay in registers (rows i = 16 I + slot_row(4 g4 + e), column j = 16 J + r).
  constexpr int NB = (10 + NW - 1) / NW;
  f32x4 cb[NB], wsum[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    wsum[b] = zero4();
    cb[b] = reinterpret_cast<const f32x4*>(a.cb)[((int64_t)(cslot * a.G + grp) * 10 + min(b * NW + w, 9)) * 64 + l];
  }
  f32x4 dC[NTW], dB[NTW];
#pragma unroll
  for (int i = 0; i < NTW; ++i) dC[i] = dB[i] = zero4();

  if (h0 < h1) fetch(h0);
  for (int h = h0; h < h1; ++h) {
    lds_barrier();  // tiles free
    rx.store(sx, LV, threadIdx.x);
    ry.store(sy, LV, threadIdx.x);
    put_state(ss, rs);
    put_state(sd, rd);
    {
      float hd = 0.f;
#pragma unroll
      for (int j = 0; j < TileRegs<T, V, K, NTH>::N; ++j) {
        float u[VEC<T>], v[VEC<T>];
        frag_get<T>(u, rs.r[j]);
        frag_get<T>(v, rd.r[j]);
        if (threadIdx.x + j * NTH < TileRegs<T, V, K, NTH>::TOTAL) {
#pragma unroll
          for (int e = 0; e < VEC<T>; ++e) hd += u[e] * v[e];
        }
      }
      hd = rows_sum(row16_sum(hd));
      if (l == 0) shd[w] = hd;
    }
    if (w == 0) {
      sG[l] = tG[slot_of<T>(l)] = gt.G;
      sGl[l] = tGl[slot_of<T>(l)] = gt.Glo;
      sdt[l] = gt.dt;
      seG[l] = fexp2(gt.G);
      seE[l] = fexp2(gt.E);
    }
    lds_barrier();
    if (h + 1 < h1) fetch(h + 1);
    float dd = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int blk = b * NW + w;
      if (blk < 10) {
        int I, J;
        tri_block(blk, I, J);
        f32x4 p = zero4();
#pragma unroll
        for (int q = 0; q < VQ; ++q)
          mma16B<T>(p, frag_row_slot<T>(sy, LV, 16 * I, q * KG<T>), frag_row<T>(sx, LV, 16 * J, q * KG<T>));
        const int sl = slot_base4<T>(I, g4), j = 16 * J + r;
        const f32x4 Gi = *reinterpret_cast<const f32x4*>(tG + sl), Gil = *reinterpret_cast<const f32x4*>(tGl + sl);
        const float Gj = sG[j], Gjl = sGl[j], dj = sdt[j];
        f32x4 m;
        float col = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 16 * I + slot_row<T>(4 * g4 + e);
          const float dec = j <= i ? fexp2((Gi[e] - Gj) + (Gil[e] - Gjl)) : 0.f;
          m[e] = cb[b][e] * dec;
          float cm = m[e] * p[e];
          if (j == i) {
            dd += p[e];
            scd[j] = cm;
            cm = 0.f;
          }
          col += cm;
          wsum[b][e] += p[e] * dec * dj;
          const float row = row16_sum(cm * dj);
          if (r == 0) srp[J][i] = row;
        }
        st4<T>(sm + j * LM + sl, m);
        col = rows_sum(col);
        if (g4 == 0) scp[I][j] = col;
      }
    }
    dd = rows_sum(row16_sum(dd));
    if (l == 0) sdd[w] = dd;
    lds_barrier();
    if (w == 0) {
      const int I = l >> 4;
      float rr = 0.f, cc = 0.f;
#pragma unroll
      for (int b = 0; b < 3; ++b) {
        if (b < I) rr += srp[b][l];
        if (b + 1 > I) cc += scp[b + 1][l];
      }
      const float u = row16_sum(I >= 2 ? srp[0][l] : 0.f), v = row16_sum(I == 3 ? srp[1][l] : 0.f);
      float* tot = a.tot + ((int64_t)cslot * a.H + h) * 4;
      if (l == 32 || l == 48) tot[I - 2] = u;
      if (l == 48) tot[2] = v;
      if (l < len) {
        const int64_t o = (int64_t)h * a.seq.total + tok + l, in = (int64_t)a.H * a.seq.total;
        a.ri[o] = rr;
        a.ri[in + o] = srp[I][l];
        a.ci[o] = cc;
        a.ci[in + o] = scp[I][l];
        a.cd[o] = scd[l];
      }
    }
    if (w == 1 && l == 0) {
      float s = 0.f;
      for (int i = 0; i < NW; ++i) s += sdd[i];
      a.dpart[(int64_t)cslot * a.H + h] = s;
    }
    if (w == 2 && l == 0) {
      float s = 0.f;
      for (int i = 0; i < NW; ++i) s += shd[i];
      a.hdot[(int64_t)cslot * a.H + h] = s;
    }
    // dX^T, rows p of this wave's share, columns j = 16 tb + r
    {
      const int j = 16 * tb + r;
      const float eE = seE[j], dt = sdt[j], D = a.d ? a.d[h] : 0.f;
#pragma unroll
      for (int pi = 0; pi < PTW; ++pi) {
        const int pt = sh * PTW + pi;
        f32x4 u = zero4(), v = zero4();
        const T* sdp = sd + slot_place<T>(16 * pt + r) * LK + VEC<T> * g4;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
          if ((q + 1) * KG<T> > 16 * tb)
            mma16B<T>(u, frag_col<T>(sy, LV, q * KG<T>, 16 * pt), frag_row<T>(sm, LM, 16 * tb, q * KG<T>));
#pragma unroll
        for (int q = 0; q < KQ; ++q)
          mma16B<T>(v, *reinterpret_cast<const uint4*>(sdp + q * KG<T>), frag_row<T>(sb, LK, 16 * tb, q * KG<T>));
        const int p = 16 * pt + 4 * g4;
        const f32x4 dyv = ld4<T>(sy + j * LV + p);
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = dt * (u[e] + eE * v[e]) + D * dyv[e];
        if (j < len) st4<T>(reinterpret_cast<T*>(a.dx) + (int64_t)(tok + j) * a.dxs + h * V + p, u);
      }
    }
    // dC, dB through the states: rows 16 tb + 4 g4 + e
    {
      uint4 yf[VQ], xf[VQ];
#pragma unroll
      for (int q = 0; q < VQ; ++q) {
        yf[q] = frag_row<T>(sy, LV, 16 * tb, q * KG<T>);
        xf[q] = frag_row<T>(sx, LV, 16 * tb, q * KG<T>);
      }
      const f32x4 eG = *reinterpret_cast<const f32x4*>(seG + 16 * tb + 4 * g4);
      const f32x4 eE = *reinterpret_cast<const f32x4*>(seE + 16 * tb + 4 * g4);
      const f32x4 dt = *reinterpret_cast<const f32x4*>(sdt + 16 * tb + 4 * g4);
#pragma unroll
      for (int ni = 0; ni < NTW; ++ni) {
        const int nt = sh * NTW + ni;
        f32x4 u = zero4(), v = zero4();
#pragma unroll
        for (int q = 0; q < VQ; ++q) {
          mma16B<T>(u, yf[q], frag_col<T>(ss, LK, q * KG<T>, 16 * nt));
          mma16B<T>(v, xf[q], frag_col<T>(sd, LK, q * KG<T>, 16 * nt));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dC[ni][e] += eG[e] * u[e];
          dB[ni][e] += eE[e] * dt[e] * v[e];
        }
      }
    }
  }
  // The heads' W: as W^T [j][i] for dB, then as W [i][j] for dC (columns in slot order);
  // for bf16 in two pieces, as it is rounded once for all heads at little cost.
#pragma unroll
  for (int piece = 0; piece < (std::is_same_v<T, bf16> ? 2 : 1); ++piece) {
    lds_barrier();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int blk = b * NW + w;
      if (blk < 10) {
        int I, J;
        tri_block(blk, I, J);
        if (piece) {
#pragma unroll
          for (int e = 0; e < 4; ++e) wsum[b][e] -= (float)(T)wsum[b][e];
        }
        T* p = sm + (16 * J + r) * LM;
        st4<T>(p + slot_base4<T>(I, g4), wsum[b]);
        // the block left of the diagonal that shares a contraction with it
        if (I == J && (I & 1)) st4<T>(p + slot_base4<T>(I - 1, g4), zero4());
      }
    }
    lds_barrier();
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      if ((q + 1) * KG<T> > 16 * tb) {
        const uint4 wf = frag_row<T>(sm, LM, 16 * tb, q * KG<T>);  // row j, contraction i
#pragma unroll
        for (int ni = 0; ni < NTW; ++ni) mma16B<T>(dB[ni], wf, frag_col<T>(sc, LK, q * KG<T>, 16 * (sh * NTW + ni)));
      }
    lds_barrier();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int blk = b * NW + w;
      if (blk < 10) {
        int I, J;
        tri_block(blk, I, J);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          T* p = sm + (16 * I + slot_row<T>(4 * g4 + e)) * LM;
          p[slot_of<T>(16 * J + r)] = (T)wsum[b][e];
          // the block right of the diagonal that shares a contraction with it
          if (I == J && (I & 1) == 0) p[slot_of<T>(16 * (J + 1) + r)] = (T)0.f;
        }
      }
    }
    lds_barrier();
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      if (q * KG<T> <= 16 * tb) {
        const uint4 wf = frag_row<T>(sm, LM, 16 * tb, q * KG<T>);  // row i, contraction j
#pragma unroll
        for (int ni = 0; ni < NTW; ++ni) mma16B<T>(dC[ni], wf, frag_col<T>(sb, LK, q * KG<T>, 16 * (sh * NTW + ni)));
      }
  }
#pragma unroll
  for (int ni = 0; ni < NTW; ++ni) {
    const int n = 16 * (sh * NTW + ni) + r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * tb + 4 * g4 + e;
      if (i < len) {
        if (a.split > 1) {
          const int64_t rows = (int64_t)a.seq.total * a.G;
          const int64_t o = ((int64_t)part * rows + (int64_t)(tok + i) * a.G + grp) * K + n;
          a.bcpart[o] = dB[ni][e];
          a.bcpart[(int64_t)a.split * rows * K + o] = dC[ni][e];
        } else {
          reinterpret_cast<T*>(a.db)[(int64_t)(tok + i) * a.dbs + grp * K + n] = (T)dB[ni][e];
          reinterpret_cast<T*>(a.dc)[(int64_t)(tok + i) * a.dcs + grp * K + n] = (T)dC[ni][e];
        }
      }
    }
  }
}

// dB or dC from the partial sums of the head ranges, elements i .. i + 3 of the packed rows.
template <typename T>
__device__ __forceinline__ void sum_ranges(const SsmArgs& a, bool dc, int64_t i) {
  const int64_t rows = (int64_t)a.seq.total * a.G, row = i / a.K, tok = row / a.G;
  const int k = (int)(i - row * a.K), grp = (int)(row - tok * a.G);
  if (row >= rows || tok >= seq_start(a.seq, a.seq.N)) return;
  const float* p = a.bcpart + (dc ? (int64_t)a.split * rows * a.K : 0) + i;
  f32x4 s = zero4();
  for (int j = 0; j < a.split; ++j) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(p + (int64_t)j * rows * a.K);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += v[e];
  }
  st4<T>(reinterpret_cast<T*>(dc ? a.dc : a.db) + tok * (dc ? a.dcs : a.dbs) + grp * a.K + k, s);
}

// Gate gradients of one chunk and head, one wave, lane t its token.  dg_t is the sum
// over what passes token t's decay: the entering state into the rows i >= t (rx), the
// rows j < t into the leaving state (dt cx), the pairs j < t <= i of the chunk, and what
// goes from the entering into the leaving state, H = exp(G_L) <S_in, dS>.
// H is small beside E = <S_out, dS> where a chunk decays strongly, and dg_t is
// multiplied by a g_t that is large there, so it may not inherit the rounding of E: it
// is formed from the states that the chunk backward read (fp32: always).  As bf16
// these give it to about 2^-9, so a decay over DIRECT takes it from E instead: H = E -
// sum dt cx, and E one chunk earlier is H + sum rx, or the other way round.  E is
// known where the walks meet, at the ends of the segments, and behind and before a
// chunk that needs no E; the nearest of these is taken, as every chunk in between adds
// its rounding.  Workgroups behind the first ngate sum dB (nsum) and dC (nsum): 32 MB, at
// the side of the gates' chains of small loads (8192 x 32 heads: 12.9 and 5.5 us apart).
template <typename T>
__global__ __launch_bounds__(256) void k_ssm_gate(SsmArgs a, int ngate, int nsum) {
  if ((int)blockIdx.x >= ngate) {
    const int b = blockIdx.x - ngate;
    sum_ranges<T>(a, b >= nsum, ((b >= nsum ? b - nsum : b) * (int64_t)256 + threadIdx.x) * 4);
    return;
  }
  // log2 of the decay: 2^-12 2^-9 is about the rounding of E and of the sum
  constexpr float DIRECT = std::is_same_v<T, bf16> ? -12.f : 1.f;
  const int wk = blockIdx.x * 4 + wave_id(), l = lane_id();
  if (wk >= a.nchunk * a.H) return;
  const int cslot = wk / a.H, h = wk - cslot * a.H;
  const Piece pc = find_piece(a.seq, cslot, CH);
  const int t0 = pc.bos + pc.k * CH, per = a.seg / CH, k = pc.k / per;  // segment of the chunk
  if (!pc.on || t0 >= pc.eos) {
    if (l < 2) a.apart[((int64_t)cslot * 2 + l) * a.H + h] = 0.;
    return;
  }
  const int t1 = min(t0 + CH, pc.eos), t2 = min(pc.bos + (k + 1) * a.seg, pc.eos);
  const int64_t row = (int64_t)h * a.seq.total;
  const float bias = gate_bias(a, h);
  // (sums in 64 bits: their terms cancel, and what they leave is summed once more
  // over the tokens)
  auto wave_sum = [](double v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d, 64);
    return v;
  };
  float dt = 0.f, z = 0.f;
  double rx = 0., dcx = 0., srx = 0., sdcx = 0.;  // a chunk's, by token and summed; last this chunk's
  auto sums = [&](int c) {  // of chunk ci + c
    const int t = t0 + c * CH + l;
    dt = 0.f;
    rx = dcx = 0.;
    if (t < t2) {
      dt = chunk_gates(a, cslot + c, h)[l].dt;
      rx = a.rx[row + t];
      dcx = (double)dt * a.cx[row + t];
    }
    srx = wave_sum(rx);
    sdcx = wave_sum(dcx);
  };
  auto direct = [&](int c) {
    return (double)fexp2(chunk_gates(a, cslot + c, h)[CH - 1].G) * a.hdot[(int64_t)(cslot + c) * a.H + h];
  };
  double H;
  if constexpr (std::is_same_v<T, bf16>) {
    const int ci = pc.k - k * per, nc = ci + (t2 - t0 + CH - 1) / CH;  // this chunk, chunks of the segment
    const uint64_t none = __ballot(l < nc && chunk_gates(a, cslot - ci + min(l, nc - 1), h)[CH - 1].G < DIRECT);
    const uint64_t later = none >> ci, before = none << (63 - ci);
    const double* ends = a.ends + ((int64_t)slot_base(a.seq, pc.n, a.seg) + k) * a.H + h;
    const int up = later ? __builtin_ctzll(later) : nc - 1 - ci;
    const int down = before ? __builtin_clzll(before) : k > 0 || !a.h0 ? ci : SEG_CHUNKS;
    double E = 0.;
    bool known = true;
    if (up <= down) {
      if (later) H = direct(up);
      else E = *ends, known = false;
      for (int c = up; c >= 0; --c) {
        sums(c);
        if (c < up || !known) H = E - sdcx;
        E = H + srx;
      }
    } else {
      if (before) H = direct(-down);
      else E = k > 0 ? ends[-a.H] : 0., known = false;
      for (int c = -down; c <= 0; ++c) {
        sums(c);
        if (c > -down || !known) H = E - srx;
        E = H + sdcx;
      }
    }
  } else {
    sums(0);
    H = direct(0);
  }
  // Pairs j < t <= i: with b the block of 16 that t lies in, the blocks right below and
  // left of it whole (tot), the rows i >= t of b left of it, the columns j < t of b below
  // it, and in its own block the suffix sum of ri - dt ci, in which the pairs on one
  // side of t cancel (over the whole chunk they would cancel 64 tokens' roundings).
  const int t = t0 + l, blk = l >> 4;
  const bool on = t < t1;
  const int64_t in = (int64_t)a.H * a.seq.total;
  double cc = 0., s = rx, pre = dcx, rb = 0., cb = 0.;  // suffix and prefix over the chunk; over the block
  if (on) {
    z = ld_beta(a.dt, a.dt_f32, (int64_t)t * a.H + h) + bias;
    const float co = a.ci[row + t], ci = a.ci[in + row + t];
    rb = (double)a.ri[row + t] + a.ri[in + row + t] - (double)dt * ci;
    cb = (double)dt * co;
    cc = (double)a.cx[row + t] + co + ci + a.cd[row + t];
  }
  const double cb0 = cb;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double u = __shfl_down(s, d, 64), v = __shfl_up(pre, d, 64);
    if (l + d < 64) s += u;
    if (l >= d) pre += v;
    if (d < 16) {
      const double p = __shfl_down(rb, d, 16), q = __shfl_up(cb, d, 16);
      if ((l & 15) + d < 16) rb += p;
      if ((l & 15) >= d) cb += q;
    }
  }
  const f32x4 tot = *reinterpret_cast<const f32x4*>(a.tot + ((int64_t)cslot * a.H + h) * 4);
  const double far = blk == 1 ? (double)tot[0] + tot[1] : blk == 2 ? (double)tot[1] + tot[2] : 0.;
  double dA = 0., db = 0.;
  if (on) {
    const double A = -exp((double)a.a_log[h]), dg = H + s + (pre - dcx) + rb + (cb - cb0) + far;
    const float e = expf(-fabsf(z)), sg = (z >= 0.f ? 1.f : e) / (1.f + e);
    db = (cc + A * dg) * sg;
    st_beta(a.ddt, a.dt_f32, (int64_t)t * a.H + h, (float)db);
    dA = dg * (A * dt);
  }
  dA = wave_sum(dA);
  db = wave_sum(db);
  if (l == 0) {
    a.apart[((int64_t)cslot * 2 + 0) * a.H + h] = dA;
    a.apart[((int64_t)cslot * 2 + 1) * a.H + h] = db;
  }
}

// dA_log, ddt_bias and dD [H], sums over the chunks (of dD's a slot that no sequence
// uses holds nothing and is skipped).
__global__ __launch_bounds__(256) void k_ssm_params(SsmArgs a) {
  __shared__ double buf[4];
  const int h = blockIdx.x, what = blockIdx.y;
  double s = 0.;
  if (what < 2) {
    for (int i = threadIdx.x; i < a.nchunk; i += 256) s += a.apart[((int64_t)i * 2 + what) * a.H + h];
  } else {
    for (int i = threadIdx.x; i < a.nchunk; i += 256) {
      const Piece pc = find_piece(a.seq, i, CH);
      if (pc.on && pc.bos + pc.k * CH < pc.eos) s += a.dpart[(int64_t)i * a.H + h];
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d, 64);
  if (lane_id() == 0) buf[wave_id()] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    float* o = what == 0 ? a.da_log : what == 1 ? a.ddt_bias : a.dd;
    if (o) o[h] = (float)((buf[0] + buf[1]) + (buf[2] + buf[3]));
  }
}

}  // namespace

hipError_t launch_ssm_walk(const SsmArgs& a, bool f32, hipStream_t s) {
  return ssm_kv_heads<64>(a, f32, [&](auto t, auto k, auto v, auto hb) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value, V = decltype(v)::value, HB = decltype(hb)::value;
    REWY_LAUNCH((k_ssm_walk<T, K, V, HB>), dim3(a.nslot * ssm_head_blocks(a, HB), 2), dim3(4 * HB * V), s, a);
    return hipGetLastError();
  });
}
hipError_t launch_ssm_chunk(const SsmArgs& a, bool f32, hipStream_t s) {
  return ssm_kv(a.K, a.V, f32, [&](auto t, auto k, auto v) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value, V = decltype(v)::value;
    REWY_LAUNCH((k_ssm_chunk<T, K, V>), dim3(a.nchunk * a.G * a.split), dim3(64 * cb_waves(K, V)), s, a);
    return hipGetLastError();
  });
}
hipError_t launch_ssm_gate(const SsmArgs& a, bool f32, hipStream_t s) {
  const int ngate = (a.nchunk * a.H + 3) / 4;
  const int nsum = a.split > 1 ? (int)(((int64_t)a.seq.total * a.G * a.K / 4 + 255) / 256) : 0;
  const dim3 grid(ngate + 2 * nsum);
  if (f32) REWY_LAUNCH((k_ssm_gate<float>), grid, dim3(256), s, a, ngate, nsum);
  else REWY_LAUNCH((k_ssm_gate<bf16>), grid, dim3(256), s, a, ngate, nsum);
  return hipGetLastError();
}
hipError_t launch_ssm_params(const SsmArgs& a, hipStream_t s) {
  REWY_LAUNCH(k_ssm_params, dim3(a.H, 3), dim3(256), s, a);
  return hipGetLastError();
}
}  // namespace rewy
