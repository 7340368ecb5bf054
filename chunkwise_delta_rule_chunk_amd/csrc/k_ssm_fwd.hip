// Selective state space scan, forward: the local end states of the segments,
// the pass that joins them, and the walk that forms y; and the token-serial
// form.
#include "ssm.hpp"

#ifndef SSM_WAVES
#define SSM_WAVES 4
#endif
namespace rewy {

namespace {

// The gates of all chunks: one wave per chunk and head, lane t its token.
__global__ __launch_bounds__(256) void k_ssm_gates(SsmArgs a) {
  const int wk = blockIdx.x * 4 + wave_id(), t = lane_id();
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
// tokens send to the state that enters it, all but the first.
template <typename T, int K, int V, int HB>
__global__ __launch_bounds__(4 * HB * V, SSM_WAVES) void k_ssm_state(SsmArgs a) {
  constexpr int CW = HB * V, NTH = 4 * CW, LK = pitch<T>(K), LV = pitch<T>(CW);
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
  const int nch = (t1 - t0 + CH - 1) / CH, w = wave_id(), l = lane_id(), hw = 16 * w / V;
  const int cbase = slot_base(a.seq, pc.n, CH) + pc.k * (a.seg / CH);
  f32x4 S[K / 16];
#pragma unroll
  for (int i = 0; i < K / 16; ++i) S[i] = zero4();
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
    if (w < HB) {
      sal[w][slot_of<T>(l)] = dir ? fexp2(gt.G) : fexp2(gt.E) * gt.dt;
      if (l == 63) sdec[w] = fexp2(gt.G);
      gs += gt.G;
    }
    lds_barrier();
    if (c + 1 < nch) fetch(c + 1);
    state_update<T, K>(S, sk, LK, su, LV, 16 * w, sal[hw], sdec[hw]);
    lds_barrier();
  }
  // (forward and reverse sum the same decays, each for the segments it takes)
  if (w < nh && l == 63) a.gsum[((int64_t)dir * a.nslot + slot) * a.H + h0 + w] = gs;
  if (hw >= nh) return;
  float* o = (dir ? a.sr : a.sf) + ((int64_t)slot * a.H + h0 + hw) * K * V + 16 * w - hw * V + (l & 15);
#pragma unroll
  for (int nt = 0; nt < K / 16; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[(int64_t)(16 * nt + 4 * (l >> 4) + i) * V] = S[nt][i];
}

// In place: the local states of a sequence's segments become the states that
// enter them (forward; from h0) or the adjoints of the states that leave them
// (reverse; from dht).
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
// state; the chunk's coefficients M, one 64 x 64 matrix a head, are formed block
// by block by all waves (C B^T once for the heads) and shared through LDS.
template <typename T, int K, int V, int HB>
__global__ __launch_bounds__(4 * HB * V, SSM_WAVES) void k_ssm_fwd(SsmArgs a) {
  constexpr int CW = HB * V, NTH = 4 * CW, NW = CW / 16, LK = pitch<T>(K), LV = pitch<T>(CW), LM = pitch<T>(CH);
  constexpr int NQ = CH / KG<T>, NT = K / 16, KQ = K / KG<T>;
  __shared__ __align__(16) T sb[CH * LK];
  __shared__ __align__(16) T sc[CH * LK];
  __shared__ __align__(16) T sx[CH * LV];
  __shared__ __align__(16) T sm[HB][CH * LM];  // columns in slot order
  // gates of each head: by token, and in slot order
  __shared__ __align__(16) float sG[HB][CH], sGl[HB][CH], seq[HB][CH], tG[HB][CH], tGl[HB][CH], tdt[HB][CH], sal[HB][CH];
  __shared__ float sdec[HB];
  const int nhb = head_blocks(a, HB), wk = xcd_range(blockIdx.x, a.nslot * nhb), slot = wk / nhb, hb = wk - slot * nhb;
  const Piece pc = find_piece(a.seq, slot, a.seg);
  if (!pc.on) return;
  const int t0 = pc.bos + pc.k * a.seg, t1 = min(t0 + a.seg, pc.eos);
  const int gb = (a.per + HB - 1) / HB, grp = hb / gb, h0 = grp * a.per + (hb - grp * gb) * HB;
  const int nh = min(HB, (grp + 1) * a.per - h0);  // heads of this block
  const int nch = (t1 - t0 + CH - 1) / CH, w = wave_id(), l = lane_id(), g4 = l >> 4, r = l & 15;
  const int hw = 16 * w / V, h = min(h0 + hw, h0 + nh - 1), pc0 = 16 * w - hw * V;  // the wave's head, its columns
  const bool live = hw < nh;
  const int cbase = slot_base(a.seq, pc.n, CH) + pc.k * (a.seg / CH);
  const float D = a.d ? a.d[h] : 0.f;
  const int64_t head = ((int64_t)pc.n * a.H + h) * K * V + pc0 + r;
  // (an empty sequence has no segment of its own: its state is given through)
  const float* init = a.two && nch > 0 ? a.sf + ((int64_t)slot * a.H + h) * K * V + pc0 + r
                      : a.h0           ? a.h0 + head
                                       : nullptr;
  f32x4 S[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) S[nt][i] = init ? init[(int64_t)(16 * nt + 4 * g4 + i) * V] : 0.f;
  // a pair of blocks above the diagonal lies inside a contraction of 32: zeros, written once
  for (int i = threadIdx.x; i < HB * CH * LM; i += NTH) sm[0][i] = (T)0.f;

  TileRegs<T, CH, K, NTH> rb, rc;
  TileRegs<T, CH, CW, NTH> rx;
  Gate gt = {};
  auto fetch = [&](int c) {
    const int tok = t0 + c * CH, len = min(CH, t1 - tok);
    if (w < nh) gt = chunk_gates(a, cbase + c, h0 + w)[l];
    load_tile<T, K, NTH>(rb, a.b, tok, a.bs, grp * K, len, K);
    load_tile<T, K, NTH>(rc, a.c, tok, a.cs, grp * K, len, K);
    load_tile<T, CW, NTH>(rx, a.x, tok, a.xs, h0 * V, len, nh * V);
  };
  if (nch > 0) fetch(0);
  for (int c = 0; c < nch; ++c) {
    const int tok = t0 + c * CH, len = min(CH, t1 - tok);
    rb.store(sb, LK, threadIdx.x);
    rc.store(sc, LK, threadIdx.x);
    rx.store(sx, LV, threadIdx.x);
    if (w < HB) {
      const float eG = fexp2(gt.G);
      const int sl = slot_of<T>(l);
      sG[w][l] = gt.G;
      sGl[w][l] = gt.Glo;
      seq[w][l] = eG;
      tG[w][sl] = gt.G;
      tGl[w][sl] = gt.Glo;
      tdt[w][sl] = gt.dt;
      sal[w][sl] = fexp2(gt.E) * gt.dt;
      if (l == 63) sdec[w] = eG;
    }
    lds_barrier();
    if (c + 1 < nch) fetch(c + 1);
    // coefficients: block (I, J) of the lower triangle, as its transpose (rows j in
    // slot order, columns i), so that a lane holds four neighbours of a row of M
#pragma unroll
    for (int b0 = 0; b0 < 10; b0 += NW) {
      const int blk = b0 + w;
      if (blk < 10) {
        const int I = blk >= 6 ? 3 : blk >= 3 ? 2 : blk >= 1 ? 1 : 0, J = blk - I * (I + 1) / 2;
        f32x4 acc = zero4();
#pragma unroll
        for (int q = 0; q < KQ; ++q)
          mma16B<T>(acc, frag_row_slot<T>(sb, LK, 16 * J, q * KG<T>), frag_row<T>(sc, LK, 16 * I, q * KG<T>));
        const int i = 16 * I + r, sl = slot_base4<T>(J, g4);
#pragma unroll
        for (int k = 0; k < HB; ++k) {
          const float Gi = sG[k][i], Gil = sGl[k][i];
          const f32x4 Gj = *reinterpret_cast<const f32x4*>(tG[k] + sl), Gjl = *reinterpret_cast<const f32x4*>(tGl[k] + sl);
          const f32x4 dj = *reinterpret_cast<const f32x4*>(tdt[k] + sl);
          f32x4 m;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m[e] = 16 * J + slot_row<T>(4 * g4 + e) <= i ? acc[e] * fexp2((Gi - Gj[e]) + (Gil - Gjl[e])) * dj[e] : 0.f;
          st4<T>(sm[k] + i * LM + sl, m);
        }
      }
    }
    // entering state: Y^T = S^T C^T, columns scaled by exp(G)
    f32x4 Y[4];
#pragma unroll
    for (int I = 0; I < 4; ++I) Y[I] = zero4();
#pragma unroll
    for (int q = 0; q < KQ; ++q) {
      uint4 sf[1];
      frag_acc<T, 1>(sf, S, q);
#pragma unroll
      for (int I = 0; I < 4; ++I) mma16B<T>(Y[I], sf[0], frag_row_acc<T>(sc, LK, 16 * I, q));
    }
#pragma unroll
    for (int I = 0; I < 4; ++I) {
      const float e = seq[hw][16 * I + r];
#pragma unroll
      for (int i = 0; i < 4; ++i) Y[I][i] *= e;
    }
    lds_barrier();  // M complete
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const uint4 xt = frag_col<T>(sx, LV, q * KG<T>, 16 * w);
#pragma unroll
      for (int I = 0; I < 4; ++I)
        if (q * KG<T> <= 16 * I) mma16B<T>(Y[I], xt, frag_row<T>(sm[hw], LM, 16 * I, q * KG<T>));
    }
#pragma unroll
    for (int I = 0; I < 4; ++I) {
      const int t = 16 * I + r;
      const f32x4 xv = ld4<T>(sx + t * LV + 16 * w + 4 * g4);
#pragma unroll
      for (int i = 0; i < 4; ++i) Y[I][i] += D * xv[i];
      if (live && t < len)
        st4<T>(reinterpret_cast<T*>(a.y) + (int64_t)(tok + t) * a.ys + h * V + pc0 + 4 * g4, Y[I]);
    }
    state_update<T, K>(S, sb, LK, sx, LV, 16 * w, sal[hw], sdec[hw]);
    lds_barrier();  // tiles free
  }
  if (a.ht && live && t1 >= pc.eos) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) a.ht[head + (int64_t)(16 * nt + 4 * g4 + i) * V] = S[nt][i];
  }
}

// Token by token: one workgroup per sequence and head, the state in registers,
// four neighbouring columns of K V / 1024 rows a thread.  For one new token it
// costs the state's bytes, read and written once.
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

hipError_t launch_ssm_gates(const SsmArgs& a, hipStream_t s) {
  REWY_LAUNCH(k_ssm_gates, dim3((a.nchunk * a.H + 3) / 4), dim3(256), s, a);
  return hipGetLastError();
}
int ssm_head_blocks(const SsmArgs& a, int hb) { return a.G * ((a.per + hb - 1) / hb); }

hipError_t launch_ssm_state(const SsmArgs& a, bool f32, bool both, hipStream_t s) {
  return ssm_kv_heads(a, f32, [&](auto t, auto k, auto v, auto hb) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value, V = decltype(v)::value, HB = decltype(hb)::value;
    REWY_LAUNCH((k_ssm_state<T, K, V, HB>), dim3(a.nslot * ssm_head_blocks(a, HB), both ? 2 : 1), dim3(4 * HB * V), s, a);
    return hipGetLastError();
  });
}
hipError_t launch_ssm_pass(const SsmArgs& a, bool both, hipStream_t s) {
  REWY_LAUNCH(k_ssm_pass, dim3(a.seq.N * a.H, (a.K * a.V + 1023) / 1024, both ? 2 : 1), dim3(256), s, a);
  return hipGetLastError();
}
hipError_t launch_ssm_fwd(const SsmArgs& a, bool f32, hipStream_t s) {
  return ssm_kv_heads(a, f32, [&](auto t, auto k, auto v, auto hb) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value, V = decltype(v)::value, HB = decltype(hb)::value;
    REWY_LAUNCH((k_ssm_fwd<T, K, V, HB>), dim3(a.nslot * ssm_head_blocks(a, HB)), dim3(4 * HB * V), s, a);
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
