// Selective state space scan, forward: the local end states of the segments,
// the pass that joins them, and the walk that forms y; and the token-serial
// form.
#include "ssm.hpp"

namespace rewy {

namespace {

// Local state of one segment and head: forward (dir 0), from zero, all but a
// sequence's last segment; reverse (dir 1), the adjoint that the segment's own
// tokens send to the state that enters it, all but the first.
template <typename T, int K, int V>
__global__ __launch_bounds__(4 * V) void k_ssm_state(SsmArgs a) {
  constexpr int NTH = 4 * V, LK = pitch<T>(K), LV = pitch<T>(V), NQ = CH / KG<T>;
  __shared__ __align__(16) T sk[CH * LK];
  __shared__ __align__(16) T su[CH * LV];
  __shared__ __align__(16) float sal[CH];
  __shared__ float sdec;
  const int dir = blockIdx.y;
  const int wk = xcd_range(blockIdx.x, a.nslot * a.H), slot = wk / a.H, h = wk - slot * a.H, grp = h / a.per;
  const Piece pc = find_piece(a.seq, slot, a.seg);
  if (!pc.on) return;
  const int t0 = pc.bos + pc.k * a.seg, t1 = min(t0 + a.seg, pc.eos);
  if (dir == 0 ? t1 >= pc.eos : pc.k == 0) return;
  const int nch = (t1 - t0 + CH - 1) / CH, w = wave_id(), l = lane_id();
  const float A2 = gate_rate(a, h), bias = gate_bias(a, h);
  f32x4 S[K / 16];
#pragma unroll
  for (int i = 0; i < K / 16; ++i) S[i] = zero4();
  float gs = 0.f;
  TileRegs<T, CH, K, NTH> rk;
  TileRegs<T, CH, V, NTH> ru;
  auto fetch = [&](int c) {
    const int tok = t0 + (dir ? nch - 1 - c : c) * CH, len = min(CH, t1 - tok);
    load_tile<T, K, NTH>(rk, dir ? a.c : a.b, tok, dir ? a.cs : a.bs, grp * K, len);
    load_tile<T, V, NTH>(ru, dir ? a.dy : a.x, tok, dir ? a.ys : a.xs, h * V, len);
  };
  fetch(0);
  for (int c = 0; c < nch; ++c) {
    const int tok = t0 + (dir ? nch - 1 - c : c) * CH, len = min(CH, t1 - tok);
    rk.store(sk, LK, threadIdx.x);
    ru.store(su, LV, threadIdx.x);
    if (w == 0) {
      const ChunkGate g = chunk_gate(a, tok, len, h, A2, bias);
      sal[l] = dir ? fexp2(g.G) : fexp2(g.E) * g.dt;
      if (l == 0) sdec = fexp2(g.GL);
      gs += g.GL;
    }
    __syncthreads();
    if (c + 1 < nch) fetch(c + 1);
    uint4 ut[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) ut[q] = frag_col<T>(su, LV, q * KG<T>, 16 * w);
    state_update<T, K>(S, sk, LK, ut, sal, sdec);
    __syncthreads();
  }
  float* o = (dir ? a.sr : a.sf) + ((int64_t)slot * a.H + h) * K * V + 16 * w + (l & 15);
#pragma unroll
  for (int nt = 0; nt < K / 16; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[(int64_t)(16 * nt + 4 * (l >> 4) + i) * V] = S[nt][i];
  // (forward and reverse sum the same decays; a segment that both take writes it twice)
  if (w == 0 && l == 0) a.gsum[((int64_t)dir * a.nslot + slot) * a.H + h] = gs;
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

// The walk of one segment and head.  V / 16 waves, wave w the columns 16 w ..
// + 15 of y and of the state; the chunk's 64 x 64 coefficients M are formed
// block by block by all waves and shared through LDS.
template <typename T, int K, int V>
__global__ __launch_bounds__(4 * V) void k_ssm_fwd(SsmArgs a) {
  constexpr int NTH = 4 * V, NW = V / 16, LK = pitch<T>(K), LV = pitch<T>(V), LM = pitch<T>(CH), NQ = CH / KG<T>;
  constexpr int NT = K / 16, KQ = K / KG<T>;
  __shared__ __align__(16) T sb[CH * LK];
  __shared__ __align__(16) T sc[CH * LK];
  __shared__ __align__(16) T sx[CH * LV];
  __shared__ __align__(16) T sm[CH * LM];
  __shared__ __align__(16) float sG[CH], sdt[CH], sal[CH], seq[CH];
  __shared__ float sdec;
  const int wk = xcd_range(blockIdx.x, a.nslot * a.H), slot = wk / a.H, h = wk - slot * a.H, grp = h / a.per;
  const Piece pc = find_piece(a.seq, slot, a.seg);
  if (!pc.on) return;
  const int t0 = pc.bos + pc.k * a.seg, t1 = min(t0 + a.seg, pc.eos);
  const int nch = (t1 - t0 + CH - 1) / CH, w = wave_id(), l = lane_id(), g4 = l >> 4, r = l & 15;
  const float A2 = gate_rate(a, h), bias = gate_bias(a, h), D = a.d ? a.d[h] : 0.f;
  const int64_t head = ((int64_t)pc.n * a.H + h) * K * V + 16 * w + r;
  // (an empty sequence has no segment of its own: its state is given through)
  const float* init = a.two && nch > 0 ? a.sf + ((int64_t)slot * a.H + h) * K * V + 16 * w + r
                      : a.h0           ? a.h0 + head
                                       : nullptr;
  f32x4 S[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) S[nt][i] = init ? init[(int64_t)(16 * nt + 4 * g4 + i) * V] : 0.f;
  // a pair of blocks above the diagonal lies inside a contraction of 32: zeros, written once
  for (int i = threadIdx.x; i < CH * LM; i += NTH) sm[i] = (T)0.f;

  TileRegs<T, CH, K, NTH> rb, rc;
  TileRegs<T, CH, V, NTH> rx;
  auto fetch = [&](int c) {
    const int tok = t0 + c * CH, len = min(CH, t1 - tok);
    load_tile<T, K, NTH>(rb, a.b, tok, a.bs, grp * K, len);
    load_tile<T, K, NTH>(rc, a.c, tok, a.cs, grp * K, len);
    load_tile<T, V, NTH>(rx, a.x, tok, a.xs, h * V, len);
  };
  if (nch > 0) fetch(0);
  for (int c = 0; c < nch; ++c) {
    const int tok = t0 + c * CH, len = min(CH, t1 - tok);
    rb.store(sb, LK, threadIdx.x);
    rc.store(sc, LK, threadIdx.x);
    rx.store(sx, LV, threadIdx.x);
    if (w == 0) {
      const ChunkGate g = chunk_gate(a, tok, len, h, A2, bias);
      sG[l] = g.G;
      sdt[l] = g.dt;
      sal[l] = fexp2(g.E) * g.dt;
      seq[l] = fexp2(g.G);
      if (l == 0) sdec = fexp2(g.GL);
    }
    __syncthreads();
    if (c + 1 < nch) fetch(c + 1);
    // coefficients: block (I, J) of the lower triangle, as its transpose (rows j,
    // columns i), so that a lane holds four neighbours of one row of M
#pragma unroll
    for (int b0 = 0; b0 < 10; b0 += NW) {
      const int blk = b0 + w;
      if (blk < 10) {
        const int I = blk >= 6 ? 3 : blk >= 3 ? 2 : blk >= 1 ? 1 : 0, J = blk - I * (I + 1) / 2;
        f32x4 acc = zero4();
#pragma unroll
        for (int q = 0; q < KQ; ++q)
          mma16B<T>(acc, frag_row<T>(sb, LK, 16 * J, q * KG<T>), frag_row<T>(sc, LK, 16 * I, q * KG<T>));
        const int i = 16 * I + r, j = 16 * J + 4 * g4;
        const float Gi = sG[i];
        const f32x4 Gj = *reinterpret_cast<const f32x4*>(sG + j), dj = *reinterpret_cast<const f32x4*>(sdt + j);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = j + e <= i ? acc[e] * fexp2(Gi - Gj[e]) * dj[e] : 0.f;
        st4<T>(sm + i * LM + j, acc);
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
      const float e = seq[16 * I + r];
#pragma unroll
      for (int i = 0; i < 4; ++i) Y[I][i] *= e;
    }
    uint4 xt[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) xt[q] = frag_col<T>(sx, LV, q * KG<T>, 16 * w);
    state_update<T, K>(S, sb, LK, xt, sal, sdec);
    __syncthreads();  // M complete
#pragma unroll
    for (int I = 0; I < 4; ++I) {
#pragma unroll
      for (int q = 0; q < NQ; ++q)
        if (q * KG<T> <= 16 * I) mma16B<T>(Y[I], xt[q], frag_row<T>(sm, LM, 16 * I, q * KG<T>));
      const int t = 16 * I + r, p = 16 * w + 4 * g4;
      const f32x4 xv = ld4<T>(sx + t * LV + p);
#pragma unroll
      for (int i = 0; i < 4; ++i) Y[I][i] += D * xv[i];
      if (t < len) st4<T>(reinterpret_cast<T*>(a.y) + (int64_t)(tok + t) * a.ys + h * V + p, Y[I]);
    }
    __syncthreads();  // tiles free
  }
  if (a.ht && t1 >= pc.eos) {
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
  const float A2 = gate_rate(a, h), bias = gate_bias(a, h), D = a.d ? a.d[h] : 0.f;
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
    __syncthreads();
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
    __syncthreads();
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

hipError_t launch_ssm_state(const SsmArgs& a, bool f32, bool both, hipStream_t s) {
  return ssm_kv(a.K, a.V, f32, [&](auto t, auto k, auto v) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value, V = decltype(v)::value;
    REWY_LAUNCH((k_ssm_state<T, K, V>), dim3(a.nslot * a.H, both ? 2 : 1), dim3(4 * V), s, a);
    return hipGetLastError();
  });
}
hipError_t launch_ssm_pass(const SsmArgs& a, bool both, hipStream_t s) {
  REWY_LAUNCH(k_ssm_pass, dim3(a.seq.N * a.H, (a.K * a.V + 1023) / 1024, both ? 2 : 1), dim3(256), s, a);
  return hipGetLastError();
}
hipError_t launch_ssm_fwd(const SsmArgs& a, bool f32, hipStream_t s) {
  return ssm_kv(a.K, a.V, f32, [&](auto t, auto k, auto v) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value, V = decltype(v)::value;
    REWY_LAUNCH((k_ssm_fwd<T, K, V>), dim3(a.nslot * a.H), dim3(4 * V), s, a);
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
