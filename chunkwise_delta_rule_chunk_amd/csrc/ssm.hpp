// Selective state space scan: argument record, launchers and the device
// pieces its kernels share.
//
// Per sequence and head, with the fp32 state S [K, V] and one scalar decay per
// token,
//   dt_t = softplus(raw_t + dt_bias),  g_t = -exp(A_log) dt_t,
//   S_t = exp(g_t) S_{t-1} + dt_t B_t x_t^T,   y_t = S_t^T C_t + D x_t.
// In a chunk of 64 tokens, G the inclusive prefix sum of g,
//   y_i = sum_{j<=i} exp(G_i - G_j) (C_i . B_j) dt_j x_j + exp(G_i) S_in^T C_i + D x_i
//   S_out = exp(G_L) S_in + sum_j exp(G_L - G_j) dt_j B_j x_j^T.
// Every exponent is at most 0.  A sequence is cut into segments of whole chunks;
// one workgroup walks a segment of one head with the state in its registers,
// and the states that enter the segments come from a first pass over them.
#pragma once
#include "layer.hpp"

namespace rewy {

struct SsmArgs {
  SeqArgs seq;
  int H, G, K, V, per;     // per = H / G heads share a group's B and C
  int dt_f32;
  int seg;                 // tokens of a segment (whole chunks)
  int nslot, nchunk;       // segment slots, chunk slots
  int split;               // backward: head ranges that share a group's dB and dC
  int two;                 // more than one segment per sequence is possible
  int64_t xs, bs, cs, ys, dxs, dbs, dcs;  // token strides
  const void* x;
  const void* dt;          // raw [tokens, H]
  const float* a_log;
  const float* dt_bias;
  const void* b;
  const void* c;
  const float* d;
  const float* h0;
  void* y;
  float* ht;
  // backward
  const void* dy;
  const float* dht;
  void* dx;
  void* ddt;
  float* da_log;
  void* db;
  void* dc;
  float* dd;
  float* ddt_bias;
  float* dh0;
  // workspace
  void* gates;             // [nchunk, H, 64] Gate
  float* cb;               // [nchunk, G, 10, 64 lanes, 4] C B^T, blocks of the lower triangle as C fragments
  float* sf;               // [nslot, H, K, V] local end states, then the states that enter the segments
  float* sr;               // [nslot, H, K, V] local adjoints, then the adjoints of the states that leave them
  float* gsum;             // [2, nslot, H] sum of g (log2 units) over a segment, for each direction
  void* hs;                // [nchunk, H, V/16, K/16, 64 lanes, 4] state entering each chunk (operand type)
  void* hd;                // same: adjoint of the state leaving each chunk
  float* rx;               // [H, tokens] row part of the decay gradient through the entering state
  float* cx;               // [H, tokens] column part (per unit of dt) through the leaving state
  float* ri;               // [2, H, tokens] row part inside the chunk (i > j): left of the diagonal's block of 16, in it
  float* ci;               // [2, H, tokens] column part inside the chunk (i > j): below the block, in it
  float* tot;              // [nchunk, H, 4] sums of the blocks (2, 0), (3, 0), (3, 1)
  float* cd;               // [H, tokens] the term i = j, which belongs to c and cancels in the decay gradient
  double* ends;            // [nslot, H] <state, adjoint> at each segment's end
  float* hdot;             // [nchunk, H] <S_in, dS> of the handed-over states
  float* dpart;            // [nchunk, H] partial sums of dD
  double* apart;           // [nchunk, 2, H] partial sums of dA_log and ddt_bias
  float* bcpart;           // [2, split, tokens, G, K] partial sums of dB and dC (split > 1)
};

int ssm_head_blocks(const SsmArgs& a, int hb);
hipError_t launch_ssm_prep(const SsmArgs& a, bool f32, bool bwd, hipStream_t s);
hipError_t launch_ssm_state(const SsmArgs& a, bool f32, bool both, hipStream_t s);
hipError_t launch_ssm_pass(const SsmArgs& a, bool both, hipStream_t s);
hipError_t launch_ssm_fwd(const SsmArgs& a, bool f32, hipStream_t s);
hipError_t launch_ssm_walk(const SsmArgs& a, bool f32, hipStream_t s);
hipError_t launch_ssm_chunk(const SsmArgs& a, bool f32, hipStream_t s);
hipError_t launch_ssm_gate(const SsmArgs& a, bool f32, hipStream_t s);
hipError_t launch_ssm_params(const SsmArgs& a, hipStream_t s);
hipError_t launch_ssm_recurrent(const SsmArgs& a, bool f32, hipStream_t s);

// most chunks of a segment of the bf16 backward: 512 tokens (k_ssm_gate's chains)
constexpr int SEG_CHUNKS = 8;

// ---- slots --------------------------------------------------------------------
// Pieces of L tokens of every sequence, numbered without a table.  Sequences of
// one length take ceil(T / L) slots each (at least one), all in use.  Packed ones: the
// pieces of sequence n take the slots start(n) / L + n, + 1, ...  Slots of
// different sequences never meet (a sequence of len tokens moves start / L by at
// least ceil(len / L) - 1), every sequence has at least one, and there are at
// most total / L + N.
struct Piece {
  int n;         // sequence
  int bos, eos;  // its tokens
  int k;         // piece of the sequence
  bool on;       // the slot is used
};
__device__ __forceinline__ int slots_each(const SeqArgs& q, int L) { return max((q.T + L - 1) / L, 1); }
__device__ __forceinline__ int slot_base(const SeqArgs& q, int n, int L) {
  return q.cu ? seq_start(q, n) / L + n : n * slots_each(q, L);
}
__device__ __forceinline__ Piece find_piece(const SeqArgs& q, int slot, int L) {
  int lo = 0, hi = q.N - 1;
  if (!q.cu) lo = min(slot / slots_each(q, L), hi);
  while (q.cu && lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (slot_base(q, mid, L) <= slot) lo = mid;
    else hi = mid - 1;
  }
  Piece p;
  p.n = lo;
  seq_range(q, lo, p.bos, p.eos);
  p.k = slot - slot_base(q, lo, L);
  // (an empty sequence keeps its first slot, for its final state)
  p.on = p.k >= 0 && (p.k == 0 || (int64_t)p.bos + (int64_t)p.k * L < p.eos);
  return p;
}

// Workgroup b of n in an order that gives each XCD (workgroups go to the 8 XCDs
// in turn) one contiguous range, so that neighbours, which share B and C, share
// an L2.
__device__ __forceinline__ int xcd_range(int b, int n) {
  const int x = b & 7, per = n >> 3, rem = n & 7;
  return x * per + min(x, rem) + (b >> 3);
}

// ---- gates ----------------------------------------------------------------------
// softplus at full fp32 precision (small steps dt matter relative to themselves)
__device__ __forceinline__ float softplus_full(float z) { return fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))); }

// The gates of one token, formed once per call by k_ssm_prep and read by every
// walk: dt, the chunk's inclusive prefix sum G of g (log2 units) and the
// exclusive suffix sum E = G_L - G.  The sums are taken in 64 bits.  G is kept as
// hi + lo, so that a difference G_i - G_j of neighbours is as exact after a long,
// strongly decaying stretch of the chunk as at its start (one float would be off by
// a step of G there, and the exponential by as much relative to itself).  Rows
// past the sequence's end have dt = g = 0, so G of row 63 is the chunk's total.
struct Gate {
  float dt, G, Glo, E;
};
__device__ __forceinline__ const Gate* chunk_gates(const SsmArgs& a, int cslot, int h) {
  return reinterpret_cast<const Gate*>(a.gates) + ((int64_t)cslot * a.H + h) * CH;
}
__device__ __forceinline__ float gate_bias(const SsmArgs& a, int h) { return a.dt_bias ? a.dt_bias[h] : 0.f; }

// ---- operand fragments ------------------------------------------------------------
// One 16-byte fragment per lane serves a contraction of KG<T> indices (bf16 32,
// fp32 16); lane l gives row (A) or column (B) l & 15.
template <typename T>
constexpr int KG = 64 / (int)sizeof(T);
template <typename T>
constexpr int VEC = 16 / (int)sizeof(T);

// row r0 + (l & 15) of an LDS tile, contraction k0 + VEC (l >> 4) + e
template <typename T>
__device__ __forceinline__ uint4 frag_row(const T* p, int ld, int r0, int k0) {
  const int l = lane_id();
  return *reinterpret_cast<const uint4*>(p + (r0 + (l & 15)) * ld + k0 + VEC<T> * (l >> 4));
}
// the same with the rows of a 16-row block in slot order (below)
template <typename T>
__device__ __forceinline__ uint4 frag_row_slot(const T* p, int ld, int r0, int k0);
// column c0 + (l & 15) of an LDS tile, contraction over its rows t0 .. t0 + KG - 1.
// fp32: slot 4 (l >> 4) + e is row t0 + 4 (l >> 4) + e.  bf16: two transposing
// reads, each of which gives lane l of a 16-lane group column l of the four rows
// that the group reads as 32 contiguous bytes each.  A row's pitch is 16 bytes
// past a multiple of the banks, so the eight rows that half a wave reads together
// are taken two apart (32 bytes apart in the banks: no conflicts): slot 8 (l >> 4) +
// 4 hf + e is row t0 + 16 hf + tr_row(l >> 4, e).  slot_of() gives a row's slot.
__device__ __forceinline__ int tr_row(int g, int e) { return 8 * (g & 1) + 2 * e + (g >> 1); }
template <typename T>
__device__ __forceinline__ int slot_of(int t) {
  if constexpr (std::is_same_v<T, bf16>)
    return (t & 32) + 8 * (((t >> 3) & 1) + 2 * (t & 1)) + 4 * ((t >> 4) & 1) + ((t >> 1) & 3);
  else return t;
}
// Row of a 16-row block whose slots a lane group finds together: rows in this order,
// as the rows of a product, put its C fragment's four values into neighbouring slots.
template <typename T>
__device__ __forceinline__ int slot_row(int i) {
  if constexpr (std::is_same_v<T, bf16>) return tr_row(i >> 2, i & 3);
  else return i;
}
template <typename T>
__device__ __forceinline__ uint4 frag_row_slot(const T* p, int ld, int r0, int k0) {
  const int l = lane_id();
  return *reinterpret_cast<const uint4*>(p + (r0 + slot_row<T>(l & 15)) * ld + k0 + VEC<T> * (l >> 4));
}
// LDS row for row i of a tile whose frag_col fragments shall have slot k at row k
template <typename T>
__device__ __forceinline__ int slot_place(int i) {
  if constexpr (std::is_same_v<T, bf16>) return (i & ~31) + 16 * ((i >> 2) & 1) + tr_row((i >> 3) & 3, i & 3);
  else return i;
}
// first of the four neighbouring slots of rows 16 J + slot_row(4 g + e)
template <typename T>
__device__ __forceinline__ int slot_base4(int J, int g) {
  if constexpr (std::is_same_v<T, bf16>) return 32 * (J >> 1) + 8 * g + 4 * (J & 1);
  else return 16 * J + 4 * g;
}
template <typename T>
__device__ __forceinline__ uint4 frag_col(const T* p, int ld, int t0, int c0) {
  const int l = lane_id(), g = l >> 4, r = l & 15;
  if constexpr (std::is_same_v<T, bf16>) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    const T* q = p + (t0 + tr_row(g, r >> 2)) * ld + c0 + 4 * (r & 3);
    const s16x4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(q));
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(q + 16 * ld));
    const uint2 x = __builtin_bit_cast(uint2, u), y = __builtin_bit_cast(uint2, v);
    return uint4{x.x, x.y, y.x, y.y};
  } else {
    const T* q = p + (t0 + 4 * g) * ld + c0 + r;
    return uint4{__float_as_uint(q[0]), __float_as_uint(q[ld]), __float_as_uint(q[2 * ld]), __float_as_uint(q[3 * ld])};
  }
}
// Element e of a fragment as fp32 / fragment of VEC fp32 values.
template <typename T>
__device__ __forceinline__ void frag_get(float (&f)[VEC<T>], uint4 v) {
  if constexpr (std::is_same_v<T, bf16>) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
}
// An fp32 value that meets a 16-bit operand in a product whose sum is kept in fp32
// (states, decay gradients) is given as the sum of SPLIT bf16 values, hi + mid +
// lo: 24 bits, as many as fp32 has, whether or not the call hands out the final state (two
// pieces, 17 bits, would make a prompt's y depend on that).  fp32 operands are one piece.
template <typename T>
constexpr int SPLIT = std::is_same_v<T, bf16> ? 3 : 1;
template <typename T, int NS>
__device__ __forceinline__ void frag_split(uint4 (&out)[NS], const float (&f)[VEC<T>]) {
  if constexpr (std::is_same_v<T, bf16>) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = f[e];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = __builtin_bit_cast(uint32_t, bf16x2{(bf16)x[2 * i], (bf16)x[2 * i + 1]});
        asm("" : "+v"(w[i]));
        if (s + 1 < NS) {
          x[2 * i] -= __uint_as_float(w[i] << 16);
          x[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
        }
      }
      out[s] = uint4{w[0], w[1], w[2], w[3]};
    }
  } else {
    static_assert(NS == 1, "");
    out[0] = uint4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  }
}
// Fragment q of a contraction over the rows of a matrix held as C fragments, acc[i]
// = rows 16 i + 4 (l >> 4) .. + 3 (partner: frag_row of a tile
// that store_acc_order wrote).
template <typename T, int NS, int NT>
__device__ __forceinline__ void frag_acc(uint4 (&out)[NS], const f32x4 (&acc)[NT], int q) {
  float f[VEC<T>];
  if constexpr (std::is_same_v<T, bf16>) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = acc[2 * q][e];
      f[4 + e] = acc[2 * q + 1][e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = acc[q][e];
  }
  frag_split<T, NS>(out, f);
}
// four values as one store of the type
template <typename T>
__device__ __forceinline__ void st4(T* p, const f32x4& v) {
  if constexpr (std::is_same_v<T, bf16>) {
    bf16x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = (bf16)v[e];
    *reinterpret_cast<bf16x4*>(p) = o;
  } else {
    *reinterpret_cast<f32x4*>(p) = v;
  }
}
template <typename T>
__device__ __forceinline__ f32x4 ld4(const T* p) {
  if constexpr (std::is_same_v<T, bf16>) {
    const bf16x4 v = *reinterpret_cast<const bf16x4*>(p);
    return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
  } else {
    return *reinterpret_cast<const f32x4*>(p);
  }
}

// A chunk's rows of a token-major tensor, columns col .. + C - 1, of which the first
// cols belong to the caller (rows past len read as zeros; the others hold whatever
// the row holds there, or zeros behind the last row's)
template <typename T, int C, int NTH>
__device__ __forceinline__ void load_tile(TileRegs<T, CH, C, NTH>& r, const void* base, int64_t tok, int64_t stride,
                                          int col, int len, int cols) {
  const T* p = reinterpret_cast<const T*>(base) + tok * stride + col;
  r.load(gbuf(p, tile_bytes<T>(len, stride, cols)), stride, threadIdx.x);
}

// State update S = exp(G_L) S + sum_t K_t (al_t u_t)^T for the wave's CT tiles of 16
// columns: A operand K^T (columns of sk, read once for the CT tiles), B operand al u
// (ut: columns of the u tile; scaled and split; sal holds al in slot order).
template <typename T, int K, int CT, int NS>
__device__ __forceinline__ void state_update(f32x4 (&S)[CT][K / 16], const T* sk, int ldk,
                                             const uint4 (&ut)[CT][CH / KG<T>], const float* sal, float dec) {
  constexpr int NQ = CH / KG<T>, VE = VEC<T>;
  const int g = lane_id() >> 4;
  uint4 uf[CT][NQ][NS];
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      float f[VE];
      frag_get<T>(f, ut[ct][q]);
#pragma unroll
      for (int e = 0; e < VE; e += 4) {
        const f32x4 al = *reinterpret_cast<const f32x4*>(sal + q * KG<T> + VE * g + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[e + i] *= al[i];
      }
      frag_split<T, NS>(uf[ct][q], f);
    }
#pragma unroll
  for (int nt = 0; nt < K / 16; ++nt) {
    f32x4 u[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) u[ct] = zero4();
    uint4 kf[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) kf[q] = frag_col<T>(sk, ldk, q * KG<T>, 16 * nt);
#pragma unroll
    for (int s = NS - 1; s >= 0; --s)
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) mma16B<T>(u[ct], kf[q], uf[ct][q][s]);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[ct][nt][i] = dec * S[ct][nt][i] + u[ct][i];
  }
}

// Whether a register tile holds an infinity or NaN (an exponent of ones).
template <typename T, int C, int NTH>
__device__ __forceinline__ bool tile_not_finite(const TileRegs<T, CH, C, NTH>& t) {
  constexpr uint32_t EXP = std::is_same_v<T, bf16> ? 0x7f807f80u : 0x7f800000u;
  constexpr uint32_t ONE = std::is_same_v<T, bf16> ? 0x00800080u : 0x00800000u;
  uint32_t s = 0;  // (the largest exponent plus one reaches the sign's place)
#pragma unroll
  for (int j = 0; j < TileRegs<T, CH, C, NTH>::N; ++j)
    s |= ((t.r[j].x & EXP) + ONE) | ((t.r[j].y & EXP) + ONE) | ((t.r[j].z & EXP) + ONE) | ((t.r[j].w & EXP) + ONE);
  return (s & ((EXP + ONE) & 0x80008000u)) != 0;
}

// Block b = 0 .. 9 of the lower triangle of 4 x 4 blocks, row by row.
__device__ __forceinline__ void tri_block(int b, int& I, int& J) {
  I = b >= 6 ? 3 : b >= 3 ? 2 : b >= 1 ? 1 : 0;
  J = b - I * (I + 1) / 2;
}

// A tile into LDS with the columns of each 32 in the slot order of frag_acc, so that
// frag_row gives the partner of a fragment made of C fragments (fp32: as they are).
template <typename T, int C, int NTH>
__device__ __forceinline__ void store_acc_order(const TileRegs<T, CH, C, NTH>& t, T* s, int ls) {
  if constexpr (std::is_same_v<T, bf16>) {
#pragma unroll
    for (int j = 0; j < TileRegs<T, CH, C, NTH>::N; ++j) {
      const int idx = threadIdx.x + j * NTH, row = idx / (C / 8), c = (idx - row * (C / 8)) * 8;
      if (idx < TileRegs<T, CH, C, NTH>::TOTAL) {
        T* p = s + row * ls + (c & ~31) + 8 * ((c >> 2) & 3) + 4 * ((c >> 4) & 1);
        *reinterpret_cast<uint2*>(p) = uint2{t.r[j].x, t.r[j].y};
        *reinterpret_cast<uint2*>(p + 8) = uint2{t.r[j].z, t.r[j].w};
      }
    }
  } else {
    t.store(s, ls, threadIdx.x);
  }
}

// Heads side by side in one workgroup: as many heads of a group as fit in its columns
// share the B and C tiles.
template <typename T>
constexpr int HEAD_COLS = std::is_same_v<T, bf16> ? 128 : 64;
// blocks of HB heads of all groups
__device__ __forceinline__ int head_blocks(const SsmArgs& a, int HB) { return a.G * ((a.per + HB - 1) / HB); }

// the (type, K, V) variants of a kernel
template <typename F>
hipError_t ssm_kv(int K, int V, bool f32, F&& f) {
  auto v_of = [&](auto t, auto k) -> hipError_t {
    if (V == 32) return f(t, k, std::integral_constant<int, 32>{});
    if (V == 64) return f(t, k, std::integral_constant<int, 64>{});
    if constexpr (std::is_same_v<decltype(t), bf16>)
      if (V == 128) return f(t, k, std::integral_constant<int, 128>{});
    return hipErrorInvalidValue;
  };
  auto k_of = [&](auto t) -> hipError_t {
    if (K == 32) return v_of(t, std::integral_constant<int, 32>{});
    if (K == 64) return v_of(t, std::integral_constant<int, 64>{});
    if constexpr (std::is_same_v<decltype(t), bf16>)
      if (K == 128) return v_of(t, std::integral_constant<int, 128>{});
    return hipErrorInvalidValue;
  };
  return f32 ? k_of(float{}) : k_of(bf16{});
}
// the same with the heads of a workgroup: as many as fit in COLS columns, or one where a
// group has no two heads to put side by side
template <int COLS, typename F>
hipError_t ssm_kv_heads(const SsmArgs& a, bool f32, F&& f) {
  return ssm_kv(a.K, a.V, f32, [&](auto t, auto k, auto v) -> hipError_t {
    constexpr int HB = std::max(std::min(COLS, HEAD_COLS<decltype(t)>) / decltype(v)::value, 1);
    if constexpr (HB > 1)
      if (a.per == 1) return f(t, k, v, std::integral_constant<int, 1>{});
    return f(t, k, v, std::integral_constant<int, HB>{});
  });
}

}  // namespace rewy
