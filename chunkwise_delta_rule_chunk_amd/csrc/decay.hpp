// Linear attention with one constant decay for each head: argument record and
// launchers.
//
// Per sequence and head, with the fp32 state S [K, V] and lam = exp(g),
//   S_t = lam S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,
// and backward, with L_t the adjoint of S_t from what follows token t (L of the
// last token: dht) and R_t = L_t + scale q_t do_t^T, L_{t-1} = lam R_t,
//   dq_t = scale S_t do_t,  dk_t = R_t v_t,  dv_t = R_t^T k_t,  dh0 = lam R_0.
// In a chunk of n tokens (rows i, j), S_in the state that enters and L the
// adjoint of the state that leaves it,
//   o_i  = scale (sum_{j<=i} lam^(i-j) (q_i . k_j) v_j + lam^(i+1) S_in^T q_i)
//   dq_i = scale (sum_{j<=i} lam^(i-j) (do_i . v_j) k_j + lam^(i+1) S_in do_i)
//   dv_j = sum_{i>=j} scale lam^(i-j) (k_j . q_i) do_i + lam^(n-1-j) L^T k_j
//   dk_j = sum_{i>=j} scale lam^(i-j) (v_j . do_i) q_i + lam^(n-1-j) L v_j
//   S_out = lam^n S_in + sum_j lam^(n-1-j) k_j v_j^T
//   L_in  = lam^n L    + sum_i scale lam^(i+1) q_i do_i^T.
// The four outputs are one walk with the operands in other places: rows A and B
// meet in the coefficients, rows C are summed by them, and the state is that of B
// and C.  Every exponent of lam is at least 0.
#pragma once
#include "ssm.hpp"

namespace rewy {

// what a walk forms
enum { DECAY_O = 0, DECAY_DQ = 1, DECAY_DV = 2, DECAY_DK = 3 };

struct DecayArgs {
  SeqArgs seq;
  int H, G, K, V, per;     // per = H / G heads share a key and value head
  int seg;                 // tokens of a segment (whole chunks)
  int nslot;               // segment slots (ssm.hpp)
  int two;                 // more than one segment per sequence is possible
  float scale;
  int64_t qs, ks, vs, os;  // token strides of q, k, v, o (backward: do)
  int64_t dqs, dks, dvs;
  const void* q;
  const void* k;
  const void* v;
  const float* g;          // [H], log of the decay
  const float* h0;
  void* o;
  float* ht;
  // backward
  const void* dO;
  const float* dht;
  void* dq;
  void* dk;
  void* dv;
  float* dh0;
  // workspace
  float* sf;               // [nslot, H, K, V] the segments' own end states, then the states that enter them
  float* sr;               // [nslot, H, K, V] the segments' own adjoints, then the adjoints of the states that leave them
  float* kpart;            // [tokens, H, K] dk before the heads of a group are summed (per > 1)
  float* vpart;            // [tokens, H, V] dv, the same
};

// directions of the states: bit 0 forward, bit 1 reverse
hipError_t launch_decay_state(const DecayArgs& a, bool f32, int dirs, hipStream_t s);
hipError_t launch_decay_pass(const DecayArgs& a, int dirs, hipStream_t s);
hipError_t launch_decay_fwd(const DecayArgs& a, bool f32, hipStream_t s);
hipError_t launch_decay_bwd(const DecayArgs& a, bool f32, hipStream_t s);
hipError_t launch_decay_sum(const DecayArgs& a, bool f32, hipStream_t s);
hipError_t launch_decay_recurrent(const DecayArgs& a, bool f32, hipStream_t s);

}  // namespace rewy
