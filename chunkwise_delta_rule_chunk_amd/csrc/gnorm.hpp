// Group norm over a token's channels with an activation or a gate, and an 8-bit
// output: argument record and launchers.
#pragma once
#include "row.hpp"

namespace rewy {

struct GnormArgs {
  int64_t M;
  int D, G, L;             // channels, groups, channels of a group
  int act, center, quant, group, ng;  // ng: scales per row
  float eps;
  int lanes;               // lanes that hold a group, 0: any other group length
  float rL;                // 1 / L (exact where lanes hold a group)
  int64_t xs, zs, ys, dxs, dzs;  // row strides (ys: y and dy)
  const void* x;
  const void* z;
  const void* w;
  const void* b;
  const void* dy;
  void* y;
  void* q;
  float* scale;
  float* mean;             // [M, G], nullptr without center
  float* rstd;             // [M, G]
  void* dx;
  void* dz;
  void* dw;
  void* db;
  float* part;             // [nblk, 2, D] partial sums of dw and db
  int nblk;
};
// lanes that hold a group of L channels, or 0
int gnorm_lanes(int L, bool f32);
int gnorm_bwd_blocks(int64_t M, int D, bool f32);
hipError_t launch_gnorm_fwd(const GnormArgs& a, bool f32, bool wf32, hipStream_t s);
hipError_t launch_gnorm_bwd(const GnormArgs& a, bool f32, bool wf32, hipStream_t s);

}  // namespace rewy
