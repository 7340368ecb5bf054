// Product of e4m3 operands with a scale for each block of 128: argument record and
// launcher.
#pragma once
#include "layer.hpp"

namespace rewy {

struct Mm8Args {
  int M, N, K, nb;      // nb: blocks of 128 along K
  int ablk;             // 1: a scale for each row and block of a; 0: for each row
  int wrow;             // 1: a scale for each row and block of w; 0: for 128 rows
  int bias_f32;
  int64_t as, ws, ys;   // row strides of a, w (bytes) and y (elements)
  const uint8_t* a;     // [M, K]
  const uint8_t* w;     // [N, K]
  const float* sa;
  const float* sw;
  const void* bias;
  void* y;
};
// name of the kernel that the sizes take
const char* mm8_kernel(const Mm8Args& a);
hipError_t launch_mm8(const Mm8Args& a, bool f32, hipStream_t s);

}  // namespace rewy
