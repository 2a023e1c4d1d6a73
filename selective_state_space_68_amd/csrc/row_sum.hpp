// Sums over parts of a wave, for the kernels whose rows are parts of one.  (Apart from device_common.hpp, by whose text the
// stored counters of the scans are known to be of the present kernels.)
#pragma once

#include "device_common.hpp"

namespace ssm {
namespace {

// The sum over N = 8 or 16 neighbouring lanes: quads, then the quads of 8, then of 16.
template <int N>
__device__ __forceinline__ float row_sum(float v) {
  static_assert(N == 8 || N == 16, "");
  v += dpp_mov<0xb1, 0xf, true>(0.0f, v);           // quad_perm [1, 0, 3, 2]
  v += dpp_mov<0x4e, 0xf, true>(0.0f, v);           // quad_perm [2, 3, 0, 1]
  v += dpp_mov<0x141, 0xf, true>(0.0f, v);          // row_half_mirror
  if constexpr (N == 16) v += dpp_mov<0x140, 0xf, true>(0.0f, v);   // row_mirror
  return v;
}

}  // namespace
}  // namespace ssm
