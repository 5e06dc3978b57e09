// Sums over lanes of a wave, shared by the norm kernels.
#pragma once

#include "mx4.h"

namespace convrot {

// Sum over 2^shift lanes, the same bits in each: DPP exchanges within 16 lanes,
// then swaps of 16-lane rows and of the wave's halves.
__device__ __forceinline__ float lanes_sum(float v, int shift) {
  typedef uint32_t u2v __attribute__((ext_vector_type(2)));
  v += mx4_dpp<kDppXor1>(v);
  v += mx4_dpp<kDppXor2>(v);
  v += mx4_dpp<kDppMirror8>(v);
  if (shift > 3) v += mx4_dpp<kDppMirror16>(v);
  if (shift > 4) {
    const uint32_t a = __float_as_uint(v);
    const u2v r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    v = __uint_as_float(r.x) + __uint_as_float(r.y);
  }
  if (shift > 5) {
    const uint32_t a = __float_as_uint(v);
    const u2v r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    v = __uint_as_float(r.x) + __uint_as_float(r.y);
  }
  return v;
}

}  // namespace convrot
