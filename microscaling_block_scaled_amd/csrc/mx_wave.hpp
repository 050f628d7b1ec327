// mx_wave.hpp -- reductions over a 64-lane wave on gfx950, all on the vector
// ALU: quads and rows of 16 lanes by DPP, rows and halves by permlane swaps.
// Every lane ends with the result; the order of the operations is fixed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
// the two values that lanes 16 apart (rows 0/1, 2/3), or 32 apart, hold
struct Pair { float a, b; };
__device__ __forceinline__ Pair rows_of(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return {__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])};
}
__device__ __forceinline__ Pair halves_of(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return {__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])};
}

__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0xB1>(v);   // lanes [1,0,3,2]
  v += dpp<0x4E>(v);   // lanes [2,3,0,1]
  v += dpp<0x141>(v);  // mirrored in 8 lanes
  v += dpp<0x140>(v);  // mirrored in 16 lanes
  const Pair r = rows_of(v);
  v = r.a + r.b;
  const Pair h = halves_of(v);
  return h.a + h.b;
}

// over the four lanes l, l + 16, l + 32, l + 48 only
__device__ __forceinline__ float rows_sum(float v) {
  const Pair r = rows_of(v);
  v = r.a + r.b;
  const Pair h = halves_of(v);
  return h.a + h.b;
}
__device__ __forceinline__ float rows_max(float v) {
  const Pair r = rows_of(v);
  v = __builtin_fmaxf(r.a, r.b);
  const Pair h = halves_of(v);
  return __builtin_fmaxf(h.a, h.b);
}

}  // namespace mx
