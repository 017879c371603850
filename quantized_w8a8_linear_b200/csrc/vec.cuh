// vec.cuh -- 16-byte vectors of 16-bit values and warp sums, shared by the
// layer norm and the adapters.
#pragma once
#include <type_traits>

#include "common.cuh"

namespace qlin {

// 8 16-bit values <-> fp32
template <typename T>
__device__ __forceinline__ void widen8(const uint4& u, float (&f)[8]) {
  uint16_t h[8];
  unpack8(u, h);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = to_f<T>(h[i]);
}

// Two fp32 values rounded to a 16-bit pair (lo in the lower half), one conversion.
template <typename T>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  uint32_t d;
  if constexpr (std::is_same<T, __nv_bfloat16>::value) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
template <typename T>
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
  return make_uint4(narrow2<T>(f[0], f[1]), narrow2<T>(f[2], f[3]), narrow2<T>(f[4], f[5]), narrow2<T>(f[6], f[7]));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace qlin
