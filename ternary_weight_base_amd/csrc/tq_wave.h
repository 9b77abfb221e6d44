// tq_wave.h -- sums over a wave's lanes in fp32 and double, and a double's
// rounding to fp32, for the kernels between the projections.  Internal to the
// library.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq_device.h"

namespace tqdev {

// In every lane: the sum over its row of 16 lanes, in a fixed order.
__device__ __forceinline__ float row16_sum(float v) {
  v += __int_as_float(dpp_move<kDppSwap1>(__float_as_int(v)));
  v += __int_as_float(dpp_move<kDppSwap2>(__float_as_int(v)));
  v += __int_as_float(dpp_move<kDppRor4>(__float_as_int(v)));
  return v + __int_as_float(dpp_move<kDppRor8>(__float_as_int(v)));
}

// The double sum over the 64 lanes, wave-uniform, in a fixed order.
template <int CTRL>
__device__ __forceinline__ double dpp_move(double v) {
  const long long b = __double_as_longlong(v);
  const int lo = dpp_move<CTRL>((int)b), hi = dpp_move<CTRL>((int)(b >> 32));
  return __longlong_as_double(((long long)hi << 32) | (uint32_t)lo);
}
__device__ __forceinline__ double wave_sum64(double v) {
  v += dpp_move<kDppSwap1>(v);
  v += dpp_move<kDppSwap2>(v);
  v += dpp_move<kDppRor4>(v);
  v += dpp_move<kDppRor8>(v);
  const long long b = __double_as_longlong(v);
  double r[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int lo = __builtin_amdgcn_readlane((int)b, 16 * i), hi = __builtin_amdgcn_readlane((int)(b >> 32), 16 * i);
    r[i] = __longlong_as_double(((long long)hi << 32) | (uint32_t)lo);
  }
  return (r[0] + r[1]) + (r[2] + r[3]);
}

// A double rounded to fp32, kept as such: where the result is rounded on to
// fp16 the compiler would otherwise merge the two roundings into one from
// the double, a long software conversion.  (The two together are off by at
// most 2^-24 of the value more than half an fp16 step.)
__device__ __forceinline__ float round_f32(double d) {
  float f = (float)d;
  asm("" : "+v"(f));
  return f;
}

}  // namespace tqdev
