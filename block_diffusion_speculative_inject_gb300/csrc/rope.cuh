// Shared by the kernels that turn rows by their positions: the angle of a phase, the turned pair, wide accesses.
#pragma once
#include "kv8.cuh"

namespace dflash {

// (cos, sin) of a phase in units of 2^-64 turns: the nearest quarter turn is split off exactly,
// the rest, at most an eighth of a turn, goes to sincospif
__device__ __forceinline__ float2 phase_cs(uint64_t ph) {
  const uint32_t quarter = (uint32_t)((ph + (1ull << 61)) >> 62);
  const int64_t rest = (int64_t)(ph - ((uint64_t)quarter << 62));
  float s, c;
  sincospif((float)rest * 0x1p-63f, &s, &c);
  if (quarter & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  return (quarter & 2) ? make_float2(-c, -s) : make_float2(c, s);
}

// the turned pair; one contraction for every instance, so that all of them give the same bits
__device__ __forceinline__ float2 turned(float x, float y, float2 k) {
  return make_float2(fmaf(x, k.x, -__fmul_rn(y, k.y)), fmaf(y, k.x, __fmul_rn(x, k.y)));
}

template <typename T, int N>
struct alignas(N * sizeof(T)) Vec {
  T v[N];
};

}  // namespace dflash
