// norm_device.hpp -- sums over a wave and the roundings of the RMS norm, shared
// by the kernels that normalise.
#pragma once

#include "pqm_device.hpp"

namespace pqm {

namespace {

// 8 weights from column c on, as binary32.
template <bool WF32>
__device__ __forceinline__ void load_w8(const void *__restrict__ w, int64_t c, float (&o)[8]) {
  if constexpr (WF32) {
    const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + c);
    const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + c + 4);
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
    o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w) + c);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = bf16_lo_f32(u[i]);
      o[2 * i + 1] = bf16_hi_f32(u[i]);
    }
  }
}

__device__ __forceinline__ double join(uint32_t lo, uint32_t hi) {
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// v of another lane of the same 16, of the other 16 of 32, of the other 32.
template <int CTRL>
__device__ __forceinline__ float other(float v) {
  return __uint_as_float(
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double other(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, 0xF, 0xF, false);
  return join(lo, hi);
}
__device__ __forceinline__ float add_halves(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t w = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
__device__ __forceinline__ double add_halves(double v) {
  uint64_t u = __builtin_bit_cast(uint64_t, v);
  const auto al = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
  const auto ah = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  u = __builtin_bit_cast(uint64_t, join(al[0], ah[0]) + join(al[1], ah[1]));
  const auto bl = __builtin_amdgcn_permlane32_swap((uint32_t)u, (uint32_t)u, false, false);
  const auto bh = __builtin_amdgcn_permlane32_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  return join(bl[0], bh[0]) + join(bl[1], bh[1]);
}

// Sum over a wave, the same in every lane, through the vector unit alone: six
// shuffles, which pass through LDS, take about four times as long.
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
  v += other<0xB1>(v);   // lane ^ 1
  v += other<0x4E>(v);   // lane ^ 2
  v += other<0x141>(v);  // 7 - lane
  v += other<0x140>(v);  // 15 - lane
  return add_halves(v);
}

// 1 / sqrt(m): the hardware's estimate (about 2^-27) and one Newton step, which
// would make a NaN of the 0 that an infinite m gives.
__device__ __forceinline__ double inverse_root(double m) {
  const double r = __builtin_amdgcn_rsq(m);
  const double s = __builtin_fma(0.5 * r, __builtin_fma(-m * r, r, 1.0), r);
  return r == 0.0 ? r : s;
}

// The binary32 value from which d rounds to bf16 as it would at once: where the
// nearest one is the middle of two, its neighbour on d's side.
__device__ __forceinline__ float before_bf16(double d) {
  const float f = (float)d;
  const double a = __builtin_fabs((double)f), b = __builtin_fabs(d);
  const uint32_t u = __float_as_uint(f);
  return (u & 0xFFFFu) == 0x8000u && a != b ? __uint_as_float(a < b ? u + 1 : u - 1) : f;
}

}  // namespace

}  // namespace pqm
