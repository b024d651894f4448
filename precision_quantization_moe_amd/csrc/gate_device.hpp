// gate_device.hpp -- reductions over the lanes of one token, and the scores of
// the router's gate, shared by the kernels that choose experts.
#pragma once

#include "pqm_device.hpp"

namespace pqm {

namespace {

template <typename F>
__device__ __forceinline__ uint32_t dpp_step(uint32_t v, F f) {
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));    // lane ^ 1
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));    // lane ^ 2
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));   // 7 - lane
  return f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));  // 15 - lane
}

// Reductions over the LPT lanes (16, a DPP row, or 64) that hold one token, the
// result in all of them.  Through the vector unit alone: with shuffles, which
// pass through LDS, a choice of 8 among 256 took 8 us for 16 tokens, most of
// it their latency.
template <int LPT, typename F>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, F f) {
  v = dpp_step(v, f);
  if constexpr (LPT == 64) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = f(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = f(b[0], b[1]);
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
  return __uint_as_float(group_reduce<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int LPT>
__device__ __forceinline__ float group_fmax(float v) {
  return __uint_as_float(group_reduce<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int LPT>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_reduce<LPT>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int LPT>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return group_reduce<LPT>(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}

// e^x of x <= 0 to about 2 ulp: 2^t with t = x log2(e) in two parts, the second
// through its first-order term.  Results below 2^-126 are 0; below -200 they are
// so in any case; a NaN stays one.  (Above 0 the first part may overflow, where
// the correction would make a NaN of it.)
__device__ __forceinline__ float exp_f32(float x) {
  x = __builtin_elementwise_maximum(x, -200.0f);
  const float t = x * 0x1.715476p+0f;
  const float r = __builtin_fmaf(x, 0x1.4ae0cp-26f, __builtin_fmaf(x, 0x1.715476p+0f, -t));
  const float p = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(p, r * 0x1.62e43p-1f, p);
}

// Order-preserving key of a logit, never 0 (0 marks "no expert here" and
// "already chosen").  -0 counts as +0.  The offset makes -inf 1, and of the NaN,
// which lie above inf or, with a sign, below -inf, the largest: a row's largest
// key shows whether it holds one.
constexpr uint32_t GATE_KEY_LOW = 0x007FFFFEu;
__device__ __forceinline__ uint32_t logit_key(float z) {
  const uint32_t u = __float_as_uint(z + 0.0f);  // and no signalling NaN
  return (u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u)) - GATE_KEY_LOW;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  k += GATE_KEY_LOW;
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// Through the exponential of -|z|, which cannot overflow.
__device__ __forceinline__ float sigmoid(float z) {
  const float t = exp_f32(-fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + t);
  return z < 0.0f ? t * r : r;
}

}  // namespace

}  // namespace pqm
