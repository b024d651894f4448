// moe_gate.hip -- the router's gate: from logits [T, E] to the k experts of
// each token and their probabilities, the per-expert counts and the balance
// loss, and the gradient of both with respect to the logits.
//
// v = softmax(z) or sigmoid(z); p = v / sum_e v (a token's shares; softmax: v).
// The choice is the k largest logits, ties to the lowest index: v grows with
// z, so no rounding of v decides it.  prob_j = scale v_j / sum over the
// chosen (renormalised) or scale v_j.  With c_e the valid tokens that chose e,
// P_e = sum of p over the valid tokens, Tv their number:
//   loss = coef E / (k Tv^2) sum_e c_e P_e.
// Gradient, the counts held fixed: u_e = d prob / d v at the chosen experts,
// h_e = d_loss coef E c_e / (k Tv^2) at every expert's share:
//   softmax: dz = p (u + h - sum p (u + h))
//   sigmoid: dz = v (1 - v) (u + (h - sum p h) / sum v).
#include "gate_device.hpp"
#include "pqm_device.hpp"
#include "pqm_internal.hpp"
#include "pqmoe.h"

#include <type_traits>

namespace pqm {

namespace {

constexpr int GATE_MAX_EXPERTS = 1024;
constexpr int GATE_MAX_K = 16;
constexpr int64_t GATE_MAX_VALUES = 0x7FFFFFFF;  // tokens (k + 1)
constexpr int64_t GATE_GROUPS = 256;  // workgroups whose partial sums the last kernel joins

template <int J>
using lane_c = std::integral_constant<int, J>;

// The value of the group's lane J in all its lanes.
template <int LPT, int J>
__device__ __forceinline__ uint32_t group_lane(uint32_t v) {
  if constexpr (LPT == 64) return (uint32_t)__builtin_amdgcn_readlane((int)v, J);
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x150 + J, 0xF, 0xF, false);
}

constexpr uint32_t GATE_NONE = 0x80000000u;  // an offset past every buffer

__device__ __forceinline__ __amdgpu_buffer_rsrc_t gate_buffer(const void *p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, bytes, 0x00020000);
}

// The logits of the tokens t0 .. t0 + groups - 1 as a buffer: what lies past the
// last token reads as 0, and writes there are dropped.
template <int B>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t gate_rows(const void *z, int64_t t0, int64_t T,
                                                            int groups, int E) {
  const int64_t n = min(T - t0, (int64_t)groups);
  return gate_buffer(static_cast<const uint8_t *>(z) + t0 * E * B, (int)(n * E * B));
}

template <bool ZF32>
__device__ __forceinline__ float load_logit(const __amdgpu_buffer_rsrc_t &r, uint32_t i) {
  if constexpr (ZF32)
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)(4 * i), 0, 0));
  return __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)(2 * i), 0, 0) << 16);
}

}  // namespace

// LPT lanes hold one token, VPL logits each (expert i LPT + lane); the choice
// takes k turns of a maximum over the keys, the lowest index that has it, and
// its removal.  Bound by those turns' vector instructions (about 40 a turn for
// 128 experts, shared by four tokens) and, for few tokens, by their latency:
// 16384 x 128, top-8, with the loss 13.2 us (k_moe_balance 4 of them, floor
// 1.8), 16 x 256 without 4.2 (an empty launch: 1.6); 0.4 us more with the removal
// found by comparing each index again.  SUMS: each workgroup also leaves its
// counts and share sums in part_cnt / part_sum [gridDim.x][E] (and its valid
// tokens in part_valid).
template <int LPT, int VPL, bool ZF32, bool SOFTMAX, bool SUMS>
__global__ __launch_bounds__(1024) void k_moe_gate(
    const void *__restrict__ z, const uint8_t *__restrict__ mask, int64_t T, int E, int k,
    int renorm, float scale, int32_t *__restrict__ ids, float *__restrict__ prob,
    int32_t *__restrict__ part_cnt, float *__restrict__ part_sum, int32_t *__restrict__ part_valid,
    uint32_t *__restrict__ ticket) {
  extern __shared__ int32_t sh[];  // SUMS: counts [E], share sums [waves][E]
  const int l = threadIdx.x % LPT;
  const int groups = blockDim.x / LPT;
  float acc[VPL] = {};
  int nvalid = 0;
  if constexpr (SUMS) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;  // for k_moe_balance
    for (int e = threadIdx.x; e < E; e += blockDim.x) sh[e] = 0;
    __syncthreads();
  }
  for (int64_t t0 = (int64_t)blockIdx.x * groups; t0 < T; t0 += (int64_t)gridDim.x * groups) {
    const int n = (int)min(T - t0, (int64_t)groups), mine = threadIdx.x / LPT;
    const int64_t t = t0 + mine;
    const bool live = mine < n;
    const __amdgpu_buffer_rsrc_t zr = gate_rows<ZF32 ? 4 : 2>(z, t0, T, groups, E);
    const uint32_t row = mine * E;
    float v[VPL];
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = load_logit<ZF32>(zr, row + i * LPT + l);
    const uint32_t mk = __builtin_amdgcn_raw_buffer_load_b8(
        gate_buffer(mask + (mask ? t0 : 0), mask ? n : 0), mine, 0, 0);
    const bool valid = live && (!mask || mk);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const bool in = i * LPT + l < E;
      v[i] = in && valid ? v[i] : -__builtin_inff();
      key[i] = in ? logit_key(v[i]) : 0u;
    }
    int my_id = 0;
    uint32_t my_key = 0;
    for (int j = 0; j < k; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) m = max(m, key[i]);
      m = group_max<LPT>(m);
      // this lane's first expert that has the maximum, and the lowest lane's of
      // them: the conditions stay in scalar registers
      uint32_t mine_at = UINT32_MAX;
      bool hit[VPL], seen = false;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const bool eq = key[i] == m;
        hit[i] = eq && !seen;
        seen = seen || eq;
        mine_at = hit[i] ? (uint32_t)(i * LPT + l) : mine_at;
      }
      const uint32_t at = group_min<LPT>(mine_at);
      const bool won = at == mine_at;
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = hit[i] && won ? 0u : key[i];
      if (l == j) {
        my_id = (int)at;
        my_key = m;
      }
    }
    float top = key_logit(group_lane<LPT, 0>(my_key));
    const float my_z = l < k ? key_logit(my_key) : -__builtin_inff();
    // shares: exp(z - top) or sigmoid(z), and their sum; an all -inf row has none,
    // and one with a NaN, which is its top then, NaN
    if (top == -__builtin_inff()) top = 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      v[i] = SOFTMAX ? exp_f32(v[i] - top) : sigmoid(v[i]);
      if (i * LPT + l >= E) v[i] = 0.0f;
      sum += v[i];
    }
    sum = group_sum<LPT>(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // a NaN stays one
    float w = l < k ? (SOFTMAX ? exp_f32(my_z - top) : sigmoid(my_z)) : 0.0f;
    if (renorm) {
      const float total = group_sum<LPT>(w);
      w = total == 0.0f ? 0.0f : w / total;
    } else if (SOFTMAX) {
      w *= inv;
    }
    if (!SOFTMAX && top != top) w = top;
    if (live && l < k) {
      // a token that the mask leaves out is not read: experts in turn, so that
      // padding loads all of them alike, and no weight
      ids[t * k + l] = valid ? my_id : (int32_t)((uint32_t)(t * k + l) % (uint32_t)E);
      prob[t * k + l] = valid ? w * scale : 0.0f;
    }
    if constexpr (SUMS) {
      if (valid) {
        if (l < k) atomicAdd(&sh[my_id], 1);
        if (l == 0) ++nvalid;
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] += v[i] * inv;
      }
    }
  }
  if constexpr (SUMS) {
    float *shs = reinterpret_cast<float *>(sh + E);
    const int wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
#pragma unroll
      for (int o = LPT; o < 64; o <<= 1) acc[i] += __shfl_xor(acc[i], o, 64);
      const int e = i * LPT + l;
      if ((threadIdx.x & 63) < LPT && e < E) shs[wave * E + e] = acc[i];
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) nvalid += __shfl_xor(nvalid, o, 64);
    int32_t *shv = sh + E + nw * E;
    if ((threadIdx.x & 63) == 0) shv[wave] = nvalid;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      float s = 0.0f;
      for (int w = 0; w < nw; ++w) s += shs[w * E + e];
      part_sum[(int64_t)blockIdx.x * E + e] = s;
      part_cnt[(int64_t)blockIdx.x * E + e] = sh[e];
    }
    if (threadIdx.x == 0) {
      int n = 0;
      for (int w = 0; w < nw; ++w) n += shv[w];
      part_valid[blockIdx.x] = n;
    }
  }
}

// Joins the P workgroups' sums, 32 columns a workgroup (32 row groups of them,
// eight rows of a group in flight), and forms the loss: each workgroup leaves
// its columns' part, and the one that draws the last ticket adds the parts.
// Every sum has one order, whichever workgroup comes last.
__global__ __launch_bounds__(1024) void k_moe_balance(
    const int32_t *__restrict__ part_cnt, const float *__restrict__ part_sum,
    const int32_t *__restrict__ part_valid, int P, int E, int k, float coef, float *part_dot,
    uint32_t *ticket, int32_t *__restrict__ counts, float *__restrict__ prob_sum,
    float *__restrict__ loss) {
  __shared__ float fs[32][33];
  __shared__ int32_t is[32][33], vs[16];
  __shared__ bool last;
  const int col = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + col;
  float s = 0.0f;
  int c = 0, nv = 0;
  for (int p0 = grp; p0 < P; p0 += 256) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int p = p0 + 32 * i;
      const bool in = p < P && e < E;
      s += in ? part_sum[(int64_t)p * E + e] : 0.0f;
      c += in ? part_cnt[(int64_t)p * E + e] : 0;
    }
  }
  for (int p = threadIdx.x; p < P; p += 1024) nv += part_valid[p];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) nv += __shfl_xor(nv, o, 64);
  if ((threadIdx.x & 63) == 0) vs[threadIdx.x >> 6] = nv;
  fs[grp][col] = s;
  is[grp][col] = c;
  __syncthreads();
  for (int w = 16; w > 0; w >>= 1) {
    if (grp < w) {
      fs[grp][col] += fs[grp + w][col];
      is[grp][col] += is[grp + w][col];
    }
    __syncthreads();
  }
  int valid = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) valid += vs[w];
  if (threadIdx.x < 64) {
    float dot = 0.0f;
    if (threadIdx.x < 32 && e < E) {
      s = fs[0][col];
      c = is[0][col];
      prob_sum[e] = s;
      counts[e] = c;
      // the share of the assignments times the mean share of the probability
      if (valid) dot = (float)c / ((float)k * (float)valid) * (s / (float)valid);
    }
    dot = group_sum<64>(dot);
    if (threadIdx.x == 0) {
      __hip_atomic_store(&part_dot[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
             gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last || threadIdx.x >= 64) return;
  float dot = threadIdx.x < gridDim.x  // at most 32 workgroups
                  ? __hip_atomic_load(&part_dot[threadIdx.x], __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT)
                  : 0.0f;
  dot = group_sum<64>(dot);
  if (threadIdx.x == 0) {
    counts[E] = valid;
    loss[0] = coef * (float)E * dot;
  }
}

// The gradient, laid out as the forward kernel.  16384 x 128 6.6 us, 4093 x 256
// in bf16 4.6 (floors 3.5 and 0.9; an empty launch takes 1.6).  Every load goes
// out before the first is used (2.2 and 2.8 us more with the counts, the ids
// and the chosen logits waited for in turn); comparing each expert with each of
// the k ids instead of the row in LDS took 0.8 us more.
template <int LPT, int VPL, bool ZF32, bool SOFTMAX>
__global__ __launch_bounds__(256) void k_moe_gate_backward(
    const void *__restrict__ z, const uint8_t *__restrict__ mask, int64_t T, int E, int k,
    int renorm, float scale, float coef, const int32_t *__restrict__ ids,
    const float *__restrict__ d_prob, const int32_t *__restrict__ counts,
    const float *__restrict__ d_loss, void *__restrict__ d_z, int out_f32) {
  const int l = threadIdx.x % LPT;
  constexpr int groups = 256 / LPT;
  // A token's row of E values, for what one lane has and another needs: its
  // shares, then u, 0 but at the chosen experts.  (16 more: tokens in other
  // banks.)  One wave's LDS accesses keep their order, so the fences hold only
  // the compiler.
  __shared__ float rows[groups][VPL * LPT + 16];
  float *mine = rows[threadIdx.x / LPT];
  // counts, empty without a loss: every load below goes out before one is used
  const __amdgpu_buffer_rsrc_t cr = gate_buffer(counts, counts ? 4 * (E + 1) : 0);
  int cnt[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    cnt[i] = (int)__builtin_amdgcn_raw_buffer_load_b32(cr, 4 * (i * LPT + l), 0, 0);
  const float valid_tokens = counts ? (float)counts[E] : 0.0f, dl = counts ? d_loss[0] : 0.0f;
  for (int64_t t0 = (int64_t)blockIdx.x * groups; t0 < T; t0 += (int64_t)gridDim.x * groups) {
    const int n = (int)min(T - t0, (int64_t)groups), in = threadIdx.x / LPT;
    const __amdgpu_buffer_rsrc_t zr = gate_rows<ZF32 ? 4 : 2>(z, t0, T, groups, E);
    const uint32_t row = in * E, at = l < k ? 4 * (in * k + l) : GATE_NONE;
    float v[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = load_logit<ZF32>(zr, row + i * LPT + l);
    const int id =
        (int)__builtin_amdgcn_raw_buffer_load_b32(gate_buffer(ids + t0 * k, 4 * n * k), (int)at, 0, 0);
    const float dp = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
        gate_buffer(d_prob + (d_prob ? t0 * k : 0), d_prob ? 4 * n * k : 0), (int)at, 0, 0));
    const uint32_t mk = __builtin_amdgcn_raw_buffer_load_b8(
        gate_buffer(mask + (mask ? t0 : 0), mask ? n : 0), in, 0, 0);
    const bool valid = in < n && (!mask || mk);
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      v[i] = i * LPT + l < E && valid ? v[i] : -__builtin_inff();
      top = fmaxf(top, v[i]);
    }
    if constexpr (SOFTMAX) {
      top = group_fmax<LPT>(top);
      if (!(top > -__builtin_inff())) top = 0.0f;
    }
    // slope: v (1 - v) of a sigmoid, the same for z and -z; 1 - v of a rounded v
    // would have no digits left near 1
    float sum = 0.0f, slope[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if constexpr (SOFTMAX) {
        v[i] = exp_f32(v[i] - top);
      } else {
        const float t = exp_f32(-fabsf(v[i])), r = __builtin_amdgcn_rcpf(1.0f + t);
        slope[i] = t * r * r;
        v[i] = v[i] < 0.0f ? t * r : r;
      }
      if (i * LPT + l >= E) v[i] = 0.0f;
      sum += v[i];
    }
    sum = group_sum<LPT>(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // a NaN stays one, in every term below
    // From here on v is the share, and u of a renormalised sigmoid the gradient
    // by the share.  By the score it would be 1 / sum v times as large, which
    // leaves binary32 where all scores are near 2^-120.
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] *= inv;
    // the chosen experts' shares, from the lanes that hold them
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < VPL; ++i) mine[i * LPT + l] = v[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int my_id = valid && l < k && id >= 0 && id < E ? id : -1;
    const float my_v = my_id >= 0 ? mine[my_id] : 0.0f;
    float my_d = my_id >= 0 ? dp * scale : 0.0f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < VPL; ++i) mine[i * LPT + l] = 0.0f;
    if (renorm) {
      const float total = group_sum<LPT>(my_v);
      const float dot = group_sum<LPT>(my_d * my_v);
      const float it = total > 0.0f ? 1.0f / total : 0.0f;
      // d (total - v) - (dot - d v) over total^2: 0 of itself where k is 1, while
      // d - dot / total leaves a rounding of d
      my_d = (my_d * (total - my_v) - (dot - my_d * my_v)) * it * it;
    }
    // An expert chosen twice gets the sum, in both its places; then each place
    // lays its value where the expert's lane finds it.
    float total = 0.0f;
    const auto add = [&](auto j) {
      if (decltype(j)::value >= k) return;  // the same for every lane
      const int id = (int)group_lane<LPT, decltype(j)::value>((uint32_t)my_id);
      const float d = __uint_as_float(group_lane<LPT, decltype(j)::value>(__float_as_uint(my_d)));
      total += id == my_id ? d : 0.0f;
    };
    add(lane_c<0>{}); add(lane_c<1>{}); add(lane_c<2>{}); add(lane_c<3>{});
    add(lane_c<4>{}); add(lane_c<5>{}); add(lane_c<6>{}); add(lane_c<7>{});
    if (k > 8) {
      add(lane_c<8>{}); add(lane_c<9>{}); add(lane_c<10>{}); add(lane_c<11>{});
      add(lane_c<12>{}); add(lane_c<13>{}); add(lane_c<14>{}); add(lane_c<15>{});
    }
    float u[VPL];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (my_id >= 0) mine[my_id] = total;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < VPL; ++i) u[i] = mine[i * LPT + l];
    const float hc =
        valid_tokens > 0.0f ? dl * coef * (float)E / (float)k / valid_tokens / valid_tokens : 0.0f;
    float h[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) h[i] = i * LPT + l < E ? hc * (float)cnt[i] : 0.0f;
    float dot = 0.0f;  // softmax: sum p (u + h); sigmoid: sum p h
#pragma unroll
    for (int i = 0; i < VPL; ++i) dot += SOFTMAX ? v[i] * (u[i] + h[i]) : v[i] * h[i];
    dot = group_sum<LPT>(dot);
    float gz[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if constexpr (SOFTMAX) {
        gz[i] = v[i] * (u[i] + h[i] - dot);
      } else {
        const float si = slope[i] * inv;
        gz[i] = (renorm ? si : slope[i]) * u[i] + si * (h[i] - dot);
      }
      if (!valid) gz[i] = 0.0f;
    }
    if (out_f32) {
      const __amdgpu_buffer_rsrc_t o = gate_rows<4>(d_z, t0, T, groups, E);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        __builtin_amdgcn_raw_buffer_store_b32(
            __float_as_uint(gz[i]), o,
            (int)(i * LPT + l < E ? 4 * (row + i * LPT + l) : GATE_NONE), 0, 0);
    } else {
      const __amdgpu_buffer_rsrc_t o = gate_rows<2>(d_z, t0, T, groups, E);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        __builtin_amdgcn_raw_buffer_store_b16(
            (uint16_t)pk_bf16_rne(gz[i], 0.0f), o,
            (int)(i * LPT + l < E ? 2 * (row + i * LPT + l) : GATE_NONE), 0, 0);
    }
  }
}

namespace {

// Threads of a workgroup that leaves sums: their shares in LDS, one row of E a
// wave, stay under 64 KB.
int gate_block(int64_t E) { return E <= 512 ? 1024 : 512; }

int64_t gate_groups(int64_t T, int64_t E) {
  const int64_t per = gate_block(E) / (E <= 256 ? 16 : 64);
  const int64_t g = (T + per - 1) / per;
  return g < 1 ? 1 : g < GATE_GROUPS ? g : GATE_GROUPS;
}

size_t gate_workspace_bytes(int64_t T, int64_t E) {
  const int64_t P = gate_groups(T, E);
  return (size_t)(P * E * 8 + P * 4 + 33 * 4);  // and the loss's parts and ticket
}

struct GateArgs {
  const void *z;
  const uint8_t *mask;
  int64_t T;
  int E, k, renorm;
  float scale, coef;
  int32_t *ids;
  float *prob;
  int32_t *counts;
  float *prob_sum, *loss;
  void *ws;
  hipStream_t st;
};

template <int LPT, int VPL, bool ZF32, bool SOFTMAX>
hipError_t go_gate(const GateArgs &a) {
  const int64_t P = gate_groups(a.T, a.E);
  if (!a.loss) {
    // no sums to join: as many workgroups as there are tokens for (a grid has
    // fewer than 2^32 threads, so at most 2^20; their loop takes the rest)
    const int64_t per = 256 / LPT, g = (a.T + per - 1) / per, most = 1 << 20;
    hipLaunchKernelGGL((k_moe_gate<LPT, VPL, ZF32, SOFTMAX, false>),
                       dim3((unsigned)(g < most ? g : most)), dim3(256), 0, a.st, a.z, a.mask, a.T, a.E,
                       a.k, a.renorm, a.scale, a.ids, a.prob, (int32_t *)nullptr, (float *)nullptr,
                       (int32_t *)nullptr, (uint32_t *)nullptr);
    return hipGetLastError();
  }
  float *ps = static_cast<float *>(a.ws);
  int32_t *pc = reinterpret_cast<int32_t *>(ps + P * a.E), *pv = pc + P * a.E;
  float *pd = reinterpret_cast<float *>(pv + P);
  uint32_t *ticket = reinterpret_cast<uint32_t *>(pd + 32);
  const int block = gate_block(a.E), waves = block / 64;
  const size_t lds = (size_t)(a.E * (1 + waves) + waves) * 4;
  hipLaunchKernelGGL((k_moe_gate<LPT, VPL, ZF32, SOFTMAX, true>), dim3((unsigned)P), dim3(block),
                     lds, a.st, a.z, a.mask, a.T, a.E, a.k, a.renorm, a.scale, a.ids, a.prob, pc, ps,
                     pv, ticket);
  hipLaunchKernelGGL(k_moe_balance, dim3((a.E + 31) / 32), dim3(1024), 0, a.st, pc, ps, pv, (int)P,
                     a.E, a.k, a.coef, pd, ticket, a.counts, a.prob_sum, a.loss);
  return hipGetLastError();
}

struct GateBackArgs {
  const void *z;
  const uint8_t *mask;
  int64_t T;
  int E, k, renorm;
  float scale, coef;
  const int32_t *ids;
  const float *d_prob;
  const int32_t *counts;
  const float *d_loss;
  void *d_z;
  int out_f32;
  hipStream_t st;
};

template <int LPT, int VPL, bool ZF32, bool SOFTMAX>
hipError_t go_gate_back(const GateBackArgs &a) {
  const int64_t per = 256 / LPT, g = (a.T + per - 1) / per;
  hipLaunchKernelGGL((k_moe_gate_backward<LPT, VPL, ZF32, SOFTMAX>),
                     dim3((unsigned)(g < 8192 ? g : 8192)), dim3(256), 0, a.st, a.z, a.mask, a.T,
                     a.E, a.k, a.renorm, a.scale, a.coef, a.ids, a.d_prob, a.counts, a.d_loss,
                     a.d_z, a.out_f32);
  return hipGetLastError();
}

// Sixteen lanes a token up to 256 experts (their reductions take four lane
// steps instead of six, for four tokens at once), a wave a token beyond.
#define PQM_GATE_PICK2(FN, Z, S, A)                \
  (A.E <= 64    ? FN<16, 4, Z, S>(A)               \
   : A.E <= 128 ? FN<16, 8, Z, S>(A)               \
   : A.E <= 256 ? FN<16, 16, Z, S>(A)              \
   : A.E <= 512 ? FN<64, 8, Z, S>(A)               \
                : FN<64, 16, Z, S>(A))
#define PQM_GATE_PICK(FN, F32, SM, A)                                                   \
  ((F32) ? ((SM) ? PQM_GATE_PICK2(FN, true, true, A) : PQM_GATE_PICK2(FN, true, false, A)) \
         : ((SM) ? PQM_GATE_PICK2(FN, false, true, A) : PQM_GATE_PICK2(FN, false, false, A)))

bool al(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
pqm_status st_of(hipError_t e) { return e == hipSuccess ? PQM_OK : PQM_ERR_HIP; }

// What the forward and the backward call check alike.
pqm_status gate_shape(pqm_dtype dtype, pqm_score score, int64_t T, int64_t E, int64_t k,
                      int renorm) {
  if (dtype != PQM_OUT_BF16 && dtype != PQM_OUT_FP32) return PQM_ERR_ENUM;
  if (score != PQM_SCORE_SOFTMAX && score != PQM_SCORE_SIGMOID) return PQM_ERR_ENUM;
  if (renorm != 0 && renorm != 1) return PQM_ERR_ENUM;
  if (T < 0 || E < 1 || E > GATE_MAX_EXPERTS || k < 1 || k > GATE_MAX_K || k > E)
    return PQM_ERR_SHAPE;
  if (T > GATE_MAX_VALUES / (k + 1)) return PQM_ERR_SHAPE;  // the product may leave 64 bits
  return PQM_OK;
}

}  // namespace
}  // namespace pqm

extern "C" {

size_t pqm_moe_gate_workspace(int64_t tokens, int64_t num_experts) {
  if (tokens < 0 || tokens > pqm::GATE_MAX_VALUES || num_experts < 1 ||
      num_experts > pqm::GATE_MAX_EXPERTS)
    return 0;
  return pqm::gate_workspace_bytes(tokens, num_experts);
}

pqm_status pqm_moe_gate(const void *logits, pqm_dtype logits_dtype, const uint8_t *mask,
                        int64_t tokens, int64_t num_experts, int64_t k, pqm_score score,
                        int renormalize, float scale, int32_t *topk_ids, float *prob,
                        float loss_coef, int32_t *counts, float *prob_sum, float *loss,
                        void *workspace, size_t workspace_bytes, hipStream_t stream) {
  using namespace pqm;
  const pqm_status bad = gate_shape(logits_dtype, score, tokens, num_experts, k, renormalize);
  if (bad != PQM_OK) return bad;
  if (tokens > 0 && (!logits || !topk_ids || !prob)) return PQM_ERR_NULL;
  const bool sums = counts || prob_sum || loss;
  if (sums && (!counts || !prob_sum || !loss || !workspace)) return PQM_ERR_NULL;
  if (sums && workspace_bytes < gate_workspace_bytes(tokens, num_experts)) return PQM_ERR_WORKSPACE;
  if (!al(logits, logits_dtype == PQM_OUT_FP32 ? 4 : 2) || !al(topk_ids, 4) || !al(prob, 4) ||
      !al(counts, 4) || !al(prob_sum, 4) || !al(loss, 4) || (sums && !al(workspace, 4)))
    return PQM_ERR_ALIGN;
  if (tokens == 0 && !sums) return PQM_OK;
  const GateArgs a = {logits, mask, tokens, (int)num_experts, (int)k, renormalize, scale,
                      loss_coef, topk_ids, prob, counts, prob_sum, loss, workspace, stream};
  return st_of(PQM_GATE_PICK(go_gate, logits_dtype == PQM_OUT_FP32, score == PQM_SCORE_SOFTMAX, a));
}

pqm_status pqm_moe_gate_backward(const void *logits, pqm_dtype logits_dtype, const uint8_t *mask,
                                 int64_t tokens, int64_t num_experts, int64_t k, pqm_score score,
                                 int renormalize, float scale, const int32_t *topk_ids,
                                 const float *d_prob, float loss_coef, const int32_t *counts,
                                 const float *d_loss, void *d_logits, pqm_dtype d_logits_dtype,
                                 hipStream_t stream) {
  using namespace pqm;
  const pqm_status bad = gate_shape(logits_dtype, score, tokens, num_experts, k, renormalize);
  if (bad != PQM_OK) return bad;
  if (d_logits_dtype != PQM_OUT_BF16 && d_logits_dtype != PQM_OUT_FP32) return PQM_ERR_ENUM;
  if (tokens == 0) return PQM_OK;
  if (!logits || !topk_ids || !d_logits || (!d_prob && !counts)) return PQM_ERR_NULL;
  if ((counts == nullptr) != (d_loss == nullptr)) return PQM_ERR_NULL;
  if (!al(logits, logits_dtype == PQM_OUT_FP32 ? 4 : 2) ||
      !al(d_logits, d_logits_dtype == PQM_OUT_FP32 ? 4 : 2) || !al(topk_ids, 4) || !al(d_prob, 4) || !al(counts, 4) ||
      !al(d_loss, 4))
    return PQM_ERR_ALIGN;
  const GateBackArgs a = {logits, mask, tokens, (int)num_experts, (int)k, renormalize, scale,
                          loss_coef, topk_ids, d_prob, counts, d_loss, d_logits,
                          d_logits_dtype == PQM_OUT_FP32, stream};
  return st_of(
      PQM_GATE_PICK(go_gate_back, logits_dtype == PQM_OUT_FP32, score == PQM_SCORE_SOFTMAX, a));
}

}  // extern "C"
