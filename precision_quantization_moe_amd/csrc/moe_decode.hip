// moe_decode.hip -- a whole expert layer for a few tokens (decode), from the
// residual stream on, with NVFP4 expert weights:
//
//   h = bf16(x + residual),  y = bf16(h rstd w),  z = y W_gate^T,
//   the k experts of the largest z and their probabilities p (as pqm_moe_gate),
//   d[t, j] = bf16(silu(g) u p[t, j]),  (g, u) = y[t] W1_e^T,  e = ids[t, j],
//   out[t] = bf16(sum over j of d[t, j] W2_e^T),
// a shared expert as one more j with p = 1.  What counts is that each weight is
// read once and that few steps wait for one another: a layer of one token takes
// 21 MB, 4 us of the memory's time.
//
// An expert meets a token at most once, so its rows are a 64-bit set of tokens.
#include "gate_device.hpp"
#include "gemv_device.hpp"
#include "norm_device.hpp"
#include "pqm_device.hpp"
#include "pqm_internal.hpp"
#include "pqmoe.h"

namespace pqm {

namespace {

constexpr int DC_TOKENS = 64, DC_EXPERTS = 1024, DC_K = 16, DC_WIDTH = 16384;
// Tokens of a workgroup of the router, whose rows are 8 KB of LDS each at NC 1.
constexpr int dr_tokens(int nc) { return 4 / nc; }

struct DcArgs {
  const uint16_t *x, *res;
  const void *norm_w;
  float eps;
  const uint16_t *gate_w;
  int T, H, I, E, k, c;  // c: rows of d a token, k and the shared expert's
  int softmax, renorm;
  float scale;
  const uint8_t *w1, *s1;
  const float *g1;
  const uint8_t *w2, *s2;
  const float *g2;
  uint16_t *h, *y;
  int32_t *ids;
  float *prob;
  uint16_t *d, *out;
  float *logits;    // [T][E]
  float *partial;   // [S][T][H]
  uint32_t *count;  // [H / 16]
  int ks, S;        // waves that share a contraction; parts of the experts
};

__device__ __forceinline__ int dc_uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

}  // namespace

// Norm and router: 16 experts by a few tokens a workgroup, each of which
// normalises its tokens itself (the first column of workgroups writes h and y).
// A wave takes every eighth 64-wide block of the contraction, its first four
// asked for before the norm.  The order of two logits decides which experts a
// token meets, so the matrix instructions' sums of 32 products are added up in
// binary64: a logit is off by little more than its last rounding.
template <int NC, bool WF32>
__global__ __launch_bounds__(512) void k_decode_router(DcArgs a) {
  constexpr int DR_TOKENS = dr_tokens(NC);
  extern __shared__ __align__(16) uint8_t lds[];  // y: rows of H values and 16 bytes
  __shared__ double red[8][DR_TOKENS];
  __shared__ double sums[8][DR_TOKENS][16];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, ln = lane & 15;
  const int wave = dc_uniform(tid >> 6);
  const int t0 = blockIdx.y * DR_TOKENS, n = min(DR_TOKENS, a.T - t0), e0 = blockIdx.x * 16;
  const int H = a.H, pitch = 2 * H + 16, blocks = (H + 63) / 64;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = tid; i < H / 16; i += 512) a.count[i] = 0;
  const __amdgpu_buffer_rsrc_t wb =
      gv_buffer(a.gate_w + (int64_t)e0 * H, (int64_t)min(16, a.E - e0) * H * 2);
  const auto load = [&](gv_u4 (&w)[8], int i0) {  // four blocks of this wave
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int kk = 64 * (wave + 8 * (i0 + i / 2)) + 32 * (i & 1) + 8 * g;
      w[i] = __builtin_amdgcn_raw_buffer_load_b128(
          wb, (int)(kk < H ? (uint32_t)(ln * H + kk) * 2 : GV_NONE), 0, 0);
    }
  };
  gv_u4 w[8];
  load(w, 0);

  uint32_t v[DR_TOKENS][NC][4];
  double sq[DR_TOKENS] = {};
#pragma unroll
  for (int t = 0; t < DR_TOKENS; ++t)
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * 512 + tid) * 8;
      uint4 u = make_uint4(0, 0, 0, 0), r = u;
      if (t < n && c < H) {
        u = *reinterpret_cast<const uint4 *>(a.x + (int64_t)(t0 + t) * H + c);
        if (a.res) r = *reinterpret_cast<const uint4 *>(a.res + (int64_t)(t0 + t) * H + c);
      }
      const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[t][i][j] = a.res ? pk_bf16_rne(bf16_lo_f32(uu[j]) + bf16_lo_f32(rr[j]),
                                         bf16_hi_f32(uu[j]) + bf16_hi_f32(rr[j]))
                           : uu[j];
    }
#pragma unroll
  for (int t = 0; t < DR_TOKENS; ++t) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const double lo = bf16_lo_f32(v[t][i][j]), hi = bf16_hi_f32(v[t][i][j]);
        sq[t] = __builtin_fma(lo, lo, sq[t]);
        sq[t] = __builtin_fma(hi, hi, sq[t]);
      }
    sq[t] = wave_sum(sq[t]);
    if (lane == 0) red[wave][t] = sq[t];
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < DR_TOKENS; ++t) {
    if (t >= n) break;
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) total += red[i][t];
    const double root = inverse_root(total / (double)H + (double)a.eps);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * 512 + tid) * 8;
      if (c >= H) continue;
      float wf[8];
      load_w8<WF32>(a.norm_w, c, wf);
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)  // binary64 throughout: y is the nearest bf16 value
        o[j] = pk_bf16_rne(
            before_bf16((double)bf16_lo_f32(v[t][i][j]) * (double)wf[2 * j] * root),
            before_bf16((double)bf16_hi_f32(v[t][i][j]) * (double)wf[2 * j + 1] * root));
      *reinterpret_cast<uint4 *>(lds + t * pitch + 2 * c) = make_uint4(o[0], o[1], o[2], o[3]);
      if (blockIdx.x == 0) {
        const int64_t at = (int64_t)(t0 + t) * H + c;
        *reinterpret_cast<uint4 *>(a.h + at) =
            make_uint4(v[t][i][0], v[t][i][1], v[t][i][2], v[t][i][3]);
        *reinterpret_cast<uint4 *>(a.y + at) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  __syncthreads();

  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  for (int i0 = 0; wave + 8 * i0 < blocks; i0 += 4) {
    if (i0) load(w, i0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int kk = 64 * (wave + 8 * (i0 + i / 2)) + 32 * (i & 1) + 8 * g;
      gv_u4 b = {0, 0, 0, 0};
      if (ln < n && kk < H) b = *reinterpret_cast<const gv_u4 *>(lds + ln * pitch + 2 * kk);
      gv_f4 s = {0, 0, 0, 0};
      s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(gv_bf8, w[i]),
                                                  __builtin_bit_cast(gv_bf8, b), s, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] += (double)s[j];
    }
  }
  if (ln < DR_TOKENS) {
#pragma unroll
    for (int j = 0; j < 4; ++j) sums[wave][ln][4 * g + j] = acc[j];
  }
  __syncthreads();
  const int t = tid >> 4, e = e0 + (tid & 15);
  if (t < n && e < a.E) {
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) z += sums[i][t][tid & 15];
    a.logits[(t0 + t) * a.E + e] = (float)z;
  }
}

namespace {

// The gate of token t by one wave, expert 64 i + lane in register i: the choice,
// the scores and the renormalisation of pqm_moe_gate.
template <int VPL>
__device__ __forceinline__ void dc_gate(const DcArgs &a, const float (&z)[VPL], int t, int32_t *ids,
                                        float *prob) {
  const int l = threadIdx.x & 63;
  float v[VPL];
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const bool in = 64 * i + l < a.E;
    v[i] = in ? z[i] : -__builtin_inff();
    key[i] = in ? logit_key(v[i]) : 0u;
  }
  int my_id = 0;
  uint32_t my_key = 0, first = 0;
  for (int j = 0; j < a.k; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = max(m, key[i]);
    m = group_max<64>(m);
    uint32_t mine_at = UINT32_MAX;
    bool hit[VPL], seen = false;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const bool eq = key[i] == m;
      hit[i] = eq && !seen;
      seen = seen || eq;
      mine_at = hit[i] ? (uint32_t)(64 * i + l) : mine_at;
    }
    const uint32_t at = group_min<64>(mine_at);
    const bool won = at == mine_at;
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = hit[i] && won ? 0u : key[i];
    if (j == 0) first = m;
    if (l == j) {
      my_id = (int)at;
      my_key = m;
    }
  }
  float top = key_logit(first);
  const float my_z = l < a.k ? key_logit(my_key) : -__builtin_inff();
  if (top == -__builtin_inff()) top = 0.0f;
  float w = l < a.k ? (a.softmax ? exp_f32(my_z - top) : sigmoid(my_z)) : 0.0f;
  if (a.renorm) {
    const float total = group_sum<64>(w);
    w = total == 0.0f ? 0.0f : w / total;
  } else if (a.softmax) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) sum += 64 * i + l < a.E ? exp_f32(v[i] - top) : 0.0f;
    sum = group_sum<64>(sum);
    w *= sum == 0.0f ? 0.0f : 1.0f / sum;
  }
  if (!a.softmax && top != top) w = top;
  if (l < a.k) {
    ids[t * a.k + l] = my_id;
    prob[t * a.k + l] = w * a.scale;
  }
}

// Every token's gate, one wave a token, the next one's logits ahead.
template <int VPL>
__device__ __forceinline__ void dc_gates(const DcArgs &a, int32_t *ids, float *prob) {
  const int l = threadIdx.x & 63, wave = dc_uniform(threadIdx.x >> 6);
  const __amdgpu_buffer_rsrc_t zb = gv_buffer(a.logits, (int64_t)a.T * a.E * 4);
  const auto load = [&](float (&z)[VPL], int t) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      z[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
          zb, (int)(64 * i + l < a.E ? (uint32_t)(t * a.E + 64 * i + l) * 4 : GV_NONE), 0, 0));
  };
  float z[VPL];
  load(z, wave);  // past the last token: zeros
  for (int t = wave; t < a.T; t += 8) {
    float next[VPL];
    load(next, t + 8);
    dc_gate<VPL>(a, z, t, ids, prob);
#pragma unroll
    for (int i = 0; i < VPL; ++i) z[i] = next[i];
  }
}

// Which experts are met, and by which tokens.
struct DcSets {
  uint64_t rows[DC_EXPERTS + 1];
  uint16_t met[DC_EXPERTS + 1];
  int32_t ids[DC_TOKENS * DC_K];
  int count[8];
};

// Fills s.rows and s.met from s.ids; the number of experts met.  All threads call
// it, after a barrier behind the ids.
__device__ __forceinline__ int dc_sets(const DcArgs &a, DcSets &s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int groups = a.E + (a.c - a.k);
  for (int e = tid; e < groups; e += 512)
    s.rows[e] = e < a.E ? 0 : a.T == 64 ? ~0ull : (1ull << a.T) - 1;
  __syncthreads();
  for (int i = tid; i < a.T * a.k; i += 512)
    atomicOr(reinterpret_cast<unsigned long long *>(&s.rows[s.ids[i]]), 1ull << (i / a.k));
  __syncthreads();
  int n = 0;
  for (int e0 = 0; e0 < groups; e0 += 512) {
    const int e = e0 + tid;
    const uint64_t b = __ballot(e < groups && s.rows[e] != 0);
    if (lane == 0) s.count[wave] = __popcll(b);
    __syncthreads();
    int at = n + __popcll(b & ((1ull << lane) - 1));
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w < wave) at += s.count[w];
      n += s.count[w];
    }
    if (b >> lane & 1) s.met[at] = (uint16_t)e;
    __syncthreads();
  }
  return dc_uniform(n);
}

// Lane r gets the token of row r of a set (its r-th member; behind the members
// come the others).
__device__ __forceinline__ int dc_members(uint64_t rows) {
  const int lane = threadIdx.x & 63, c = __popcll(rows);
  const int before = __popcll(rows & ((1ull << lane) - 1));
  const int at = rows >> lane & 1 ? before : c + lane - before;
  return __builtin_amdgcn_ds_permute(4 * at, lane);
}

__device__ __forceinline__ uint64_t dc_uniform64(uint64_t v) {
  return (uint64_t)(uint32_t)dc_uniform((int)(v >> 32)) << 32 | (uint32_t)dc_uniform((int)v);
}

// Which of its token's rows an expert's row is.
__device__ __forceinline__ int dc_slot(const DcArgs &a, const DcSets &s, int t, int e) {
  int j = a.k;  // the shared expert's
  for (int i = 0; i < a.k; ++i) j = s.ids[t * a.k + i] == e ? i : j;
  return j;
}

// A 16-row weight tile's part of a 256-wide chunk: eight rows a load, eight lanes
// each; of the scales a row's 16 bytes in four lanes.
struct DcChunk {
  gv_u4 q[2];
  uint32_t s;
};

template <bool WORDS>
__device__ __forceinline__ void dc_load(DcChunk &b, __amdgpu_buffer_rsrc_t wq,
                                        __amdgpu_buffer_rsrc_t ws, int K, int ch, bool in) {
  const int lane = threadIdx.x & 63;
  const uint32_t oq = in ? ch * 128u : GV_NONE, os = in ? ch * 16u : GV_NONE;
  const int vq = (int)((lane >> 3) * (uint32_t)(K / 2) + 16 * (lane & 7) + oq);
  const int vs = (int)((lane >> 2) * (uint32_t)(K / 16) + 4 * (lane & 3) + os);
  b.q[0] = __builtin_amdgcn_raw_buffer_load_b128(wq, vq, 0, 0);
  b.q[1] = __builtin_amdgcn_raw_buffer_load_b128(wq, vq + 8 * (K / 2), 0, 0);
  if constexpr (WORDS)
    b.s = __builtin_amdgcn_raw_buffer_load_b32(ws, vs, 0, 0);
  else  // rows of scales start at any even byte
    b.s = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(ws, vs, 0, 0) |
          (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(ws, vs + 2, 0, 0) << 16;
}

// A chunk of N weight tiles times MT tiles of 16 rows, whose values start at xo
// (GV_NONE: no row) of xb.  Few of the rows' values are held at a time: 8 tiles'
// worth of registers.
template <int MT, int N>
__device__ __forceinline__ void dc_multiply(gv_f4 (&acc)[N][MT], const DcChunk (&b)[N],
                                            __amdgpu_buffer_rsrc_t xb, const uint32_t (&xo)[MT],
                                            const GvTurn &turn, int K, int ch) {
  constexpr int JB = 8 / MT;
  const int lane = threadIdx.x & 63, g = lane >> 4, ln = lane & 15;
  // past the row's end stand the next row's scales, maybe NaN: x is 0 there, the
  // scale has to be so too
  const int left = K - 256 * ch - 64 * g;
  gv_u4 x[JB][MT];
  const auto load_x = [&](int j0) {
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        x[j][m] = __builtin_amdgcn_raw_buffer_load_b128(
            xb,
            (int)(8 * (j0 + j) < left && xo[m] != GV_NONE
                      ? xo[m] + 2 * (256 * ch + 64 * g + 8 * (j0 + j))
                      : GV_NONE),
            0, 0);
  };
  load_x(0);
  gv_u4 q[N][2];
  float f[N][4];
#pragma unroll
  for (int t = 0; t < N; ++t) {
    turn(b[t].q, q[t]);
    int sw = __builtin_amdgcn_ds_bpermute(16 * ln + 4 * g, (int)b[t].s);
    if (left < 64) sw = left == 32 ? sw & 0xFFFF : 0;
    f[t][0] = __builtin_amdgcn_cvt_f32_fp8(sw, 0);
    f[t][1] = __builtin_amdgcn_cvt_f32_fp8(sw, 1);
    f[t][2] = __builtin_amdgcn_cvt_f32_fp8(sw, 2);
    f[t][3] = __builtin_amdgcn_cvt_f32_fp8(sw, 3);
  }
#pragma unroll
  for (int j0 = 0; j0 < 8; j0 += JB) {
    if (j0) load_x(j0);
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int t = 0; t < N; ++t) {
        const gv_bf8 w = gv_decode(q[t][(j0 + j) >> 2][(j0 + j) & 3], f[t][(j0 + j) >> 1]);
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[t][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              w, __builtin_bit_cast(gv_bf8, x[j][m]), acc[t][m], 0, 0, 0);
      }
  }
}

// One expert's 16 columns of d, its rows m0 .. m0 + 16 MT - 1: ks waves share the
// contraction.
template <int MT, bool WORDS>
__device__ __forceinline__ void dc_up(const DcArgs &a, const DcSets &s, const float *prob, int e,
                                      uint64_t rows, int m0, int tile, const GvTurn &turn,
                                      gv_f4 (*red)[2][64]) {
  const int lane = threadIdx.x & 63, g = lane >> 4, ln = lane & 15;
  const int wave = dc_uniform(threadIdx.x >> 6), kw = wave & (a.ks - 1);
  const int K = a.H, chunks = (K + 255) / 256, c = __popcll(rows);
  const bool live = 16 * tile < a.I;  // otherwise a wave past the last tile
  const int64_t r0 = (int64_t)e * 2 * a.I + (live ? 16 * tile : 0), r1 = r0 + a.I;
  const int n = live ? 16 : 0;
  const __amdgpu_buffer_rsrc_t gq = gv_buffer(a.w1 + r0 * (K / 2), (int64_t)n * (K / 2)),
                               gs = gv_buffer(a.s1 + r0 * (K / 16), (int64_t)n * (K / 16)),
                               uq = gv_buffer(a.w1 + r1 * (K / 2), (int64_t)n * (K / 2)),
                               us = gv_buffer(a.s1 + r1 * (K / 16), (int64_t)n * (K / 16)),
                               xb = gv_buffer(a.y, (int64_t)a.T * K * 2);
  const int token = dc_members(rows);
  uint32_t xo[MT];
  int tok[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    tok[m] = __builtin_amdgcn_ds_bpermute(4 * (m0 + 16 * m + ln), token);
    xo[m] = m0 + 16 * m + ln < c ? (uint32_t)tok[m] * K * 2 : GV_NONE;
  }
  gv_f4 acc[2][MT] = {};
  DcChunk b[2];
  const auto load = [&](int ch) {
    dc_load<WORDS>(b[0], gq, gs, K, ch, ch < chunks);
    dc_load<WORDS>(b[1], uq, us, K, ch, ch < chunks);
  };
  load(kw);
  for (int ch = kw; ch < chunks; ch += a.ks) {
    const DcChunk cur[2] = {b[0], b[1]};
    load(ch + a.ks);
    dc_multiply<MT, 2>(acc, cur, xb, xo, turn, K, ch);
  }
  const float outer = a.g1[e];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    gv_f4 vg = acc[0][m], vu = acc[1][m];
    if (a.ks > 1) {
      red[wave][0][lane] = vg;
      red[wave][1][lane] = vu;
      __syncthreads();
      if (kw == 0) {
        for (int i = 1; i < a.ks; ++i) {
          vg += red[wave + i][0][lane];
          vu += red[wave + i][1][lane];
        }
      }
      __syncthreads();
    }
    if (kw == 0 && live && xo[m] != GV_NONE) {
      const int t = tok[m], j = dc_slot(a, s, t, e);
      const float p = j < a.k ? prob[t * a.k + j] : 1.0f;
      float o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = swiglu_f32(vg[i] * outer, vu[i] * outer, p);
      *reinterpret_cast<uint2 *>(a.d + (int64_t)(t * a.c + j) * a.I + 16 * tile + 4 * g) =
          make_uint2(pk_bf16_rne(o[0], o[1]), pk_bf16_rne(o[2], o[3]));
    }
  }
}

}  // namespace

// Gate and gate_up.
template <int MAXMT, int VPL, bool WORDS>
__global__ __launch_bounds__(512, 4) void k_decode_up(DcArgs a) {
  __shared__ DcSets s;
  __shared__ float prob[DC_TOKENS * DC_K];
  __shared__ __align__(16) uint8_t turns[8][2048];
  __shared__ gv_f4 red[8][2][64];
  dc_gates<VPL>(a, s.ids, prob);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.T * a.k; i += 512) {
      a.ids[i] = s.ids[i];
      a.prob[i] = prob[i];
    }
  const int D = dc_sets(a, s);
  const int wave = dc_uniform(threadIdx.x >> 6), per = 8 / a.ks;
  const int tg = (a.I / 16 + per - 1) / per;
  const GvTurn turn(turns[wave], threadIdx.x & 63);
  for (int item = blockIdx.x; item < D * tg; item += gridDim.x) {
    const int i = item / tg, tile = (item - i * tg) * per + wave / a.ks;
    const int e = dc_uniform(s.met[i]);
    const uint64_t rows = dc_uniform64(s.rows[e]);
    const int c = __popcll(rows);
    // more than 32 rows of an expert read its weights again
    for (int m0 = 0; m0 < c; m0 += 32) {
      if (MAXMT == 1 || c - m0 <= 16) dc_up<1, WORDS>(a, s, prob, e, rows, m0, tile, turn, red);
      else dc_up<MAXMT, WORDS>(a, s, prob, e, rows, m0, tile, turn, red);
    }
  }
}

namespace {

// One chunk of one expert's part of 16 output columns, its rows m0 .., added to the
// wave's sums.
template <int MT>
__device__ __forceinline__ void dc_down(const DcArgs &a, const DcSets &s, int e, uint64_t rows,
                                        int m0, const DcChunk &b, float outer, const GvTurn &turn, int ch,
                                        float *sums) {
  const int lane = threadIdx.x & 63, g = lane >> 4, ln = lane & 15;
  const int K = a.I, c = __popcll(rows);
  const __amdgpu_buffer_rsrc_t xb = gv_buffer(a.d, (int64_t)a.T * a.c * K * 2);
  const int token = dc_members(rows);
  uint32_t xo[MT];
  int tok[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    tok[m] = __builtin_amdgcn_ds_bpermute(4 * (m0 + 16 * m + ln), token);
    xo[m] = GV_NONE;
    if (m0 + 16 * m + ln < c) xo[m] = (uint32_t)(tok[m] * a.c + dc_slot(a, s, tok[m], e)) * K * 2;
  }
  gv_f4 acc[1][MT] = {};
  const DcChunk one[1] = {b};
  dc_multiply<MT, 1>(acc, one, xb, xo, turn, K, ch);
#pragma unroll
  for (int m = 0; m < MT; ++m)
    if (xo[m] != GV_NONE) {
      gv_f4 *p = reinterpret_cast<gv_f4 *>(sums + tok[m] * 16 + 4 * g);
      *p += acc[0][m] * outer;
    }
}

}  // namespace

// Down projection and sum: a workgroup takes 16 output columns and a part of the
// experts met; its waves take their chunks in turn, each with sums of its own.
// The workgroup that finishes a column's last part adds the parts in their order.
template <int MAXMT, bool WORDS>
__global__ __launch_bounds__(512, 4) void k_decode_down(DcArgs a) {
  extern __shared__ __align__(16) float sums[];  // [8][T][16]
  __shared__ DcSets s;
  __shared__ __align__(16) uint8_t turns[8][2048];
  __shared__ int last;
  const int tid = threadIdx.x, wave = dc_uniform(tid >> 6);
  for (int i = tid; i < a.T * a.k; i += 512) s.ids[i] = a.ids[i];
  __syncthreads();
  const int D = dc_sets(a, s);
  const int K = a.I, chunks = (K + 255) / 256, NT = a.H / 16;
  const GvTurn turn(turns[wave], tid & 63);
  float *mine = sums + wave * a.T * 16;
  for (int item = blockIdx.x; item < NT * a.S; item += gridDim.x) {
    const int part = item / NT, tile = item - part * NT;
    const int i0 = D * part / a.S, i1 = D * (part + 1) / a.S, units = (i1 - i0) * chunks;
    for (int i = tid & 63; i < a.T * 4; i += 64)
      reinterpret_cast<gv_f4 *>(mine)[i] = gv_f4{0, 0, 0, 0};
    const auto load = [&](DcChunk &b, float &outer, int u) {
      const bool in = u < units;
      const int e = in ? dc_uniform(s.met[i0 + u / chunks]) : 0;
      const int64_t r0 = (int64_t)e * a.H + 16 * tile;
      dc_load<WORDS>(b, gv_buffer(a.w2 + r0 * (K / 2), 8 * (int64_t)K),
                     gv_buffer(a.s2 + r0 * (K / 16), (int64_t)K), K, u % chunks, in);
      outer = a.g2[e];
    };
    DcChunk b;
    float outer;
    load(b, outer, wave);
    for (int u = wave; u < units; u += 8) {
      const DcChunk cur = b;
      const float o = outer;
      load(b, outer, u + 8);
      const int e = dc_uniform(s.met[i0 + u / chunks]);
      const uint64_t rows = dc_uniform64(s.rows[e]);
      const int c = __popcll(rows);
      for (int m0 = 0; m0 < c; m0 += 32) {
        if (MAXMT == 1 || c - m0 <= 16) dc_down<1>(a, s, e, rows, m0, cur, o, turn, u % chunks, mine);
        else dc_down<MAXMT>(a, s, e, rows, m0, cur, o, turn, u % chunks, mine);
      }
    }
    __syncthreads();
    for (int i = tid; i < a.T * 8; i += 512) {
      const int t = i >> 3, c = 2 * (i & 7);
      float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        v0 += sums[(w * a.T + t) * 16 + c];
        v1 += sums[(w * a.T + t) * 16 + c + 1];
      }
      if (a.S == 1) {
        *reinterpret_cast<uint32_t *>(a.out + (int64_t)t * a.H + 16 * tile + c) =
            pk_bf16_rne(v0, v1);
      } else {
        float *p = a.partial + ((int64_t)part * a.T + t) * a.H + 16 * tile + c;
        __hip_atomic_store(p, v0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(p + 1, v1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    if (a.S > 1) {
      __threadfence();
      __syncthreads();
      if (tid == 0)
        last = __hip_atomic_fetch_add(&a.count[tile], 1u, __ATOMIC_ACQ_REL,
                                      __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)a.S - 1;
      __syncthreads();
      if (last) {
        for (int i = tid; i < a.T * 8; i += 512) {
          const int t = i >> 3, c = 2 * (i & 7);
          float v0 = 0.0f, v1 = 0.0f;
          for (int q = 0; q < a.S; ++q) {
            const float *p = a.partial + ((int64_t)q * a.T + t) * a.H + 16 * tile + c;
            v0 += __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            v1 += __hip_atomic_load(p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          }
          *reinterpret_cast<uint32_t *>(a.out + (int64_t)t * a.H + 16 * tile + c) =
              pk_bf16_rne(v0, v1);
        }
      }
    }
    __syncthreads();
  }
}

namespace {

struct DcPlan {
  int ks, S;
};

// By size alone: waves share a contraction until there are 4096 of them, and the
// experts are parted until there are 1024 workgroups of the down projection, each
// wave with a chunk at least.
DcPlan dc_plan(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int shared) {
  const int64_t met = (T * k < E ? T * k : E) + shared;
  DcPlan p = {1, 1};
  while (p.ks < 8 && met * (I / 16) * p.ks < 4096 && 2 * p.ks <= (H + 255) / 256) p.ks *= 2;
  int64_t s = (1024 + H / 16 - 1) / (H / 16);
  const int64_t most = met * ((I + 255) / 256) / 8;
  if (s > most) s = most;
  if (s > met) s = met;
  p.S = (int)(s < 1 ? 1 : s);
  return p;
}

bool dc_sizes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k) {
  return T >= 0 && T <= DC_TOKENS && H >= 32 && H <= DC_WIDTH && H % 32 == 0 && I >= 32 &&
         I <= DC_WIDTH && I % 32 == 0 && E >= 1 && E <= DC_EXPERTS && k >= 1 && k <= DC_K && k <= E;
}

struct DcLayout {
  size_t partial, count, bytes;
};

DcLayout dc_layout(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int shared) {
  const DcPlan p = dc_plan(T, H, I, E, k, shared);
  DcLayout l;
  l.partial = (size_t)(T * E * 4 + 15) / 16 * 16;
  l.count = l.partial + (p.S > 1 ? (size_t)p.S * T * H * 4 : 0);
  l.bytes = l.count + (size_t)H / 16 * 4;
  return l;
}

bool al(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

template <int NC>
void dc_router(const DcArgs &a, bool wf32, hipStream_t st) {
  constexpr int N = dr_tokens(NC);
  const dim3 grid((unsigned)((a.E + 15) / 16), (unsigned)((a.T + N - 1) / N));
  const size_t lds = (size_t)N * (2 * a.H + 16);
  if (wf32) hipLaunchKernelGGL((k_decode_router<NC, true>), grid, dim3(512), lds, st, a);
  else hipLaunchKernelGGL((k_decode_router<NC, false>), grid, dim3(512), lds, st, a);
}

template <int MAXMT, int VPL>
void dc_launch_up(const DcArgs &a, unsigned grid, hipStream_t st) {
  if (a.H % 64 == 0)
    hipLaunchKernelGGL((k_decode_up<MAXMT, VPL, true>), dim3(grid), dim3(512), 0, st, a);
  else
    hipLaunchKernelGGL((k_decode_up<MAXMT, VPL, false>), dim3(grid), dim3(512), 0, st, a);
}

template <int MAXMT>
hipError_t dc_experts(const DcArgs &a, hipStream_t st) {
  const int64_t met = (a.T * a.k < a.E ? a.T * a.k : a.E) + (a.c - a.k);
  const int64_t per = 8 / a.ks, items = met * ((a.I / 16 + per - 1) / per);
  const unsigned grid = (unsigned)(items < 512 ? items : 512);
  if (a.E <= 64) dc_launch_up<MAXMT, 1>(a, grid, st);
  else if (a.E <= 128) dc_launch_up<MAXMT, 2>(a, grid, st);
  else if (a.E <= 256) dc_launch_up<MAXMT, 4>(a, grid, st);
  else dc_launch_up<MAXMT, 16>(a, grid, st);
  const hipError_t r = hipGetLastError();
  if (r != hipSuccess) return r;
  const int64_t down = (int64_t)(a.H / 16) * a.S;
  const dim3 dgrid((unsigned)(down < 512 ? down : 512));
  const size_t lds = (size_t)8 * a.T * 16 * 4;
  if (a.I % 64 == 0) hipLaunchKernelGGL((k_decode_down<MAXMT, true>), dgrid, dim3(512), lds, st, a);
  else hipLaunchKernelGGL((k_decode_down<MAXMT, false>), dgrid, dim3(512), lds, st, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace pqm

extern "C" {

size_t pqm_moe_decode_nvfp4_workspace(int64_t tokens, int64_t hidden, int64_t inter,
                                      int64_t num_experts, int64_t k, int shared_expert) {
  using namespace pqm;
  if (!dc_sizes(tokens, hidden, inter, num_experts, k) || tokens == 0) return 0;
  return dc_layout(tokens, hidden, inter, num_experts, k, shared_expert ? 1 : 0).bytes;
}

pqm_status pqm_moe_decode_nvfp4(const uint16_t *x, const uint16_t *residual, const void *norm_w,
                                pqm_dtype norm_dtype, float eps, const uint16_t *gate_w,
                                int64_t tokens, int64_t hidden, int64_t inter, int64_t num_experts,
                                int64_t k, int shared_expert, pqm_score score, int renormalize,
                                float scale, const uint8_t *w1_q, const uint8_t *w1_scale,
                                const float *w1_outer, const uint8_t *w2_q,
                                const uint8_t *w2_scale, const float *w2_outer, uint16_t *h,
                                uint16_t *y, int32_t *topk_ids, float *prob, uint16_t *d,
                                uint16_t *out, void *workspace, size_t workspace_bytes,
                                hipStream_t stream) {
  using namespace pqm;
  if ((norm_dtype != PQM_OUT_BF16 && norm_dtype != PQM_OUT_FP32) ||
      (score != PQM_SCORE_SOFTMAX && score != PQM_SCORE_SIGMOID) || renormalize < 0 ||
      renormalize > 1 || shared_expert < 0 || shared_expert > 1)
    return PQM_ERR_ENUM;
  if (!dc_sizes(tokens, hidden, inter, num_experts, k)) return PQM_ERR_SHAPE;
  if (!(eps >= 0x1p-100f && eps <= 3.4e38f)) return PQM_ERR_SHAPE;
  if (tokens == 0) return PQM_OK;
  if (!x || !norm_w || !gate_w || !w1_q || !w1_scale || !w1_outer || !w2_q || !w2_scale ||
      !w2_outer || !h || !y || !topk_ids || !prob || !d || !out || !workspace)
    return PQM_ERR_NULL;
  if (!al(x, 16) || !al(residual, 16) || !al(norm_w, 16) || !al(gate_w, 16) || !al(w1_q, 16) ||
      !al(w2_q, 16) || !al(w1_scale, 4) || !al(w2_scale, 4) || !al(w1_outer, 4) ||
      !al(w2_outer, 4) || !al(h, 16) || !al(y, 16) || !al(topk_ids, 4) || !al(prob, 4) ||
      !al(d, 16) || !al(out, 16) || !al(workspace, 16))
    return PQM_ERR_ALIGN;
  const DcLayout l = dc_layout(tokens, hidden, inter, num_experts, k, shared_expert);
  if (workspace_bytes < l.bytes) return PQM_ERR_WORKSPACE;
  const DcPlan p = dc_plan(tokens, hidden, inter, num_experts, k, shared_expert);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const DcArgs a = {x, residual, norm_w, eps, gate_w, (int)tokens, (int)hidden, (int)inter,
                    (int)num_experts, (int)k, (int)k + shared_expert, score == PQM_SCORE_SOFTMAX,
                    renormalize, scale, w1_q, w1_scale, w1_outer, w2_q, w2_scale, w2_outer, h, y,
                    topk_ids, prob, d, out, reinterpret_cast<float *>(ws),
                    reinterpret_cast<float *>(ws + l.partial),
                    reinterpret_cast<uint32_t *>(ws + l.count), p.ks, p.S};
  const bool wf32 = norm_dtype == PQM_OUT_FP32;
  if (hidden <= 4096) dc_router<1>(a, wf32, stream);
  else if (hidden <= 8192) dc_router<2>(a, wf32, stream);
  else dc_router<4>(a, wf32, stream);
  if (hipGetLastError() != hipSuccess) return PQM_ERR_HIP;
  const hipError_t r = tokens <= 16 ? dc_experts<1>(a, stream) : dc_experts<2>(a, stream);
  return r == hipSuccess ? PQM_OK : PQM_ERR_HIP;
}

}  // extern "C"
