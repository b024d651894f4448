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
// An expert meets a token at most once, so the rows of one are a set of tokens.
#include "gate_device.hpp"
#include "gemv_device.hpp"
#include "norm_device.hpp"
#include "pqm_device.hpp"
#include "pqm_internal.hpp"
#include "pqmoe.h"

namespace pqm {

namespace {

constexpr int DC_TOKENS = 64, DC_EXPERTS = 1024, DC_K = 16, DC_WIDTH = 16384;
constexpr int DC_FEW = 8;        // tokens of the one-kernel form
constexpr int DC_WAVES = 16;     // of a workgroup of that form, one workgroup a CU
constexpr int DC_GRID = 256;
static_assert(DC_FEW <= 16, "an expert's rows are one tile");
constexpr int DC_CLASSES = 8;    // tickets and signals, a cache line each

// Tokens of a workgroup of the router, whose rows are 8 KB of LDS each at NC 1.
constexpr int dr_tokens(int nc) { return 4 / nc; }

struct DcSync {
  struct {
    uint32_t ticket, pad0[63], done, pad1[63];
  } of[DC_CLASSES];
};

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
  // workspace
  float *logits;        // [T][E]
  uint16_t *y16;        // [T][H] y in scaled binary16; null: the form of separate products
  float *back;          // [T] what undoes the scale
  float *partial;       // [S][T][H]
  uint32_t *count;      // [H / 16]
  DcSync *sync;
  int32_t *all_ids;     // [T][c], the shared expert's among them
  float *all_prob;
  int ks, S;            // waves that share a contraction; parts of the experts
  uint32_t tg_inv;      // 2^32 over the items of an expert, rounded up
};

__device__ __forceinline__ int dc_uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

}  // namespace

// Norm and router: 16 experts by a few tokens a workgroup, each of which
// normalises its tokens itself (the first column of workgroups writes h and y).
// A wave takes every eighth 64-wide block of the contraction, its first four
// asked for before the norm.  The order of two logits decides which experts a token
// meets, so the matrix instructions' sums of 32 products are added up in binary64: a
// logit is off by little more than its last rounding.  Bound by the chain
// of its steps (load, sum, root, products, join): 6.0 us for up to 4 tokens of 2048
// and 128 experts, 10.8 for 37 of 5120 and 64, of which an empty launch is 1.6; eight
// blocks asked for ahead take 0.7 us longer, the norm's loads waiting behind them.
template <int NC, bool WF32>
__global__ __launch_bounds__(512) void k_decode_router(DcArgs a) {
  constexpr int DR_TOKENS = dr_tokens(NC);
  extern __shared__ __align__(16) uint8_t lds[];  // y: rows of H values and 16 bytes
  __shared__ double red[8][DR_TOKENS];
  __shared__ uint32_t top[8][DR_TOKENS];
  __shared__ double sums[8][DR_TOKENS][16];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, ln = lane & 15;
  const int wave = dc_uniform(tid >> 6);
  const int t0 = blockIdx.y * DR_TOKENS, n = min(DR_TOKENS, a.T - t0), e0 = blockIdx.x * 16;
  const int H = a.H, pitch = 2 * H + 16, blocks = (H + 63) / 64;
  if (blockIdx.x == 0 && blockIdx.y == 0) {  // for the kernel behind this one
    for (int i = tid; i < H / 16; i += 512) a.count[i] = 0;
    if (tid < DC_CLASSES) a.sync->of[tid].ticket = a.sync->of[tid].done = 0;
  }
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

  float wf[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (i * 512 + tid) * 8;
    if (c < H) load_w8<WF32>(a.norm_w, c, wf[i]);
  }
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
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * 512 + tid) * 8;
      if (c >= H) continue;
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)  // binary64 throughout: y is the nearest bf16 value
        o[j] = pk_bf16_rne(
            before_bf16((double)bf16_lo_f32(v[t][i][j]) * (double)wf[i][2 * j] * root),
            before_bf16((double)bf16_hi_f32(v[t][i][j]) * (double)wf[i][2 * j + 1] * root));
      *reinterpret_cast<uint4 *>(lds + t * pitch + 2 * c) = make_uint4(o[0], o[1], o[2], o[3]);
      if (blockIdx.x == 0) {
        const int64_t at = (int64_t)(t0 + t) * H + c;
        *reinterpret_cast<uint4 *>(a.h + at) =
            make_uint4(v[t][i][0], v[t][i][1], v[t][i][2], v[t][i][3]);
        *reinterpret_cast<uint4 *>(a.y + at) = make_uint4(o[0], o[1], o[2], o[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[t][i][j] = o[j];
          most = pk_max_u16(most, o[j] & 0x7FFF7FFFu);
        }
      }
    }
    if (blockIdx.x == 0) {
      most = max(most & 0xFFFFu, most >> 16);
      most = group_max<64>(most);
      if (lane == 0) top[wave][t] = most;
    }
  }
  __syncthreads();
  // y again in binary16, under the power of two that brings the row's largest value
  // to 2^14 .. 2^15: bf16 has 8 significant bits, so values down to 2^-31 of the
  // largest stay exact, and weights in binary16 take half the instructions of bf16.
  if (blockIdx.x == 0 && a.y16) {
#pragma unroll
    for (int t = 0; t < DR_TOKENS; ++t) {
      if (t >= n) break;
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) most = max(most, top[i][t]);
      const int ex = min(127, 14 + 127 - (int)(most >> 7));
      const float up = __builtin_ldexpf(1.0f, ex);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = (i * 512 + tid) * 8;
        if (c >= H) continue;
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = __builtin_bit_cast(
              uint32_t, __builtin_amdgcn_cvt_pkrtz(bf16_lo_f32(v[t][i][j]) * up,
                                                   bf16_hi_f32(v[t][i][j]) * up));
        *reinterpret_cast<uint4 *>(a.y16 + (int64_t)(t0 + t) * H + c) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (tid == 0) a.back[t0 + t] = __builtin_ldexpf(1.0f, -ex);
    }
  }

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

// A token's gate by one wave, expert 64 i + lane in register i: the choice, the
// scores and the renormalisation of pqm_moe_gate, to the token's k ids and probs.
template <int VPL>
__device__ __forceinline__ void dc_gate(const DcArgs &a, const float (&z)[VPL], int32_t *ids,
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
    ids[l] = my_id;
    prob[l] = w * a.scale;
  }
}

// The same from the logits; past the last token nothing.
template <int VPL>
__device__ __forceinline__ void dc_gate_of(const DcArgs &a, int t, int32_t *ids, float *prob) {
  const int l = threadIdx.x & 63;
  if (t >= a.T) return;
  const __amdgpu_buffer_rsrc_t zb = gv_buffer(a.logits, (int64_t)a.T * a.E * 4);
  float z[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    z[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
        zb, (int)(64 * i + l < a.E ? (uint32_t)(t * a.E + 64 * i + l) * 4 : GV_NONE), 0, 0));
  dc_gate<VPL>(a, z, ids, prob);
}

// Which tokens meet an expert, and as which of their choices.
struct DcSets {
  uint32_t rows[DC_EXPERTS];
  uint8_t slot[DC_FEW][DC_EXPERTS];
};

// The experts met, in order, the shared one last: every wave keeps them as sets of
// 64 in scalar registers, which takes no barrier and no list.
template <int VPL>
struct DcMet {
  uint64_t in[VPL];
  int n;

  __device__ __forceinline__ DcMet(const DcArgs &a, const DcSets &s) {
    const int lane = threadIdx.x & 63;
    n = a.c - a.k;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = 64 * i + lane;
      in[i] = __ballot(e < a.E && s.rows[e] != 0);
      n += __popcll(in[i]);
    }
  }
  // The i-th.
  __device__ __forceinline__ int operator()(const DcArgs &a, int i) const {
    const int lane = threadIdx.x & 63;
    int e = a.E;
#pragma unroll
    for (int w = 0; w < VPL; ++w) {
      const int here = __popcll(in[w]);
      if (i >= 0 && i < here) {
        const uint64_t at = __ballot((in[w] >> lane & 1) &&
                                     __popcll(in[w] & ((1ull << lane) - 1)) == i);
        e = 64 * w + __ffsll((unsigned long long)at) - 1;
      }
      i -= here;
    }
    return dc_uniform(e);
  }
};

__device__ __forceinline__ uint32_t dc_rows(const DcArgs &a, const DcSets &s, int e) {
  return e == a.E ? (1u << a.T) - 1 : (uint32_t)dc_uniform((int)s.rows[e]);
}

// The token of row l % 16 of a set of up to 16 (its members in order).
__device__ __forceinline__ int dc_member(uint32_t rows) {
  const int lane = threadIdx.x & 63, c = __popc(rows);
  const int before = __popc(rows & ((1u << (lane & 31)) - 1));
  const int at = rows >> (lane & 31) & 1 ? before : c + (lane & 31) - before;
  const int members = __builtin_amdgcn_ds_permute(4 * (at + (lane & 32)), lane & 31);
  return __builtin_amdgcn_ds_bpermute(4 * (lane & 15), members);
}

// Which of its token's rows an expert's row is.
__device__ __forceinline__ int dc_slot(const DcArgs &a, const DcSets &s, int t, int e) {
  return e == a.E ? a.k : s.slot[t & (DC_FEW - 1)][e];
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

// What a chunk's product takes of 16 rows, whose values start at xo (GV_NONE: no
// row) of xb: lane group g has the chunk's values 64 g .. + 63.  No branch: the
// loads have to stay in their order, or the waits for them would wait for the next
// chunk's weights too.
__device__ __forceinline__ void dc_load_x(gv_u4 (&x)[8], __amdgpu_buffer_rsrc_t xb, uint32_t xo,
                                          int K, int ch) {
  const uint32_t kk = 256 * ch + 64 * ((threadIdx.x & 63) >> 4);
  const uint32_t lo = (xo + 2 * kk) | (kk < (uint32_t)K ? 0 : GV_NONE);
  const uint32_t hi = (xo + 2 * kk) | (kk + 32 < (uint32_t)K ? 0 : GV_NONE);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    x[j] = __builtin_amdgcn_raw_buffer_load_b128(xb, (int)(j < 4 ? lo : hi), 16 * j, 0);
}

// Eight weights in binary16: exact, and half the instructions of bf16.
__device__ __forceinline__ gv_h8 dc_decode16(uint32_t u, _Float16 f) {
  const gv_h2 s = {f, f};
  const gv_h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.0f, 0) * s;
  const gv_h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.0f, 1) * s;
  const gv_h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.0f, 2) * s;
  const gv_h2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.0f, 3) * s;
  return gv_h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A chunk of a weight tile times 16 rows, in binary16 or bf16.
template <bool HALF>
__device__ __forceinline__ void dc_multiply(gv_f4 &acc, const DcChunk &b, const gv_u4 (&x)[8],
                                            const GvTurn &turn, int K, int ch) {
  const int lane = threadIdx.x & 63, g = lane >> 4, ln = lane & 15;
  gv_u4 q[2];
  turn(b.q, q);
  int sw = __builtin_amdgcn_ds_bpermute(16 * ln + 4 * g, (int)b.s);
  // past the row's end stand the next row's scales, maybe NaN: x is 0 there, the
  // scale has to be so too
  const int left = K - 256 * ch - 64 * g;
  if (left < 64) sw = left == 32 ? sw & 0xFFFF : 0;
  if constexpr (HALF) {
    const gv_h2 f[2] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sw, 1.0f, false),
                        __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sw, 1.0f, true)};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(
          dc_decode16(q[j >> 2][j & 3], f[j >> 2][(j >> 1) & 1]),
          __builtin_bit_cast(gv_h8, x[j]), acc, 0, 0, 0);
  } else {
    const float f[4] = {__builtin_amdgcn_cvt_f32_fp8(sw, 0), __builtin_amdgcn_cvt_f32_fp8(sw, 1),
                        __builtin_amdgcn_cvt_f32_fp8(sw, 2), __builtin_amdgcn_cvt_f32_fp8(sw, 3)};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(gv_decode(q[j >> 2][j & 3], f[j >> 1]),
                                                    __builtin_bit_cast(gv_bf8, x[j]), acc, 0, 0, 0);
  }
}

// The next ticket of a class (one lane).
__device__ __forceinline__ uint32_t dc_draw(DcSync *sync, int cls) {
  return __hip_atomic_fetch_add(&sync->of[cls].ticket, 1u, __ATOMIC_RELAXED,
                                __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ int dc_drawn(uint32_t ticket, int cls, int total) {
  return ticket < (uint32_t)((total - cls + DC_CLASSES - 1) / DC_CLASSES)
             ? cls + DC_CLASSES * (int)ticket
             : -1;
}

// With its own class at an end, a workgroup looks at all of them at once (the first
// wave) and draws where there are any left.  -1: every item is drawn, each by a
// workgroup that runs.
__device__ __forceinline__ int dc_sweep(DcSync *sync, int total) {
  const int lane = threadIdx.x & 63, cls = lane % DC_CLASSES;
  int got = -1;
  uint32_t v = lane < DC_CLASSES ? __hip_atomic_load(&sync->of[cls].ticket, __ATOMIC_RELAXED,
                                                     __HIP_MEMORY_SCOPE_AGENT)
                                 : 0xFFFFFFFFu;
  uint64_t open = __ballot(dc_drawn(v, cls, total) >= 0);
  while (got < 0 && open) {  // each turn draws or closes a class
    const int who = __ffsll((unsigned long long)open) - 1;
    if (lane == who) v = dc_draw(sync, cls);
    got = __builtin_amdgcn_readlane(dc_drawn(v, cls, total), who);
    open &= ~(1ull << who);
  }
  return got;
}

}  // namespace

// Gate, gate_up, down projection and sum in one kernel, one workgroup a CU.
//
// gate_up's items (an expert, 16 / ks tiles of 16 columns; ks waves share a tile's
// contraction) are drawn by ticket, so whoever waits for the last of them waits for
// workgroups that run and wait for nothing themselves: the wait ends however many
// workgroups the card holds at once, also beside other calls.  Eight counters, since
// one address takes 10 ns a draw: 256 workgroups draw in 2.8 us from one and in 1.1
// from eight, and meet in 3.8 and 1.4.  d goes past the L2, of which each XCD has its
// own, and nothing of it is read before the wait.
//
// The down projection's items are 16 columns and a part of the experts met; its waves
// take (expert, chunk) in turn, each with sums of its own, the first chunk's weights
// asked for before the wait.  The workgroup that finishes a column's last part adds
// the parts in their order.
//
// Bound by the chain gate, weights, join, weights, join; one token, top-8 of 128 experts
// of 2048 x 768: 21 MB in 15.2 to 17 us (4.2 at a copy's rate).  Above 256 experts the 16
// sets of those met leave the registers (44 bytes a lane in scratch): the whole layer
// 24.2 us for 256 experts and 30.4 for 512, for three tokens 35.7 and 44.8.
template <int VPL, bool WORDS1, bool WORDS2>
__global__ __launch_bounds__(64 * DC_WAVES, 4) void k_decode_experts(DcArgs a) {
  __shared__ DcSets s;
  __shared__ int32_t ids[DC_FEW * DC_K];
  __shared__ float prob[DC_FEW * DC_K];
  __shared__ __align__(16) uint8_t turns[DC_WAVES][2048];
  __shared__ gv_f4 red[2][DC_WAVES][2][64];
  __shared__ int drawn[2], last;
  float(*const sums)[DC_FEW * 16] = reinterpret_cast<float(*)[DC_FEW * 16]>(red);
  static_assert(sizeof(red) >= 4 * DC_WAVES * DC_FEW * 16, "the down projection's sums");
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, ln = lane & 15;
  const int wave = dc_uniform(tid >> 6);
  const GvTurn turn(turns[wave], lane);

  uint32_t ticket = 0;
  const int cls = blockIdx.x % DC_CLASSES;
  if (tid == 0) ticket = dc_draw(a.sync, cls);
  for (int e = tid; e < a.E; e += 64 * DC_WAVES) s.rows[e] = 0;
  __syncthreads();
  for (int t = wave; t < a.T; t += DC_WAVES) {
    dc_gate_of<VPL>(a, t, ids + t * a.k, prob + t * a.k);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (lane < a.k) {
      const int e = ids[t * a.k + lane];
      atomicOr(&s.rows[e], 1u << t);
      s.slot[t][e] = (uint8_t)lane;
      if (blockIdx.x == 0) {
        a.ids[t * a.k + lane] = e;
        a.prob[t * a.k + lane] = prob[t * a.k + lane];
      }
    }
  }
  __syncthreads();
  const DcMet<VPL> met(a, s);

  const int per = DC_WAVES / a.ks, kw = wave & (a.ks - 1), tiles = a.I / 16;
  const int tg = (tiles + per - 1) / per, total = met.n * tg;
  {
    const int K = a.H, chunks = (K + 255) / 256;
    const __amdgpu_buffer_rsrc_t xb = gv_buffer(a.y16, (int64_t)a.T * K * 2);
    if (tid == 0) drawn[1] = dc_drawn(ticket, cls, total);
    __syncthreads();
    // the item, its expert and that one's rows, and this wave's tile of it
    int item = dc_uniform(drawn[1]), buf = 0, finished = 0, ch = kw, e = 0, first = 0, tok = 0;
    bool row = false;
    float outer = 0.0f, back = 0.0f;
    const auto open = [&]() {
      const int i = tg == 1 ? item : (int)__umulhi((uint32_t)item, a.tg_inv);  // item / tg
      first = (item - i * tg) * per;
      e = met(a, i);
      const uint32_t rows = dc_rows(a, s, e);
      tok = dc_member(rows);
      row = ln < __popc(rows);
      ch = kw;
      outer = a.g1[e];
      back = a.back[tok & (DC_FEW - 1)];
    };
    const auto load = [&](DcChunk (&b)[2], int ch) {
      const int tile = first + wave / a.ks;
      const bool in = tile < tiles && ch < chunks;
      const int64_t r0 = (int64_t)e * 2 * a.I + (tile < tiles ? 16 * tile : 0), r1 = r0 + a.I;
      dc_load<WORDS1>(b[0], gv_buffer(a.w1 + r0 * (K / 2), 8 * (int64_t)K),
                      gv_buffer(a.s1 + r0 * (K / 16), (int64_t)K), K, ch, in);
      dc_load<WORDS1>(b[1], gv_buffer(a.w1 + r1 * (K / 2), 8 * (int64_t)K),
                      gv_buffer(a.s1 + r1 * (K / 16), (int64_t)K), K, ch, in);
    };
    gv_f4 acc[2] = {};
    // A chunk, whose weights are in b; the next one's go out behind this one's rows, so
    // that the wait for the rows leaves them in flight.  Two sets of registers in turn,
    // since a copy would wait, and no more than two copies of this code: what runs once
    // waits for its own instructions.  False: no item is left anywhere.
    const auto step = [&](const DcChunk (&b)[2], DcChunk (&next)[2]) {
      gv_u4 x[8];
      dc_load_x(x, xb, row ? (uint32_t)tok * K * 2 : GV_NONE, K, ch);
      __builtin_amdgcn_sched_barrier(0);
      if (ch == kw && tid == 0) ticket = dc_draw(a.sync, cls);
      load(next, ch + a.ks);
      __builtin_amdgcn_sched_barrier(0);
      dc_multiply<true>(acc[0], b[0], x, turn, K, ch);
      dc_multiply<true>(acc[1], b[1], x, turn, K, ch);
      ch += a.ks;
      if (ch < chunks) return true;
      red[buf][wave][0][lane] = acc[0];
      red[buf][wave][1][lane] = acc[1];
      acc[0] = acc[1] = gv_f4{0, 0, 0, 0};
      if (tid == 0) drawn[buf] = dc_drawn(ticket, cls, total);
      // tile t of the item is wave t's to finish
      const int mine = first + wave, at = tok, j = dc_slot(a, s, tok, e);
      const bool ends = wave < per && mine < tiles && row;
      const float out1 = outer, undo = back;
      float p = 1.0f;
      if (ends && j < a.k) p = prob[tok * a.k + j];
      __syncthreads();
      item = dc_uniform(drawn[buf]);
      const int was = buf;
      buf ^= 1;
      ++finished;
      if (item >= 0) {
        open();
        load(next, ch);
      }
      if (ends) {
        gv_f4 vg = red[was][wave * a.ks][0][lane], vu = red[was][wave * a.ks][1][lane];
        for (int q = 1; q < a.ks; ++q) {
          vg += red[was][wave * a.ks + q][0][lane];
          vu += red[was][wave * a.ks + q][1][lane];
        }
        float o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = swiglu_f32(vg[q] * undo * out1, vu[q] * undo * out1, p);
        __hip_atomic_store(
            reinterpret_cast<uint64_t *>(a.d + (int64_t)(at * a.c + j) * a.I + 16 * mine + 4 * g),
            (uint64_t)pk_bf16_rne(o[2], o[3]) << 32 | pk_bf16_rne(o[0], o[1]), __ATOMIC_RELAXED,
            __HIP_MEMORY_SCOPE_AGENT);
      }
      return item >= 0;
    };
    for (;;) {
      if (item >= 0) {
        open();
        DcChunk b0[2], b1[2];
        load(b0, ch);
        while (step(b0, b1) && step(b1, b0)) {
        }
      }
      // Its class is at an end: every wave's part of d has to arrive before the
      // workgroup says so, and what is left of other classes is taken.
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (tid == 0 && finished)
        __hip_atomic_fetch_add(&a.sync->of[cls].done, (uint32_t)finished, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
      finished = 0;
      if (wave == 0) {
        const int t = dc_sweep(a.sync, total);
        if (lane == 0) drawn[buf ^ 1] = t;
      }
      __syncthreads();
      item = dc_uniform(drawn[buf ^ 1]);
      if (item < 0) break;
    }
  }

  const int K = a.I, chunks = (K + 255) / 256, NT = a.H / 16;
  const __amdgpu_buffer_rsrc_t xb = gv_buffer(a.d, (int64_t)a.T * a.c * K * 2);
  bool waited = false;
  for (int item = blockIdx.x; item < NT * a.S; item += DC_GRID) {
    const int part = item / NT, tile = item - part * NT;
    const int i0 = met.n * part / a.S, i1 = met.n * (part + 1) / a.S, units = (i1 - i0) * chunks;
    // a chunk of an expert: its weights, and where the rows' values start
    struct Unit {
      DcChunk b;
      float outer;
      uint32_t xo;
      int tok, ch;
    };
    const auto load = [&](Unit &t, int u) {
      const bool in = u < units;
      const int i = u / chunks, e = in ? met(a, i0 + i) : 0;
      t.ch = u - i * chunks;
      const int64_t r0 = (int64_t)e * a.H + 16 * tile;
      dc_load<WORDS2>(t.b, gv_buffer(a.w2 + r0 * (K / 2), 8 * (int64_t)K),
                      gv_buffer(a.s2 + r0 * (K / 16), (int64_t)K), K, t.ch, in);
      t.outer = a.g2[e];
      const uint32_t rows = dc_rows(a, s, e);
      const int tok = dc_member(rows);
      const uint32_t at = (uint32_t)(tok * a.c + dc_slot(a, s, tok, e)) * K * 2;
      t.xo = ln < __popc(rows) ? at : GV_NONE;
      t.tok = tok;
    };
    Unit u0, u1;
    load(u0, wave);
    for (int i = lane; i < a.T * 4; i += 64)
      reinterpret_cast<gv_f4 *>(sums[wave])[i] = gv_f4{0, 0, 0, 0};
    if (!waited) {
      if (wave == 0) {
        for (;;) {
          const uint32_t v = lane < DC_CLASSES
                                 ? __hip_atomic_load(&a.sync->of[lane].done, __ATOMIC_RELAXED,
                                                     __HIP_MEMORY_SCOPE_AGENT)
                                 : 0;
          int n = 0;
#pragma unroll
          for (int q = 0; q < DC_CLASSES; ++q) n += __builtin_amdgcn_readlane((int)v, q);
          if (n == total) break;
          __builtin_amdgcn_s_sleep(2);
        }
        // for the whole CU: nothing of d that was cached before is read
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      }
      __syncthreads();
      waited = true;
    }
    const auto turn_of = [&](const Unit &t, Unit &next, int u) {
      gv_u4 x[8];
      dc_load_x(x, xb, t.xo, K, t.ch);
      __builtin_amdgcn_sched_barrier(0);
      load(next, u + DC_WAVES);
      __builtin_amdgcn_sched_barrier(0);
      gv_f4 acc = {0, 0, 0, 0};
      dc_multiply<false>(acc, t.b, x, turn, K, t.ch);
      if (t.xo != GV_NONE) *reinterpret_cast<gv_f4 *>(sums[wave] + t.tok * 16 + 4 * g) += acc * t.outer;
    };
    for (int u = wave; u < units; u += 2 * DC_WAVES) {
      turn_of(u0, u1, u);
      if (u + DC_WAVES >= units) break;
      turn_of(u1, u0, u + DC_WAVES);
    }
    __syncthreads();
    const int t = tid >> 3, c = 2 * (tid & 7);
    const bool one = tid < a.T * 8;
    const int64_t o = (int64_t)t * a.H + 16 * tile + c;
    float v0 = 0.0f, v1 = 0.0f;
    if (one) {
#pragma unroll
      for (int w = 0; w < DC_WAVES; ++w) {
        v0 += sums[w][t * 16 + c];
        v1 += sums[w][t * 16 + c + 1];
      }
      if (a.S == 1) {
        *reinterpret_cast<uint32_t *>(a.out + o) = pk_bf16_rne(v0, v1);
      } else {
        __hip_atomic_store(reinterpret_cast<uint64_t *>(a.partial + (int64_t)part * a.T * a.H + o),
                           (uint64_t)__float_as_uint(v1) << 32 | __float_as_uint(v0),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    if (a.S > 1) {
      // The sums went past the L2 and are waited for; a fence would write back the
      // whole L2, for each wave.
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (tid == 0)
        last = __hip_atomic_fetch_add(&a.count[tile], 1u, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)a.S - 1;
      __syncthreads();
      if (last && one) {
        v0 = v1 = 0.0f;
        for (int q = 0; q < a.S; ++q) {
          const uint64_t v =
              __hip_atomic_load(reinterpret_cast<uint64_t *>(a.partial + (int64_t)q * a.T * a.H + o),
                                __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          v0 += __uint_as_float((uint32_t)v);
          v1 += __uint_as_float((uint32_t)(v >> 32));
        }
        *reinterpret_cast<uint32_t *>(a.out + o) = pk_bf16_rne(v0, v1);
      }
    }
    __syncthreads();
  }
}

// More tokens: the gate by itself, then the few-row products of gemv_nvfp4.hip
// over all rows (the shared expert's among them, as experts of up to 16 rows behind
// the routed ones), then the sum.  Bound by the weights: 37 tokens, top-8 of 64 experts
// of 5120 x 1280 and a shared one, 719 MB: 96 + 64 us of 171 (5 launches the rest).
template <int VPL>
__global__ __launch_bounds__(256) void k_decode_gate(DcArgs a) {
  __shared__ int32_t ids[4 * DC_K];
  __shared__ float prob[4 * DC_K];
  const int wave = dc_uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + wave;
  if (t >= a.T) return;
  dc_gate_of<VPL>(a, t, ids + wave * a.k, prob + wave * a.k);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (lane < a.c) {
    const bool routed = lane < a.k;
    // the shared expert's rows in groups of 16, each an expert to the products
    const int32_t id = routed ? ids[wave * a.k + lane] : a.E + t / 16;
    const float p = routed ? prob[wave * a.k + lane] : 1.0f;
    a.all_ids[t * a.c + lane] = id;
    a.all_prob[t * a.c + lane] = p;
    if (routed) {
      a.ids[t * a.k + lane] = id;
      a.prob[t * a.k + lane] = p;
    }
  }
}

__global__ __launch_bounds__(256) void k_decode_sum(const float *__restrict__ rows, int T, int c,
                                                    int H, uint16_t *__restrict__ out) {
  const int i = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= T * H) return;
  const int t = i / H, n = i - t * H;
  gv_f4 v = {0, 0, 0, 0};
#pragma unroll 4
  for (int j = 0; j < c; ++j)
    v += *reinterpret_cast<const gv_f4 *>(rows + ((int64_t)t * c + j) * H + n);
  *reinterpret_cast<uint2 *>(out + i) = make_uint2(pk_bf16_rne(v[0], v[1]), pk_bf16_rne(v[2], v[3]));
}

namespace {

struct DcPlan {
  int ks, S;
};

// By size alone, for as many experts met as there can be: the shape that leaves the
// fewest turns of a wave, where an item costs half a turn of its own.
DcPlan dc_plan(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int shared) {
  const int64_t met = (T * k < E ? T * k : E) + shared, chunks = (H + 255) / 256;
  DcPlan p = {1, 1};
  int64_t best = 0;
  for (int ks = 1; ks <= DC_WAVES && ks <= chunks; ks *= 2) {
    const int64_t per = DC_WAVES / ks, items = met * ((I / 16 + per - 1) / per);
    const int64_t cost = (items + DC_GRID - 1) / DC_GRID * (2 * ((chunks + ks - 1) / ks) + 1);
    if (ks == 1 || cost <= best) {
      best = cost;
      p.ks = ks;
    }
  }
  const int64_t tiles = H / 16, units = met * ((I + 255) / 256);
  for (int S = 1; S <= 8 && S <= met; ++S) {
    const int64_t turns = ((units + S - 1) / S + DC_WAVES - 1) / DC_WAVES;
    const int64_t cost = (tiles * S + DC_GRID - 1) / DC_GRID * (2 * turns + 1) + (S > 1 ? 3 : 0);
    if (S == 1 || cost < best) {
      best = cost;
      p.S = S;
    }
  }
  return p;
}

// One kernel up to DC_FEW tokens whose experts hold up to 96 MB: 128 experts of
// 2048 x 768, top-8, 24.3 us for one token and 36.3 for three (26.3 and 38.4 by
// separate products), 16 of 4096 x 1024, top-2, 42.9 for eight (46.4).  Beyond, the
// separate products stream the weights faster: 64 experts of 5120 x 1280, top-8, three
// tokens 69.8 us against 92.5, 16 tokens 145 against 186.
bool dc_is_few(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int shared) {
  const int64_t met = (T * k < E ? T * k : E) + shared;
  return T <= DC_FEW && met * H * I / 16 * 27 <= (int64_t)96 << 20;
}

bool dc_sizes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k) {
  return T >= 0 && T <= DC_TOKENS && H >= 32 && H <= DC_WIDTH && H % 32 == 0 && I >= 32 &&
         I <= DC_WIDTH && I % 32 == 0 && E >= 1 && E <= DC_EXPERTS && k >= 1 && k <= DC_K && k <= E;
}

// Offsets into the workspace.
struct DcLayout {
  size_t y16, back, partial, count, sync, ids, prob, rows, bytes;
};

DcLayout dc_layout(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int shared) {
  DcLayout l;
  size_t at = 0;
  const auto take = [&](int64_t n) {
    const size_t r = at;
    at += (size_t)(n + 255) / 256 * 256;
    return r;
  };
  const bool few = dc_is_few(T, H, I, E, k, shared);
  const int64_t rows = T * (k + shared);
  take(T * E * 4);
  l.y16 = take(few ? T * H * 2 : 0);
  l.back = take(few ? T * 4 : 0);
  l.partial = take(few ? dc_plan(T, H, I, E, k, shared).S * T * H * 4 : 0);
  l.count = take(H / 16 * 4);
  l.sync = take(sizeof(DcSync));
  l.ids = take(few ? 0 : rows * 4);
  l.prob = take(few ? 0 : rows * 4);
  l.rows = take(few ? 0 : rows * H * 4);
  l.bytes = at;
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

template <int VPL>
hipError_t dc_few(const DcArgs &a, hipStream_t st) {
  const auto kernel = a.H % 64 == 0 ? a.I % 64 == 0 ? k_decode_experts<VPL, true, true>
                                                    : k_decode_experts<VPL, true, false>
                      : a.I % 64 == 0 ? k_decode_experts<VPL, false, true>
                                      : k_decode_experts<VPL, false, false>;
  hipLaunchKernelGGL(kernel, dim3(DC_GRID), dim3(64 * DC_WAVES), 0, st, a);
  return hipGetLastError();
}

template <int VPL>
hipError_t dc_many(const DcArgs &a, float *rows, hipStream_t st) {
  hipLaunchKernelGGL(k_decode_gate<VPL>, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, st, a);
  hipError_t r = hipGetLastError();
  if (r != hipSuccess) return r;
  const int64_t n = (int64_t)a.T * a.c, GW = a.E + (a.c - a.k);
  const int64_t G = a.c > a.k ? a.E + (a.T + 15) / 16 : a.E;
  r = launch_gemv_nvfp4(a.y, a.all_ids, a.all_prob, n, a.c, a.w1, a.s1, a.g1, 2 * a.I, G, GW, a.I,
                        a.H, a.d, false, st);
  if (r != hipSuccess) return r;
  r = launch_gemv_nvfp4(a.d, a.all_ids, nullptr, n, 1, a.w2, a.s2, a.g2, a.H, G, GW, a.H, a.I,
                        rows, true, st);
  if (r != hipSuccess) return r;
  hipLaunchKernelGGL(k_decode_sum, dim3((unsigned)((a.T * a.H / 4 + 255) / 256)), dim3(256), 0, st,
                     rows, a.T, a.c, a.H, a.out);
  return hipGetLastError();
}

template <int VPL>
hipError_t dc_experts(const DcArgs &a, float *rows, hipStream_t st) {
  return a.y16 ? dc_few<VPL>(a, st) : dc_many<VPL>(a, rows, st);
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
  const bool few = dc_is_few(tokens, hidden, inter, num_experts, k, shared_expert);
  // item / tg is exact for items up to 2^21 and tg from 2 to 2^10
  const int64_t per = DC_WAVES / p.ks, tg = (inter / 16 + per - 1) / per;
  const uint32_t tg_inv = tg == 1 ? 0 : (uint32_t)((((int64_t)1 << 32) + tg - 1) / tg);
  const DcArgs a = {x, residual, norm_w, eps, gate_w, (int)tokens, (int)hidden, (int)inter,
                    (int)num_experts, (int)k, (int)k + shared_expert, score == PQM_SCORE_SOFTMAX,
                    renormalize, scale, w1_q, w1_scale, w1_outer, w2_q, w2_scale, w2_outer, h, y,
                    topk_ids, prob, d, out, reinterpret_cast<float *>(ws),
                    few ? reinterpret_cast<uint16_t *>(ws + l.y16) : nullptr,
                    reinterpret_cast<float *>(ws + l.back),
                    reinterpret_cast<float *>(ws + l.partial),
                    reinterpret_cast<uint32_t *>(ws + l.count),
                    reinterpret_cast<DcSync *>(ws + l.sync),
                    reinterpret_cast<int32_t *>(ws + l.ids),
                    reinterpret_cast<float *>(ws + l.prob), p.ks, p.S, tg_inv};
  const bool wf32 = norm_dtype == PQM_OUT_FP32;
  if (hidden <= 4096) dc_router<1>(a, wf32, stream);
  else if (hidden <= 8192) dc_router<2>(a, wf32, stream);
  else dc_router<4>(a, wf32, stream);
  if (hipGetLastError() != hipSuccess) return PQM_ERR_HIP;
  float *rows = reinterpret_cast<float *>(ws + l.rows);
  const hipError_t r = num_experts <= 64    ? dc_experts<1>(a, rows, stream)
                       : num_experts <= 128 ? dc_experts<2>(a, rows, stream)
                       : num_experts <= 256 ? dc_experts<4>(a, rows, stream)
                                            : dc_experts<16>(a, rows, stream);
  return r == hipSuccess ? PQM_OK : PQM_ERR_HIP;
}

}  // extern "C"
