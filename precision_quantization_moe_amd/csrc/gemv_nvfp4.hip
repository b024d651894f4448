// gemv_nvfp4.hip -- the experts' products for a few routed rows: bf16
// activations times NVFP4 weights, the decode form of the grouped GEMM.
//
//   y[r, n] = s_g sum_k x[r / div, k] q[e, n, k] s_b[e, n, k / 16],  e = ids[r],
// and for the gate_up projection d[r, n] = bf16(silu(g) u p[r]) of the rows n
// (gate) and I + n (up).  The weights are read once per expert that a row
// chose (and per 16 rows of it); rows of the same expert are found in `ids` by
// the workgroups themselves, so no sort, gather or offsets go before.
//
// A wave multiplies 16 weight rows by up to 16 activation rows with a 16x16x32
// matrix instruction; the sums are binary32 and the outer scale multiplies
// them at the end.  q s_b has at most 6 significant bits, exact in bf16 and in
// f16.
#include "pqm_device.hpp"
#include "pqm_internal.hpp"
#include "pqmoe.h"

namespace pqm {

namespace {

typedef __bf16 gv_bf8 __attribute__((ext_vector_type(8)));
typedef float gv_f4 __attribute__((ext_vector_type(4)));
typedef float gv_f2 __attribute__((ext_vector_type(2)));
typedef uint32_t gv_u4 __attribute__((ext_vector_type(4)));
typedef _Float16 gv_h2 __attribute__((ext_vector_type(2)));
typedef _Float16 gv_h8 __attribute__((ext_vector_type(8)));

constexpr int GEMV_MAX_ROWS = 4096;
constexpr uint32_t GV_NONE = 0x80000000u;  // an offset past every buffer below: reads give 0

struct GemvArgs {
  const uint16_t *x;
  int rows, div;
  const uint8_t *w, *ws;
  const float *wo;
  int64_t rps;
  int G;
  int64_t N, K;  // N: output columns; ACT weights have 2 N rows
  const float *prob;
  void *out;
  int byrow;  // blockIdx.y is a row of ids and stands for its expert if no earlier row chose it;
              // otherwise it is the expert, and G the rows without one
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t gv_buffer(const void *p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, 0x00020000);
}

// This workgroup's expert, -1 for none.
__device__ __forceinline__ int gv_expert(const GemvArgs &a, const int32_t *ids) {
  const int e = a.byrow ? ids[blockIdx.y] : (int)blockIdx.y;
  return __builtin_amdgcn_readfirstlane(e < 0 || e >= a.G ? -1 : e);
}

// ids[r], 0 past the end.
__device__ __forceinline__ int gv_id(const GemvArgs &a, const int32_t *ids, int r) {
  return (int)__builtin_amdgcn_raw_buffer_load_b32(gv_buffer(ids, 4 * a.rows), 4 * r, 0, 0);
}

// The rows of expert e in order, and their number: 0 where another workgroup
// serves them.  `id` is gv_id of this thread's row.
template <int WAVES>
__device__ __forceinline__ int gv_rows(const GemvArgs &a, const int32_t *ids, int id, int e,
                                       uint16_t *list, int *cnt) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int c = 0;
  bool mine_first = true;
  for (int r0 = 0; r0 < a.rows; r0 += 64 * WAVES) {
    const int r = r0 + tid;
    if (r0 > 0) id = gv_id(a, ids, r);
    const bool mine = r < a.rows && (id < 0 || id >= a.G ? -1 : id) == e;
    const uint64_t b = __ballot(mine), before = __ballot(a.byrow && mine && r < (int)blockIdx.y);
    if (lane == 0) cnt[wave] = __popcll(b) | (before ? 256 : 0);
    __syncthreads();
    int pos = c + __popcll(b & ((1ull << lane) - 1));
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const int n = cnt[w] & 255;
      if (cnt[w] & 256) mine_first = false;
      c += n;
      if (w < wave) pos += n;
    }
    if (mine) list[pos] = (uint16_t)r;
    __syncthreads();
  }
  return __builtin_amdgcn_readfirstlane(mine_first ? c : 0);
}

template <bool OUTF32>
__device__ __forceinline__ void gv_store(const GemvArgs &a, int64_t at, float v) {
  if (OUTF32) static_cast<float *>(a.out)[at] = v;
  else static_cast<uint16_t *>(a.out)[at] = (uint16_t)pk_bf16_rne(v, 0.0f);
}

// Zeros for the rows without an expert, columns n0 .. n0 + cols - 1.
template <bool OUTF32>
__device__ __forceinline__ void gv_zero(const GemvArgs &a, const uint16_t *list, int c, int64_t n0,
                                        int cols) {
  for (int i = threadIdx.x; i < c * cols; i += blockDim.x)
    gv_store<OUTF32>(a, (int64_t)list[i / cols] * a.N + n0 + i % cols, 0.0f);
}

// The outer scale of weight row n of expert e.
__device__ __forceinline__ float gv_outer(const GemvArgs &a, int e, int64_t NW, int64_t n) {
  return a.rps == NW ? a.wo[e] : a.wo[((int64_t)e * NW + n) / a.rps];
}

// Eight weights (the nibbles of w, lowest first) times their block's scale.
__device__ __forceinline__ gv_bf8 gv_decode(uint32_t w, float s) {
  const gv_f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
  const gv_f2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const gv_f2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
  const gv_f2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  const uint4 u = make_uint4(pk_bf16_rne(a[0] * s, a[1] * s), pk_bf16_rne(b[0] * s, b[1] * s),
                             pk_bf16_rne(c[0] * s, c[1] * s), pk_bf16_rne(d[0] * s, d[1] * s));
  return __builtin_bit_cast(gv_bf8, u);
}

// The matrix instruction wants row n in lanes n, n + 16, n + 32, n + 48, while
// a load is cheapest where neighbouring lanes continue a cache line (a lane
// that starts a line of its own costs a cycle of the L1's address path, which
// was 85 % busy with rows in lanes).  So the words pass through 2 KB of the
// wave's own LDS: row r's 16-byte piece p goes to slot p ^ (r / 2 mod 8), which
// spreads 16 rows' same piece over all banks.  Lane group g takes pieces 2 g
// and 2 g + 1: k = 64 g .. 64 g + 63 of the chunk.
struct GvTurn {
  uint8_t *mine;
  int wr[2], rd;
  __device__ __forceinline__ GvTurn(uint8_t *m, int lane) : mine(m) {
    wr[0] = (lane >> 3) * 128 + 16 * ((lane & 7) ^ (lane >> 4));
    wr[1] = (lane >> 3) * 128 + 1024 + 16 * ((lane & 7) ^ ((lane >> 4) + 4));
    rd = (lane & 15) * 128 + 16 * ((2 * (lane >> 4)) ^ ((lane & 15) >> 1));
  }
  __device__ __forceinline__ void operator()(const gv_u4 (&in)[2], gv_u4 (&out)[2]) const {
    // one wave's LDS accesses keep their order: only the compiler is held
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    *reinterpret_cast<gv_u4 *>(mine + wr[0]) = in[0];
    *reinterpret_cast<gv_u4 *>(mine + wr[1]) = in[1];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    out[0] = *reinterpret_cast<const gv_u4 *>(mine + rd);
    out[1] = *reinterpret_cast<const gv_u4 *>(mine + (rd ^ 16));
  }
};

// A lane's part of a 256-wide chunk of a tile: eight rows a load, eight lanes
// each; of the scales a row's 16 bytes in four lanes.
struct GdChunk {
  gv_u4 q[2];
  uint32_t s;
};

}  // namespace

// Few workgroups: everything straight from memory to registers.  Of a
// workgroup's eight waves each takes one of two 16-row tiles (ACT: a gate tile
// and its up tile) and a quarter of the contraction in 256-wide chunks, so a
// chain is short: what bounds this kernel is latency (ids, weights, x, then
// the joining).  One decode step of top-8 of 128 experts, 2048 x 768, in a
// captured graph: gate_up 7.4 us, down 5.7, of which an empty launch is 1.6.
// Measured against 8.9 and 6.0 of this form (kernel durations): two tiles a wave
// 10.4 and 6.7; waiting for the rows before the first weights were asked for,
// 12; the next chunk's loads ahead of this one's products, 9.0 and 7.1 (the
// registers halve what a CU holds).
//
// WORDS: K % 64 == 0, so that a row of scales starts at a word; otherwise (any
// K % 32 == 0) it starts at any even byte and its words come in halves, which
// the compiler joins, and waits for, before the rows are known: 9.6 and 6.2.
template <bool ACT, bool OUTF32, bool WORDS>
__global__ __launch_bounds__(512, 4) void k_gemv_direct(GemvArgs a,
                                                        const int32_t *__restrict__ ids) {
  constexpr int KS = 4;
  constexpr int COLS = ACT ? 16 : 32;
  extern __shared__ uint16_t list[];  // the rows of this expert, in order
  __shared__ gv_f4 red[KS][2][64];
  __shared__ __align__(16) uint8_t turns[2 * KS][2048];
  __shared__ int cnt[2 * KS];
  const int lane = threadIdx.x & 63, g = lane >> 4, ln = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), kw = wave >> 1, t = wave & 1;
  const int id = gv_id(a, ids, threadIdx.x);
  const int e = gv_expert(a, ids);
  const int64_t n0 = (int64_t)blockIdx.x * COLS, NW = ACT ? 2 * a.N : a.N;
  const int cols = (int)min((int64_t)COLS, a.N - n0);
  const int K = (int)a.K, chunks = (K + 255) / 256;
  // The tile's weight rows as buffers: what lies past their end reads as 0.
  const int64_t r0 = (int64_t)(e < 0 ? 0 : e) * NW + n0 + (t ? (ACT ? a.N : 16) : 0);
  const int rows = ACT ? cols : max(0, min(16, cols - 16 * t));
  const __amdgpu_buffer_rsrc_t wq = gv_buffer(a.w + r0 * (K / 2), (int64_t)rows * (K / 2));
  const __amdgpu_buffer_rsrc_t ws = gv_buffer(a.ws + r0 * (K / 16), (int64_t)rows * (K / 16));
  const auto load = [&](GdChunk &b, int ch) {
    const uint32_t oq = ch < chunks ? ch * 128u : GV_NONE, os = ch < chunks ? ch * 16u : GV_NONE;
    const int vq = (int)((lane >> 3) * (uint32_t)(K / 2) + 16 * (lane & 7) + oq);
    const int vs = (int)((lane >> 2) * (uint32_t)(K / 16) + 4 * (lane & 3) + os);
    b.q[0] = __builtin_amdgcn_raw_buffer_load_b128(wq, vq, 0, 0);
    b.q[1] = __builtin_amdgcn_raw_buffer_load_b128(wq, vq + 8 * (K / 2), 0, 0);
    if constexpr (WORDS)
      b.s = __builtin_amdgcn_raw_buffer_load_b32(ws, vs, 0, 0);
    else
      b.s = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(ws, vs, 0, 0) |
            (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(ws, vs + 2, 0, 0) << 16;
  };
  // the first chunk's loads go out before the rows are known
  GdChunk b;
  const bool early = a.byrow && e >= 0;
  load(b, early ? kw : chunks);
  const float one = e >= 0 && a.rps == NW ? a.wo[e] : 0.0f;
  const int c = gv_rows<2 * KS>(a, ids, id, e, list, cnt);
  if (c == 0) return;
  if (e < 0) return gv_zero<OUTF32>(a, list, c, n0, cols);
  const GvTurn turn(turns[wave], lane);
  for (int m0 = 0; m0 < c; m0 += 16) {
    const int row = list[min(m0 + ln, c - 1)];
    const uint16_t *xr = a.x + (int64_t)(row / a.div) * K;
    const float pr = ACT ? a.prob[row] : 0.0f;
    const auto load_x = [&](uint4 (&x)[8], int ch) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = ch * 256 + 64 * g + 8 * j;
        x[j] = *reinterpret_cast<const uint4 *>(xr + min(k, K - 8));
        if (k >= K) x[j] = make_uint4(0, 0, 0, 0);
      }
    };
    gv_f4 acc = {0, 0, 0, 0};
    const auto multiply = [&](const GdChunk &b, const uint4 (&x)[8], int ch) {
      gv_u4 q[2];
      turn(b.q, q);
      int sw = __builtin_amdgcn_ds_bpermute(16 * ln + 4 * g, (int)b.s);
      // past the row's end stand the next row's scales, maybe NaN: x is 0 there,
      // the scale has to be so too
      const int left = K - 256 * ch - 64 * g;
      if (left < 64) sw = left == 32 ? sw & 0xFFFF : 0;
      const float f[4] = {__builtin_amdgcn_cvt_f32_fp8(sw, 0), __builtin_amdgcn_cvt_f32_fp8(sw, 1),
                          __builtin_amdgcn_cvt_f32_fp8(sw, 2), __builtin_amdgcn_cvt_f32_fp8(sw, 3)};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(gv_decode(q[j >> 2][j & 3], f[j >> 1]),
                                                      __builtin_bit_cast(gv_bf8, x[j]), acc, 0, 0, 0);
    };
    for (int ch = kw; ch < chunks; ch += KS) {
      if (!early || m0 > 0 || ch > kw) load(b, ch);
      uint4 x[8];
      load_x(x, ch);
      multiply(b, x, ch);
    }
    red[kw][t][lane] = acc;
    __syncthreads();
    if (wave < (ACT ? 1 : 2) && m0 + ln < c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t n = n0 + 16 * wave + 4 * g + i;
        if (n >= a.N) break;
        float v = red[0][wave][lane][i];
#pragma unroll
        for (int w = 1; w < KS; ++w) v += red[w][wave][lane][i];
        v *= a.rps == NW ? one : gv_outer(a, e, NW, n);
        if constexpr (ACT) {
          float u = red[0][1][lane][i];
#pragma unroll
          for (int w = 1; w < KS; ++w) u += red[w][1][lane][i];
          u *= a.rps == NW ? one : gv_outer(a, e, NW, a.N + n);
          v = swiglu_f32(v, u, pr);
        }
        gv_store<OUTF32>(a, (int64_t)row * a.N + n, v);
      }
    }
    __syncthreads();
  }
}

namespace {

constexpr int GS_KB = 512;              // k of a staged block
constexpr int GS_STR = GS_KB * 2 + 16;  // its row stride in LDS: 16 rows in distinct banks
constexpr int gs_cols(bool act) { return act ? 64 : 128; }  // output columns of a workgroup
__host__ __device__ constexpr int gs_list_bytes(int rows) { return (2 * rows + 15) / 16 * 16; }
constexpr int gs_lds(int rows) {
  return gs_list_bytes(rows) + 2 * 16 * GS_STR + 4 * (2048 + 2 * 1280);
}
static_assert(gs_lds(GEMV_MAX_ROWS) <= 65536, "LDS of a workgroup");

// Two tiles' part of a 256-wide chunk: eight rows a load, eight lanes each.
struct GvChunk {
  gv_u4 q[2][2];
};

}  // namespace

// Many workgroups: bandwidth counts.  Four waves, each two 16-row weight tiles
// (ACT: a gate tile and its up tile) and the whole contraction, two chunks of
// weights in flight in registers.  x is staged through LDS for the four, 512
// values a row at a time, one block ahead.
//
// It is staged as f16, since decoding the weights to f16 takes half the
// instructions of bf16 (a conversion and a packed multiply per two values).
// Each row is scaled by the power of two that brings its largest value so far
// to 2^14 .. 2^15; when a block raises that value, the sums move to the new
// power, exactly.  bf16 has 8 significant bits, so values down to 2^-31 of the
// largest stay exact; what smaller ones lose is below 2^-38 of the largest,
// 2^14 times less than what the binary32 sum may round.
//
// STREAM: the weights (not their scales) pass by the L2, which then keeps x for
// the workgroups of an expert: its fetches fall from 524 to 483 MB in the case
// below.  It loses where a workgroup reads its weights again for every 16 rows.
//
// Measured, 37 tokens x top-8 of 64 experts, 5120 x 1280: gate_up 472 MB in
// 90 us (5.2 TB/s; a copy here moves 5.1), 29 tokens: down 55 us.
// What made it so, gate_up: 174 us with a row of weights in each lane (see
// GvTurn); 150 -> 136 by waits that count loads (no load in a branch); 125
// after the scales' loads became whole lines; 111 without a pass that found
// each row's maximum first; 100 with four chunks' scales in one load; 90 with
// STREAM.  The rest is a short grid's last round and the start of each
// workgroup (ids, x).
template <bool ACT, bool OUTF32, bool STREAM>
__global__ __launch_bounds__(256, 3) void k_gemv_staged(GemvArgs a,
                                                        const int32_t *__restrict__ ids) {
  constexpr int COLS = gs_cols(ACT), OT = ACT ? 1 : 2;  // output columns; output tiles a wave
  extern __shared__ __align__(16) uint8_t lds[];  // the list, then x blocks [2][16][GS_STR]
  __shared__ int cnt[4];
  __shared__ int sexp[2][16];
  uint16_t *list = reinterpret_cast<uint16_t *>(lds);
  uint8_t *smem = lds + gs_list_bytes(a.rows);
  const int id = gv_id(a, ids, threadIdx.x), e = gv_expert(a, ids);
  const int c = gv_rows<4>(a, ids, id, e, list, cnt);
  if (c == 0) return;
  const int64_t n0 = (int64_t)blockIdx.x * COLS;
  const int cols = (int)min((int64_t)COLS, a.N - n0);
  if (e < 0) return gv_zero<OUTF32>(a, list, c, n0, cols);

  const int lane = threadIdx.x & 63, g = lane >> 4, ln = lane & 15;
  const int uw = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t NW = ACT ? 2 * a.N : a.N;
  const int K = (int)a.K, chunks = (K + 255) / 256, blocks = (K + GS_KB - 1) / GS_KB;
  // The workgroup's weight rows as buffers: what lies past their end reads as
  // 0; past the end of one row, x and the scales are made 0 at their use.
  const int64_t r0 = (int64_t)e * NW + n0;
  const __amdgpu_buffer_rsrc_t wq = gv_buffer(a.w + r0 * (K / 2), (int64_t)cols * (K / 2));
  const __amdgpu_buffer_rsrc_t ws = gv_buffer(a.ws + r0 * (K / 16), (int64_t)cols * (K / 16));
  const int64_t r1 = ACT ? r0 + a.N : r0;
  const __amdgpu_buffer_rsrc_t uq = gv_buffer(a.w + r1 * (K / 2), (int64_t)cols * (K / 2));
  const __amdgpu_buffer_rsrc_t us = gv_buffer(a.ws + r1 * (K / 16), (int64_t)cols * (K / 16));
  const uint32_t row0 = 16 * (uw * OT);
  const auto load = [&](GvChunk &b, int ch) {
    const uint32_t oq = ch < chunks ? ch * 128u : GV_NONE;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint32_t row = row0 + 16 * (t % OT);
      const int vq = (int)((row + (lane >> 3)) * (uint32_t)(K / 2) + 16 * (lane & 7) + oq);
      b.q[t][0] = __builtin_amdgcn_raw_buffer_load_b128(t < OT ? wq : uq, vq, 0, STREAM ? 2 : 0);
      b.q[t][1] = __builtin_amdgcn_raw_buffer_load_b128(t < OT ? wq : uq, vq + 8 * (K / 2), 0,
                                                        STREAM ? 2 : 0);
    }
  };
  // The scales of four chunks, 64 bytes of a row in four lanes.
  gv_u4 sv[2];
  const auto load_s = [&](int ch) {
    const uint32_t os = ch < chunks ? ch * 16u : GV_NONE;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint32_t row = row0 + 16 * (t % OT) + (lane >> 2);
      sv[t] = __builtin_amdgcn_raw_buffer_load_b128(
          t < OT ? ws : us, (int)(row * (uint32_t)(K / 16) + 16 * (lane & 3) + os), 0, 0);
    }
  };
  for (int m0 = 0; m0 < c; m0 += 16) {
    const int mr = min(16, c - m0);
    GvChunk b0, b1;
    load_s(0);
    load(b0, 0);
    load(b1, 1);
    // This wave's rows of x: uw, uw + 4, ...  They are staged as f16, each under
    // the power of two that brings the largest value of the row so far to
    // 2^14 .. 2^15; when that value grows, the sums move to the new power.
    __amdgpu_buffer_rsrc_t xr[4];
    int xe[4] = {127, 127, 127, 127};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = uw + 4 * i < mr;  // the others: empty buffers, read as 0
      const int row = __builtin_amdgcn_readfirstlane(list[m0 + (in ? uw + 4 * i : 0)]);
      xr[i] = gv_buffer(a.x + (int64_t)(row / a.div) * K, in ? 2 * K : 0);
    }
    const bool wide = mr > 4;  // more than one row a wave
    gv_u4 xs[4];
    const auto load_x = [&](int blk) {
      const int o = blk * (2 * GS_KB) + lane * 16;
      xs[0] = __builtin_amdgcn_raw_buffer_load_b128(xr[0], o, 0, 0);
      if (wide) {
#pragma unroll
        for (int i = 1; i < 4; ++i) xs[i] = __builtin_amdgcn_raw_buffer_load_b128(xr[i], o, 0, 0);
      }
    };
    const auto stage1 = [&](int buf, int i) {
      uint32_t m = xs[i][0] & 0x7FFF7FFFu;
#pragma unroll
      for (int j = 1; j < 4; ++j) m = pk_max_u16(m, xs[i][j] & 0x7FFF7FFFu);
      m = max(m & 0xFFFFu, m >> 16);
      m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));   // xor 1
      m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));   // xor 2
      m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));  // 7 - i
      m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, false));  // 15 - i
      const uint32_t top = max(max((uint32_t)__builtin_amdgcn_readlane((int)m, 0),
                                   (uint32_t)__builtin_amdgcn_readlane((int)m, 16)),
                               max((uint32_t)__builtin_amdgcn_readlane((int)m, 32),
                                   (uint32_t)__builtin_amdgcn_readlane((int)m, 48)));
      xe[i] = min(xe[i], 14 + 127 - (int)(top >> 7));
      const float f = __builtin_ldexpf(1.0f, xe[i]);
      gv_u4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(bf16_lo_f32(xs[i][j]) * f,
                                                                      bf16_hi_f32(xs[i][j]) * f));
      *reinterpret_cast<gv_u4 *>(smem + (buf * 16 + uw + 4 * i) * GS_STR + lane * 16) = o;
      if (lane == 0) sexp[buf][uw + 4 * i] = xe[i];
    };
    const auto stage = [&](int buf) {
      stage1(buf, 0);
      if (wide) {
#pragma unroll
        for (int i = 1; i < 4; ++i) stage1(buf, i);
      }
    };
    int se = 127;  // the power the sums of this lane's row are under
    gv_f4 acc[2] = {};
    uint8_t *mine = smem + 2 * 16 * GS_STR + uw * (2048 + 2 * 1280);
    uint8_t *mys = mine + 2048;  // scales: rows of 80 bytes, 64 of them used
    const GvTurn turn(mine, lane);
    const auto rescale = [&](int buf) {
      const int n = sexp[buf][min(ln, mr - 1)];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_ldexpf(acc[t][i], n - se);
      se = n;
    };
    const auto put_s = [&]() {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int t = 0; t < 2; ++t)
        *reinterpret_cast<gv_u4 *>(mys + (16 * t + (lane >> 2)) * 80 + 16 * (lane & 3)) = sv[t];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    // ch: the chunk's place in its block; sc: its place among the four whose
    // scales are in LDS; left: what the rows hold from it on
    const auto multiply = [&](const GvChunk &b, int buf, int ch, int sc, int left) {
      const uint8_t *xp = smem + (buf * 16 + min(ln, mr - 1)) * GS_STR + ch * 512 + g * 128;
      gv_h2 f[2][2];
      gv_u4 q[2][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        turn(b.q[t], q[t]);
        int sw = *reinterpret_cast<const int *>(mys + (16 * t + ln) * 80 + sc * 16 + 4 * g);
        if (64 * g >= left) sw = 0;  // the next row's, maybe NaN; x is 0 there
        f[t][0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sw, 1.0f, false);
        f[t][1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sw, 1.0f, true);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const gv_h8 x = *reinterpret_cast<const gv_h8 *>(xp + 16 * j);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t u = q[t][j >> 2][j & 3];
          const _Float16 sc = f[t][j >> 2][(j >> 1) & 1];
          const gv_h2 s2 = {sc, sc};
          const gv_h2 w0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.0f, 0) * s2;
          const gv_h2 w1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.0f, 1) * s2;
          const gv_h2 w2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.0f, 2) * s2;
          const gv_h2 w3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.0f, 3) * s2;
          const gv_h8 w = {w0[0], w0[1], w1[0], w1[1], w2[0], w2[1], w3[0], w3[1]};
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, x, acc[t], 0, 0, 0);
        }
      }
    };
    load_x(0);
    stage(0);
    // nothing in flight at the loop's entry, so that the waits in it count the
    // loads of its own turns alone
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
    const auto block = [&](int blk, int i) {
      load_x(blk + 1);
      rescale(i);
      multiply(b0, i, 0, 2 * i, K - 512 * blk);
      load(b0, 2 * blk + 2);
      if (2 * blk + 1 < chunks) multiply(b1, i, 1, 2 * i + 1, K - 512 * blk - 256);
      load(b1, 2 * blk + 3);
      stage(i ^ 1);
      __syncthreads();
    };
    // two blocks a turn: the scales of their four chunks come together
    for (int blk = 0;;) {
      put_s();
      load_s(2 * blk + 4);
      block(blk, 0);
      if (++blk >= blocks) break;
      block(blk, 1);
      if (++blk >= blocks) break;
    }
    if (ln < mr) {
      const int row = list[m0 + ln];
      const float back = __builtin_ldexpf(1.0f, -se);
      const int64_t o = (int64_t)row * a.N;
#pragma unroll
      for (int t = 0; t < OT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t n = n0 + 16 * (uw * OT + t) + 4 * g + i;
          if (n >= a.N) break;
          float v = acc[t][i] * back * gv_outer(a, e, NW, n);
          if constexpr (ACT) {
            const float u = acc[t + OT][i] * back * gv_outer(a, e, NW, a.N + n);
            v = swiglu_f32(v, u, a.prob[row]);
          }
          gv_store<OUTF32>(a, o + n, v);
        }
    }
    __syncthreads();
  }
}

namespace {

template <typename L>
hipError_t gv_launch(const GemvArgs &a, int per, int threads, int lds, L kernel,
                     const int32_t *ids, hipStream_t st) {
  const dim3 grid((unsigned)((a.N + per - 1) / per), (unsigned)(a.byrow ? a.rows : a.G + 1));
  hipLaunchKernelGGL(kernel, grid, dim3(threads), lds, st, a, ids);
  return hipGetLastError();
}

hipError_t launch_gemv(GemvArgs a, const int32_t *ids, bool act, bool f32, hipStream_t st) {
  // Fewer rows than experts: a workgroup row per row of ids.  Otherwise one
  // per expert, and one for the rows without an expert.
  a.byrow = a.rows < a.G;
  // The staged kernel from 160 workgroups on.  Its loads of scales need K % 64;
  // without it the direct kernel runs at any size (gate_up of 37 tokens, K =
  // 5088: 160 us, 5120: 92).
  // Measured, direct against staged: 96 workgroups 8.9 / 10.9 us, 128: 6.1 /
  // 7.6 and 12.8 / 16.3, 160: 22.5 / 21.3, 192: 12.4 / 11.6, 384: 21.9 / 15.4,
  // 1280: 133 / 85.
  const int64_t tiles = (a.N + gs_cols(act) - 1) / gs_cols(act);
  if (a.K % 64 == 0 && tiles * (a.byrow ? a.rows : a.G) >= 160) {
    // Streamed weights while an expert's rows are one pass of 16 on average.
    // Streamed against not, 2560 x 5120 gate_up (us), rows per expert 4.6:
    // 87.5 / 96.3, 8: 37.0 / 38.2, 12: 49.5 / 51.0, 16: 62.1 / 62.6, 24: 75.5 /
    // 75.2, 64: 115 / 113; 5120 x 1280 down, 16: 31.5 / 30.4, 64: 59.2 / 54.5.
    const bool stream = a.rows < 16 * (int64_t)a.G;
    const auto kernel = act   ? stream ? k_gemv_staged<true, false, true>
                                       : k_gemv_staged<true, false, false>
                        : f32 ? stream ? k_gemv_staged<false, true, true>
                                       : k_gemv_staged<false, true, false>
                        : stream ? k_gemv_staged<false, false, true>
                                 : k_gemv_staged<false, false, false>;
    return gv_launch(a, gs_cols(act), 256, gs_lds(a.rows), kernel, ids, st);
  }
  const int lds = 2 * a.rows;
  const bool w = a.K % 64 == 0;
  const auto kernel = act   ? w ? k_gemv_direct<true, false, true> : k_gemv_direct<true, false, false>
                      : f32 ? w ? k_gemv_direct<false, true, true> : k_gemv_direct<false, true, false>
                      : w   ? k_gemv_direct<false, false, true>
                            : k_gemv_direct<false, false, false>;
  return gv_launch(a, act ? 16 : 32, 512, lds, kernel, ids, st);
}

bool al(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
pqm_status st_of(hipError_t e) { return e == hipSuccess ? PQM_OK : PQM_ERR_HIP; }

pqm_status gemv_check(const GemvArgs &a, const int32_t *ids, int64_t rows, int64_t divisor, int64_t G, int64_t NW) {
  if (rows < 0 || rows > GEMV_MAX_ROWS || divisor < 1 || divisor > GEMV_MAX_ROWS || G < 1 ||
      G > 4096)
    return PQM_ERR_SHAPE;
  if (a.N < 0 || a.N > (1 << 20) || a.K < 32 || a.K > (1 << 20) || a.K % 32) return PQM_ERR_SHAPE;
  if (a.rps < 1 || (G * NW) % a.rps) return PQM_ERR_SHAPE;
  if (rows == 0 || a.N == 0) return PQM_OK;
  if (!a.x || !ids || !a.w || !a.ws || !a.wo || !a.out) return PQM_ERR_NULL;
  if (!al(a.x, 16) || !al(a.w, 16) || !al(a.out, 16) || !al(ids, 4) || !al(a.ws, 4) ||
      !al(a.wo, 4) || !al(a.prob, 4))
    return PQM_ERR_ALIGN;
  return PQM_OK;
}

}  // namespace
}  // namespace pqm

extern "C" {

pqm_status pqm_moe_gemv_nvfp4(const uint16_t *x, const int32_t *ids, int64_t rows, int64_t divisor,
                              const uint8_t *w_q, const uint8_t *w_scale, const float *w_outer,
                              int64_t w_rows_per_scale, int64_t G, int64_t N, int64_t K, void *out,
                              pqm_dtype out_dtype, hipStream_t stream) {
  using namespace pqm;
  if (out_dtype != PQM_OUT_BF16 && out_dtype != PQM_OUT_FP32) return PQM_ERR_ENUM;
  const GemvArgs a = {x, (int)rows, (int)divisor, w_q, w_scale, w_outer, w_rows_per_scale,
                      (int)G, N, K, nullptr, out, 0};
  const pqm_status bad = gemv_check(a, ids, rows, divisor, G, N);
  if (bad != PQM_OK || rows == 0 || N == 0) return bad;
  return st_of(launch_gemv(a, ids, false, out_dtype == PQM_OUT_FP32, stream));
}

pqm_status pqm_moe_gemv_swiglu_nvfp4(const uint16_t *x, const int32_t *ids, const float *prob,
                                     int64_t rows, int64_t divisor, const uint8_t *w_q,
                                     const uint8_t *w_scale, const float *w_outer,
                                     int64_t w_rows_per_scale, int64_t G, int64_t inter, int64_t K,
                                     uint16_t *d, hipStream_t stream) {
  using namespace pqm;
  const GemvArgs a = {x, (int)rows, (int)divisor, w_q, w_scale, w_outer, w_rows_per_scale,
                      (int)G, inter, K, prob, d, 0};
  const pqm_status bad = gemv_check(a, ids, rows, divisor, G, 2 * inter);
  if (bad != PQM_OK || rows == 0 || inter == 0) return bad;
  if (!prob) return PQM_ERR_NULL;
  return st_of(launch_gemv(a, ids, true, false, stream));
}

}  // extern "C"
