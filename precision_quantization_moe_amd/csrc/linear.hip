// linear.hip -- dense bf16 products with their epilogue, and their gradients.
//
//   z = x W^T + bias,  y = act(z) + residual      x [M, K], W [N, K]
//   dz = dy act'(z),   dx = dz W + d_x,  dW = dz^T x,  dbias = sum of dz's rows
//
// All three products are C[i, j] = sum_k A(i, k) B(j, k) with each operand
// either "KL" (the contraction contiguous in memory: x, W, dz of the first
// two) or "ML" (contraction rows, the outputs contiguous: W of dx, both of
// dW).  act(z) = z / (1 + e^-s(z)), s(z) = z (SiLU) or 2 sqrt(2/pi)
// (z + 0.044715 z^3) (GELU with its tanh, since (1 + tanh u) / 2 is the
// sigmoid of 2 u).  Sums are binary32; y, z, dx and dz are rounded once.
#include "norm_device.hpp"
#include "pqm_device.hpp"
#include "pqm_internal.hpp"
#include "pqmoe.h"

namespace pqm {

namespace {

typedef __bf16 ln_bf8 __attribute__((ext_vector_type(8)));
typedef float ln_f4 __attribute__((ext_vector_type(4)));
typedef float ln_f16 __attribute__((ext_vector_type(16)));
typedef uint32_t ln_u4 __attribute__((ext_vector_type(4)));
typedef uint32_t ln_u2 __attribute__((ext_vector_type(2)));
typedef short ln_v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) ln_v4s ln_lds_v4s;

constexpr uint32_t LN_NONE = 0x80000000u;  // an offset past every buffer below: reads give 0
constexpr int64_t LN_MAX = 1 << 22;        // row strides: 256 rows of 2-byte values stay below 2^31
constexpr int LN_FEW = 64;                 // rows of the few-row kernel
constexpr int64_t LN_SHARE = 4096;         // outputs from which its tiles share

__device__ __forceinline__ __amdgpu_buffer_rsrc_t ln_buffer(const void *p, int64_t bytes) {
  const int n = (int)(bytes < 0 ? 0 : bytes > 0x7FFFFFFF ? 0x7FFFFFFF : bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, n, 0x00020000);
}

// ---------------------------------------------------------------- epilogue

struct LnEpi {
  const float *bias;
  const uint16_t *res;
  int64_t ldr;
  void *y;
  uint16_t *z;
  int64_t N;
  int act, f32;
  int vec;  // rows of y, z and res hold whole, aligned groups of eight
  int stream;  // 1: bf16 outputs go past the caches; 2: the residual too
};

// -s(z) log2(e) of the activation, times `of`.
__device__ __forceinline__ float ln_squash(float z, int act, float of = 1.0f) {
  constexpr float G = 1.5957691216057308f;  // 2 sqrt(2 / pi)
  const float L = of * 1.4426950408889634f;
  return act == PQM_ACT_SILU ? -L * z : z * __builtin_fmaf(z * z, -L * G * 0.044715f, -L * G);
}
// z / (1 + e^-s) as (z 2^-15) / (2^-15 + 2^-15 h h) with h = e^(-s / 2): z e^s is a value
// of bf16 where e^-s has left binary32 (SiLU of -88: -5.3e-37), so the reciprocal takes
// up to 2^141; where that is too much, the value rounds to 0.  The plain form, 0 from 2^126
// on, takes 162.8 us for 8190 x 4096 x 2048, this one 164.1, a branch for the far values
// 168.5.  A z below 2^-111 loses bits below 2^-135.
__device__ __forceinline__ float ln_act(float z, int act) {
  if (act == PQM_ACT_NONE) return z;
  const float h = __builtin_amdgcn_exp2f(ln_squash(z, act, 0.5f));
  return z * 0x1p-15f * __builtin_amdgcn_rcpf(__builtin_fmaf(h * 0x1p-15f, h, 0x1p-15f));
}
// act'(z) = v + z v (1 - v) s'(z) with v the sigmoid of s; v (1 - v) is even in
// s, so it is formed with e^-|s|, which cannot overflow.
__device__ __attribute__((noinline)) float ln_dz_near(float g, float z, int act) {
  constexpr double G = 1.5957691216057307;  // 2 sqrt(2 / pi)
  const double x = z, s = act == PQM_ACT_SILU ? x : G * (x + 0.044715 * x * x * x);
  const double ds = act == PQM_ACT_SILU ? 1.0 : G * (1.0 + 0.134145 * x * x);
  const double t = exp(-__builtin_fabs(s)), r = 1.0 / (1.0 + t);
  const double v = s < 0.0 ? t * r : r, w = t * r * r;
  return before_bf16((double)g * (w == 0.0 ? v : v + x * ds * w));
}
// g act'(z), to be rounded to bf16: the nearest value.  dW and dbias keep binary32 sums
// of it, in which one step of bf16 to the wrong side shows where there are few rows; so
// a binary32 value within its own error of the middle of two is formed again in binary64.
__device__ __forceinline__ float ln_dz(float g, float z, int act) {
  const float s = ln_squash(z, act);
  const float ds = act == PQM_ACT_SILU
                       ? 1.0f
                       : __builtin_fmaf(z * z, 1.5957691216057308f * 0.134145f, 1.5957691216057308f);
  const float t = __builtin_amdgcn_exp2f(-fabsf(s)), r = __builtin_amdgcn_rcpf(1.0f + t);
  const float v = s > 0.0f ? t * r : r, w = t * r * r;
  // far out w is 0 and z ds may be infinite
  const float a = w == 0.0f && s == s ? 0.0f : z * ds * w, d = g * (v + a);
  // half steps (2^-24): three of the argument times ln 2 |s|; two of the exponential; two
  // of the reciprocal, twice, and of 1 + t; the products and the sum
  const float e = fabsf(g) * (v + fabsf(a)) *
                  __builtin_fmaf(fminf(fabsf(s), 256.0f), 2.125f * 0x1p-24f, 14.0f * 0x1p-24f);
  const uint32_t both = pk_bf16_rne(d - e, d + e);
  // s over 99: e^-s is about to leave binary32, z s'(z) times it need not
  if (((both ^ (both >> 16)) & 0xFFFFu) || s > 99.0f) return ln_dz_near(g, z, act);
  return d;
}

// The output of row r, column c.
__device__ __forceinline__ void ln_put1(const LnEpi &e, int64_t r, int64_t c, float v) {
  const int64_t at = r * e.N + c;
  if (e.bias) v += e.bias[c];
  if (e.z) e.z[at] = (uint16_t)pk_bf16_rne(v, 0.0f);
  v = ln_act(v, e.act);
  if (e.res) v += bf16_lo_f32(e.res[r * e.ldr + c]);
  if (e.f32)
    static_cast<float *>(e.y)[at] = v;
  else
    static_cast<uint16_t *>(e.y)[at] = (uint16_t)pk_bf16_rne(v, 0.0f);
}

// Keeps a streaming access from being joined with the plain one of the other branch,
// which makes both plain.
#define LN_APART asm volatile("")

// Eight neighbouring outputs of row r from column c on, where rows hold whole,
// aligned groups of eight (e.vec); q, b: ln_res8 and ln_bias8 of them, which their
// callers ask for early.  ACT: whether there may be an activation; gradients have none,
// and without its code theirs of 8190 x 4096 x 2048 take 334 us, with it 343.
__device__ __forceinline__ ln_u4 ln_res8(const LnEpi &e, int64_t r, int64_t c) {
  if (!e.res) return ln_u4{0, 0, 0, 0};
  const ln_u4 *p = reinterpret_cast<const ln_u4 *>(e.res + r * e.ldr + c);
  if (e.stream < 2) return *p;
  LN_APART;
  const ln_u4 q = __builtin_nontemporal_load(p);
  LN_APART;
  return q;
}
__device__ __forceinline__ void ln_store8(const LnEpi &e, uint16_t *to, const ln_u4 &o) {
  if (e.stream) {
    LN_APART;
    __builtin_nontemporal_store(o, reinterpret_cast<ln_u4 *>(to));
    LN_APART;
  } else {
    *reinterpret_cast<ln_u4 *>(to) = o;
  }
}
__device__ __forceinline__ void ln_bias8(const LnEpi &e, int64_t c, float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = e.bias ? e.bias[c + i] : 0.0f;
}
template <bool ACT>
__device__ __forceinline__ void ln_put8(const LnEpi &e, int64_t r, int64_t c, float (&v)[8],
                                        const ln_u4 &q, const float (&b)[8]) {
  const int64_t at = r * e.N + c;
  if (e.bias) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  if (e.z) {
    const ln_u4 o = {pk_bf16_rne(v[0], v[1]), pk_bf16_rne(v[2], v[3]), pk_bf16_rne(v[4], v[5]),
                     pk_bf16_rne(v[6], v[7])};
    ln_store8(e, e.z + at, o);
  }
  if (ACT && e.act != PQM_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = ln_act(v[i], e.act);
  }
  if (e.res) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] += bf16_lo_f32(q[i]);
      v[2 * i + 1] += bf16_hi_f32(q[i]);
    }
  }
  if (e.f32) {
    ln_f4 *o = reinterpret_cast<ln_f4 *>(static_cast<float *>(e.y) + at);
    o[0] = ln_f4{v[0], v[1], v[2], v[3]};
    o[1] = ln_f4{v[4], v[5], v[6], v[7]};
  } else {
    const ln_u4 o = {pk_bf16_rne(v[0], v[1]), pk_bf16_rne(v[2], v[3]), pk_bf16_rne(v[4], v[5]),
                     pk_bf16_rne(v[6], v[7])};
    ln_store8(e, static_cast<uint16_t *>(e.y) + at, o);
  }
}

// ------------------------------------------------------------ tile products
//
// Four waves, 2 x 2, a tile; operands by DMA into a ring of LDS slots of 32 of the
// contraction, fragments read one step ahead.  256 x 256: a wave's 128 x 128 outputs
// take half the LDS bytes of 128 x 128 tiles a product, at one workgroup a CU.
// 8190 x 4096 x 2048 with GELU, bias, residual and z kept 164 us (the product alone by
// the library 111): the steps 131 (1050 TFLOP/s) and two epilogues of 16, in which all
// CUs move their 384 KB of residual, y and z at once and multiply nothing.  The matrix
// cores are busy 36 % of its cycles, 46 % without the epilogue (141 us), where a wave
// waits for loads or the barrier 21 % of its time and no LDS access meets a conflict.
// dx of the same layer takes 126 to 137 (library 120), dW 151 to 160 (174).  The router,
// 16384 x 128 x 2048, 22.6 us: 75 MB at 3.3 TB/s, which is what its 128 workgroups, on
// half of the CUs, draw; its dx 36, 138 MB.

enum { LN_NT = 0, LN_NN = 1, LN_TN = 2 };  // y; dx (B is ML); dW (both are ML)

struct LnTile {
  const uint16_t *a, *b;
  int64_t lda, ldb;   // row strides in elements
  int64_t I, J, K;    // output rows, output columns, contraction
  int64_t part;       // contraction of one split, a multiple of 32
  int mt, nt;         // tiles
  float *partial;     // [splits][I][J] when the contraction is split
};

template <int TM_, int TN_, int NS_>
struct Ln {
  static constexpr int TM = TM_, TN = TN_, NS = NS_;
  static constexpr int SLOT = (TM + TN) * 64, RING = NS * SLOT;
  static constexpr int FI = TM / 64, FJ = TN / 64;  // 32-wide fragments of a wave (2 x 2 waves)
  static constexpr int CA = TM / 64, CB = TN / 64, OPS = CA + CB;
  static constexpr int PITCH = TN / 2 * 4 + 16;     // epilogue: a wave's 32 rows of its columns
  static constexpr int LDS = RING > 4 * 32 * PITCH ? RING : 4 * 32 * PITCH;
};

template <int n>
__device__ __forceinline__ void ln_vm_wait() {
  __builtin_amdgcn_s_waitcnt((n & 0xF) | ((n >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
__device__ __forceinline__ void ln_lgkm_wait0() { __builtin_amdgcn_s_waitcnt(0xC07F); }

// The swizzle of contraction row r of an ML tile W outputs wide, in units of
// 64 bytes: the rows that one transposing read touches go to different banks.
template <int W>
__device__ __forceinline__ int ln_swz(int r) {
  return W >= 256 ? (r & 3) | (((r >> 3) & 1) << 2) : (r & 3);
}

// One operand's loads.  A lane's 16-byte chunk c of a step is row c / 4, piece
// c % 4 (KL) or contraction row c / (W / 8), piece c % (W / 8) (ML); it goes to
// LDS byte 16 c, so the swizzle is in where it comes from.  What lies past the
// operand's end reads as 0: rows and, of an ML operand, contraction past the end of
// the buffer; a KL operand's contraction past its end by an offset past the buffer.
template <int W, bool ML>
struct LnSrc {
  const uint8_t *base;    // of the next step to load
  int64_t step;           // base's way per step, bytes
  int left;               // contraction left from base on
  int rows, ld2;          // KL: bytes to the end of the last row's start; ML: of a row used
  uint32_t off[W / 64];
  int piece;              // KL: the lane's piece of a step

  __device__ __forceinline__ void init(const uint16_t *p, int64_t ld, int64_t first, int64_t lines,
                                       int64_t k0, int64_t K) {
    const int tid = threadIdx.x;
    const int n = (int)min((int64_t)W, lines - first);
    left = (int)(K - k0);
    ld2 = (int)ld * 2;
    if (ML) {  // lines: outputs; first: the first of them
      base = reinterpret_cast<const uint8_t *>(p + k0 * ld + first);
      step = 64 * ld;
      rows = 2 * n;
      piece = 0;
#pragma unroll
      for (int i = 0; i < W / 64; ++i) {
        const int c = tid + 256 * i, r = c / (W / 8), x = (c % (W / 8)) ^ (4 * ln_swz<W>(r));
        off[i] = (uint32_t)(r * ld2 + 16 * x);
      }
    } else {
      base = reinterpret_cast<const uint8_t *>(p + first * ld + k0);
      step = 64;
      rows = (n - 1) * ld2;
      piece = 8 * ((tid & 3) ^ ((tid >> 4) & 3));
#pragma unroll
      for (int i = 0; i < W / 64; ++i)
        off[i] = (uint32_t)(((tid >> 2) + 64 * i) * ld2 + 2 * piece);
    }
  }
  // Chunk i of the next step to LDS address m0 (the wave's).
  __device__ __forceinline__ void load(int i, uint32_t m0) const {
    const int l = min(left, 32), bytes = ML ? (l - 1) * ld2 + rows : rows + 2 * min(left, 32);
    const uint32_t o = ML || piece < left ? off[i] : LN_NONE;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), (short)0,
                                          left > 0 ? bytes : 0, 0x00020000),
        (__attribute__((address_space(3))) void *)(uintptr_t)m0, 16, (int)o, 0, 0, 0);
  }
  __device__ __forceinline__ void next() {
    base += step;
    left -= 32;
  }
};

template <int TM, int TN>
struct LnFrags {
  ln_u4 a[TM / 64][2], b[TN / 64][2];  // [fragment][16-wide half of the step]
};

// A fragment of 32 outputs (32x32x16: lane l holds output l % 32, contraction
// 8 (l / 32) .. + 7 of the half).  KL: two plain reads.  ML: the transposing read
// gives lane i of a group of 16, as its element e, element i % 4 of the 8
// bytes that lane 4 e + i / 4 addresses; so lanes 16 q + j address row
// 8 (q / 2) + j / 4 (+ 4 for the second read), outputs 16 (q % 2) + 4 (j % 4).
template <int W, bool ML>
__device__ __forceinline__ void ln_read(const uint8_t *reg, int first, ln_u4 (&f)[2]) {
  const int lane = threadIdx.x & 63;
  if constexpr (ML) {
    const int q = lane >> 4, j = lane & 15, r = 8 * (q >> 1) + (j >> 2);
    const int out = 2 * (first + 16 * (q & 1) + 4 * (j & 3));
    const uint8_t *p = reg + r * (2 * W) + (out ^ (64 * ln_swz<W>(r)));
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const ln_u2 lo = __builtin_bit_cast(
          ln_u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                     (ln_lds_v4s *)(const_cast<uint8_t *>(p + (16 * s) * (2 * W)))));
      const ln_u2 hi = __builtin_bit_cast(
          ln_u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                     (ln_lds_v4s *)(const_cast<uint8_t *>(p + (16 * s + 4) * (2 * W)))));
      f[s] = ln_u4{lo[0], lo[1], hi[0], hi[1]};
    }
  } else {
    const int r = first + (lane & 31), x = (r >> 2) & 3, h = lane >> 5;
    f[0] = *reinterpret_cast<const ln_u4 *>(reg + r * 64 + 16 * (h ^ x));
    f[1] = *reinterpret_cast<const ln_u4 *>(reg + r * 64 + 16 * ((2 + h) ^ x));
  }
}

}  // namespace

template <int KIND, int TM, int TN, int NS>
__global__ __launch_bounds__(256, NS * (TM + TN) * 64 > 81920 ? 1 : 2) void k_linear(LnTile t,
                                                                                  LnEpi e) {
  using C = Ln<TM, TN, NS>;
  constexpr bool AM = KIND == LN_TN, BM = KIND != LN_NT;
  constexpr int FI = C::FI, FJ = C::FJ;
  __shared__ __align__(16) uint8_t lds[C::LDS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave >> 1, wn = wave & 1;

  // Workgroup b runs on XCD b % 8: each XCD gets a run of tiles, eight tile
  // rows at a time, so that its L2 serves both operands' panels.
  const int tiles = t.mt * t.nt, all = gridDim.x;
  const int per = (all + 7) / 8, full = all - 8 * (per - 1);  // the first `full` XCDs hold per
  const int x = blockIdx.x & 7;
  const int T = x * per - max(0, x - full) + (int)(blockIdx.x >> 3);
  const int split = T / tiles, u = T - split * tiles;
  const int band = u / (8 * t.nt), rows8 = min(8, t.mt - 8 * band), v = u - band * 8 * t.nt;
  const int64_t i0 = (int64_t)(8 * band + v % rows8) * TM, j0 = (int64_t)(v / rows8) * TN;
  const int64_t k0 = split * t.part, k1 = min(t.K, k0 + t.part);

  LnSrc<TM, AM> A;
  LnSrc<TN, BM> B;
  A.init(t.a, t.lda, i0, t.I, k0, k1);
  B.init(t.b, t.ldb, j0, t.J, k0, k1);
  const uint32_t dst =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds + (uint32_t)wave * 1024u);
  const auto load = [&](int slot, int q) {
    const uint32_t m0 = dst + slot * C::SLOT;
    if (q < C::CA) A.load(q, m0 + q * 4096);
    else B.load(q - C::CA, m0 + TM * 64 + (q - C::CA) * 4096);
    if (q == C::CA - 1) A.next();
    if (q == C::OPS - 1) B.next();
  };
  const auto read_a = [&](int slot, int f, LnFrags<TM, TN> &F) {
    ln_read<TM, AM>(lds + slot * C::SLOT, wm * (TM / 2) + 32 * f, F.a[f]);
  };
  const auto read_b = [&](int slot, int f, LnFrags<TM, TN> &F) {
    ln_read<TN, BM>(lds + slot * C::SLOT + TM * 64, wn * (TN / 2) + 32 * f, F.b[f]);
  };

  ln_f16 acc[FI][FJ];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  const int nk = (int)((k1 - k0 + 31) / 32);
#pragma unroll 1  // code that runs once waits for its own instructions
  for (int s = 0; s < C::NS; ++s)
#pragma unroll
    for (int q = 0; q < C::OPS; ++q) load(s, q);
  LnFrags<TM, TN> F0, F1;
  ln_vm_wait<(C::NS - 1) * C::OPS>();
  __builtin_amdgcn_s_barrier();
#pragma unroll
  for (int f = 0; f < FI; ++f) read_a(0, f, F0);
#pragma unroll
  for (int f = 0; f < FJ; ++f) read_b(0, f, F0);

  // A step: its fragments are in registers; after each matrix instruction comes a
  // slice of the other work: the fragments of the next step, and the loads of the step
  // NS ahead into the slot that every wave has left.
  const auto step = [&](int slot, const LnFrags<TM, TN> &cur, LnFrags<TM, TN> &next) {
    ln_vm_wait<(C::NS - 2) * C::OPS>();  // the next step has landed
    ln_lgkm_wait0();
    __builtin_amdgcn_s_barrier();
    const int after = slot == C::NS - 1 ? 0 : slot + 1;
    constexpr int NM = 2 * FI * FJ, NW = C::OPS + FI + FJ, PER = (NW + NM - 1) / NM;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const int s = m / (FI * FJ), j = (m / FI) % FJ, i = m % FI;
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          __builtin_bit_cast(ln_bf8, cur.b[j][s]), __builtin_bit_cast(ln_bf8, cur.a[i][s]),
          acc[i][j], 0, 0, 0);
#pragma unroll
      for (int w = m * PER; w < (m + 1) * PER && w < NW; ++w) {
        // the next fragments first: the next step waits for them
        if (w < FI) read_a(after, w, next);
        else if (w < FI + FJ) read_b(after, w - FI, next);
        else load(slot, w - FI - FJ);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int slot = 0;
  for (int kt = 0; kt < nk; kt += 2) {
    step(slot, F0, F1);
    slot = slot == C::NS - 1 ? 0 : slot + 1;
    step(slot, F1, F0);  // past the end it multiplies zeros
    slot = slot == C::NS - 1 ? 0 : slot + 1;
  }
  ln_vm_wait<0>();  // no load may still target the LDS that the epilogue uses
  __syncthreads();

  // A lane holds row l % 32, columns 8 (i / 4) + 4 (l / 32) + i % 4: through LDS,
  // 32 rows of the wave at a time, so that rows leave as whole lines.
  uint8_t *mine = lds + wave * 32 * C::PITCH;
  constexpr int LPR = TN / 2 / 8, RPI = 64 / LPR, NR = 32 / RPI;  // lanes a row, rows a turn, turns
  const int64_t col = j0 + wn * (TN / 2) + 8 * (lane % LPR);
  const float *p = reinterpret_cast<const float *>(mine + lane / LPR * C::PITCH) + 8 * (lane % LPR);
  const bool vec = t.partial ? t.J % 8 == 0 : e.vec;
  float bias[8];
  if (vec && !t.partial) ln_bias8(e, min(col, t.J - 8), bias);
#pragma unroll
  for (int i = 0; i < FI; ++i) {
    const int64_t row = i0 + wm * (TM / 2) + 32 * i + lane / LPR;  // of the first turn
    ln_u4 res[NR];
    if (vec && !t.partial) {  // all 32 rows' residual at once
#pragma unroll
      for (int r = 0; r < NR; ++r)
        res[r] = ln_res8(e, min(row + r * RPI, t.I - 1), min(col, t.J - 8));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<ln_f4 *>(mine + (lane & 31) * C::PITCH + 4 * (32 * j + 8 * q) +
                                   16 * (lane >> 5)) =
            ln_f4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                  acc[i][j][4 * q + 3]};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (vec) {
      float *w = t.partial + (split * t.I + row) * t.J + col;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const ln_f4 *o = reinterpret_cast<const ln_f4 *>(p + r * RPI * (C::PITCH / 4));
        const ln_f4 lo = o[0], hi = o[1];
        if (row + r * RPI >= t.I || col >= t.J) continue;
        if (t.partial) {
          ln_f4 *to = reinterpret_cast<ln_f4 *>(w + r * RPI * t.J);
          to[0] = lo;
          to[1] = hi;
        } else {
          float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          ln_put8<KIND == LN_NT>(e, row + r * RPI, col, v, res[r], bias);
        }
      }
    } else {
      // one output at a time: 8190 x 4095 x 2048 203 us where 4096 outputs take 141, with
      // an activation, bias, residual and z 402 and 168
      const int n = (int)min((int64_t)8, t.J - col);
#pragma unroll 1
      for (int r = 0; r < NR && row + r * RPI < t.I; ++r)
#pragma unroll 1
        for (int c = 0; c < n; ++c) {
          const float v = p[r * RPI * (C::PITCH / 4) + c];
          if (t.partial) t.partial[(split * t.I + row + r * RPI) * t.J + col + c] = v;
          else ln_put1(e, row + r * RPI, col + c, v);
        }
    }
  }
}

// The splits' sums in order, and the epilogue: eight outputs a thread.
__global__ __launch_bounds__(256) void k_linear_join(const float *__restrict__ partial, int splits,
                                                     int64_t I, int64_t J, LnEpi e) {
  const int64_t groups = (J + 7) / 8;
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < I * groups;
       g += (int64_t)gridDim.x * 256) {
    const int64_t row = g / groups, col = 8 * (g - row * groups);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const float *p = partial + row * J + col;
    const int64_t step = I * J;
    ln_u4 res = {0, 0, 0, 0};
    float bias[8];
    if (e.vec) {
      res = ln_res8(e, row, col);
      ln_bias8(e, col, bias);
    }
    if (J % 8 == 0) {
#pragma unroll 4
      for (int s = 0; s < splits; ++s) {
        const ln_f4 lo = *reinterpret_cast<const ln_f4 *>(p + s * step);
        const ln_f4 hi = *reinterpret_cast<const ln_f4 *>(p + s * step + 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          v[c] += lo[c];
          v[4 + c] += hi[c];
        }
      }
    } else {
      for (int s = 0; s < splits; ++s)
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (col + c < J) v[c] += p[s * step + c];
    }
    if (e.vec) {
      ln_put8<true>(e, row, col, v, res, bias);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (col + c < J) ln_put1(e, row, col + c, v[c]);
    }
  }
}

// ------------------------------------------------------------- few rows
//
// Up to 64 rows of x: what counts is reading W once.  A wave multiplies NT tiles of
// 16 rows of W, straight from memory to registers, by MT tiles of 16 rows of x with a
// 16x16x32 matrix instruction; ks of a workgroup's waves share a contraction and are
// joined through LDS.  Bound by memory (8 rows to 32768 outputs of 2048: 134 MB in
// 29.9 us, 4.5 TB/s) and from 32 rows on by the L1, which brings x to every wave.
// Every load of a turn goes out before the first is used; a streaming hint costs a
// tenth, since two loads share a line.
template <int MT, int NT>
__global__ __launch_bounds__(512, 4) void k_linear_few(const uint16_t *__restrict__ x, int64_t ldx,
                                                       const uint16_t *__restrict__ w, int64_t M,
                                                       int64_t K, int ks, LnEpi e) {
  __shared__ ln_f4 red[8][MT * NT][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, ln = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = wave % ks, tile = wave / ks;
  const int64_t n0 = ((int64_t)blockIdx.x * (8 / ks) + tile) * (16 * NT);
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  const __amdgpu_buffer_rsrc_t wb = ln_buffer(w + n0 * K, min((int64_t)16 * NT, e.N - n0) * K * 2);
  const int rows = (int)min((int64_t)16 * MT, M - m0);
  const __amdgpu_buffer_rsrc_t xb = ln_buffer(x + m0 * ldx, ((rows - 1) * ldx + K) * 2);
  uint32_t wo[NT], xo[MT];
#pragma unroll
  for (int t = 0; t < NT; ++t) wo[t] = (uint32_t)((16 * t + ln) * K + 8 * g) * 2;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = 16 * m + ln;
    xo[m] = r < rows ? (uint32_t)(r * ldx + 8 * g) * 2 : LN_NONE;
  }
  ln_f4 acc[MT][NT] = {};
  constexpr int U = MT == 1 ? 8 / NT : MT == 2 ? 4 : MT == 3 ? 3 : 2;  // steps of 32 in flight
  const int steps = (int)((K + 31) / 32), each = (steps + ks - 1) / ks;
  const int s1 = min(steps, (kw + 1) * each);
  for (int s = kw * each; s < s1; s += U) {
    ln_u4 wv[U][NT], xv[U][MT];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t none = s + i < s1 && 32 * (s + i) + 8 * g < K ? 0 : LN_NONE;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        wv[i][t] = __builtin_amdgcn_raw_buffer_load_b128(wb, (int)((wo[t] + 64 * (s + i)) | none),
                                                         0, 0);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        xv[i][m] = __builtin_amdgcn_raw_buffer_load_b128(xb, (int)((xo[m] + 64 * (s + i)) | none),
                                                         0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(ln_bf8, wv[i][t]), __builtin_bit_cast(ln_bf8, xv[i][m]),
              acc[m][t], 0, 0, 0);
  }
  if (ks > 1) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) red[wave][m * NT + t][lane] = acc[m][t];
    __syncthreads();
    if (kw > 0) return;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        for (int s = 1; s < ks; ++s) acc[m][t] += red[wave + s][m * NT + t][lane];
  }
  // lane: row 16 m + l % 16 of x, outputs n0 + 16 t + 4 (l / 16) ..: joined in pairs of
  // lane groups to eight neighbouring outputs
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t col = n0 + 16 * t + 4 * g;
    float bias[8] = {};
    if (e.vec && col + 8 <= e.N) ln_bias8(e, col, bias);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = acc[m][t][i];
        v[4 + i] = __shfl_down(acc[m][t][i], 16, 64);
      }
      const int64_t row = m0 + 16 * m + ln;
      if ((g & 1) || row >= M || col >= e.N) continue;
      if (e.vec) {
        ln_put8<true>(e, row, col, v, ln_res8(e, row, col), bias);
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (col + c < e.N) ln_put1(e, row, col + c, v[c]);
      }
    }
  }
}

// ------------------------------------------------- dz and the bias gradient

constexpr int LZ_ROWS = 32;  // rows of a workgroup's partial sums

// dz = bf16(dy act'(z)) (act none: dy itself, not written) and, per LZ_ROWS
// rows, the column sums of dz.  A thread takes eight columns of every 256 / CT-th
// row, four rows asked for at once; CT threads a row, as many as fill it.  Bound by
// memory and by the values formed again: 8190 x 4096 in 54 us (201 MB, 40 at a copy's
// rate and without them).
template <int CT>
__global__ __launch_bounds__(256) void k_linear_dz(const uint16_t *__restrict__ dy, int64_t lddy,
                                                   const uint16_t *z, int act, int64_t M,
                                                   int64_t N, uint16_t *dz,
                                                   float *__restrict__ sums) {
  constexpr int RT = 256 / CT, NR = LZ_ROWS / RT, NB = NR < 4 ? NR : 4;
  __shared__ float part[RT][CT][9];
  const int c8 = threadIdx.x % CT, q = threadIdx.x / CT;
  const int64_t col = ((int64_t)blockIdx.y * CT + c8) * 8;
  const int64_t r0 = (int64_t)blockIdx.x * LZ_ROWS + q;
  float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
  for (int h = 0; h < NR; h += NB) {
    ln_u4 d[NB], zz[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int64_t r = r0 + (h + i) * RT;
      const bool in = col < N && r < M;
      d[i] = zz[i] = ln_u4{0, 0, 0, 0};
      if (in) d[i] = *reinterpret_cast<const ln_u4 *>(dy + r * lddy + col);
      if (in && act != PQM_ACT_NONE) zz[i] = *reinterpret_cast<const ln_u4 *>(z + r * N + col);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int64_t r = r0 + (h + i) * RT;
      if (act != PQM_ACT_NONE) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          d[i][j] = pk_bf16_rne(ln_dz(bf16_lo_f32(d[i][j]), bf16_lo_f32(zz[i][j]), act),
                                ln_dz(bf16_hi_f32(d[i][j]), bf16_hi_f32(zz[i][j]), act));
        if (col < N && r < M) *reinterpret_cast<ln_u4 *>(dz + r * N + col) = d[i];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[2 * j] += bf16_lo_f32(d[i][j]);
        s[2 * j + 1] += bf16_hi_f32(d[i][j]);
      }
    }
  }
  if (!sums) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) part[q][c8][j] = s[j];
  __syncthreads();
  for (int c = threadIdx.x; c < 8 * CT; c += 256) {
    const int64_t at = (int64_t)blockIdx.y * CT * 8 + c;
    float v = 0.0f;
#pragma unroll
    for (int p = 0; p < RT; ++p) v += part[p][c >> 3][c & 7];
    if (at < N) sums[blockIdx.x * N + at] = v;
  }
}

// The partial sums' sum in one order: 16 columns a workgroup, 16 threads a column.
__global__ __launch_bounds__(256) void k_linear_colsum(const float *__restrict__ sums, int64_t parts,
                                                       int64_t N, float *__restrict__ out) {
  __shared__ float s[16][17];
  const int c = threadIdx.x & 15, q = threadIdx.x >> 4;
  const int64_t col = (int64_t)blockIdx.x * 16 + c;
  float v = 0.0f;
  if (col < N) {
#pragma unroll 8
    for (int64_t p = q; p < parts; p += 16) v += sums[p * N + col];
  }
  s[q][c] = v;
  __syncthreads();
  if (q > 0 || col >= N) return;
#pragma unroll
  for (int p = 1; p < 16; ++p) v += s[p][c];
  out[col] = v;
}

__global__ __launch_bounds__(256) void k_linear_zero(float *__restrict__ p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = 0.0f;
}

// ------------------------------------------------------------------- host

namespace {

struct LnPlan {
  int tm, tn, splits;
  int64_t part, ns;  // ns: an estimate, for 128 x 128 tiles
};

int64_t ln_tiles(int64_t I, int64_t J, int tm, int tn) {
  return ((I + tm - 1) / tm) * ((J + tn - 1) / tn);
}

// Outputs of 3 * 2^23 values on (50 MB) leave past the caches: the operands keep them
// (8190 x 4096 x 2048 with SiLU, bias, residual and z: 168 us, 162 so; dx of 16384 x 128
// x 2048: 46, 36, though a norm's gradients behind it, which read it, give back 13; two
// layers of 8192 x 2048 x 8192 in a row: 549, 518).  Fewer are still
// there for whoever reads them next (the same two layers with 1024 rows and 4096
// outputs: 64, 73).  A residual of 2^26 values does too: it is not there anyway
// (8192 x 8192 x 2048: 334, 306), where one of 2^25 may be (36, 46).
int ln_stream(int64_t I, int64_t J) {
  return I * J >= (int64_t)1 << 26 ? 2 : I * J >= (int64_t)3 << 23 ? 1 : 0;
}

// Tiles and splits by size alone.
//
// 256 x 256 tiles from 200 of them on (8190 x 4096 x 2048: 976 TFLOP/s, 128 x 128
// 750), unless the contraction is so short that the epilogue counts, which two
// workgroups a CU overlap (dx of 8192 x 256 x 2048: 27.7 us, 23.6 in 128 x 128; of
// 4096 x 128 x 7168: 37.4, 32.0).  Else 128 x 128; splitting the contraction pays where
// the steps of 32 saved outweigh a launch of 4 us and the partial sums' way out and
// back.  A step takes 0.24 us on a CU (LDS) and, from about 200 workgroups on, 1.25 ns
// a workgroup (the L2s give 13 TB/s).  Where both operands are read across the
// contraction (dW), whose rows come from memory and never again, one workgroup a CU
// waits for them (0.5 us a step) and two hide half of that: up to 512 workgroups
// (dW of 16384 x 256 x 2048: 60 us in 160, 42 in 512; 8192 x 512 x 2048: 55, 40).
LnPlan ln_plan(int kind, int64_t I, int64_t J, int64_t K) {
  LnPlan p = {128, 128, 1, (K + 31) / 32 * 32, 0};
  if (K > 256 && ln_tiles(I, J, 256, 256) >= 200) {
    p.tm = p.tn = 256;
    return p;
  }
  const int64_t tiles = ln_tiles(I, J, 128, 128), steps = (K + 31) / 32;
  const int64_t most = kind == LN_TN ? 512 : 256;
  for (int64_t s = 1; s <= 64 && (s == 1 || (tiles * s <= most && steps / s >= 4)); ++s) {
    const int64_t each = (steps + s - 1) / s, n = tiles * s;
    const int64_t step = kind == LN_TN ? (n > 256 ? 650 : 500) : n > 192 ? n * 5 / 4 : 240;
    const int64_t join = s == 1 ? 0 : 4000 + s * I * J / (kind == LN_TN ? 450 : 600);
    const int64_t ns = each * step + join;
    if (s == 1 || ns < p.ns) {
      p.ns = ns;
      p.part = each * 32;
      p.splits = (int)((steps + each - 1) / each);
    }
  }
  return p;
}

size_t ln_partial_bytes(const LnPlan &p, int64_t I, int64_t J) {
  return p.splits > 1 ? (size_t)p.splits * I * J * 4 : 0;
}

template <int KIND, int TM, int TN, int NS>
hipError_t ln_launch_tile(const LnTile &t, const LnEpi &e, int splits, hipStream_t st) {
  hipLaunchKernelGGL((k_linear<KIND, TM, TN, NS>),
                     dim3((unsigned)((int64_t)t.mt * t.nt * splits)), dim3(256), 0, st, t, e);
  return hipGetLastError();
}

template <int KIND>
hipError_t ln_product(const uint16_t *a, int64_t lda, const uint16_t *b, int64_t ldb, int64_t I,
                      int64_t J, int64_t K, const LnEpi &e, float *ws, hipStream_t st) {
  const LnPlan p = ln_plan(KIND, I, J, K);
  const LnTile t = {a, b, lda, ldb, I, J, K, p.part, (int)((I + p.tm - 1) / p.tm),
                    (int)((J + p.tn - 1) / p.tn), p.splits > 1 ? ws : nullptr};
  // Up to one workgroup a CU: eight steps in flight; more: four, two workgroups a CU.
  const bool deep = (int64_t)t.mt * t.nt * p.splits <= 256;
  const hipError_t r = p.tm == 256 ? ln_launch_tile<KIND, 256, 256, 4>(t, e, p.splits, st)
                       : deep      ? ln_launch_tile<KIND, 128, 128, 8>(t, e, p.splits, st)
                                   : ln_launch_tile<KIND, 128, 128, 4>(t, e, p.splits, st);
  if (r != hipSuccess || p.splits == 1) return r;
  const int64_t groups = I * ((J + 7) / 8);
  const unsigned grid = (unsigned)(groups > 256 * 4096 ? 4096 : (groups + 255) / 256);
  hipLaunchKernelGGL(k_linear_join, dim3(grid), dim3(256), 0, st, ws, p.splits, I, J, e);
  return hipGetLastError();
}

template <int MT, int NT>
hipError_t ln_launch_few(const uint16_t *x, int64_t ldx, const uint16_t *w, int64_t M, int64_t N,
                         int64_t K, const LnEpi &e, hipStream_t st) {
  const int64_t tiles = (N + 16 * NT - 1) / (16 * NT), steps = (K + 31) / 32;
  int ks = 1;
  while (ks < 8 && tiles * ks < 4096 && steps / (2 * ks) >= 4) ks *= 2;
  const dim3 grid((unsigned)((tiles + 8 / ks - 1) / (8 / ks)), (unsigned)((M + 16 * MT - 1) / (16 * MT)));
  hipLaunchKernelGGL((k_linear_few<MT, NT>), grid, dim3(512), 0, st, x, ldx, w, M, K, ks, e);
  return hipGetLastError();
}

// Whether rows straight from memory are the faster way: up to LN_FEW rows always
// (64 rows to 2048 outputs of 2048: 10.3 us, 16 in tiles), and while 16 x 16 outputs a
// wave, each with its operands from the L2, cost less than tiles (256 rows to 128
// outputs of 2048: 6.5 us, 10 in tiles; 512 rows to 512 of 2048: 17.6, 13.2).
bool ln_is_few(int64_t M, int64_t N, int64_t K) {
  if (M <= LN_FEW) return true;
  const int64_t units = ((M + 15) / 16) * ((N + 15) / 16);
  if (units > (1 << 16) || ln_tiles(M, N, 256, 256) >= 200) return false;
  return units * K / 160 < 2000 + ln_plan(LN_NT, M, N, K).ns;
}

// Few tiles of W: each 16 rows of x are a workgroup's own, since W comes from the L2
// a second time for less than x takes through one CU.  Many: x's tiles share W, and
// W's tiles share x in pairs.
hipError_t ln_few(const uint16_t *x, int64_t ldx, const uint16_t *w, int64_t M, int64_t N,
                  int64_t K, const LnEpi &e, hipStream_t st) {
  if (M <= 16 || M > LN_FEW || N < LN_SHARE) return ln_launch_few<1, 1>(x, ldx, w, M, N, K, e, st);
  if (M <= 32) return ln_launch_few<2, 2>(x, ldx, w, M, N, K, e, st);
  if (M <= 48) return ln_launch_few<3, 2>(x, ldx, w, M, N, K, e, st);
  return ln_launch_few<4, 2>(x, ldx, w, M, N, K, e, st);
}

bool al(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
pqm_status st_of(hipError_t e) { return e == hipSuccess ? PQM_OK : PQM_ERR_HIP; }

// Sizes that every product here takes.
bool ln_sizes(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N >= 0 && K >= 8 && K % 8 == 0 && M < ((int64_t)1 << 29) && N <= LN_MAX &&
         K <= LN_MAX && ln_tiles(M, N, 128, 128) < (1 << 24) && M <= ((int64_t)1 << 40) / (N + K);
}

// And their gradients: a launch holds fewer than 2^32 threads, 256 for each tile of dx
// and of dW and for each LZ_ROWS rows of dz.
bool ln_backward_sizes(int64_t M, int64_t N, int64_t K) {
  return ln_sizes(M, N, K) && N >= 8 && N % 8 == 0 && M <= ((int64_t)1 << 29) - LZ_ROWS &&
         ln_tiles(M, K, 128, 128) < (1 << 24) && ln_tiles(N, K, 128, 128) < (1 << 24);
}

size_t ln_forward_bytes(int64_t M, int64_t N, int64_t K) {
  return ln_is_few(M, N, K) ? 0 : ln_partial_bytes(ln_plan(LN_NT, M, N, K), M, N);
}

size_t ln_backward_bytes(int64_t M, int64_t N, int64_t K) {
  const size_t a = ln_partial_bytes(ln_plan(LN_NN, M, K, N), M, K);
  const size_t b = ln_partial_bytes(ln_plan(LN_TN, N, K, M), N, K);
  const size_t c = (size_t)((M + LZ_ROWS - 1) / LZ_ROWS) * N * 4;
  return a > b ? (a > c ? a : c) : (b > c ? b : c);
}

}  // namespace
}  // namespace pqm

extern "C" {

size_t pqm_linear_workspace(int64_t M, int64_t N, int64_t K) {
  using namespace pqm;
  return !ln_sizes(M, N, K) || M == 0 || N == 0 ? 0 : ln_forward_bytes(M, N, K);
}

size_t pqm_linear_backward_workspace(int64_t M, int64_t N, int64_t K) {
  using namespace pqm;
  return !ln_backward_sizes(M, N, K) || M == 0 ? 0 : ln_backward_bytes(M, N, K);
}

pqm_status pqm_linear(const uint16_t *x, int64_t ldx, const uint16_t *w, const float *bias,
                      pqm_act act, const uint16_t *residual, int64_t ldr, int64_t M, int64_t N,
                      int64_t K, void *y, pqm_dtype y_dtype, uint16_t *z, void *workspace,
                      size_t workspace_bytes, hipStream_t stream) {
  using namespace pqm;
  if (y_dtype != PQM_OUT_BF16 && y_dtype != PQM_OUT_FP32) return PQM_ERR_ENUM;
  if (act != PQM_ACT_NONE && act != PQM_ACT_SILU && act != PQM_ACT_GELU) return PQM_ERR_ENUM;
  if (!ln_sizes(M, N, K) || ldx < K || ldx > LN_MAX || (residual && (ldr < N || ldr > LN_MAX)))
    return PQM_ERR_SHAPE;
  if (residual && residual == y && (ldr != N || y_dtype != PQM_OUT_BF16)) return PQM_ERR_SHAPE;
  if (M == 0 || N == 0) return PQM_OK;
  if (!x || !w || !y) return PQM_ERR_NULL;
  if (!al(x, 16) || ldx % 8 || !al(w, 16) || !al(y, 16) || !al(z, 16) || !al(bias, 4) ||
      !al(residual, 2))
    return PQM_ERR_ALIGN;
  const size_t need = ln_forward_bytes(M, N, K);
  if (need) {
    if (!workspace) return PQM_ERR_NULL;
    if (workspace_bytes < need) return PQM_ERR_WORKSPACE;
    if (!al(workspace, 16)) return PQM_ERR_ALIGN;
  }
  const int vec = N % 8 == 0 && (!residual || (al(residual, 16) && ldr % 8 == 0));
  const LnEpi e = {bias, residual, ldr, y, z, N, act, y_dtype == PQM_OUT_FP32, vec,
                   ln_stream(M, N)};
  return st_of(ln_is_few(M, N, K) ? ln_few(x, ldx, w, M, N, K, e, stream)
                           : ln_product<LN_NT>(x, ldx, w, K, M, N, K, e,
                                               static_cast<float *>(workspace), stream));
}

pqm_status pqm_linear_backward(const uint16_t *dy, int64_t lddy, const uint16_t *x, int64_t ldx,
                               const uint16_t *w, pqm_act act, const uint16_t *z,
                               const uint16_t *d_x, int64_t ldd, int64_t M, int64_t N, int64_t K,
                               uint16_t *dz, uint16_t *dx, float *dw, float *dbias,
                               void *workspace, size_t workspace_bytes, hipStream_t stream) {
  using namespace pqm;
  if (act != PQM_ACT_NONE && act != PQM_ACT_SILU && act != PQM_ACT_GELU) return PQM_ERR_ENUM;
  if (!ln_backward_sizes(M, N, K) || lddy < N || lddy > LN_MAX ||
      (dw && (ldx < K || ldx > LN_MAX)) || (dx && d_x && (ldd < K || ldd > LN_MAX)) ||
      (dx && d_x == dx && ldd != K))
    return PQM_ERR_SHAPE;
  if (!dx && !dw && !dbias) return PQM_ERR_NULL;
  if (M > 0 &&
      (!dy || (dw && !x) || (dx && !w) || (act != PQM_ACT_NONE && (!z || !dz))))
    return PQM_ERR_NULL;
  if (!al(dy, 16) || lddy % 8 || (dw && (!al(x, 16) || ldx % 8)) || !al(w, 16) || !al(z, 16) ||
      !al(d_x, 2) || !al(dz, 16) || !al(dx, 16) || !al(dw, 16) || !al(dbias, 16))
    return PQM_ERR_ALIGN;
  if (M == 0) {  // sums over no rows
    for (int i = 0; i < 2; ++i) {
      float *p = i ? dbias : dw;
      const int64_t n = i ? N : N * K;
      if (!p) continue;
      hipLaunchKernelGGL(k_linear_zero, dim3((unsigned)(n > (1 << 20) ? 4096 : (n + 255) / 256)),
                         dim3(256), 0, stream, p, n);
      if (hipGetLastError() != hipSuccess) return PQM_ERR_HIP;
    }
    return PQM_OK;
  }
  const size_t need = ln_backward_bytes(M, N, K);
  if (need) {
    if (!workspace) return PQM_ERR_NULL;
    if (workspace_bytes < need) return PQM_ERR_WORKSPACE;
    if (!al(workspace, 16)) return PQM_ERR_ALIGN;
  }
  float *ws = static_cast<float *>(workspace);
  if (act != PQM_ACT_NONE || dbias) {
    const unsigned parts = (unsigned)((M + LZ_ROWS - 1) / LZ_ROWS);
    const int ct = N > 256 ? 64 : N > 128 ? 32 : 16;
    const auto kernel = ct == 64 ? k_linear_dz<64> : ct == 32 ? k_linear_dz<32> : k_linear_dz<16>;
    hipLaunchKernelGGL(kernel, dim3(parts, (unsigned)((N + 8 * ct - 1) / (8 * ct))), dim3(256), 0,
                       stream, dy, lddy, z, act, M, N, dz, dbias ? ws : nullptr);
    if (hipGetLastError() != hipSuccess) return PQM_ERR_HIP;
    if (dbias) {
      hipLaunchKernelGGL(k_linear_colsum, dim3((unsigned)((N + 15) / 16)), dim3(256), 0, stream, ws,
                         parts, N, dbias);
      if (hipGetLastError() != hipSuccess) return PQM_ERR_HIP;
    }
  }
  const uint16_t *g = act == PQM_ACT_NONE ? dy : dz;
  const int64_t ldg = act == PQM_ACT_NONE ? lddy : N;
  if (dx) {
    const LnEpi e = {nullptr, d_x, ldd, dx, nullptr, K, PQM_ACT_NONE, 0,
                     !d_x || (al(d_x, 16) && ldd % 8 == 0),
                     ln_stream(M, K)};
    const hipError_t r = ln_product<LN_NN>(g, ldg, w, K, M, K, N, e, ws, stream);
    if (r != hipSuccess) return PQM_ERR_HIP;
  }
  if (dw) {
    const LnEpi e = {nullptr, nullptr, 0, dw, nullptr, K, PQM_ACT_NONE, 1, 1, 0};
    const hipError_t r = ln_product<LN_TN>(g, ldg, x, ldx, N, K, M, e, ws, stream);
    if (r != hipSuccess) return PQM_ERR_HIP;
  }
  return PQM_OK;
}

}  // extern "C"
