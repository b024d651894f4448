// token_logprobs.hip -- what a policy's logits [T, V] say of given tokens: their
// log probabilities, the entropy of each row, its best alternatives, and the
// gradient of the first two.
//
// With x a row of logits, t the temperature, M its largest logit,
//   u_i = (x_i - M) / t,  S = sum e^u,  log p_i = u_i - log S,
//   H = log S - (sum e^u u) / S,
//   d x_i = (g [i = id] - p_i (g + h (log p_i + H))) / t
// for the gradients g of log p_id and h of H.  One pass reads the row: each
// thread carries its running maximum, sum (without the maximum's own 1) and weighted
// sum, and moves the sums when its maximum grows.  u is formed from the difference, which neither
// overflows nor loses digits where all logits are far from 0; in powers of two,
// u log2(e).
//
// Both directions are bound by memory where there are many rows: 4093 rows of 32768
// bf16, a fifth of them left out, in 42 us (5.1 TB/s of the rows that are read);
// gradient of 2048 rows of 151936 bf16, a fifth left out, in 190 us (5.8 TB/s, read and
// written), of 509 rows of 50257 binary32, an odd length, in 44 (4.6).  One row of 151936 is split over workgroups and bound by
// the chain of load, choice of the best, join: 17.5 us with 20 alternatives.
#include "pqm_device.hpp"
#include "pqm_internal.hpp"
#include "pqmoe.h"

#include <type_traits>

namespace pqm {

namespace {

constexpr int TL_TOP = 32;         // alternatives at most
constexpr int TL_TILE = 2048;      // logits of a workgroup's turn: 256 threads, eight each
constexpr int TL_PARTS = 128;      // parts of a row at most
constexpr int TL_JOIN = 2048;      // candidates of a row's parts at most
constexpr float TL_LOG2E = 1.44269504088896341f, TL_LN2 = 0.69314718055994531f;

typedef uint64_t tl_key;  // a logit's order, then the lower index; 0: none

// Sixteen bytes at any element's address: rows of an odd length start anywhere.
struct __attribute__((packed, aligned(2))) TlWords {
  uint32_t w[4];
};

template <bool F32>
__device__ __forceinline__ float tl_one(const void *row, int64_t i) {
  if (F32) return static_cast<const float *>(row)[i];
  return bf16_lo_f32(static_cast<const uint16_t *>(row)[i]);
}

// The same, past the caches with NT: what no cache holds until its next reader comes
// only takes the place of something else.
typedef uint32_t tl_v4 __attribute__((ext_vector_type(4), aligned(2)));
template <bool NT>
__device__ __forceinline__ TlWords tl_get(const void *at) {
  if (!NT) return *static_cast<const TlWords *>(at);
  return __builtin_bit_cast(TlWords, __builtin_nontemporal_load(static_cast<const tl_v4 *>(at)));
}
template <bool NT>
__device__ __forceinline__ void tl_put(void *at, const TlWords &w) {
  if (!NT) *static_cast<TlWords *>(at) = w;
  else __builtin_nontemporal_store(__builtin_bit_cast(tl_v4, w), static_cast<tl_v4 *>(at));
}

// Eight logits from i on, -inf past the end.
template <bool F32, bool NT>
__device__ __forceinline__ void tl_load8(const void *row, int64_t i, int64_t end, float (&x)[8]) {
  if (i + 8 <= end) {
    if (F32) {
      const float *p = static_cast<const float *>(row) + i;
      const TlWords a = tl_get<NT>(p), b = tl_get<NT>(p + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = __uint_as_float(a.w[j]);
        x[4 + j] = __uint_as_float(b.w[j]);
      }
    } else {
      const TlWords a = tl_get<NT>(static_cast<const uint16_t *>(row) + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = bf16_lo_f32(a.w[j]);
        x[2 * j + 1] = bf16_hi_f32(a.w[j]);
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = i + j < end ? tl_one<F32>(row, i + j) : -__builtin_inff();
}

// Running statistics: the maximum, the sum of e^u without the maximum's own 1, and the
// sum of e^u u log2(e).  Without that 1 a nearly certain row keeps its entropy and its
// log S = log(1 + r), which are as small as r: next to the 1 they would lose what lies
// below half a step of it.  A NaN is no maximum, but reaches the sum.
struct TlSums {
  float m, r, t;
};

// Where nothing but -inf was seen, differences are taken from 0.
__device__ __forceinline__ float tl_from(float m) { return m == -__builtin_inff() ? 0.0f : m; }

// The exponent of a logit d below the maximum; from -200 on down all are 0 in
// binary32, and -inf times 0 would be a NaN.
__device__ __forceinline__ float tl_exponent(float d, float c) {
  return __builtin_elementwise_maximum(d * c, -200.0f);
}

// Takes b, of a maximum not above a's, into a; with nothing seen its share is 0.
__device__ __forceinline__ void tl_take(TlSums &a, const TlSums &b, float c) {
  const float d = tl_exponent(b.m - tl_from(a.m), c), f = __builtin_amdgcn_exp2f(d);
  const float all = 1.0f + b.r;
  a.t = __builtin_fmaf(f, __builtin_fmaf(all, d, b.t), a.t);
  a.r = __builtin_fmaf(f, all, a.r);
}

__device__ __forceinline__ void tl_join(TlSums &a, const TlSums &b, float c) {
  const bool up = b.m > a.m;
  TlSums hi = up ? b : a;
  const TlSums lo = up ? a : b;
  tl_take(hi, lo, c);
  a = hi;
}

// Takes in 8 U logits.  All at once, since a wave finds a new maximum in one of its
// lanes nearly every time (4093 rows of 32768: 52.8 us by 32, 53.6 by eight).
template <int U>
__device__ __forceinline__ void tl_add(TlSums &a, const float (&v)[U][8], float c) {
  float x[U][8], m = v[0][0];
#pragma unroll
  for (int j = 0; j < 8 * U; ++j) {
    x[j / 8][j % 8] = v[j / 8][j % 8];
    m = fmaxf(m, v[j / 8][j % 8]);
  }
  if (m > a.m) {  // a new maximum: its 1 is no part of r
    TlSums b = {m, 0.0f, 0.0f};
    tl_take(b, a, c);
    a = b;
    bool left = m < __builtin_inff();  // inf stays: inf - inf makes the row NaN
#pragma unroll
    for (int j = 0; j < 8 * U; ++j) {
      const bool it = left && x[j / 8][j % 8] == m;
      x[j / 8][j % 8] = it ? -__builtin_inff() : x[j / 8][j % 8];
      left = left && !it;
    }
  }
  const float from = tl_from(a.m);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float s[2] = {0, 0}, t[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float u = tl_exponent(x[i][j] - from, c), e = __builtin_amdgcn_exp2f(u);
      s[j & 1] += e;
      t[j & 1] = __builtin_fmaf(e, u, t[j & 1]);
    }
    a.r += s[0] + s[1];
    a.t += t[0] + t[1];
  }
}

// The workgroup's statistics in thread 0.
__device__ __forceinline__ TlSums tl_reduce(TlSums a, float c, TlSums *sh) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const TlSums b = {__shfl_down(a.m, o, 64), __shfl_down(a.r, o, 64), __shfl_down(a.t, o, 64)};
    tl_join(a, b, c);
  }
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < 4; ++w) tl_join(a, sh[w], c);
  }
  return a;
}

// A logit's place in the order: NaN first, -0 as +0; above 0 for every logit.
__device__ __forceinline__ uint32_t tl_order(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return x != x ? 0xFFFFFFFFu : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float tl_value(uint32_t o) {
  return o == 0xFFFFFFFFu ? __builtin_nanf("")
                          : __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ tl_key tl_make(float x, int64_t i) {
  return (tl_key)tl_order(x) << 32 | (0xFFFFFFFFu - (uint32_t)i);
}

// The n best keys so far, in order.
struct TlTop {
  tl_key kept[TL_TOP];
  tl_key bar[4];
  __align__(16) tl_key cand[TL_TOP + 4 * 8 * TL_TOP + 8];
  int count;
};

__device__ __forceinline__ void tl_top_init(TlTop &s) {
  if (threadIdx.x < TL_TOP) s.kept[threadIdx.x] = 0;
  __syncthreads();
}

// Takes in eight keys a thread.  With b the n-th of the lanes' own best in a wave, at
// least n keys are not below b, so none below the largest of the waves' b is among the
// n best; and no wave has more than n lanes whose best reaches it, so no more than 32 n
// candidates are left however the logits are ordered (n and a few as a rule), and
// ranking them by counting stays cheap.
__device__ __forceinline__ void tl_top_add(TlTop &s, const tl_key (&k)[8], int n) {
  const int wave = threadIdx.x >> 6;
  tl_key top = k[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) top = k[j] > top ? k[j] : top;
  const tl_key last = s.kept[n - 1];
  if (__syncthreads_count(top > last) == 0) return;
  int above = 0;
#pragma unroll 16
  for (int i = 0; i < 64; ++i) {
    const tl_key o = (tl_key)(uint32_t)__builtin_amdgcn_readlane((int)(top >> 32), i) << 32 |
                     (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)top, i);
    above += o > top ? 1 : 0;
  }
  const uint64_t at = __ballot(above == n - 1 && top > last);  // keys differ: one lane, or none
  if ((threadIdx.x & 63) == 0) s.bar[wave] = last + 1;
  if (at >> (threadIdx.x & 63) & 1) s.bar[wave] = top;
  for (int i = threadIdx.x; i < (int)(sizeof(s.cand) / sizeof(tl_key)); i += 256)
    s.cand[i] = i < n ? s.kept[i] : 0;
  if (threadIdx.x == 0) s.count = n;
  __syncthreads();
  tl_key bar = s.bar[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) bar = s.bar[w] > bar ? s.bar[w] : bar;
  if (top >= bar) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k[j] >= bar) s.cand[atomicAdd(&s.count, 1)] = k[j];
  }
  __syncthreads();
  const int count = s.count;
  for (int i = threadIdx.x; i < count; i += 256) {
    const tl_key mine = s.cand[i];
    int better = 0;
    for (int j = 0; j < count; j += 8) {  // zeros behind the last
      const ulonglong2 *p = reinterpret_cast<const ulonglong2 *>(s.cand + j);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const ulonglong2 v = p[q];
        better += (v.x > mine ? 1 : 0) + (v.y > mine ? 1 : 0);
      }
    }
    if (better < n && mine != 0) s.kept[better] = mine;
  }
  __syncthreads();
}

struct TlArgs {
  const void *x;
  int64_t ld;
  const int32_t *ids;
  int64_t V;
  float temperature, c;  // c = log2(e) / temperature
  float *logprob, *entropy, *stats;
  int32_t *top_ids;
  float *top_logprob;
  int n;
  int parts;
  int64_t part;  // logits of a part
  uint8_t *ws;
};

// A part's record: its statistics, then its keys.
__device__ __forceinline__ uint8_t *tl_record(const TlArgs &a, int64_t row, int part) {
  return a.ws + (row * a.parts + part) * (16 + 8 * a.n);
}

// The row's id; -1 for a row to leave out, 0 without ids.
__device__ __forceinline__ int64_t tl_id(const TlArgs &a, int64_t row) {
  if (!a.ids) return 0;
  const int64_t i = a.ids[row];
  return i < 0 || i >= a.V ? -1 : i;
}

// The row's results from its statistics (thread 0) and keys.
template <bool F32>
__device__ __forceinline__ void tl_finish(const TlArgs &a, int64_t row, int64_t id, const TlSums &s,
                                          const TlTop *top, float *sh) {
  const bool none = s.m == -__builtin_inff() && s.r == 0.0f;  // -inf alone
  if (threadIdx.x == 0) {
    const float log_s = none ? 0.0f : log1pf(s.r);
    if (a.stats) {
      a.stats[2 * row] = s.m;
      a.stats[2 * row + 1] = log_s;
    }
    if (a.entropy) a.entropy[row] = none ? 0.0f : fmaxf(log_s - TL_LN2 * (s.t / (1.0f + s.r)), 0.0f);
    if (a.entropy && !none && s.r != s.r) a.entropy[row] = s.r;
    if (a.logprob) {
      const float x = tl_one<F32>(static_cast<const uint8_t *>(a.x) +
                                      row * a.ld * (F32 ? 4 : 2), id);
      a.logprob[row] = (x - tl_from(s.m)) / a.temperature - log_s;
    }
    sh[0] = s.m;
    sh[1] = log_s;
  }
  if (!top) return;
  __syncthreads();
  if (threadIdx.x < a.n) {
    const tl_key k = top->kept[threadIdx.x];
    a.top_ids[row * a.n + threadIdx.x] = (int32_t)(0xFFFFFFFFu - (uint32_t)k);
    a.top_logprob[row * a.n + threadIdx.x] =
        (tl_value((uint32_t)(k >> 32)) - tl_from(sh[0])) / a.temperature - sh[1];
  }
}

// A row that is left out.
__device__ __forceinline__ void tl_skip(const TlArgs &a, int64_t row) {
  if (threadIdx.x == 0) {
    if (a.logprob) a.logprob[row] = 0.0f;
    if (a.entropy) a.entropy[row] = 0.0f;
    if (a.stats) a.stats[2 * row] = a.stats[2 * row + 1] = 0.0f;
  }
  if (threadIdx.x < a.n) {
    a.top_ids[row * a.n + threadIdx.x] = -1;
    a.top_logprob[row * a.n + threadIdx.x] = 0.0f;
  }
}

}  // namespace

// One part of one row a workgroup; a row of one part is finished here.
template <bool F32, bool TOP, bool NT>
__global__ __launch_bounds__(256) void k_token_logprobs(TlArgs a) {
  __shared__ TlSums sh[4];
  __shared__ float fin[2];
  __shared__ typename std::conditional<TOP, TlTop, int>::type top;
  const int64_t row = blockIdx.x / a.parts;
  const int part = (int)(blockIdx.x - row * a.parts);
  const int64_t id = tl_id(a, row);
  if (id < 0) {
    if (a.parts == 1) tl_skip(a, row);
    return;
  }
  const uint8_t *x = static_cast<const uint8_t *>(a.x) + row * a.ld * (F32 ? 4 : 2);
  const int64_t i0 = part * a.part, end = min(a.V, i0 + a.part);
  TlSums s = {-__builtin_inff(), 0.0f, 0.0f};
  if constexpr (TOP) {
    tl_top_init(top);
    for (int64_t i = i0; i < end; i += TL_TILE) {  // every thread takes every turn
      const int64_t at = i + 8 * threadIdx.x;
      float v[1][8];
      tl_load8<F32, NT>(x, at, end, v[0]);
      tl_add<1>(s, v, a.c);
      tl_key k[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) k[j] = at + j < end ? tl_make(v[0][j], at + j) : 0;
      tl_top_add(top, k, a.n);
    }
  } else {
    int64_t at = i0 + 8 * threadIdx.x;
    for (; at + 3 * TL_TILE + 8 <= end; at += 4 * TL_TILE) {
      float v[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u) tl_load8<F32, NT>(x, at + u * TL_TILE, a.V, v[u]);
      tl_add<4>(s, v, a.c);
    }
    for (; at < end; at += TL_TILE) {
      float v[1][8];
      tl_load8<F32, NT>(x, at, end, v[0]);
      tl_add<1>(s, v, a.c);
    }
  }
  s = tl_reduce(s, a.c, sh);
  if (a.parts == 1) {
    if constexpr (TOP) tl_finish<F32>(a, row, id, s, &top, fin);
    else tl_finish<F32>(a, row, id, s, nullptr, fin);
    return;
  }
  uint8_t *rec = tl_record(a, row, part);
  if (threadIdx.x == 0) {
    float *f = reinterpret_cast<float *>(rec);
    f[0] = s.m;
    f[1] = s.r;
    f[2] = s.t;
  }
  if constexpr (TOP) {
    if (threadIdx.x < a.n)
      reinterpret_cast<tl_key *>(rec + 16)[threadIdx.x] = top.kept[threadIdx.x];
  }
}

// The parts of a row, joined in one order.
template <bool F32, bool TOP>
__global__ __launch_bounds__(256) void k_token_logprobs_join(TlArgs a) {
  __shared__ TlSums sh[4];
  __shared__ float fin[2];
  __shared__ typename std::conditional<TOP, TlTop, int>::type top;
  const int64_t row = blockIdx.x, id = tl_id(a, row);
  if (id < 0) return tl_skip(a, row);
  TlSums s = {-__builtin_inff(), 0.0f, 0.0f};
  if (threadIdx.x < a.parts) {
    const float *f = reinterpret_cast<const float *>(tl_record(a, row, threadIdx.x));
    s = TlSums{f[0], f[1], f[2]};
  }
  if constexpr (TOP) {
    tl_top_init(top);
    tl_key k[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = threadIdx.x + 256 * j;
      k[j] = i < a.parts * a.n
                 ? reinterpret_cast<const tl_key *>(tl_record(a, row, i / a.n) + 16)[i % a.n]
                 : 0;
    }
    tl_top_add(top, k, a.n);
  }
  s = tl_reduce(s, a.c, sh);
  if constexpr (TOP) tl_finish<F32>(a, row, id, s, &top, fin);
  else tl_finish<F32>(a, row, id, s, nullptr, fin);
}

namespace {

struct TlBack {
  const void *x;
  int64_t ld;
  const int32_t *ids;
  int64_t V;
  float temperature, c;
  const float *stats, *entropy, *d_logprob, *d_entropy;
  void *dx;
  int64_t ldd;
  int parts;
};

constexpr int TB_TURNS = 4;  // eight logits a thread each

template <bool F32, bool NT>
__device__ __forceinline__ void tl_store8(void *row, int64_t i, int64_t end, const float (&v)[8]) {
  if (i + 8 <= end) {
    if (F32) {
      float *p = static_cast<float *>(row) + i;
      TlWords a, b;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a.w[j] = __float_as_uint(v[j]);
        b.w[j] = __float_as_uint(v[4 + j]);
      }
      tl_put<NT>(p, a);
      tl_put<NT>(p + 4, b);
    } else {
      TlWords a;
#pragma unroll
      for (int j = 0; j < 4; ++j) a.w[j] = pk_bf16_rne(v[2 * j], v[2 * j + 1]);
      tl_put<NT>(static_cast<uint16_t *>(row) + i, a);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (i + j >= end) break;
    if (F32) static_cast<float *>(row)[i + j] = v[j];
    else static_cast<uint16_t *>(row)[i + j] = (uint16_t)pk_bf16_rne(v[j], 0.0f);
  }
}

}  // namespace

// Gradient: with l = log2 p, d x = -p (A + B l), A = (g + h H) / t, B = h ln 2 / t, but
// for the taken token's.
template <bool F32, bool OUTF32, bool NT>
__global__ __launch_bounds__(256) void k_token_logprobs_backward(TlBack a) {
  const int64_t row = blockIdx.x / a.parts;
  const int64_t at = (blockIdx.x - row * a.parts) * (int64_t)(TB_TURNS * TL_TILE) +
                     8 * threadIdx.x;
  const uint8_t *x = static_cast<const uint8_t *>(a.x) + row * a.ld * (F32 ? 4 : 2);
  uint8_t *dx = static_cast<uint8_t *>(a.dx) + row * a.ldd * (OUTF32 ? 4 : 2);
  int64_t id = a.ids ? a.ids[row] : 0;
  const float m = a.stats[2 * row], log_s = a.stats[2 * row + 1];
  const bool skip = id < 0 || id >= a.V || (m == -__builtin_inff() && log_s == 0.0f);
  if (!a.ids) id = -1;
  if (skip) {
    const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < TB_TURNS; ++u) tl_store8<OUTF32, NT>(dx, at + u * TL_TILE, a.V, zero);
    return;
  }
  const float ls = log_s * TL_LOG2E;
  const float g = a.d_logprob ? a.d_logprob[row] / a.temperature : 0.0f;
  const float h = a.d_entropy ? a.d_entropy[row] / a.temperature : 0.0f;
  const float H = a.d_entropy ? a.entropy[row] : 0.0f;
  const float A = __builtin_fmaf(h, H, g), B = h * TL_LN2;
  // The taken token: g (1 - p) as -g (e^(log p) - 1), since p of a nearly certain token
  // is 1 in binary32 long before 1 - p is 0 (what is left of 2^-30 came out as 0), and
  // the entropy's term apart, which next to g would lose as much.
  float taken = 0.0f;
  if (id >= at && (id - at) % TL_TILE < 8 && id - at < TB_TURNS * TL_TILE) {
    const float d = tl_one<F32>(x, id) - m;
    const float l = __builtin_elementwise_maximum(__builtin_fmaf(d, a.c, -ls), -200.0f);
    taken = -g * expm1f(d / a.temperature - log_s) -
            __builtin_amdgcn_exp2f(l) * __builtin_fmaf(B, l, h * H);
  }
  float v[TB_TURNS][8];
#pragma unroll
  for (int u = 0; u < TB_TURNS; ++u) tl_load8<F32, NT>(x, at + u * TL_TILE, a.V, v[u]);
#pragma unroll
  for (int u = 0; u < TB_TURNS; ++u) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float l =
          __builtin_elementwise_maximum(__builtin_fmaf(v[u][j] - m, a.c, -ls), -200.0f);
      v[u][j] = -__builtin_amdgcn_exp2f(l) * __builtin_fmaf(B, l, A);
    }
    const int64_t rel = id - (at + u * TL_TILE);
    if (rel >= 0 && rel < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (rel == j) v[u][j] = taken;
    }
    tl_store8<OUTF32, NT>(dx, at + u * TL_TILE, a.V, v[u]);
  }
}

// ------------------------------------------------------------------- host

namespace {

struct TlPlan {
  int parts;
  int64_t part;
};

// Parts of a row: as many as give the card 1024 workgroups, none below a turn.
TlPlan tl_plan(int64_t tokens, int64_t V, int64_t n) {
  const int64_t turns = (V + TL_TILE - 1) / TL_TILE;
  int64_t parts = (1024 + tokens - 1) / tokens;
  if (parts > TL_PARTS) parts = TL_PARTS;
  if (n && parts > TL_JOIN / n) parts = TL_JOIN / n;
  if (parts > turns) parts = turns;
  const int64_t each = (turns + parts - 1) / parts;
  return {(int)((turns + each - 1) / each), each * TL_TILE};
}

size_t tl_bytes(int64_t tokens, int64_t V, int64_t n) {
  const TlPlan p = tl_plan(tokens, V, n);
  return p.parts == 1 ? 0 : (size_t)tokens * p.parts * (16 + 8 * n);
}

bool tl_sizes(int64_t tokens, int64_t V, int64_t n) {
  return tokens >= 0 && tokens < ((int64_t)1 << 24) && V >= 1 && V <= ((int64_t)1 << 30) && n >= 0 &&
         n <= TL_TOP && n <= V;
}

bool al(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
pqm_status st_of(hipError_t e) { return e == hipSuccess ? PQM_OK : PQM_ERR_HIP; }

// Logits of 3 * 2^26 bytes on (200 MB) go past the caches, which cannot hold them for
// the backward pass anyway, and so does their gradient: 2048 rows of 151936 bf16 125 and
// 235 us, 125 and 221 so, one after the other 370 and 331; 4093 of 32768 57 and 103, 53
// and 92, 168 and 145.  Fewer may still be there (509 of 50257 binary32: 25 and 39, 27
// and 47 so).
bool tl_streams(int64_t tokens, int64_t V, bool f32) {
  return tokens * V * (f32 ? 4 : 2) >= (int64_t)3 << 26;
}

template <bool F32, bool NT>
hipError_t tl_forward(const TlArgs &a, int64_t tokens, hipStream_t st) {
  const dim3 grid((unsigned)(tokens * a.parts)), rows((unsigned)tokens), block(256);
  if (a.n) hipLaunchKernelGGL((k_token_logprobs<F32, true, NT>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_token_logprobs<F32, false, NT>), grid, block, 0, st, a);
  const hipError_t r = hipGetLastError();
  if (r != hipSuccess || a.parts == 1) return r;
  if (a.n) hipLaunchKernelGGL((k_token_logprobs_join<F32, true>), rows, block, 0, st, a);
  else hipLaunchKernelGGL((k_token_logprobs_join<F32, false>), rows, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace pqm

extern "C" {

size_t pqm_token_logprobs_workspace(int64_t tokens, int64_t vocab, int64_t top_n) {
  using namespace pqm;
  return !tl_sizes(tokens, vocab, top_n) || tokens == 0 ? 0 : tl_bytes(tokens, vocab, top_n);
}

pqm_status pqm_token_logprobs(const void *logits, pqm_dtype logits_dtype, int64_t ld,
                              const int32_t *ids, int64_t tokens, int64_t vocab, float temperature,
                              float *logprob, float *entropy, float *stats, int32_t *top_ids,
                              float *top_logprob, int64_t top_n, void *workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  using namespace pqm;
  if (logits_dtype != PQM_OUT_BF16 && logits_dtype != PQM_OUT_FP32) return PQM_ERR_ENUM;
  if (!tl_sizes(tokens, vocab, top_n) || ld < vocab || ld > ((int64_t)1 << 30))
    return PQM_ERR_SHAPE;
  if (!(temperature >= 0x1p-60f && temperature <= 0x1p60f)) return PQM_ERR_SHAPE;
  const bool f32 = logits_dtype == PQM_OUT_FP32;
  const TlPlan p = tokens ? tl_plan(tokens, vocab, top_n) : TlPlan{1, vocab};
  if (tokens * p.parts >= ((int64_t)1 << 24)) return PQM_ERR_SHAPE;
  if (tokens == 0) return PQM_OK;
  if (!logits || (!logprob && !entropy && !stats && !top_n) || (logprob && !ids) ||
      (top_n && (!top_ids || !top_logprob)))
    return PQM_ERR_NULL;
  if (!al(logits, f32 ? 4 : 2) || !al(ids, 4) || !al(logprob, 4) || !al(entropy, 4) ||
      !al(stats, 4) || !al(top_ids, 4) || !al(top_logprob, 4))
    return PQM_ERR_ALIGN;
  const size_t need = tl_bytes(tokens, vocab, top_n);
  if (need) {
    if (!workspace) return PQM_ERR_NULL;
    if (workspace_bytes < need) return PQM_ERR_WORKSPACE;
    if (!al(workspace, 8)) return PQM_ERR_ALIGN;
  }
  const TlArgs a = {logits, ld, ids, vocab, temperature, (float)(1.4426950408889634 / temperature),
                    logprob, entropy, stats, top_ids, top_logprob, (int)top_n, p.parts, p.part,
                    static_cast<uint8_t *>(workspace)};
  const bool nt = tl_streams(tokens, vocab, f32);
  return st_of(f32 ? nt ? tl_forward<true, true>(a, tokens, stream)
                        : tl_forward<true, false>(a, tokens, stream)
               : nt ? tl_forward<false, true>(a, tokens, stream)
                    : tl_forward<false, false>(a, tokens, stream));
}

pqm_status pqm_token_logprobs_backward(const void *logits, pqm_dtype logits_dtype, int64_t ld,
                                       const int32_t *ids, int64_t tokens, int64_t vocab,
                                       float temperature, const float *stats,
                                       const float *entropy, const float *d_logprob,
                                       const float *d_entropy, void *d_logits,
                                       pqm_dtype d_logits_dtype, int64_t ldd,
                                       hipStream_t stream) {
  using namespace pqm;
  if ((logits_dtype != PQM_OUT_BF16 && logits_dtype != PQM_OUT_FP32) ||
      (d_logits_dtype != PQM_OUT_BF16 && d_logits_dtype != PQM_OUT_FP32))
    return PQM_ERR_ENUM;
  if (!tl_sizes(tokens, vocab, 0) || ld < vocab || ld > ((int64_t)1 << 30) || ldd < vocab ||
      ldd > ((int64_t)1 << 30))
    return PQM_ERR_SHAPE;
  if (!(temperature >= 0x1p-60f && temperature <= 0x1p60f)) return PQM_ERR_SHAPE;
  if (d_logits && d_logits == logits && (ld != ldd || logits_dtype != d_logits_dtype))
    return PQM_ERR_SHAPE;
  const int64_t parts = (vocab + TB_TURNS * TL_TILE - 1) / (TB_TURNS * TL_TILE);
  if (tokens * parts >= ((int64_t)1 << 24)) return PQM_ERR_SHAPE;
  if (tokens == 0) return PQM_OK;
  if (!logits || !stats || !d_logits || (!d_logprob && !d_entropy) || (d_logprob && !ids) ||
      (d_entropy && !entropy))
    return PQM_ERR_NULL;
  const bool f32 = logits_dtype == PQM_OUT_FP32, o32 = d_logits_dtype == PQM_OUT_FP32;
  if (!al(logits, f32 ? 4 : 2) || !al(d_logits, o32 ? 4 : 2) || !al(ids, 4) || !al(stats, 4) ||
      !al(entropy, 4) || !al(d_logprob, 4) || !al(d_entropy, 4))
    return PQM_ERR_ALIGN;
  const TlBack a = {logits, ld, ids, vocab, temperature, (float)(1.4426950408889634 / temperature),
                    stats, entropy, d_logprob, d_entropy, d_logits, ldd, (int)parts};
  const auto pick = [&](auto nt) {
    constexpr bool NT = decltype(nt)::value;
    return f32 ? o32 ? k_token_logprobs_backward<true, true, NT>
                     : k_token_logprobs_backward<true, false, NT>
           : o32 ? k_token_logprobs_backward<false, true, NT>
                 : k_token_logprobs_backward<false, false, NT>;
  };
  const auto kernel = tl_streams(tokens, vocab, f32) ? pick(std::true_type()) : pick(std::false_type());
  hipLaunchKernelGGL(kernel, dim3((unsigned)(tokens * parts)), dim3(256), 0, stream, a);
  return st_of(hipGetLastError());
}

}  // extern "C"
