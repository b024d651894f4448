// gemv_nvfp4.hip -- the experts' products for a few routed rows: bf16
// activations times NVFP4 weights, the decode form of the grouped GEMM.
//
//   y[r, n] = s_g sum_k x[r / div, k] q[e, n, k] s_b[e, n, k / 16],  e = ids[r],
// and for the gate_up projection d[r, n] = bf16(silu(g) u p[r]) of the rows n
// (gate) and I + n (up).  The weights are read once per expert that a row
// chose; rows of the same expert are found in `ids` by the workgroups
// themselves, so no sort, gather or offsets go before.
//
// q s_b has at most 6 significant bits: exact in bf16.  A wave multiplies 16
// weight rows by up to 16 activation rows with v_mfma_f32_16x16x32_bf16; the
// sums are binary32 and the outer scale multiplies them at the end.
#include "pqm_device.hpp"
#include "pqm_internal.hpp"
#include "pqmoe.h"

namespace pqm {

namespace {

typedef __bf16 gv_bf8 __attribute__((ext_vector_type(8)));
typedef float gv_f4 __attribute__((ext_vector_type(4)));
typedef float gv_f2 __attribute__((ext_vector_type(2)));

constexpr int GEMV_MAX_ROWS = 4096;

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

struct GemvArgs {
  const uint16_t *x;
  const int32_t *ids;
  int rows, div;
  const uint8_t *w, *ws;
  const float *wo;
  int64_t rps;
  int G;
  int64_t N, K;  // N: output columns; ACT weights have 2 N rows
  const float *prob;
  void *out;
};

}  // namespace

// One workgroup: 32 weight rows of one expert (ACT: 16 gate rows and their 16
// up rows), the contraction dealt to its four waves in 128-wide chunks and
// their sums joined through LDS in wave order.  byrow: blockIdx.y is a row of
// ids and stands for its expert if no earlier row chose it; otherwise it is
// the expert, and G the rows without one.
template <bool ACT, bool OUTF32>
__global__ __launch_bounds__(256) void k_gemv_nvfp4(GemvArgs a, int byrow) {
  extern __shared__ int list[];  // the rows of this expert, in order
  __shared__ gv_f4 red[4][2][64];
  __shared__ int cnt[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int e = byrow ? a.ids[blockIdx.y] : (int)blockIdx.y;
  if (e < 0 || e >= a.G) e = -1;
  int c = 0;
  bool earlier = false;
  for (int r0 = 0; r0 < a.rows; r0 += 256) {
    const int r = r0 + tid;
    int id = r < a.rows ? a.ids[r] : -2;
    if (id != -2 && (id < 0 || id >= a.G)) id = -1;
    const bool mine = id == e;
    if (byrow && mine && r < (int)blockIdx.y) earlier = true;
    const uint64_t b = __ballot(mine);
    if (lane == 0) cnt[wave] = __popcll(b);
    __syncthreads();
    int pos = c + __popcll(b & ((1ull << lane) - 1));
    for (int w = 0; w < wave; ++w) pos += cnt[w];
    if (mine) list[pos] = r;
    c += cnt[0] + cnt[1] + cnt[2] + cnt[3];
    __syncthreads();
  }
  if (__syncthreads_or(earlier) || c == 0) return;

  const int n0 = blockIdx.x * (ACT ? 16 : 32);
  if (e < 0) {  // rows without an expert give zero
    const int cols = min((int64_t)(ACT ? 16 : 32), a.N - n0);
    for (int i = tid; i < c * cols; i += 256) {
      const int64_t o = (int64_t)list[i / cols] * a.N + n0 + i % cols;
      if (OUTF32) static_cast<float *>(a.out)[o] = 0.0f;
      else static_cast<uint16_t *>(a.out)[o] = 0;
    }
    return;
  }
  const int g = lane >> 4, ln = lane & 15;
  const int64_t NW = ACT ? 2 * a.N : a.N, K = a.K;
  // this lane's weight row of either 16-row tile (past the end: the last row,
  // computed and not stored)
  const int64_t w0 = (int64_t)e * NW + min((int64_t)n0 + ln, a.N - 1);
  const int64_t w1 = ACT ? w0 + a.N : (int64_t)e * NW + min((int64_t)n0 + 16 + ln, a.N - 1);
  for (int m0 = 0; m0 < c; m0 += 16) {
    const int row = list[min(m0 + ln, c - 1)];
    const uint16_t *xr = a.x + (int64_t)(row / a.div) * K;
    gv_f4 acc0 = {0, 0, 0, 0}, acc1 = {0, 0, 0, 0};
    for (int64_t kc = (int64_t)wave * 128; kc < K; kc += 512) {
      const int64_t k = kc + g * 32;
      uint4 q0 = make_uint4(0, 0, 0, 0), q1 = q0, xv[4] = {q0, q0, q0, q0};
      uint32_t s0 = 0, s1 = 0;
      if (k < K) {
        q0 = *reinterpret_cast<const uint4 *>(a.w + (w0 * K + k) / 2);
        q1 = *reinterpret_cast<const uint4 *>(a.w + (w1 * K + k) / 2);
        s0 = *reinterpret_cast<const uint16_t *>(a.ws + (w0 * K + k) / 16);
        s1 = *reinterpret_cast<const uint16_t *>(a.ws + (w1 * K + k) / 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) xv[j] = *reinterpret_cast<const uint4 *>(xr + k + 8 * j);
      }
      const uint32_t u0[4] = {q0.x, q0.y, q0.z, q0.w}, u1[4] = {q1.x, q1.y, q1.z, q1.w};
      const float f0[2] = {__builtin_amdgcn_cvt_f32_fp8((int)s0, 0),
                           __builtin_amdgcn_cvt_f32_fp8((int)s0, 1)};
      const float f1[2] = {__builtin_amdgcn_cvt_f32_fp8((int)s1, 0),
                           __builtin_amdgcn_cvt_f32_fp8((int)s1, 1)};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const gv_bf8 b = __builtin_bit_cast(gv_bf8, xv[j]);
        acc0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(gv_decode(u0[j], f0[j / 2]), b, acc0, 0, 0, 0);
        acc1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(gv_decode(u1[j], f1[j / 2]), b, acc1, 0, 0, 0);
      }
    }
    red[wave][0][lane] = acc0;
    red[wave][1][lane] = acc1;
    __syncthreads();
    if (tid < (ACT ? 64 : 128) && m0 + ln < c) {
      const int t = ACT ? 0 : wave;
      const int64_t o = (int64_t)row * a.N;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t n = n0 + 16 * t + 4 * g + i;
        if (n >= a.N) break;
        float v = (red[0][t][lane][i] + red[1][t][lane][i]) +
                  (red[2][t][lane][i] + red[3][t][lane][i]);
        v *= a.wo[((int64_t)e * NW + n) / a.rps];
        if constexpr (ACT) {
          float u = (red[0][1][lane][i] + red[1][1][lane][i]) +
                    (red[2][1][lane][i] + red[3][1][lane][i]);
          u *= a.wo[((int64_t)e * NW + a.N + n) / a.rps];
          v = swiglu_f32(v, u, a.prob[row]);
        }
        if (OUTF32) static_cast<float *>(a.out)[o + n] = v;
        else static_cast<uint16_t *>(a.out)[o + n] = (uint16_t)pk_bf16_rne(v, 0.0f);
      }
    }
    __syncthreads();
  }
}

namespace {

hipError_t launch_gemv(const GemvArgs &a, bool act, bool f32, hipStream_t st) {
  const int per = act ? 16 : 32;
  // Fewer rows than experts: a workgroup row per row of ids.  Otherwise one
  // per expert, and one for the rows without an expert.
  const int byrow = a.rows < a.G;
  const dim3 grid((unsigned)((a.N + per - 1) / per), (unsigned)(byrow ? a.rows : a.G + 1));
  const size_t lds = (size_t)a.rows * sizeof(int);
  if (act)
    hipLaunchKernelGGL((k_gemv_nvfp4<true, false>), grid, dim3(256), lds, st, a, byrow);
  else if (f32)
    hipLaunchKernelGGL((k_gemv_nvfp4<false, true>), grid, dim3(256), lds, st, a, byrow);
  else
    hipLaunchKernelGGL((k_gemv_nvfp4<false, false>), grid, dim3(256), lds, st, a, byrow);
  return hipGetLastError();
}

bool al(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
pqm_status st_of(hipError_t e) { return e == hipSuccess ? PQM_OK : PQM_ERR_HIP; }

pqm_status gemv_check(const GemvArgs &a, int64_t rows, int64_t divisor, int64_t G, int64_t NW) {
  if (rows < 0 || rows > GEMV_MAX_ROWS || divisor < 1 || divisor > GEMV_MAX_ROWS || G < 1 ||
      G > 4096)
    return PQM_ERR_SHAPE;
  if (a.N < 0 || a.N > (1 << 20) || a.K < 32 || a.K > (1 << 20) || a.K % 32) return PQM_ERR_SHAPE;
  if (a.rps < 1 || (G * NW) % a.rps) return PQM_ERR_SHAPE;
  if (rows == 0 || a.N == 0) return PQM_OK;
  if (!a.x || !a.ids || !a.w || !a.ws || !a.wo || !a.out) return PQM_ERR_NULL;
  if (!al(a.x, 16) || !al(a.w, 16) || !al(a.out, 16) || !al(a.ids, 4) || !al(a.ws, 4) ||
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
  const GemvArgs a = {x, ids, (int)rows, (int)divisor, w_q, w_scale, w_outer, w_rows_per_scale,
                      (int)G, N, K, nullptr, out};
  const pqm_status bad = gemv_check(a, rows, divisor, G, N);
  if (bad != PQM_OK || rows == 0 || N == 0) return bad;
  return st_of(launch_gemv(a, false, out_dtype == PQM_OUT_FP32, stream));
}

pqm_status pqm_moe_gemv_swiglu_nvfp4(const uint16_t *x, const int32_t *ids, const float *prob,
                                     int64_t rows, int64_t divisor, const uint8_t *w_q,
                                     const uint8_t *w_scale, const float *w_outer,
                                     int64_t w_rows_per_scale, int64_t G, int64_t inter, int64_t K,
                                     uint16_t *d, hipStream_t stream) {
  using namespace pqm;
  const GemvArgs a = {x, ids, (int)rows, (int)divisor, w_q, w_scale, w_outer, w_rows_per_scale,
                      (int)G, inter, K, prob, d};
  const pqm_status bad = gemv_check(a, rows, divisor, G, 2 * inter);
  if (bad != PQM_OK || rows == 0 || inter == 0) return bad;
  if (!prob) return PQM_ERR_NULL;
  return st_of(launch_gemv(a, true, false, stream));
}

}  // extern "C"
