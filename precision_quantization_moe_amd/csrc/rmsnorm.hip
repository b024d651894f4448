// rmsnorm.hip -- the norm in front of an expert layer: residual addition, RMS
// norm and the row-wise MXFP8 encoding of its output in one pass, and the
// gradients of that norm.
//
// Forward, one row of C values:  s = bf16(x + r);  rstd = 1 / sqrt(mean(s^2) +
// eps);  y = bf16(s rstd w);  (q, E8M0) = MXFP8 1x32 blocks of y.  The sum is
// rounded first because that rounded sum is what the residual stream carries
// on and what the backward pass reads again; y is rounded to bf16 before the
// encoding, so that the bytes are those of pqm_quantize_mxfp8 of the y that a
// caller may keep.  The sum of squares and the root are binary64 (no square
// overflows, and their cost hides behind the loads), and a binary32 product that
// lies within its own error of the middle of two bf16 values is formed again in
// binary64, and so is one whose factors may be subnormal: y is the nearest bf16
// value.
//
// Backward (straight through both roundings), g = dy w, h = s rstd:
//   dx = rstd (g - h mean(g h)) + d_sum,   dw_c = sum over rows of dy h.
#include "norm_device.hpp"
#include "pqm_device.hpp"
#include "pqm_internal.hpp"
#include "pqmoe.h"

namespace pqm {

namespace {

typedef uint32_t nb_u4 __attribute__((ext_vector_type(4)));
typedef uint32_t nb_u2 __attribute__((ext_vector_type(2)));

// A store or load that streams past the caches, or an ordinary one.
template <bool STREAM, typename V>
__device__ __forceinline__ void put(void *p, V v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, static_cast<V *>(p));
  else *static_cast<V *>(p) = v;
}

template <bool STREAM>
__device__ __forceinline__ nb_u4 get(const uint16_t *p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const nb_u4 *>(p));
  else return *reinterpret_cast<const nb_u4 *>(p);
}

// Sum over the TPR threads of a row (64: one wave; 256: the workgroup, through
// `red`, 4 slots).  Every thread of the workgroup must call it.
template <int TPR>
__device__ __forceinline__ double row_sum(double v, double *red) {
  v = wave_sum(v);
  if constexpr (TPR == 64) return v;
  __syncthreads();  // the slots' last readers are done
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// Smaller halves of a and of b's bf16 magnitudes, each as twice its bits less
// one (0 becomes the largest): three packed instructions for two values.
__device__ __forceinline__ uint32_t low_magnitudes(uint32_t a, uint32_t b) {
  const pqm_us2 v = __builtin_bit_cast(pqm_us2, b) * (uint16_t)2 + (uint16_t)0xFFFF;
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(pqm_us2, a), v));
}

// The same of the magnitude below which v rstd may be subnormal in binary32
// (with a subnormal rstd: all but 0), where a product keeps fewer bits than
// to_middle counts on.  From the exponents: v rstd >= 2^-126 where the two
// fields add up to 128 and v is normal.
__device__ __forceinline__ uint32_t short_products(float rstd) {
  const int e = (int)(__float_as_uint(rstd) >> 23);
  return e == 0 ? 0xFFFFu : (uint32_t)max(1, 128 - e) << 8;
}

// At most 6 where v, nearest but for 3 units in the last place, is so close to
// the middle of two bf16 values that those units may decide.
__device__ __forceinline__ uint16_t to_middle(float v) {
  return (uint16_t)((uint16_t)__float_as_uint(v) + (uint16_t)0x8003);
}

}  // namespace

// One row per TPR threads, NC chunks of 8 values per thread, kept in registers
// between the sum of squares and the scaling, so each input is read once.
// `sum` may be x or r itself: a thread reads what it overwrites before it does.
// Bound by memory: 16384 x 2048 with residual, 235 MB, 41.3 us (5.7 TB/s; a copy
// here moves 5.1); 8 x 2048 by latency, 4.6 us (an empty launch: 1.6).  The
// binary64 sum, root and middles cost 0.1 us there and 0.5 for 256 to 2048 rows;
// the look for factors that may be subnormal 0.13 for 8 rows and nothing for
// 16384.
template <int TPR, int NC, bool WF32, bool STREAM>
__global__ __launch_bounds__(256) void k_rmsnorm_quant(
    const uint16_t *x, int64_t ldx, const uint16_t *r, int64_t ldr, const void *__restrict__ w,
    int64_t rows, int64_t C, double inv_c, float eps, uint16_t *sum, uint16_t *__restrict__ y,
    uint8_t *__restrict__ q, uint8_t *__restrict__ s, float *__restrict__ rstd_out) {
  __shared__ double red[4];
  const int l = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  const bool live = row < rows;  // with 64 threads a row: the last workgroup's spare waves
  uint32_t v[NC][4];
  uint32_t low = 0xFFFFFFFFu;  // of this thread's smallest magnitudes but 0
  double sq = 0.0;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t c = ((int64_t)i * TPR + l) * 8;
    uint4 a = make_uint4(0, 0, 0, 0);
    if (live && c < C) {
      a = *reinterpret_cast<const uint4 *>(x + row * ldx + c);
      if (r) {
        const nb_u4 b = get<STREAM>(r + row * ldr + c);
        a.x = pk_bf16_rne(bf16_lo_f32(a.x) + bf16_lo_f32(b[0]), bf16_hi_f32(a.x) + bf16_hi_f32(b[0]));
        a.y = pk_bf16_rne(bf16_lo_f32(a.y) + bf16_lo_f32(b[1]), bf16_hi_f32(a.y) + bf16_hi_f32(b[1]));
        a.z = pk_bf16_rne(bf16_lo_f32(a.z) + bf16_lo_f32(b[2]), bf16_hi_f32(a.z) + bf16_hi_f32(b[2]));
        a.w = pk_bf16_rne(bf16_lo_f32(a.w) + bf16_lo_f32(b[3]), bf16_hi_f32(a.w) + bf16_hi_f32(b[3]));
      }
    }
    v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      low = low_magnitudes(low, v[i][j]);
      const double lo = bf16_lo_f32(v[i][j]), hi = bf16_hi_f32(v[i][j]);
      sq = __builtin_fma(lo, lo, sq);
      sq = __builtin_fma(hi, hi, sq);
    }
  }
  if (sum) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t c = ((int64_t)i * TPR + l) * 8;
      if (live && c < C)
        put<STREAM>(sum + row * C + c, nb_u4{v[i][0], v[i][1], v[i][2], v[i][3]});
    }
  }
  const double total = row_sum<TPR>(sq, red);
  const double root = inverse_root(total * inv_c + eps);  // no square of bf16 leaves binary64
  const float rstd = (float)root;
  const bool all_close = min(low & 0xFFFFu, low >> 16) < short_products(rstd);
  if (!live) return;
  if (rstd_out && l == 0) rstd_out[row] = rstd;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t c = ((int64_t)i * TPR + l) * 8;
    if (c >= C) continue;  // whole quads: C is a multiple of 32 where q is written
    float wf[8];
    load_w8<WF32>(w, c, wf);
    float f[8];
    uint16_t close = 0xFFFF;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[j] = (j & 1 ? bf16_hi_f32(v[i][j / 2]) : bf16_lo_f32(v[i][j / 2])) * rstd * wf[j];
      close = min(close, to_middle(f[j]));
    }
    if (close <= 6 || all_close) {  // one lane in a thousand; all eight, which keeps the code short
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t u = v[i][j / 2];
        asm("" : "+v"(u));  // or the sum's conversions would be kept for here, 16 registers a chunk
        f[j] = before_bf16((double)(j & 1 ? bf16_hi_f32(u) : bf16_lo_f32(u)) * (double)wf[j] * root);
      }
    }
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = pk_bf16_rne(f[2 * j], f[2 * j + 1]);
    if (y) put<STREAM>(y + row * C + c, nb_u4{o[0], o[1], o[2], o[3]});
    if (q) {
      uint32_t mm = pk_max_u16(pk_max_u16(o[0] & 0x7FFF7FFFu, o[1] & 0x7FFF7FFFu),
                               pk_max_u16(o[2] & 0x7FFF7FFFu, o[3] & 0x7FFF7FFFu));
      mm = max(mm & 0xFFFFu, mm >> 16);
      mm = max(mm, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mm, 0xB1, 0xF, 0xF, false));
      mm = max(mm, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mm, 0x4E, 0xF, 0xF, false));
      const uint32_t b = mx_scale_byte(mm);
      const float scale = __uint_as_float(b << 23);
      put<STREAM>(q + row * C + c,
                  nb_u2{cvt4_e4m3_bf16(o[0], o[1], scale), cvt4_e4m3_bf16(o[2], o[3], scale)});
      if ((threadIdx.x & 3) == 0) s[row * (C / 32) + c / 32] = (uint8_t)b;
    }
  }
}

// Gradients.  One workgroup a CU takes rows blockIdx.x, + gridDim.x, ... (four
// at a time with one wave a row); a thread owns the same columns of every row,
// so dw's sums and the weights stay in registers, and the sums leave once, as
// the workgroup's row of `part`.  The next row's loads go out before the
// current row is reduced.  Rows are read and written as buffers of their own
// length: past their end reads give 0 and writes are dropped, and a row that
// is none is an empty buffer.
//
// Bound by memory: 16384 x 2048 with d_sum, 268 MB, 48.5 us with k_rmsnorm_dw's
// 4 (5.5 TB/s; a copy here moves 5.1).  70 us without the next row in flight and
// with weights read again for every row; two workgroups a CU, whose sums are
// twice the bytes, 2 us more.  1021 x 7168: 18 us, half of it the start of two
// kernels and their sums of dw.
template <int TPR, int NC, bool WF32, bool STREAM>
__global__ __launch_bounds__(TPR == 512 ? 512 : 256, 2) void k_rmsnorm_backward(
    const uint16_t *__restrict__ dy, const uint16_t *__restrict__ sx, const void *__restrict__ w,
    const float *__restrict__ rstd, const uint16_t *dsum, int64_t rows, int64_t C, uint16_t *dx,
    float *__restrict__ part) {
  constexpr int RPB = TPR == 64 ? 4 : 1, WAVES = TPR == 512 ? 8 : 4;
  extern __shared__ float lds[];  // [4][C] with one wave a row
  __shared__ float red[2][WAVES];
  const int l = threadIdx.x % TPR;
  const int sub = RPB == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
  const int64_t step = (int64_t)gridDim.x * RPB;
  struct Row {
    nb_u4 g[NC], s[NC], d[NC];
    float rs;
  };
  const auto buffer = [&](const uint16_t *p, int64_t row) {
    const bool in = p && row < rows;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(p) + (in ? row * C : 0), (short)0,
                                             in ? (int)(2 * C) : 0, 0x00020000);
  };
  const auto load = [&](Row &r, int64_t row) {
    const __amdgpu_buffer_rsrc_t g = buffer(dy, row), s = buffer(sx, row), d = buffer(dsum, row);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int o = (i * TPR + l) * 16;
      r.g[i] = __builtin_amdgcn_raw_buffer_load_b128(g, o, 0, STREAM ? 2 : 0);
      r.s[i] = __builtin_amdgcn_raw_buffer_load_b128(s, o, 0, STREAM ? 2 : 0);
      r.d[i] = __builtin_amdgcn_raw_buffer_load_b128(d, o, 0, STREAM ? 2 : 0);
    }
    r.rs = row < rows ? rstd[row] : 0.0f;
  };
  // the weights of this thread's columns, kept as they are stored
  const __amdgpu_buffer_rsrc_t wb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<void *>(w), (short)0, (int)(C * (WF32 ? 4 : 2)), 0x00020000);
  nb_u4 wr[NC][WF32 ? 2 : 1];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int h = 0; h < (WF32 ? 2 : 1); ++h)
      wr[i][h] = __builtin_amdgcn_raw_buffer_load_b128(wb, (i * TPR + l) * (WF32 ? 32 : 16) + 16 * h,
                                                       0, 0);
  const auto weight = [&](int i, int j) {
    if constexpr (WF32) return __uint_as_float(wr[i][j / 4][j % 4]);
    else return j & 1 ? bf16_hi_f32(wr[i][0][j / 2]) : bf16_lo_f32(wr[i][0][j / 2]);
  };
  float acc[NC][8] = {};
  const auto use = [&](const Row &r, int64_t row, int turn) {
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = j & 1 ? bf16_hi_f32(r.g[i][j / 2]) : bf16_lo_f32(r.g[i][j / 2]);
        const float h = (j & 1 ? bf16_hi_f32(r.s[i][j / 2]) : bf16_lo_f32(r.s[i][j / 2])) * r.rs;
        const float t = d * h;
        acc[i][j] += t;
        dot += t * weight(i, j);
      }
    }
    dot = wave_sum(dot);
    if constexpr (TPR != 64) {  // two sets of slots: one barrier a row
      if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = dot;
      __syncthreads();
      dot = 0.0f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) dot += red[turn][i];
    }
    const float m = dot / (float)C;
    const __amdgpu_buffer_rsrc_t out = buffer(dx, row);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      nb_u4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float lo = r.rs * (bf16_lo_f32(r.g[i][j]) * weight(i, 2 * j) - bf16_lo_f32(r.s[i][j]) * r.rs * m);
        const float hi =
            r.rs * (bf16_hi_f32(r.g[i][j]) * weight(i, 2 * j + 1) - bf16_hi_f32(r.s[i][j]) * r.rs * m);
        o[j] = pk_bf16_rne(lo + bf16_lo_f32(r.d[i][j]), hi + bf16_hi_f32(r.d[i][j]));
      }
      // streaming (2): 16384 x 2048 53.5 -> 51.7 us, 1021 x 7168 19.2 -> 18.4
      __builtin_amdgcn_raw_buffer_store_b128(o, out, (i * TPR + l) * 16, 0, 2);
    }
  };
  const int64_t first = (int64_t)blockIdx.x * RPB;  // every wave takes the same turns
  Row a, b;
  load(a, first + sub);
  for (int64_t r0 = first; r0 < rows; r0 += 2 * step) {
    load(b, r0 + step + sub);
    use(a, r0 + sub, 0);
    if (r0 + step >= rows) break;
    load(a, r0 + 2 * step + sub);
    use(b, r0 + step + sub, 1);
  }
  if constexpr (TPR != 64) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t c = ((int64_t)i * TPR + l) * 8;
      if (c >= C) continue;
      float *p = part + blockIdx.x * C + c;
      *reinterpret_cast<float4 *>(p) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      *reinterpret_cast<float4 *>(p + 4) = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t c = ((int64_t)i * TPR + l) * 8;
      if (c >= C) continue;
      float *p = lds + sub * C + c;
      *reinterpret_cast<float4 *>(p) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      *reinterpret_cast<float4 *>(p + 4) = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
    __syncthreads();
    for (int64_t c = threadIdx.x; c < C; c += 256)
      part[blockIdx.x * C + c] = (lds[c] + lds[C + c]) + (lds[2 * C + c] + lds[3 * C + c]);
  }
}

// dw = sum of the P rows of part, always in the same order: 16 columns x 64
// row groups a workgroup, eight rows of a group in flight, the groups' sums
// joined through LDS.
__global__ __launch_bounds__(1024) void k_rmsnorm_dw(const float *__restrict__ part, int64_t P,
                                                     int64_t C, float *__restrict__ dw) {
  __shared__ float sh[64][17];
  const int col = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * 16 + col;
  float a[8] = {};
  if (c < C)
    for (int64_t p0 = grp; p0 < P; p0 += 512) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t p = p0 + 64 * i;
        a[i] += p < P ? part[p * C + c] : 0.0f;
      }
    }
  sh[grp][col] = ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
  __syncthreads();
  for (int w = 32; w > 0; w >>= 1) {
    if (grp < w) sh[grp][col] += sh[grp + w][col];
    __syncthreads();
  }
  if (grp == 0 && c < C) dw[c] = sh[0][col];
}

namespace {

constexpr int64_t NORM_MAX_COLS = 16384;  // 8 chunks of 8 values for each of 256 threads

// Workgroups of the backward kernel, i.e. rows of its partial sums of dw.
int64_t norm_backward_groups(int64_t rows, int64_t C) {
  const int64_t per = C <= 2048 ? 4 : 1;
  const int64_t g = (rows + per - 1) / per;
  return g < 256 ? g : 256;
}

template <int TPR, int NC>
hipError_t go_quant(bool wf32, const uint16_t *x, int64_t ldx, const uint16_t *r, int64_t ldr,
                    const void *w, int64_t rows, int64_t C, float eps, uint16_t *sum, uint16_t *y,
                    uint8_t *q, uint8_t *s, float *rstd, hipStream_t st) {
  // Streaming from 2^21 values on.  The stores: 16384 x 2048 with residual 51 ->
  // 47 us, 4096 x 7168 47 -> 42.6, 2048 x 2048 9.3 -> 8.1, 1024 x 2048 7.5 -> 7.0,
  // 256 x 2048 5.6 -> 5.9; with a gather that reads q and y afterwards the sum of
  // the two stays within 4 % either way.  The residual, which a layer before
  // wrote: 16384 x 2048 47.7 -> 41.7 with nothing in the caches; after a kernel that
  // wrote x, 1024 to 32768 rows, its time included, within 1 % either way (all of
  // it still in a cache: 2048 x 2048 6.3 -> 8.3).  x itself streamed as well took
  // 44.2.
  const bool stream = rows * C >= (1 << 21);
  const auto kernel = wf32 ? stream ? k_rmsnorm_quant<TPR, NC, true, true>
                                    : k_rmsnorm_quant<TPR, NC, true, false>
                           : stream ? k_rmsnorm_quant<TPR, NC, false, true>
                                    : k_rmsnorm_quant<TPR, NC, false, false>;
  // a grid has fewer than 2^32 threads: at most 2^23 workgroups a launch
  constexpr int64_t RPB = 256 / TPR, most = RPB << 23;
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    const int64_t n = rows - r0 < most ? rows - r0 : most, o = r0 * C;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((n + RPB - 1) / RPB)), dim3(256), 0, st,
                       x + r0 * ldx, ldx, r ? r + r0 * ldr : r, ldr, w, n, C, 1.0 / (double)C, eps,
                       sum ? sum + o : sum, y ? y + o : y, q ? q + o : q, s ? s + o / 32 : s,
                       rstd ? rstd + r0 : rstd);
  }
  return hipGetLastError();
}

template <int TPR, int NC>
hipError_t go_back(bool wf32, const uint16_t *dy, const uint16_t *x, const void *w,
                   const float *rstd, const uint16_t *dsum, int64_t rows, int64_t C, uint16_t *dx,
                   float *part, hipStream_t st) {
  const dim3 grid((unsigned)norm_backward_groups(rows, C));
  const size_t lds = TPR == 64 ? 4 * C * sizeof(float) : 0;
  const dim3 block(TPR == 512 ? 512 : 256);
  // Streaming loads once the four tensors (2^25 values: 268 MB) outgrow the 256
  // MB of the last cache.  Streaming against not, after a kernel that wrote dy,
  // its time included (us): 16384 x 2048 63.5 / 66.3, 8192 x 7168 114 / 123, 32768
  // x 2048 120 / 150; with nothing in the caches 16384 x 2048 48.5 / 51.8; below,
  // 4096 x 2048 15.9 / 15.7, 1024 x 7168 21.2 / 18.2.
  const bool stream = rows * C >= (1 << 25);
  const auto kernel = wf32 ? stream ? k_rmsnorm_backward<TPR, NC, true, true>
                                    : k_rmsnorm_backward<TPR, NC, true, false>
                           : stream ? k_rmsnorm_backward<TPR, NC, false, true>
                                    : k_rmsnorm_backward<TPR, NC, false, false>;
  hipLaunchKernelGGL(kernel, grid, block, lds, st, dy, x, w, rstd, dsum, rows, C, dx, part);
  return hipGetLastError();
}

// One wave a row up to 2048 columns (no barrier between a row's sum and its
// use), the workgroup a row beyond (a wave would hold over 32 values a lane
// of each tensor).  The gradients hold two rows of three tensors, the weights
// and dw's sums: at most four chunks a thread, hence 512 threads from 4097
// columns on (1021 x 7168: 18.0 us, with 256 threads 17.9; 16384 columns
// would spill 124 registers).
#define PQM_NORM_PICK(FN, ...)                               \
  (C <= 512     ? FN<64, 1>(__VA_ARGS__)                     \
   : C <= 1024  ? FN<64, 2>(__VA_ARGS__)                     \
   : C <= 2048  ? FN<64, 4>(__VA_ARGS__)                     \
   : C <= 4096  ? FN<256, 2>(__VA_ARGS__)                    \
   : C <= 8192  ? FN<256, 4>(__VA_ARGS__)                    \
                : FN<256, 8>(__VA_ARGS__))
#define PQM_NORM_BACK_PICK(FN, ...)                          \
  (C <= 512     ? FN<64, 1>(__VA_ARGS__)                     \
   : C <= 1024  ? FN<64, 2>(__VA_ARGS__)                     \
   : C <= 2048  ? FN<64, 4>(__VA_ARGS__)                     \
   : C <= 4096  ? FN<256, 2>(__VA_ARGS__)                    \
   : C <= 8192  ? FN<512, 2>(__VA_ARGS__)                    \
                : FN<512, 4>(__VA_ARGS__))

bool al(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
pqm_status st_of(hipError_t e) { return e == hipSuccess ? PQM_OK : PQM_ERR_HIP; }

}  // namespace
}  // namespace pqm

extern "C" {

pqm_status pqm_rmsnorm_quantize_mxfp8(const uint16_t *x, int64_t ldx, const uint16_t *residual,
                                      int64_t ldr, const void *weight, pqm_dtype weight_dtype,
                                      int64_t rows, int64_t cols, float eps, uint16_t *sum,
                                      uint16_t *y, uint8_t *q, uint8_t *s, float *rstd,
                                      hipStream_t stream) {
  using namespace pqm;
  if (weight_dtype != PQM_OUT_BF16 && weight_dtype != PQM_OUT_FP32) return PQM_ERR_ENUM;
  if (rows < 0 || cols < 0 || cols % 8 || cols > NORM_MAX_COLS || rows >= ((int64_t)1 << 31))
    return PQM_ERR_SHAPE;
  if (ldx < cols || (residual && ldr < cols)) return PQM_ERR_SHAPE;
  if ((q || s) && cols % 32) return PQM_ERR_SHAPE;
  // in place only where the rows of sum lie where they were read
  if (sum && ((sum == x && ldx != cols) || (sum == residual && ldr != cols))) return PQM_ERR_SHAPE;
  if (!(eps >= 0x1p-100f) || !(eps < __builtin_inff())) return PQM_ERR_SHAPE;
  if (rows == 0 || cols == 0) return PQM_OK;
  if (!x || !weight || (!q && !y) || (q == nullptr) != (s == nullptr)) return PQM_ERR_NULL;
  if (!al(x, 16) || ldx % 8 || !al(weight, 16) || !al(sum, 16) || !al(y, 16) || !al(q, 8) ||
      !al(rstd, 4))
    return PQM_ERR_ALIGN;
  if (residual && (!al(residual, 16) || ldr % 8)) return PQM_ERR_ALIGN;
  const int64_t C = cols;
  return st_of(PQM_NORM_PICK(go_quant, weight_dtype == PQM_OUT_FP32, x, ldx, residual, ldr, weight,
                             rows, C, eps, sum, y, q, s, rstd, stream));
}

size_t pqm_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || rows >= ((int64_t)1 << 31) || cols <= 0 || cols > pqm::NORM_MAX_COLS) return 0;
  return (size_t)(pqm::norm_backward_groups(rows, cols) * cols) * sizeof(float);
}

pqm_status pqm_rmsnorm_backward(const uint16_t *dy, const uint16_t *x, const void *weight,
                                pqm_dtype weight_dtype, const float *rstd, const uint16_t *d_sum,
                                int64_t rows, int64_t cols, uint16_t *dx, float *dweight,
                                void *workspace, size_t workspace_bytes, hipStream_t stream) {
  using namespace pqm;
  if (weight_dtype != PQM_OUT_BF16 && weight_dtype != PQM_OUT_FP32) return PQM_ERR_ENUM;
  if (rows < 0 || cols < 0 || cols % 8 || cols > NORM_MAX_COLS || rows >= ((int64_t)1 << 31))
    return PQM_ERR_SHAPE;
  if (cols == 0) return PQM_OK;
  if (!dweight || (rows > 0 && (!dy || !x || !weight || !rstd || !dx || !workspace)))
    return PQM_ERR_NULL;
  if (workspace_bytes < pqm_rmsnorm_backward_workspace(rows, cols)) return PQM_ERR_WORKSPACE;
  if (!al(dy, 16) || !al(x, 16) || !al(weight, 16) || !al(rstd, 4) || !al(d_sum, 16) ||
      !al(dx, 16) || !al(dweight, 4) || !al(workspace, 16))
    return PQM_ERR_ALIGN;
  const int64_t C = cols;
  float *part = static_cast<float *>(workspace);
  if (rows > 0) {
    const hipError_t e = PQM_NORM_BACK_PICK(go_back, weight_dtype == PQM_OUT_FP32, dy, x, weight, rstd,
                                       d_sum, rows, C, dx, part, stream);
    if (e != hipSuccess) return PQM_ERR_HIP;
  }
  // no rows: the sum over none of them is zero
  hipLaunchKernelGGL(k_rmsnorm_dw, dim3((unsigned)((C + 15) / 16)), dim3(1024), 0, stream, part,
                     rows > 0 ? norm_backward_groups(rows, C) : 0, C, dweight);
  return st_of(hipGetLastError());
}

}  // extern "C"
