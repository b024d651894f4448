// gemv_device.hpp -- NVFP4 weights on their way to the matrix core, shared by
// the kernels that multiply a few rows.
#pragma once

#include "pqm_device.hpp"

namespace pqm {

namespace {

typedef __bf16 gv_bf8 __attribute__((ext_vector_type(8)));
typedef float gv_f4 __attribute__((ext_vector_type(4)));
typedef float gv_f2 __attribute__((ext_vector_type(2)));
typedef uint32_t gv_u4 __attribute__((ext_vector_type(4)));
typedef _Float16 gv_h2 __attribute__((ext_vector_type(2)));
typedef _Float16 gv_h8 __attribute__((ext_vector_type(8)));

constexpr uint32_t GV_NONE = 0x80000000u;  // an offset past every buffer below: reads give 0

__device__ __forceinline__ __amdgpu_buffer_rsrc_t gv_buffer(const void *p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, 0x00020000);
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

}  // namespace pqm
