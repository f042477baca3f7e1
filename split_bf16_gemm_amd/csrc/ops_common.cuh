// ops_common.cuh -- what the operators of include/lowm_ops.h share: typed row
// access, reductions over a wavefront or a group of wavefronts, and the host
// side of a launch.
#pragma once

#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "lowm_ops.h"
#include "lowm_types.h"

namespace lowm {

extern thread_local int g_last_hip_error;

// The result of a launch: the error code of the kernel that hipGetLastError
// reports, kept for lowm_last_hip_error().
inline int launched(hipError_t err) {
  if (err == hipSuccess) err = hipGetLastError();
  if (err == hipSuccess) return LOWM_OK;
  g_last_hip_error = (int)err;
  return LOWM_ERR_LAUNCH;
}

// Bytes [lo, hi) of a [rows, cols] array whose rows start `ld` elements apart.
struct Span {
  uintptr_t lo, hi;
};
inline Span span_of(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
  const uintptr_t lo = (uintptr_t)p;
  return {lo, p ? lo + (uintptr_t)(((rows - 1) * ld + cols) * elem) : lo};
}
inline bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

inline int type_bytes(int type) { return type == LOWM_F32 ? 4 : type == LOWM_BF16 ? 2 : 1; }

typedef uint32_t ops_u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t ops_u32x2 __attribute__((ext_vector_type(2)));
typedef float ops_f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) {
  return __builtin_bit_cast(float, w & 0xffff0000u);
}
// fp32 to bf16, round to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const uint16_t a = __builtin_bit_cast(uint16_t, static_cast<__bf16>(lo));
  const uint16_t b = __builtin_bit_cast(uint16_t, static_cast<__bf16>(hi));
  return (uint32_t)a | ((uint32_t)b << 16);
}

// Eight consecutive elements from 16-byte aligned memory.
__device__ __forceinline__ void load8(const void* base, int64_t at, bool f32, float (&v)[8]) {
  if (f32) {
    const ops_f32x4* p = reinterpret_cast<const ops_f32x4*>(static_cast<const float*>(base) + at);
    const ops_f32x4 a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    const ops_u32x4 a =
        *reinterpret_cast<const ops_u32x4*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(a[i]);
      v[2 * i + 1] = bf16_hi(a[i]);
    }
  }
}
__device__ __forceinline__ float load1(const void* base, int64_t at, bool f32) {
  return f32 ? static_cast<const float*>(base)[at]
             : bf16_lo(static_cast<const uint16_t*>(base)[at]);
}
__device__ __forceinline__ void store8(void* base, int64_t at, bool f32, const float (&v)[8]) {
  if (f32) {
    ops_f32x4* p = reinterpret_cast<ops_f32x4*>(static_cast<float*>(base) + at);
    p[0] = ops_f32x4{v[0], v[1], v[2], v[3]};
    p[1] = ops_f32x4{v[4], v[5], v[6], v[7]};
  } else {
    ops_u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<ops_u32x4*>(static_cast<uint16_t*>(base) + at) = w;
  }
}
__device__ __forceinline__ void store1(void* base, int64_t at, bool f32, float v) {
  if (f32)
    static_cast<float*>(base)[at] = v;
  else
    static_cast<__bf16*>(base)[at] = static_cast<__bf16>(v);
}

// Reductions over the wavefront; every lane gets the result.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) {
    const uint32_t o = __shfl_xor(v, off);
    v = o > v ? o : v;
  }
  return v;
}

}  // namespace lowm
