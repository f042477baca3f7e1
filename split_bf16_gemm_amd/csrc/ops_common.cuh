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

// A launch has fewer than 2^32 threads; more rows than fit go in several, each of
// at most this many.
constexpr int64_t kMaxThreads = 1ll << 31;

// Bytes [lo, hi) of a [rows, cols] array whose rows, `width` bytes each, start
// `ld` elements, `pitch` bytes, apart.
struct Span {
  uintptr_t lo, hi, pitch, width;
};
inline Span span_of(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
  const uintptr_t lo = (uintptr_t)p;
  return {lo, p ? lo + (uintptr_t)(((rows - 1) * ld + cols) * elem) : lo, (uintptr_t)(ld * elem),
          (uintptr_t)(cols * elem)};
}
// Whether two arrays share a byte.  Rows of one pitch may lie between one another,
// as column ranges of one buffer do; of two pitches the whole spans are compared.
inline bool meet(const Span& a, const Span& b) {
  if (a.lo >= b.hi || b.lo >= a.hi) return false;
  if (a.pitch != b.pitch || a.pitch == 0) return true;
  const Span &first = a.lo <= b.lo ? a : b, &other = a.lo <= b.lo ? b : a;
  const uintptr_t off = (other.lo - first.lo) % a.pitch;
  return off < first.width || off + other.width > a.pitch;
}

inline int type_bytes(int type) { return type == LOWM_F32 ? 4 : type == LOWM_BF16 ? 2 : 1; }

typedef uint32_t ops_u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t ops_u32x2 __attribute__((ext_vector_type(2)));

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

// Vectors at any address (the GPU's unaligned access): rows of an odd length or
// pitch start anywhere.
struct __attribute__((packed, aligned(1))) AnyU32x4 {
  ops_u32x4 v;
};
struct __attribute__((packed, aligned(1))) AnyU32x2 {
  ops_u32x2 v;
};

// Eight consecutive elements as they lie in memory; their values are taken out
// later, so that a kernel's loads do not wait for one another in the branches on
// its operands' types.
struct Raw8 {
  ops_u32x4 a, b;
};
__device__ __forceinline__ Raw8 load8(const void* base, int64_t at, bool f32) {
  Raw8 r;
  if (f32) {
    const AnyU32x4* p = reinterpret_cast<const AnyU32x4*>(static_cast<const float*>(base) + at);
    r.a = p[0].v;
    r.b = p[1].v;
  } else {
    r.a = reinterpret_cast<const AnyU32x4*>(static_cast<const uint16_t*>(base) + at)->v;
    r.b = ops_u32x4{0u, 0u, 0u, 0u};
  }
  return r;
}
__device__ __forceinline__ void values8(const Raw8& r, bool f32, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = r.a[i], b = r.b[i];
    v[i] = __builtin_bit_cast(float, a);
    v[4 + i] = __builtin_bit_cast(float, b);
  }
  if (!f32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = r.a[i];
      v[2 * i] = bf16_lo(w);
      v[2 * i + 1] = bf16_hi(w);
    }
  }
}
__device__ __forceinline__ float load1(const void* base, int64_t at, bool f32) {
  return f32 ? static_cast<const float*>(base)[at]
             : bf16_lo(static_cast<const uint16_t*>(base)[at]);
}
__device__ __forceinline__ void store8(void* base, int64_t at, bool f32, const float (&v)[8]) {
  if (f32) {
    AnyU32x4* p = reinterpret_cast<AnyU32x4*>(static_cast<float*>(base) + at);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      ops_u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(uint32_t, v[4 * h + i]);
      p[h].v = w;
    }
  } else {
    ops_u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    reinterpret_cast<AnyU32x4*>(static_cast<uint16_t*>(base) + at)->v = w;
  }
}
__device__ __forceinline__ void store1(void* base, int64_t at, bool f32, float v) {
  if (f32)
    static_cast<float*>(base)[at] = v;
  else
    static_cast<__bf16*>(base)[at] = static_cast<__bf16>(v);
}

// Reductions over the wavefront by data-parallel moves within the vector unit
// (four shifts within rows of 16 lanes, then two broadcasts across rows); lanes
// a move does not reach take the operation's neutral 0.  Every lane gets the
// result, the last lane's.  All 64 lanes must be active.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t lane_move(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
template <typename Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, Op op) {
  v = op(v, lane_move<0x111, 0xf>(v));   // row_shr 1, 2, 4, 8
  v = op(v, lane_move<0x112, 0xf>(v));
  v = op(v, lane_move<0x114, 0xf>(v));
  v = op(v, lane_move<0x118, 0xf>(v));
  v = op(v, lane_move<0x142, 0xa>(v));   // row_bcast 15 into rows 1 and 3
  v = op(v, lane_move<0x143, 0xc>(v));   // row_bcast 31 into rows 2 and 3
  return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}
__device__ __forceinline__ float wave_sum(float v) {
  return __builtin_bit_cast(
      float, wave_reduce(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(
            uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
      }));
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  return wave_reduce(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// fp32 bits as unsigned integers in the order of their values: -0 as +0, any
// NaN above +infinity; never 0.
__device__ __forceinline__ uint32_t order(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
  return x != x ? 0xffffffffu : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __builtin_bit_cast(float, o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

// A row's scale for int8 from the bits of its largest magnitude: a row of zeros
// has scale 0, one with an infinity or a NaN (whose bits are the greatest) scale
// NaN; the q of both are 0.
struct RowScale {
  float scale, recip;
  bool some;
  __device__ __forceinline__ explicit RowScale(uint32_t top) {
    const bool finite = top < 0x7f800000u;
    const float s = __builtin_bit_cast(float, top) / 127.0f;
    scale = finite ? s : __builtin_nanf("");
    some = finite && s > 0.f;
    // no reciprocal for a subnormal scale: its values all take the divide
    recip = s >= 1.17549435e-38f ? 1.0f / s : __builtin_nanf("");
  }
  // Four of rint(x / scale), as bytes, the divide correctly rounded so that q is
  // the same number on any machine.  x recip is within 127 * 2^-22 of the
  // quotient: away from the halves it rounds to the same integer, and next to one
  // the divide itself decides.  (Adding 1.5 * 2^23 rounds to an integer and leaves
  // it in the low bits.  A subnormal scale can be rounded far enough that a
  // quotient passes 127: such a value is held there.)
  __device__ __forceinline__ uint32_t quantise4(float x0, float x1, float x2, float x3) const {
    constexpr float kRound = 12582912.f;
    const float x[4] = {x0, x1, x2, x3};
    uint32_t b[4];
    bool clear = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float y = __builtin_fmaf(x[i], recip, kRound);
      clear = clear && fabsf(__builtin_fmaf(x[i], recip, kRound - y)) <= 0.4998f;
      b[i] = __builtin_bit_cast(uint32_t, y);
    }
    if (__builtin_expect(!clear, 0)) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        b[i] = some ? (uint32_t)(int)fminf(fmaxf(rintf(x[i] / scale), -127.f), 127.f) : 0u;
    }
    return (b[0] & 255u) | (b[1] & 255u) << 8 | (b[2] & 255u) << 16 | b[3] << 24;
  }
};

}  // namespace lowm
