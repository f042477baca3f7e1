// ops_rotary.hip -- rotary positions for queries and keys (include/lowm_cache.h)
// for gfx950.
//
//   a = pos freq ;  (x, y) -> scale (x cos a - y sin a, x sin a + y cos a)
//
// Elementwise but for the angles, which all heads of a token share: a thread owns 16
// elements of a token's heads, eight pairs or 16 that are only copied, forms their sines
// and cosines once and goes through heads with them.  Few heads to a thread cost
// arithmetic, many leave lanes idle (launch_rotary).  Bound by HBM (8192 tokens of 72 heads of
// 128, half of each turned: 66 to 71 us, 4.3 to 4.6 TB/s read and written, a large copy 5.0), one token by
// its chain of position, angle and sine (4.0 us).  The angle is taken modulo a turn in
// fp64, where position and frequency are exact to 2^-53, and goes to the fp32 sine in half
// turns.
#include "ops_cache.cuh"

namespace lowm {
namespace {

struct RotaryArgs {
  lowm_rotary_args u;
  int64_t first_token, tokens;   // of this launch
  int head_lanes;                // threads that share a token's heads
  int pair_groups, groups;       // of eight pairs; with those of 16 copied elements
};

// Eight (or, at the end of a stretch, n) elements.
template <bool F32, bool WHOLE>
__device__ __forceinline__ void take(const void* p, int64_t at, int n, float (&v)[8]) {
  if (WHOLE || n >= 8) {
    values8(load8(p, at, F32), F32, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? load1(p, at + i, F32) : 0.f;
  }
}
template <bool F32, bool WHOLE>
__device__ __forceinline__ void put(void* p, int64_t at, int n, const float (&v)[8]) {
  if (WHOLE || n >= 8) {
    store8(p, at, F32, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) store1(p, at + i, F32, v[i]);
  }
}

// WHOLE: every thread has all its 16 elements, so that a loop's loads do not wait for one
// another.
template <bool F32, bool HALF, bool WHOLE>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a) {
  const lowm_rotary_args& u = a.u;
  // (fewer than 2^31 threads to a launch)
  const uint32_t at = blockIdx.x * 256u + threadIdx.x;
  const uint32_t th = at / (uint32_t)a.groups, local = th / (uint32_t)a.head_lanes;
  const int g = (int)(at - th * a.groups), lane = (int)(th - local * a.head_lanes);
  if (local >= a.tokens) return;
  const int64_t t = a.first_token + local;
  const int heads = u.Hq + u.Hk, pairs = u.R / 2;

  // two runs of up to eight elements, at d0 and d1: n0 and n1 of them
  const bool turn = g < a.pair_groups;
  int d0, d1, n0, n1;
  float c[8], s[8];
  if (turn) {
    const int p0 = 8 * g, n = pairs - p0 < 8 ? pairs - p0 : 8;
    d0 = u.first + (HALF ? p0 : 2 * p0);
    d1 = HALF ? d0 + pairs : d0 + 8;
    n0 = HALF ? n : 2 * n;
    n1 = HALF ? n : 2 * n - 8;
    const double pos = u.positions_bytes == 8
                           ? (double)static_cast<const int64_t*>(u.positions)[t]
                           : (double)static_cast<const int32_t*>(u.positions)[t];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double half_turns = pos * u.freqs[p0 + (i < n ? i : 0)] * 0.31830988618379067154;
      const float part = (float)(half_turns - 2.0 * rint(0.5 * half_turns));
      float si, co;
      sincospif(part, &si, &co);
      c[i] = u.scale * co;
      s[i] = u.scale * (u.flags & LOWM_ROTARY_INVERSE ? -si : si);
    }
  } else {
    // those before the turned ones, then those behind them, groups of each apart
    const int before = (u.first + 15) / 16, k = g - a.pair_groups;
    d0 = k < before ? 16 * k : u.first + u.R + 16 * (k - before);
    d1 = d0 + 8;
    n0 = (k < before ? u.first : u.D) - d0;
    n1 = n0 - 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = s[i] = 0.f;
  }
  if (n0 > 8) n0 = 8;
  if (n1 > 8) n1 = 8;

#pragma unroll 4
  for (int h = lane; h < heads; h += a.head_lanes) {
    const bool q = h < u.Hq;
    const int i = q ? h : h - u.Hq;
    const void* x = q ? u.q : u.k;
    void* y = q ? u.q_out : u.k_out;
    const int64_t from = t * (q ? u.q_row : u.k_row) + i * (q ? u.q_head : u.k_head);
    const int64_t to = t * (q ? u.q_out_row : u.k_out_row) + i * (q ? u.q_out_head : u.k_out_head);
    float v[8], w[8], v2[8], w2[8];
    take<F32, WHOLE>(x, from + d0, n0, v);
    take<F32, WHOLE>(x, from + d1, n1, w);
    if (HALF) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v2[i] = v[i] * c[i] - w[i] * s[i];
        w2[i] = v[i] * s[i] + w[i] * c[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v2[2 * i] = v[2 * i] * c[i] - v[2 * i + 1] * s[i];
        v2[2 * i + 1] = v[2 * i] * s[i] + v[2 * i + 1] * c[i];
        w2[2 * i] = w[2 * i] * c[4 + i] - w[2 * i + 1] * s[4 + i];
        w2[2 * i + 1] = w[2 * i] * s[4 + i] + w[2 * i + 1] * c[4 + i];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v2[i] = turn ? v2[i] : v[i];
      w2[i] = turn ? w2[i] : w[i];
    }
    put<F32, WHOLE>(y, to + d0, n0, v2);
    put<F32, WHOLE>(y, to + d1, n1, w2);
  }
}

template <bool F32, bool HALF>
const void* kernel_for(bool whole) {
  return whole ? (const void*)&rotary_kernel<F32, HALF, true>
               : (const void*)&rotary_kernel<F32, HALF, false>;
}

// copy: whether what is not turned has to be copied (in place it is there).
int launch_rotary(RotaryArgs a, bool copy, hipStream_t stream) {
  const lowm_rotary_args& u = a.u;
  const int pairs = u.R / 2, heads = u.Hq + u.Hk, behind = u.D - u.first - u.R;
  a.pair_groups = (pairs + 7) / 8;
  a.groups = a.pair_groups + (copy ? (u.first + 15) / 16 + (behind + 15) / 16 : 0);
  const bool whole = pairs % 8 == 0 && (!copy || (u.first % 16 == 0 && behind % 16 == 0));
  // As many threads to a token's heads as fill the GPU with 16 wavefronts to a CU (8192
  // tokens of 72 heads, all of 128 elements turned: 72 us; with half as many 84).
  const int64_t per = (int64_t)u.T * a.groups;
  const int64_t lanes = (256 * 16 * kWave + per - 1) / per;
  a.head_lanes = (int)(lanes < heads ? lanes : heads);
  const bool half = !(u.flags & LOWM_ROTARY_INTERLEAVED);
  const void* fn = u.type == LOWM_F32
                       ? (half ? kernel_for<true, true>(whole) : kernel_for<true, false>(whole))
                       : (half ? kernel_for<false, true>(whole) : kernel_for<false, false>(whole));
  const int64_t threads = (int64_t)a.groups * a.head_lanes, most = kMaxThreads / threads;
  void* args[] = {&a};
  int rc = LOWM_OK;
  for (int64_t t = 0; t < u.T && rc == LOWM_OK; t += most) {
    a.first_token = t;
    a.tokens = u.T - t < most ? u.T - t : most;
    rc = launched(hipLaunchKernel(fn, dim3((unsigned)((a.tokens * threads + 255) / 256)),
                                  dim3(256), args, 0, stream));
  }
  return rc;
}

int rotary(const lowm_rotary_args* u, hipStream_t stream) {
  if (!u || u->T < 0 || u->Hq < 1 || u->D < 1 || u->R < 2 || u->R % 2 || u->first < 0 ||
      u->first > u->D - u->R || (u->k && u->Hk < 1))
    return LOWM_ERR_INVALID_ARG;
  if (u->type != LOWM_BF16 && u->type != LOWM_F32) return LOWM_ERR_INVALID_ARG;
  if (u->positions_bytes != 8 && u->positions_bytes != 4) return LOWM_ERR_INVALID_ARG;
  if (u->flags & ~(LOWM_ROTARY_INTERLEAVED | LOWM_ROTARY_INVERSE)) return LOWM_ERR_INVALID_ARG;
  if (u->D > LOWM_ROTARY_MAX_D || u->Hq > LOWM_CACHE_MAX_HEADS || u->Hk > LOWM_CACHE_MAX_HEADS)
    return LOWM_ERR_UNSUPPORTED;
  if (u->T == 0) return LOWM_OK;
  if (!u->q || !u->q_out || !u->positions || !u->freqs || (u->k && !u->k_out))
    return LOWM_ERR_INVALID_ARG;
  lowm_rotary_args v = *u;
  if (!v.k) {
    v.Hk = 0;
    v.k_out = nullptr;
    v.k_row = v.k_head = v.k_out_row = v.k_out_head = 0;
  }
  const int b = type_bytes(v.type);
  if (!aligned_to(v.q, b) || !aligned_to(v.k, b) || !aligned_to(v.q_out, b) ||
      !aligned_to(v.k_out, b) || !aligned_to(v.positions, v.positions_bytes) ||
      !aligned_to(v.freqs, 8))
    return LOWM_ERR_UNSUPPORTED;
  if (!heads_apart(v.T, v.Hq, v.D, v.q_row, v.q_head) ||
      !heads_apart(v.T, v.Hq, v.D, v.q_out_row, v.q_out_head) ||
      (v.k && (!heads_apart(v.T, v.Hk, v.D, v.k_row, v.k_head) ||
               !heads_apart(v.T, v.Hk, v.D, v.k_out_row, v.k_out_head))))
    return LOWM_ERR_INVALID_ARG;
  const bool q_in = v.q == v.q_out && v.q_row == v.q_out_row && v.q_head == v.q_out_head;
  const bool k_in = v.k && v.k == v.k_out && v.k_row == v.k_out_row && v.k_head == v.k_out_head;
  const Heads q{v.q, v.T, v.Hq, v.D, v.q_row, v.q_head, b},
      qo{v.q_out, v.T, v.Hq, v.D, v.q_out_row, v.q_out_head, b},
      k{v.k, v.T, v.Hk, v.D, v.k_row, v.k_head, b},
      ko{v.k_out, v.T, v.Hk, v.D, v.k_out_row, v.k_out_head, b};
  const Span pos = span_of(v.positions, 1, v.T, v.T, v.positions_bytes),
             fr = span_of(v.freqs, 1, v.R / 2, v.R / 2, 8);
  if ((!q_in && meet(qo, q)) || (!k_in && meet(ko, k)) || meet(qo, k) || meet(ko, q) ||
      meet(qo, ko) || meet(qo, pos) || meet(qo, fr) || meet(ko, pos) || meet(ko, fr))
    return LOWM_ERR_INVALID_ARG;
  RotaryArgs a{};
  a.u = v;
  return launch_rotary(a, !q_in || (v.k && !k_in), stream);
}

}  // namespace
}  // namespace lowm

extern "C" int lowm_rotary(const lowm_rotary_args* args, void* stream) {
  return lowm::rotary(args, static_cast<hipStream_t>(stream));
}
