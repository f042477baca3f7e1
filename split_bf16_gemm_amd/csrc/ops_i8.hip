// ops_i8.hip -- the int8 product of up to 64 rows (include/lowm_ops.h) for
// gfx950.
//
//   C[m][n] = (sum_k A[m][k] W[n][k]) a_scale[m] w_scale[n]
//
// The sum is exact (int8 products in int32), so no order of it changes a bit;
// it is scaled in fp32 and rounded once to the output's type.  Bound by HBM:
// the N K bytes of W are read once.  Each workgroup takes 16*NB rows of W, its
// wavefronts a stretch of K each (ops_stream.cuh), and adds their sums through
// LDS.
#include "ops_stream.cuh"

namespace lowm {

int quantize_rows(const void* x, int x_type, int64_t ld, int M, int K, void* q, float* scale,
                  hipStream_t stream);

struct I8Args {
  const uint8_t* A;
  const uint8_t* W;
  const float* a_scale;
  const float* w_scale;
  void* C;
  int M, N, K, f32;
};

template <int MB, int NB, int R>
struct I8Shape {
  using S = StreamShape<NB, MB, R>;
  static constexpr int kBlocks = NB * MB;
  static constexpr int kRings = kWaves * S::kRing * 16;                  // bytes
  static constexpr int kSums = kWaves * kBlocks * kWave * 16;
  static constexpr int lds_bytes = kRings > kSums ? kRings : kSums;
  static constexpr bool valid = (R - 1) * S::G <= 63 && lds_bytes <= 160 * 1024;
};

template <int MB, int NB, int R>
__global__ __launch_bounds__(kThreads) void gemm_i8_kernel(I8Args a) {
#if defined(__HIP_DEVICE_COMPILE__)
  using SH = I8Shape<MB, NB, R>;
  constexpr int G = SH::S::G;
  __shared__ u32x4 lds[SH::lds_bytes / 16];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int g = lane >> 4, l16 = lane & 15;
  const int n0 = blockIdx.x * 16 * NB;

  const int steps = (a.K + 127) / 128, per = (steps + kWaves - 1) / kWaves;
  const int s0 = wave * per;
  const int P = steps - s0 < per ? steps - s0 : per;
  const int k0 = s0 * 128 + stream_piece(lane) * 16;
  i32x4 acc[SH::kBlocks];
#pragma unroll
  for (int i = 0; i < SH::kBlocks; ++i) acc[i] = i32x4{0, 0, 0, 0};
  if (P > 0) {
    const uint8_t* src[G];
#pragma unroll
    for (int t = 0; t < G; ++t) {
      // rows past the end read the last row: their results are not stored
      int r = 8 * (t < 2 * NB ? t : t - 2 * NB) + stream_row(lane);
      if (t < 2 * NB) {
        r = n0 + r < a.N ? n0 + r : a.N - 1;
        src[t] = a.W + (size_t)r * a.K + k0;
      } else {
        r = r < a.M ? r : a.M - 1;
        src[t] = a.A + (size_t)r * a.K + k0;
      }
    }
    stream_tile<NB, MB, R>(lds + wave * SH::S::kRing, src, a.K - k0, P, acc);
  }
  stream_settle(acc);

  // Sum i of block q from wavefront w at sums[((w * kBlocks + q) * 64 + lane)][i].
  i32x4* sums = reinterpret_cast<i32x4*>(lds);
  __syncthreads();
#pragma unroll
  for (int q = 0; q < SH::kBlocks; ++q) sums[(wave * SH::kBlocks + q) * kWave + lane] = acc[q];
  __syncthreads();
#pragma unroll
  for (int q0 = 0; q0 < SH::kBlocks; q0 += kWaves) {
    const int q = q0 + wave;
    if (q >= SH::kBlocks) break;
    i32x4 v = sums[q * kWave + lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += sums[(w * SH::kBlocks + q) * kWave + lane];
    const int n = n0 + 16 * (q / MB) + l16;
    if (n >= a.N) continue;
    const float sw = a.w_scale[n];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = 16 * (q % MB) + 4 * g + i;
      if (m >= a.M) continue;
      const int sum = v[i];
      // int32 to fp32 rounds a sum past 2^24 by half a step of fp32.
      const float c = (float)sum * a.a_scale[m] * sw;
      const size_t at = (size_t)m * a.N + n;
      if (a.f32)
        static_cast<float*>(a.C)[at] = c;
      else
        static_cast<__bf16*>(a.C)[at] = static_cast<__bf16>(c);
    }
  }
#endif
}

namespace {

template <int MB, int NB>
const void* kernel_of() {
  constexpr int R = I8Shape<MB, NB, 4>::valid ? 4 : I8Shape<MB, NB, 3>::valid ? 3 : 2;
  static_assert(I8Shape<MB, NB, R>::valid, "the ring fits");
  return reinterpret_cast<const void*>(&gemm_i8_kernel<MB, NB, R>);
}
const void* pick_kernel(int MB, int NB) {
  static const void* const table[4][4] = {
      {kernel_of<1, 1>(), kernel_of<1, 2>(), kernel_of<1, 3>(), kernel_of<1, 4>()},
      {kernel_of<2, 1>(), kernel_of<2, 2>(), kernel_of<2, 3>(), kernel_of<2, 4>()},
      {kernel_of<3, 1>(), kernel_of<3, 2>(), kernel_of<3, 3>(), kernel_of<3, 4>()},
      {kernel_of<4, 1>(), kernel_of<4, 2>(), kernel_of<4, 3>(), kernel_of<4, 4>()}};
  return table[MB - 1][NB - 1];
}

// The width of 16..64 weight rows whose workgroups load the fewest rows in all:
// rounds of 256 workgroups (one per CU) times a step's rows.
int pick_width(int M, int N) {
  const int act = (M + 15) / 16;
  int best = 1;
  long best_cost = 0;
  for (int nb = 1; nb <= 4; ++nb) {
    const long tiles = ((long)N + 16 * nb - 1) / (16 * nb);
    const long cost = (tiles + 255) / 256 * (act + nb);
    if (nb == 1 || cost < best_cost) {
      best = nb;
      best_cost = cost;
    }
  }
  return best;
}

constexpr int64_t kI8MaxK = 131056;   // 128 * 128 * K stays below 2^31

size_t i8_workspace(int M, int N, int K) {
  if (M < 1 || M > LOWM_MAX_M || N < 1 || K < 1 || K % 16 || K > LOWM_QUANTIZE_MAX_K) return 0;
  return ((size_t)M * K + 255) / 256 * 256 + LOWM_MAX_M * sizeof(float);
}

int gemm_i8(const lowm_gemm_i8_args* u, hipStream_t stream) {
  if (!u || u->M < 1 || u->N < 1 || u->K < 1) return LOWM_ERR_INVALID_ARG;
  if (!u->A || !u->W || !u->w_scale || !u->C) return LOWM_ERR_INVALID_ARG;
  const bool quantised = u->a_type == LOWM_I8;
  if ((!quantised && u->a_type != LOWM_BF16) || (quantised && !u->a_scale) ||
      (u->c_type != LOWM_BF16 && u->c_type != LOWM_F32))
    return LOWM_ERR_INVALID_ARG;
  if (u->M > LOWM_MAX_M || u->K % 16 || u->K > (quantised ? kI8MaxK : LOWM_QUANTIZE_MAX_K))
    return LOWM_ERR_UNSUPPORTED;
  const size_t need = quantised ? 0 : i8_workspace(u->M, u->N, u->K);
  if (need && (!u->workspace || u->workspace_bytes < need)) return LOWM_ERR_WORKSPACE;
  const int cb = type_bytes(u->c_type), ab = type_bytes(u->a_type);
  if ((((uintptr_t)u->A | (uintptr_t)u->W | (need ? (uintptr_t)u->workspace : 0)) & 15) ||
      ((uintptr_t)u->C & (cb - 1)) || ((uintptr_t)u->w_scale & 3) ||
      (quantised && ((uintptr_t)u->a_scale & 3)))
    return LOWM_ERR_UNSUPPORTED;
  const int64_t M = u->M, N = u->N, K = u->K;
  const Span in[] = {span_of(u->A, M, K, K, ab), span_of(u->W, N, K, K, 1),
                     span_of(u->w_scale, 1, N, N, 4),
                     span_of(quantised ? u->a_scale : nullptr, 1, M, M, 4)};
  const Span c = span_of(u->C, M, N, N, cb),
             ws = span_of(need ? u->workspace : nullptr, 1, (int64_t)need, (int64_t)need, 1);
  for (const Span& s : in)
    if (meet(c, s) || meet(ws, s)) return LOWM_ERR_INVALID_ARG;
  if (meet(c, ws)) return LOWM_ERR_INVALID_ARG;

  I8Args a{static_cast<const uint8_t*>(u->A), static_cast<const uint8_t*>(u->W), u->a_scale,
           u->w_scale, u->C, u->M, u->N, u->K, u->c_type == LOWM_F32};
  if (!quantised) {
    uint8_t* q = static_cast<uint8_t*>(u->workspace);
    float* s = reinterpret_cast<float*>(q + (need - LOWM_MAX_M * sizeof(float)));
    const int rc = quantize_rows(u->A, LOWM_BF16, K, u->M, u->K, q, s, stream);
    if (rc != LOWM_OK) return rc;
    a.A = q;
    a.a_scale = s;
  }
  const int NB = pick_width(u->M, u->N);
  void* args[] = {&a};
  return launched(hipLaunchKernel(pick_kernel((u->M + 15) / 16, NB),
                                  dim3((unsigned)((N + 16 * NB - 1) / (16 * NB))), dim3(kThreads),
                                  args, 0, stream));
}

}  // namespace
}  // namespace lowm

extern "C" {

size_t lowm_gemm_i8_workspace_bytes(int M, int N, int K) { return lowm::i8_workspace(M, N, K); }

int lowm_gemm_i8(const lowm_gemm_i8_args* args, void* stream) {
  return lowm::gemm_i8(args, static_cast<hipStream_t>(stream));
}

}  // extern "C"
