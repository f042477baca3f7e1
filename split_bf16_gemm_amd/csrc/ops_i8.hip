// ops_i8.hip -- the int8 product of up to 64 rows (include/lowm_ops.h) for
// gfx950.
//
//   C[m][n] = (sum_k A[m][k] W[n][k]) a_scale[m] w_scale[n]
//
// The sum is exact (int8 products in int32), so no order of it changes a bit;
// it is scaled in fp32 and rounded once to the output's type.  Bound by HBM:
// the N K bytes of W are read once, the M K of A by every workgroup from the
// caches.  Two kinds of workgroup:
//   stretch  16*NB rows of W, its four wavefronts a stretch of K each
//            (ops_stream.cuh), their sums added through LDS;
//   panel    16 rows of W to each of 4 to 16 wavefronts, all of K for each, with
//            one panel of A per step for all of them: more rows of W for each
//            byte of A read.
// Where they are too few for the CUs, K is split over several workgroups whose
// int32 sums the last to arrive adds.  A few rows of bf16 are quantised by each
// workgroup for itself while its first rows of W are on their way (few); more
// rows once, by a kernel of their own.
//
// Measured on MI355X, us a call, W from HBM, beside a plain read of W's bytes: M 1,
// N 6144, K 4096 from bf16 7.6 (3.8); M 23, N 2304, K 12288 10.9 (4.3); M 64,
// N 49152, K 4096 37 (31), with 4.6 to quantise its rows before; M 16, N 16384,
// K 12288 36 (30).
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
  uint32_t* lines;                        // [tiles] counter lines
  uint32_t* slots;                        // [tiles][splits][blocks][64][4]
  int M, N, K, f32, splits;
};

constexpr int kI8MaxSplits = 4;

// Tile and split of this workgroup.  The grid is round_up(tiles, 8) * splits; a
// tile's splits share their index modulo 8, so they run on one XCD.
__device__ __forceinline__ void i8_place(const I8Args& a, int& tile, int& split) {
  const int row = blockIdx.x / kXcds;
  tile = blockIdx.x % kXcds + kXcds * (row / a.splits);
  split = row % a.splits;
}
// The split's steps [s0, s0 + P) of 128 bytes, of this part of `parts`.
__device__ __forceinline__ void i8_steps(const I8Args& a, int part, int parts, int& s0, int& P) {
  const int steps = (a.K + 127) / 128;
  s0 = (int)((int64_t)steps * part / parts);
  P = (int)((int64_t)steps * (part + 1) / parts) - s0;
}

// A sum in a slot: never zero, since a sum of K <= 131056 products of magnitude
// at most 2^14 is above -2^31.
__device__ __forceinline__ uint32_t i8_encode(int v) { return (uint32_t)v ^ 0x80000000u; }
__device__ __forceinline__ int i8_decode(uint32_t w) { return (int)(w ^ 0x80000000u); }

// Row 4 g + i of block b, column n: element i of v.
__device__ __forceinline__ void i8_store(const I8Args& a, const float* a_scale, const i32x4& v,
                                         int b, int n, int g) {
  if (n >= a.N) return;
  const float sw = a.w_scale[n];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = 16 * b + 4 * g + i;
    if (m >= a.M) continue;
    const int sum = v[i];
    // int32 to fp32 rounds a sum past 2^24 by half a step of fp32.
    const float c = (float)sum * a_scale[m] * sw;
    const size_t at = (size_t)m * a.N + n;
    if (a.f32)
      static_cast<float*>(a.C)[at] = c;
    else
      static_cast<__bf16*>(a.C)[at] = static_cast<__bf16>(c);
  }
}

// The splits' sums of a tile.  Thread by thread: v[j] is block first + j * step of
// the tile's `blocks`.  Returns whether this workgroup, the last to arrive, now
// holds the whole sums.
template <int NV>
__device__ __forceinline__ bool i8_join(const I8Args& a, i32x4 (&v)[NV], int tile, int split,
                                        int blocks, int first, int step, int* lds) {
  const int lane = threadIdx.x & (kWave - 1);
  const size_t per = (size_t)blocks * kWave * 4;
  uint32_t* slots = a.slots + (size_t)tile * a.splits * per;
  auto slot = [&](int s, int j, int i) {
    return slots + s * per + ((size_t)(first + j * step) * kWave + lane) * 4 + i;
  };
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (first + j * step < blocks) {
#pragma unroll
      for (int i = 0; i < 4; ++i) store_slot(slot(split, j, i), i8_encode(v[j][i]));
    }
  uint32_t* line = a.lines + (size_t)tile * kCtrStride;
  if (!arrive_last(line, a.splits, lds)) return false;
  uint32_t w[NV][kI8MaxSplits][4];       // every load before the first use
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int s = 0; s < kI8MaxSplits; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (s < a.splits && first + j * step < blocks) w[j][s][i] = load_slot(slot(s, j, i));
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (first + j * step < blocks) {
      v[j] = i32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < kI8MaxSplits; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (s < a.splits) v[j][i] += i8_decode(take_slot(slot(s, j, i), w[j][s][i], line));
    }
  return true;
}

template <int AP, int NB, int R>
struct I8Shape {
  using S = StreamShape<NB, AP, R>;
  static constexpr int kBlocks = NB * S::MB;
  static constexpr int kRings = kWaves * S::kRing * 16;                  // bytes
  static constexpr int kSums = kWaves * kBlocks * kWave * 16;
  static constexpr int lds_bytes = kRings > kSums ? kRings : kSums;
  static constexpr bool valid = S::valid && lds_bytes <= 160 * 1024 - 64;
};

// WHOLE, here and below: W's rows are whole lines of memory.
template <int AP, int NB, int R, bool WHOLE>
__global__ __launch_bounds__(kThreads) void gemm_i8_stretch_kernel(I8Args a) {
#if defined(__HIP_DEVICE_COMPILE__)
  using SH = I8Shape<AP, NB, R>;
  constexpr int G = SH::S::G, MB = SH::S::MB;
  __shared__ u32x4 lds[SH::lds_bytes / 16];
  __shared__ int last;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int g = lane >> 4, l16 = lane & 15;
  int tile, split;
  i8_place(a, tile, split);
  const int n0 = tile * 16 * NB;
  if (n0 >= a.N) return;                  // the grid's padding

  int s0, P;
  i8_steps(a, split * kWaves + wave, a.splits * kWaves, s0, P);
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
    u32x4* ring = lds + wave * SH::S::kRing;
    if constexpr (WHOLE)
      stream_tile<NB, AP, R>(ring, src, a.K - k0, P, acc);
    else
      stream_tile_shifted<NB, AP, R>(ring, src, k0, a.K - k0, P, acc);
  }
  stream_settle(acc);

  // Wavefront w's block q at sums[(w * kBlocks + q) * 64 + lane]; wavefront w adds
  // up blocks w, w + 4, ...
  i32x4* sums = reinterpret_cast<i32x4*>(lds);
  __syncthreads();
#pragma unroll
  for (int q = 0; q < SH::kBlocks; ++q) sums[(wave * SH::kBlocks + q) * kWave + lane] = acc[q];
  __syncthreads();
  constexpr int NV = (SH::kBlocks + kWaves - 1) / kWaves;
  i32x4 v[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int q = wave + j * kWaves;
    v[j] = i32x4{0, 0, 0, 0};
    if (q < SH::kBlocks) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v[j] += sums[(w * SH::kBlocks + q) * kWave + lane];
    }
  }
  if (a.splits > 1 && !i8_join(a, v, tile, split, SH::kBlocks, wave, kWaves, &last)) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int q = wave + j * kWaves;
    if (q < SH::kBlocks) i8_store(a, a.a_scale, v[j], q % MB, n0 + 16 * (q / MB) + l16, g);
  }
#endif
}

// Few bf16 rows (M <= 4 * RQ, at most 8), each workgroup quantising them for
// itself: stretch tiles whose wavefronts hold their stretch of A, PM steps at
// most, in LDS: first as it is (the row's scale needs all of K, so all
// wavefronts'), then, through registers, as int8 in the same place.  The ring
// streams W alone, and its first steps are on their way before A is looked at.
template <int RQ, int PM, int NB, int R>
struct I8Few {
  static constexpr int kPP = 68;
  static constexpr int G = 2 * NB;                       // loads per step
  static constexpr int kSlot = G * kPP;
  static constexpr int kRing = R * kSlot;
  // Each step's 4 * RQ rows of 256 bytes, then its int8 piece of 8 rows; that
  // block's other piece holds rows that are not there: whatever follows (one
  // piece of room after the last).
  static constexpr int kRaw = RQ * kWave;
  static constexpr int kRows = PM * (kRaw > kPP ? kRaw : kPP);
  static constexpr int kElems = kWaves * (kRing + kRows) + kPP;
  static constexpr int kSums = kWaves * NB * kWave;
  static constexpr bool valid = R >= 2 && (R - 1) * G <= 63 && kSums <= kWaves * kRing &&
                                kElems * 16 <= 160 * 1024 - 512;
};

template <int RQ, int PM, int NB, int R, bool WHOLE>
__global__ __launch_bounds__(kThreads) void gemm_i8_few_kernel(I8Args a) {
#if defined(__HIP_DEVICE_COMPILE__)
  using SH = I8Few<RQ, PM, NB, R>;
  constexpr int G = SH::G, kPP = SH::kPP;
  __shared__ u32x4 lds[SH::kElems];
  __shared__ u32x4 tops[4 * RQ];         // [row][wavefront]
  __shared__ float scales[4 * RQ];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int g = lane >> 4, l16 = lane & 15;
  const int n0 = blockIdx.x * 16 * NB;
  const int steps = (a.K + 127) / 128;
  const int s0 = steps * wave / kWaves, P = steps * (wave + 1) / kWaves - s0;

  u32x4* ring = lds + wave * SH::kRing;
  u32x4* rows = lds + kWaves * SH::kRing + wave * SH::kRows;
  const int k0 = s0 * 128 + stream_piece(lane) * 16, left = a.K - k0;
  const int line = __builtin_amdgcn_readfirstlane(left);
  const uint8_t* src[G];
#pragma unroll
  for (int t = 0; t < G; ++t) {
    const int r = n0 + 8 * t + stream_row(lane);
    src[t] = a.W + (size_t)(r < a.N ? r : a.N - 1) * a.K + k0;
  }
  const StreamRows<WHOLE, NB, SH::kSlot, SH::kRing, kPP> w_rows(src);
  const int lines = w_rows.lines(P, line);
  auto issue = [&](u32x4* slot, int p) {
    const int at = p * 128;
    if (line - at >= 128 && (WHOLE || (p > 0 && p + 1 < lines))) {
      static_for<G>([&](auto t_c) {
        constexpr int t = decltype(t_c)::value;
        __builtin_amdgcn_global_load_lds(
            src[t] + at, (__attribute__((address_space(3))) void*)(slot + t * kPP), 16, 0,
            kStreamAux);
      });
    } else {
      static_for<G>([&](auto t_c) {
        constexpr int t = decltype(t_c)::value;
        __builtin_amdgcn_global_load_lds(
            w_rows.from(src[t], t, at, k0, left),
            (__attribute__((address_space(3))) void*)(slot + t * kPP), 16, 0, 0);
      });
    }
    pin_issue();
  };
  u32x4* const end = ring + SH::kRing;
  u32x4 *fill = ring, *use = ring;
  auto next = [&](u32x4* s) { return s + SH::kSlot == end ? ring : s + SH::kSlot; };
  // Lane (g, l16) takes elements 8 l16 .. 8 l16 + 7 of a step's 128, of rows g and,
  // for RQ 2, g + 4; zeros past the end.
  const uint16_t* A = reinterpret_cast<const uint16_t*>(a.A);
  static_for<PM * RQ>([&](auto i_c) {
    constexpr int p = decltype(i_c)::value / RQ, q = decltype(i_c)::value % RQ;
    const int m = g + 4 * q < a.M ? g + 4 * q : a.M - 1;
    const int k = (s0 + p) * 128 + 8 * l16;
    const void* from = p < P && k < a.K ? static_cast<const void*>(A + (size_t)m * a.K + k)
                                        : static_cast<const void*>(&kZeroPiece);
    __builtin_amdgcn_global_load_lds(
        from, (__attribute__((address_space(3))) void*)(rows + (p * RQ + q) * kWave), 16, 0, 0);
  });
  // All of the ring's slots, whether there are as many steps or not (past them
  // there are zeros to read), so that the wait for A below knows how many loads
  // may stay in flight.
  static_for<R - 1>([&](auto i_c) {
    issue(fill, decltype(i_c)::value);
    fill = next(fill);
  });

  wait_vmcnt<(R - 1) * G>();
  u32x4 raw[PM * RQ];                    // step p's rows g + 4 q at p * RQ + q
#pragma unroll
  for (int i = 0; i < PM * RQ; ++i) raw[i] = lds_read_opaque(rows + i * kWave + lane);
  lds_wait(raw);
  // The rows' largest magnitudes, as bit patterns: over the 16 lanes that share
  // a row, then over the wavefronts.
#pragma unroll
  for (int q = 0; q < RQ; ++q) {
    uint32_t top = 0;
#pragma unroll
    for (int p = 0; p < PM; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = raw[p * RQ + q][i], hi = w & 0x7fff0000u, lo = (w & 0x7fffu) << 16;
        top = hi > top ? hi : top;
        top = lo > top ? lo : top;
      }
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) {
      const uint32_t o = __shfl_xor(top, off);
      top = o > top ? o : top;
    }
    if (l16 == 0) reinterpret_cast<uint32_t*>(&tops[g + 4 * q])[wave] = top;
  }
  // (the ring's loads stay in flight)
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
  for (int q = 0; q < RQ; ++q) {
    u32x4 all[1] = {lds_read_opaque(&tops[g + 4 * q])};
    lds_wait(all);
    uint32_t top = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const uint32_t o = all[0][w];
      top = o > top ? o : top;
    }
    const RowScale rs(top);
    if (wave == 0 && l16 == 0) scales[g + 4 * q] = rs.scale;
    // Row m's 16-byte piece j of a line lies at place (j + m / 2) mod 8 of the row,
    // as the loads into the ring place it.
    const int m = g + 4 * q, at = (m * 8 + (((l16 >> 1) + (m >> 1)) & 7)) * 16 + (l16 & 1) * 8;
#pragma unroll
    for (int p = 0; p < PM; ++p) {
      ops_u32x2 q8;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t lo = raw[p * RQ + q][2 * h], hi = raw[p * RQ + q][2 * h + 1];
        q8[h] = rs.quantise4(bf16_lo(lo), bf16_hi(lo), bf16_lo(hi), bf16_hi(hi));
      }
      if (p < P) lds_write8_opaque(reinterpret_cast<char*>(rows + p * kPP) + at, q8);
    }
  }
  wait_lgkmcnt0();                       // (a wavefront reads only its own rows)

  int rpos[2];
#pragma unroll
  for (int c = 0; c < 2; ++c)
    rpos[c] = (l16 >> 3) * kPP + (l16 & 7) * 8 + ((4 * c + g + ((l16 & 7) >> 1)) & 7);
  i32x4 acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = i32x4{0, 0, 0, 0};
  auto multiply = [&](int p) {
    u32x4 v[2 * (NB + 1)];
    const bool turned = next(use) == ring;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int j = 0; j < NB; ++j) v[c * (NB + 1) + j] = w_rows.read(use, turned, c, j);
      v[c * (NB + 1) + NB] = lds_read_opaque(rows + p * kPP + rpos[c]);
    }
    lds_wait(v);
    if (!WHOLE && p + 1 == lines) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < NB; ++j) w_rows.cut(v[c * (NB + 1) + j], c, j);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        acc[j] = stream_mfma(v[c * (NB + 1) + NB], v[c * (NB + 1) + j], acc[j]);
    use = next(use);
  };
  int p = 0;
  if constexpr (WHOLE) {
    for (; p + R - 1 < P; ++p) {
      wait_vmcnt<(R - 2) * G>();
      issue(fill, p + R - 1);
      fill = next(fill);
      multiply(p);
    }
    static_for<R - 1>([&](auto i_c) {
      constexpr int younger = R - 2 - decltype(i_c)::value;
      if (P - p == younger + 1) {
        wait_vmcnt<younger * G>();
        multiply(p);
        ++p;
      }
    });
  } else {
    static_assert(R >= 3, "two slots to read from");
    for (; p < P; ++p) {
      if (p + R - 1 < lines) {
        issue(fill, p + R - 1);
        fill = next(fill);
      }
      const int issued = lines < R - 1 ? R - 1 : p + R < lines ? p + R : lines;
      stream_wait<R - 2, G>(issued - (p + 2 < lines ? p + 2 : lines));
      multiply(p);
    }
  }
  stream_settle(acc);
  // Where there were fewer steps than slots, the others' loads may still be on their
  // way into LDS, which the sums take next.
  wait_vmcnt<0>();
  i32x4* sums = reinterpret_cast<i32x4*>(lds);
  __syncthreads();
#pragma unroll
  for (int q = 0; q < NB; ++q) sums[(wave * NB + q) * kWave + lane] = acc[q];
  __syncthreads();
  if (wave < NB) {
    i32x4 v = sums[wave * kWave + lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += sums[(w * NB + wave) * kWave + lane];
    i8_store(a, scales, v, 0, n0 + 16 * wave + l16, g);
  }
#endif
}

// A step's slot of the panel kernel: the panel's pieces, then each of the PW
// wavefronts' two pieces of W.
template <int AP, int PW, int R>
struct I8Panel {
  static constexpr int MB = (AP + 1) / 2;
  static constexpr int kPP = 68;
  static constexpr int kEach = AP / PW, kRest = AP % PW;   // panel pieces a wavefront loads
  static constexpr int kSlot = (2 * MB + 2 * PW) * kPP;
  static constexpr int lds_bytes = R * kSlot * 16;
  static constexpr bool valid =
      R >= 2 && (R - 1) * (kEach + 1 + 2) <= 63 && lds_bytes <= 160 * 1024 - 64;
};

// The loop of one wavefront; MINE: how many pieces of the panel it loads (its
// waits count those loads too).
template <int AP, int PW, int R, int MINE, bool WHOLE>
__device__ __forceinline__ void i8_panel_loop(const I8Args& a, u32x4* lds, int n0, int P,
                                              i32x4 (&acc)[(AP + 1) / 2]) {
  using SH = I8Panel<AP, PW, R>;
  constexpr int G = 2 + MINE, kPP = SH::kPP, MB = SH::MB;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int g = lane >> 4, l16 = lane & 15;
  const int k0 = stream_piece(lane) * 16, left = a.K - k0;
  const int line = __builtin_amdgcn_readfirstlane(left);
  const int my_w = (2 * MB + wave * 2) * kPP;       // within a slot
  const uint8_t* src[G];
#pragma unroll
  for (int t = 0; t < G; ++t) {
    if (t < 2) {
      const int r = n0 + 8 * t + stream_row(lane);
      src[t] = a.W + (size_t)(r < a.N ? r : a.N - 1) * a.K + k0;
    } else {
      const int r = 8 * (wave + (t - 2) * PW) + stream_row(lane);
      src[t] = a.A + (size_t)(r < a.M ? r : a.M - 1) * a.K + k0;
    }
  }
  int rpos[2];
#pragma unroll
  for (int c = 0; c < 2; ++c)
    rpos[c] = (l16 >> 3) * kPP + (l16 & 7) * 8 + ((4 * c + g + ((l16 & 7) >> 1)) & 7);

  const StreamRows<WHOLE, 1, SH::kSlot, R * SH::kSlot, kPP> w_rows(src);
  const int lines = w_rows.lines(P, line);
  // Neighbours start at different steps and go round: else all ask at one time for
  // one column of rows a power of two of bytes apart, that is, of a few memory
  // channels (K 4096: M 40, N 32768 34.5 against 28 us, M 64, N 49152 38.9 against 37;
  // M 24, N 33000, K 8192 61.5 against 48; K 4224 the same; whole-K panels only: the
  // stretch kind's wavefronts start K / 4 apart and gain nothing).
  const int start = WHOLE ? (int)(blockIdx.x % (unsigned)P) : 0;
  auto issue = [&](u32x4* slot, int p) {
    const int at = (WHOLE && p + start >= P ? p + start - P : p + start) * 128;
    auto load = [&](auto t_c, const uint8_t* from, auto aux_c) {
      constexpr int t = decltype(t_c)::value;
      u32x4* to = slot + (t < 2 ? my_w + t * kPP : (wave + (t - 2) * PW) * kPP);
      __builtin_amdgcn_global_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, 0,
                                       decltype(aux_c)::value);
    };
    if (line - at >= 128 && (WHOLE || (p > 0 && p + 1 < lines)))
      static_for<G>([&](auto t_c) {
        constexpr int t = decltype(t_c)::value;
        load(t_c, src[t] + at, std::integral_constant<int, t < 2 ? kStreamAux : 0>{});
      });
    else
      static_for<G>([&](auto t_c) {
        constexpr int t = decltype(t_c)::value;
        const uint8_t* from = src[t] + at;
        if constexpr (t < 2)
          from = w_rows.from(src[t], t, at, k0, left);
        else
          from = left - at >= 16 ? from : reinterpret_cast<const uint8_t*>(&kZeroPiece);
        load(t_c, from, std::integral_constant<int, 0>{});
      });
    pin_issue();
  };
  u32x4* const end = lds + R * SH::kSlot;
  u32x4 *fill = lds, *use = lds;
  auto next = [&](u32x4* s) { return s + SH::kSlot == end ? lds : s + SH::kSlot; };
  auto multiply = [&](int p) {
    u32x4 v[2 * (1 + MB)];
    const bool turned = next(use) == lds;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      v[c * (1 + MB)] = w_rows.read(use + my_w, turned, c, 0);
#pragma unroll
      for (int b = 0; b < MB; ++b)
        v[c * (1 + MB) + 1 + b] = lds_read_opaque(use + 2 * b * kPP + rpos[c]);
    }
    lds_wait(v);
    if (!WHOLE && p + 1 == lines) {
#pragma unroll
      for (int c = 0; c < 2; ++c) w_rows.cut(v[c * (1 + MB)], c, 0);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int b = 0; b < MB; ++b)
        acc[b] = stream_mfma(v[c * (1 + MB) + 1 + b], v[c * (1 + MB)], acc[b]);
    use = next(use);
  };
  for (int p = 0; p < R - 1 && p < lines; ++p) {
    issue(fill, p);
    fill = next(fill);
  }
  int p = 0;
  if constexpr (WHOLE) {
    for (; p + R - 1 < P; ++p) {
      wait_vmcnt<(R - 2) * G>();
      // Every wavefront's loads of step p have landed, and every wavefront's reads
      // of step p-1, whose slot is filled next, have completed (lds_wait).  Every
      // wavefront passes P barriers.
      barrier_keep_loads();
      issue(fill, p + R - 1);
      fill = next(fill);
      multiply(p);
    }
    static_for<R - 1>([&](auto i_c) {
      constexpr int younger = R - 2 - decltype(i_c)::value;
      if (P - p == younger + 1) {
        wait_vmcnt<younger * G>();
        barrier_keep_loads();
        multiply(p);
        ++p;
      }
    });
  } else {
    static_assert(R >= 3, "two slots to read from");
    for (; p < P; ++p) {
      // As above; then the wavefront's own rows' next line, after which the slot
      // freed by the barrier is being filled again.
      const int before = p + R - 1 < lines ? p + R - 1 : lines;
      stream_wait<R - 2, G>(before - (p + 1));
      barrier_keep_loads();
      if (p + R - 1 < lines) {
        issue(fill, p + R - 1);
        fill = next(fill);
      }
      stream_wait<R - 2, G>((p + R < lines ? p + R : lines) - (p + 2 < lines ? p + 2 : lines));
      multiply(p);
    }
  }
}

template <int AP, int PW, int R, bool WHOLE>
__global__ __launch_bounds__(PW* kWave) void gemm_i8_panel_kernel(I8Args a) {
#if defined(__HIP_DEVICE_COMPILE__)
  using SH = I8Panel<AP, PW, R>;
  constexpr int MB = SH::MB;
  __shared__ u32x4 lds[R * SH::kSlot];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int n0 = ((int)blockIdx.x * PW + wave) * 16;
  const int P = (a.K + 127) / 128;
  i32x4 acc[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) acc[i] = i32x4{0, 0, 0, 0};
  if (wave < SH::kRest)
    i8_panel_loop<AP, PW, R, SH::kEach + 1, WHOLE>(a, lds, n0, P, acc);
  else
    i8_panel_loop<AP, PW, R, SH::kEach, WHOLE>(a, lds, n0, P, acc);
  stream_settle(acc);
#pragma unroll
  for (int b = 0; b < MB; ++b) i8_store(a, a.a_scale, acc[b], b, n0 + (lane & 15), lane >> 4);
#endif
}

namespace {

// From this many bytes of W on, rows that are not whole lines are read line by line
// (ShiftedRows); below, what it costs to find one's place in the lines is more than
// the bytes read twice (16 rows: N 2048, K 4112 6.9 against 7.5 us, N 8192, K 1040
// 6.0 against 5.8; 1 row: N 2048, K 8208 8.2 against 7.8, N 8192, K 2064 6.6 against
// 7.1, N 16000, K 8208 25.3 against 38.8).
constexpr int64_t kI8ShiftFrom = 1 << 24;

// The deepest ring, up to R slots, that LDS and the wait counter allow.
template <int AP, int NB, int R>
constexpr int stretch_ring() {
  if constexpr (I8Shape<AP, NB, R>::valid) return R;
  else return stretch_ring<AP, NB, R - 1>();
}
// A kernel for W of whole lines, and the one for other rows, which there is for
// rings of three slots and more.
struct Pair {
  const void *whole, *shifted;
};
constexpr bool three_slots(int MB, int NB) { return MB + NB <= 6; }
template <int AP, int NB>
Pair stretch_of() {
  constexpr int R = stretch_ring<AP, NB, 4>();
  static_assert(three_slots(AP / 2, NB) == (R >= 3), "what the plan takes it for");
  Pair k{reinterpret_cast<const void*>(&gemm_i8_stretch_kernel<AP, NB, R, true>), nullptr};
  if constexpr (R >= 3)
    k.shifted = reinterpret_cast<const void*>(&gemm_i8_stretch_kernel<AP, NB, R, false>);
  return k;
}
template <int AP, int PW>
Pair panel_of() {
  static_assert(I8Panel<AP, PW, 3>::valid, "the ring fits");
  return {reinterpret_cast<const void*>(&gemm_i8_panel_kernel<AP, PW, 3, true>),
          reinterpret_cast<const void*>(&gemm_i8_panel_kernel<AP, PW, 3, false>)};
}
constexpr int kPanelWaves[] = {4, 6, 8, 12, 16};
template <int AP>
Pair panel_by_waves(int waves) {
  return waves == 4    ? panel_of<AP, 4>()
         : waves == 6  ? panel_of<AP, 6>()
         : waves == 8  ? panel_of<AP, 8>()
         : waves == 12 ? panel_of<AP, 12>()
                       : panel_of<AP, 16>();
}

struct I8Plan {
  int panel;                              // the panel kind's wavefronts, 0 for the stretch kind
  int NB, splits;
  int width() const { return 16 * (panel ? panel : 1) * NB; }
  int tiles(int N) const { return (int)(((int64_t)N + width() - 1) / width()); }
};

template <int RQ, int PM, int NB, int R>
constexpr int few_ring() {
  if constexpr (I8Few<RQ, PM, NB, R>::valid) return R;
  else return few_ring<RQ, PM, NB, R - 1>();
}
template <int RQ, int PM, int NB>
Pair few_of() {
  constexpr int R = few_ring<RQ, PM, NB, 8>();
  Pair k{reinterpret_cast<const void*>(&gemm_i8_few_kernel<RQ, PM, NB, R, true>), nullptr};
  if constexpr (R >= 3)
    k.shifted = reinterpret_cast<const void*>(&gemm_i8_few_kernel<RQ, PM, NB, R, false>);
  return k;
}
// The kernel that quantises M bf16 rows itself, if there is one: M <= 8 rows whose
// stretches fit a wavefront's registers, in one round of workgroups.
Pair few_kernel(int M, int K, const I8Plan& p, int tiles) {
  static const Pair table[3][4] = {
      {few_of<1, 8, 1>(), few_of<1, 8, 2>(), few_of<1, 8, 3>(), few_of<1, 8, 4>()},
      {few_of<1, 16, 1>(), few_of<1, 16, 2>(), few_of<1, 16, 3>(), few_of<1, 16, 4>()},
      {few_of<2, 8, 1>(), few_of<2, 8, 2>(), few_of<2, 8, 3>(), few_of<2, 8, 4>()}};
  if (M > 8 || p.panel || tiles > 256) return {};
  const int steps = ((K + 127) / 128 + kWaves - 1) / kWaves;
  const int row = steps <= 8 ? (M <= 4 ? 0 : 2) : steps <= 16 && M <= 4 ? 1 : -1;
  return row < 0 ? Pair{} : table[row][p.NB - 1];
}

Pair i8_kernel(int MB, const I8Plan& p) {
  static const Pair stretch[4][4] = {
      {stretch_of<2, 1>(), stretch_of<2, 2>(), stretch_of<2, 3>(), stretch_of<2, 4>()},
      {stretch_of<4, 1>(), stretch_of<4, 2>(), stretch_of<4, 3>(), stretch_of<4, 4>()},
      {stretch_of<6, 1>(), stretch_of<6, 2>(), stretch_of<6, 3>(), stretch_of<6, 4>()},
      {stretch_of<8, 1>(), stretch_of<8, 2>(), stretch_of<8, 3>(), stretch_of<8, 4>()}};
  if (!p.panel) return stretch[MB - 1][p.NB - 1];
  return MB == 1   ? panel_by_waves<2>(p.panel)
         : MB == 2 ? panel_by_waves<4>(p.panel)
         : MB == 3 ? panel_by_waves<6>(p.panel)
                   : panel_by_waves<8>(p.panel);
}

constexpr int64_t kI8MaxK = 131056;   // 128 * 128 * K stays below 2^31
// The panel kind's four threads to a column, in tiles of up to 256 columns, are
// fewer than 2^32, what a launch takes.
static_assert(4ll * (LOWM_I8_MAX_N + 255) < 1ll << 32, "one launch");
// What a split launch may use of the workspace: counter lines, one for each
// tile, and blocks of 16 x 16 partial sums.
constexpr int kI8MaxTiles = LOWM_I8_STATUS_N / 16;
constexpr long kI8MaxBlocks = 8192;
constexpr size_t kI8LineBytes = 256 * (size_t)kI8MaxTiles;
constexpr size_t kI8SlotBytes = (size_t)kI8MaxBlocks * kWave * 4 * 4;

// How to cut the product.  Measured on MI355X, W from HBM, us a call:
//   - from 16385 columns on the panel kind (a workgroup then loads 64 rows of A for
//     up to 256 of W, not for 64), of the width with the fewest rounds of 256
//     workgroups times rows loaded.  M 64, K 4096: N 20000 with 6 wavefronts 24.4 (4:
//     28.9, 8: 27.1), N 32768 with 8 31.3 (4: 34.4, 16: 39.5), N 49152 with 12 39.9
//     (4: 48.4, 16: 41.4; stretch 56.2).  Up to 16 rows, where A is little to save,
//     from 32768 columns on: M 16, K 4096 N 20000 19.2 against 19.8, but K 8192 37.0
//     against 34.2; N 49152 35.6 against 40.2, N 32768, K 8192 44.9 against 49.1.  At
//     N 16384 its tiles are too few (M 64, K 8192 38.6 against 33.8).
//   - otherwise stretch tiles of the width, and the split of K, of least cost:
//     rounds times bytes loaded by a workgroup, at 67 KB a us, and for a split's
//     exchange 1 us, 0.25 a split and 0.2 a block of 16 x 16 sums sent.  M 16,
//     N 6144, K 4096 NB 2 7.5 us (NB 1 8.3, NB 3 8.6); M 64, N 12288, K 8192 NB 3
//     25.2 (NB 4 29.2); M 64, N 1536, K 8192 NB 1 in two splits 10.9 (whole 13.2);
//     M 23, N 2304, K 12288 NB 2 in three 11.4 (NB 1 whole 12.5); M 64, N 4096,
//     K 4096 NB 1 whole 9.2 (two splits 16.3).
//   - the panel kind of 4 wavefronts competes by the same cost where K is short (no
//     sums to add up at the end: N 16384, K 512, M 64 7.3 against 9.0, M 32 5.5
//     against 6.6; K 4096 22.4 against 21.6, 19.3 against 16.4), and for rows of W
//     that are not whole lines where the wide tiles' rings are too short for those
//     (M 64, N 16384, K 4112 25.8 against 29.7; K 12272 64.5 against 72.6).
I8Plan i8_plan(int M, int N, int K, bool split, bool whole) {
  const int MB = (M + 15) / 16;
  if (N >= (M > 16 ? 16385 : 32768)) {
    I8Plan best{0, 1, 1};
    int64_t best_cost = 0;
    for (int waves : kPanelWaves) {
      const I8Plan p{waves, 1, 1};
      const int64_t cost = (int64_t)(p.tiles(N) + 255) / 256 * (16 * MB + p.width());
      if (best.panel == 0 || cost < best_cost) {
        best = p;
        best_cost = cost;
      }
    }
    return best;
  }
  I8Plan best{0, 1, 1};
  double best_us = 0;
  if (MB >= 2 && (K <= 1536 || (!whole && MB >= 3))) {
    best = I8Plan{4, 1, 1};
    best_us = (double)((best.tiles(N) + 255) / 256) * (16 * MB + best.width()) * K / 67.0e3;
  }
  for (int nb = 1; nb <= 4 && (whole || three_slots(MB, nb)); ++nb)
    for (int s = 1; s <= (split ? kI8MaxSplits : 1); ++s) {
      const I8Plan p{0, nb, s};
      const int64_t tiles = p.tiles(N);
      if (s > 1 && (tiles > kI8MaxTiles || tiles * s * nb * MB > kI8MaxBlocks)) continue;
      if (s > 1 && K / s < 128 * kWaves) continue;       // a step for every wavefront
      const double us = (double)((tiles * s + 255) / 256) * (16 * (MB + nb)) * K / s / 67.0e3 +
                        (s > 1 ? 1.0 + 0.25 * s + 0.2 * (nb * MB) * (s - 1) : 0.0);
      if (best_us == 0 || us < best_us) {
        best = p;
        best_us = us;
      }
    }
  return best;
}

size_t i8_workspace(int M, int N, int K) {
  if (M < 1 || M > LOWM_MAX_M || N < 1 || N > LOWM_I8_MAX_N || K < 1 || K % 16 || K > kI8MaxK) return 0;
  return kI8LineBytes + kI8SlotBytes + ((size_t)M * K + 255) / 256 * 256 +
         LOWM_MAX_M * sizeof(float);
}

int gemm_i8(const lowm_gemm_i8_args* u, hipStream_t stream) {
  if (!u || u->M < 1 || u->N < 1 || u->K < 1) return LOWM_ERR_INVALID_ARG;
  if (!u->A || !u->W || !u->w_scale || !u->C) return LOWM_ERR_INVALID_ARG;
  const bool quantised = u->a_type == LOWM_I8;
  if ((!quantised && u->a_type != LOWM_BF16) || (quantised && !u->a_scale) ||
      (u->c_type != LOWM_BF16 && u->c_type != LOWM_F32))
    return LOWM_ERR_INVALID_ARG;
  if (u->M > LOWM_MAX_M || u->N > LOWM_I8_MAX_N || u->K % 16 || u->K > (quantised ? kI8MaxK : LOWM_QUANTIZE_MAX_K))
    return LOWM_ERR_UNSUPPORTED;
  const size_t need = i8_workspace(u->M, u->N, u->K);
  if (u->workspace ? u->workspace_bytes < need : !quantised) return LOWM_ERR_WORKSPACE;
  const int cb = type_bytes(u->c_type), ab = type_bytes(u->a_type);
  if ((((uintptr_t)u->A | (uintptr_t)u->W) & 15) || ((uintptr_t)u->workspace & 255) ||
      ((uintptr_t)u->C & (cb - 1)) || ((uintptr_t)u->w_scale & 3) ||
      (quantised && ((uintptr_t)u->a_scale & 3)))
    return LOWM_ERR_UNSUPPORTED;
  const int64_t M = u->M, N = u->N, K = u->K;
  const Span in[] = {span_of(u->A, M, K, K, ab), span_of(u->W, N, K, K, 1),
                     span_of(u->w_scale, 1, N, N, 4),
                     span_of(quantised ? u->a_scale : nullptr, 1, M, M, 4)};
  const Span c = span_of(u->C, M, N, N, cb),
             ws = span_of(u->workspace, 1, (int64_t)need, (int64_t)need, 1);
  for (const Span& s : in)
    if (meet(c, s) || meet(ws, s)) return LOWM_ERR_INVALID_ARG;
  if (meet(c, ws)) return LOWM_ERR_INVALID_ARG;

  I8Args a{};
  a.A = static_cast<const uint8_t*>(u->A);
  a.W = static_cast<const uint8_t*>(u->W);
  a.a_scale = u->a_scale;
  a.w_scale = u->w_scale;
  a.C = u->C;
  a.M = u->M;
  a.N = u->N;
  a.K = u->K;
  a.f32 = u->c_type == LOWM_F32;
  uint8_t* w = static_cast<uint8_t*>(u->workspace);
  void* args[] = {&a};
  const bool whole = !(((uintptr_t)a.W | (uintptr_t)u->K) & 127) || N * K < kI8ShiftFrom;
  auto in_lines = [whole](const Pair& k) { return whole ? k.whole : k.shifted; };
  if (!quantised) {
    const I8Plan p = i8_plan(u->M, u->N, u->K, false, whole);
    const int tiles = p.tiles(u->N);
    if (const void* fn = in_lines(few_kernel(u->M, u->K, p, tiles)))
      return launched(hipLaunchKernel(fn, dim3((unsigned)tiles), dim3(kThreads), args, 0, stream));
    uint8_t* q = w + kI8LineBytes + kI8SlotBytes;
    float* s = reinterpret_cast<float*>(w + need - LOWM_MAX_M * sizeof(float));
    const int rc = quantize_rows(u->A, LOWM_BF16, K, u->M, u->K, q, s, stream);
    if (rc != LOWM_OK) return rc;
    a.A = q;
    a.a_scale = s;
  }
  const I8Plan p = i8_plan(u->M, u->N, u->K, w != nullptr, whole);
  a.splits = p.splits;
  a.lines = reinterpret_cast<uint32_t*>(w);
  a.slots = reinterpret_cast<uint32_t*>(w + (w ? kI8LineBytes : 0));
  const size_t tiles = (size_t)p.tiles(u->N);
  const size_t grid = p.panel ? tiles : (tiles + kXcds - 1) / kXcds * kXcds * p.splits;
  return launched(hipLaunchKernel(in_lines(i8_kernel((u->M + 15) / 16, p)), dim3((unsigned)grid),
                                  dim3(p.panel ? p.panel * kWave : kThreads), args, 0,
                                  stream));
}

}  // namespace
}  // namespace lowm

extern "C" {

size_t lowm_gemm_i8_workspace_bytes(int M, int N, int K) { return lowm::i8_workspace(M, N, K); }

int lowm_gemm_i8(const lowm_gemm_i8_args* args, void* stream) {
  return lowm::gemm_i8(args, static_cast<hipStream_t>(stream));
}

}  // extern "C"
