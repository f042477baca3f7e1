// ops_stream.cuh -- one wavefront's product of a few rows with 16*NB weight rows
// over a stretch of the inner dimension, both operands streamed through an LDS
// ring of the wavefront's own.  Shared by the operators that read weights once
// (the int8 product, the experts' products).
//
// Bytes are all this file knows of the element type: a step is one 128-byte
// line of every row, two matrix instructions of 64 bytes each.  A line goes
// straight into LDS in whole requests (8 rows x 128 B), its 16-byte pieces
// rotated by row/2 so that the matrix layout's reads of 16 rows fall in
// distinct banks.  There is no barrier in the loop: a slot is refilled only
// after the wavefront's own reads of it have completed.
#pragma once

#include "lowm_kernels.cuh"
#include "ops_common.cuh"

namespace lowm {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// What pieces past a row's end read instead: they then add nothing.
__device__ const u32x4 kZeroPiece = {0u, 0u, 0u, 0u};

__device__ __forceinline__ f32x4 stream_mfma(u32x4 a, u32x4 b, f32x4 c) { return mfma(a, b, c); }
__device__ __forceinline__ i32x4 stream_mfma(u32x4 a, u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                               __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}
// See mfma_settle (lowm_kernels.cuh): wait states between the last matrix
// instruction and the first read of its result on every path.
template <int N>
__device__ __forceinline__ void stream_settle(f32x4 (&acc)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" : "+a"(acc[i]));
}
template <int N>
__device__ __forceinline__ void stream_settle(i32x4 (&acc)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" : "+a"(acc[i]));
}

// LDS accesses the compiler does not see, for use while loads into LDS are in
// flight (it would wait for all of those first).  A wavefront's own complete in
// order; the read waits for itself.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}
__device__ __forceinline__ ops_u32x2 lds_read8_opaque(const void* p) {
  ops_u32x2 v;
  asm volatile("ds_read_b64 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=v"(v) : "v"(lds_address(p)) : "memory");
  return v;
}
__device__ __forceinline__ void lds_write8_opaque(void* p, ops_u32x2 v) {
  asm volatile("ds_write_b64 %0, %1" : : "v"(lds_address(p)), "v"(v) : "memory");
}
__device__ __forceinline__ void lds_add_opaque(float* p, float v) {
  asm volatile("ds_add_f32 %0, %1" : : "v"(lds_address(p)), "v"(v) : "memory");
}

// NB blocks of 16 weight rows, AP pieces of 8 activation rows, R ring slots.
template <int NB, int AP, int R>
struct StreamShape {
  static constexpr int MB = (AP + 1) / 2;        // blocks of 16 activation rows
  static constexpr int kPP = 68;                 // u32x4 per piece of 8 rows (1088 B)
  static constexpr int G = 2 * NB + AP;          // pieces, and loads, per step
  // An odd last piece leaves the upper half of its block unwritten: rows whose
  // results nobody takes.
  static constexpr int kSlot = (2 * NB + 2 * MB) * kPP;   // u32x4 per slot
  static constexpr int kRing = R * kSlot;        // u32x4 per wavefront
  static constexpr bool valid = R >= 2 && (R - 1) * G <= 63;   // the wait counter is 6 bits
};

// Lane's row within a piece of 8 and its 16-byte piece of the row's line.
__device__ __forceinline__ int stream_row(int lane) { return lane >> 3; }
__device__ __forceinline__ int stream_piece(int lane) { return ((lane & 7) - (lane >> 4)) & 7; }

// acc[j * MB + b] += rows of block b times weight rows of block j over P steps.
// src[t]: this lane's 16 bytes of piece t in the first step (pieces 0 .. 2NB-1
// weight rows, then activation rows); left: bytes from there to the row's end,
// the same for every t.  Every address up to the row's end must be readable;
// none past it is read.
template <int NB, int AP, int R, typename Acc>
__device__ __forceinline__ void stream_tile(u32x4* ring, const uint8_t* (&src)[2 * NB + AP],
                                            int left, int P,
                                            Acc (&acc)[NB * ((AP + 1) / 2)]) {
  using SH = StreamShape<NB, AP, R>;
  static_assert(SH::valid, "a ring the waits can count");
  constexpr int G = SH::G, kPP = SH::kPP, MB = SH::MB;
  const int lane = threadIdx.x & (kWave - 1);
  const int g = lane >> 4, l16 = lane & 15;
  // Lane 7 of each 8-row piece's row 0 holds the line's last 16 bytes: a step is
  // whole when they are inside.
  const int line = __builtin_amdgcn_readfirstlane(left);   // lane 0: piece 0
  int rpos[2];
#pragma unroll
  for (int c = 0; c < 2; ++c)
    rpos[c] = (l16 >> 3) * kPP + (l16 & 7) * 8 + ((4 * c + g + ((l16 & 7) >> 1)) & 7);

  auto issue = [&](u32x4* slot, int p) {
    const int at = p * 128;
    const bool whole = line - at >= 128;
    static_for<G>([&](auto t_c) {
      constexpr int t = decltype(t_c)::value;
      const uint8_t* from = src[t] + at;
      if (!whole) from = left - at >= 16 ? from : reinterpret_cast<const uint8_t*>(&kZeroPiece);
      __builtin_amdgcn_global_load_lds(from, (__attribute__((address_space(3))) void*)(slot + t * kPP),
                                       16, 0, t < 2 * NB ? kStreamAux : 0);
    });
    pin_issue();
  };
  auto multiply = [&](const u32x4* slot) {
    u32x4 v[2 * (NB + MB)];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int t = 0; t < NB + MB; ++t)
        v[c * (NB + MB) + t] = lds_read_opaque(slot + 2 * t * kPP + rpos[c]);
    lds_wait(v);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int b = 0; b < MB; ++b)
          acc[j * MB + b] =
              stream_mfma(v[c * (NB + MB) + NB + b], v[c * (NB + MB) + j], acc[j * MB + b]);
  };

  u32x4* const end = ring + SH::kRing;
  u32x4 *fill = ring, *use = ring;
  auto next = [&](u32x4* s) { return s + SH::kSlot == end ? ring : s + SH::kSlot; };
  for (int p = 0; p < R - 1 && p < P; ++p) {
    issue(fill, p);
    fill = next(fill);
  }
  int p = 0;
  for (; p + R - 1 < P; ++p) {
    // steps p .. p+R-2 are in flight; step p has landed when R-2 are
    wait_vmcnt<(R - 2) * G>();
    issue(fill, p + R - 1);        // into the slot step p-1 was read from
    fill = next(fill);
    multiply(use);
    use = next(use);
  }
  static_for<R - 1>([&](auto i_c) {
    constexpr int younger = R - 2 - decltype(i_c)::value;   // steps after this one
    if (P - p == younger + 1) {
      wait_vmcnt<younger * G>();
      multiply(use);
      use = next(use);
      ++p;
    }
  });
}

// Waits until at most `young` steps' loads of G each are in flight, 0 <= young <= MOST.
template <int MOST, int G>
__device__ __forceinline__ void stream_wait(int young) {
  if (young >= MOST) {
    wait_vmcnt<MOST * G>();
    return;
  }
  static_for<MOST>([&](auto i_c) {
    constexpr int i = decltype(i_c)::value;
    if (young == i) wait_vmcnt<i * G>();
  });
}

// Weight rows that start anywhere in a line (a multiple of 16 bytes).  A request
// for bytes 0 .. 127 of such a row touches two lines, and with the streaming hint
// both are fetched again for the row's next request.  So the ring takes whole
// lines of memory, `shift` 16-byte pieces of which lie before the step's own, and
// the reads find piece z of the step at piece z + shift: in the step's slot or in
// the one after it, which therefore has to have landed too.  Only the lines at a
// stretch's ends, which a neighbour reads as well, go without the hint.  (The
// experts' up kernel, 64 experts of 1552 rows of 6064 bytes, 593 MB: 94 us against
// 139 us through stream_tile, which fetched 1.5 times as much, and 119 us through
// stream_tile without the hint.)
//
// NB blocks of 16 rows, read by a lane whose loads are pieces 0 .. 2NB-1 of 8 rows;
// KSLOT, KRING: u32x4 in a slot and in the ring, PP in a piece.
template <int NB, int KSLOT, int KRING, int PP>
struct ShiftedRows {
  int back[2 * NB];                      // bytes from the lane's first back to its line's
  int place[2][NB];                      // of the lane's 16 bytes of each block, in the slot
  int turn[2][NB];                       // if in the next slot: what that is away after the last
  int most;                              // the largest of back, over the lanes

  // src[t]: this lane's 16 bytes of piece t in the first step; moved back to the
  // line's.  Before any load into LDS.
  template <int G>
  __device__ __forceinline__ explicit ShiftedRows(const uint8_t* (&src)[G]) {
    const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, l16 = lane & 15;
    uint32_t top = 0;
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t) {
      const uint32_t s = ((uint32_t)((uintptr_t)src[t] >> 4) - (uint32_t)stream_piece(lane)) & 7u;
      top = s > top ? s : top;
      back[t] = 16 * (int)s;
      src[t] -= back[t];
    }
    most = 16 * (int)wave_umax(top);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      // row l16's shift is with the lanes that load it
      const int lo = __shfl(back[2 * j], 8 * (l16 & 7)), hi = __shfl(back[2 * j + 1], 8 * (l16 & 7));
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int z = 4 * c + g + (l16 < 8 ? lo : hi) / 16;
        place[c][j] = (2 * j + (l16 >> 3)) * PP + (l16 & 7) * 8 + ((z + ((l16 & 7) >> 1)) & 7) +
                      (z > 7 ? KSLOT : 0);
        turn[c][j] = z > 7 ? KRING : 0;
      }
    }
  }
  // How many lines hold P steps of rows with `line` bytes left.
  __device__ __forceinline__ int lines(int P, int line) const {
    return P + (128 * P < line + most ? 1 : 0);
  }
  // Where load t finds its 16 bytes of the line `at` bytes on, in a row with k0
  // bytes before the lane's first and `left` after: the rows' ends read zeros.
  __device__ __forceinline__ const uint8_t* from(const uint8_t* src, int t, int at, int k0,
                                                 int left) const {
    const int to = at - back[t];
    return left - to >= 16 && k0 + to >= 0 ? src + at
                                           : reinterpret_cast<const uint8_t*>(&kZeroPiece);
  }
  // The reads of block j's half c; `turned`: from the ring's last slot.
  __device__ __forceinline__ u32x4 read(const u32x4* slot, bool turned, int c, int j) const {
    return lds_read_opaque(slot + place[c][j] - (turned ? turn[c][j] : 0));
  }
  // After the wait, in a last step that has no line after it: nothing is there.
  __device__ __forceinline__ void cut(u32x4& v, int c, int j) const {
    if (turn[c][j]) v = u32x4{0u, 0u, 0u, 0u};
  }
};

// The same for rows of whole lines, for code that serves both.
template <int NB, int KSLOT, int KRING, int PP>
struct WholeRows {
  int place[2];
  template <int G>
  __device__ __forceinline__ explicit WholeRows(const uint8_t* (&)[G]) {
    const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, l16 = lane & 15;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      place[c] = (l16 >> 3) * PP + (l16 & 7) * 8 + ((4 * c + g + ((l16 & 7) >> 1)) & 7);
  }
  __device__ __forceinline__ int lines(int P, int) const { return P; }
  __device__ __forceinline__ const uint8_t* from(const uint8_t* src, int, int at, int,
                                                 int left) const {
    return left - at >= 16 ? src + at : reinterpret_cast<const uint8_t*>(&kZeroPiece);
  }
  __device__ __forceinline__ u32x4 read(const u32x4* slot, bool, int c, int j) const {
    return lds_read_opaque(slot + 2 * j * PP + place[c]);
  }
  __device__ __forceinline__ void cut(u32x4&, int, int) const {}
};
template <bool WHOLE, int NB, int KSLOT, int KRING, int PP>
using StreamRows = std::conditional_t<WHOLE, WholeRows<NB, KSLOT, KRING, PP>,
                                      ShiftedRows<NB, KSLOT, KRING, PP>>;

// stream_tile for such rows; k0: bytes from the row's start to this lane's first.
template <int NB, int AP, int R, typename Acc>
__device__ __forceinline__ void stream_tile_shifted(u32x4* ring,
                                                    const uint8_t* (&src)[2 * NB + AP], int k0,
                                                    int left, int P,
                                                    Acc (&acc)[NB * ((AP + 1) / 2)]) {
  using SH = StreamShape<NB, AP, R>;
  static_assert(SH::valid && R >= 3, "a ring the waits can count, and two slots to read from");
  constexpr int G = SH::G, kPP = SH::kPP, MB = SH::MB;
  const int lane = threadIdx.x & (kWave - 1);
  const int g = lane >> 4, l16 = lane & 15;
  const int line = __builtin_amdgcn_readfirstlane(left);
  const ShiftedRows<NB, SH::kSlot, SH::kRing, kPP> rows(src);
  const int lines = rows.lines(P, line);
  int rpos[2];
#pragma unroll
  for (int c = 0; c < 2; ++c)
    rpos[c] = (l16 >> 3) * kPP + (l16 & 7) * 8 + ((4 * c + g + ((l16 & 7) >> 1)) & 7);

  auto issue = [&](u32x4* slot, int p) {
    const int at = p * 128;
    if (p > 0 && p + 1 < lines && line - at >= 128) {
      static_for<G>([&](auto t_c) {
        constexpr int t = decltype(t_c)::value;
        __builtin_amdgcn_global_load_lds(
            src[t] + at, (__attribute__((address_space(3))) void*)(slot + t * kPP), 16, 0,
            t < 2 * NB ? kStreamAux : 0);
      });
    } else {
      static_for<G>([&](auto t_c) {
        constexpr int t = decltype(t_c)::value;
        const uint8_t* from = src[t] + at;
        if constexpr (t < 2 * NB)
          from = rows.from(src[t], t, at, k0, left);
        else
          from = left - at >= 16 ? from : reinterpret_cast<const uint8_t*>(&kZeroPiece);
        __builtin_amdgcn_global_load_lds(
            from, (__attribute__((address_space(3))) void*)(slot + t * kPP), 16, 0, 0);
      });
    }
    pin_issue();
  };
  u32x4* const end = ring + SH::kRing;
  u32x4 *fill = ring, *use = ring;
  auto next = [&](u32x4* s) { return s + SH::kSlot == end ? ring : s + SH::kSlot; };
  for (int p = 0; p < R - 1 && p < lines; ++p) {
    issue(fill, p);
    fill = next(fill);
  }
  for (int p = 0; p < P; ++p) {
    if (p + R - 1 < lines) {
      issue(fill, p + R - 1);            // into the slot step p-1 was read from
      fill = next(fill);
    }
    stream_wait<R - 2, G>((p + R < lines ? p + R : lines) - (p + 2 < lines ? p + 2 : lines));
    u32x4 v[2 * (NB + MB)];
    const bool turned = next(use) == ring;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int t = 0; t < NB + MB; ++t)
        v[c * (NB + MB) + t] =
            t < NB ? rows.read(use, turned, c, t < NB ? t : 0)
                   : lds_read_opaque(use + 2 * t * kPP + rpos[c]);
    lds_wait(v);
    if (p + 1 == lines) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < NB; ++j) rows.cut(v[c * (NB + MB) + j], c, j);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int b = 0; b < MB; ++b)
          acc[j * MB + b] =
              stream_mfma(v[c * (NB + MB) + NB + b], v[c * (NB + MB) + j], acc[j * MB + b]);
    use = next(use);
  }
}

// Exchange between workgroups.  A slot is a word that is zero until its owner
// writes it, once in a call, with a word that is not (an fp32 value's complement,
// a biased integer); the reader waits for it, whatever order the counter and the
// slots become visible in, and sets it back to zero.  The wait is bounded: a slot
// that stays zero sets the counter line's fault word.
__device__ __forceinline__ uint32_t take_slot(uint32_t* slot, uint32_t w, uint32_t* line) {
  if (w == 0u) {
    const uint64_t t0 = __builtin_amdgcn_s_memrealtime();
    while ((w = load_slot(slot)) == 0u) {
      if (__builtin_amdgcn_s_memrealtime() - t0 > kFoldPollTicks) {
        store_slot(line + kFaultWord, 1u);
        break;
      }
      __builtin_amdgcn_s_sleep(4);
    }
  }
  store_slot(slot, 0u);
  return w;
}

// Whether this workgroup is the last of `total` to arrive at the line; the
// last one sets the count back to zero.
__device__ __forceinline__ bool arrive_last(uint32_t* line, int total, int* lds) {
  if (threadIdx.x == 0) {
    const uint32_t before =
        __hip_atomic_fetch_add(line, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *lds = before == (uint32_t)(total - 1);
    if (*lds) store_slot(line, 0u);
  }
  __syncthreads();
  return *lds != 0;
}

}  // namespace lowm
