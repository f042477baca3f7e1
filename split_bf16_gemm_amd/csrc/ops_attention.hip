// ops_attention.hip -- attention over the paged 8-bit cache (include/lowm_cache.h)
// for gfx950.
//
//   x_t = scale q . k_t ;  out = sum_t e^(x_t - lse) v_t ;  lse = log sum_t e^x_t
//
// One pass over the pages with a running maximum and sum (attend_kernel), and the
// joining of sequences that several workgroups shared (join_kernel).  Bound by HBM
// for few rows: a byte of the cache is read once for up to 32 rows of a key head.
//
// Layout.  Up to 16 RT rows of one key head (a token's query heads that share it,
// token after token) are a tile.  A wavefront takes a page of 64 tokens at a time:
// S^T = K Q^T by v_mfma_f32_16x16x32_f16, tokens as the 16 rows of the result and
// query rows as its columns, so that a lane holds 16 scores of one query row and all
// softmax state is one number a lane.  The tokens of the four score blocks are dealt
// so that a lane's scores are, in order, what the second product O^T = V^T P^T wants
// of that lane: scores go from one matrix instruction to the other without leaving
// their lane.  The cache's layout is what the two products read: a load of 16 bytes a
// lane takes 16 elements of a token's key, or 16 tokens of a value's element, whole
// lines at a time and straight into registers.  The next page's keys load while this
// page's scores are worked on, its values while the keys multiply.
//
// Bytes become fp16 exactly (an int8 by two byte permutations to 1024 + 128 + b and a
// packed subtraction).  A row of q is scaled by a power of two to just below 2^15; e^(x
// - max of the page) by 2^14, so that fp16 keeps what is within 2^-28 of a page's
// largest; the scale of the values and the page's distance to the running maximum are
// one factor on the page's fp32 result.
//
// Work.  The pages of all sequences, heads and tiles are one list that is cut into
// equal runs, one to a workgroup, whatever the lengths are; they are read on the
// device.  A workgroup has at most two tiles that others share, its first and its
// last, and leaves their unfinished sums in two places of its own in the workspace.
#include "ops_cache.cuh"

namespace lowm {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kGroupsLog = 9;                // workgroups: two to a CU
constexpr int kGroups = 1 << kGroupsLog;
constexpr float kLift = 14.f;                // log2 of what e^(x - max) is scaled by
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct AttendArgs {
  lowm_kv_cache cache;
  lowm_sequences seq;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  float* sums;       // [2 kGroups][rows of a tile][D]
  float* stats;      // [2 kGroups][rows of a tile][2]: maximum, sum
  int64_t q_row, q_head;
  int Hq, G, window, rows;   // rows: of a tile
  float scale;               // times log2 e
};

// A sequence's share of the list: its tiles' pages, tile after tile.
struct Share {
  Rows rows;
  int tiles;          // of a key head
  int first, pages;   // first page that a row may see; how many from there
  int64_t units;
  __device__ __forceinline__ Share(const AttendArgs& a, int b) {
    rows = rows_of(a.seq, b);
    tiles = (rows.n * a.G + a.rows - 1) / a.rows;
    const int64_t most = (int64_t)a.seq.W * LOWM_PAGE;
    const int tokens = rows.len < most ? rows.len : (int)most;
    const int64_t from = (int64_t)rows.len - rows.n - a.window + 1;
    first = a.window > 0 && from > 0 ? (int)(from / LOWM_PAGE) : 0;
    pages = (tokens + LOWM_PAGE - 1) / LOWM_PAGE - first;
    if (pages < 0) pages = 0;
    units = (int64_t)a.cache.H * tiles * pages;
  }
};

__device__ __forceinline__ int64_t wave_scan64(int64_t v) {
  uint64_t x = (uint64_t)v;
  auto add = [&](auto move) {
    const uint32_t lo = move((uint32_t)x), hi = move((uint32_t)(x >> 32));
    x += (uint64_t)hi << 32 | lo;
  };
  add([](uint32_t w) { return lane_move<0x111, 0xf>(w); });
  add([](uint32_t w) { return lane_move<0x112, 0xf>(w); });
  add([](uint32_t w) { return lane_move<0x114, 0xf>(w); });
  add([](uint32_t w) { return lane_move<0x118, 0xf>(w); });
  add([](uint32_t w) { return lane_move<0x142, 0xa>(w); });
  add([](uint32_t w) { return lane_move<0x143, 0xc>(w); });
  return (int64_t)x;
}
__device__ __forceinline__ int64_t lane_value(int64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane),
                 hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)v >> 32), lane);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// The whole list, as every wavefront sums it for itself, 64 sequences at a time.
struct List {
  int64_t total;
  int64_t own, upto;     // of sequence `lane`, and up to it (the only step of up to 64)
  __device__ __forceinline__ explicit List(const AttendArgs& a) {
    const int lane = threadIdx.x & (kWave - 1);
    total = 0;
    for (int at = 0; at < a.seq.B; at += kWave) {
      own = at + lane < a.seq.B ? Share(a, at + lane).units : 0;
      upto = wave_scan64(own);
      total += lane_value(upto, kWave - 1);
    }
  }
  // Units of a workgroup's run: a multiple of its wavefronts.
  __device__ __forceinline__ int64_t run() const {
    const int64_t r = (total + kGroups - 1) >> kGroupsLog;
    return (r + kWaves - 1) & ~(int64_t)(kWaves - 1);
  }
  // The sequence that unit u belongs to, and the first of its units.
  __device__ __forceinline__ int find(const AttendArgs& a, int64_t u, int64_t* start) const {
    const int lane = threadIdx.x & (kWave - 1);
    int64_t before = 0, mine = own, sum = upto;
    for (int at = 0; at < a.seq.B; at += kWave) {
      if (a.seq.B > kWave) {
        mine = at + lane < a.seq.B ? Share(a, at + lane).units : 0;
        sum = wave_scan64(mine);
      }
      const int64_t all = lane_value(sum, kWave - 1);
      if (u - before < all) {
        const int first = __builtin_ctzll(__ballot(sum > u - before));
        *start = before + lane_value(sum - mine, first);
        return at + first;
      }
      before += all;
    }
    *start = before;
    return a.seq.B;
  }
};

// Where workgroup w's unfinished sums of a tile are: of the tile that its run begins
// with, or of the one that it ends with.
__device__ __forceinline__ int place_of(int64_t w, bool begins) {
  return 2 * (int)w + (begins ? 0 : 1);
}

__device__ __forceinline__ float bits_float(uint32_t b) { return __builtin_bit_cast(float, b); }
__device__ __forceinline__ uint32_t float_bits(float f) { return __builtin_bit_cast(uint32_t, f); }

// Over the four lanes that share a query row (lane % 16).
template <typename Op>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, Op op) {
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = op(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return op(b[0], b[1]);
}
__device__ __forceinline__ float row_max(float v) {
  return bits_float(row_reduce(float_bits(v), [](uint32_t a, uint32_t b) {
    return float_bits(fmaxf(bits_float(a), bits_float(b)));
  }));
}
__device__ __forceinline__ float row_sum(float v) {
  return bits_float(row_reduce(float_bits(v), [](uint32_t a, uint32_t b) {
    return float_bits(bits_float(a) + bits_float(b));
  }));
}
__device__ __forceinline__ uint32_t row_umax(uint32_t v) {
  return row_reduce(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// Eight bytes of the cache as fp16.
template <bool E4M3>
__device__ __forceinline__ f16x8 widen(uint32_t a, uint32_t b) {
  f16x2 h[4];
  if constexpr (E4M3) {
    h[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, false);
    h[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, true);
    h[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, false);
    h[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, true);
  } else {
    const f16x2 bias = {(_Float16)1152.f, (_Float16)1152.f};
    a ^= 0x80808080u;
    b ^= 0x80808080u;
    h[0] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, a, 0x04010400u)) - bias;
    h[1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u)) - bias;
    h[2] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u)) - bias;
    h[3] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u)) - bias;
  }
  f16x8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[2 * i] = h[i][0];
    r[2 * i + 1] = h[i][1];
  }
  return r;
}
__device__ __forceinline__ f32x4 product(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
// Keeps the loads above it above what follows.
__device__ __forceinline__ void pin_loads() { asm volatile("" ::: "memory"); }

// DP blocks of 64 elements of a head, all of them there (FULL) or not, RT blocks of 16
// rows to a tile.
template <int DP, bool FULL, int RT, bool E4M3>
__global__ __launch_bounds__(kThreads, DP * RT <= 2 ? 2 : 1) void attend_kernel(AttendArgs a) {
  constexpr int NT = 4 * DP;                // blocks of 16 elements
  constexpr int kRows = 16 * RT;
  constexpr int kPart = DP == 1 ? 4 : DP == 3 ? 6 : 8;   // joined through LDS at a time
  static_assert(NT % kPart == 0, "whole parts");
  constexpr int kPitch = 16 * kPart + 4;    // lanes' rows in distinct banks
  __shared__ __align__(16) float joint[kWaves][kRows][kPitch];
  __shared__ float joint_max[kWaves][kRows], joint_sum[kWaves][kRows];

  const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const lowm_kv_cache& c = a.cache;
  const int D = FULL ? 64 * DP : c.D, nt = FULL ? NT : D / 16;

  const List list(a);
  const int64_t run = list.run();
  int64_t u = (int64_t)blockIdx.x * run;
  const int64_t begin = u, end = u + run < list.total ? u + run : list.total;
  if (u >= end) return;
  int64_t start;
  int b = list.find(a, u, &start);

  while (u < end) {
    const Share s(a, b);
    if (u - start >= s.units) {
      start += s.units;
      ++b;
      continue;
    }
    const int64_t tile_at = (u - start) / s.pages;
    const int page_at = (int)(u - start - tile_at * s.pages);
    const int64_t room = end - u;
    const int pages = s.pages - page_at < room ? s.pages - page_at : (int)room;
    const int head = (int)(tile_at / s.tiles), tile = (int)(tile_at - (int64_t)head * s.tiles);
    const int row0 = tile * kRows, last_row = s.rows.n * a.G - 1;

    // rows: what they see, and their queries as the matrix operand
    int see_lo[RT], see_hi[RT];
    float unit[RT];
    f16x8 q[RT][2 * DP];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int r = row0 + 16 * t + col, in = r <= last_row ? r : last_row;
      const int j = in / a.G, h = head * a.G + (in - j * a.G), pos = s.rows.position(j);
      see_hi[t] = r <= last_row ? pos : -1;
      see_lo[t] = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
      const uint16_t* x = a.q + (s.rows.first + j) * a.q_row + h * a.q_head;
      ops_u32x4 raw[2 * DP];
      uint32_t top = 0;
#pragma unroll
      for (int m = 0; m < 2 * DP; ++m) {
        const int d = 64 * (m / 2) + 16 * g + 8 * (m % 2);
        raw[m] = ops_u32x4{0u, 0u, 0u, 0u};
        if (FULL || m < 2 * DP - 2 || d < D) raw[m] = *reinterpret_cast<const ops_u32x4*>(x + d);
      }
#pragma unroll
      for (int m = 0; m < 2 * DP; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = raw[m][i], lo = w << 16 & 0x7fffffffu, hi = w & 0x7fff0000u;
          top = top > lo ? top : lo;
          top = top > hi ? top : hi;
        }
      top = row_umax(top);
      // 2^(14 - exponent of the largest), within what fp32 has
      const int e = (int)(top >> 23), up = 127 + 14 - (e - 127);
      const float lift = bits_float((uint32_t)(up < 1 ? 1 : up > 254 ? 254 : up) << 23);
      unit[t] = top < 0x7f800000u ? a.scale / lift : __builtin_nanf("");
#pragma unroll
      for (int m = 0; m < 2 * DP; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = raw[m][i];
          q[t][m][2 * i] = (_Float16)(bf16_lo(w) * lift);
          q[t][m][2 * i + 1] = (_Float16)(bf16_hi(w) * lift);
        }
    }
    // positions of the tile's first and last row: pages past the last are not seen
    const int low = s.rows.position(row0 / a.G);
    const int high = s.rows.position((row0 + kRows - 1 < last_row ? row0 + kRows - 1 : last_row) / a.G);
    const int high_lo = a.window > 0 && high >= a.window ? high - a.window + 1 : 0;
    const int seen = high < 0 ? 0 : high / LOWM_PAGE + 1 - s.first;
    const int stop = page_at + pages < seen ? page_at + pages : seen;
    const int* table = a.seq.table + b * a.seq.table_ld + s.first;

    float most[RT], sum[RT];
    f32x4 o[RT][NT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      most[t] = -__builtin_inff();
      sum[t] = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) o[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    ops_u32x4 keys[4][DP], vals[NT];
    float k_scale = 0.f, v_scale = 0.f;
    int page = -1;
    // The token of row r of score block i is 16 (r / 4) + 4 i + r % 4: then lane group
    // g has tokens 16 g .. 16 g + 15, in the order of the values' bytes.
    auto load_keys = [&](int at) {
      page = table[at];
      const bool some = page >= 0 && page < c.P;
      const int64_t from = (int64_t)(some ? page : 0) * c.H + head;
      const uint8_t* p = static_cast<const uint8_t*>(c.k) + from * (LOWM_PAGE * D);
      k_scale = some ? c.k_scale[from] : 0.f;
      v_scale = some ? c.v_scale[from] : 0.f;
      if (!some) page = -1;
#pragma unroll
      for (int m = 0; m < DP; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int piece = 4 * m + g;
          const uint8_t* x = p + (piece * LOWM_PAGE + 16 * (col >> 2) + 4 * i + (col & 3)) * 16;
          keys[i][m] = ops_u32x4{0u, 0u, 0u, 0u};
          if (FULL || m < DP - 1 || piece * 16 < D) keys[i][m] = *reinterpret_cast<const ops_u32x4*>(x);
        }
      pin_loads();
    };
    auto load_vals = [&]() {
      const uint8_t* p = static_cast<const uint8_t*>(c.v) +
                         ((int64_t)(page < 0 ? 0 : page) * c.H + head) * (LOWM_PAGE * D);
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (FULL || n < NT - 4 || n < nt)
          vals[n] = *reinterpret_cast<const ops_u32x4*>(p + (g * D + 16 * n + col) * 16);
      pin_loads();
    };

    int at = page_at + wave;
    if (at < stop) load_keys(at);
    for (; at < stop; at += kWaves) {
      const int token0 = (s.first + at) * LOWM_PAGE;
      // tokens of the page that are there at all
      int live = s.rows.len - token0;
      live = page < 0 ? 0 : live < LOWM_PAGE ? live : LOWM_PAGE;
      const float ks = k_scale, vs = v_scale;
      load_vals();

      f32x4 x[RT][4];
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < DP; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f16x8 k0 = widen<E4M3>(keys[i][m][0], keys[i][m][1]),
                      k1 = widen<E4M3>(keys[i][m][2], keys[i][m][3]);
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            x[t][i] = product(k0, q[t][2 * m], x[t][i]);
            x[t][i] = product(k1, q[t][2 * m + 1], x[t][i]);
          }
        }
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[t][i] *= unit[t] * ks;
      if (at + kWaves < stop) load_keys(at + kWaves);

      if (live < LOWM_PAGE || token0 + LOWM_PAGE - 1 > low || token0 < high_lo) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int token = token0 + 16 * g + 4 * i + e;
              const bool sees = live > 0 && token >= see_lo[t] && token <= see_hi[t];
              x[t][i][e] = sees ? x[t][i][e] : -__builtin_inff();
            }
      }

      f16x8 p[RT][2];
      float keep[RT], take[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        float here = x[t][0][0];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) here = fmaxf(here, x[t][i][e]);
        here = row_max(here);
        const bool none = here == -__builtin_inff();
        const float from = none ? 0.f : here - kLift;
        const float now = fmaxf(most[t], here), base = now == -__builtin_inff() ? 0.f : now;
        const float rise = __builtin_amdgcn_exp2f(here - base);
        keep[t] = __builtin_amdgcn_exp2f(most[t] - base);
        take[t] = none ? 0.f : rise * vs;
        most[t] = now;
        float add = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w = __builtin_amdgcn_exp2f(x[t][i][e] - from);
            add += w;
            p[t][i / 2][4 * (i % 2) + e] = (_Float16)w;
          }
        sum[t] = sum[t] * keep[t] + add * rise;
      }
      if (E4M3 && live < LOWM_PAGE) {
        // what lies behind the sequence may be any byte, a NaN among them
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int left = live - 16 * g - 4 * i;
            const uint32_t mask = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << 8 * left) - 1;
            vals[n][i] &= mask;
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (!FULL && n >= NT - 4 && n >= nt) continue;
        const f16x8 v0 = widen<E4M3>(vals[n][0], vals[n][1]),
                    v1 = widen<E4M3>(vals[n][2], vals[n][3]);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          f32x4 y = {0.f, 0.f, 0.f, 0.f};
          y = product(v0, p[t][0], y);
          y = product(v1, p[t][1], y);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][n][e] = o[t][n][e] * keep[t] + y[e] * take[t];
        }
      }
    }

    // the four wavefronts' sums of the tile
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float all = row_sum(sum[t]);
      if (g == 0) {
        joint_max[wave][16 * t + col] = most[t];
        joint_sum[wave][16 * t + col] = all;
      }
    }
    const bool whole = page_at == 0 && pages == s.pages;
    const int place = place_of(blockIdx.x, u == begin);
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += kPart) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int n = 0; n < kPart; ++n)
          *reinterpret_cast<f32x4*>(&joint[wave][16 * t + col][16 * n + 4 * g]) = o[t][n0 + n];
      __syncthreads();
      for (int i = threadIdx.x; i < kRows * 4 * kPart; i += kThreads) {
        const int r = i / (4 * kPart), d4 = i % (4 * kPart), d = 16 * n0 + 4 * d4;
        if (row0 + r > last_row || (!FULL && d >= D)) continue;
        float top = joint_max[0][r];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, joint_max[w][r]);
        const float base = top == -__builtin_inff() ? 0.f : top;
        float all = 0.f;
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float f = __builtin_amdgcn_exp2f(joint_max[w][r] - base);
          all += f * joint_sum[w][r];
          const f32x4 z = *reinterpret_cast<const f32x4*>(&joint[w][r][4 * d4]);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] += f * z[e];
        }
        if (whole) {
          const int j = (row0 + r) / a.G, h = head * a.G + (row0 + r - j * a.G);
          const int64_t row = (int64_t)(s.rows.first + j) * a.Hq + h;
          const float k = all == 0.f ? 0.f : 1.f / all;
          *reinterpret_cast<ops_u32x2*>(a.out + row * D + d) =
              ops_u32x2{pack_bf16(y[0] * k, y[1] * k), pack_bf16(y[2] * k, y[3] * k)};
          if (a.lse && d == 0)
            a.lse[row] = (top + __builtin_amdgcn_logf(all) - kLift) * kLn2;
        } else {
          const int64_t row = (int64_t)place * kRows + r;
          *reinterpret_cast<f32x4*>(a.sums + row * D + d) = y;
          if (d == 0) {
            a.stats[2 * row] = top;
            a.stats[2 * row + 1] = all;
          }
        }
      }
      __syncthreads();
    }
    u += pages;
  }
}

// A workgroup to a row: nothing to do for tiles that one workgroup had whole; zeros
// for rows of sequences without pages; the sums of the others joined in the order of
// their pages, 64 at a time.
__global__ __launch_bounds__(kThreads) void join_kernel(AttendArgs a) {
  constexpr int kStep = 64;
  __shared__ float factor[kStep];
  __shared__ float total[2];
  __shared__ __align__(16) f32x4 part[kThreads];
  const int lane = threadIdx.x & (kWave - 1);
  const int D = a.cache.D;
  const int64_t row = blockIdx.x;
  const int token = (int)(row / a.Hq), h = (int)(row % a.Hq), head = h / a.G;

  // the sequence that the row belongs to, and the units before its own
  int b = -1;
  int64_t start = 0;
  const List list(a);
  if (!a.seq.row_starts) {
    b = token / (a.seq.T / a.seq.B);
  } else {
    for (int at = 0; at < a.seq.B && b < 0; at += kWave) {
      bool mine = false;
      if (at + lane < a.seq.B) {
        const Rows r = rows_of(a.seq, at + lane);
        mine = token >= r.first && token < r.first + r.n;
      }
      const uint64_t who = __ballot(mine);
      if (who) b = at + __builtin_ctzll(who);
    }
    if (b < 0) return;
  }
  if (a.seq.B <= kWave) {
    start = lane_value(list.upto - list.own, b);
  } else {
    for (int at = 0; at <= b; at += kWave) {
      const int64_t own = at + lane < b ? Share(a, at + lane).units : 0;
      start += lane_value(wave_scan64(own), kWave - 1);
    }
  }
  const Share s(a, b);
  if (s.pages == 0) {
    for (int d = threadIdx.x; d < D; d += kThreads) a.out[row * D + d] = 0;
    if (a.lse && threadIdx.x == 0) a.lse[row] = -__builtin_inff();
    return;
  }
  const int r = (token - s.rows.first) * a.G + (h - head * a.G), tile = r / a.rows,
            in = r - tile * a.rows;
  const int64_t run = list.run();
  const int64_t first = start + ((int64_t)head * s.tiles + tile) * s.pages,
                last = first + s.pages - 1;
  const int64_t w0 = first / run, w1 = last / run;
  if (w0 == w1) return;
  const int n = (int)(w1 - w0) + 1;
  const bool begins = first == w0 * run;
  auto at = [&](int i) {
    return (int64_t)place_of(w0 + i, i > 0 || begins) * a.rows + in;
  };

  // 16, 32 or 64 lanes to a place's row, four elements to a lane
  const int lanes = D <= 64 ? 16 : D <= 128 ? 32 : 64;
  const int sets = kThreads / lanes, set = threadIdx.x / lanes, d = (int)threadIdx.x % lanes * 4;
  float most = -__builtin_inff(), sum = 0.f;
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
  for (int i0 = 0; i0 < n; i0 += kStep) {
    const int m = n - i0 < kStep ? n - i0 : kStep;
    float keep = 1.f;
    if (i0 > 0) __syncthreads();
    if (threadIdx.x < kWave) {
      float x = -__builtin_inff(), z = 0.f;
      if (lane < m) {
        const float* p = a.stats + 2 * at(i0 + lane);
        x = p[0];
        z = p[1];
      }
      float now = x;
#pragma unroll
      for (int k = 1; k < kWave; k *= 2) now = fmaxf(now, __shfl_xor(now, k));
      now = fmaxf(now, most);
      const float base = now == -__builtin_inff() ? 0.f : now;
      const float f = __builtin_amdgcn_exp2f(x - base);
      keep = __builtin_amdgcn_exp2f(most - base);
      sum = sum * keep + wave_sum(lane < m ? f * z : 0.f);
      most = now;
      factor[lane] = f;
      if (lane == 0) total[0] = keep;
    }
    __syncthreads();
    keep = total[0];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] *= keep;
    if (d < D) {
#pragma unroll 8
      for (int i = set; i < m; i += sets) {
        const f32x4 z = *reinterpret_cast<const f32x4*>(a.sums + at(i0 + i) * D + d);
        const float f = factor[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += f * z[e];
      }
    }
  }
  part[threadIdx.x] = y;
  if (threadIdx.x == 0) {
    total[1] = sum;
    if (a.lse) a.lse[row] = (most + __builtin_amdgcn_logf(sum) - kLift) * kLn2;
  }
  __syncthreads();
  if (set > 0 || d >= D) return;
  for (int i = 1; i < sets; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] += part[i * lanes + threadIdx.x][e];
  const float k = total[1] == 0.f ? 0.f : 1.f / total[1];
  *reinterpret_cast<ops_u32x2*>(a.out + row * D + d) =
      ops_u32x2{pack_bf16(y[0] * k, y[1] * k), pack_bf16(y[2] * k, y[3] * k)};
}

template <int DP, bool FULL>
const void* kernel_for(int rt, bool e4m3) {
  if (rt == 1)
    return e4m3 ? (const void*)&attend_kernel<DP, FULL, 1, true>
                : (const void*)&attend_kernel<DP, FULL, 1, false>;
  return e4m3 ? (const void*)&attend_kernel<DP, FULL, 2, true>
              : (const void*)&attend_kernel<DP, FULL, 2, false>;
}
const void* kernel_for(int D, int rt, bool e4m3) {
  switch ((D + 63) / 64) {
    case 1: return D == 64 ? kernel_for<1, true>(rt, e4m3) : kernel_for<1, false>(rt, e4m3);
    case 2: return D == 128 ? kernel_for<2, true>(rt, e4m3) : kernel_for<2, false>(rt, e4m3);
    case 3: return D == 192 ? kernel_for<3, true>(rt, e4m3) : kernel_for<3, false>(rt, e4m3);
    default: return D == 256 ? kernel_for<4, true>(rt, e4m3) : kernel_for<4, false>(rt, e4m3);
  }
}

// Rows of a tile that a workspace has room for.
int64_t room_rows(int T, int G) { return (int64_t)T * G <= 16 ? 16 : 32; }
size_t workspace_bytes(int T, int G, int D) {
  return (size_t)(2 * kGroups * room_rows(T, G) * (D + 2) * 4);
}

int cache_attention(const lowm_cache_attention_args* u, hipStream_t stream) {
  if (!u) return LOWM_ERR_INVALID_ARG;
  const lowm_kv_cache& c = u->cache;
  const lowm_sequences& s = u->seq;
  int rc = check_sequences(s);
  if (rc == LOWM_OK) rc = check_cache(c);
  if (rc != LOWM_OK) return rc;
  if (c.layers != 1 || u->Hq < 1 || u->Hq % c.H || u->window < 0) return LOWM_ERR_INVALID_ARG;
  if (u->Hq > LOWM_CACHE_MAX_HEADS || (int64_t)s.T * u->Hq > INT32_MAX) return LOWM_ERR_UNSUPPORTED;
  if (s.T == 0) return LOWM_OK;
  if (!u->q || !u->out) return LOWM_ERR_INVALID_ARG;
  if (!aligned_to(u->q, 16) || !aligned_to(u->out, 16) || !aligned_to(u->lse, 4) ||
      u->q_row % 8 || u->q_head % 8)
    return LOWM_ERR_UNSUPPORTED;
  if (!heads_apart(s.T, u->Hq, c.D, u->q_row, u->q_head)) return LOWM_ERR_INVALID_ARG;
  const int G = u->Hq / c.H;
  const size_t need = workspace_bytes(s.T, G, c.D);
  if (!u->workspace || u->workspace_bytes < need) return LOWM_ERR_WORKSPACE;
  if (!aligned_to(u->workspace, 256)) return LOWM_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)s.T * u->Hq;
  const Span q = span_of(Heads{u->q, s.T, u->Hq, c.D, u->q_row, u->q_head, 2}),
             out[] = {plain_span(u->out, rows * c.D, 2), plain_span(u->lse, rows, 4),
                      plain_span(u->workspace, (int64_t)need, 1)};
  const CacheSpans cs(c);
  const SequenceSpans ss(s);
  for (int i = 0; i < 3; ++i) {
    if (meet(out[i], q) || cs.meets(out[i]) || ss.meets(out[i])) return LOWM_ERR_INVALID_ARG;
    for (int k = 0; k < i; ++k)
      if (meet(out[i], out[k])) return LOWM_ERR_INVALID_ARG;
  }
  // Two blocks of rows to a tile where a sequence has more than one block, on average.
  const int rt = room_rows(s.T, G) == 32 && (int64_t)s.T * G > (int64_t)s.B * 16 ? 2 : 1;
  AttendArgs a{};
  a.cache = c;
  a.seq = s;
  a.q = static_cast<const uint16_t*>(u->q);
  a.out = static_cast<uint16_t*>(u->out);
  a.lse = u->lse;
  a.rows = 16 * rt;
  a.stats = static_cast<float*>(u->workspace);
  a.sums = a.stats + 2 * kGroups * a.rows * 2;
  a.q_row = u->q_row;
  a.q_head = u->q_head;
  a.Hq = u->Hq;
  a.G = G;
  a.window = u->window;
  a.scale = u->scale * kLog2e;
  void* args[] = {&a};
  rc = launched(hipLaunchKernel(kernel_for(c.D, rt, c.type == LOWM_E4M3), dim3(kGroups),
                                dim3(kThreads), args, 0, stream));
  if (rc != LOWM_OK) return rc;
  return launched(hipLaunchKernel((const void*)&join_kernel, dim3((unsigned)rows), dim3(kThreads),
                                  args, 0, stream));
}

}  // namespace
}  // namespace lowm

extern "C" {

size_t lowm_cache_attention_workspace_bytes(int T, int Hq, int H, int D) {
  if (T < 1 || H < 1 || Hq < 1 || Hq % H || Hq > LOWM_CACHE_MAX_HEADS || D < 16 || D % 16 ||
      D > LOWM_CACHE_MAX_D || (int64_t)T * Hq > INT32_MAX)
    return 0;
  return lowm::workspace_bytes(T, Hq / H, D);
}

int lowm_cache_attention(const lowm_cache_attention_args* args, void* stream) {
  return lowm::cache_attention(args, static_cast<hipStream_t>(stream));
}

}  // extern "C"
