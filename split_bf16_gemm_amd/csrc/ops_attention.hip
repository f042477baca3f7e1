// ops_attention.hip -- attention over the paged 8-bit cache (include/lowm_cache.h)
// for gfx950.
//
//   x_t = scale q . k_t ;  out = sum_t e^(x_t - lse) v_t ;  lse = log sum_t e^x_t
//
// One pass over the pages with a running maximum and sum, in one launch.  Bound by HBM
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
// device.  A tile counts as kTileCost pages more than it has, so that many short
// sequences are spread like one long one.  A run has at most two tiles that others
// share, its first and its last, and leaves its sums of them in two places of its own
// in the workspace; the last of a tile's runs to arrive at its counter joins them, in the
// order of the pages, so that the bits do not depend on who that is.
//
// The exchange.  Sums go to the workspace with device-scope stores, which pass the
// XCDs' own caches; a workgroup waits until its stores are acknowledged there and then
// adds to the counter, and who finds the others' additions reads with device-scope
// loads.  No cache is written back or invalidated, and nobody waits for another
// workgroup.  Counters are zero between calls: who joins clears them.
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
constexpr int kJoin = 32;                    // places joined at once
constexpr int kTileCost = 8;                 // what a tile costs beside its pages, in pages
constexpr float kLift = 7.f;                 // log2 of what weights are scaled by, and how
constexpr float kSlack = 8.f;                // far the largest may pass its reference
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct AttendArgs {
  lowm_kv_cache cache;
  lowm_sequences seq;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int* counts;       // [2][2 kGroups]: arrivals in a group of places, and of groups
  float* sums;       // [2 kGroups][rows of a tile][D]
  float* stats;      // [2 kGroups][rows of a tile][2]: maximum, sum
  int64_t q_row, q_head;
  int Hq, G, window, rows;   // rows: of a tile
  float scale;               // times log2 e
};

// A sequence's share of the list: its tiles, each kTileCost units that stand for no page,
// then its pages.
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
    units = (int64_t)a.cache.H * tiles * (pages + kTileCost);
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

// Where the unfinished sums of a tile that run w has a part of are: of the one tile that
// an earlier run began, or of the one that this run begins and a later one ends.
__device__ __forceinline__ int place_of(int64_t w, bool begun) { return 2 * (int)w + !begun; }

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
// Device-scope accesses, eight bytes at a time.
__device__ __forceinline__ void put2(float* p, float a, float b) {
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), (uint64_t)float_bits(b) << 32 | float_bits(a),
                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
struct Two {
  float a, b;
};
__device__ __forceinline__ Two get2(const float* p) {
  const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
  return {bits_float((uint32_t)v), bits_float((uint32_t)(v >> 32))};
}

// One more arrival at a counter, after all stores of the workgroup; whether it was the
// last of n, which clears the counter.  Every thread gets the answer.
__device__ __forceinline__ bool arrive(int* count, int n, int* lds) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) {
    const int before =
        __hip_atomic_fetch_add(count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (before == n - 1)
      __hip_atomic_store(count, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *lds = before == n - 1;
  }
  __syncthreads();
  const bool last = *lds != 0;
  __syncthreads();
  return last;
}

// Where a tile's rows go.
struct TileRows {
  int row0, last_row, head, first;   // first row of the tile, last of the sequence's
  __device__ __forceinline__ int64_t at(const AttendArgs& a, int r) const {
    const int j = (row0 + r) / a.G;
    return (int64_t)(first + j) * a.Hq + head * a.G + (row0 + r - j * a.G);
  }
};
__device__ __forceinline__ void finish(const AttendArgs& a, const TileRows& rows, int r, int d,
                                       float most, float sum, const f32x4& y) {
  const int64_t row = rows.at(a, r);
  const float k = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<ops_u32x2*>(a.out + row * a.cache.D + d) =
      ops_u32x2{pack_bf16(y[0] * k, y[1] * k), pack_bf16(y[2] * k, y[3] * k)};
  if (a.lse && d == 0) a.lse[row] = (most + __builtin_amdgcn_logf(sum) - kLift) * kLn2;
}

// m places' sums joined: place i is of run w + i * step, of the tile that it begins
// (w + i * step == w0) or of the one it continues.  To the rows, or to place 0.
__device__ void join(const AttendArgs& a, const TileRows& rows, int64_t w0, int64_t w, int step,
                     int m, bool last, float* lds) {
  const int n = rows.last_row - rows.row0 + 1 < a.rows ? rows.last_row - rows.row0 + 1 : a.rows;
  const int D = a.cache.D;
  float *most = lds, *sum = lds + kJoin * a.rows;
  auto at = [&](int i, int r) {
    const int64_t run = w + (int64_t)i * step;
    return (int64_t)place_of(run, run > w0) * a.rows + r;
  };
  for (int i = threadIdx.x; i < m * n; i += kThreads) {
    const Two v = get2(a.stats + 2 * at(i / n, i % n));
    most[i] = v.a;
    sum[i] = v.b;
  }
  __syncthreads();
  for (int item = threadIdx.x; item < n * (D / 4); item += kThreads) {
    const int r = item / (D / 4), d = item % (D / 4) * 4;
    float top = -__builtin_inff();
    for (int i = 0; i < m; ++i) top = fmaxf(top, most[i * n + r]);
    const float base = top == -__builtin_inff() ? 0.f : top;
    float all = 0.f;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int i = 0; i < m; ++i) {
      const float* p = a.sums + at(i, r) * D + d;
      const Two lo = get2(p), hi = get2(p + 2);
      const float f = __builtin_amdgcn_exp2f(most[i * n + r] - base);
      all += f * sum[i * n + r];
      y[0] += f * lo.a;
      y[1] += f * lo.b;
      y[2] += f * hi.a;
      y[3] += f * hi.b;
    }
    if (last) {
      finish(a, rows, r, d, top, all, y);
    } else {
      float* p = a.sums + at(0, r) * D + d;
      put2(p, y[0], y[1]);
      put2(p + 2, y[2], y[3]);
      if (d == 0) put2(a.stats + 2 * at(0, r), top, all);
    }
  }
  __syncthreads();
}

// Keeps the loads above it above what follows.
__device__ __forceinline__ void pin_loads() { asm volatile("" ::: "memory"); }

// DP blocks of 64 elements of a head, all of them there (FULL) or not, RT blocks of 16
// rows to a tile.
template <int DP, bool FULL, int RT, bool E4M3>
__global__ __launch_bounds__(kThreads, DP * RT <= 4 ? 2 : 1) void attend_kernel(AttendArgs a) {
  constexpr int NT = 4 * DP;                // blocks of 16 elements
  constexpr int kRows = 16 * RT;
  constexpr int kPart = DP == 1 ? 4 : DP == 3 ? 6 : 8;   // joined through LDS at a time
  static_assert(NT % kPart == 0, "whole parts");
  constexpr int kPitch = 16 * kPart + 4;    // lanes' rows in distinct banks
  __shared__ __align__(16) float joint[kWaves][kRows][kPitch];
  __shared__ float joint_max[kWaves][kRows], joint_sum[kWaves][kRows];
  __shared__ int arrived;
  static_assert(sizeof(joint) >= 2 * kJoin * kRows * sizeof(float), "room to join");

  const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const lowm_kv_cache& c = a.cache;
  const int D = FULL ? 64 * DP : c.D, nt = FULL ? NT : D / 16;

  const List list(a);
  const int64_t run = list.run();
  // runs that have units, an eighth of them to each XCD: neighbours, which may share a
  // head's pages, share an L2
  const int64_t runs = (list.total + run - 1) / (run > 0 ? run : 1);
  const int64_t w = (blockIdx.x % 8) * ((runs + 7) / 8) + blockIdx.x / 8;
  if ((int64_t)blockIdx.x / 8 >= (runs + 7) / 8 || w >= runs) return;
  int64_t u = w * run;
  const int64_t end = u + run < list.total ? u + run : list.total;
  int64_t start;
  int b = list.find(a, u, &start);

  while (u < end) {
    const Share s(a, b);
    if (u - start >= s.units) {
      start += s.units;
      ++b;
      continue;
    }
    // a tile's units: kTileCost that stand for no page, then its pages
    const int64_t tile_at = (u - start) / (s.pages + kTileCost);
    const int from = (int)(u - start - tile_at * (s.pages + kTileCost));
    const int64_t room = end - u;
    const int units = s.pages + kTileCost - from < room ? s.pages + kTileCost - from : (int)room;
    u += units;
    const int page_at = from > kTileCost ? from - kTileCost : 0,
              pages = from + units - kTileCost - page_at;
    const int head = (int)(tile_at / s.tiles), tile = (int)(tile_at - (int64_t)head * s.tiles);
    const int row0 = tile * kRows, last_row = s.rows.n * a.G - 1;
    const TileRows rows{row0, last_row, head, s.rows.first};
    if (pages <= 0) {
      // whoever has the first unit of a tile without pages writes its rows
      if (s.pages == 0 && from == 0)
        for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads)
          if (row0 + i / (D / 4) <= last_row)
            finish(a, rows, i / (D / 4), i % (D / 4) * 4, -__builtin_inff(), 0.f,
                   f32x4{0.f, 0.f, 0.f, 0.f});
      continue;
    }
    // positions of the tile's first and last row: pages past the last are not seen
    const int low = s.rows.position(row0 / a.G);
    const int high = s.rows.position((row0 + kRows - 1 < last_row ? row0 + kRows - 1 : last_row) / a.G);
    const int high_lo = a.window > 0 && high >= a.window ? high - a.window + 1 : 0;
    const int seen = high < 0 ? 0 : high / LOWM_PAGE + 1 - s.first;
    const int stop = page_at + pages < seen ? page_at + pages : seen;
    const int* table = a.seq.table + b * a.seq.table_ld + s.first;

    ops_u32x4 keys[4][DP], vals[NT];
    float k_scale = 0.f, v_scale = 0.f;
    int page = -1, next_page = -1;
    // The token of row r of score block i is 16 (r / 4) + 4 i + r % 4: then lane group
    // g has tokens 16 g .. 16 g + 15, in the order of the values' bytes.
    auto load_keys = [&]() {
      page = next_page >= 0 && next_page < c.P ? next_page : -1;
      const int64_t at = (int64_t)(page < 0 ? 0 : page) * c.H + head;
      const uint8_t* p = static_cast<const uint8_t*>(c.k) + at * (LOWM_PAGE * D);
      k_scale = c.k_scale[at];
      v_scale = c.v_scale[at];
#pragma unroll
      for (int m = 0; m < DP; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int piece = 4 * m + g;
          const uint8_t* x = p + (piece * LOWM_PAGE + 16 * (col >> 2) + 4 * i + (col & 3)) * 16;
          keys[i][m] = ops_u32x4{0u, 0u, 0u, 0u};
          if (FULL || m < DP - 1 || piece * 16 < D)
            keys[i][m] = *reinterpret_cast<const ops_u32x4*>(x);
        }
      pin_loads();
    };
    auto load_vals = [&]() {
      const uint8_t* p = static_cast<const uint8_t*>(c.v) +
                         ((int64_t)(page < 0 ? 0 : page) * c.H + head) * (LOWM_PAGE * D);
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (FULL || n < NT - 4 || n < nt)
          vals[n] = __builtin_nontemporal_load(
              reinterpret_cast<const ops_u32x4*>(p + (g * D + 16 * n + col) * 16));
      pin_loads();
    };
    // the number of a page is read a turn before its keys
    int at = page_at + wave;
    if (at < stop) {
      next_page = table[at];
      load_keys();
      next_page = table[at + kWaves < stop ? at + kWaves : at];
    }

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
      // 2^(14 - exponent of the largest), within what fp32 has; with the sign of the
      // scale, so that larger products are larger scores
      const int e = (int)(top >> 23), up = 127 + 14 - (e - 127);
      const float lift = bits_float((uint32_t)(up < 1 ? 1 : up > 254 ? 254 : up) << 23);
      const float signed_lift = a.scale < 0.f ? -lift : lift;
      unit[t] = top < 0x7f800000u ? a.scale / signed_lift : __builtin_nanf("");
#pragma unroll
      for (int m = 0; m < 2 * DP; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = raw[m][i];
          q[t][m][2 * i] = (_Float16)(bf16_lo(w) * signed_lift);
          q[t][m][2 * i + 1] = (_Float16)(bf16_hi(w) * signed_lift);
        }
    }

    // Weights are e^(x + log vs - ref) 2^kLift with vs the page's scale of the values in
    // units of the first page's, v0: they multiply the bytes as they are, and go into the
    // sums o without another factor.  ref is the largest x + log vs so far, or up to
    // kSlack less: the sums are scaled anew only when a page passes that.
    float ref[RT], sum[RT], v0 = 0.f;
    f32x4 o[RT][NT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      ref[t] = -__builtin_inff();
      sum[t] = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) o[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    for (; at < stop; at += kWaves) {
      const int token0 = (s.first + at) * LOWM_PAGE;
      // tokens of the page that are there at all
      int live = s.rows.len - token0;
      live = page < 0 ? 0 : live < LOWM_PAGE ? live : LOWM_PAGE;
      const float ks = live > 0 ? k_scale : 0.f, vs = live > 0 ? v_scale : 0.f;
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
      if (at + kWaves < stop) {
        load_keys();
        next_page = table[at + 2 * kWaves < stop ? at + 2 * kWaves : at];
      }

      // a scale of 0 (or one too small to be a number with a logarithm) leaves no value
      const bool some = !(fabsf(vs) < 1.17549435e-38f);
      if (v0 == 0.f && some && vs > 0.f && vs < __builtin_inff()) v0 = vs;
      const float vs_here = some ? vs / (v0 == 0.f ? 1.f : v0) : 1.f,
                  log_vs = __builtin_amdgcn_logf(vs_here), per_vs = 1.f / vs_here;

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
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        // never 0, which would make NaN of the masked ones
        float per = unit[t] * ks;
        per = per == 0.f ? 1e-38f : per;
        float here = x[t][0][0];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) here = fmaxf(here, x[t][i][e]);
        here = row_max(here);
        // a row that sees none of the page is not touched by its scales
        const bool none = here == -__builtin_inff();
        here = here * per + log_vs;
        per = none ? 1.f : per;
        if (__any(here > ref[t] + kSlack)) {
          const float now = here > ref[t] + kSlack ? here : ref[t];
          const float keep = now == ref[t] ? 1.f : __builtin_amdgcn_exp2f(ref[t] - now);
          ref[t] = now;
          sum[t] *= keep;
#pragma unroll
          for (int n = 0; n < NT; ++n) o[t][n] *= keep;
        }
        const float lift =
            none ? 0.f : log_vs + kLift - (ref[t] == -__builtin_inff() ? 0.f : ref[t]);
        float add = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][i][e], per, lift));
            add += w;
            p[t][i / 2][4 * (i % 2) + e] = (_Float16)w;
          }
        sum[t] += add * (none ? 1.f : per_vs);
      }
      if (!some) {
#pragma unroll
        for (int t = 0; t < RT; ++t) p[t][0] = p[t][1] = f16x8{};
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
        const f16x8 y0 = widen<E4M3>(vals[n][0], vals[n][1]),
                    y1 = widen<E4M3>(vals[n][2], vals[n][3]);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          o[t][n] = product(y0, p[t][0], o[t][n]);
          o[t][n] = product(y1, p[t][1], o[t][n]);
        }
      }
    }

    // the four wavefronts' sums of the tile
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float all = row_sum(sum[t]);
      if (g == 0) {
        joint_max[wave][16 * t + col] = ref[t];
        joint_sum[wave][16 * t + col] = all;
      }
    }
    const bool whole = page_at == 0 && pages == s.pages;
    const int place = place_of(w, page_at > 0);
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += kPart) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int n = 0; n < kPart; ++n)
          *reinterpret_cast<f32x4*>(&joint[wave][16 * t + col][16 * n + 4 * g]) =
              o[t][n0 + n] * v0;
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
          finish(a, rows, r, d, top, all, y);
        } else {
          const int64_t row = (int64_t)place * kRows + r;
          put2(a.sums + row * D + d, y[0], y[1]);
          put2(a.sums + row * D + d + 2, y[2], y[3]);
          if (d == 0) put2(a.stats + 2 * row, top, all);
        }
      }
      __syncthreads();
    }
    if (whole) continue;

    // the runs that share the tile, in groups of kJoin, and then the groups
    const int64_t first_page = start + tile_at * (s.pages + kTileCost) + kTileCost;
    const int64_t w0 = first_page / run;
    const int n = (int)((first_page + s.pages - 1) / run - w0) + 1;
    const int group = (int)(w - w0) / kJoin, groups = (n + kJoin - 1) / kJoin;
    const int64_t leader = w0 + group * kJoin;
    const int members = n - group * kJoin < kJoin ? n - group * kJoin : kJoin;
    if (!arrive(a.counts + place_of(leader, group > 0), members, &arrived)) continue;
    float* lds = &joint[0][0][0];
    join(a, rows, w0, leader, 1, members, groups == 1, lds);
    if (groups == 1) continue;
    if (arrive(a.counts + 2 * kGroups + place_of(w0, false), groups, &arrived))
      join(a, rows, w0, w0, kJoin, groups, true, lds);
  }
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
  return (size_t)(2 * kGroups * (2 * 4 + room_rows(T, G) * (D + 2) * 4));
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
  a.counts = static_cast<int*>(u->workspace);
  a.stats = static_cast<float*>(u->workspace) + 4 * kGroups;
  a.sums = a.stats + 2 * kGroups * a.rows * 2;
  a.q_row = u->q_row;
  a.q_head = u->q_head;
  a.Hq = u->Hq;
  a.G = G;
  a.window = u->window;
  a.scale = u->scale * kLog2e;
  void* args[] = {&a};
  return launched(hipLaunchKernel(kernel_for(c.D, rt, c.type == LOWM_E4M3), dim3(kGroups),
                                  dim3(kThreads), args, 0, stream));
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
