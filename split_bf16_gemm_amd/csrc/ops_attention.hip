// ops_attention.hip -- attention over the paged 8-bit cache (include/lowm_cache.h)
// for gfx950.
//
//   x_t = scale q . k_t ;  out = sum_t e^(x_t - lse) v_t ;  lse = log sum_t e^x_t
//
// One pass over the pages with a running maximum and sum.  Bound by HBM for few rows, where
// a byte of the cache is read once for all rows of a key head (2 x 131001 tokens, 64 heads on
// 8 of 128, e4m3: 96 us, 5.6 TB/s, inputs changing from call to call); by the matrix unit and
// the vector unit, which hardly overlap, for many (1024 rows over 8192 tokens, the same heads:
// 296 to 303 us, 850 TFLOP/s and more of 1470 that a large product reaches; matrix
// instructions take 38 % of a SIMD's cycles, others 48 %); by round trips where the work is
// small (640 tokens: 9.5 us).
//
// Layout.  Rows of one key head (a token's query heads that share it, token after token)
// are taken in tiles, blocks of 16 to a wavefront.  S^T = K Q^T by
// v_mfma_f32_16x16x32_f16, 64 tokens of a page as the rows of four results and query rows
// as their columns, so that a lane holds 16 scores of one query row and all softmax state
// is one number a lane.  The tokens of the four score blocks are dealt so that a lane's
// scores are, in order, what the second product O^T = V^T P^T wants of that lane: scores
// go from one matrix instruction to the other without leaving their lane.  The cache's
// layout is what the two products read: a load of 16 bytes a lane takes 16 elements of a
// token's key, or 16 tokens of a value's element, whole lines at a time.
//
// Up to 32 rows (attend_kernel) each wavefront has pages of its own, straight into
// registers: the next page's keys load while this page's scores are worked on, its values
// while the keys multiply.  With more (attend_wide_kernel) all wavefronts of a workgroup take
// the same page, each for other rows, and it becomes fp16 once, in LDS.
//
// Bytes become fp16 exactly (an int8 by two byte permutations to 1024 + 128 + b and a
// packed subtraction).  A row of q is scaled by a power of two to just below 2^15.  Weights
// are taken times the scale of their page's values, which is part of the exponent, as
// 2^7 e^(x + log vs - ref), ref at most 8 (as a power of two) below the largest: fp16 keeps
// all 11 bits of what is within 2^-21 of that, and sums are seldom scaled anew.
//
// Work is cut on the device, whatever the lengths are (List, Walk).  Runs of the list have
// at most two tiles that others share, their first and their last, and leave what they have
// of them (a row's average of the values, its weights' sum and largest score) in two places
// of their own in the workspace; they are joined in the order of the pages, so that the
// bits do not depend on who does it.
//
// The join, for few rows: sums go to the workspace with device-scope stores, which pass the
// XCDs' own caches; a workgroup waits until its stores are acknowledged there and then
// adds to the tile's counter, and who finds all the others' additions reads with device-scope
// loads.  No cache is written back or invalidated, and nobody waits for another
// workgroup.  Counters are zero between calls: who joins clears them.  Sums of more rows
// are too many to pass the caches (64 KB of a part of 128 rows of 128): a second launch,
// join_kernel, reads them, and finds the tiles in notes that the first one leaves.
#include <type_traits>

#include "ops_cache.cuh"

namespace lowm {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kGroups = 512;                 // workgroups at most: two to a CU
constexpr int kWideRows = 128;               // rows of a tile of attend_wide_kernel
constexpr int kGroup = 16;                   // places joined at first
constexpr int kJoin = kGroups / kGroup;      // and at most, groups of them
constexpr int kJoinGroups = 1024;            // workgroups of join_kernel
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
  int* notes;        // for join_kernel: [8] how many runs there are, [kGroups][8] a Note each
  float* sums;       // [2 kGroups][rows of a tile][D]: averages of the values so far
  float* stats;      // [2 kGroups][rows of a tile][2]: maximum, sum
  int64_t q_row, q_head;
  int Hq, G, window, rows;   // rows: of a tile
  int most_pages;            // that a tile's rows may see together through the window
  int groups;                // workgroups
  uint32_t g_magic, g_shift; // for division by G
  float scale;               // times log2 e
};

// x / G for x of 31 bits: G's reciprocal rounded up, so that no quotient is too small,
// with enough bits that none is too large.
struct Divisor {
  uint32_t magic, shift;
  explicit Divisor(int d) {
    shift = 0;
    while ((1 << shift) < d) ++shift;
    magic = (uint32_t)(((1ull << (31 + shift)) + d - 1) / d);
  }
};
__device__ __forceinline__ int by_g(const AttendArgs& a, int x) {
  return a.G == 1 ? x : (int)(__umulhi((uint32_t)x, a.g_magic) >> (a.g_shift - 1));
}

// A sequence's share of the list.
struct Share {
  Rows rows;
  int tiles;          // of a key head
  int first, end;     // pages that a row may see
  int pages;          // that the rows of one tile may see, at most
  __device__ __forceinline__ Share() {}
  __device__ __forceinline__ Share(const AttendArgs& a, int b) {
    rows = rows_of(a.seq, b);
    tiles = (rows.n * a.G + a.rows - 1) / a.rows;   // a.rows: a power of two
    const int64_t most = (int64_t)a.seq.W * LOWM_PAGE;
    const int tokens = rows.len < most ? rows.len : (int)most;
    const int64_t from = (int64_t)rows.len - rows.n - a.window + 1;
    first = a.window > 0 && from > 0 ? (int)(from / LOWM_PAGE) : 0;
    end = (tokens + LOWM_PAGE - 1) / LOWM_PAGE;
    pages = end - first < a.most_pages ? end - first : a.most_pages;
    if (pages < 0) pages = 0;
  }
  // The share of the wavefront's lane `from`.
  __device__ __forceinline__ Share of_lane(int from) const {
    auto get = [&](int v) { return __builtin_amdgcn_readlane(v, from); };
    Share s;
    s.rows = Rows{get(rows.first), get(rows.n), get(rows.len)};
    s.tiles = get(tiles);
    s.first = get(first);
    s.end = get(end);
    s.pages = get(pages);
    return s;
  }
};

// The list: every sequence's tiles, head after head, and how they are cut into runs, one
// to a workgroup.  Where there are workgroups enough, each tile is cut by itself
// (`apart`): into parts of 2^per_log pages, a unit each, or none if it is small, and a
// run is a unit.  Else a tile is kTileCost units that stand for no page and then its
// pages, and all tiles are one list of equal runs, which may end inside a tile.  Every
// wavefront works that out for itself, 64 sequences at a time.  The host sees to it that
// 32 bits hold the units.
//
// A workgroup of attend_kernel takes four pages at a time, one of attend_wide_kernel (WIDE)
// one.  WIDE, parts of less than 8 pages pay while up to kFine workgroups leave sums (64 rows over 1024 tokens, 16 tiles: 21 us in parts of
// 2 pages, 29 in parts of 8; 512 rows over themselves, 128 tiles: 27 whole, 35 in parts of 4).
template <bool WIDE>
struct List {
  static constexpr int kTurn = WIDE ? 1 : kWaves;
  static constexpr int kLogs = WIDE ? 3 : 2, kLeast = WIDE ? 1 : 3;   // log2 of a part's pages
  // Pages of a tile that is not cut (10 to 12 pages 9.7 us, 11 in parts of 8; 19 pages 12.5 whole, 11
  // in parts).
  static constexpr int kSmall = WIDE ? 0 : 12;
  static constexpr int kFine = WIDE ? 128 : kGroups;   // runs at most for parts not the largest
  static constexpr int kLone = 24;   // units to a workgroup from which half as many take them
  int total, run, per_log, lane;
  bool apart;
  Share own;                         // of sequence `lane` (of the last 64)
  __device__ __forceinline__ int parts(int pages, int log) const {
    const int alone = kSmall > 1 << log ? kSmall : 1 << log;
    return pages <= alone ? 1 : (pages + (1 << log) - 1) >> log;
  }
  __device__ __forceinline__ explicit List(const AttendArgs& a) {
    lane = threadIdx.x & (kWave - 1);
    int units = 0, runs[kLogs] = {};   // for parts of 2^kLeast pages, of twice as many ..
    float rows = 0.f;
    for (int at = 0; at < a.seq.B; at += kWave) {
      own = Share(a, at + lane < a.seq.B ? at + lane : a.seq.B - 1);
      const int tiles = at + lane < a.seq.B ? a.cache.H * own.tiles : 0;
      auto all = [&](int v) { return __builtin_amdgcn_readlane(wave_scan(v), kWave - 1); };
      units += all(tiles * (own.pages + kTileCost));
#pragma unroll
      for (int i = 0; i < kLogs; ++i) runs[i] += all(tiles * parts(own.pages, kLeast + i));
      rows += wave_sum(at + lane < a.seq.B ? (float)own.rows.n : 0.f);
    }
    // row_starts that fall may count rows twice, and more units than 32 bits hold
    if (rows > 1.001f * (float)a.seq.T) units = runs[0] = 0;
    apart = false;
    per_log = 0;
    total = units;
#pragma unroll
    for (int i = kLogs - 1; i >= 0; --i) {
      if (runs[i] > a.groups || (i < kLogs - 1 && runs[i] > kFine)) continue;
      apart = true;
      per_log = kLeast + i;
      total = runs[i];
    }
    // long runs do better with one to a CU
    const bool half = !WIDE && a.groups == kGroups && units / kLone >= kGroups;
    const int groups = half ? kGroups / 2 : a.groups;
    run = apart ? 1 : ((units + groups - 1) / groups + kTurn - 1) & ~(kTurn - 1);
  }
  // Units from one tile to the next.
  __device__ __forceinline__ int span(const Share& s) const {
    return apart ? parts(s.pages, per_log) : s.pages + kTileCost;
  }
  // The sequence that unit u belongs to, the first of its units, and its share.
  __device__ __forceinline__ int find(const AttendArgs& a, int u, int* start, Share* s) const {
    int before = 0;
    for (int at = 0; at < a.seq.B; at += kWave) {
      Share mine = own;
      if (a.seq.B > kWave) mine = Share(a, at + lane < a.seq.B ? at + lane : a.seq.B - 1);
      const int units = at + lane < a.seq.B ? a.cache.H * mine.tiles * span(mine) : 0;
      const int sum = wave_scan(units);
      const int all = __builtin_amdgcn_readlane(sum, kWave - 1);
      if (u - before < all) {
        const int first = __builtin_ctzll(__ballot(sum > u - before));
        *start = before + __builtin_amdgcn_readlane(sum - units, first);
        *s = mine.of_lane(first);
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
__device__ __forceinline__ int place_of(int w, bool begun) { return 2 * w + !begun; }

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
    const int j = by_g(a, row0 + r);
    return (int64_t)(first + j) * a.Hq + head * a.G + (row0 + r - j * a.G);
  }
};
// 1 / the sum of a row's weights, to one unit in the last place; of one that saw nothing, 0.
__device__ __forceinline__ float over(float sum) {
  return sum == 0.f ? 0.f : __builtin_amdgcn_rcpf(sum);
}
// y: a row's outputs, the average of the values that it saw, which is no larger than they
// are (weights times values would be: 2^20 times and more).  So are those of a part.
__device__ __forceinline__ void finish(const AttendArgs& a, const TileRows& rows, int r, int d,
                                       float most, float sum, const f32x4& y) {
  const int64_t row = rows.at(a, r);
  *reinterpret_cast<ops_u32x2*>(a.out + row * a.cache.D + d) =
      ops_u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
  if (a.lse && d == 0) a.lse[row] = (most + __builtin_amdgcn_logf(sum) - kLift) * kLn2;
}

// Averages of the values of several parts, which saw weights of these sums in units of
// e^most each, given the largest of those units.  A part counts for its factor
// e^(its most - top) times its sum over all of them.  Where a factor nears the end of
// fp32's range (`far`) the values, which may be as large, take it as two halves.
struct Joined {
  float base;
  __device__ __forceinline__ explicit Joined(float top)
      : base(top == -__builtin_inff() ? 0.f : top) {}
  __device__ __forceinline__ float factor(float most) const {
    return __builtin_amdgcn_exp2f(most - base);
  }
  __device__ __forceinline__ float half(float most) const {
    return __builtin_amdgcn_exp2f(0.5f * (most - base));
  }
  __device__ __forceinline__ bool far(float most) const {
    return most - base < -100.f && most != -__builtin_inff();
  }
};
__device__ __forceinline__ void add_part(f32x4& y, const f32x4& z, float k) {
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] += z[e] * k;
}
__device__ __forceinline__ void add_part(f32x4& y, const f32x4& z, float half, float share) {
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] += z[e] * half * share;
}
// Over the 16 lanes of a row of them.
template <typename Op>
__device__ __forceinline__ float lanes_reduce(float v, Op op) {
  v = op(v, bits_float(lane_move<0x128, 0xf>(float_bits(v))));   // row_ror 8, 4, 2, 1
  v = op(v, bits_float(lane_move<0x124, 0xf>(float_bits(v))));
  v = op(v, bits_float(lane_move<0x122, 0xf>(float_bits(v))));
  return op(v, bits_float(lane_move<0x121, 0xf>(float_bits(v))));
}

// What a tile that others have a part of has so far, into its place: for a workgroup of
// this launch, or for the next one.
template <bool NOW>
__device__ __forceinline__ void leave(const AttendArgs& a, int place, int r, int d, float most,
                                      float sum, const f32x4& y) {
  const int64_t row = (int64_t)place * a.rows + r;
  if constexpr (!NOW) {
    *reinterpret_cast<f32x4*>(a.sums + row * a.cache.D + d) = y;
    if (d == 0) {
      a.stats[2 * row] = most;
      a.stats[2 * row + 1] = sum;
    }
    return;
  }
  put2(a.sums + row * a.cache.D + d, y[0], y[1]);
  put2(a.sums + row * a.cache.D + d + 2, y[2], y[3]);
  if (d == 0) put2(a.stats + 2 * row, most, sum);
}

// m places' sums joined: place i is of run w + i * step, of the tile that it begins
// (w + i * step == w0) or of the one it continues.  To the rows, or to place 0.
__device__ void join(const AttendArgs& a, const TileRows& rows, int w0, int w, int step,
                     int m, bool last, float* lds) {
  const int n = rows.last_row - rows.row0 + 1 < a.rows ? rows.last_row - rows.row0 + 1 : a.rows;
  const int D = a.cache.D;
  float *half = lds, *share = lds + kJoin * a.rows;    // of part i and row r: i * n + r
  float *tops = lds + 2 * kJoin * a.rows, *sums = tops + a.rows;
  auto at = [&](int i, int r) {
    const int run = w + i * step;
    return (int64_t)place_of(run, run > w0) * a.rows + r;
  };
  // 16 lanes to each of up to 16 rows
  static_assert(kThreads == 16 * kGroup && kGroup == 16 && kJoin <= 2 * kGroup, "all rows at once");
  const int row = threadIdx.x / kGroup, lane = threadIdx.x % kGroup;
  if (row < n) {
    Two part[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      part[k] = lane + kGroup * k < m ? get2(a.stats + 2 * at(lane + kGroup * k, row))
                                      : Two{-__builtin_inff(), 0.f};
    const float top =
        lanes_reduce(fmaxf(part[0].a, part[1].a), [](float x, float y) { return fmaxf(x, y); });
    const Joined join(top);
    const float h[2] = {join.half(part[0].a), join.half(part[1].a)};
    const float all = lanes_reduce(h[0] * h[0] * part[0].b + h[1] * h[1] * part[1].b,
                                   [](float x, float y) { return x + y; });
    const float inverse = over(all);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (lane + kGroup * k < m) {
        half[(lane + kGroup * k) * n + row] = h[k];
        share[(lane + kGroup * k) * n + row] = h[k] * (part[k].b * inverse);
      }
    if (lane == 0) {
      tops[row] = top;
      sums[row] = all;
    }
  }
  __syncthreads();
  for (int item = threadIdx.x; item < n * (D / 4); item += kThreads) {
    const int r = item / (D / 4), d = item % (D / 4) * 4;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < m; i0 += kGroup) {
      Two lo[kGroup], hi[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const float* p = a.sums + at(i0 + i < m ? i0 + i : i0, r) * D + d;
        lo[i] = get2(p);
        hi[i] = get2(p + 2);
      }
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const int k = (i0 + i) * n + r;
        if (i0 + i < m)
          add_part(y, f32x4{lo[i].a, lo[i].b, hi[i].a, hi[i].b}, half[k], share[k]);
      }
    }
    if (last) {
      finish(a, rows, r, d, tops[r], sums[r], y);
    } else {
      float* p = a.sums + at(0, r) * D + d;
      put2(p, y[0], y[1]);
      put2(p + 2, y[2], y[3]);
      if (d == 0) put2(a.stats + 2 * at(0, r), tops[r], sums[r]);
    }
  }
  __syncthreads();
}

// Keeps the loads above it above what follows.
__device__ __forceinline__ void pin_loads() { asm volatile("" ::: "memory"); }

// What join_kernel needs to know of the tile that a run begins and others end.
struct Note {
  int parts;         // runs that have a part of it; 0: there is no such tile
  TileRows rows;
};

// A workgroup's run of the list, part of a tile after part of a tile.
template <bool WIDE>
struct Walk {
  int total, run, per_log, w, u, end, start;   // its units are u .. end - 1; start: of b
  bool apart;
  int b;
  Share s;                         // of sequence b
  // the part of a tile at hand
  TileRows rows;
  int page_at, pages;              // of the tile's pages, this part's
  int w0, n;                       // the runs that share the tile: w0 .. w0 + n - 1
  int low, high;                   // positions of the tile's first and last row
  int first;                       // the tile's first page
  bool noted;                      // whether the run's note is written, or there is no run

  __device__ __forceinline__ explicit Walk(const AttendArgs& a) {
    const List<WIDE> list(a);
    total = list.total;
    run = list.run;
    per_log = list.per_log;
    apart = list.apart;
    // runs that have units, an eighth of them to each XCD: neighbours, which may share a
    // head's pages, share an L2
    const int runs = apart ? total : run > 0 ? (total + run - 1) / run : 0;
    const int each = (runs + 7) / 8;
    w = (blockIdx.x % 8) * each + blockIdx.x / 8;
    u = w * run;
    end = u + run < total ? u + run : total;
    if ((int)blockIdx.x / 8 >= each || w >= runs) u = end = 0;
    noted = u >= end;
    if (u >= end) return;
    b = list.find(a, u, &start, &s);
    if (b >= a.seq.B) u = end;
    if (apart) {
      // the only part there is
      const int span = list.span(s);
      const int tile_at = (int)((uint32_t)(u - start) / (uint32_t)span);
      const int part = u - start - tile_at * span;
      take(a, tile_at);
      w0 = w - part;
      page_at = part << per_log;
      pages = span == 1 || s.pages - page_at < 1 << per_log ? s.pages - page_at : 1 << per_log;
      n = span == 1 ? 1 : (seen() + (1 << per_log) - 1) >> per_log;
      if (part >= n) u = end;   // no row of the tile sees these pages
    }
  }
  // The tile's rows and first page.  Without a window later rows see more pages, so that
  // tiles are taken from both ends in turn, and equal runs have equal work in them (8192
  // rows over themselves, 64 heads on 8 of 128: 2045 us in order, 1243 so).
  __device__ __forceinline__ void take(const AttendArgs& a, int tile_at) {
    const int head = (int)((uint32_t)tile_at / (uint32_t)s.tiles), nth = tile_at - head * s.tiles;
    const int tile = !WIDE || a.window > 0 ? nth : nth % 2 ? s.tiles - 1 - nth / 2 : nth / 2;
    rows = TileRows{tile * a.rows, s.rows.n * a.G - 1, head, s.rows.first};
    const int last = rows.row0 + a.rows - 1 < rows.last_row ? rows.row0 + a.rows - 1 : rows.last_row;
    low = s.rows.position(by_g(a, rows.row0));
    high = s.rows.position(by_g(a, last));
    first = a.window > 0 && low >= a.window ? (low - a.window + 1) / LOWM_PAGE : 0;
    if (first < s.first) first = s.first;
  }
  __device__ __forceinline__ void zeros(const AttendArgs& a) const {
    const int quads = a.cache.D / 4;
    for (int i = threadIdx.x; i < a.rows * quads; i += blockDim.x)
      if (rows.row0 + i / quads <= rows.last_row)
        finish(a, rows, i / quads, i % quads * 4, -__builtin_inff(), 0.f, f32x4{0.f, 0.f, 0.f, 0.f});
  }
  // The next part that has pages; rows of sequences without any get their zeros here.
  __device__ __forceinline__ bool next(const AttendArgs& a) {
    while (u < end) {
      if (apart) {
        ++u;
        if (pages > 0) return true;
        zeros(a);
        return false;
      }
      const int span = s.pages + kTileCost;
      if ((uint32_t)(u - start) >= (uint32_t)(a.cache.H * s.tiles * span)) {
        start += a.cache.H * s.tiles * span;
        if (++b >= a.seq.B) return false;
        s = Share(a, b);
        continue;
      }
      const int tile_at = (int)((uint32_t)(u - start) / (uint32_t)span);
      const int from = u - start - tile_at * span;
      const int to = from + end - u < span ? from + end - u : span;
      const int first_page = u - from + kTileCost;   // unit of the tile's first page
      u += to - from;
      page_at = from > kTileCost ? from - kTileCost : 0;
      pages = to - kTileCost - page_at;
      take(a, tile_at);
      if (pages > 0) {
        if (page_at >= seen()) continue;
        w0 = first_page / run;
        n = (first_page + seen() - 1) / run - w0 + 1;
        return true;
      }
      // whoever has the first unit of a tile without pages writes its rows
      if (s.pages == 0 && from == 0) zeros(a);
    }
    return false;
  }
  __device__ __forceinline__ const int* table(const AttendArgs& a) const {
    return a.seq.table + b * a.seq.table_ld + first;
  }
  // The tile's pages that a row of it may see: how many are left from its first one on
  // (none, or less, where a window begins past the table).
  __device__ __forceinline__ int left() const {
    const int past = high < 0 ? 0 : high / LOWM_PAGE + 1;
    return (past < s.end ? past : s.end) - first;
  }
  // That, but one at least, which is somebody's part, and no more than the list has; for few
  // rows, all of which see about the same, what the list has.
  __device__ __forceinline__ int seen() const {
    if (!WIDE) return s.pages;
    return left() > 1 ? left() < s.pages ? left() : s.pages : 1;
  }
  // Where this part stops: no page past it is read.
  __device__ __forceinline__ int stop() const {
    return page_at + pages < left() ? page_at + pages : left();
  }
  // The first token that a row at a position sees.
  __device__ __forceinline__ int window_of(const AttendArgs& a, int position) const {
    return a.window > 0 && position >= a.window ? position - a.window + 1 : 0;
  }
  __device__ __forceinline__ bool whole() const { return n == 1; }
  __device__ __forceinline__ int place() const { return place_of(w, w > w0); }

  // Leaves the run's note: of the tile at hand if it begins here and ends elsewhere, in
  // any case before the workgroup ends.
  __device__ __forceinline__ void note(const AttendArgs& a, bool last_call) {
    if (blockIdx.x == 0 && last_call && threadIdx.x == 0)
      a.notes[0] = run > 0 ? (total + run - 1) / run : 0;
    if (noted) return;
    if (!last_call && (w > w0 || whole())) return;
    noted = true;
    if (threadIdx.x != 0) return;
    Note mine{0, rows};
    if (!last_call) mine.parts = n;
    *reinterpret_cast<Note*>(a.notes + 8 * (1 + w)) = mine;
  }
  // After the sums of a part that is not whole are in their place: the runs that share
  // the tile, in groups of kGroup, and then the groups.
  __device__ __forceinline__ void share(const AttendArgs& a, int* arrived, float* lds) const {
    const int group = (w - w0) / kGroup, groups = (n + kGroup - 1) / kGroup;
    const int leader = w0 + group * kGroup;
    const int members = n - group * kGroup < kGroup ? n - group * kGroup : kGroup;
    if (!arrive(a.counts + place_of(leader, group > 0), members, arrived)) return;
    join(a, rows, w0, leader, 1, members, groups == 1, lds);
    if (groups == 1) return;
    if (arrive(a.counts + 2 * kGroups + place_of(w0, false), groups, arrived))
      join(a, rows, w0, w0, kGroup, groups, true, lds);
  }
};

// Sixteen rows for each t: what they see, and their queries as the matrix operand.
template <int DP, bool FULL, int RT>
struct Queries {
  int see_lo[RT], see_hi[RT];
  float unit[RT];             // what a product of operands stands for, times log2 e
  f16x8 q[RT][2 * DP];

  // Rows row0 + 16 t + lane % 16 of the tile's sequence.
  template <typename W>
  __device__ __forceinline__ Queries(const AttendArgs& a, const W& walk, int row0) {
    const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, col = lane & 15;
    const int D = a.cache.D;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int r = row0 + 16 * t + col;
      const int in = r <= walk.rows.last_row ? r : walk.rows.last_row;
      const int j = by_g(a, in), h = walk.rows.head * a.G + (in - j * a.G);
      const int pos = walk.s.rows.position(j);
      see_hi[t] = r <= walk.rows.last_row ? pos : -1;
      see_lo[t] = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
      const uint16_t* x = a.q + (walk.s.rows.first + j) * a.q_row + h * a.q_head;
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
      const float size = bits_float((uint32_t)(up < 1 ? 1 : up > 254 ? 254 : up) << 23);
      const float lift = a.scale < 0.f ? -size : size;
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
  }
};

// The softmax's state.  Weights are e^(x + log vs - ref) 2^kLift with vs the page's scale
// of the values in units of 2^unit, the first page's exponent: they multiply the bytes as
// they are, and go into the sums o without another factor.  ref is the largest x + log vs
// so far, or up to kSlack less: the sums are scaled anew only when a page passes that.
//
// The sum of the weights has them without vs, in units of e^low, low being to x what ref is
// to x + log vs: a page's weights count for 2^(ref - low - log vs) times as much there.
// Scales may lie anywhere in fp32's range; where a page's is so small that its values are
// nothing beside those that a row has seen (kNothing), or 0, its weights are taken in units
// of e^low and its values as 0.
constexpr float kNothing = 90.f;
template <int NT, int RT>
struct Softmax {
  static constexpr int kNoUnit = 1000;
  float ref[RT], low[RT], sum[RT];
  int unit = kNoUnit;
  f32x4 o[RT][NT];
  __device__ __forceinline__ Softmax() {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      ref[t] = low[t] = -__builtin_inff();
      sum[t] = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) o[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
  // What makes the sums o[t] averages of the values, given the sum of a row's weights.
  __device__ __forceinline__ float to_average(int t, float all) {
    const float k = over(all), none = -__builtin_inff();
    const float up = ref[t] == none ? none : ref[t] - low[t] + (float)unit;
    if (__builtin_expect(!__any(up > 60.f || (up < -60.f && up > none)), 1))
      return k * __builtin_amdgcn_exp2f(up);
    // in steps, or the factor could be subnormal, or infinite
    const float half = __builtin_amdgcn_exp2f(0.5f * up);
#pragma unroll
    for (int n = 0; n < NT; ++n) o[t][n] = o[t][n] * k * half;
    return half;
  }
  // A page's products x to weights p, for its first `live` tokens from token0 on; masked:
  // whether a row may not see some of them.
  template <typename Q>
  __device__ __forceinline__ void weigh(const Q& q, f32x4 (&x)[RT][4], f16x8 (&p)[RT][2],
                                        bool masked, int live, int token0, float ks, float vs) {
    const int g = (threadIdx.x & (kWave - 1)) >> 4;
    const int exponent = __builtin_amdgcn_frexp_expf(vs);
    if (unit == kNoUnit && vs > 0.f) unit = exponent;
    const float log_vs =
        (float)(exponent - unit) + __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(vs));
    const float not_nan = vs - vs;   // 0, or NaN, which the rows that see the page get
    if (masked) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int token = token0 + 16 * g + 4 * i + e;
            const bool sees = live > 0 && token >= q.see_lo[t] && token <= q.see_hi[t];
            x[t][i][e] = sees ? x[t][i][e] : -__builtin_inff();
          }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      // never 0, which would make NaN of the masked ones
      float per = __builtin_fmaf(q.unit[t], ks, not_nan);
      per = per == 0.f ? 1.17549435e-38f : per;
      float here = x[t][0][0];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) here = fmaxf(here, x[t][i][e]);
      here = row_max(here);
      // a row that sees none of the page is not touched by its scales
      const bool none = here == -__builtin_inff();
      here *= per;
      per = none ? 1.f : per;
      const float value = here + log_vs;
      if (__any(value > ref[t] + kSlack || here > low[t] + kSlack)) {
        const float now = value > ref[t] + kSlack ? value : ref[t];
        const float keep = now == ref[t] ? 1.f : __builtin_amdgcn_exp2f(ref[t] - now);
        ref[t] = now;
#pragma unroll
        for (int n = 0; n < NT; ++n) o[t][n] *= keep;
        const float most = here > low[t] + kSlack ? here : low[t];
        sum[t] *= most == low[t] ? 1.f : __builtin_amdgcn_exp2f(low[t] - most);
        low[t] = most;
      }
      const float apart = ref[t] - low[t] - log_vs;
      // (also where ref is -infinity: a scale of 0)
      const bool nothing = !none && !(apart <= kNothing);
      const float lift = none ? 0.f : kLift + (nothing ? -low[t] : log_vs - ref[t]);
      float add = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][i][e], per, lift));
          add += w;
          p[t][i / 2][4 * (i % 2) + e] = (_Float16)w;
        }
      sum[t] += add * (none || nothing ? 1.f : __builtin_amdgcn_exp2f(apart));
      if (__builtin_expect(__any(nothing), 0))
        if (nothing) p[t][0] = p[t][1] = f16x8{};
    }
  }
};

// What lies behind a sequence may be any byte, a NaN of e4m3 among them: a piece of 16
// tokens, of which `left` are there.
__device__ __forceinline__ void clear_behind(ops_u32x4& v, int left) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = left - 4 * i;
    v[i] &= n >= 4 ? ~0u : n <= 0 ? 0u : (1u << 8 * n) - 1;
  }
}
// And so may what lies before every row's window: the first `gone` of a piece.
__device__ __forceinline__ void clear_before(ops_u32x4& v, int gone) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = gone - 4 * i;
    v[i] &= n >= 4 ? 0u : n <= 0 ? ~0u : ~((1u << 8 * n) - 1);
  }
}

// The token of row r of score block i is 16 (r / 4) + 4 i + r % 4: then lane group g has
// tokens 16 g .. 16 g + 15, in the order of the values' bytes.
__device__ __forceinline__ int key_piece(int g, int col, int m, int i) {
  return (4 * m + g) * LOWM_PAGE + 16 * (col >> 2) + 4 * i + (col & 3);
}

// One word for the whole wavefront by a vector load.  A scalar load would share the
// counter of LDS accesses, and those would wait for it (first_lane() at its use makes it
// one number again).
template <typename T>
__device__ __forceinline__ T load_apart(const T* p) {
  uint32_t none = 0;
  asm volatile("" : "+v"(none));
  return p[none];
}
__device__ __forceinline__ int first_lane(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float first_lane(float v) {
  return bits_float((uint32_t)__builtin_amdgcn_readfirstlane((int)float_bits(v)));
}

// A barrier for LDS alone: loads in flight stay so.
__device__ __forceinline__ void meet_in_lds() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Whether the registers of two workgroups fit a CU; and whether they do with the queries
// in LDS.
constexpr bool queries_in_lds(int DP, int RT) { return DP == 2 && RT == 2; }
constexpr bool two_to_a_cu(int DP, int RT) {
  return DP * RT <= 2 || (DP == 3 && RT == 1) || (DP == 2 && RT == 2);
}

// DP blocks of 64 elements of a head, all of them there (FULL) or not, RT blocks of 16
// rows to a tile.  Each wavefront takes every fourth page of the part.
template <int DP, bool FULL, int RT, bool E4M3>
__global__ __launch_bounds__(kThreads, two_to_a_cu(DP, RT) ? 2 : 1)
void attend_kernel(AttendArgs a) {
  constexpr int NT = 4 * DP;                // blocks of 16 elements
  constexpr int kRows = 16 * RT;
  constexpr int kPart = DP == 1 ? 4 : DP == 3 ? 6 : 8;   // joined through LDS at a time
  static_assert(NT % kPart == 0, "whole parts");
  constexpr int kPitch = 16 * kPart + 4;    // lanes' rows in distinct banks
  __shared__ __align__(16) float joint[kWaves][kRows][kPitch];
  __shared__ float joint_max[kWaves][kRows], joint_sum[kWaves][kRows];
  __shared__ int arrived;
  constexpr bool kInLds = queries_in_lds(DP, RT);
  __shared__ f16x8 queries[kInLds ? RT : 1][kInLds ? 2 * DP : 1][kWave];
  constexpr bool kNow = RT == 1;            // few rows are joined here, others by join_kernel
  static_assert(!kNow || sizeof(joint) >= 2 * (kJoin + 1) * kRows * sizeof(float), "room to join");

  const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const lowm_kv_cache& c = a.cache;
  const int D = FULL ? 64 * DP : c.D, nt = FULL ? NT : D / 16;

  Walk<false> walk(a);
  while (walk.next(a)) {
    const int stop = walk.stop(), head = walk.rows.head;
    const int high_lo = walk.window_of(a, walk.high), low_lo = walk.window_of(a, walk.low);
    const int* table = walk.table(a);

    ops_u32x4 keys[4][DP], vals[NT];
    float k_scale = 0.f, v_scale = 0.f;
    int page = -1, next_page = -1;
    auto load_keys = [&](int next) {
      page = first_lane(next_page);
      page = page >= 0 && page < c.P ? page : -1;
      const int64_t at = (int64_t)(page < 0 ? 0 : page) * c.H + head;
      next_page = load_apart(table + next);
      const ops_u32x4* p =
          reinterpret_cast<const ops_u32x4*>(static_cast<const uint8_t*>(c.k) + at * (LOWM_PAGE * D));
      k_scale = load_apart(c.k_scale + at);
      v_scale = load_apart(c.v_scale + at);
#pragma unroll
      for (int m = 0; m < DP; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          keys[i][m] = ops_u32x4{0u, 0u, 0u, 0u};
          if (FULL || m < DP - 1 || (4 * m + g) * 16 < D) keys[i][m] = p[key_piece(g, col, m, i)];
        }
      pin_loads();
    };
    // Values are read once: with the streaming hint (the keys' lines are shared by two
    // loads each, and would be fetched twice: 2 x 131001 tokens 91 us, 95 with the hint
    // on both, 102 on neither).
    auto load_vals = [&]() {
      const ops_u32x4* p = reinterpret_cast<const ops_u32x4*>(
          static_cast<const uint8_t*>(c.v) +
          ((int64_t)(page < 0 ? 0 : page) * c.H + head) * (LOWM_PAGE * D));
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (!FULL && n >= NT - 4) vals[n] = ops_u32x4{0u, 0u, 0u, 0u};
        if (FULL || n < NT - 4 || n < nt)
          vals[n] = __builtin_nontemporal_load(p + g * D + 16 * n + col);
      }
      pin_loads();
    };
    // the number of a page is read a turn before its keys
    int at = walk.page_at + wave;
    if (at < stop) {
      next_page = load_apart(table + at);
      load_keys(at + kWaves < stop ? at + kWaves : at);
    }
    const Queries<DP, FULL, RT> rows(a, walk, walk.rows.row0);
    if constexpr (kInLds) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int m = 0; m < 2 * DP; ++m)
          if (m % kWaves == wave) queries[t][m][lane] = rows.q[t][m];
      meet_in_lds();
    }
    Softmax<NT, RT> sm;

    for (; at < stop; at += kWaves) {
      const int token0 = (walk.first + at) * LOWM_PAGE;
      // tokens of the page that are there at all
      int live = walk.s.rows.len - token0;
      live = page < 0 ? 0 : live < LOWM_PAGE ? live : LOWM_PAGE;
      const float ks = live > 0 ? first_lane(k_scale) : 0.f, vs = live > 0 ? first_lane(v_scale) : 0.f;
      load_vals();

      f32x4 x[RT][4];
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
      // four operands are widened while the matrix unit takes the four before
      f16x8 ops[2][4];
      auto widen_keys = [&](int step) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          ops[step % 2][i] = widen<E4M3>(keys[i][step / 2][step % 2 * 2],
                                         keys[i][step / 2][step % 2 * 2 + 1]);
      };
      auto widen_vals = [&](int step) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          ops[step % 2][i] = widen<E4M3>(vals[2 * step + i / 2][i % 2 * 2],
                                         vals[2 * step + i / 2][i % 2 * 2 + 1]);
      };
      widen_keys(0);
#pragma unroll
      for (int step = 0; step < 2 * DP; ++step) {
        __builtin_amdgcn_sched_barrier(0);
        if (step + 1 < 2 * DP) widen_keys(step + 1);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int t = 0; t < RT; ++t)
            x[t][i] = product(ops[step % 2][i], kInLds ? queries[t][step][lane] : rows.q[t][step],
                              x[t][i]);
      }
      if (at + kWaves < stop) {
        load_keys(at + 2 * kWaves < stop ? at + 2 * kWaves : at);
      }
      f16x8 p[RT][2];
      sm.weigh(rows, x, p,
               live < LOWM_PAGE || token0 + LOWM_PAGE - 1 > walk.low || token0 < high_lo, live,
               token0, ks, vs);
      if (E4M3 && live < LOWM_PAGE) {
#pragma unroll
        for (int n = 0; n < NT; ++n) clear_behind(vals[n], live - 16 * g);
      }
      if (E4M3 && token0 < low_lo) {
#pragma unroll
        for (int n = 0; n < NT; ++n) clear_before(vals[n], low_lo - token0 - 16 * g);
      }
      // (blocks past D are zeros)
      widen_vals(0);
#pragma unroll
      for (int step = 0; step < NT / 2; ++step) {
        __builtin_amdgcn_sched_barrier(0);
        if (step + 1 < NT / 2) widen_vals(step + 1);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int t = 0; t < RT; ++t)
              sm.o[t][2 * step + n] =
                  product(ops[step % 2][2 * n + i], p[t][i], sm.o[t][2 * step + n]);
      }
    }

    // the four wavefronts' parts of the tile
    float to_average[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float all = row_sum(sm.sum[t]);
      to_average[t] = sm.to_average(t, all);
      if (g == 0) {
        joint_max[wave][16 * t + col] = sm.low[t];
        joint_sum[wave][16 * t + col] = all;
      }
    }
    const bool whole = walk.whole();
    const int place = walk.place();
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += kPart) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int n = 0; n < kPart; ++n)
          *reinterpret_cast<f32x4*>(&joint[wave][16 * t + col][16 * n + 4 * g]) =
              sm.o[t][n0 + n] * to_average[t];
      __syncthreads();
      for (int i = threadIdx.x; i < kRows * 4 * kPart; i += kThreads) {
        const int r = i / (4 * kPart), d4 = i % (4 * kPart), d = 16 * n0 + 4 * d4;
        if (walk.rows.row0 + r > walk.rows.last_row || (!FULL && d >= D)) continue;
        float top = joint_max[0][r];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, joint_max[w][r]);
        const Joined join(top);
        float k[kWaves], all = 0.f;
        bool far = false;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float most = joint_max[w][r];
          k[w] = join.factor(most) * joint_sum[w][r];
          all += k[w];
          far |= join.far(most);
        }
        const float inverse = over(all);
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const f32x4 z = *reinterpret_cast<const f32x4*>(&joint[w][r][4 * d4]);
          if (__builtin_expect(!far, 1)) {
            add_part(y, z, k[w] * inverse);
          } else {
            const float h = join.half(joint_max[w][r]);
            add_part(y, z, h, h * (joint_sum[w][r] * inverse));
          }
        }
        if (whole)
          finish(a, walk.rows, r, d, top, all, y);
        else
          leave<kNow>(a, place, r, d, top, all, y);
      }
      __syncthreads();
    }
    if constexpr (kNow) {
      if (!whole) walk.share(a, &arrived, &joint[0][0][0]);
    } else {
      walk.note(a, false);
    }
  }
  if constexpr (!kNow) walk.note(a, true);
}

// The same for many rows: 16 RT to each of WAVES wavefronts, all on the same page.  A
// page becomes fp16 once, in LDS, a share by each wavefront, in the order in which the
// matrix instructions take it (a lane's 16 bytes after another: no bank is hit twice);
// the next two pages are on their way in registers meanwhile, and go into the other half
// of the LDS in turn.  One barrier a page, which waits for LDS alone.
template <int DP, bool FULL, int RT, int WAVES, bool E4M3>
__global__ __launch_bounds__(kWave* WAVES, DP <= 2 || WAVES == 8 ? 2 : 1)
void attend_wide_kernel(AttendArgs a) {
  constexpr int NT = 4 * DP;
  constexpr int kShare = 8 * DP / WAVES;   // pieces of a page to a wavefront
  static_assert(8 * DP % WAVES == 0, "equal shares");
  // keys of score block i and 64 elements m: 4 m + i; values of 16 elements n: 4 DP + n
  __shared__ f16x8 stage[2][8 * DP][2][kWave];

  const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const lowm_kv_cache& c = a.cache;
  const int D = FULL ? 64 * DP : c.D, nt = FULL ? NT : D / 16;

  Walk<true> walk(a);
  while (walk.next(a)) {
    const int stop = walk.stop(), head = walk.rows.head;
    const int* table = walk.table(a);
    // the wavefront's own rows
    const int row0 = walk.rows.row0 + 16 * RT * wave;
    const int last = row0 + 16 * RT - 1 < walk.rows.last_row ? row0 + 16 * RT - 1
                                                             : walk.rows.last_row;
    const bool mine = row0 <= walk.rows.last_row;
    const int low = mine ? walk.s.rows.position(by_g(a, row0)) : -1,
              high = mine ? walk.s.rows.position(by_g(a, last)) : -1;
    const int high_lo = walk.window_of(a, high), low_lo = walk.window_of(a, low);
    const int tile_lo = walk.window_of(a, walk.low);

    // Two pages are on their way, one for each half of the LDS: pieces wave + WAVES k.
    ops_u32x4 raw[2][kShare];
    struct Page {
      float ks, vs;
      int live, gone;   // tokens that are there, and those before every row's window
    } on_way[2] = {}, here = {};
    int next_page = 0;
    auto load = [&](auto half_c, int at) {
      constexpr int half = decltype(half_c)::value;
      const int page = first_lane(next_page);
      const bool some = page >= 0 && page < c.P;
      const int64_t from = (int64_t)(some ? page : 0) * c.H + head;
      // the next page's number first: waiting for it is not waiting for what follows
      next_page = load_apart(table + (at + 1 < stop ? at + 1 : at));
      const ops_u32x4* pk = reinterpret_cast<const ops_u32x4*>(static_cast<const uint8_t*>(c.k) +
                                                               from * (LOWM_PAGE * D));
      const ops_u32x4* pv = reinterpret_cast<const ops_u32x4*>(static_cast<const uint8_t*>(c.v) +
                                                               from * (LOWM_PAGE * D));
      const int live = walk.s.rows.len - (walk.first + at) * LOWM_PAGE;
      on_way[half].live = !some ? 0 : live < LOWM_PAGE ? live : LOWM_PAGE;
      on_way[half].gone = tile_lo - (walk.first + at) * LOWM_PAGE;
      on_way[half].ks = load_apart(c.k_scale + from);
      on_way[half].vs = load_apart(c.v_scale + from);
#pragma unroll
      for (int k = 0; k < kShare; ++k) {
        const int piece = wave + WAVES * k;
        const bool key = piece < 4 * DP;
        const int m = piece / 4, n = piece - 4 * DP;
        const bool there = FULL || (key ? (4 * m + g) * 16 < D : n < nt);
        const ops_u32x4* x =
            key ? pk + key_piece(g, col, m, piece % 4) : pv + g * D + 16 * n + col;
        raw[half][k] = ops_u32x4{0u, 0u, 0u, 0u};
        if (there) raw[half][k] = *x;
      }
      pin_loads();
    };
    auto put = [&](auto half_c) {
      constexpr int half = decltype(half_c)::value;
#pragma unroll
      for (int k = 0; k < kShare; ++k) {
        const int piece = wave + WAVES * k;
        ops_u32x4 v = raw[half][k];
        if (E4M3 && piece >= 4 * DP && on_way[half].live < LOWM_PAGE)
          clear_behind(v, on_way[half].live - 16 * g);
        if (E4M3 && piece >= 4 * DP && on_way[half].gone > 0)
          clear_before(v, on_way[half].gone - 16 * g);
        stage[half][piece][0][lane] = widen<E4M3>(v[0], v[1]);
        stage[half][piece][1][lane] = widen<E4M3>(v[2], v[3]);
      }
      here.live = on_way[half].live;
      here.ks = first_lane(on_way[half].ks);
      here.vs = first_lane(on_way[half].vs);
    };
    constexpr std::integral_constant<int, 0> even{};
    constexpr std::integral_constant<int, 1> odd{};
    int at = walk.page_at;
    if (at < stop) {
      next_page = load_apart(table + at);
      load(even, at);
      if (at + 1 < stop) load(odd, at + 1);
    }
    const Queries<DP, FULL, RT> rows(a, walk, row0);
    Softmax<NT, RT> sm;
    if (at < stop) {
      put(even);
      if (at + 2 < stop) load(even, at + 2);
      meet_in_lds();
    }
    auto turn = [&](auto half_c, auto other, int at) {
      constexpr int half = decltype(half_c)::value;
      const int token0 = (walk.first + at) * LOWM_PAGE;
      // wavefronts whose rows do not see the page only pass it on
      if (mine && token0 <= high && token0 + LOWM_PAGE > low_lo) {
        f32x4 x[RT][4];
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        // four operands are read while eight instructions take the four before
        f16x8 ops[2][4];
        auto read_keys = [&](int step) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            ops[step % 2][i] = stage[half][step / 2 * 4 + i][step % 2][lane];
        };
        auto read_vals = [&](int step) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            ops[step % 2][i] = stage[half][4 * DP + 2 * step + i / 2][i % 2][lane];
        };
        read_keys(0);
#pragma unroll
        for (int step = 0; step < 2 * DP; ++step) {
          if (step + 1 < 2 * DP)
            read_keys(step + 1);
          else
            read_vals(0);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < RT; ++t)
              x[t][i] = product(ops[step % 2][i], rows.q[t][step], x[t][i]);
          __builtin_amdgcn_sched_barrier(0);
        }
        const float ks = here.live > 0 ? here.ks : 0.f, vs = here.live > 0 ? here.vs : 0.f;
        f16x8 p[RT][2];
        sm.weigh(rows, x, p,
                 here.live < LOWM_PAGE || token0 + LOWM_PAGE - 1 > low || token0 < high_lo,
                 here.live, token0, ks, vs);
        // (blocks past D are zeros)
#pragma unroll
        for (int step = 0; step < NT / 2; ++step) {
          if (step + 1 < NT / 2) read_vals(step + 1);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int t = 0; t < RT; ++t)
                sm.o[t][2 * step + n] =
                    product(ops[step % 2][2 * n + i], p[t][i], sm.o[t][2 * step + n]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (at + 1 < stop) {
        put(other);
        if (at + 3 < stop) load(other, at + 3);
      }
      meet_in_lds();
    };
    for (; at < stop; at += 2) {
      turn(even, odd, at);
      if (at + 1 < stop) turn(odd, even, at + 1);
    }

    const bool whole = walk.whole();
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float all = row_sum(sm.sum[t]), to_average = sm.to_average(t, all);
      const int r = 16 * RT * wave + 16 * t + col;
      if (walk.rows.row0 + r > walk.rows.last_row) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (!FULL && n >= NT - 4 && n >= nt) continue;
        const int d = 16 * n + 4 * g;
        if (whole)
          finish(a, walk.rows, r, d, sm.low[t], all, sm.o[t][n] * to_average);
        else
          leave<false>(a, walk.place(), r, d, sm.low[t], all, sm.o[t][n] * to_average);
      }
    }
    walk.note(a, false);
  }
  walk.note(a, true);
}

__host__ __device__ inline int join_lanes(int D) { return D <= 64 ? 16 : D <= 128 ? 32 : 64; }
// Joins the tiles that several runs have a part of, in the order of join().  Each
// wavefront finds out which runs begin one, and takes 64 / lanes rows at a time.
__global__ __launch_bounds__(kThreads) void join_kernel(AttendArgs a) {
  constexpr int kSets = kGroups / kWave;
  const int lane = threadIdx.x & (kWave - 1);
  const int runs = a.notes[0];
  uint64_t begun[kSets];
  int tiles = 0;
#pragma unroll
  for (int k = 0; k < kSets; ++k) {
    const int w = kWave * k + lane;
    const int parts = reinterpret_cast<const Note*>(a.notes + 8 * (1 + w))->parts;
    begun[k] = __ballot(w < runs && parts > 0);
    tiles += __builtin_popcountll(begun[k]);
  }
  const int D = a.cache.D, lanes = join_lanes(D);
  const int per = a.rows * lanes / kWave;   // turns to a tile
  const int d = lane % lanes * 4;
  for (int item = blockIdx.x * kWaves + (int)threadIdx.x / kWave; item < tiles * per;
       item += kWaves * gridDim.x) {
    int skip = item / per;
    int w0 = 0;
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      const int here = __builtin_popcountll(begun[k]);
      if (skip >= 0 && skip < here) {
        uint64_t left = begun[k];
        for (int i = 0; i < skip; ++i) left &= left - 1;
        w0 = kWave * k + __builtin_ctzll(left);
      }
      skip -= here;
    }
    const Note note = *reinterpret_cast<const Note*>(a.notes + 8 * (1 + w0));
    const int n = note.parts, r = item % per * (kWave / lanes) + lane / lanes;
    if (note.rows.row0 + r > note.rows.last_row || d >= D) continue;
    float most = -__builtin_inff(), sum = 0.f;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
    auto fold = [&](auto ahead_c) {
      constexpr int ahead = decltype(ahead_c)::value;
      for (int i0 = 0; i0 < n; i0 += ahead) {
        float top[ahead], part[ahead];
        f32x4 z[ahead];
#pragma unroll
        for (int i = 0; i < ahead; ++i) {
          const int in = i0 + i < n ? i0 + i : n - 1;
          const int64_t row = (int64_t)place_of(w0 + in, in > 0) * a.rows + r;
          top[i] = i0 + i < n ? a.stats[2 * row] : -__builtin_inff();
          part[i] = a.stats[2 * row + 1];
          z[i] = *reinterpret_cast<const f32x4*>(a.sums + row * D + d);
        }
        float now = most;
#pragma unroll
        for (int i = 0; i < ahead; ++i) now = fmaxf(now, top[i]);
        const Joined join(now);
        // (the sum so far is 0 where the loop begins)
        bool far = join.far(most);
        const float before = join.factor(most) * sum;
        float all = before;
#pragma unroll
        for (int i = 0; i < ahead; ++i) {
          far |= join.far(top[i]);
          part[i] *= join.factor(top[i]);   // (of parts past the last: 0)
          all += part[i];
        }
        const float inverse = over(all);
        if (__builtin_expect(!far, 1)) {
          y *= before * inverse;
#pragma unroll
          for (int i = 0; i < ahead; ++i) add_part(y, z[i], part[i] * inverse);
        } else {
          const float h = join.half(most);
          f32x4 x = {0.f, 0.f, 0.f, 0.f};
          add_part(x, y, h, h * (sum * inverse));
          for (int i = i0; i < n && i < i0 + ahead; ++i) {
            // (read again, rather than kept in registers for this)
            const int64_t row = (int64_t)place_of(w0 + i, i > 0) * a.rows + r;
            const float h = join.half(a.stats[2 * row]);
            add_part(x, *reinterpret_cast<const f32x4*>(a.sums + row * D + d), h,
                     h * (a.stats[2 * row + 1] * inverse));
          }
          y = x;
        }
        most = now;
        sum = all;
      }
    };
    // (most tiles of a prompt have two parts or three)
    if (n <= 4)
      fold(std::integral_constant<int, 4>{});
    else
      fold(std::integral_constant<int, 16>{});
    finish(a, note.rows, r, d, most, sum, y);
  }
}

// A sequence's rows of a key head, on average, choose the kernel: up to 16, 32 or 64, or
// more.
enum Kind { kFew = 16, kSome = 32, kMore = 64, kMany = kWideRows };
Kind kind_for(int64_t T, int G, int B) {
  const int64_t rows = T * G;
  return rows <= (int64_t)B * kFew    ? kFew
         : rows <= (int64_t)B * kSome ? kSome
         : rows <= (int64_t)B * kMore ? kMore
                                      : kMany;
}
// Wavefronts of a workgroup.  Past 128 elements a page's fp16 take more than half of the
// LDS, and 16 rows to each of eight wavefronts keep two on each SIMD where 32 to each of
// four would keep one.
int waves_for(Kind k, int D) { return k == kMany && D > 128 ? 8 : 4; }
template <int DP, bool FULL, bool E4M3>
const void* kernel_for(Kind k) {
  switch (k) {
    case kFew: return (const void*)&attend_kernel<DP, FULL, 1, E4M3>;
    case kSome: return (const void*)&attend_kernel<DP, FULL, 2, E4M3>;
    case kMore: return (const void*)&attend_wide_kernel<DP, FULL, 1, 4, E4M3>;
    default:
      return (const void*)&attend_wide_kernel<DP, FULL, DP <= 2 ? 2 : 1, DP <= 2 ? 4 : 8, E4M3>;
  }
}
template <int DP>
const void* kernel_for(Kind k, bool full, bool e4m3) {
  return full ? (e4m3 ? kernel_for<DP, true, true>(k) : kernel_for<DP, true, false>(k))
              : (e4m3 ? kernel_for<DP, false, true>(k) : kernel_for<DP, false, false>(k));
}
const void* kernel_for(int D, Kind k, bool e4m3) {
  switch ((D + 63) / 64) {
    case 1: return kernel_for<1>(k, D == 64, e4m3);
    case 2: return kernel_for<2>(k, D == 128, e4m3);
    case 3: return kernel_for<3>(k, D == 192, e4m3);
    default: return kernel_for<4>(k, D == 256, e4m3);
  }
}

// Rows of the largest tile that T rows may take.
int64_t room_rows(int T, int G) {
  const int64_t rows = (int64_t)T * G;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : kWideRows;
}
size_t workspace_bytes(int T, int G, int D) {
  return (size_t)(4 * (4 * kGroups + 8 * (1 + kGroups) + 2 * kGroups * room_rows(T, G) * (D + 2)));
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
  const Kind kind = kind_for(s.T, G, s.B);
  // units of the list (see List), at most
  if ((rows / c.H / kind + s.B + 1) * c.H * (s.W + kTileCost + 64) > INT32_MAX / 2)
    return LOWM_ERR_UNSUPPORTED;
  AttendArgs a{};
  a.cache = c;
  a.seq = s;
  a.q = static_cast<const uint16_t*>(u->q);
  a.out = static_cast<uint16_t*>(u->out);
  a.lse = u->lse;
  a.rows = kind;
  // One workgroup to a CU streams best (2 x 131001 tokens 89 us; 92 with two), and is all
  // that fits where a page takes more than half of the LDS; two where tiles are many and
  // short (64 sequences of 300 tokens, 512 tiles: 11.3 us; 21.7 with one), or rows many.
  const int64_t tiles = (int64_t)c.H * (s.B < s.T ? s.B : s.T);
  a.groups = (kind >= kMore ? c.D <= 128 : tiles > 128) ? kGroups : kGroups / 2;
  // positions p to p + (rows + G - 2) / G of a tile's rows, and the window before p
  const int64_t most = ((int64_t)u->window + (a.rows + G - 2) / G + LOWM_PAGE - 2) / LOWM_PAGE + 1;
  a.most_pages = u->window > 0 && most < INT32_MAX ? (int)most : INT32_MAX;
  const Divisor g(G);
  a.g_magic = g.magic;
  a.g_shift = g.shift;
  a.counts = static_cast<int*>(u->workspace);
  a.notes = a.counts + 4 * kGroups;
  a.stats = reinterpret_cast<float*>(a.notes + 8 * (1 + kGroups));
  a.sums = a.stats + 2 * kGroups * a.rows * 2;
  a.q_row = u->q_row;
  a.q_head = u->q_head;
  a.Hq = u->Hq;
  a.G = G;
  a.window = u->window;
  a.scale = u->scale * kLog2e;
  void* args[] = {&a};
  rc = launched(hipLaunchKernel(kernel_for(c.D, kind, c.type == LOWM_E4M3),
                                dim3((unsigned)a.groups), dim3(kWave * waves_for(kind, c.D)), args,
                                0, stream));
  if (rc != LOWM_OK || kind == kFew) return rc;
  const int64_t joins = (rows / c.H / kind + (s.B < s.T ? s.B : s.T)) * c.H *
                        (kind * join_lanes(c.D) / kWave) / kWaves;
  return launched(hipLaunchKernel((const void*)&join_kernel,
                                  dim3((unsigned)(joins < kJoinGroups ? joins : kJoinGroups)),
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
