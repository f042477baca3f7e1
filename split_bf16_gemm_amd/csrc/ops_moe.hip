// ops_moe.hip -- a mixture-of-experts layer for a few tokens
// (include/lowm_ops.h) for gfx950.
//
// With few tokens the layer is a stream of weights: every expert that some
// token chose is read once, 6 D I bytes, against a few rows of activations.
// Three kernels:
//   route  l = x router^T by tiles of 16 experts and 16 tokens (and, with few of
//          those, stretches of D); the last workgroup of a block of tokens picks
//          their experts, and the last block's sorts the (token, expert) pairs by
//          expert into segments of up to 16 rows, the matrix instructions' height
//          (32 or 64 where experts get many);
//   up     one workgroup per segment and 16 columns of h: 16 gate and 16 up rows;
//   down   one workgroup per 16 output columns walks the segments as one long
//          inner dimension, cut evenly over its wavefronts (and, for a narrow D,
//          over several workgroups), and adds gate * result to the pair's token.
// A segment's weights are all that its workgroups read from HBM; a further
// segment of the same expert finds them in the caches.  No atomic adds, no
// order that changes: equal inputs give equal bits.
//
// Bound by HBM.  Measured on MI355X, us a call, beside the time of a plain read of
// the chosen experts: T 1, D 4096, I 1024, E 64, top_k 4 27 (15); T 64, E 128,
// top_k 8 483 (473).  What is left at T 1 is 6 us of routing, which one kernel has to
// finish before the next can know what to read, and 5 us in up and down, which take
// 12.4 and 7.8 us for 67 and 34 MB and load 16 rows of activations a step where one
// is there.
//
// Roundings: h = silu(gate) up is rounded to bf16, the matrix instructions' type,
// from fp32 sums; that is the one rounding besides the result's own, and makes the
// error against 64 bits 1.4 times that of a layer that keeps h in fp32.
#include "ops_stream.cuh"

namespace lowm {

constexpr int kMaxT = LOWM_MOE_MAX_T;
constexpr int kMaxE = LOWM_MOE_MAX_E;
constexpr int kMaxK = LOWM_MOE_MAX_K;
constexpr int kCols = 16;                 // columns of h, and of the output, per workgroup
constexpr int kMaxDownSplits = 8;
constexpr int kRouteWaves = 16;
constexpr int kRouteThreads = kRouteWaves * kWave;
constexpr int kMaxSize = 65536;

struct Segment {
  int expert, first, rows, unused;        // pairs first .. first + rows - 1
};
struct Pair {
  int token;
  float gate;
};

// The workspace: arrival counters (one 256-byte line each: count, fault word)
// and exchange slots, zero between calls, then what one call's kernels hand on.
// The first part has one place and size for all calls, so that a call never
// finds another size's leavings where its zeros have to be.
constexpr size_t up256(size_t b) { return (b + 255) / 256 * 256; }
constexpr int kFirstTileLine = 1 + kMaxT / 16;   // after the router's
constexpr size_t kCounterBytes = 256 * (kFirstTileLine + (size_t)kMaxSize / kCols);
constexpr size_t kPairSlots = 2 * (size_t)kMaxT * kMaxK;
constexpr int kMaxRouteSplits = 4;
constexpr size_t kRouteSlots = kMaxRouteSplits * (size_t)kMaxT * kMaxE;
constexpr size_t kDownSlots = 512 * (size_t)kMaxT * kCols;       // most tiles * splits, times the tile
constexpr size_t kRouteAt = kCounterBytes;
constexpr size_t kDownAt = kRouteAt + 4 * kRouteSlots;
constexpr size_t kPairsAt = kDownAt + 4 * kDownSlots;
constexpr size_t kListsAt = kPairsAt + 4 * kPairSlots;

struct Layout {
  int seg_rows, route_splits, down_splits, max_segments;
  size_t pairs, h, bytes;
};

// Rows of a segment, by the rows that an expert gets on average.  A further segment
// reads the expert's weights again, from the caches at best, while a larger one
// keeps the LDS of more rows.  us at 16, 32 and 64 rows: T 48, D 4096, I 1024, E 20,
// top_k 5 (12 rows on average) 101, 108, 134; T 64, D 4096, I 1024, E 8, top_k 2 (16)
// 60.8, 55.2, 64.8; T 47, D 4000, I 488, E 20, top_k 8 (19) 97, 82, 92; T 64,
// D 4096, I 1024, E 16, top_k 8 (32) 153, 131, 119.
static int seg_rows_of(int T, int E, int K) {
  return T * K >= 28 * E ? 64 : T * K >= 14 * E ? 32 : 16;
}

static Layout layout_of(int T, int D, int I, int E, int K) {
  Layout l{};
  // Router: a tile's weights come from far and slowly to one CU, so few tiles
  // are cut along D: up to 64 workgroups, a step at least for each wavefront.
  const int router_tiles = ((E + 15) / 16) * ((T + 15) / 16), steps = (2 * D + 127) / 128;
  l.route_splits = 1;
  while (l.route_splits < kMaxRouteSplits && router_tiles * l.route_splits * 2 <= 64 &&
         steps >= 2 * l.route_splits * kRouteWaves)
    l.route_splits *= 2;
  // Down: enough workgroups for 256 CUs.  Nearly enough will do: a split costs its
  // join (T 27, D 3632, 227 tiles: 91 us whole, 96 us in two; T 52, D 3008, 188
  // tiles: 162 us whole, 154 us in two).
  const int tiles = (D + kCols - 1) / kCols;
  l.down_splits = 1;
  while (l.down_splits < kMaxDownSplits && tiles * l.down_splits < 200) l.down_splits *= 2;
  const int pairs = T * K, active = pairs < E ? pairs : E;
  l.seg_rows = seg_rows_of(T, E, K);
  // sum of ceil(n / rows) over the active experts, each with 1 <= n <= T pairs
  auto segments = [&](int rows) {
    return T <= rows ? active : (pairs + (rows - 1) * active) / rows;
  };
  l.max_segments = segments(l.seg_rows);
  // (room for segments of 16, so that fewer tokens never need more bytes)
  l.pairs = kListsAt + up256(16 + sizeof(Segment) * (size_t)segments(16));
  l.h = l.pairs + up256(sizeof(Pair) * (size_t)pairs);
  l.bytes = l.h + up256((size_t)2 * pairs * I);
  return l;
}

struct MoeArgs {
  const uint8_t* x;
  const uint8_t* router;
  const float* bias;
  const uint8_t* w13;
  const uint8_t* w2;
  __bf16* out;
  int* ids;
  float* gates;
  uint32_t* counters;                     // lines: the router's, its blocks', the down tiles'
  uint32_t* route_slots;                  // [route_splits][T][E]
  uint32_t* pair_slots;                   // [T][top_k][2]: id + 1, gate
  uint32_t* down_slots;                   // [tiles][down_splits][T][kCols]
  int* lists;                             // number of segments, 3 unused, then the segments
  Pair* pairs;
  uint8_t* h;                             // [T * top_k, I] bf16, in the pairs' order
  int T, D, I, E, top_k, flags;
  float routed_scale;
  int seg_rows, route_splits, down_splits;
};

// ---------------------------------------------------------------------------
// route
// ---------------------------------------------------------------------------
// 64 tokens, D 4096, 128 experts 11.8 us; one token, 64 experts 6.2 (whole D in one
// workgroup to a tile instead of four: 10).
// The wavefronts cut D between them and load their operands straight into
// registers in the matrix layout, kRouteBatch steps at a time: there is little
// to read and one round trip to wait for, so a ring would only add trips.
[[maybe_unused]] constexpr int kRouteBatch = 4;

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

constexpr int kBlock = 16;                // tokens of a router tile

struct RouteLds {
  float logits[kBlock * kMaxE];           // of one block of tokens
  int chosen[kMaxT][kMaxK];
  float gates[kMaxT][kMaxK];
  uint32_t mask[kMaxE][2];
  uint32_t starts[kMaxE];
  uint32_t ends[kMaxE / kWave];
  int last;
};

// One token's experts in order and their gates, by one wavefront: lane l holds
// experts l, l + 64, ... (NJ of them), and in the end the l-th choice.
template <int NJ>
__device__ __forceinline__ void pick_experts(const MoeArgs& a, const float* logits, int& my_id,
                                             float& my_gate) {
  const int lane = threadIdx.x & (kWave - 1);
  const bool sig = a.flags & LOWM_MOE_SIGMOID, renorm = !(a.flags & LOWM_MOE_NO_RENORM);
  float l[NJ];
  uint32_t o[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = lane + kWave * j;
    l[j] = logits[e < a.E ? e : 0];
    o[j] = e < a.E ? order(l[j]) : 0u;
  }
  // Softmax over all experts only where it shows: in a choice by score + bias, or
  // in gates that are not divided by the chosen ones' sum.
  const bool whole = !sig && (!renorm || a.bias);
  float most = 0.f, total = 1.f;
  if (whole) {
    uint32_t top = o[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) top = o[j] > top ? o[j] : top;
    most = value_of(wave_umax(top));
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) s += lane + kWave * j < a.E ? expf(l[j] - most) : 0.f;
    total = wave_sum(s);
  }
  if (a.bias) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = lane + kWave * j;
      const float score = sig ? sigmoid(l[j]) : expf(l[j] - most) / total;
      o[j] = e < a.E ? order(score + a.bias[e < a.E ? e : 0]) : 0u;
    }
  }
  my_id = 0;
  for (int i = 0; i < a.top_k; ++i) {
    uint32_t top = o[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) top = o[j] > top ? o[j] : top;
    top = wave_umax(top);
    // the lowest id among equals: the first j, then the first lane
    uint64_t at = __ballot(o[0] == top);
    int first = 0;
#pragma unroll
    for (int j = 1; j < NJ; ++j)
      if (!at) {
        at = __ballot(o[j] == top);
        first = kWave * j;
      }
    const int e = first + __builtin_ctzll(at);
#pragma unroll
    for (int j = 0; j < NJ; ++j) o[j] = lane + kWave * j == e ? 0u : o[j];
    my_id = lane == i ? e : my_id;
  }
  const bool mine = lane < a.top_k;
  const float v = logits[my_id];
  float score;
  if (renorm) {
    // Scores as multiples of one that no chosen expert's is far above, so that their
    // ratios stay where the scores themselves are below fp32's smallest number: e^l
    // by the chosen ones' largest l, which is the first choice's without a bias, and
    // a sigmoid too where that l is negative.
    const uint32_t bits = __builtin_bit_cast(uint32_t, v);
    const float top = a.bias ? value_of(wave_umax(mine ? order(v) : 0u))
                             : __builtin_bit_cast(
                                   float, (uint32_t)__builtin_amdgcn_readfirstlane((int)bits));
    score = sig && top >= 0.f ? sigmoid(v) : expf(v - top) / (sig ? 1.0f + expf(v) : 1.0f);
  } else {
    score = sig ? sigmoid(v) : expf(v - most) / total;
  }
  score = mine ? score : 0.f;
  const float sum = wave_sum(score);
  my_gate = (renorm ? score / sum : score) * a.routed_scale;
}

// The pairs in order of expert, then token, and their segments.  Each expert's
// tokens are the bits of a mask, so a pair's place is a count of bits below.
__device__ __forceinline__ void sort_pairs(const MoeArgs& a, RouteLds& r) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int pairs = a.T * a.top_k;
  for (int p = tid; p < pairs; p += kRouteThreads) {
    const int t = p / a.top_k;
    atomicOr(&r.mask[r.chosen[t][p - t * a.top_k]][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  // thread e: expert e's pairs (low half) and segments (high half), summed over
  // the experts before it
  const bool one = tid < kMaxE;
  const int rows = one ? __popc(r.mask[tid][0]) + __popc(r.mask[tid][1]) : 0;
  const int most = a.seg_rows;            // a power of 2
  const uint32_t own = (uint32_t)rows | (uint32_t)((rows + most - 1) >> __builtin_ctz(most)) << 16;
  uint32_t before = own;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const uint32_t v = __shfl_up(before, off);
    if (lane >= off) before += v;
  }
  if (one && lane == kWave - 1) r.ends[wave] = before;
  __syncthreads();
  if (one) {
    uint32_t total = 0;
#pragma unroll
    for (int w = 0; w < kMaxE / kWave; ++w) {
      if (w < wave) before += r.ends[w];
      total += r.ends[w];
    }
    before -= own;
    r.starts[tid] = before & 0xffffu;
    Segment* segments = reinterpret_cast<Segment*>(a.lists + 4);
    for (int s = 0; s * most < rows; ++s)
      segments[(before >> 16) + s] =
          Segment{tid, (int)(before & 0xffffu) + s * most,
                  rows - s * most < most ? rows - s * most : most, 0};
    if (tid == 0) a.lists[0] = (int)(total >> 16);
  }
  __syncthreads();
  for (int p = tid; p < pairs; p += kRouteThreads) {
    const int t = p / a.top_k, e = r.chosen[t][p - t * a.top_k];
    const uint32_t lo = r.mask[e][0], hi = r.mask[e][1];
    const int below = t < 32 ? __popc(lo & ((1u << t) - 1u))
                             : __popc(lo) + __popc(hi & ((1u << (t - 32)) - 1u));
    a.pairs[r.starts[e] + below] = Pair{t, r.gates[t][p - t * a.top_k]};
  }
}

__global__ __launch_bounds__(kRouteThreads) void moe_route_kernel(MoeArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ RouteLds r;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int g = lane >> 4, l16 = lane & 15;
  const int tiles = (a.E + 15) / 16;
  const int split = blockIdx.x % a.route_splits, place = blockIdx.x / a.route_splits;
  const int e0 = place % tiles * 16, block = place / tiles, t0 = block * kBlock;

  const int steps = (2 * a.D + 127) / 128, parts = a.route_splits * kRouteWaves;
  const int part = split * kRouteWaves + wave;
  const int s0 = steps * part / parts, s1 = steps * (part + 1) / parts;
  const uint8_t* w =
      a.router + (size_t)(e0 + l16 < a.E ? e0 + l16 : a.E - 1) * a.D * 2;
  const uint8_t* x = a.x + (size_t)(t0 + l16 < a.T ? t0 + l16 : a.T - 1) * a.D * 2;
  f32x4 acc[1] = {{0.f, 0.f, 0.f, 0.f}};
  auto batch = [&](auto n_c, int s) {
    constexpr int N = 2 * decltype(n_c)::value;
    u32x4 wv[N], xv[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int k = (2 * s + j) * 64 + 16 * g;           // the lane's 16 bytes
      // (past the end something is read and dropped: loads under a branch wait
      // for one another)
      wv[j] = *reinterpret_cast<const u32x4*>(w + (k < 2 * a.D ? k : 0));
      xv[j] = *reinterpret_cast<const u32x4*>(x + (k < 2 * a.D ? k : 0));
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const bool in = (2 * s + j) * 64 + 16 * g < 2 * a.D;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wv[j][i] = in ? wv[j][i] : 0u;
        xv[j][i] = in ? xv[j][i] : 0u;
      }
      acc[0] = mfma(xv[j], wv[j], acc[0]);
    }
  };
  int s = s0;
  for (; s + kRouteBatch <= s1; s += kRouteBatch)
    batch(std::integral_constant<int, kRouteBatch>{}, s);
  for (; s < s1; ++s) batch(std::integral_constant<int, 1>{}, s);
  stream_settle(acc);
  f32x4* sums = reinterpret_cast<f32x4*>(r.logits);
  static_assert(sizeof(r.logits) >= kRouteThreads * sizeof(f32x4), "the sums fit");
  sums[wave * kWave + lane] = acc[0];
  if (threadIdx.x < 2 * kMaxE) (&r.mask[0][0])[threadIdx.x] = 0u;
  __syncthreads();
  // Wavefront i adds row 4 g + i of lane group g, in 64 bits so that experts next
  // to the border are told apart as well as fp32 can.
  if (wave < 4) {
    double v = 0.0;
#pragma unroll
    for (int p = 0; p < kRouteWaves; ++p)
      v += (double)reinterpret_cast<const float*>(sums + p * kWave + lane)[wave];
    const int t = t0 + 4 * g + wave, e = e0 + l16;
    if (t < a.T && e < a.E)
      store_slot(a.route_slots + ((size_t)split * a.T + t) * a.E + e, enc_partial((float)v));
  }
  uint32_t* line = a.counters + (size_t)(1 + block) * kCtrStride;
  if (!arrive_last(line, tiles * a.route_splits, &r.last)) return;

  // The last workgroup of a block of tokens has all its logits before it.
  const int rows = a.T - t0 < kBlock ? a.T - t0 : kBlock, cells = rows * a.E;
  constexpr int kAtOnce = 4;              // cells a thread asks for in one trip
  auto slot = [&](int c, int s) {
    return a.route_slots + ((size_t)s * a.T + t0) * a.E + c;
  };
  for (int c0 = threadIdx.x; c0 < cells; c0 += kAtOnce * kRouteThreads) {
    uint32_t v[kAtOnce][kMaxRouteSplits];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
      for (int s = 0; s < kMaxRouteSplits; ++s) {
        const int c = c0 + j * kRouteThreads;
        v[j][s] = load_slot(slot(c < cells ? c : c0, s < a.route_splits ? s : 0));
      }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int c = c0 + j * kRouteThreads;
      if (c >= cells) break;
      double sum = 0.0;
#pragma unroll
      for (int s = 0; s < kMaxRouteSplits; ++s)
        if (s < a.route_splits) sum += (double)dec_partial(take_slot(slot(c, s), v[j][s], line));
      r.logits[c] = (float)sum;
    }
  }
  __syncthreads();
  const int blocks = (a.T + kBlock - 1) / kBlock;
  if (wave < rows) {
    int id;
    float gate;
    const float* l = r.logits + wave * a.E;
    if (a.E <= kWave) pick_experts<1>(a, l, id, gate);
    else if (a.E <= 2 * kWave) pick_experts<2>(a, l, id, gate);
    else pick_experts<kMaxE / kWave>(a, l, id, gate);
    const int t = t0 + wave;
    if (lane < a.top_k) {
      const int p = t * a.top_k + lane;
      if (a.ids) a.ids[p] = id;
      if (a.gates) a.gates[p] = gate;
      if (blocks == 1) {
        r.chosen[t][lane] = id;
        r.gates[t][lane] = gate;
      } else {
        store_slot(a.pair_slots + 2 * p, (uint32_t)id + 1u);
        store_slot(a.pair_slots + 2 * p + 1, enc_partial(gate));
      }
    }
  }
  if (blocks > 1) {
    // The last block's workgroup has every token's choice before it.
    if (!arrive_last(a.counters, blocks, &r.last)) return;
    for (int p = threadIdx.x; p < a.T * a.top_k; p += kRouteThreads) {
      const int t = p / a.top_k, i = p - t * a.top_k;
      const uint32_t w0 = load_slot(a.pair_slots + 2 * p), w1 = load_slot(a.pair_slots + 2 * p + 1);
      // (held in range whatever a workspace that was not zero makes of it: an
      // expert taken twice then only leaves a pair that no segment counts)
      const int id = (int)take_slot(a.pair_slots + 2 * p, w0, a.counters) - 1;
      r.chosen[t][i] = id < 0 ? 0 : id < a.E ? id : a.E - 1;
      r.gates[t][i] = dec_partial(take_slot(a.pair_slots + 2 * p + 1, w1, a.counters));
    }
  }
  __syncthreads();
  sort_pairs(a, r);
#endif
}

// ---------------------------------------------------------------------------
// up
// ---------------------------------------------------------------------------
// 16 gate rows and the 16 up rows of the same columns, so that h is there where both
// sums are; the four wavefronts a stretch of D each (a workgroup's 32 weight rows
// are few, and this way it waits for a quarter of them).  64 tokens, D 4096,
// I 1024, 126 active experts, 2.1 GB: 306 us (6.9 TB/s).
//
// AP pieces of 8 rows to a segment.
template <int AP, int R>
struct UpShape {
  using S = StreamShape<2, AP, R>;
  static constexpr int kRings = kWaves * S::kRing * 16;
};

template <int AP, int R, bool WHOLE>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(MoeArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  using SH = UpShape<AP, R>;
  constexpr int G = SH::S::G, MB = SH::S::MB;
  __shared__ u32x4 lds[SH::kRings / 16];
  const int tiles = (a.I + kCols - 1) / kCols;
  const int seg = blockIdx.x / tiles, i0 = blockIdx.x % tiles * kCols;
  if (seg >= a.lists[0]) return;
  const Segment s = reinterpret_cast<const Segment*>(a.lists + 4)[seg];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;

  const int steps = (2 * a.D + 127) / 128;
  const int s0 = steps * wave / kWaves, P = steps * (wave + 1) / kWaves - s0;
  const int k0 = s0 * 128 + stream_piece(lane) * 16;
  f32x4 acc[2 * MB];                      // gate's blocks of 16 rows, then up's
#pragma unroll
  for (int q = 0; q < 2 * MB; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (P > 0) {
    const uint8_t* w = a.w13 + (size_t)s.expert * 4 * a.I * a.D + k0;
    const uint8_t* src[G];
#pragma unroll
    for (int t = 0; t < G; ++t) {
      // 16 gate rows, the 16 up rows of the same columns, then the segment's tokens
      int r = 8 * (t < 4 ? t & 1 : t - 4) + stream_row(lane);
      if (t < 4) {
        r = i0 + r < a.I ? i0 + r : a.I - 1;
        src[t] = w + (size_t)(t < 2 ? r : a.I + r) * a.D * 2;
      } else {
        r = r < s.rows ? r : s.rows - 1;
        src[t] = a.x + (size_t)a.pairs[s.first + r].token * a.D * 2 + k0;
      }
    }
    u32x4* ring = lds + wave * SH::S::kRing;
    if constexpr (WHOLE)
      stream_tile<2, AP, R>(ring, src, 2 * a.D - k0, P, acc);
    else
      stream_tile_shifted<2, AP, R>(ring, src, k0, 2 * a.D - k0, P, acc);
  }
  stream_settle(acc);
  f32x4* sums = reinterpret_cast<f32x4*>(lds);
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2 * MB; ++q) sums[(wave * 2 * MB + q) * kWave + lane] = acc[q];
  __syncthreads();
  // wavefront i takes rows 4 g + i of lane group g
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    float gate = 0.f, up = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      gate += reinterpret_cast<const float*>(sums + (w * 2 * MB + b) * kWave + lane)[wave];
      up += reinterpret_cast<const float*>(sums + (w * 2 * MB + MB + b) * kWave + lane)[wave];
    }
    const int row = 16 * b + 4 * (lane >> 4) + wave, i = i0 + (lane & 15);
    if (row < s.rows && i < a.I)
      reinterpret_cast<__bf16*>(a.h)[(size_t)(s.first + row) * a.I + i] =
          static_cast<__bf16>(gate * sigmoid(gate) * up);
  }
#endif
}

// ---------------------------------------------------------------------------
// down
// ---------------------------------------------------------------------------
// One workgroup has all of an output tile's inner dimension, or a fixed part of it,
// so the experts' results are added where they are, gate by gate, with no exchange
// but the splits'.  64 tokens, D 4096, I 1024, 126 active experts, 1.06 GB: 152 us
// (7.0 TB/s).
template <int AP, int R>
struct DownShape {
  using S = StreamShape<1, AP, R>;
  static constexpr int kRings = kWaves * S::kRing * 16;
};

// The segments' steps as one sequence: step q is step q mod n of segment q / n.
// WHOLE: rows are whole lines, which are read once and need no place in the
// caches.  Otherwise two requests share a line, and the second finds it in the L2
// if it was read without the streaming hint (T 52, D 3032, I 776, E 64: 85 us
// against 95; with whole lines through the ring as in stream_tile_shifted, whose
// extra line every run pays, 125).
template <int AP, int R, bool WHOLE>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  using S = typename DownShape<AP, R>::S;
  constexpr int G = S::G, kPP = S::kPP, MB = S::MB;
  extern __shared__ u32x4 dyn[];
  __shared__ u32x4 rings[DownShape<AP, R>::kRings / 16];
  __shared__ int last;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int g = lane >> 4, l16 = lane & 15;
  const int split = blockIdx.x % a.down_splits, tile = blockIdx.x / a.down_splits;
  const int n0 = tile * kCols;
  const int segments = a.lists[0], n_pairs = a.T * a.top_k;

  // dynamic LDS: the segments, the pairs, each wavefront's [T][kCols] sums
  Segment* segs = reinterpret_cast<Segment*>(dyn);
  Pair* pairs = reinterpret_cast<Pair*>(segs + segments);
  float* sums = reinterpret_cast<float*>(pairs + (n_pairs + 1) / 2 * 2);
  for (int i = threadIdx.x; i < segments; i += kThreads)
    segs[i] = reinterpret_cast<const Segment*>(a.lists + 4)[i];
  for (int i = threadIdx.x; i < n_pairs; i += kThreads) pairs[i] = a.pairs[i];
  const int cells = a.T * kCols;
  for (int i = threadIdx.x; i < kWaves * cells; i += kThreads) sums[i] = 0.f;
  __syncthreads();

  const int per = (2 * a.I + 127) / 128;               // steps of a segment
  const int steps = segments * per;
  const int parts = a.down_splits * kWaves, part = split * kWaves + wave;
  const int q0 = (int)((int64_t)steps * part / parts);
  const int q1 = (int)((int64_t)steps * (part + 1) / parts);
  const int P = q1 - q0;
  u32x4* ring = rings + wave * S::kRing;
  float* mine = sums + wave * cells;

  const int piece = stream_piece(lane) * 16, qr = stream_row(lane);
  int rpos[2];
#pragma unroll
  for (int c = 0; c < 2; ++c)
    rpos[c] = (l16 >> 3) * kPP + (l16 & 7) * 8 + ((4 * c + g + ((l16 & 7) >> 1)) & 7);
  // this tile's rows of w2 within an expert
  size_t wrow[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int n = n0 + 8 * t + qr;
    wrow[t] = (size_t)(n < a.D ? n : a.D - 1) * a.I * 2 + piece;
  }

  auto segment_at = [&](int s) {
    u32x4 v[1] = {lds_read_opaque(reinterpret_cast<const u32x4*>(segs + s))};
    lds_wait(v);
    Segment out;
    const uint32_t e = v[0][0], f = v[0][1], r = v[0][2];
    out.expert = __builtin_amdgcn_readfirstlane((int)e);
    out.first = __builtin_amdgcn_readfirstlane((int)f);
    out.rows = __builtin_amdgcn_readfirstlane((int)r);
    out.unused = 0;
    return out;
  };
  // the next step to load
  int ls = per > 0 ? q0 / per : 0, lk = q0 - ls * per;
  const uint8_t* src[G];
  auto point = [&]() {
    const Segment s = segment_at(ls);
    const uint8_t* w = a.w2 + (size_t)s.expert * a.D * a.I * 2;
#pragma unroll
    for (int t = 0; t < 2; ++t) src[t] = w + wrow[t];
#pragma unroll
    for (int t = 0; t < AP; ++t) {
      int r = 8 * t + qr;
      r = r < s.rows ? r : s.rows - 1;
      src[2 + t] = a.h + (size_t)(s.first + r) * a.I * 2 + piece;
    }
  };
  int loaded = 0;
  auto issue = [&](u32x4* slot) {
    const int at = lk * 128;
    const bool whole = 2 * a.I - at >= 128;
    static_for<G>([&](auto t_c) {
      constexpr int t = decltype(t_c)::value;
      const uint8_t* from = src[t] + at;
      if (!whole)
        from = 2 * a.I - piece - at >= 16 ? from : reinterpret_cast<const uint8_t*>(&kZeroPiece);
      __builtin_amdgcn_global_load_lds(from, (__attribute__((address_space(3))) void*)(slot + t * kPP),
                                       16, 0, WHOLE && t < 2 ? kStreamAux : 0);
    });
    pin_issue();
    ++loaded;
    if (++lk == per) {
      lk = 0;
      ++ls;
      if (loaded < P) point();
    }
  };
  f32x4 acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  int us = ls, uk = lk, used = 0;                        // the next step to use
  auto flush = [&]() {
    stream_settle(acc);
    const Segment s = segment_at(us);
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      if (b > 0 && 16 * b >= s.rows) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 16 * b + 4 * g + i;
        const ops_u32x2 p = lds_read8_opaque(pairs + s.first + (row < s.rows ? row : 0));
        const uint32_t token = p[0], gate_bits = p[1];
        const float gate = __builtin_bit_cast(float, gate_bits);
        const float v = acc[b][i];
        if (row < s.rows) lds_add_opaque(mine + token * kCols + l16, gate * v);
      }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  auto multiply = [&](const u32x4* slot) {
    u32x4 v[2 * (1 + MB)];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int t = 0; t < 1 + MB; ++t)
        v[c * (1 + MB) + t] = lds_read_opaque(slot + 2 * t * kPP + rpos[c]);
    lds_wait(v);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int b = 0; b < MB; ++b)
        acc[b] = mfma(v[c * (1 + MB) + 1 + b], v[c * (1 + MB)], acc[b]);
    ++used;
    if (++uk == per || used == P) {
      flush();
      uk = 0;
      ++us;
    }
  };

  u32x4* const end = ring + S::kRing;
  u32x4 *fill = ring, *use = ring;
  auto next = [&](u32x4* s) { return s + S::kSlot == end ? ring : s + S::kSlot; };
  if (P > 0) point();
  for (int p = 0; p < R - 1 && p < P; ++p) {
    issue(fill);
    fill = next(fill);
  }
  int p = 0;
  for (; p + R - 1 < P; ++p) {
    wait_vmcnt<(R - 2) * G>();
    issue(fill);
    fill = next(fill);
    multiply(use);
    use = next(use);
  }
  static_for<R - 1>([&](auto i_c) {
    constexpr int younger = R - 2 - decltype(i_c)::value;
    if (P - p == younger + 1) {
      wait_vmcnt<younger * G>();
      multiply(use);
      use = next(use);
      ++p;
    }
  });
  wait_lgkmcnt0();
  __syncthreads();

  // The wavefronts' sums in order; then, with several workgroups to a tile, the
  // workgroups' in order, by the last to arrive.
  constexpr int kMine = kMaxT * kCols / kThreads;
  float v[kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int c = threadIdx.x + j * kThreads;
    v[j] = 0.f;
    if (c < cells) {
      v[j] = sums[c];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v[j] += sums[w * cells + c];
    }
  }
  if (a.down_splits > 1) {
    uint32_t* slots = a.down_slots + (size_t)tile * a.down_splits * cells;
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int c = threadIdx.x + j * kThreads;
      if (c < cells) store_slot(slots + (size_t)split * cells + c, enc_partial(v[j]));
    }
    uint32_t* line = a.counters + (size_t)(kFirstTileLine + tile) * kCtrStride;
    if (!arrive_last(line, a.down_splits, &last)) return;
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int c = threadIdx.x + j * kThreads;
      if (c < cells) {
        uint32_t w[kMaxDownSplits];
#pragma unroll
        for (int r = 0; r < kMaxDownSplits; ++r)
          if (r < a.down_splits) w[r] = load_slot(slots + (size_t)r * cells + c);
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < kMaxDownSplits; ++r)
          if (r < a.down_splits) {
            const float part_sum =
                dec_partial(take_slot(slots + (size_t)r * cells + c, w[r], line));
            sum = r == 0 ? part_sum : sum + part_sum;
          }
        v[j] = sum;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int c = threadIdx.x + j * kThreads;
    const int n = n0 + c % kCols;
    if (c < cells && n < a.D) a.out[(size_t)(c / kCols) * a.D + n] = static_cast<__bf16>(v[j]);
  }
#endif
}

namespace {

bool moe_sizes(int T, int D, int I, int E, int K) {
  return T >= 1 && T <= kMaxT && D >= 8 && D % 8 == 0 && D <= kMaxSize && I >= 8 && I % 8 == 0 &&
         I <= kMaxSize && E >= 1 && E <= kMaxE && K >= 1 && K <= kMaxK && K <= E;
}

int moe(const lowm_moe_args* u, hipStream_t stream) {
  if (!u || u->T < 0 || u->D < 1 || u->I < 1 || u->E < 1 || u->top_k < 1 || u->top_k > u->E)
    return LOWM_ERR_INVALID_ARG;
  if (u->flags & ~(LOWM_MOE_SIGMOID | LOWM_MOE_NO_RENORM)) return LOWM_ERR_INVALID_ARG;
  if (u->T == 0) return LOWM_OK;
  if (!u->x || !u->router || !u->w13 || !u->w2 || !u->out) return LOWM_ERR_INVALID_ARG;
  const int T = u->T, D = u->D, I = u->I, E = u->E, K = u->top_k;
  if (!moe_sizes(T, D, I, E, K)) return LOWM_ERR_UNSUPPORTED;
  const Layout l = layout_of(T, D, I, E, K);
  if (!u->workspace || u->workspace_bytes < l.bytes) return LOWM_ERR_WORKSPACE;
  if (((uintptr_t)u->x | (uintptr_t)u->router | (uintptr_t)u->w13 | (uintptr_t)u->w2 |
       (uintptr_t)u->out) & 15 ||
      ((uintptr_t)u->bias | (uintptr_t)u->ids | (uintptr_t)u->gates) & 3 ||
      (uintptr_t)u->workspace & 255)
    return LOWM_ERR_UNSUPPORTED;
  const Span in[] = {span_of(u->x, T, D, D, 2), span_of(u->router, E, D, D, 2),
                     span_of(u->bias, 1, E, E, 4), span_of(u->w13, E, 2ll * I * D, 2ll * I * D, 2),
                     span_of(u->w2, E, (int64_t)I * D, (int64_t)I * D, 2)};
  const Span out[] = {span_of(u->out, T, D, D, 2), span_of(u->ids, T, K, K, 4),
                      span_of(u->gates, T, K, K, 4),
                      span_of(u->workspace, 1, (int64_t)l.bytes, (int64_t)l.bytes, 1)};
  for (int i = 0; i < 4; ++i) {
    for (const Span& s : in)
      if (meet(out[i], s)) return LOWM_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return LOWM_ERR_INVALID_ARG;
  }
  char* ws = static_cast<char*>(u->workspace);
  MoeArgs a{};
  a.x = static_cast<const uint8_t*>(u->x);
  a.router = static_cast<const uint8_t*>(u->router);
  a.bias = u->bias;
  a.w13 = static_cast<const uint8_t*>(u->w13);
  a.w2 = static_cast<const uint8_t*>(u->w2);
  a.out = static_cast<__bf16*>(u->out);
  a.ids = u->ids;
  a.gates = u->gates;
  a.counters = reinterpret_cast<uint32_t*>(ws);
  a.route_slots = reinterpret_cast<uint32_t*>(ws + kRouteAt);
  a.down_slots = reinterpret_cast<uint32_t*>(ws + kDownAt);
  a.pair_slots = reinterpret_cast<uint32_t*>(ws + kPairsAt);
  a.lists = reinterpret_cast<int*>(ws + kListsAt);
  a.pairs = reinterpret_cast<Pair*>(ws + l.pairs);
  a.h = reinterpret_cast<uint8_t*>(ws + l.h);
  a.T = T;
  a.D = D;
  a.I = I;
  a.E = E;
  a.top_k = K;
  a.flags = u->flags;
  a.routed_scale = u->routed_scale;
  a.seg_rows = l.seg_rows;
  a.route_splits = l.route_splits;
  a.down_splits = l.down_splits;
  void* args[] = {&a};
  auto go = [&](const void* fn, size_t grid, size_t lds, int threads = kThreads) {
    return launched(hipLaunchKernel(fn, dim3((unsigned)grid), dim3(threads), args, lds, stream));
  };
  // Rows of weights that are not whole lines of memory.
  using Kernel = void (*)(MoeArgs);
  auto in_lines = [](int cols, const void* w, Kernel shifted, Kernel whole) {
    const bool any = ((uintptr_t)w | (uintptr_t)cols * 2) & 127;
    return reinterpret_cast<const void*>(any ? shifted : whole);
  };
  int rc = go(reinterpret_cast<const void*>(&moe_route_kernel),
              (size_t)((E + 15) / 16) * ((T + 15) / 16) * l.route_splits, 0, kRouteThreads);
  // Up to one workgroup to a CU the ring is as deep as a CU's LDS (T 2, D 4096, I 512,
  // two experts each: 22.8 us a call with 6 slots, 24.1 with 3); more share a CU.
  const size_t up_grid = (size_t)l.max_segments * ((I + kCols - 1) / kCols);
  if (rc == LOWM_OK)
    rc = go(l.seg_rows == 64
                ? in_lines(D, u->w13, &moe_up_kernel<8, 3, false>, &moe_up_kernel<8, 3, true>)
            : l.seg_rows == 32
                ? in_lines(D, u->w13, &moe_up_kernel<4, 4, false>, &moe_up_kernel<4, 4, true>)
            : up_grid <= 256
                ? in_lines(D, u->w13, &moe_up_kernel<2, 6, false>, &moe_up_kernel<2, 6, true>)
                : in_lines(D, u->w13, &moe_up_kernel<2, 3, false>, &moe_up_kernel<2, 3, true>),
            up_grid, 0);
  const size_t lds = sizeof(Segment) * (size_t)l.max_segments +
                     sizeof(Pair) * (size_t)((T * K + 1) / 2 * 2) +
                     sizeof(float) * kWaves * (size_t)T * kCols;
  const size_t down_grid = (size_t)((D + kCols - 1) / kCols) * l.down_splits;
  if (rc == LOWM_OK)
    // Up to one workgroup to a CU each has a CU to itself: a ring of 6 slots, 102 KB,
    // beside up to 29 KB of lists and sums (8 slots are no faster).  More share a CU
    // in pairs, with 3 slots, rather than leave the last ones a round of their own
    // (T 16, D 2488, I 272, E 128, 312 workgroups: 66 us with 3 slots, 76 with 6;
    // T 64, D 4096, I 1024, E 64, 256 workgroups: 289 and 261).
    rc = go(l.seg_rows == 64
                ? in_lines(I, u->w2, &moe_down_kernel<8, 3, false>, &moe_down_kernel<8, 3, true>)
            : l.seg_rows == 32
                ? in_lines(I, u->w2, &moe_down_kernel<4, 5, false>, &moe_down_kernel<4, 5, true>)
            : down_grid <= 256
                ? in_lines(I, u->w2, &moe_down_kernel<2, 6, false>, &moe_down_kernel<2, 6, true>)
                : in_lines(I, u->w2, &moe_down_kernel<2, 3, false>, &moe_down_kernel<2, 3, true>),
            down_grid, lds);
  return rc;
}

}  // namespace
}  // namespace lowm

extern "C" {

size_t lowm_moe_workspace_bytes(int T, int D, int I, int E, int top_k) {
  return lowm::moe_sizes(T, D, I, E, top_k) ? lowm::layout_of(T, D, I, E, top_k).bytes : 0;
}

int lowm_moe(const lowm_moe_args* args, void* stream) {
  return lowm::moe(args, static_cast<hipStream_t>(stream));
}

}  // extern "C"
