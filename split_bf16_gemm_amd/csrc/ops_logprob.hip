// ops_logprob.hip -- log probabilities of given tokens, with entropy, rank and
// the most likely alternatives (include/lowm_ops.h), for gfx950.
//
// One pass over a row of logits with a running maximum m, each lane its own and
// joined at the row's end.  With L = log2 e and c = m L, rounded,
//
//   d = l L - c ;  S = sum 2^d ;  T = sum 2^d d
//   m' > m:  T' = (T + S (c-c')) 2^(c-c') ;  S' = S 2^(c-c')
//   log p = l - m - (log S + (c - m L) log 2) ;  entropy = log S - log 2 T / S
//
// (d is one fused multiply-add, rounded once; what c's own rounding moves all the
// terms by is known and put back where sums join and at the end).  That is under
// 1/16 up to a maximum of 2^20; past it the terms take d = (l - m) L, which needs
// nothing put back.  So no term is above 2^(1/16), whatever the finite logits are,
// and the logits are read once.  The alternatives cost the
// pass nothing: each lane's running maximum is its greatest logit, the top_n-th
// of those bounds the row's top_n-th from below, and only the few lanes whose
// maximum passes the bound have their logits read again (from the caches).
// What passes is sorted by a 64-bit key: the logit's bits in an order that
// integers compare, then the complement of its id, so equal logits go by id and
// no two keys are equal.
// Bound by HBM and the vector unit alike for many rows (2 or 4 bytes a logit
// against some 12 vector instructions, the exponential a quarter-rate one): 2048
// rows of 49152 bf16, 201 MB, 45 us (4.5 TB/s), where a plain read takes 30.  Few
// rows are cut into up to kMaxSplits pieces, joined by the last workgroup of a row
// to arrive, and are bound by the chain of latencies: read, reduce, pick, hand on,
// join (one row of 49152 8.7 us; 61 rows of 50001 fp32 with 20 alternatives 13.5).
#include "ops_stream.cuh"

namespace lowm {
namespace {

constexpr int kTh = 256;                 // threads of a workgroup
constexpr int kW = kTh / kWave;
constexpr int kPerThread = 16;           // logits a thread takes from a chunk
constexpr int kCap = kTh;                // keys that are sorted
constexpr int kPiece = 4096;             // least logits of a piece of a row
constexpr int kMaxSplits = 32;
constexpr int kMaxTop = LOWM_LOGPROBS_MAX_TOP;
constexpr uint32_t kMasked = 0x007fffffu;   // order() of -infinity
constexpr float kNone = -__builtin_inff();

struct LogprobArgs {
  lowm_token_logprobs_args u;
  int splits, per;                       // pieces of a row, logits in each
  int64_t first;                         // row of this launch
  uint32_t* lines;
  uint64_t* records;
};

// The workspace: a counter line for each row, then a record for each piece of a
// row, 64-bit slots that are zero between calls: the maximum and S, T and the
// count of greater logits, the top_n keys.  Rows are cut only while they are
// fewer than kSplitBelow, into about that many pieces in all.
constexpr int kSplitBelow = 512;
constexpr size_t kRecord = 2 + kMaxTop;
constexpr size_t kLineBytes = 256 * (size_t)kSplitBelow;
constexpr size_t kWorkspace = kLineBytes + 8 * kRecord * 2 * kSplitBelow;
constexpr uint64_t kNoKey = 1;           // an empty key's slot (no key is that small)

__device__ __forceinline__ void store_slot64(uint64_t* p, uint64_t w) {
  __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t load_slot64(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// See take_slot.
__device__ __forceinline__ uint64_t take_slot64(uint64_t* slot, uint64_t w, uint32_t* line) {
  if (w == 0u) {
    const uint64_t t0 = __builtin_amdgcn_s_memrealtime();
    while ((w = load_slot64(slot)) == 0u) {
      if (__builtin_amdgcn_s_memrealtime() - t0 > kFoldPollTicks) {
        store_slot(line + kFaultWord, 1u);
        break;
      }
      __builtin_amdgcn_s_sleep(4);
    }
  }
  store_slot64(slot, 0u);
  return w;
}
// Two words as the complement of their bits: zero only for two words of all
// ones, which a maximum and a count never are.
__device__ __forceinline__ uint64_t pack_words(uint32_t lo, uint32_t hi) {
  return ~((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ uint64_t key_of(float x, int id) {
  return (uint64_t)order(x) << 32 | (uint32_t)~id;
}

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// A difference for a factor that multiplies 2^d: below -300 2^d is 0 in fp32, and
// 0 * -infinity would be NaN.
__device__ __forceinline__ float held(float d) { return fmaxf(d, -300.f); }

// A maximum m past which c = round(m L) is off by too much: half a step of c is
// 1/16 at 2^20, but 128 and more, a factor 2^d past fp32's range, from 2^31 on.
// Its terms take d = (l - m) L, two roundings instead of one; ordinary logits stay
// below.  Infinities are far.
constexpr float kFar = 0x1p20f;
__device__ __forceinline__ bool far(float m) { return fabsf(m) > kFar; }

// c, rounded: the product is not to be fused into the sums it is used in.
__device__ __forceinline__ float scaled(float m) {
#pragma clang fp contract(off)
  return m * kLog2e;
}
// By how much the terms' exponents are too large: m L - c, in one rounding.
__device__ __forceinline__ float offset(float m) {
  return far(m) ? 0.f : __builtin_fmaf(m, kLog2e, -scaled(m));
}

struct Sums {
  float m, s, t;
  // What the terms are relative to, where m is not far; 0 while there is nothing
  // but masked logits.
  __device__ __forceinline__ float base() const { return m == kNone ? 0.f : scaled(m); }
  // Rescales to the maximum m2 >= m.
  __device__ __forceinline__ void to(float m2) {
    // (Nothing there yet: s and t are 0 and stay so.  Of an infinite maximum s is a
    // NaN already.)
    const float m1 = m, from = m1 == kNone ? kNone : base();
    m = m2;
    float d = held(from - base());
    // (where m1 is far above, so is m2)
    const bool apart = (m2 != kNone && far(m2)) || (m1 != kNone && m1 < -kFar);
    if (__builtin_expect(__ballot(apart) != 0, 0) && apart)
      d = m1 == m2 ? 0.f : held((m1 - m2) * kLog2e - (offset(m1) - offset(m2)));
    const float k = __builtin_amdgcn_exp2f(d);
    t = (t + s * d) * k;
    s *= k;
  }
};

__device__ __forceinline__ Sums wave_join(Sums a) {
  a.to(value_of(wave_umax(order(a.m))));
  a.s = wave_sum(a.s);
  a.t = wave_sum(a.t);
  return a;
}

// The greatest bound that what is at or above t passes.  Below +0 lie the bits
// of -0, which order() never gives: the bound is taken further down there, so
// that +0 compares as greater than it.
__device__ __forceinline__ uint32_t below(uint32_t t) {
  return t == 0x80000000u ? 0x7f7fffffu : t - 1;
}

// A bound that at least n of the workgroup's logits pass: the n-th greatest of its
// lanes' own greatest ones (their order()s), to 16 bits.  Every wavefront finds it
// for itself.  (n <= 32, so there always are n.)
__device__ __forceinline__ uint32_t bound_of(const uint32_t* orders, int n) {
  const int lane = threadIdx.x & (kWave - 1);
  uint32_t o[kW];
#pragma unroll
  for (int w = 0; w < kW; ++w) o[w] = orders[w * kWave + lane];
  uint32_t t = 0;
  for (int bit = 31; bit >= 16; --bit) {
    const uint32_t more = t | 1u << bit;
    int have = 0;
#pragma unroll
    for (int w = 0; w < kW; ++w) have += __popcll(__ballot(o[w] >= more));
    if (have >= n) t = more;
  }
  t = below(t);
  return t > kMasked ? t : kMasked;
}

// The logits in 16 bytes.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  static constexpr int kPer = 4;
  static constexpr uint32_t kMask = 0xff800000u;         // -infinity throughout
  __device__ static __forceinline__ float get(const ops_u32x4& w, int i) {
    const uint32_t bits = w[i];          // a bit cast of w[i] itself reads element 0
    return __builtin_bit_cast(float, bits);
  }
};
template <>
struct Raw<uint16_t> {
  static constexpr int kPer = 8;
  static constexpr uint32_t kMask = 0xff80ff80u;
  __device__ static __forceinline__ float get(const ops_u32x4& w, int i) {
    return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  }
};

// N logits of each lane; the greatest of them is `most`.  `above` is the
// wavefront's.
template <int N>
__device__ __forceinline__ void add_logits(Sums& sum, int& above, const float (&x)[N], float most,
                                           float token_logit) {
  sum.to(fmaxf(sum.m, most));
  const float c = sum.base();
  auto term = [&](float d) {
    const float e = __builtin_amdgcn_exp2f(d);
    sum.s += e;                          // a NaN logit shows here
    sum.t = __builtin_fmaf(e, held(d), sum.t);
  };
  const bool apart = sum.m != kNone && far(sum.m);
  if (__builtin_expect(__ballot(apart) != 0, 0)) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      term(apart ? (x[i] - sum.m) * kLog2e : __builtin_fmaf(x[i], kLog2e, -c));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) term(__builtin_fmaf(x[i], kLog2e, -c));
  }
  // Counted by the scalar unit, which has little else to do; and not at all
  // where no lane has a logit that counts.
  if (__ballot(most > token_logit)) {
#pragma unroll
    for (int i = 0; i < N; ++i) above += __popcll(__ballot(x[i] > token_logit));
  }
}

// What a row's sums come to, by one thread.
__device__ __forceinline__ void finish_row(const lowm_token_logprobs_args& u, int64_t row,
                                           const Sums& a, int above, float token_logit,
                                           bool token_ok, float* log_s, bool* bad) {
  // An infinity or a NaN among the logits makes S a NaN (inf - inf).
  *bad = !(a.s >= 0.f) || a.m == -kNone;
  const bool empty = a.m == kNone;
  const float ls = empty ? 0.f : logf(a.s) - offset(a.m) * kLn2;
  const float nan = __builtin_nanf("");
  u.logprob[row] = *bad || !token_ok ? nan : empty ? kNone : token_logit - a.m - ls;
  u.entropy[row] = *bad ? nan : empty ? 0.f : logf(a.s) - kLn2 * (a.t / a.s);
  u.rank[row] = token_ok ? above : -1;
  *log_s = ls;
}
__device__ __forceinline__ void finish_top(const lowm_token_logprobs_args& u, int64_t row, int i,
                                           uint64_t key, float m, float log_s, bool bad) {
  const bool some = key != 0 && !bad;
  const int64_t at = row * u.top_n + i;
  u.top_logprob[at] = bad ? __builtin_nanf("")
                          : some ? value_of((uint32_t)(key >> 32)) - m - log_s : kNone;
  u.top_id[at] = some ? (int32_t)~(uint32_t)key : -1;
}

__device__ __forceinline__ bool token_of(const lowm_token_logprobs_args& u, int64_t row,
                                         float* logit) {
  const int64_t id = u.tokens_bytes == 8 ? static_cast<const int64_t*>(u.tokens)[row]
                                         : static_cast<const int32_t*>(u.tokens)[row];
  const bool ok = id >= 0 && id < u.V;
  *logit = ok ? load1(u.logits, row * u.ld + id, u.logits_type == LOWM_F32) : 0.f;
  return ok;
}

template <typename T>
__global__ __launch_bounds__(kTh, 8) void token_logprobs_kernel(LogprobArgs a) {
  using R = Raw<T>;
  constexpr int kRuns = kPerThread / R::kPer;   // of 16 bytes
  __shared__ uint64_t keys[kMaxSplits * kMaxTop];
  __shared__ uint64_t list[kMaxTop];
  __shared__ uint64_t best[kW];
  __shared__ Sums sums[kW];
  __shared__ int totals[kW];
  __shared__ uint32_t orders[kTh];
  __shared__ int lanes[kTh];
  __shared__ int n_lanes, n_keys, last;
  const lowm_token_logprobs_args& u = a.u;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int64_t row = a.first + blockIdx.x / a.splits;
  const int piece = blockIdx.x % a.splits;
  const int first = piece * a.per;                       // this piece: [first, first + len)
  const int len = first + a.per < u.V ? a.per : u.V - first;
  const T* src = static_cast<const T*>(u.logits) + row * u.ld + first;
  // Whole 16-byte runs between the first and the last 16-byte boundary in the
  // piece, and up to 2 (kPer - 1) single logits beside them.
  const int gap = (int)((16 - ((uintptr_t)src & 15)) & 15) / (int)sizeof(T);
  const int head = gap < len ? gap : len;
  const int runs = (len - head) / R::kPer;
  const int chunks = (runs + kTh * kRuns - 1) / (kTh * kRuns);
  const ops_u32x4* body = reinterpret_cast<const ops_u32x4*>(src + head);

  auto fetch = [&](int c, ops_u32x4 (&w)[kRuns]) {
    const int j0 = c * kRuns * kTh;
    if (j0 + kRuns * kTh <= runs) {
#pragma unroll
      for (int r = 0; r < kRuns; ++r) w[r] = body[j0 + r * kTh + tid];
    } else {
#pragma unroll
      for (int r = 0; r < kRuns; ++r) {
        // (read something and drop it: loads under a branch wait for one another)
        const int j = j0 + r * kTh + tid;
        w[r] = body[j < runs ? j : runs - 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[r][i] = j < runs ? w[r][i] : R::kMask;
      }
    }
  };

  ops_u32x4 even[kRuns], odd[kRuns];
  if (chunks > 0) fetch(0, even);
  float token_logit;
  const bool token_ok = token_of(u, row, &token_logit);
  Sums sum{kNone, 0.f, 0.f};
  int above = 0;
  const int n = u.top_n;
  if (tid == 0) n_lanes = n_keys = 0;
  if (tid < kMaxTop) list[tid] = 0;

  auto take = [&](const ops_u32x4 (&w)[kRuns]) {
    float x[kPerThread];
#pragma unroll
    for (int r = 0; r < kRuns; ++r)
#pragma unroll
      for (int i = 0; i < R::kPer; ++i) x[r * R::kPer + i] = R::get(w[r], i);
    float most = x[0];
#pragma unroll
    for (int i = 1; i < kPerThread; ++i) most = fmaxf(most, x[i]);
    add_logits(sum, above, x, most, token_logit);
  };
  for (int c = 0; c < chunks; c += 2) {
    if (c + 1 < chunks) fetch(c + 1, odd);
    take(even);
    if (c + 1 < chunks) {
      if (c + 2 < chunks) fetch(c + 2, even);
      take(odd);
    }
  }
  const float most = sum.m;              // of the lane's runs
  // The single logits beside the runs, one for each of the first lanes.
  const int tail = head + runs * R::kPer;
  const int single = tid < head ? tid : tail + tid - head;
  float x1[1] = {kNone};
  if (wave == 0) {
    if (single < len) x1[0] = load1(src, single, sizeof(T) == 4);
    add_logits(sum, above, x1, x1[0], token_logit);
  }

  sum = wave_join(sum);
  if (lane == 0) {
    sums[wave] = sum;
    totals[wave] = above;
  }
  orders[tid] = order(most);
  __syncthreads();
  if (n > 0) {
    const float bar = value_of(bound_of(orders, n));
    auto add = [&](float v, int e) {
      if (v > bar) {
        const int to = atomicAdd(&n_keys, 1);
        if (to < kCap) keys[to] = key_of(v, first + e);
      }
    };
    if (wave == 0) add(x1[0], single);
    if (chunks <= 1) {                   // all there is is still in registers
      if (most > bar) {
#pragma unroll
        for (int r = 0; r < kRuns; ++r)
#pragma unroll
          for (int i = 0; i < R::kPer; ++i)
            add(R::get(even[r], i), head + (r * kTh + tid) * R::kPer + i);
      }
    } else {
      if (most > bar) lanes[atomicAdd(&n_lanes, 1)] = tid;
      __syncthreads();
      const int per_lane = (runs + kTh - 1) / kTh, tasks = n_lanes * per_lane;
      for (int q = tid; q < tasks; q += kTh) {
        const int j = q % per_lane * kTh + lanes[q / per_lane];
        if (j < runs) {
          const ops_u32x4 again = body[j];
#pragma unroll
          for (int i = 0; i < R::kPer; ++i) add(R::get(again, i), head + j * R::kPer + i);
        }
      }
    }
    __syncthreads();
    int count = n_keys;
    if (count > kCap) {
      // More equal logits at the bound than there is room for: the greatest
      // keys one by one, each from the whole piece.
      uint64_t last = ~0ull;
      for (int k = 0; k < n && last; ++k) {
        uint64_t mine = 0;
        for (int e = tid; e < len; e += kTh) {
          const float v = load1(src, e, sizeof(T) == 4);
          const uint64_t key = key_of(v, first + e);
          if (v > kNone && key < last && key > mine) mine = key;
        }
        const uint32_t hi = wave_umax((uint32_t)(mine >> 32));
        const uint32_t lo = wave_umax((uint32_t)(mine >> 32) == hi ? (uint32_t)mine : 0u);
        __syncthreads();
        if (lane == 0) best[wave] = (uint64_t)hi << 32 | lo;
        __syncthreads();
        last = best[0];
#pragma unroll
        for (int v = 1; v < kW; ++v) last = best[v] > last ? best[v] : last;
        if (tid == 0) list[k] = last;
      }
    } else if (tid < count) {            // a key's place is the number of greater ones
      const uint64_t key = keys[tid];
      int place = 0;
      for (int j = 0; j < count; ++j) place += keys[j] > key;
      if (place < n) list[place] = key;
    }
    __syncthreads();
  }
  Sums all = sums[0];
  int total = totals[0];
#pragma unroll
  for (int v = 1; v < kW; ++v) {
    Sums o = sums[v];
    const float m = fmaxf(all.m, o.m);
    all.to(m);
    o.to(m);
    all.s += o.s;
    all.t += o.t;
    total += totals[v];
  }
  if (a.splits > 1) {
    uint64_t* record = a.records + (size_t)row * a.splits * (2 + n);
    uint64_t* own = record + (size_t)piece * (2 + n);
    if (tid == 0) {
      store_slot64(own, pack_words(__builtin_bit_cast(uint32_t, all.s),
                                   __builtin_bit_cast(uint32_t, all.m)));
      store_slot64(own + 1, pack_words(__builtin_bit_cast(uint32_t, all.t), (uint32_t)total));
    }
    if (tid < n) store_slot64(own + 2 + tid, list[tid] ? list[tid] : kNoKey);
    uint32_t* line = a.lines + row * kCtrStride;
    if (!arrive_last(line, a.splits, &last)) return;
    // The pieces' sums by the first wavefront, their keys by all.  Each piece's
    // keys are in order, so the greatest of the pieces' last keys bounds the
    // row's n-th from below.
    uint64_t w0 = 0, w1 = 0, w[kMaxSplits * kMaxTop / kTh];
    if (tid < a.splits) {
      w0 = load_slot64(record + (size_t)tid * (2 + n));
      w1 = load_slot64(record + (size_t)tid * (2 + n) + 1);
    }
    const int slots = a.splits * n;
    auto slot = [&](int j) {
      const int i = tid + j * kTh;
      return record + (size_t)(i / n) * (2 + n) + 2 + i % n;
    };
#pragma unroll
    for (int j = 0; j < kMaxSplits * kMaxTop / kTh; ++j)
      if (tid + j * kTh < slots) w[j] = load_slot64(slot(j));
    if (tid == 0) {
      best[0] = 0;
      n_keys = 0;
    }
    if (tid < kMaxTop) list[tid] = 0;
    if (tid < kWave) {
      all = Sums{kNone, 0.f, 0.f};
      total = 0;
      if (tid < a.splits) {
        w0 = ~take_slot64(record + (size_t)tid * (2 + n), w0, line);
        w1 = ~take_slot64(record + (size_t)tid * (2 + n) + 1, w1, line);
        all = Sums{__builtin_bit_cast(float, (uint32_t)(w0 >> 32)),
                   __builtin_bit_cast(float, (uint32_t)w0),
                   __builtin_bit_cast(float, (uint32_t)w1)};
        total = (int)(w1 >> 32);
      }
      all = wave_join(all);
#pragma unroll
      for (int o = kWave / 2; o > 0; o >>= 1) total += __shfl_xor(total, o);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMaxSplits * kMaxTop / kTh; ++j)
      if (tid + j * kTh < slots) {
        w[j] = take_slot64(slot(j), w[j], line);
        if ((tid + j * kTh) % n == n - 1)
          atomicMax(reinterpret_cast<unsigned long long*>(&best[0]), (unsigned long long)w[j]);
      }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMaxSplits * kMaxTop / kTh; ++j)
      if (tid + j * kTh < slots && w[j] >= best[0] && w[j] > kNoKey)
        keys[atomicAdd(&n_keys, 1)] = w[j];
    __syncthreads();
    const int found = n_keys;
    for (int i = tid; i < found; i += kTh) {
      const uint64_t key = keys[i];
      int place = 0;
      for (int j = 0; j < found; ++j) place += keys[j] > key;
      if (place < n) list[place] = key;
    }
    __syncthreads();
  }
  float log_s = 0.f;
  bool bad = false;
  if (tid < kWave) {                     // one wavefront: no value has to cross
    if (tid == 0) finish_row(u, row, all, total, token_logit, token_ok, &log_s, &bad);
    log_s = __shfl(log_s, 0);
    bad = __shfl((int)bad, 0);
    if (tid < n) finish_top(u, row, tid, list[tid], all.m, log_s, bad);
  }
}

// Pieces of a row: enough that the rows' pieces number kSplitBelow (two
// workgroups per CU), each at least kPiece long.  Measured on MI355X at 256 / 512
// / 1024: M 64, V 49152 bf16 10.4 / 10.9 / 11.0 us, M 128 12.9 / 11.9 / 13.2,
// M 512 16.9 / 16.7 / 18.2, M 800 22.5 / 22.4 / 24.6.
int splits_of(int M, int V) {
  const int want = (kSplitBelow + M - 1) / M, most = (V + kPiece - 1) / kPiece;
  const int s = want < most ? want : most;
  return s < kMaxSplits ? s : kMaxSplits;
}

size_t logprobs_workspace(int M, int V, int n) {
  if (M < 1 || V < 1 || V > (1 << 30) || n < 0 || n > kMaxTop) return 0;
  return splits_of(M, V) > 1 ? kWorkspace : 0;
}

int token_logprobs(const lowm_token_logprobs_args* u, hipStream_t stream) {
  if (!u || u->M < 0 || u->V < 1 || u->ld < u->V || u->top_n < 0) return LOWM_ERR_INVALID_ARG;
  if ((u->logits_type != LOWM_BF16 && u->logits_type != LOWM_F32) ||
      (u->tokens_bytes != 4 && u->tokens_bytes != 8))
    return LOWM_ERR_INVALID_ARG;
  if (u->M == 0) return LOWM_OK;
  if (!u->logits || !u->tokens || !u->logprob || !u->entropy || !u->rank ||
      (u->top_n > 0 && (!u->top_logprob || !u->top_id)))
    return LOWM_ERR_INVALID_ARG;
  if (u->top_n > kMaxTop || u->V > (1 << 30)) return LOWM_ERR_UNSUPPORTED;
  const int es = type_bytes(u->logits_type);
  const size_t need = logprobs_workspace(u->M, u->V, u->top_n);
  if (need > 0 && (!u->workspace || u->workspace_bytes < need)) return LOWM_ERR_WORKSPACE;
  if (((uintptr_t)u->logits & (es - 1)) || ((uintptr_t)u->tokens & (u->tokens_bytes - 1)) ||
      (((uintptr_t)u->logprob | (uintptr_t)u->entropy | (uintptr_t)u->rank) & 3) ||
      (u->top_n > 0 && (((uintptr_t)u->top_logprob | (uintptr_t)u->top_id) & 3)) ||
      (need > 0 && ((uintptr_t)u->workspace & 255)))
    return LOWM_ERR_UNSUPPORTED;
  const int64_t M = u->M, n = u->top_n;
  const Span in[] = {span_of(u->logits, M, u->V, u->ld, es),
                     span_of(u->tokens, 1, M, M, u->tokens_bytes)};
  const Span out[] = {span_of(u->logprob, 1, M, M, 4), span_of(u->entropy, 1, M, M, 4),
                      span_of(u->rank, 1, M, M, 4),
                      span_of(n ? u->top_logprob : nullptr, 1, M * n, M * n, 4),
                      span_of(n ? u->top_id : nullptr, 1, M * n, M * n, 4),
                      span_of(need ? u->workspace : nullptr, 1, (int64_t)need, (int64_t)need, 1)};
  for (int i = 0; i < 6; ++i) {
    for (const Span& s : in)
      if (meet(out[i], s)) return LOWM_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return LOWM_ERR_INVALID_ARG;
  }
  char* w = static_cast<char*>(u->workspace);
  LogprobArgs a{*u, splits_of(u->M, u->V), 0, 0, reinterpret_cast<uint32_t*>(w),
                reinterpret_cast<uint64_t*>(w + (need ? kLineBytes : 0))};
  // Pieces of whole 16-byte runs, so that an aligned row has aligned pieces.
  a.per = ((u->V + a.splits - 1) / a.splits + 7) / 8 * 8;
  a.splits = (u->V + a.per - 1) / a.per;
  void* args[] = {&a};
  const void* fn = u->logits_type == LOWM_F32
                       ? reinterpret_cast<const void*>(&token_logprobs_kernel<float>)
                       : reinterpret_cast<const void*>(&token_logprobs_kernel<uint16_t>);
  constexpr int64_t most = kMaxThreads / kTh;            // (rows in pieces are far fewer)
  int rc = LOWM_OK;
  for (int64_t& row = a.first; row < M && rc == LOWM_OK; row += most)
    rc = launched(hipLaunchKernel(fn, dim3((unsigned)(a.splits * (M - row < most ? M - row : most))),
                                  dim3(kTh), args, 0, stream));
  return rc;
}

}  // namespace
}  // namespace lowm

extern "C" {

size_t lowm_token_logprobs_workspace_bytes(int M, int V, int top_n) {
  return lowm::logprobs_workspace(M, V, top_n);
}

int lowm_token_logprobs(const lowm_token_logprobs_args* args, void* stream) {
  return lowm::token_logprobs(args, static_cast<hipStream_t>(stream));
}

}  // extern "C"
