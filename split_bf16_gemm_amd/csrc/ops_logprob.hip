// ops_logprob.hip -- log probabilities of given tokens, with entropy, rank and
// the most likely alternatives (include/lowm_ops.h), for gfx950.
//
// One pass over a row of logits with a running maximum m, S = sum e^(l-m) and
// T = sum e^(l-m) (l-m), each lane its own and joined at the row's end:
//
//   m' = max(m, l) ;  S' = S e^(m-m') + e^(l-m') ;  T' = (T + S (m-m')) e^(m-m') + ...
//   log p = l - m - log S ;  entropy = log S - T / S
//
// so nothing overflows and the logits are read once.  The alternatives cost the
// pass nothing: each lane's running maximum is its greatest logit, the top_n-th
// of them bounds the row's top_n-th from below, and only the few lanes whose
// maximum passes the bound have their logits read again (from the caches).
// What passes is sorted by a 64-bit key: the logit's bits in an order that
// integers compare, then the complement of its id, so equal logits go by id and
// no two keys are equal.
// Bound by HBM for many rows (2 or 4 bytes a logit against some 12 vector
// instructions); few rows are cut into up to kMaxSplits pieces, joined by a
// second small kernel.
#include "ops_common.cuh"

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
};

// A piece's part of a row's sums, followed by its top_n keys.
struct Part {
  float m, s, t;
  int32_t above;                         // logits greater than the token's
};
__host__ __device__ constexpr size_t part_bytes(int n) { return sizeof(Part) + 8 * (size_t)n; }

__device__ __forceinline__ uint64_t key_of(float x, int id) {
  return (uint64_t)order(x) << 32 | (uint32_t)~id;
}

// e^d for d <= 0: the difference is exact to a rounding before the scaling.
__device__ __forceinline__ float exp_of(float d) {
  return __builtin_amdgcn_exp2f(d * 1.44269504088896340736f);
}
// A difference of logits for a factor that multiplies e^d: below -200 e^d is 0
// in fp32, and 0 * -infinity would be NaN.
__device__ __forceinline__ float held(float d) { return fmaxf(d, -200.f); }

struct Sums {
  float m, s, t;
  // Rescales to the maximum m2 >= m.
  __device__ __forceinline__ void to(float m2) {
    const float d = held(m - m2);        // NaN (both -infinity) becomes -200: s and t are 0
    const float k = exp_of(d);
    t = (t + s * d) * k;
    s *= k;
    m = m2;
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

// An order() that at least n of the wavefront's logits are above: the n-th of
// its 64 lanes' own greatest logits, to 16 bits.  (n <= 32, so there always are n.)
__device__ __forceinline__ uint32_t wave_bound(float most, int n) {
  const uint32_t o = order(most);
  uint32_t t = 0;
  for (int bit = 31; bit >= 16; --bit) {
    const uint32_t more = t | 1u << bit;
    if (__popcll(__ballot(o >= more)) >= n) t = more;
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

// The sums' part of N logits of each lane; the greatest of them is `most`.
template <int N>
__device__ __forceinline__ void add_logits(Sums& sum, int& above, const float (&x)[N], float most,
                                           float token_logit) {
  sum.to(fmaxf(sum.m, most));
  const float m = sum.m == kNone ? 0.f : sum.m;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float d = x[i] - m, e = exp_of(d);
    sum.s += e;                          // a NaN logit shows here
    sum.t += e * held(d);
    above += x[i] > token_logit;
  }
}

// What a row's sums come to, by one thread.
__device__ __forceinline__ void finish_row(const lowm_token_logprobs_args& u, int64_t row,
                                           const Sums& a, int above, float token_logit,
                                           bool token_ok, float* log_s, bool* bad) {
  // An infinity or a NaN among the logits makes S a NaN (inf - inf).
  *bad = !(a.s >= 0.f) || a.m == -kNone;
  const bool empty = a.m == kNone;
  const float ls = empty ? 0.f : logf(a.s);
  const float nan = __builtin_nanf("");
  u.logprob[row] = *bad || !token_ok ? nan : empty ? kNone : token_logit - a.m - ls;
  u.entropy[row] = *bad ? nan : empty ? 0.f : ls - a.t / a.s;
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
__global__ __launch_bounds__(kTh) void token_logprobs_kernel(LogprobArgs a) {
  using R = Raw<T>;
  constexpr int kRuns = kPerThread / R::kPer;   // of 16 bytes
  __shared__ uint64_t keys[kCap];
  __shared__ uint64_t list[kMaxTop];
  __shared__ uint64_t best[kW];
  __shared__ Sums sums[kW];
  __shared__ int totals[kW];
  __shared__ uint32_t bounds[kW];
  __shared__ int lanes[kTh];
  __shared__ int n_lanes, n_keys;
  const lowm_token_logprobs_args& u = a.u;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int64_t row = blockIdx.x / a.splits;
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

  auto run_at = [&](int c, int r) { return (c * kRuns + r) * kTh + tid; };
  auto fetch = [&](int c, ops_u32x4 (&w)[kRuns]) {
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      w[r] = ops_u32x4{R::kMask, R::kMask, R::kMask, R::kMask};
      const int j = run_at(c, r);
      if (j < runs) w[r] = body[j];
    }
  };

  ops_u32x4 w[kRuns], ahead[kRuns];
  fetch(0, w);
  float token_logit;
  const bool token_ok = token_of(u, row, &token_logit);
  Sums sum{kNone, 0.f, 0.f};
  int above = 0;
  const int n = u.top_n;
  if (tid == 0) n_lanes = n_keys = 0;
  if (tid < kMaxTop) list[tid] = 0;

  for (int c = 0; c < chunks; ++c) {
    if (c + 1 < chunks) fetch(c + 1, ahead);
    float x[kPerThread];
#pragma unroll
    for (int r = 0; r < kRuns; ++r)
#pragma unroll
      for (int i = 0; i < R::kPer; ++i) x[r * R::kPer + i] = R::get(w[r], i);
    float most = x[0];
#pragma unroll
    for (int i = 1; i < kPerThread; ++i) most = fmaxf(most, x[i]);
    add_logits(sum, above, x, most, token_logit);
#pragma unroll
    for (int r = 0; r < kRuns; ++r) w[r] = ahead[r];
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
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) above += __shfl_xor(above, o);
  if (lane == 0) {
    sums[wave] = sum;
    totals[wave] = above;
  }
  if (n > 0) {
    const uint32_t own = wave_bound(most, n);
    if (lane == 0) bounds[wave] = own;
  }
  __syncthreads();
  if (n > 0) {
    uint32_t thr = bounds[0];
#pragma unroll
    for (int v = 1; v < kW; ++v) thr = bounds[v] > thr ? bounds[v] : thr;
    const float bar = value_of(thr);
    if (most > bar) lanes[atomicAdd(&n_lanes, 1)] = tid;
    auto add = [&](float v, int e) {
      if (v > bar) {
        const int to = atomicAdd(&n_keys, 1);
        if (to < kCap) keys[to] = key_of(v, first + e);
      }
    };
    if (wave == 0) add(x1[0], single);
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
    char* part = static_cast<char*>(u.workspace) + (size_t)blockIdx.x * part_bytes(n);
    if (tid == 0) *reinterpret_cast<Part*>(part) = Part{all.m, all.s, all.t, total};
    if (tid < n) reinterpret_cast<uint64_t*>(part + sizeof(Part))[tid] = list[tid];
    return;
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
// Joins a row's pieces.  Each piece's keys are in order, so the greatest of the
// pieces' last keys bounds the row's n-th from below.
__global__ __launch_bounds__(kTh) void token_logprobs_join_kernel(LogprobArgs a) {
  __shared__ uint64_t buf[kMaxSplits * kMaxTop];
  __shared__ uint64_t list[kMaxTop];
  __shared__ int count;
  __shared__ float scale[2];
  __shared__ int is_bad;
  const lowm_token_logprobs_args& u = a.u;
  const int tid = threadIdx.x, n = u.top_n;
  const int64_t row = blockIdx.x;
  const char* parts = static_cast<const char*>(u.workspace) + (size_t)row * a.splits * part_bytes(n);
  if (tid == 0) count = 0;
  if (tid < kMaxTop) list[tid] = 0;
  __syncthreads();
  if (tid < kWave) {
    float token_logit;
    const bool token_ok = token_of(u, row, &token_logit);
    Part p{kNone, 0.f, 0.f, 0};
    uint64_t last = 0;
    if (tid < a.splits) {
      const char* at = parts + (size_t)tid * part_bytes(n);
      p = *reinterpret_cast<const Part*>(at);
      if (n > 0) last = reinterpret_cast<const uint64_t*>(at + sizeof(Part))[n - 1];
    }
    const Sums all = wave_join(Sums{p.m, p.s, p.t});
    int above = p.above;
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) {
      above += __shfl_xor(above, off);
      const uint64_t o = __shfl_xor(last, off);
      last = o > last ? o : last;
    }
    if (tid == 0) {
      float log_s;
      bool bad;
      finish_row(u, row, all, above, token_logit, token_ok, &log_s, &bad);
      scale[0] = all.m;
      scale[1] = log_s;
      is_bad = bad;
      list[0] = last;                    // for a moment: the bound
    }
  }
  if (n == 0) return;
  __syncthreads();
  const uint64_t bound = list[0];
  __syncthreads();
  if (tid == 0) list[0] = 0;
  for (int i = tid; i < a.splits * n; i += kTh) {
    const uint64_t key =
        reinterpret_cast<const uint64_t*>(parts + (size_t)(i / n) * part_bytes(n) + sizeof(Part))[i % n];
    if (key >= bound && key) buf[atomicAdd(&count, 1)] = key;
  }
  __syncthreads();
  const int found = count;
  for (int i = tid; i < found; i += kTh) {
    const uint64_t key = buf[i];
    int place = 0;
    for (int j = 0; j < found; ++j) place += buf[j] > key;
    if (place < n) list[place] = key;
  }
  __syncthreads();
  if (tid < n) finish_top(u, row, tid, list[tid], scale[0], scale[1], is_bad != 0);
}

// Pieces of a row: enough that the rows' pieces number 1024 (four workgroups
// per CU), each at least kPiece long.
int splits_of(int M, int V) {
  const int want = (1024 + M - 1) / M, most = (V + kPiece - 1) / kPiece;
  const int s = want < most ? want : most;
  return s < kMaxSplits ? s : kMaxSplits;
}

size_t logprobs_workspace(int M, int V, int n) {
  if (M < 1 || V < 1 || V > (1 << 30) || n < 0 || n > kMaxTop) return 0;
  const int s = splits_of(M, V);
  return s > 1 ? (size_t)M * s * part_bytes(n) : 0;
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
      (need > 0 && ((uintptr_t)u->workspace & 15)))
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
  LogprobArgs a{*u, splits_of(u->M, u->V), 0};
  // Pieces of whole 16-byte runs, so that an aligned row has aligned pieces.
  a.per = ((u->V + a.splits - 1) / a.splits + 7) / 8 * 8;
  a.splits = (u->V + a.per - 1) / a.per;
  if ((int64_t)a.splits * M > 0x7fffffff) return LOWM_ERR_UNSUPPORTED;
  void* args[] = {&a};
  const void* fn = u->logits_type == LOWM_F32
                       ? reinterpret_cast<const void*>(&token_logprobs_kernel<float>)
                       : reinterpret_cast<const void*>(&token_logprobs_kernel<uint16_t>);
  int rc = launched(hipLaunchKernel(fn, dim3((unsigned)(a.splits * M)), dim3(kTh), args, 0, stream));
  if (rc == LOWM_OK && a.splits > 1)
    rc = launched(hipLaunchKernel(reinterpret_cast<const void*>(&token_logprobs_join_kernel),
                                  dim3((unsigned)M), dim3(kTh), args, 0, stream));
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
