// ops_logprob.hip -- log probabilities of given tokens, with entropy, rank and
// the most likely alternatives (include/lowm_ops.h), for gfx950.
//
// One pass over a row of logits with a running maximum m, S = sum e^(l-m) and
// T = sum e^(l-m) (l-m), each lane its own and joined at the row's end:
//
//   m' = max(m, l) ;  S' = S e^(m-m') + e^(l-m') ;  T' = (T + S (m-m')) e^(m-m') + ...
//   log p = l - m - log S ;  entropy = log S - T / S
//
// so nothing overflows and the logits are read once.  The alternatives are kept
// as a sorted list of 64-bit keys (the logit's bits in an order that integers
// compare, then the complement of its id, so equal logits go by id and no two
// keys are equal); a later chunk only adds what passes the list's last key.
// Bound by HBM for many rows (2 or 4 bytes a logit against some 13 vector
// instructions); few rows are cut into up to kMaxSplits pieces, joined by a
// second small kernel.
#include "ops_common.cuh"

namespace lowm {
namespace {

constexpr int kTh = 256;                 // threads of a workgroup
constexpr int kW = kTh / kWave;
constexpr int kPerThread = 16;           // logits a thread takes from a chunk
constexpr int kChunk = kTh * kPerThread;
constexpr int kCap = 512;                // candidates a chunk may add at once
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

struct Shared {
  uint64_t list[2][kMaxTop];             // the best so far, greatest first; 0: none
  uint64_t buf[kCap];
  uint64_t best[kW];
  uint32_t thr[kW];
  int count[3];
  Sums sums[kW];
};

// Greatest key of the workgroup; every thread gets it.
__device__ __forceinline__ uint64_t group_max(uint64_t v, uint64_t* lds) {
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) {
    const uint64_t o = __shfl_xor(v, off);
    v = o > v ? o : v;
  }
  __syncthreads();
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < kW; ++w) v = lds[w] > v ? lds[w] : v;
  return v;
}

// The n greatest of list[0..n) and buf[0..count), in order, into next[0..n).
// All keys but the empty ones differ, so each key's place is the number of
// greater ones.  Barriers on both sides are the caller's.
__device__ __forceinline__ void merge_lists(const uint64_t* list, const uint64_t* buf, int count,
                                            int n, uint64_t* next) {
  for (int i = threadIdx.x; i < count + n; i += kTh) {
    const uint64_t key = i < n ? list[i] : buf[i - n];
    int place = 0;
    if (key) {
      for (int j = 0; j < n; ++j) place += list[j] > key;
      for (int j = 0; j < count; ++j) place += buf[j] > key;
      if (place < n) next[place] = key;
    }
  }
}

// An order() that at least n of the workgroup's logits are above, at least thr:
// of each wavefront's 64 lanes' own greatest logits the n-th, to 16 bits, and
// the best of the wavefronts' bounds.  (n <= 32, so there always are n.)
__device__ __forceinline__ uint32_t chunk_bound(float most, int n, uint32_t thr, uint32_t* lds) {
  const uint32_t o = order(most);
  uint32_t t = 0;
  for (int bit = 31; bit >= 16; --bit) {
    const uint32_t more = t | 1u << bit;
    if (__popcll(__ballot(o >= more)) >= n) t = more;
  }
  // Above t - 1.  Below +0 lie the bits of -0, which order() never gives: the
  // next bound down is taken there, so that +0 compares as greater than it.
  t = t == 0x80000000u ? 0x7f7fffffu : t - 1;
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = t;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kW; ++w) thr = lds[w] > thr ? lds[w] : thr;
  return thr;
}

template <typename T>
struct Raw;
template <>
struct Raw<float> {
  static constexpr int kPer = 4;         // logits in 16 bytes
  static constexpr uint32_t kMask = 0xff800000u;
  __device__ static __forceinline__ float get(const ops_u32x4& w, int i) {
    const uint32_t bits = w[i];          // a bit cast of w[i] itself reads element 0
    return __builtin_bit_cast(float, bits);
  }
  __device__ static __forceinline__ void set(ops_u32x4& w, int i, uint32_t bits) { w[i] = bits; }
  using Word = uint32_t;
};
template <>
struct Raw<uint16_t> {
  static constexpr int kPer = 8;
  static constexpr uint32_t kMask = 0xff80u;
  __device__ static __forceinline__ float get(const ops_u32x4& w, int i) {
    return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  }
  __device__ static __forceinline__ void set(ops_u32x4& w, int i, uint32_t bits) {
    w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | bits << 16 : (w[i / 2] & 0xffff0000u) | bits;
  }
  using Word = uint16_t;
};

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
  constexpr int kRuns = kPerThread / R::kPer;
  __shared__ Shared sh;
  const lowm_token_logprobs_args& u = a.u;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int64_t row = blockIdx.x / a.splits;
  const int piece = blockIdx.x % a.splits;
  const int first = piece * a.per;                       // this piece: [first, first + len)
  const int len = first + a.per < u.V ? a.per : u.V - first;
  const T* src = static_cast<const T*>(u.logits) + row * u.ld + first;
  // Logits between the 16-byte boundary below src and src: run j holds the
  // logits [j * kPer - off, (j + 1) * kPer - off) of the piece.
  const int off = (int)(((uintptr_t)src & 15) / sizeof(T));
  const int chunks = (len + off + kChunk - 1) / kChunk;
  const int n = u.top_n;

  float token_logit;
  const bool token_ok = token_of(u, row, &token_logit);

  if (tid < 3) sh.count[tid] = 0;
  if (tid < kMaxTop) sh.list[0][tid] = sh.list[1][tid] = 0;
  __syncthreads();

  auto at = [&](int c, int r) { return (c * kChunk + (r * kTh + tid) * R::kPer) - off; };
  auto fetch = [&](int c, ops_u32x4 (&w)[kRuns]) {
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      const int e = at(c, r);
      if (e >= 0 && e + R::kPer <= len) {
        w[r] = *reinterpret_cast<const ops_u32x4*>(src + e);
      } else {
#pragma unroll
        for (int i = 0; i < R::kPer; ++i)
          R::set(w[r], i,
                 e + i >= 0 && e + i < len
                     ? (uint32_t) reinterpret_cast<const typename R::Word*>(src)[e + i]
                     : R::kMask);
      }
    }
  };

  Sums sum{kNone, 0.f, 0.f};
  int above = 0;                         // of the wavefront
  int cur = 0;                           // which list is the current one
  ops_u32x4 w[kRuns], ahead[kRuns];
  fetch(0, w);
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
    sum.to(fmaxf(sum.m, most));
    const float m = sum.m == kNone ? 0.f : sum.m;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const float d = x[i] - m, e = exp_of(d);
      sum.s += e;                        // a NaN logit shows here
      sum.t += e * held(d);
      above += __popcll(__ballot(x[i] > token_logit));
    }

    if (n > 0) {
      const uint64_t* list = sh.list[cur];
      int* count = &sh.count[c % 3];
      // The third of the counters is cleared here for the next chunk: every
      // thread has passed the barrier after which the last reads of it ended.
      if (tid == 0) sh.count[(c + 1) % 3] = 0;
      // A candidate's order() is above thr: that of the list's last key (an
      // equal logit further on has a greater id, so it comes after it).
      uint32_t thr = (uint32_t)(list[n - 1] >> 32);
      thr = thr > kMasked ? thr : kMasked;
      bool tried = false;
      if (c == 0) {
        thr = chunk_bound(most, n, thr, sh.thr);
        tried = true;
      }
      int found;
      while (true) {
        const float bar = value_of(thr);
        if (most > bar) {
#pragma unroll
          for (int i = 0; i < kPerThread; ++i)
            if (x[i] > bar) {
              const int to = atomicAdd(count, 1);
              if (to < kCap)
                sh.buf[to] = key_of(x[i], first + at(c, i / R::kPer) + i % R::kPer);
            }
        }
        __syncthreads();
        found = *count;
        if (found <= kCap) break;
        // Too many: raise the bound by this chunk's own, or, where that does
        // not do (many equal logits), take the chunk's greatest one by one.
        __syncthreads();
        if (tid == 0) *count = 0;
        if (!tried) {
          thr = chunk_bound(most, n, thr, sh.thr);
          tried = true;
          continue;
        }
        uint64_t last = ~0ull;
        for (int k = 0; k < n; ++k) {
          uint64_t mine = 0;
#pragma unroll
          for (int i = 0; i < kPerThread; ++i)
            if (x[i] > kNone) {
              const uint64_t key = key_of(x[i], first + at(c, i / R::kPer) + i % R::kPer);
              if (key < last && key > mine) mine = key;
            }
          last = group_max(mine, sh.best);
          if (tid == 0) sh.buf[k] = last;      // 0 once there are none left
        }
        __syncthreads();
        found = n;
        break;
      }
      if (found > 0) {
        uint64_t* next = sh.list[cur ^ 1];
        if (tid < n) next[tid] = 0;
        __syncthreads();
        merge_lists(list, sh.buf, found, n, next);
        __syncthreads();
        cur ^= 1;
      }
    }
#pragma unroll
    for (int r = 0; r < kRuns; ++r) w[r] = ahead[r];
  }

  sum = wave_join(sum);
  if (lane == 0) {
    sh.sums[wave] = sum;
    sh.thr[wave] = (uint32_t)above;
  }
  __syncthreads();
  Sums all = sh.sums[0];
  int total = (int)sh.thr[0];
#pragma unroll
  for (int v = 1; v < kW; ++v) {
    Sums o = sh.sums[v];
    const float m = fmaxf(all.m, o.m);
    all.to(m);
    o.to(m);
    all.s += o.s;
    all.t += o.t;
    total += (int)sh.thr[v];
  }
  if (a.splits > 1) {
    char* part = static_cast<char*>(u.workspace) + (size_t)blockIdx.x * part_bytes(n);
    if (tid == 0) *reinterpret_cast<Part*>(part) = Part{all.m, all.s, all.t, total};
    if (tid < n) reinterpret_cast<uint64_t*>(part + sizeof(Part))[tid] = sh.list[cur][tid];
    return;
  }
  float log_s = 0.f;
  bool bad = false;
  if (tid < kWave) {                     // one wavefront: no value has to cross
    if (tid == 0) finish_row(u, row, all, total, token_logit, token_ok, &log_s, &bad);
    log_s = __shfl(log_s, 0);
    bad = __shfl((int)bad, 0);
    if (tid < n) finish_top(u, row, tid, sh.list[cur][tid], all.m, log_s, bad);
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
// per CU), each at least a chunk long.
int splits_of(int M, int V) {
  const int want = (1024 + M - 1) / M, most = (V + kChunk - 1) / kChunk;
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
