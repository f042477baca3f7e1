// ops_cache.hip -- rows into and out of the paged 8-bit cache
// (include/lowm_cache.h) for gfx950.
//
//   append:  s' = max(s, max|new| / top) ;  q = round(new / s') ;  q_old = round(q_old s / s')
//   read:    bf16(q s)
//
// A workgroup owns one head of one page, its keys or its values, so nothing it
// reads or writes is another's: 256 threads for long rows of a sequence, a wavefront
// where a page gets a token or two (61 sequences of one token: as many workgroups, a
// quarter of the wavefronts to start).  A thread holds four tokens by eight elements:
// the bytes meet in LDS, values turned into pieces of 16 tokens, padded so that the
// lanes' words lie in distinct banks, and go from there to memory in whole pieces, one
// after another.  A page that is being filled token by token keeps its bytes
// and its scale until a token is larger than all before it; only then are the
// earlier ones rounded again, to the new step, which is at most half a step off
// for each time the scale has grown.
//
// Bound by HBM for long rows (4 x 16384 rows of 8 heads of 128: 107 us, 3.8 TB/s read and
// written, and 83 us, 4.9 TB/s, back; a large copy 5.0): a workgroup has to have its page's
// maximum before it writes (2 x 4100 rows: 20 us for 51 MB; 7 workgroups fit a CU, so that
// 1792 of the 2112 run at once).  One token to a sequence is a chain of lengths, table, scale and
// page (61 sequences 4.7 us in a graph).
#include "ops_cache.cuh"

namespace lowm {
namespace {

// The page of a sequence that a workgroup serves, by its number among the pages
// that the call's rows touch.
struct Touched {
  Rows rows;
  int lo, hi;          // positions of the call's rows on it
  int page;            // -1: none
  int begin;           // position of its first token
};
__device__ __forceinline__ Touched page_of(const lowm_sequences& s, int P, int item,
                                           int uniform_pages) {
  Touched t;
  t.page = -1;
  int b = 0, nth = 0;
  if (!s.row_starts) {
    b = item / uniform_pages;
    nth = item % uniform_pages;
    t.rows = rows_of(s, b);
  } else {
    // every wavefront looks for itself, 64 sequences at a time
    const int lane = threadIdx.x & (kWave - 1);
    b = -1;
    for (int at = 0; at < s.B; at += kWave) {
      const Rows mine = rows_of(s, at + lane < s.B ? at + lane : s.B - 1);
      const int n = at + lane < s.B ? Stretch(s, mine).pages() : 0;
      const int sum = wave_scan(n);
      const int total = __builtin_amdgcn_readlane(sum, kWave - 1);
      if (item - nth < total) {
        const uint64_t past = __ballot(sum > item - nth);
        const int first = __builtin_ctzll(past);
        b = at + first;
        nth = item - nth - __builtin_amdgcn_readlane(sum - n, first);
        t.rows = Rows{__builtin_amdgcn_readlane(mine.first, first),
                      __builtin_amdgcn_readlane(mine.n, first),
                      __builtin_amdgcn_readlane(mine.len, first)};
        break;
      }
      nth += total;
    }
    if (b < 0) return t;
  }
  const Stretch all(s, t.rows);
  if (nth < 0 || nth >= all.pages()) return t;
  const int p = all.lo / LOWM_PAGE + nth;
  t.begin = p * LOWM_PAGE;
  t.lo = all.lo > t.begin ? all.lo : t.begin;
  t.hi = all.hi - t.begin < LOWM_PAGE ? all.hi : t.begin + LOWM_PAGE;
  const int page = s.table[b * s.table_ld + p];
  if (page >= 0 && page < P) t.page = page;
  return t;
}

// Values in LDS: 16 bytes of four tokens' quads for each element, one more piece
// for every eight of them.
__device__ __forceinline__ int turned(int D, int group, int d) {   // in words
  return (group * (D + D / 8) + d + d / 8) * 4;
}
inline int turned_words(int D) { return 4 * (D + D / 8) * 4; }

// Keys in LDS: the page's pieces, one more for every 64 of them.
__device__ __forceinline__ int key_words(int chunk, int token) {
  return (chunk * (LOWM_PAGE + 1) + token) * 4;
}

struct Levels {
  float scale;
  bool e4m3;
  RowScale i8;
  __device__ __forceinline__ Levels(float s, bool e) : scale(s), e4m3(e), i8(s) {}
  // Four elements as bytes.
  __device__ __forceinline__ uint32_t of(float a, float b, float c, float d) const {
    if (!e4m3) return i8.quantise4(a, b, c, d);
    if (!i8.some) return 0u;
    return bytes(a / scale, b / scale, c / scale, d / scale);
  }
  static __device__ __forceinline__ float held(float x) { return fminf(fmaxf(x, -448.f), 448.f); }
  static __device__ __forceinline__ uint32_t bytes(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(held(a), held(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(held(c), held(d), w, true);
  }
};
// The four values of a word of bytes.
__device__ __forceinline__ void unpack4(uint32_t w, bool e4m3, float (&v)[4]) {
  if (e4m3) {
    v[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0);
    v[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1);
    v[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2);
    v[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(w >> 8 * i);
  }
}
// A word of earlier bytes at the new scale.
__device__ __forceinline__ uint32_t again4(uint32_t w, bool e4m3, float ratio) {
  float v[4];
  unpack4(w, e4m3, v);
  if (e4m3) return Levels::bytes(v[0] * ratio, v[1] * ratio, v[2] * ratio, v[3] * ratio);
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= ((uint32_t)(int)rintf(v[i] * ratio) & 255u) << 8 * i;
  return r;
}

struct AppendArgs {
  lowm_cache_append_args u;
  int uniform_pages;
  int first_item;
};

// Q items, each four tokens by eight elements, stay in a thread's registers; where a page
// has more of them they are read a second time.
template <int Q, int THREADS>
__global__ __launch_bounds__(THREADS) void append_kernel(AppendArgs a) {
  const lowm_cache_append_args& u = a.u;
  const lowm_kv_cache& c = u.cache;
  __shared__ uint32_t tops[THREADS / kWave];
  extern __shared__ __align__(16) uint32_t turn[];
  const Touched t = page_of(u.seq, c.P, a.first_item + (int)blockIdx.x, a.uniform_pages);
  if (t.page < 0) return;
  const int head = blockIdx.y, D = c.D, chunks = D / 8;
  const bool values = blockIdx.z, f32 = u.type == LOWM_F32, e4m3 = c.type == LOWM_E4M3;
  const void* x = values ? u.v : u.k;
  const int64_t x_row = values ? u.v_row : u.k_row,
                x_at = head * (values ? u.v_head : u.k_head);
  uint8_t* out = static_cast<uint8_t*>(values ? c.v : c.k) + page_offset(c, t.page, head);
  float* scale_at = (values ? c.v_scale : c.k_scale) + (int64_t)t.page * c.H + head;
  // tokens lo .. hi - 1 of the page are new; those before are earlier ones
  const int lo = t.lo - t.begin, hi = t.hi - t.begin;
  const float before = lo > 0 ? *scale_at : 0.f;
  // row of the call that page token 0 would be
  const int64_t row0 = (int64_t)t.rows.first + (t.begin - (t.rows.len - t.rows.n));

  // items: quad of tokens by eight elements, from the first new token's quad on
  const int first_quad = lo / 4, items = ((hi + 3) / 4 - first_quad) * chunks;
  Raw8 raw[Q][4];
  int tok[Q], el[Q];
  auto load = [&](int first) {
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int at = first + (int)threadIdx.x + i * THREADS;
      const int in = at < items ? at : 0;
      tok[i] = (first_quad + in / chunks) * 4;
      el[i] = in % chunks * 8;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = tok[i] + j;
        raw[i][j] =
            load8(x, (row0 + (k < lo ? lo : k >= hi ? hi - 1 : k)) * x_row + x_at + el[i], f32);
      }
    }
  };
  uint32_t top = 0;
  for (int first = 0; first < items; first += Q * THREADS) {
    load(first);
#pragma unroll
    for (int i = 0; i < Q; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[8];
        values8(raw[i][j], f32, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t b = __builtin_bit_cast(uint32_t, v[e]) & 0x7fffffffu;
          top = b > top ? b : top;   // repeated tokens change nothing
        }
      }
  }
  top = wave_umax(top);
  if ((threadIdx.x & (kWave - 1)) == 0) tops[threadIdx.x / kWave] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / kWave; ++w) top = tops[w] > top ? tops[w] : top;
  float now = top < 0x7f800000u ? __builtin_bit_cast(float, top) / (e4m3 ? 448.f : 127.f)
                                : __builtin_nanf("");
  if (lo > 0) now = before != before ? before : before > now ? before : now;
  const Levels levels(now, e4m3);
  const bool grown = lo > 0 && now > before;   // not where it is NaN
  const float ratio = grown ? before / now : 1.f;
  const bool one = hi - lo == 1;   // token: it needs no detour
  if (threadIdx.x == 0) *scale_at = now;

  for (int first = 0; first < items; first += Q * THREADS) {
    if (items > Q * THREADS) load(first);
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      if (first + (int)threadIdx.x + i * THREADS >= items) break;
      uint32_t q[4][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[8];
        values8(raw[i][j], f32, v);
        q[j][0] = levels.of(v[0], v[1], v[2], v[3]);
        q[j][1] = levels.of(v[4], v[5], v[6], v[7]);
      }
      if (!values) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = tok[i] + j;
          const ops_u32x2 w = {q[j][0], q[j][1]};
          if (k < lo || k >= hi) continue;
          if (one)
            *reinterpret_cast<ops_u32x2*>(out + (el[i] / 16 * LOWM_PAGE + k) * 16 + el[i] % 16) = w;
          else
            *reinterpret_cast<ops_u32x2*>(&turn[key_words(el[i] / 16, k) + el[i] % 16 / 4]) = w;
        }
      } else if (!grown && one) {
        // one more token of a page that keeps its scale: a byte an element
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint8_t b = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (tok[i] + j == lo) b = (uint8_t)(q[j][e / 4] >> 8 * (e % 4));
          out[(lo / 16 * D + el[i] + e) * 16 + lo % 16] = b;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint32_t w = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) w |= (q[j][e / 4] >> 8 * (e % 4) & 255u) << 8 * j;
          turn[turned(D, tok[i] / 16, el[i] + e) + tok[i] % 16 / 4] = w;
        }
      }
    }
  }
  if (!grown && one) return;

  ops_u32x4* pieces = reinterpret_cast<ops_u32x4*>(out);
  if (!values) {
    if (grown) {
      // earlier tokens of the keys: a piece each
      for (int at = threadIdx.x; at < D / 16 * lo; at += THREADS) {
        const int p = at / lo * LOWM_PAGE + at % lo;
        ops_u32x4 w = pieces[p];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = again4(w[i], e4m3, ratio);
        pieces[p] = w;
      }
    }
    if (one) return;
    __syncthreads();
    for (int at = threadIdx.x; at < D / 16 * LOWM_PAGE; at += THREADS) {
      const int chunk = at / LOWM_PAGE, k = at % LOWM_PAGE;
      if (k >= lo && k < hi) pieces[at] = *reinterpret_cast<ops_u32x4*>(&turn[key_words(chunk, k)]);
    }
    return;
  }
  __syncthreads();
  // pieces of the values: whole ones are written, others are merged
  const int first = grown ? 0 : lo / 16;
  for (int at = threadIdx.x; at < ((hi + 15) / 16 - first) * D; at += THREADS) {
    const int g = first + at / D, d = at % D;
    const int from = lo - 16 * g, to = hi - 16 * g;   // new tokens of the piece
    ops_u32x4 w = {0u, 0u, 0u, 0u};
    if (from > 0 || to < 16) w = pieces[g * D + d];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // bytes of this word: earlier ones below a, new ones below b, others above
      const int a = from - 4 * i < 0 ? 0 : from - 4 * i > 4 ? 4 : from - 4 * i;
      const int b = to - 4 * i < 0 ? 0 : to - 4 * i > 4 ? 4 : to - 4 * i;
      const uint32_t old_mask = (uint32_t)((1ull << 8 * a) - 1),
                     put_mask = (uint32_t)((1ull << 8 * b) - 1) & ~old_mask;
      uint32_t v = w[i];
      if (grown && old_mask) v = (again4(v, e4m3, ratio) & old_mask) | (v & ~old_mask);
      if (put_mask) v = (turn[turned(D, g, d) + i] & put_mask) | (v & ~put_mask);
      w[i] = v;
    }
    pieces[g * D + d] = w;
  }
}

struct ReadArgs {
  lowm_cache_read_args u;
  int uniform_pages;
  int first_item;
};

template <int THREADS>
__global__ __launch_bounds__(THREADS) void read_kernel(ReadArgs a) {
  const lowm_cache_read_args& u = a.u;
  const lowm_kv_cache& c = u.cache;
  extern __shared__ __align__(16) uint32_t turn[];
  const Touched t = page_of(u.seq, c.P, a.first_item + (int)blockIdx.x, a.uniform_pages);
  if (t.page < 0) return;
  const int head = blockIdx.y, D = c.D, chunks = D / 8;
  const bool values = blockIdx.z, e4m3 = c.type == LOWM_E4M3;
  const uint8_t* in =
      static_cast<const uint8_t*>(values ? c.v : c.k) + page_offset(c, t.page, head);
  const float scale = (values ? c.v_scale : c.k_scale)[(int64_t)t.page * c.H + head];
  const int lo = t.lo - t.begin, hi = t.hi - t.begin;
  const int64_t row0 = (int64_t)t.rows.first + (t.begin - (t.rows.len - t.rows.n));
  void* out = values ? u.v_out : u.k_out;
  auto store = [&](int k, int d, uint32_t lo4, uint32_t hi4) {
    float x[8], p[4];
    unpack4(lo4, e4m3, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = p[i] * scale;
    unpack4(hi4, e4m3, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[4 + i] = p[i] * scale;
    store8(out, ((row0 + k) * c.H + head) * D + d, false, x);
  };
  // several loads at a time: a loop's next load would wait for the store before it
  constexpr int kAhead = 4;
  if (!values) {
    const int items = (hi - lo) * chunks;
    for (int first = threadIdx.x; first < items; first += kAhead * THREADS) {
      ops_u32x2 w[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int at = first + i * THREADS < items ? first + i * THREADS : first;
        const int k = lo + at / chunks, d = at % chunks * 8;
        w[i] = *reinterpret_cast<const ops_u32x2*>(in + (d / 16 * LOWM_PAGE + k) * 16 + d % 16);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int at = first + i * THREADS;
        if (at < items) store(lo + at / chunks, at % chunks * 8, w[i][0], w[i][1]);
      }
    }
    return;
  }
  const ops_u32x4* pieces = reinterpret_cast<const ops_u32x4*>(in);
  const int first_piece = lo / 16 * D, all = (hi + 15) / 16 * D;
  for (int first = first_piece + threadIdx.x; first < all; first += kAhead * THREADS) {
    ops_u32x4 w[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      w[i] = pieces[first + i * THREADS < all ? first + i * THREADS : first];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = first + i * THREADS;
      if (at < all) *reinterpret_cast<ops_u32x4*>(&turn[turned(D, at / D, at % D)]) = w[i];
    }
  }
  __syncthreads();
  const int first_quad = lo / 4, items = ((hi + 3) / 4 - first_quad) * chunks;
  for (int at = threadIdx.x; at < items; at += THREADS) {
    const int k = (first_quad + at / chunks) * 4, d = at % chunks * 8;
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = turn[turned(D, k / 16, d + e) + k % 16 / 4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (k + j < lo || k + j >= hi) continue;
      uint32_t lo4 = 0, hi4 = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo4 |= (w[e] >> 8 * j & 255u) << 8 * e;
        hi4 |= (w[4 + e] >> 8 * j & 255u) << 8 * e;
      }
      store(k + j, d, lo4, hi4);
    }
  }
}

// Page-by-head workgroups, keys and values: no more pages than rows, and no more
// than the rows fill with two more for each sequence.  `one`: of a wavefront, for up to
// two rows a sequence on average; `four`: of four.
template <typename A>
int launch_pages(const void* one, const void* four, A a, const lowm_sequences& s,
                 const lowm_kv_cache& c, hipStream_t stream) {
  int64_t items;
  if (!s.row_starts) {
    const int n = s.T / s.B;
    a.uniform_pages = (n + LOWM_PAGE - 2) / LOWM_PAGE + 1;
    if (a.uniform_pages > n) a.uniform_pages = n;
    items = (int64_t)a.uniform_pages * s.B;
  } else {
    a.uniform_pages = 0;
    items = (int64_t)s.T / LOWM_PAGE + 2 * (int64_t)s.B;
    if (items > s.T) items = s.T;
  }
  const bool few = s.T <= 2 * (int64_t)s.B;
  const int threads = few ? kWave : 4 * kWave;
  const int64_t most = kMaxThreads / threads / (2 * c.H);
  void* args[] = {&a};
  int rc = LOWM_OK;
  for (int64_t i = 0; i < items && rc == LOWM_OK; i += most) {
    a.first_item = (int)i;
    rc = launched(hipLaunchKernel(few ? one : four,
                                  dim3((unsigned)(items - i < most ? items - i : most),
                                       (unsigned)c.H, 2),
                                  dim3(threads), args, 4 * turned_words(c.D), stream));
  }
  return rc;
}

int cache_append(const lowm_cache_append_args* u, hipStream_t stream) {
  if (!u) return LOWM_ERR_INVALID_ARG;
  int rc = check_sequences(u->seq);
  if (rc == LOWM_OK) rc = check_cache(u->cache);
  if (rc != LOWM_OK) return rc;
  if (u->cache.layers != 1 || (u->type != LOWM_BF16 && u->type != LOWM_F32))
    return LOWM_ERR_INVALID_ARG;
  if (u->seq.T == 0) return LOWM_OK;
  if (!u->k || !u->v) return LOWM_ERR_INVALID_ARG;
  const lowm_kv_cache& c = u->cache;
  const int b = type_bytes(u->type);
  const int64_t T = u->seq.T;
  if (!aligned_to(u->k, b) || !aligned_to(u->v, b)) return LOWM_ERR_UNSUPPORTED;
  if (!heads_apart(T, c.H, c.D, u->k_row, u->k_head) ||
      !heads_apart(T, c.H, c.D, u->v_row, u->v_head))
    return LOWM_ERR_INVALID_ARG;
  const CacheSpans cs(c);
  const SequenceSpans ss(u->seq);
  if (!cs.apart()) return LOWM_ERR_INVALID_ARG;
  for (const Span& x : {span_of(Heads{u->k, T, c.H, c.D, u->k_row, u->k_head, b}),
                        span_of(Heads{u->v, T, c.H, c.D, u->v_row, u->v_head, b})})
    if (cs.meets(x)) return LOWM_ERR_INVALID_ARG;
  for (const Span& x : cs.s)
    if (ss.meets(x)) return LOWM_ERR_INVALID_ARG;
  return launch_pages((const void*)&append_kernel<1, kWave>,
                      c.D > 128 ? (const void*)&append_kernel<2, 4 * kWave>
                                : (const void*)&append_kernel<1, 4 * kWave>,
                      AppendArgs{*u, 0, 0}, u->seq, c, stream);
}

int cache_read(const lowm_cache_read_args* u, hipStream_t stream) {
  if (!u) return LOWM_ERR_INVALID_ARG;
  int rc = check_sequences(u->seq);
  if (rc == LOWM_OK) rc = check_cache(u->cache);
  if (rc != LOWM_OK) return rc;
  if (u->cache.layers != 1) return LOWM_ERR_INVALID_ARG;
  if (u->seq.T == 0) return LOWM_OK;
  if (!u->k_out || !u->v_out) return LOWM_ERR_INVALID_ARG;
  if (!aligned_to(u->k_out, 2) || !aligned_to(u->v_out, 2)) return LOWM_ERR_UNSUPPORTED;
  const lowm_kv_cache& c = u->cache;
  const int64_t n = (int64_t)u->seq.T * c.H * c.D;
  const Span k = plain_span(u->k_out, n, 2), v = plain_span(u->v_out, n, 2);
  const CacheSpans cs(c);
  const SequenceSpans ss(u->seq);
  if (meet(k, v) || cs.meets(k) || cs.meets(v) || ss.meets(k) || ss.meets(v))
    return LOWM_ERR_INVALID_ARG;
  return launch_pages((const void*)&read_kernel<kWave>, (const void*)&read_kernel<4 * kWave>,
                      ReadArgs{*u, 0, 0}, u->seq, c, stream);
}

}  // namespace
}  // namespace lowm

extern "C" {

int lowm_cache_append(const lowm_cache_append_args* args, void* stream) {
  return lowm::cache_append(args, static_cast<hipStream_t>(stream));
}

int lowm_cache_read(const lowm_cache_read_args* args, void* stream) {
  return lowm::cache_read(args, static_cast<hipStream_t>(stream));
}

}  // extern "C"
