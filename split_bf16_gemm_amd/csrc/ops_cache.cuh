// ops_cache.cuh -- what the operators of include/lowm_cache.h share: the checks of
// their operands, where a sequence's rows stand, and the cache's layout.
#pragma once

#include "lowm_cache.h"
#include "ops_common.cuh"

namespace lowm {

inline bool aligned_to(const void* p, int bytes) {
  return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0;
}

// [T, H, D] elements, each row of D contiguous, row and head strides in elements.
struct Heads {
  const void* p;
  int64_t T, H, D, row, head;
  int bytes;
};
// Whether no two of the (token, head) rows share an element: the smaller stride
// steps over D, the larger over all that the smaller reaches.
inline bool heads_apart(int64_t T, int64_t H, int64_t D, int64_t row, int64_t head) {
  if (row < 0 || head < 0) return false;
  if (T <= 1) return H <= 1 || head >= D;
  if (H <= 1) return row >= D;
  return row >= head ? head >= D && row >= (H - 1) * head + D
                     : row >= D && head >= (T - 1) * row + D;
}
// The bytes they span, as rows of the larger stride where that says more: column
// ranges of one buffer with equal strides do not meet.
inline Span span_of(const Heads& x) {
  if (!x.p) return Span{0, 0, 0, 0};
  const bool by_token = x.T > 1 && (x.H <= 1 || x.row >= x.head);
  const int64_t outer = by_token ? x.T : x.H, inner = by_token ? x.H : x.T,
                big = by_token ? x.row : x.head, small = by_token ? x.head : x.row;
  const int64_t width = (inner - 1) * small + x.D;
  return span_of(x.p, outer, width, outer > 1 ? big : width, x.bytes);
}
inline bool meet(const Heads& a, const Heads& b) { return meet(span_of(a), span_of(b)); }
inline bool meet(const Heads& a, const Span& b) { return meet(span_of(a), b); }

inline Span plain_span(const void* p, int64_t n, int64_t bytes) {
  return span_of(p, 1, n, n, bytes);
}

inline bool cache_type(int t) { return t == LOWM_I8 || t == LOWM_E4M3; }
inline int check_cache(const lowm_kv_cache& c) {
  if (c.P < 1 || c.H < 1 || c.D < 1 || c.layers < 1 || !cache_type(c.type))
    return LOWM_ERR_INVALID_ARG;
  if (c.D % 16 || c.D > LOWM_CACHE_MAX_D || c.H > LOWM_CACHE_MAX_HEADS) return LOWM_ERR_UNSUPPORTED;
  if (!c.k || !c.v || !c.k_scale || !c.v_scale) return LOWM_ERR_INVALID_ARG;
  if (!aligned_to(c.k, 16) || !aligned_to(c.v, 16) || !aligned_to(c.k_scale, 4) ||
      !aligned_to(c.v_scale, 4))
    return LOWM_ERR_UNSUPPORTED;
  return LOWM_OK;
}
struct CacheSpans {
  Span s[4];
  explicit CacheSpans(const lowm_kv_cache& c) {
    const int64_t pages = (int64_t)c.layers * c.P * c.H, bytes = pages * LOWM_PAGE * c.D;
    s[0] = plain_span(c.k, bytes, 1);
    s[1] = plain_span(c.v, bytes, 1);
    s[2] = plain_span(c.k_scale, pages, 4);
    s[3] = plain_span(c.v_scale, pages, 4);
  }
  bool meets(const Span& x) const {
    for (const Span& y : s)
      if (meet(x, y)) return true;
    return false;
  }
  bool apart() const {
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < i; ++j)
        if (meet(s[i], s[j])) return false;
    return true;
  }
};
inline int check_sequences(const lowm_sequences& s) {
  if (s.T < 0 || s.B < 0 || s.W < 0) return LOWM_ERR_INVALID_ARG;
  if (s.B > LOWM_CACHE_MAX_B || s.W > LOWM_PAGES_MAX_W) return LOWM_ERR_UNSUPPORTED;
  if (s.T == 0) return LOWM_OK;
  if (s.B < 1 || s.W < 1 || (s.B > 1 && s.table_ld < s.W)) return LOWM_ERR_INVALID_ARG;
  if (!s.row_starts && s.T % s.B) return LOWM_ERR_INVALID_ARG;
  if (!s.table || !s.lens) return LOWM_ERR_INVALID_ARG;
  if (!aligned_to(s.table, 4) || !aligned_to(s.lens, 4) || !aligned_to(s.row_starts, 4))
    return LOWM_ERR_UNSUPPORTED;
  return LOWM_OK;
}
struct SequenceSpans {
  Span s[3];
  explicit SequenceSpans(const lowm_sequences& q) {
    s[0] = span_of(q.table, q.B, q.W, q.B > 1 ? q.table_ld : q.W, 4);
    s[1] = plain_span(q.lens, q.B, 4);
    s[2] = plain_span(q.row_starts, (int64_t)q.B + 1, 4);
  }
  bool meets(const Span& x) const {
    for (const Span& y : s)
      if (meet(x, y)) return true;
    return false;
  }
};

// A sequence's rows in the call and where they stand.
struct Rows {
  int first, n;      // rows first .. first + n - 1 of the call
  int len;           // tokens of the sequence, up to the last of these rows
  __device__ __forceinline__ int position(int j) const { return len - n + j; }
};
__device__ __forceinline__ Rows rows_of(const lowm_sequences& s, int b) {
  Rows r;
  int past = 0;   // rows behind the call's last: they are left out, each with its token
  if (s.row_starts) {
    int lo = s.row_starts[b], hi = s.row_starts[b + 1];
    past = hi > s.T ? hi - s.T : 0;
    lo = lo < 0 ? 0 : lo > s.T ? s.T : lo;
    hi -= past;
    r.first = lo;
    r.n = hi < lo ? 0 : hi - lo;
  } else {
    r.n = s.T / s.B;
    r.first = b * r.n;
  }
  const int len = s.lens[b];
  r.len = len > past ? len - past : 0;
  return r;
}

// The rows of a sequence that stand on pages of its table, as the positions
// lo .. hi - 1 (none: lo >= hi).
struct Stretch {
  int lo, hi;
  __device__ __forceinline__ explicit Stretch(const lowm_sequences& s, const Rows& r) {
    lo = r.len - r.n > 0 ? r.len - r.n : 0;
    const int64_t most = (int64_t)s.W * LOWM_PAGE;
    hi = r.len < most ? r.len : (int)most;
  }
  __device__ __forceinline__ int pages() const {
    return lo < hi ? (hi - 1) / LOWM_PAGE - lo / LOWM_PAGE + 1 : 0;
  }
};

// Inclusive sums over the wavefront's lanes, all active.
__device__ __forceinline__ int wave_scan(int v) {
  uint32_t x = (uint32_t)v;
  x += lane_move<0x111, 0xf>(x);
  x += lane_move<0x112, 0xf>(x);
  x += lane_move<0x114, 0xf>(x);
  x += lane_move<0x118, 0xf>(x);
  x += lane_move<0x142, 0xa>(x);
  x += lane_move<0x143, 0xc>(x);
  return (int)x;
}

// Bytes of a page's head before its pages' other heads.
__device__ __forceinline__ int64_t page_offset(const lowm_kv_cache& c, int page, int head) {
  return ((int64_t)page * c.H + head) * (LOWM_PAGE * c.D);
}

}  // namespace lowm
