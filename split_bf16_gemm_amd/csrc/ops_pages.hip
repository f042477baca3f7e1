// ops_pages.hip -- the pages of a cache: forking, freeing and reserving
// (lowm_fork_pages), compacting (lowm_compact_pages) and the copying of both, for
// gfx950.
//
// Whole numbers and copies.  Counting how often each page is used goes over the
// table with one atomic addition an entry, whose order does not matter; which page
// goes where is decided by one workgroup, from prefix sums over the rows and over
// the pages in ascending order, so that the same tables give the same pages.  Small
// tables go through that workgroup whole, with the counts in LDS, instead of three
// launches (8 rows: 14.6 us, 8.2 so).  Then all workgroups copy: a page of a layer is one
// run of bytes for the keys and one for the values, in units of kUnit bytes, past the caches
// (355 pages of 786 KB 118 us, 4.75 TB/s, 127 through them; 110 to 123 with the deciding).
#include "ops_cache.cuh"

namespace lowm {
namespace {

constexpr int kOne = 1024;            // threads of the workgroup that decides
constexpr int kWaves = kOne / kWave;
constexpr int kPer = 4;               // pages, or rows, to a thread and step
constexpr int kSmallP = 4096;         // pages whose counts fit its LDS,
constexpr int kSmallEntries = 16384;  // and entries of a table that it goes through alone
constexpr int kUnit = 16384;          // bytes copied by a workgroup at a time

// The workspace: 32-bit words.
struct Scratch {
  int* count;      // [4] copies to make
  int* owner;      // [P] lowest row whose unfinished page it is; where a page moves
  int* parts;      // [P] rows whose unfinished page it is
  int* list;       // [P] free pages in order
  int* src;        // [max(R, P / 2 + 1)]
  int* dst;
  int* wants;      // [R]
};
inline int64_t pair_room(int R, int P) { return R > P / 2 + 1 ? R : P / 2 + 1; }
inline size_t scratch_bytes(int R, int P) {
  return 4 * (size_t)(4 + 3 * (int64_t)P + 2 * pair_room(R, P) + R);
}
inline Scratch scratch_of(void* w, int R, int P) {
  int* p = static_cast<int*>(w);
  Scratch s;
  s.count = p;
  s.owner = s.count + 4;
  s.parts = s.owner + P;
  s.list = s.parts + P;
  s.src = s.list + P;
  s.dst = s.src + pair_room(R, P);
  s.wants = s.dst + pair_room(R, P);
  return s;
}

struct PagesArgs {
  lowm_kv_cache cache;
  Scratch w;
  const int* table;
  const int* lens;
  const int* parents;
  const int* held;
  int* table_out;
  int* lens_out;
  int* refs;
  int* result;       // missing [1], or moved and top [2]
  int R, W, reserve;
};

__device__ __forceinline__ int pages_for(int64_t tokens) {
  return (int)((tokens + LOWM_PAGE - 1) / LOWM_PAGE);
}
__device__ __forceinline__ int held_of(const PagesArgs& a, int p) {
  return a.held && a.held[p] > 0 ? a.held[p] : 0;
}

// Uses of each page, and for forking who has it as an unfinished last page: in the
// workspace and refs_out, or in LDS.
struct Counts {
  int *refs, *owner, *parts;
};
__device__ __forceinline__ void begin_page(const PagesArgs& a, const Counts& n, int p) {
  n.refs[p] = held_of(a, p);
  n.owner[p] = a.lens ? INT32_MAX : p;
  n.parts[p] = 0;
}
__global__ __launch_bounds__(256) void pages_begin_kernel(PagesArgs a) {
  const Counts n{a.refs, a.w.owner, a.w.parts};
  for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < a.cache.P;
       p += (int64_t)gridDim.x * 256)
    begin_page(a, n, (int)p);
}

// Whose pages row r takes, and how many tokens: what goes on with none, and what
// ends, has no pages.
struct Heir {
  int parent, len, pages;
  bool on;
  __device__ __forceinline__ Heir(const PagesArgs& a, int r) {
    parent = a.parents ? a.parents[r] : r;
    on = parent >= 0 && parent < a.R;
    len = on ? a.lens[parent] : 0;
    if (len < 0) len = 0;
    pages = pages_for(len);
    if (pages > a.W) {       // the table has no more: nor has the row
      pages = a.W;
      len = a.W * LOWM_PAGE;
    }
  }
};

// Entry w of row r.
__device__ __forceinline__ void fork_entry(const PagesArgs& a, const Counts& n, const Heir& h,
                                           int r, int w) {
  int page = -1;
  if (w < h.pages) {
    page = a.table[(int64_t)h.parent * a.W + w];
    if (page < 0 || page >= a.cache.P) page = -1;
  }
  a.table_out[(int64_t)r * a.W + w] = page;
  if (page >= 0) {
    atomicAdd(&n.refs[page], 1);
    if (w == h.pages - 1 && h.len % LOWM_PAGE) {
      atomicAdd(&n.parts[page], 1);
      atomicMin(&n.owner[page], r);
    }
  }
}
// A workgroup to a row and a stretch of its entries.
__global__ __launch_bounds__(256) void fork_rows_kernel(PagesArgs a) {
  const int r = blockIdx.x;
  const Heir h(a, r);
  const Counts n{a.refs, a.w.owner, a.w.parts};
  for (int w = blockIdx.y * 256 + threadIdx.x; w < a.W; w += gridDim.y * 256)
    fork_entry(a, n, h, r, w);
  if (blockIdx.y == 0 && threadIdx.x == 0) a.lens_out[r] = h.len;
}

__device__ __forceinline__ void count_entry(const PagesArgs& a, const Counts& n, int64_t i) {
  const int page = a.table[i];
  if (page >= 0 && page < a.cache.P) atomicAdd(&n.refs[page], 1);
}
__global__ __launch_bounds__(256) void count_kernel(PagesArgs a) {
  const int64_t entries = (int64_t)a.R * a.W;
  const Counts n{a.refs, a.w.owner, a.w.parts};
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < entries;
       i += (int64_t)gridDim.x * 256)
    count_entry(a, n, i);
}

// Inclusive sums over the deciding workgroup, and the sum of all.
struct GroupScan {
  int* lds;    // [2][kWaves]
  int turn = 0;
  __device__ __forceinline__ int operator()(int v, int* total) {
    const int s = wave_scan(v), wave = threadIdx.x / kWave;
    int* slot = lds + turn * kWaves;
    turn ^= 1;   // a slot is written again only after the next scan's barrier
    if ((threadIdx.x & (kWave - 1)) == kWave - 1) slot[wave] = s;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int n = slot[w];
      before += w < wave ? n : 0;
      all += n;
    }
    *total = all;
    return before + s;
  }
};

__device__ void fork_decide(const PagesArgs& a, const Counts& c) {
  __shared__ int lds[2 * kWaves];
  __shared__ int sums[3];   // copies made, pages missing, others that a row cannot have
  GroupScan scan{lds};
  if (threadIdx.x < 3) sums[threadIdx.x] = 0;
  __syncthreads();

  // what each row asks for: a copy of its last page (bit 0), and further pages
  const int P = a.cache.P;
  int asked = 0;
  for (int r0 = 0; r0 < a.R; r0 += kOne) {
    const int r = r0 + (int)threadIdx.x;
    int n = 0;
    if (r < a.R) {
      const Heir h(a, r);
      int copy = 0, more = 0;
      if (h.len % LOWM_PAGE) {
        const int page = a.table_out[(int64_t)r * a.W + h.pages - 1];
        copy = page >= 0 && !(c.owner[page] == r && c.refs[page] == c.parts[page]);
        // nothing holds the tokens that it should have: a new page would show others
        if (page < 0) atomicAdd(&sums[2], 1);
      }
      if (h.on) {
        const int want = pages_for((int64_t)h.len + a.reserve);
        more = (want < a.W ? want : a.W) - h.pages;
        if (want > a.W) atomicAdd(&sums[2], want - a.W);
      }
      n = copy + more;
      a.w.wants[r] = copy | more << 1;
    }
    int total;
    scan(n, &total);
    asked += total;
  }

  // the lowest free pages, in order
  int found = 0;
  for (int64_t p0 = 0; p0 < P && found < asked; p0 += kOne * kPer) {
    const int64_t p = p0 + (int64_t)threadIdx.x * kPer;
    bool free[kPer];
    int n = 0, total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      free[i] = p + i < P && c.refs[p + i] == 0;
      n += free[i];
    }
    int at = found + scan(n, &total) - n;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (free[i]) a.w.list[at++] = (int)p + i;
    found += total;
  }
  __syncthreads();

  // who gets them
  int given = 0;
  for (int r0 = 0; r0 < a.R; r0 += kOne) {
    const int r = r0 + (int)threadIdx.x;
    const int wants = r < a.R ? a.w.wants[r] : 0, copy = wants & 1, more = wants >> 1;
    int total;
    int at = given + scan(copy + more, &total) - copy - more;
    given += total;
    if (!wants) continue;
    const Heir h(a, r);
    int* row = a.table_out + (int64_t)r * a.W;
    int missing = 0;
    if (copy) {
      const int old = row[h.pages - 1], page = at < found ? a.w.list[at] : -1;
      atomicSub(&c.refs[old], 1);
      row[h.pages - 1] = page;
      if (page >= 0) {
        atomicAdd(&c.refs[page], 1);
        const int k = atomicAdd(&sums[0], 1);
        a.w.src[k] = old;
        a.w.dst[k] = page;
      } else {
        ++missing;
      }
      ++at;
    }
    for (int i = 0; i < more; ++i, ++at) {
      const int page = at < found ? a.w.list[at] : -1;
      row[h.pages + i] = page;
      if (page >= 0)
        atomicAdd(&c.refs[page], 1);
      else
        ++missing;
    }
    if (missing) atomicAdd(&sums[1], missing);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    a.w.count[0] = sums[0];
    a.result[0] = sums[1] + sums[2];
  }
}
__global__ __launch_bounds__(kOne) void fork_decide_kernel(PagesArgs a) {
  fork_decide(a, Counts{a.refs, a.w.owner, a.w.parts});
}
// All of it but the copies, for tables and caches that the workgroup's LDS holds.
__global__ __launch_bounds__(kOne) void fork_small_kernel(PagesArgs a) {
  __shared__ int refs[kSmallP], owner[kSmallP], parts[kSmallP];
  const Counts n{refs, owner, parts};
  for (int p = threadIdx.x; p < a.cache.P; p += kOne) begin_page(a, n, p);
  __syncthreads();
  for (int i = threadIdx.x; i < a.R * a.W; i += kOne) {
    const int r = i / a.W, w = i - r * a.W;
    const Heir h(a, r);
    fork_entry(a, n, h, r, w);
    if (w == 0) a.lens_out[r] = h.len;
  }
  __syncthreads();
  fork_decide(a, n);
  __syncthreads();
  for (int p = threadIdx.x; p < a.cache.P; p += kOne) a.refs[p] = refs[p];
}

// The i-th lowest free page takes the i-th highest movable one while that is higher:
// a free page p, the i-th, is taken if more than i movable ones lie above it, and a
// movable one moves if more free ones lie below it than movable ones above.
__device__ void compact_decide(const PagesArgs& a, const Counts& c) {
  __shared__ int lds[2 * kWaves];
  __shared__ int top;
  GroupScan scan{lds};
  if (threadIdx.x == 0) top = 0;
  const int P = a.cache.P;
  auto movable = [&](int64_t p) { return c.refs[p] > 0 && held_of(a, (int)p) == 0; };
  int count = 0;
  for (int64_t p = threadIdx.x; p < P; p += kOne) count += movable(p);
  int all;
  scan(count, &all);

  int free_before = 0, movable_before = 0, moved = 0, highest = 0;
  for (int64_t p0 = 0; p0 < P; p0 += kOne * kPer) {
    const int64_t p = p0 + (int64_t)threadIdx.x * kPer;
    int kind[kPer];   // 1: free, 2: movable, 0: held, or past the end
    int nf = 0, nm = 0, tf, tm;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      kind[i] = p + i >= P ? 0 : c.refs[p + i] == 0 ? 1 : movable(p + i) ? 2 : 0;
      if (kind[i] == 0 && p + i < P) highest = (int)p + i + 1;
      nf += kind[i] == 1;
      nm += kind[i] == 2;
    }
    int f = free_before + scan(nf, &tf) - nf, m = movable_before + scan(nm, &tm) - nm;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (kind[i] == 1) {
        if (all - m > f) {
          a.w.dst[f] = (int)p + i;
          highest = (int)p + i + 1;
        }
        ++f;
      } else if (kind[i] == 2) {
        const int above = all - ++m;
        if (f > above) {
          a.w.src[above] = (int)p + i;
          ++moved;
        } else {
          highest = (int)p + i + 1;
        }
      }
    }
    free_before += tf;
    movable_before += tm;
  }
  int pairs;
  scan(moved, &pairs);   // its barrier is behind every store of a pair
  for (int i = threadIdx.x; i < pairs; i += kOne) {
    const int s = a.w.src[i], d = a.w.dst[i];
    c.refs[d] = c.refs[s];
    c.refs[s] = 0;
    c.owner[s] = d;
  }
  atomicMax(&top, highest);
  __syncthreads();
  if (threadIdx.x == 0) {
    a.w.count[0] = pairs;
    a.result[0] = pairs;
    a.result[1] = top;
  }
}
__global__ __launch_bounds__(kOne) void compact_decide_kernel(PagesArgs a) {
  compact_decide(a, Counts{a.refs, a.w.owner, a.w.parts});
}
__global__ __launch_bounds__(kOne) void compact_small_kernel(PagesArgs a) {
  __shared__ int refs[kSmallP], owner[kSmallP], parts[kSmallP];
  const Counts n{refs, owner, parts};
  for (int p = threadIdx.x; p < a.cache.P; p += kOne) begin_page(a, n, p);
  __syncthreads();
  for (int i = threadIdx.x; i < a.R * a.W; i += kOne) count_entry(a, n, i);
  __syncthreads();
  compact_decide(a, n);
  for (int p = threadIdx.x; p < a.cache.P; p += kOne) {
    a.refs[p] = refs[p];
    a.w.owner[p] = owner[p];
  }
}

// The copies, and where compacting made them, the table's new numbers.
__global__ __launch_bounds__(256) void copy_pages_kernel(PagesArgs a, bool renumber) {
  const lowm_kv_cache& c = a.cache;
  if (renumber) {
    const int64_t n = (int64_t)a.R * a.W;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * 256) {
      const int page = a.table[i];
      a.table_out[i] = page >= 0 && page < c.P ? a.w.owner[page] : -1;
    }
  }
  const int64_t bytes = (int64_t)c.H * c.D * LOWM_PAGE;
  const int units = (int)((bytes + kUnit - 1) / kUnit);
  const int64_t all = (int64_t)a.w.count[0] * c.layers * 2 * units;
  for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
    const int unit = (int)(i % units);
    int64_t rest = i / units;
    const bool values = rest & 1;
    rest >>= 1;
    const int layer = (int)(rest % c.layers), pair = (int)(rest / c.layers);
    const int64_t from = (int64_t)layer * c.P + a.w.src[pair],
                  to = (int64_t)layer * c.P + a.w.dst[pair];
    uint8_t* p = static_cast<uint8_t*>(values ? c.v : c.k);
    const int64_t at = (int64_t)unit * kUnit;
    const int64_t left = bytes - at < kUnit ? bytes - at : kUnit;
    const ops_u32x4* x = reinterpret_cast<const ops_u32x4*>(p + from * bytes + at);
    ops_u32x4* y = reinterpret_cast<ops_u32x4*>(p + to * bytes + at);
    ops_u32x4 v[kUnit / 4096];
#pragma unroll
    for (int k = 0; k < kUnit / 4096; ++k) {
      const int e = k * 256 + (int)threadIdx.x;
      v[k] = __builtin_nontemporal_load(x + (e * 16 < left ? e : 0));
    }
#pragma unroll
    for (int k = 0; k < kUnit / 4096; ++k) {
      const int e = k * 256 + (int)threadIdx.x;
      if (e * 16 < left) __builtin_nontemporal_store(v[k], y + e);
    }
    if (unit == 0) {
      float* s = values ? c.v_scale : c.k_scale;
      for (int h = threadIdx.x; h < c.H; h += 256) s[to * c.H + h] = s[from * c.H + h];
    }
  }
}

int launch(const void* fn, dim3 grid, int threads, PagesArgs a, bool renumber,
           hipStream_t stream) {
  void* args[] = {&a, &renumber};
  return launched(hipLaunchKernel(fn, grid, dim3(threads), args, 0, stream));
}
unsigned blocks_for(int64_t n, int64_t per, int64_t most) {
  const int64_t b = (n + per - 1) / per;
  return (unsigned)(b < 1 ? 1 : b > most ? most : b);
}
bool is_small(int P, int64_t entries) { return P <= kSmallP && entries <= kSmallEntries; }
int launch_copies(const PagesArgs& a, int64_t pairs, bool renumber, hipStream_t stream) {
  const lowm_kv_cache& c = a.cache;
  const int64_t units = ((int64_t)c.H * c.D * LOWM_PAGE + kUnit - 1) / kUnit;
  const int64_t work = pairs * c.layers * 2 * units;
  return launch((const void*)&copy_pages_kernel, dim3(blocks_for(work, 1, 2048)), 256, a, renumber,
                stream);
}

int check_pages(const lowm_kv_cache& c, int R, int W, const void* table, const void* held,
                const void* table_out, const void* refs, const void* result) {
  if (R < 1 || W < 1) return LOWM_ERR_INVALID_ARG;
  const int rc = check_cache(c);
  if (rc != LOWM_OK) return rc;
  if (R > LOWM_PAGES_MAX_R || W > LOWM_PAGES_MAX_W || c.P > LOWM_PAGES_MAX_P)
    return LOWM_ERR_UNSUPPORTED;
  if (!table || !table_out || !refs || !result) return LOWM_ERR_INVALID_ARG;
  for (const void* p : {table, held, table_out, refs, result})
    if (!aligned_to(p, 4)) return LOWM_ERR_UNSUPPORTED;
  return LOWM_OK;
}
int check_workspace(const void* w, size_t bytes, int R, int P) {
  if (!w || bytes < scratch_bytes(R, P)) return LOWM_ERR_WORKSPACE;
  return aligned_to(w, 256) ? LOWM_OK : LOWM_ERR_UNSUPPORTED;
}
// No output over another, an input or the cache.
int check_apart(const CacheSpans& cache, const Span* in, int n_in, const Span* out, int n_out) {
  if (!cache.apart()) return LOWM_ERR_INVALID_ARG;
  for (int i = 0; i < n_in; ++i)
    if (cache.meets(in[i])) return LOWM_ERR_INVALID_ARG;
  for (int o = 0; o < n_out; ++o) {
    if (cache.meets(out[o])) return LOWM_ERR_INVALID_ARG;
    for (int i = 0; i < n_in; ++i)
      if (meet(out[o], in[i])) return LOWM_ERR_INVALID_ARG;
    for (int i = 0; i < o; ++i)
      if (meet(out[o], out[i])) return LOWM_ERR_INVALID_ARG;
  }
  return LOWM_OK;
}

int fork_pages(const lowm_fork_pages_args* u, hipStream_t stream) {
  if (!u) return LOWM_ERR_INVALID_ARG;
  const lowm_kv_cache& c = u->cache;
  int rc = check_pages(c, u->R, u->W, u->table, u->held, u->table_out, u->refs_out, u->missing_out);
  if (rc != LOWM_OK) return rc;
  if (!u->lens || !u->lens_out || u->reserve < 0) return LOWM_ERR_INVALID_ARG;
  if (!aligned_to(u->lens, 4) || !aligned_to(u->lens_out, 4) || !aligned_to(u->parents, 4) ||
      u->reserve > LOWM_PAGES_MAX_W * LOWM_PAGE)
    return LOWM_ERR_UNSUPPORTED;
  rc = check_workspace(u->workspace, u->workspace_bytes, u->R, c.P);
  if (rc != LOWM_OK) return rc;
  const int64_t n = (int64_t)u->R * u->W;
  const Span in[] = {plain_span(u->table, n, 4), plain_span(u->lens, u->R, 4),
                     plain_span(u->parents, u->R, 4), plain_span(u->held, c.P, 4)};
  const Span out[] = {plain_span(u->table_out, n, 4), plain_span(u->lens_out, u->R, 4),
                      plain_span(u->refs_out, c.P, 4), plain_span(u->missing_out, 1, 4),
                      plain_span(u->workspace, (int64_t)scratch_bytes(u->R, c.P), 1)};
  rc = check_apart(CacheSpans(c), in, 4, out, 5);
  if (rc != LOWM_OK) return rc;
  PagesArgs a{};
  a.cache = c;
  a.w = scratch_of(u->workspace, u->R, c.P);
  a.table = u->table;
  a.lens = u->lens;
  a.parents = u->parents;
  a.held = u->held;
  a.table_out = u->table_out;
  a.lens_out = u->lens_out;
  a.refs = u->refs_out;
  a.result = u->missing_out;
  a.R = u->R;
  a.W = u->W;
  a.reserve = u->reserve;
  if (is_small(c.P, n)) {
    rc = launch((const void*)&fork_small_kernel, dim3(1), kOne, a, false, stream);
    return rc == LOWM_OK ? launch_copies(a, u->R, false, stream) : rc;
  }
  rc = launch((const void*)&pages_begin_kernel, dim3(blocks_for(c.P, 256, 1024)), 256, a, false,
              stream);
  if (rc == LOWM_OK)
    rc = launch((const void*)&fork_rows_kernel, dim3(u->R, blocks_for(u->W, 1024, 64)), 256, a,
                false, stream);
  if (rc == LOWM_OK)
    rc = launch((const void*)&fork_decide_kernel, dim3(1), kOne, a, false, stream);
  return rc == LOWM_OK ? launch_copies(a, u->R, false, stream) : rc;
}

int compact_pages(const lowm_compact_pages_args* u, hipStream_t stream) {
  if (!u) return LOWM_ERR_INVALID_ARG;
  const lowm_kv_cache& c = u->cache;
  int rc = check_pages(c, u->R, u->W, u->table, u->held, u->table_out, u->refs_out, u->counts_out);
  if (rc != LOWM_OK) return rc;
  rc = check_workspace(u->workspace, u->workspace_bytes, u->R, c.P);
  if (rc != LOWM_OK) return rc;
  const int64_t n = (int64_t)u->R * u->W;
  const Span in[] = {plain_span(u->table, n, 4), plain_span(u->held, c.P, 4)};
  const Span out[] = {plain_span(u->table_out, n, 4), plain_span(u->refs_out, c.P, 4),
                      plain_span(u->counts_out, 2, 4),
                      plain_span(u->workspace, (int64_t)scratch_bytes(u->R, c.P), 1)};
  rc = check_apart(CacheSpans(c), in, 2, out, 4);
  if (rc != LOWM_OK) return rc;
  PagesArgs a{};
  a.cache = c;
  a.w = scratch_of(u->workspace, u->R, c.P);
  a.table = u->table;
  a.held = u->held;
  a.table_out = u->table_out;
  a.refs = u->refs_out;
  a.result = u->counts_out;
  a.R = u->R;
  a.W = u->W;
  const int64_t most = n < c.P / 2 + 1 ? n : c.P / 2 + 1;
  if (is_small(c.P, n)) {
    rc = launch((const void*)&compact_small_kernel, dim3(1), kOne, a, false, stream);
    return rc == LOWM_OK ? launch_copies(a, most, true, stream) : rc;
  }
  rc = launch((const void*)&pages_begin_kernel, dim3(blocks_for(c.P, 256, 1024)), 256, a, false,
              stream);
  if (rc == LOWM_OK)
    rc = launch((const void*)&count_kernel, dim3(blocks_for(n, 1024, 1024)), 256, a, false, stream);
  if (rc == LOWM_OK)
    rc = launch((const void*)&compact_decide_kernel, dim3(1), kOne, a, false, stream);
  return rc == LOWM_OK ? launch_copies(a, most, true, stream) : rc;
}

}  // namespace
}  // namespace lowm

extern "C" {

size_t lowm_pages_workspace_bytes(int R, int W, int P) {
  if (R < 1 || W < 1 || P < 1 || R > LOWM_PAGES_MAX_R || W > LOWM_PAGES_MAX_W ||
      P > LOWM_PAGES_MAX_P)
    return 0;
  return lowm::scratch_bytes(R, P);
}

int lowm_fork_pages(const lowm_fork_pages_args* args, void* stream) {
  return lowm::fork_pages(args, static_cast<hipStream_t>(stream));
}

int lowm_compact_pages(const lowm_compact_pages_args* args, void* stream) {
  return lowm::compact_pages(args, static_cast<hipStream_t>(stream));
}

}  // extern "C"
