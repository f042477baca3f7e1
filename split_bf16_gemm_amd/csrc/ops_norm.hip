// ops_norm.hip -- the residual norm at a block's border and the row quantiser
// (include/lowm_ops.h) for gfx950.
//
//   p = N(y) w_post ;  r' = a r + b g p ;  x = N(r') w_pre ;  q = rint(x / s)
//
// Each element is read once and written once: a row stays in the registers of
// the group of lanes that owns it (8 elements per lane and step), and its sums
// (the two norms' and, for int8, the largest magnitude) are the only values
// that cross lanes, in fp32.  Bound by HBM for many rows (8 bytes an element
// with bf16 everywhere) and by latency for few: one load's round trip, then a
// reduction per norm.  Measured on MI355X: 16384 rows of 4096 with a gate for every
// element, 671 MB, 115 us (5.8 TB/s; a plain copy reads and writes 5.1 TB/s, and
// part of these rows is still in the caches); one row of 4096 4.0 us, of which an
// empty launch is 1.6; 48 rows of 6144 to int8 6.0 us.  quantize_rows, bf16: 64 rows of
// 4096 3.1 us, 16384 of them 35 (5.7 TB/s), 16384 rows of 12288 122 (5.0 TB/s), 65536
// rows of 512 19 (5.2 TB/s).
//
// Roundings: r' is rounded once, to the residual's type, where it is stored; x comes
// from the unrounded r', which is at hand, and is rounded once, to bf16 or int8.
#include "ops_common.cuh"

namespace lowm {
namespace {

// Centred, twice: two sums a norm; and the largest magnitude.
constexpr int kMaxReductions = 5;

struct NormArgs {
  lowm_residual_norm_args u;
  int64_t first;                         // row of this launch
};

// Sums over the group of G lanes that shares a row.  A group larger than a
// wavefront joins its wavefronts' sums through LDS, each reduction in a slot
// of its own, so one barrier per reduction is enough.
template <int G>
struct Group {
  static constexpr int kWavesPer = G / kWave;
  float* lds;      // [reductions][kWavesPer]
  int at = 0;

  __device__ __forceinline__ float sum(float v) {
    v = wave_sum(v);
    if constexpr (kWavesPer > 1) {
      float* slot = lds + kWavesPer * at++;
      if ((threadIdx.x & (kWave - 1)) == 0) slot[threadIdx.x / kWave] = v;
      __syncthreads();
      v = 0.f;
#pragma unroll
      for (int w = 0; w < kWavesPer; ++w) v += slot[w];
    }
    return v;
  }
  __device__ __forceinline__ uint32_t umax(uint32_t v) {
    v = wave_umax(v);
    if constexpr (kWavesPer > 1) {
      uint32_t* slot = reinterpret_cast<uint32_t*>(lds) + kWavesPer * at++;
      if ((threadIdx.x & (kWave - 1)) == 0) slot[threadIdx.x / kWave] = v;
      __syncthreads();
      v = 0;
#pragma unroll
      for (int w = 0; w < kWavesPer; ++w) v = slot[w] > v ? slot[w] : v;
    }
    return v;
  }
};

// The elements of a row that a lane owns: V runs of 8 consecutive ones, G lanes
// apart.  kRagged: the row ends inside a run; that run's lane reads the row's last
// 8 elements instead and owns those past the run before.  kTiny (fewer than 8
// elements): 8 V single ones, G apart.  Rows may start anywhere.
enum RowKind { kWhole, kRagged, kTiny };

template <int G, int V, RowKind KIND>
struct Row {
  int lane, D;
  __device__ __forceinline__ int start(int v) const { return (v * G + lane) * 8; }
  // Where run v is read; past the row's end the row's first elements are, and
  // dropped (loads under a branch wait for one another).
  __device__ __forceinline__ int base(int v) const {
    const int s = start(v);
    if (KIND == kRagged && s < D) return s + 8 <= D ? s : D - 8;
    return s < D ? s : 0;
  }
  __device__ __forceinline__ int at(int v, int i) const {
    return KIND == kTiny ? (v * 8 + i) * G + lane : base(v) + i;
  }
  __device__ __forceinline__ bool has(int v, int i) const {
    if (KIND == kTiny) return at(v, i) < D;
    return start(v) < D && (KIND == kWhole || base(v) + i >= start(v));
  }
  __device__ __forceinline__ bool whole(int v) const { return start(v) + 8 <= D; }

  // What a lane reads of a row, and later its values.
  struct Held {
    Raw8 v[KIND == kTiny ? 1 : V];
    float s[KIND == kTiny ? V : 1][8];
  };
  __device__ __forceinline__ Held load(const void* p, int64_t row, bool f32) const {
    Held h;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (KIND != kTiny) {
        h.v[v] = load8(p, row + base(v), f32);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h.s[v][i] = load1(p, row + (has(v, i) ? at(v, i) : 0), f32);
      }
    }
    return h;
  }
  __device__ __forceinline__ void values(const Held& h, bool f32, float (&x)[V][8]) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (KIND != kTiny) values8(h.v[v], f32, x[v]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[v][i] = has(v, i) ? (KIND == kTiny ? h.s[KIND == kTiny ? v : 0][i] : x[v][i]) : 0.f;
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t row, bool f32,
                                        const float (&x)[V][8]) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (KIND != kTiny && whole(v)) {
        store8(p, row + base(v), f32, x[v]);
      } else if (KIND != kWhole) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (has(v, i)) store1(p, row + at(v, i), f32, x[v][i]);
      }
    }
  }
  __device__ __forceinline__ void store_i8(int8_t* p, int64_t row, int v, uint32_t lo,
                                           uint32_t hi) const {
    if (KIND != kTiny && whole(v)) {
      reinterpret_cast<AnyU32x2*>(p + row + base(v))->v = ops_u32x2{lo, hi};
    } else if (KIND != kWhole) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (has(v, i)) p[row + at(v, i)] = (int8_t)((i < 4 ? lo : hi) >> 8 * (i % 4));
    }
  }
};

// x -> N(x), without weights.  Elements past the row's end are zero on entry
// and are left out of the centred sum; their values on exit are not used.
template <int G, int V, RowKind KIND>
__device__ __forceinline__ void normalise(const Row<G, V, KIND>& row, Group<G>& grp, bool center,
                                          float eps, float (&x)[V][8]) {
  const float inv_d = 1.0f / (float)row.D;
  if (center) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += x[v][i];
    const float mean = grp.sum(s) * inv_d;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[v][i] = row.has(v, i) ? x[v][i] - mean : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) s += x[v][i] * x[v][i];
  const float k = 1.0f / sqrtf(grp.sum(s) * inv_d + eps);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[v][i] *= k;
}

// Row to int8 (RowScale).  The magnitudes are compared as bit patterns, so that a
// NaN or an infinity comes out on top instead of being passed over.
template <int G, int V, RowKind KIND>
__device__ __forceinline__ void quantise(const Row<G, V, KIND>& row, Group<G>& grp,
                                         const float (&x)[V][8], int8_t* q, int64_t base,
                                         float* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = __builtin_bit_cast(uint32_t, x[v][i]) & 0x7fffffffu;
      if (row.has(v, i)) top = b > top ? b : top;
    }
  top = grp.umax(top);
  const RowScale rs(top);
  if (row.lane == 0) *scale = rs.scale;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    row.store_i8(q, base, v, rs.quantise4(x[v][0], x[v][1], x[v][2], x[v][3]),
                 rs.quantise4(x[v][4], x[v][5], x[v][6], x[v][7]));
  }
}

// Threads of a workgroup whose rows belong to groups of G lanes.
constexpr int group_threads(int G) { return G < 256 ? 256 : G; }

template <int G, int V, RowKind KIND>
__global__ __launch_bounds__(group_threads(G)) void residual_norm_kernel(NormArgs a) {
  const lowm_residual_norm_args& u = a.u;
  __shared__ float lds[kMaxReductions * (G / kWave)];
  const int64_t m = a.first + (int64_t)blockIdx.x * (group_threads(G) / G) + threadIdx.x / G;
  // Whole wavefronts leave here, and only where no group spans two of them.
  if (m >= u.M) return;
  const Row<G, V, KIND> row{(int)threadIdx.x % G, u.D};
  Group<G> grp{lds};

  // Every load, then every value.  An operand that is not there reads y again.
  const bool post = u.flags & LOWM_NORM_POST, center = u.flags & LOWM_NORM_CENTER;
  const bool pre = !(u.flags & LOWM_NORM_NO_PRE);
  const bool weigh_post = post && u.w_post, weigh_pre = pre && u.w_pre;
  const bool y32 = u.y_type == LOWM_F32, r32 = u.r_type == LOWM_F32, w32 = u.w_type == LOWM_F32,
             g32 = u.gate_type == LOWM_F32, gate_row = u.gate && u.gate_col;
  const int64_t at_y = m * u.ld_y;
  const auto held_y = row.load(u.y, at_y, y32);
  const auto held_r = row.load(u.r, m * u.ld_r, r32);
  const auto held_post =
      row.load(weigh_post ? u.w_post : u.y, weigh_post ? 0 : at_y, weigh_post ? w32 : y32);
  const auto held_gate =
      row.load(gate_row ? u.gate : u.y, gate_row ? m * u.gate_row : at_y, gate_row ? g32 : y32);
  const auto held_pre =
      row.load(weigh_pre ? u.w_pre : u.y, weigh_pre ? 0 : at_y, weigh_pre ? w32 : y32);
  const float gate_one = u.gate && !u.gate_col ? load1(u.gate, m * u.gate_row, g32) : 1.f;

  float p[V][8], r[V][8], w[V][8], g[V][8];
  row.values(held_y, y32, p);
  // what multiplies the branch: gate * w_post
  row.values(held_post, w32, w);
  row.values(held_gate, g32, g);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      g[v][i] = (gate_row ? g[v][i] : gate_one) * (weigh_post ? w[v][i] : 1.f);

  if (post) normalise(row, grp, center, u.eps, p);
  row.values(held_r, r32, r);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = u.residual_scale * r[v][i] + u.branch_scale * (g[v][i] * p[v][i]);
      r[v][i] = row.has(v, i) ? t : 0.f;
    }
  row.store(u.r_out, m * u.ld_r_out, r32, r);
  if (!pre) return;
  normalise(row, grp, center, u.eps, r);
  if (weigh_pre) {
    row.values(held_pre, w32, w);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) r[v][i] *= w[v][i];
  }
  if (u.x_type == LOWM_I8)
    quantise(row, grp, r, static_cast<int8_t*>(u.x), m * u.ld_x, u.x_scale + m);
  else
    row.store(u.x, m * u.ld_x, false, r);
}

struct QuantArgs {
  const void* x;
  int8_t* q;
  float* scale;
  int64_t ld, first;
  int M, D, f32;
};

template <int G, int V, RowKind KIND>
__global__ __launch_bounds__(group_threads(G)) void quantize_rows_kernel(QuantArgs a) {
  __shared__ float lds[kMaxReductions * (G / kWave)];
  const int64_t m = a.first + (int64_t)blockIdx.x * (group_threads(G) / G) + threadIdx.x / G;
  if (m >= a.M) return;
  const Row<G, V, KIND> row{(int)threadIdx.x % G, a.D};
  Group<G> grp{lds};
  float x[V][8];
  row.values(row.load(a.x, m * a.ld, a.f32 != 0), a.f32 != 0, x);
  quantise(row, grp, x, a.q, m * (int64_t)a.D, a.scale + m);
}

// The group of lanes for rows of D elements: a wavefront up to 512 elements, 256
// lanes up to 2048 of them in one run per lane and 4096 in two, 512 lanes up to
// 8192, then 1024 lanes with up to four runs (two for the norm, whose operands
// stay in registers).  Measured on MI355X, residual_norm, us a call: 4096 rows of
// 6144 44.6 with 512 lanes and two runs, 64.7 with 1024 lanes and one (a workgroup
// of 16 wavefronts leaves the CU idle between rows); one row 4.4 against 4.2.
template <template <int, int, RowKind> class K, RowKind KIND, int VMAX, typename A>
int launch_kind(A a, int M, int D, hipStream_t stream) {
  auto go = [&](auto fn, int G) {
    const int64_t per = group_threads(G) / G, most = kMaxThreads / group_threads(G);
    const int64_t blocks = (M + per - 1) / per;
    void* args[] = {&a};
    int rc = LOWM_OK;
    for (int64_t b = 0; b < blocks && rc == LOWM_OK; b += most) {
      a.first = b * per;
      rc = launched(hipLaunchKernel(reinterpret_cast<const void*>(fn),
                                    dim3((unsigned)(blocks - b < most ? blocks - b : most)),
                                    dim3(group_threads(G)), args, 0, stream));
    }
    return rc;
  };
  if constexpr (KIND == kTiny) {
    return go(K<64, 1, KIND>::fn(), 64);
  } else {
    if (D <= 512) return go(K<64, 1, KIND>::fn(), 64);
    if (D <= 2048) return go(K<256, 1, KIND>::fn(), 256);
    if (D <= 4096) return go(K<256, 2, KIND>::fn(), 256);
    if (D <= 8192) return go(K<512, 2, KIND>::fn(), 512);
    if constexpr (VMAX > 2) {
      if (D > 16384) return go(K<1024, 4, KIND>::fn(), 1024);
    }
    return go(K<1024, 2, KIND>::fn(), 1024);
  }
}
template <template <int, int, RowKind> class K, int VMAX, typename A>
int launch_rows(const A& a, int M, int D, hipStream_t stream) {
  return D < 8        ? launch_kind<K, kTiny, VMAX>(a, M, D, stream)
         : D % 8 == 0 ? launch_kind<K, kWhole, VMAX>(a, M, D, stream)
                      : launch_kind<K, kRagged, VMAX>(a, M, D, stream);
}
template <int G, int V, RowKind KIND>
struct NormK {
  static auto fn() { return &residual_norm_kernel<G, V, KIND>; }
};
template <int G, int V, RowKind KIND>
struct QuantK {
  static auto fn() { return &quantize_rows_kernel<G, V, KIND>; }
};

bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }
bool real_type(int t) { return t == LOWM_BF16 || t == LOWM_F32; }

int residual_norm(const lowm_residual_norm_args* u, hipStream_t stream) {
  if (!u || u->M < 0 || u->D < 1) return LOWM_ERR_INVALID_ARG;
  if (u->M == 0) return LOWM_OK;
  if (!u->y || !u->r || !u->r_out) return LOWM_ERR_INVALID_ARG;
  const bool pre = !(u->flags & LOWM_NORM_NO_PRE);
  const bool i8 = pre && u->x_type == LOWM_I8;
  if (u->flags & ~(LOWM_NORM_POST | LOWM_NORM_NO_PRE | LOWM_NORM_CENTER))
    return LOWM_ERR_INVALID_ARG;
  if (!real_type(u->y_type) || !real_type(u->r_type) || !real_type(u->w_type) ||
      !real_type(u->gate_type))
    return LOWM_ERR_INVALID_ARG;
  if (pre && (!u->x || (u->x_type != LOWM_BF16 && u->x_type != LOWM_I8) || u->ld_x < u->D))
    return LOWM_ERR_INVALID_ARG;
  if (i8 && !u->x_scale) return LOWM_ERR_INVALID_ARG;
  if (u->ld_y < u->D || u->ld_r < u->D || u->ld_r_out < u->D) return LOWM_ERR_INVALID_ARG;
  if (u->gate && (u->gate_row < 0 || (u->gate_col != 0 && u->gate_col != 1)))
    return LOWM_ERR_INVALID_ARG;
  if (u->D > LOWM_NORM_MAX_D) return LOWM_ERR_UNSUPPORTED;
  const int yb = type_bytes(u->y_type), rb = type_bytes(u->r_type), wb = type_bytes(u->w_type),
            gb = type_bytes(u->gate_type), xb = type_bytes(u->x_type);
  if (!aligned(u->y, yb) || !aligned(u->r, rb) || !aligned(u->r_out, rb) ||
      !aligned(u->w_post, wb) || !aligned(u->w_pre, wb) || !aligned(u->gate, gb) ||
      (pre && !aligned(u->x, xb)) || (i8 && !aligned(u->x_scale, 4)))
    return LOWM_ERR_UNSUPPORTED;
  const int64_t M = u->M, D = u->D;
  const bool inplace = u->r_out == u->r && u->ld_r_out == u->ld_r;
  const Span y = span_of(u->y, M, D, u->ld_y, yb), r = span_of(u->r, M, D, u->ld_r, rb),
             ro = span_of(u->r_out, M, D, u->ld_r_out, rb),
             w0 = span_of(u->w_post, 1, D, D, wb), w1 = span_of(u->w_pre, 1, D, D, wb),
             g = span_of(u->gate, M, u->gate_col ? D : 1, u->gate_row, gb),
             x = span_of(pre ? u->x : nullptr, M, D, u->ld_x, xb),
             xs = span_of(i8 ? u->x_scale : nullptr, 1, M, M, 4);
  const Span in[] = {y, w0, w1, g}, out[] = {ro, x, xs};
  for (const Span& o : out)
    for (const Span& s : in)
      if (meet(o, s)) return LOWM_ERR_INVALID_ARG;
  if ((!inplace && meet(ro, r)) || meet(x, r) || meet(xs, r) || meet(ro, x) || meet(ro, xs) ||
      meet(x, xs))
    return LOWM_ERR_INVALID_ARG;
  const NormArgs a{*u, 0};
  return launch_rows<NormK, 2>(a, u->M, u->D, stream);
}

}  // namespace

// (The int8 product calls this too.)
int quantize_rows(const void* x, int x_type, int64_t ld, int M, int K, void* q, float* scale,
                  hipStream_t stream) {
  if (M < 0 || K < 1 || ld < K || !real_type(x_type)) return LOWM_ERR_INVALID_ARG;
  if (M == 0) return LOWM_OK;
  if (!x || !q || !scale) return LOWM_ERR_INVALID_ARG;
  if (K > LOWM_QUANTIZE_MAX_K) return LOWM_ERR_UNSUPPORTED;
  const int xb = type_bytes(x_type);
  if (!aligned(x, xb) || !aligned(scale, 4)) return LOWM_ERR_UNSUPPORTED;
  const Span xs = span_of(x, M, K, ld, xb), qs = span_of(q, M, K, K, 1),
             ss = span_of(scale, 1, M, M, 4);
  if (meet(xs, qs) || meet(xs, ss) || meet(qs, ss)) return LOWM_ERR_INVALID_ARG;
  const QuantArgs a{x, static_cast<int8_t*>(q), scale, ld, 0, M, K, x_type == LOWM_F32};
  return launch_rows<QuantK, 4>(a, M, K, stream);
}

}  // namespace lowm

extern "C" {

int lowm_residual_norm(const lowm_residual_norm_args* args, void* stream) {
  return lowm::residual_norm(args, static_cast<hipStream_t>(stream));
}

int lowm_quantize_rows(const void* x, int x_type, int64_t ld_x, int M, int K, void* q,
                       float* scale, void* stream) {
  return lowm::quantize_rows(x, x_type, ld_x, M, K, q, scale, static_cast<hipStream_t>(stream));
}

}  // extern "C"
