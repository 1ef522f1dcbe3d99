// Rotary positions with three axes (time, height, width).
//
// Pair p of a token's d/2 pairs belongs to one axis a (the first pairs[0]
// pairs to time, then height, then width; the rest stay unrotated) and turns
// by angle = (first_a + step_a * pos_a) * theta^(-i / pairs_a), i the pair's
// index within its axis:
//   (y0, y1) = (x0 cos - x1 sin, x0 sin + x1 cos).
// The pair's elements are 2p and 2p+1 (interleaved) or p and p + d/2.  The
// transposed rotation (sin negated) is the gradient's.
//
// The kernels are bound by HBM: every row is read once and written once (6
// flops a pair).  The cosines and sines come from a table of one row per
// axis coordinate (25 KB for a 21 x 45 x 80 grid at d = 128: it stays in
// L1), made once in 64 bits: an angle of some thousand radians in 32 bits
// would be off by 1e-4.
#include "common.cuh"

namespace paro {
namespace {

constexpr int kThreads = 256;

// Groups of four pairs: a table row holds its axis's pairs at the columns
// p - (start & ~3), its length rounded up to whole groups, so that a group
// of four pairs is 32 aligned bytes whatever the axes' numbers of pairs.
__host__ __device__ inline int row_groups(int start, int pairs) {
  return pairs == 0 ? 0 : ((start + pairs + 3) >> 2) - (start >> 2);
}

__global__ void rope_table_kernel(RopeTab t, double theta, double f0, double f1, double f2,
                                  double s0, double s1, double s2, float2* __restrict__ table) {
  const int a = blockIdx.y;
  const double first = a == 0 ? f0 : a == 1 ? f1 : f2, step = a == 0 ? s0 : a == 1 ? s1 : s2;
  const int cols = 4 * t.groups[a];
  const int64_t total = (int64_t)t.extent[a] * cols;
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < total;
       e += (int64_t)gridDim.x * blockDim.x) {
    const int pos = (int)(e / cols), col = (int)(e - (int64_t)pos * cols);
    const int i = col + (t.start[a] & ~3) - t.start[a];  // pair index within the axis
    float2 cs = make_float2(1.f, 0.f);
    if (i >= 0 && i < t.pairs[a]) {
      const double angle = (first + step * pos) * pow(theta, -(double)i / t.pairs[a]);
      double c, s;
      sincos(angle, &s, &c);
      cs = make_float2((float)c, (float)s);
    }
    table[t.offset[a] + e] = cs;
  }
}

// cos and sin of the NP pairs from p0 on (a multiple of NP) of the token at
// (pos[0], pos[1], pos[2]); pairs of no axis get (1, 0).  Most groups lie in
// one axis: one or two 16-byte loads.
template <int NP>
__device__ __forceinline__ void load_cs(const RopeTab& t, const float2* __restrict__ table,
                                        const int (&pos)[3], int p0, float2 (&cs)[NP]) {
  constexpr int G = NP < 4 ? NP : 4;
#pragma unroll
  for (int e = 0; e < NP; ++e) cs[e] = make_float2(1.f, 0.f);
#pragma unroll
  for (int g = 0; g < NP; g += G) {
#pragma unroll
    for (int a = 0; a < 3; ++a) {
      const int lo = t.start[a] - (p0 + g), hi = lo + t.pairs[a];  // the axis's pairs of the group
      if (lo >= G || hi <= 0 || t.pairs[a] == 0) continue;
      const float4* src = reinterpret_cast<const float4*>(
          table + t.offset[a] + (int64_t)pos[a] * (4 * t.groups[a]) + (p0 + g - (t.start[a] & ~3)));
#pragma unroll
      for (int e = 0; e < G; e += 2) {
        const float4 v = __ldg(src + e / 2);
        if (e >= lo && e < hi) cs[g + e] = make_float2(v.x, v.y);
        if (e + 1 >= lo && e + 1 < hi) cs[g + e + 1] = make_float2(v.z, v.w);
      }
    }
  }
}

// A unit of work: the chunks of a row that hold whole pairs.  Interleaved:
// one 16-byte chunk (E elements, E/2 pairs); halves: chunk c and the chunk
// d/2 elements on (E pairs).
template <typename T, bool kInter>
struct Unit {
  static constexpr int E = Chunk<T>::n;
  static constexpr int kChunks = kInter ? 1 : 2;
  static constexpr int kPairs = kInter ? E / 2 : E;
  uint4 u[kChunks];

  // The rotated values in f (element order of the chunks).
  __device__ __forceinline__ void rotate(const float2 (&cs)[kPairs], float sign,
                                         float (&f)[kChunks * E]) const {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) Chunk<T>::unpack(u[c], f + c * E);
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      const int i0 = kInter ? 2 * p : p, i1 = kInter ? 2 * p + 1 : E + p;
      const float a = f[i0], b = f[i1], s = sign * cs[p].y;
      f[i0] = a * cs[p].x - b * s;
      f[i1] = a * s + b * cs[p].x;
    }
  }
  __device__ __forceinline__ static uint4 pack(const float* f) {
    uint4 w;
    if constexpr (sizeof(T) == 4) {
      w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3]));
    } else {
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    }
    return w;
  }
};

// x -> y, any strides of batch, head and token.  A thread owns one unit of
// one token and goes over kHeads heads with it: the table is read once for
// them, and all their loads are in flight before the first store.  Rows of
// 16 (or 32) tokens of a head are neighbours in a head-major tensor, rows of
// kHeads heads of a token in a token-major one, so both sides move 1 KB or
// more in one piece.
template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const T* x, RowStride xs, T* y, RowStride ys, int N, int H, int W, int heads,
                const __grid_constant__ RopeTab tab, const float2* __restrict__ table,
                const int32_t* __restrict__ positions, int64_t pos_batch, float sign,
                int32_t* __restrict__ status) {
  using U = Unit<T, kInter>;
  constexpr int kUnits = D / U::E / U::kChunks;  // units of a row
  constexpr int kTokens = kThreads / kUnits;
  constexpr int kHeads = 8 / U::kChunks;
  const int c = threadIdx.x % kUnits;
  const int n = blockIdx.x * kTokens + threadIdx.x / kUnits;
  const int b = blockIdx.z;
  if (n >= N) return;
  int pos[3];
  if (positions != nullptr) {
    const int32_t* p = positions + b * pos_batch + (int64_t)n * 3;
    bool bad = false;
#pragma unroll
    for (int a = 0; a < 3; ++a) {
      pos[a] = __ldg(p + a);
      bad |= pos[a] < 0 || pos[a] >= tab.extent[a];
    }
    if (bad) {
      if (c == 0) report(status, PA_ERR_DEVICE_CHECK);
      return;
    }
  } else {
    pos[0] = n / (H * W);
    pos[1] = n / W % H;
    pos[2] = n % W;
  }
  const int h0 = blockIdx.y * kHeads;
  const T* src = x + b * xs.batch + h0 * xs.head + (int64_t)n * xs.token + c * U::E;
  T* dst = y + b * ys.batch + h0 * ys.head + (int64_t)n * ys.token + c * U::E;
  U unit[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h)
    if (h0 + h < heads)
#pragma unroll
      for (int k = 0; k < U::kChunks; ++k)
        unit[h].u[k] = *reinterpret_cast<const uint4*>(src + h * xs.head + k * (D / 2));
  float2 cs[U::kPairs];
  load_cs<U::kPairs>(tab, table, pos, c * U::kPairs, cs);
#pragma unroll
  for (int h = 0; h < kHeads; ++h)
    if (h0 + h < heads) {
      float f[U::kChunks * U::E];
      unit[h].rotate(cs, sign, f);
#pragma unroll
      for (int k = 0; k < U::kChunks; ++k)
        *reinterpret_cast<uint4*>(dst + h * ys.head + k * (D / 2)) = U::pack(f + k * U::E);
    }
}

// x (any strides) -> the permuted copy xp [B*heads, Np, D] of the rotated
// rows, pad rows zero, and the mean of each block's valid rotated rows
// (before their rounding to T) in pool.  One CTA per (block, head); a thread
// owns one unit of RPT rows and issues all its loads before the first use.
template <typename T, int D, int BLOCK, bool kInter>
__global__ void __launch_bounds__(kThreads)
    rope_reorder_kernel(const T* __restrict__ x, RowStride xs, const __grid_constant__ Grid g,
                        const __grid_constant__ RopeTab tab, const float2* __restrict__ table,
                        T* __restrict__ xp, float* __restrict__ pool) {
  using U = Unit<T, kInter>;
  constexpr int kUnits = D / U::E / U::kChunks;
  constexpr int kGroups = kThreads / kUnits;
  constexpr int RPT = BLOCK / kGroups;
  static_assert(RPT >= 1, "a block has a row for every group");
  __shared__ float red[kGroups][D];
  const int i = blockIdx.x;
  const int64_t bh = blockIdx.y;
  const int h = (int)(bh % g.heads);
  const int order = g.perm[h];
  const int c = threadIdx.x % kUnits, rg = threadIdx.x / kUnits;
  const int p0 = i * BLOCK;
  const int valid = min(BLOCK, g.N - p0);
  const T* src = x + (bh / g.heads) * xs.batch + h * xs.head + c * U::E;
  U unit[RPT];
  int nat[RPT];
#pragma unroll
  for (int k = 0; k < RPT; ++k) {
    const int r = rg + k * kGroups;
    nat[k] = r < valid ? natural_index(g, order, p0 + r) : -1;
#pragma unroll
    for (int m = 0; m < U::kChunks; ++m)
      unit[k].u[m] = nat[k] >= 0 ? __ldg(reinterpret_cast<const uint4*>(
                                       src + (int64_t)nat[k] * xs.token + m * (D / 2)))
                                 : make_uint4(0, 0, 0, 0);
  }
  T* dst = xp + (bh * (int64_t)g.Np + p0) * D + c * U::E;
  float acc[U::kChunks * U::E];
#pragma unroll
  for (int e = 0; e < U::kChunks * U::E; ++e) acc[e] = 0.f;
#pragma unroll
  for (int k = 0; k < RPT; ++k) {
    const int n = max(nat[k], 0);  // a pad row is zero: any angle keeps it so
    const int pos[3] = {n / (g.H * g.W), n / g.W % g.H, n % g.W};
    float2 cs[U::kPairs];
    load_cs<U::kPairs>(tab, table, pos, c * U::kPairs, cs);
    float f[U::kChunks * U::E];
    unit[k].rotate(cs, 1.f, f);
#pragma unroll
    for (int m = 0; m < U::kChunks; ++m)
      *reinterpret_cast<uint4*>(dst + (int64_t)(rg + k * kGroups) * D + m * (D / 2)) =
          U::pack(f + m * U::E);
#pragma unroll
    for (int e = 0; e < U::kChunks * U::E; ++e) acc[e] += f[e];
  }
  if (pool == nullptr) return;  // uniform across the CTA
#pragma unroll
  for (int m = 0; m < U::kChunks; ++m)
#pragma unroll
    for (int e = 0; e < U::E; ++e) red[rg][m * (D / 2) + c * U::E + e] = acc[m * U::E + e];
  __syncthreads();
  for (int col = threadIdx.x; col < D; col += kThreads) {
    float sum = 0.f;
    for (int r = 0; r < kGroups; ++r) sum += red[r][col];
    pool[(bh * g.NB + i) * D + col] = sum / (float)valid;
  }
}

template <typename T, int D, bool kInter>
cudaError_t launch_rope_typed(const void* x, RowStride xs, void* y, RowStride ys, const Grid& g,
                              const RopeTab& tab, const float* table, const int32_t* positions,
                              int64_t pos_batch, bool inverse, int32_t* status, cudaStream_t s) {
  using U = Unit<T, kInter>;
  constexpr int kTokens = kThreads / (D / U::E / U::kChunks);
  constexpr int kHeads = 8 / U::kChunks;
  const dim3 grid((g.N + kTokens - 1) / kTokens, (g.heads + kHeads - 1) / kHeads, g.B);
  rope_kernel<T, D, kInter><<<grid, kThreads, 0, s>>>(
      static_cast<const T*>(x), xs, static_cast<T*>(y), ys, g.N, g.H, g.W, g.heads, tab,
      reinterpret_cast<const float2*>(table), positions, pos_batch, inverse ? -1.f : 1.f, status);
  return cudaGetLastError();
}

template <typename T, int D, int BLOCK, bool kInter>
cudaError_t launch_reorder_typed(const void* x, RowStride xs, void* xp, const Grid& g,
                                 const RopeTab& tab, const float* table, float* pool,
                                 cudaStream_t s) {
  rope_reorder_kernel<T, D, BLOCK, kInter><<<dim3(g.NB, g.B * g.heads), kThreads, 0, s>>>(
      static_cast<const T*>(x), xs, g, tab, reinterpret_cast<const float2*>(table),
      static_cast<T*>(xp), pool);
  return cudaGetLastError();
}

}  // namespace

int64_t make_rope_tab(const pa_rope& r, RopeTab* t) {
  int64_t off = 0;
  int start = 0;
  for (int a = 0; a < 3; ++a) {
    t->extent[a] = r.extent[a];
    t->pairs[a] = r.pairs[a];
    t->start[a] = start;
    t->groups[a] = row_groups(start, r.pairs[a]);
    t->offset[a] = off;
    off += (int64_t)r.extent[a] * 4 * t->groups[a];
    start += r.pairs[a];
  }
  return off;
}

cudaError_t launch_rope_table(const RopeTab& t, double theta, const double* first,
                              const double* step, float* table, cudaStream_t s) {
  int64_t most = 1;
  for (int a = 0; a < 3; ++a)
    if ((int64_t)t.extent[a] * 4 * t.groups[a] > most) most = (int64_t)t.extent[a] * 4 * t.groups[a];
  const int64_t blocks = (most + 255) / 256;
  rope_table_kernel<<<dim3((unsigned)(blocks < 1024 ? blocks : 1024), 3), 256, 0, s>>>(
      t, theta, first[0], first[1], first[2], step[0], step[1], step[2],
      reinterpret_cast<float2*>(table));
  return cudaGetLastError();
}

cudaError_t launch_rope(const void* x, RowStride xs, void* y, RowStride ys, pa_dtype dt,
                        const Grid& g, const RopeTab& tab, bool interleaved, const float* table,
                        const int32_t* positions, int64_t pos_batch, bool inverse,
                        int32_t* status, cudaStream_t s) {
#define PARO_R(CODE, T, D)                                                                      \
  if (dt == CODE && g.d == D)                                                                   \
    return interleaved ? launch_rope_typed<T, D, true>(x, xs, y, ys, g, tab, table, positions,  \
                                                       pos_batch, inverse, status, s)           \
                       : launch_rope_typed<T, D, false>(x, xs, y, ys, g, tab, table, positions, \
                                                        pos_batch, inverse, status, s);
  PARO_R(PA_BF16, __nv_bfloat16, 64)
  PARO_R(PA_BF16, __nv_bfloat16, 128)
  PARO_R(PA_F32, float, 64)
  PARO_R(PA_F32, float, 128)
#undef PARO_R
  return cudaErrorInvalidValue;
}

cudaError_t launch_rope_reorder(const void* x, RowStride xs, void* xp, pa_dtype dt, const Grid& g,
                                const RopeTab& tab, bool interleaved, const float* table,
                                float* pool, cudaStream_t s) {
#define PARO_R(CODE, T, D, BL)                                                                  \
  if (dt == CODE && g.d == D && g.block == BL)                                                  \
    return interleaved                                                                          \
               ? launch_reorder_typed<T, D, BL, true>(x, xs, xp, g, tab, table, pool, s)        \
               : launch_reorder_typed<T, D, BL, false>(x, xs, xp, g, tab, table, pool, s);
  PARO_R(PA_BF16, __nv_bfloat16, 64, 64)
  PARO_R(PA_BF16, __nv_bfloat16, 64, 128)
  PARO_R(PA_BF16, __nv_bfloat16, 128, 64)
  PARO_R(PA_BF16, __nv_bfloat16, 128, 128)
  PARO_R(PA_F32, float, 64, 64)
  PARO_R(PA_F32, float, 64, 128)
  PARO_R(PA_F32, float, 128, 64)
  PARO_R(PA_F32, float, 128, 128)
#undef PARO_R
  return cudaErrorInvalidValue;
}

}  // namespace paro
