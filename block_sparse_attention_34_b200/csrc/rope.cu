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
#include "sm100.cuh"

namespace paro {
namespace {

using sm100::fadd2;
using sm100::ffma2;
using sm100::fmul2;

constexpr int kThreads = 256;

// A table row holds its axis's pairs at the columns p - (start & ~3), its
// length rounded up to whole groups of four, first the cosines, then the
// sines: a group of four pairs is 16 aligned bytes of each whatever the
// axes' numbers of pairs, and the lanes of a row read neighbouring chunks.
// A fourth axis with one row of (1, 0) holds the pairs that stay, so every
// pair has a place in the table.
__host__ __device__ inline int row_groups(int start, int pairs) {
  return pairs == 0 ? 0 : ((start + pairs + 3) >> 2) - (start >> 2);
}

__global__ void rope_table_kernel(RopeTab t, double theta, double f0, double f1, double f2,
                                  double s0, double s1, double s2, float* __restrict__ table) {
  const int a = blockIdx.y;
  const double first = a == 0 ? f0 : a == 1 ? f1 : f2, step = a == 0 ? s0 : a == 1 ? s1 : s2;
  const int cols = 4 * t.groups[a];
  const int64_t total = (int64_t)t.extent[a] * cols;
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < total;
       e += (int64_t)gridDim.x * blockDim.x) {
    const int pos = (int)(e / cols), col = (int)(e - (int64_t)pos * cols);
    const int i = col + (t.start[a] & ~3) - t.start[a];  // pair index within the axis
    double c = 1.0, s = 0.0;
    if (a < 3 && i >= 0 && i < t.pairs[a])
      sincos((first + step * pos) * pow(theta, -(double)i / t.pairs[a]), &s, &c);
    float* row = table + t.offset[a] + (int64_t)pos * 2 * cols;
    row[col] = (float)c;
    row[cols + col] = (float)s;
  }
}

// Where a thread finds the cosines and sines of its NP pairs, p0 on (a
// multiple of NP): group by group of G pairs, the axis of the group's last
// pair, and that of its first where it is another one.  The lanes of a warp
// lie in all axes, so all make the same loads and the few groups of two
// axes are put right after them (a loop over the axes with a branch each
// serialised three loads a row; pair by pair cost twice that again).
template <int NP>
struct CsPlan {
  static constexpr int G = NP < 4 ? NP : 4, NG = NP / G;
  const float* base[NG][2];
  int stride[NG][2], axis[NG][2];
  int split[NG];  // pairs of the group before the last axis's first

  __device__ __forceinline__ CsPlan(const RopeTab& t, const float* table, int p0) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int p = p0 + g * G + u * (G - 1);
        int a = 3;
#pragma unroll
        for (int x = 2; x >= 0; --x)
          if (p >= t.start[x] && p < t.start[x] + t.pairs[x]) a = x;
        axis[g][u] = a;
        stride[g][u] = 8 * t.groups[a];
        base[g][u] = table + t.offset[a] + (p0 + g * G - (t.start[a] & ~3));
        split[g] = t.start[a] - (p0 + g * G);
      }
    }
  }

  __device__ __forceinline__ static void load4(const float* src, float (&f)[G]) {
    if constexpr (G == 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(src));
      f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else {
      const float2 v = __ldg(reinterpret_cast<const float2*>(src));
      f[0] = v.x, f[1] = v.y;
    }
  }

  // of RB tokens with coordinate at[k * step + 1 + a] on axis a
  template <int RB>
  __device__ __forceinline__ void load(const int* at, int step, float2 (&cos)[RB][NP / 2],
                                       float2 (&sin)[RB][NP / 2]) const {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float c[RB][G], s[RB][G];
#pragma unroll
      for (int k = 0; k < RB; ++k) {
        const float* src = base[g][1] + (int64_t)at[k * step + 1 + axis[g][1]] * stride[g][1];
        load4(src, c[k]);
        load4(src + stride[g][1] / 2, s[k]);
      }
      if (split[g] > 0) {
        float c0[RB][G], s0[RB][G];
#pragma unroll
        for (int k = 0; k < RB; ++k) {
          const float* src = base[g][0] + (int64_t)at[k * step + 1 + axis[g][0]] * stride[g][0];
          load4(src, c0[k]);
          load4(src + stride[g][0] / 2, s0[k]);
        }
#pragma unroll
        for (int k = 0; k < RB; ++k)
#pragma unroll
          for (int e = 0; e < G; ++e) {
            c[k][e] = e < split[g] ? c0[k][e] : c[k][e];
            s[k][e] = e < split[g] ? s0[k][e] : s[k][e];
          }
      }
#pragma unroll
      for (int k = 0; k < RB; ++k)
#pragma unroll
        for (int e = 0; e < G; e += 2) {
          cos[k][(g * G + e) / 2] = make_float2(c[k][e], c[k][e + 1]);
          sin[k][(g * G + e) / 2] = make_float2(s[k][e], s[k][e + 1]);
        }
    }
  }

  // Axes of one or two pairs may put a third axis into a group (the tables'
  // `tiny`): pair by pair.
  __device__ __forceinline__ static void load_tiny(const RopeTab& t, const float* table,
                                                   const int* at, int p0,
                                                   float2 (&cos)[NP / 2], float2 (&sin)[NP / 2]) {
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      int a = 3;
#pragma unroll
      for (int x = 2; x >= 0; --x)
        if (p0 + e >= t.start[x] && p0 + e < t.start[x] + t.pairs[x]) a = x;
      const float* src = table + t.offset[a] + (int64_t)at[1 + a] * (8 * t.groups[a]) +
                         (p0 + e - (t.start[a] & ~3));
      (e & 1 ? cos[e / 2].y : cos[e / 2].x) = __ldg(src);
      (e & 1 ? sin[e / 2].y : sin[e / 2].x) = __ldg(src + 4 * t.groups[a]);
    }
  }
};

// Streamed data: read once, kept out of L1, where the table stays.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 u;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p));
  return u;
}

// A unit of work: the chunks of a row that hold whole pairs.  Interleaved:
// one 16-byte chunk (E elements, E/2 pairs); halves: chunk c and the chunk
// d/2 elements on (E pairs).
template <typename T, bool kInter>
struct Unit {
  static constexpr int E = Chunk<T>::n;
  static constexpr int kChunks = kInter ? 1 : 2;
  static constexpr int kPairs = kInter ? E / 2 : E;
  static constexpr int kTwo = kPairs / 2;  // the pairs two by two, for f32x2 arithmetic
  uint4 u[kChunks];

  // The pairs' first elements a and second elements b.
  __device__ __forceinline__ void unpack(float2 (&a)[kTwo], float2 (&b)[kTwo]) const {
    const uint32_t* w = &u[0].x;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kTwo; ++i) {
        if constexpr (kInter) {
          a[i] = make_float2(__uint_as_float(w[4 * i]), __uint_as_float(w[4 * i + 2]));
          b[i] = make_float2(__uint_as_float(w[4 * i + 1]), __uint_as_float(w[4 * i + 3]));
        } else {
          a[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
          b[i] = make_float2(__uint_as_float(w[2 * kTwo + 2 * i]),
                             __uint_as_float(w[2 * kTwo + 2 * i + 1]));
        }
      }
    } else {
      auto lo = [](uint32_t x) { return __uint_as_float(x << 16); };
      auto hi = [](uint32_t x) { return __uint_as_float(x & 0xffff0000u); };
#pragma unroll
      for (int i = 0; i < kTwo; ++i) {
        if constexpr (kInter) {
          a[i] = make_float2(lo(w[2 * i]), lo(w[2 * i + 1]));
          b[i] = make_float2(hi(w[2 * i]), hi(w[2 * i + 1]));
        } else {
          a[i] = make_float2(lo(w[i]), hi(w[i]));
          b[i] = make_float2(lo(w[kTwo + i]), hi(w[kTwo + i]));
        }
      }
    }
  }

  __device__ __forceinline__ void pack(const float2 (&a)[kTwo], const float2 (&b)[kTwo]) {
    uint32_t* w = &u[0].x;
#pragma unroll
    for (int i = 0; i < kTwo; ++i) {
      if constexpr (sizeof(T) == 4) {
        if constexpr (kInter) {
          w[4 * i] = __float_as_uint(a[i].x);
          w[4 * i + 1] = __float_as_uint(b[i].x);
          w[4 * i + 2] = __float_as_uint(a[i].y);
          w[4 * i + 3] = __float_as_uint(b[i].y);
        } else {
          w[2 * i] = __float_as_uint(a[i].x);
          w[2 * i + 1] = __float_as_uint(a[i].y);
          w[2 * kTwo + 2 * i] = __float_as_uint(b[i].x);
          w[2 * kTwo + 2 * i + 1] = __float_as_uint(b[i].y);
        }
      } else {
        if constexpr (kInter) {
          w[2 * i] = sm100::pack_bf16(a[i].x, b[i].x);
          w[2 * i + 1] = sm100::pack_bf16(a[i].y, b[i].y);
        } else {
          w[i] = sm100::pack_bf16(a[i].x, a[i].y);
          w[kTwo + i] = sm100::pack_bf16(b[i].x, b[i].y);
        }
      }
    }
  }

  // (a, b) turned by the angles of cos, sin; nsin = -sin
  __device__ __forceinline__ static void rotate(float2 (&a)[kTwo], float2 (&b)[kTwo],
                                                const float2 (&cos)[kTwo],
                                                const float2 (&sin)[kTwo],
                                                const float2 (&nsin)[kTwo]) {
#pragma unroll
    for (int i = 0; i < kTwo; ++i) {
      const float2 y = ffma2(b[i], nsin[i], fmul2(a[i], cos[i]));
      b[i] = ffma2(a[i], sin[i], fmul2(b[i], cos[i]));
      a[i] = y;
    }
  }

  // Column of the first (k = 0) or second element of pair p of chunk c.
  __device__ __forceinline__ static int column(int c, int p, int k, int d) {
    return kInter ? c * E + 2 * p + k : c * E + p + k * (d / 2);
  }
};

// x -> y, any strides of batch, head and token.  A thread owns one unit of
// one token and goes over `per` heads with it, at most kHeads: the table is
// read once for them, and all their loads are in flight before the first store.  Rows of
// 16 (or 32) tokens of a head are neighbours in a head-major tensor, rows of
// kHeads heads of a token in a token-major one: both sides move whole
// kilobytes.  Bound by HBM: 40 heads of 75,600 bf16 tokens take 233 us (6.6
// TB/s, the measured copy rate), 237 us from a token-major tensor.
template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const T* x, RowStride xs, T* y, RowStride ys, int N, int H, int W, int heads,
                int per, const __grid_constant__ RopeTab tab, const float* __restrict__ table,
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
  int at[5] = {n, 0, 0, 0, 0};
  int* pos = at + 1;
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
  const int h0 = blockIdx.y * per, mine = min(per, heads - h0);  // this CTA's heads
  const T* src = x + b * xs.batch + h0 * xs.head + (int64_t)n * xs.token + c * U::E;
  T* dst = y + b * ys.batch + h0 * ys.head + (int64_t)n * ys.token + c * U::E;
  U unit[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h)
    if (h < mine)
#pragma unroll
      for (int k = 0; k < U::kChunks; ++k)
        unit[h].u[k] = load_once(src + h * xs.head + k * (D / 2));
  float2 cos[1][U::kTwo], sin[1][U::kTwo], nsin[U::kTwo];
  if (tab.tiny)
    CsPlan<U::kPairs>::load_tiny(tab, table, at, c * U::kPairs, cos[0], sin[0]);
  else
    CsPlan<U::kPairs>(tab, table, c * U::kPairs).load(at, 0, cos, sin);
#pragma unroll
  for (int i = 0; i < U::kTwo; ++i) {
    sin[0][i] = make_float2(sign * sin[0][i].x, sign * sin[0][i].y);
    nsin[i] = make_float2(-sin[0][i].x, -sin[0][i].y);
  }
#pragma unroll
  for (int h = 0; h < kHeads; ++h)
    if (h < mine) {
      float2 a[U::kTwo], b2[U::kTwo];
      unit[h].unpack(a, b2);
      U::rotate(a, b2, cos[0], sin[0], nsin);
      unit[h].pack(a, b2);
#pragma unroll
      for (int k = 0; k < U::kChunks; ++k)
        *reinterpret_cast<uint4*>(dst + h * ys.head + k * (D / 2)) = unit[h].u[k];
    }
}

// Lists of heads of one order, each of the same length, -1 behind the last.
struct HeadLists {
  int16_t head[kMaxHeads + kOrders * 8];
};

// A CTA of rope_reorder_kernel: a thread's units of kRows rows.
template <typename T, int D, int BLOCK, bool kInter>
struct ReorderShape {
  static constexpr int kUnits = D / Unit<T, kInter>::E / Unit<T, kInter>::kChunks;
  static constexpr int kRows = kInter ? 8 : 4;
  static constexpr int kThreads = BLOCK * kUnits / kRows;
  static constexpr int kGroups = kThreads / kUnits;
  static constexpr int kStages = 3;
  static constexpr int kStageBytes = BLOCK * D * (int)sizeof(T);
  // CTAs an SM: what its shared memory holds (the stages and some 12 KB)
  static constexpr int kCtas = kStages * kStageBytes > 96 * 1024 ? 1 : 512 / kThreads;
  static_assert(kThreads % 32 == 0 && kThreads <= 512 && kUnits <= 32, "shape");
};

// x (any strides) -> the permuted copy xp [B*heads, Np, D] of the rotated
// rows, pad rows zero, and the mean of each block's valid rotated rows
// (before their rounding to T) in pool.  One CTA per block and list of heads
// of one order: the list's heads turn the same tokens by the same angles, so
// a thread keeps its rows' cosines and sines in registers and goes over the
// heads, while cp.async brings its chunks of the next two heads' rows into
// its own places in shared memory (no barrier but the means').  With the
// angles read for every head instead, their 1 KB a row from L1 bounded the
// kernel, and with the rows in registers too few were in flight (720p, 40
// heads: 310 and 300 us).  Bound by HBM: that case takes 245 us, 6.4 TB/s
// or 98% of the measured copy rate; fp32 478 us, 99%.
template <typename T, int D, int BLOCK, bool kInter>
__global__ void __launch_bounds__(ReorderShape<T, D, BLOCK, kInter>::kThreads,
                                  ReorderShape<T, D, BLOCK, kInter>::kCtas)
    rope_reorder_kernel(const T* __restrict__ x, RowStride xs, const __grid_constant__ Grid g,
                        const __grid_constant__ HeadLists heads, int lists, int length,
                        const __grid_constant__ RopeTab tab, const float* __restrict__ table,
                        T* __restrict__ xp, float* __restrict__ pool) {
  using U = Unit<T, kInter>;
  using S = ReorderShape<T, D, BLOCK, kInter>;
  constexpr int kRows = S::kRows, kWarps = S::kThreads / 32;
  extern __shared__ __align__(16) unsigned char stages[];
  __shared__ float red[2][kWarps][D];
  // a row's place in x (-1: a pad row) and its coordinates on the four axes
  __shared__ int64_t place[BLOCK];
  __shared__ int at[BLOCK][5];
  const int i = blockIdx.x;
  const int b = blockIdx.y / lists;
  const int16_t* hs = heads.head + (blockIdx.y - b * lists) * length;
  const int order = g.perm[hs[0]];
  const int c = threadIdx.x % S::kUnits, rg = threadIdx.x / S::kUnits;
  const int p0 = i * BLOCK;
  const int valid = min(BLOCK, g.N - p0);
  int count = 1;  // heads of the list
  while (count < length && hs[count] >= 0) ++count;
  // once a row, not once a chunk: the divisions cost more than the rotation
  for (int r = threadIdx.x; r < BLOCK; r += S::kThreads) {
    const int n = natural_index(g, order, p0 + min(r, valid - 1));
    at[r][1] = n / (g.H * g.W);
    at[r][2] = n / g.W % g.H;
    at[r][3] = n % g.W;
    at[r][4] = 0;
    place[r] = r < valid ? n * xs.token : -1;
  }
  __syncthreads();
  const T* src = x + b * xs.batch + c * U::E;
  unsigned char* mine = stages + (rg * D + c * U::E) * sizeof(T);
  auto fetch = [&](int t) {
    if (t < count) {
      const T* s = src + hs[t] * xs.head;
      const uint32_t to =
          sm100::smem_u32(mine) + (uint32_t)(t % S::kStages) * S::kStageBytes;
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int64_t row = place[rg + k * S::kGroups];
#pragma unroll
        for (int m = 0; m < U::kChunks; ++m)
          sm100::cp_async16(to + (k * S::kGroups * D + m * (D / 2)) * sizeof(T),
                            s + (row < 0 ? 0 : row) + m * (D / 2), row < 0 ? 0u : 16u);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(0);
  fetch(1);
  float2 cos[kRows][U::kTwo], sin[kRows][U::kTwo];
  if (tab.tiny) {
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      CsPlan<U::kPairs>::load_tiny(tab, table, at[rg + k * S::kGroups], c * U::kPairs, cos[k],
                                   sin[k]);
  } else {
    CsPlan<U::kPairs>(tab, table, c * U::kPairs).load(at[rg], S::kGroups * 5, cos, sin);
  }
#pragma unroll 1
  for (int t = 0; t < count; ++t) {
    fetch(t + 2);
    asm volatile("cp.async.wait_group 2;" ::: "memory");  // this head's rows are here
    const unsigned char* from = mine + (t % S::kStages) * S::kStageBytes;
    T* dst = xp + (((int64_t)b * g.heads + hs[t]) * g.Np + p0 + rg) * D + c * U::E;
    float2 acc[2][U::kTwo];
#pragma unroll
    for (int e = 0; e < U::kTwo; ++e) acc[0][e] = acc[1][e] = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      U u;
#pragma unroll
      for (int m = 0; m < U::kChunks; ++m)
        u.u[m] = *reinterpret_cast<const uint4*>(
            from + (k * S::kGroups * D + m * (D / 2)) * sizeof(T));
      float2 f[2][U::kTwo], nsin[U::kTwo];
#pragma unroll
      for (int e = 0; e < U::kTwo; ++e) nsin[e] = make_float2(-sin[k][e].x, -sin[k][e].y);
      u.unpack(f[0], f[1]);
      U::rotate(f[0], f[1], cos[k], sin[k], nsin);
      u.pack(f[0], f[1]);
#pragma unroll
      for (int m = 0; m < U::kChunks; ++m)
        *reinterpret_cast<uint4*>(dst + k * S::kGroups * D + m * (D / 2)) = u.u[m];
#pragma unroll
      for (int e = 0; e < U::kTwo; ++e) {
        acc[0][e] = fadd2(acc[0][e], f[0][e]);
        acc[1][e] = fadd2(acc[1][e], f[1][e]);
      }
    }
    if (pool != nullptr) {  // uniform across the grid
      // the warp's rows, then the warps; two buffers, so one barrier a head
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int p = 0; p < U::kPairs; ++p) {
          float v = p & 1 ? acc[k][p / 2].y : acc[k][p / 2].x;
#pragma unroll
          for (int off = S::kUnits; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
          if (threadIdx.x % 32 < S::kUnits)
            red[t & 1][threadIdx.x / 32][U::column(c, p, k, D)] = v;
        }
      __syncthreads();
      for (int col = threadIdx.x; col < D; col += S::kThreads) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += red[t & 1][w][col];
        pool[(((int64_t)b * g.heads + hs[t]) * g.NB + i) * D + col] = sum / (float)valid;
      }
    }
  }
}

template <typename T, int D, bool kInter>
cudaError_t launch_rope_typed(const void* x, RowStride xs, void* y, RowStride ys, const Grid& g,
                              const RopeTab& tab, const float* table, const int32_t* positions,
                              int64_t pos_batch, bool inverse, int32_t* status, cudaStream_t s) {
  using U = Unit<T, kInter>;
  constexpr int kTokens = kThreads / (D / U::E / U::kChunks);
  constexpr int kHeads = 8 / U::kChunks;
  const int groups = (g.heads + kHeads - 1) / kHeads, per = (g.heads + groups - 1) / groups;
  const dim3 grid((g.N + kTokens - 1) / kTokens, (g.heads + per - 1) / per, g.B);
  rope_kernel<T, D, kInter><<<grid, kThreads, 0, s>>>(
      static_cast<const T*>(x), xs, static_cast<T*>(y), ys, g.N, g.H, g.W, g.heads, per, tab,
      table, positions, pos_batch, inverse ? -1.f : 1.f, status);
  return cudaGetLastError();
}

template <typename T, int D, int BLOCK, bool kInter>
cudaError_t launch_reorder_typed(const void* x, RowStride xs, void* xp, const Grid& g,
                                 const RopeTab& tab, const float* table, float* pool,
                                 cudaStream_t s) {
  // heads a list: up to eight, as many as leave four CTAs for every SM (two
  // or eight instead of four changed no measured case by more than 3%)
  const int64_t blocks = (int64_t)g.NB * g.B * g.heads;
  const int64_t want = blocks / (4 * 148);
  const int length = want < 1 ? 1 : want > 8 ? 8 : (int)want;
  HeadLists l;
  int n = 0;
  for (int o = 0; o < kOrders; ++o) {
    for (int h = 0; h < g.heads; ++h)
      if (g.perm[h] == o) l.head[n++] = (int16_t)h;
    while (n % length != 0) l.head[n++] = -1;
  }
  const int lists = n / length;
  using S = ReorderShape<T, D, BLOCK, kInter>;
  auto kern = rope_reorder_kernel<T, D, BLOCK, kInter>;
  const int smem = S::kStages * S::kStageBytes;
  if (smem > 32 * 1024) {  // with the static part, more than a kernel has unasked
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<dim3(g.NB, g.B * lists), S::kThreads, smem, s>>>(static_cast<const T*>(x), xs, g, l, lists,
                                                         length, tab, table, static_cast<T*>(xp),
                                                         pool);
  return cudaGetLastError();
}

}  // namespace

int64_t make_rope_tab(const pa_rope& r, RopeTab* t) {
  int64_t off = 0;
  int start = 0;
  for (int a = 0; a < 4; ++a) {
    t->extent[a] = a < 3 ? r.extent[a] : 1;
    t->pairs[a] = a < 3 ? r.pairs[a] : 64 - start;
    t->start[a] = start;
    t->groups[a] = row_groups(start, t->pairs[a]);
    t->offset[a] = off;
    off += (int64_t)t->extent[a] * 8 * t->groups[a];
    start += t->pairs[a];
  }
  // three axes in a group: one lies wholly inside it
  t->tiny = 0;
  for (int a = 1; a < 3; ++a)
    if (t->pairs[a] > 0 && t->pairs[a] < 3 && (t->start[a] & 3) != 0 &&
        (t->start[a] & 3) + t->pairs[a] < 4)
      t->tiny = 1;
  return off;
}

cudaError_t launch_rope_table(const RopeTab& t, double theta, const double* first,
                              const double* step, float* table, cudaStream_t s) {
  int64_t most = 1;
  for (int a = 0; a < 4; ++a)
    if ((int64_t)t.extent[a] * 4 * t.groups[a] > most) most = (int64_t)t.extent[a] * 4 * t.groups[a];
  const int64_t blocks = (most + 255) / 256;
  rope_table_kernel<<<dim3((unsigned)(blocks < 1024 ? blocks : 1024), 4), 256, 0, s>>>(
      t, theta, first[0], first[1], first[2], step[0], step[1], step[2],
      table);
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
