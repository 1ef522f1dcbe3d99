// Block-sparse attention of single query tokens over a stored clip: each
// query row scores the clip's blocks by q . kbar_j (kbar_j the block's mean
// key), keeps the k best and attends to their tokens,
//   out = sum_c softmax_c(q . k_c / sqrt(d)) v_c  over the kept blocks' keys.
//
// A row reads NB block means and k blocks of keys and values and does two
// flops a byte: a call is bound by HBM, and by latency where it has few
// rows.  So it is one launch.  A cluster of CTAs takes up to kRows query
// rows of one key head: it splits the means (scores exchanged through
// distributed shared memory), each CTA repeats the cheap selection (a warp a
// row), takes an equal share of the union of the rows' kept blocks, so that
// a block several rows keep is read once, and the partial softmax states
// (maximum, sum, weighted values) join in one CTA of the cluster per row.
// No workspace, no atomics on global memory, one order of every sum.
//
// The scores are sums of two floats each (error-free transformations: the
// compensated dot product of Ogita, Rump and Oishi), some 46 bits: a row
// keeps or drops whole blocks by them, and the order of a plain 32-bit sum
// would decide near ties.  64-bit arithmetic took five times as long.
//
// bf16: the products run on mma.sync m16n8k16 with the query rows as rows of
// the tile (the scalar form, 16 lanes a key, took four times the
// instructions and held a CTA at 46 GB/s).  P is not rounded to bf16 but
// split, p = bf16(p) + rest, and both parts multiply V, so P V keeps 16 bits
// of P (off by 2^-16 at most; the sums are fp32): up to 8 query rows sit in
// rows 0-7 of the tile and the rests in rows 8-15; with more, the rests are a
// second product.  fp32: one row a cluster, fp32 arithmetic throughout.
//
// Measured: 12 heads' one row over 64 of 256 blocks (52 MB) 17.5 us, of which
// some 9 are the launch, the scores' latency and the join, the rest at 6.5
// TB/s; 40 heads' 16 rows each over 89 of 591 blocks (1.56 GB, each block read
// once) 272 us, 5.7 TB/s.
#include <atomic>
#include <mutex>
#include <type_traits>

#include "bwd.cuh"
#include "sm100.cuh"

namespace paro {
namespace {

using sm100::fadd2;
using sm100::ffma2;
using sm100::fmul2;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;  // above 8 not portable: asked for, see ClusterFit
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T>
constexpr int kRows = sizeof(T) == 2 ? 16 : 1;  // query rows of a cluster
// partial states a CTA receives: C * ceil(R / C) < R + C
template <typename T>
constexpr int kSlots = kRows<T> + kMaxCluster - 1;
// bf16: a warp's ring of units, 16 keys of K or of V each
template <int D>
constexpr int kUnitBytes = 16 * D * 2;
// Shared memory that three phases use in turn: scores and selection (keys
// [R][NB] u64, the warps' histograms, the query rows), the copies' rings,
// the warps' softmax states.
template <typename T, int D, int kUnits>
constexpr int kRingBytes = sizeof(T) == 2 ? kWarps * kUnits * kUnitBytes<D>
                                          : kWarps * (D + 2) * 4;
static_assert(kWarps * 16 * (128 + 2) * 4 <= kRingBytes<__nv_bfloat16, 128, 3>, "states");
static_assert(kWarps * 16 * (64 + 2) * 4 <= kRingBytes<__nv_bfloat16, 64, 3>, "states");

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// The address, in CTA `rank` of the cluster, of this CTA's shared address.
__device__ __forceinline__ uint32_t map_rank(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a)
               : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Error-free sum of two floats: s + e = a + b exactly (Knuth).
__device__ __forceinline__ float two_sum(float a, float b, float& e) {
  const float s = a + b, t = s - a;
  e = (a - (s - t)) + (b - t);
  return s;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  return ffma2(b, make_float2(-1.f, -1.f), a);
}

// Order-preserving map of a float to 32 bits (-0 as +0).
__device__ __forceinline__ uint32_t order32(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
// Of the score hi + lo to 64 bits, NaN as -inf.
__device__ __forceinline__ uint64_t score_key(float hi, float lo) {
  float s = hi + lo, r = lo - (s - hi);
  if (!(fabsf(hi) < INFINITY)) s = hi, r = 0.f;  // infinite or NaN: no rest
  if (s != s) s = -INFINITY;
  if (r != r) r = 0.f;
  return ((uint64_t)order32(s) << 32) | order32(r);
}
__device__ __forceinline__ float key_score(uint64_t key) {
  const uint32_t b = (uint32_t)(key >> 32);
  return __uint_as_float((b >> 31) ? b ^ 0x80000000u : ~b);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The bin, from the top of 256, where the running count reaches need: lane l
// holds the bins 8 (31 - l) .. + 7.  Returns the bin and, in *left, how many
// of its keys are kept (-1: all).  One warp.
__device__ __forceinline__ int top_bin(const uint32_t* hist, int need, int lane, int* left) {
  // hist: 16-byte aligned
  const uint4 v = reinterpret_cast<const uint4*>(hist)[2 * (31 - lane)];
  const uint4 w = reinterpret_cast<const uint4*>(hist)[2 * (31 - lane) + 1];
  const uint32_t total = v.x + v.y + v.z + v.w + w.x + w.y + w.z + w.w;
  uint32_t upto = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += t;
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, upto >= (uint32_t)need)) - 1;
  // the lane's bins, one a lane: lane x takes bin 8 (31 - src) + 7 - x
  const int above = __shfl_sync(0xffffffffu, (int)(upto - total), src);
  const int first = 8 * (31 - src) + 7;
  uint32_t run = lane < 8 ? hist[first - lane] : 0;
  const uint32_t own = run;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += t;
  }
  const int x = __ffs(__ballot_sync(0xffffffffu, above + (int)run >= need)) - 1;
  const int before = above + (int)__shfl_sync(0xffffffffu, run - own, x);
  const int here = __shfl_sync(0xffffffffu, (int)own, x);
  *left = before + here == need ? -1 : need - before;
  return first - x;
}

// One warp: the last of the `kept` largest of keys[0, nb), ties to the lower
// index.  Kept are the keys > *from, and those equal to it up to index *upto.
// Radix selection from the top, eight bits a pass; done early once every key
// that shares the prefix is kept.  hist: 256 words of this warp.
__device__ __noinline__ void select_radix(const uint64_t* keys, int nb, int kept, uint32_t* hist,
                                          int lane, uint64_t* from, int* upto) {
  uint64_t prefix = 0;
  int need = kept;
  for (int shift = 56; shift >= 0; shift -= 8) {
#pragma unroll
    for (int x = 0; x < 8; ++x) hist[x * 32 + lane] = 0;
    __syncwarp();
    const uint64_t top = shift == 56 ? 0 : ~0ull << (shift + 8);
    for (int j = lane; j < nb; j += 32)
      if ((keys[j] & top) == prefix) atomicAdd(&hist[(keys[j] >> shift) & 255], 1u);
    __syncwarp();
    int left;
    const int digit = top_bin(hist, need, lane, &left);
    __syncwarp();  // the bins are read
    prefix |= (uint64_t)digit << shift;
    if (left < 0) {  // all that share the prefix: those > prefix - 1
      *from = prefix - 1;
      *upto = -1;
      return;
    }
    need = left;
  }
  int last = 0;  // the need-th key equal to the prefix
  for (int j0 = 0, seen = 0; j0 < nb && seen < need; j0 += 32) {
    const bool in = j0 + lane < nb && keys[j0 + lane] == prefix;
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    const uint32_t here =
        __ballot_sync(0xffffffffu, in && seen + __popc(m & ((1u << lane) - 1u)) == need - 1);
    if (here) last = j0 + __ffs(here) - 1;
    seen += __popc(m);
  }
  *from = prefix;
  *upto = last;
}

// The same, mostly in one pass: 256 equal bins between the smallest and the
// largest score (monotone in the score, so whole bins are kept or not), then
// the few keys of the bin at the border in order, one a lane.  Scores that
// are not finite or crowd one bin go through the radix passes, up to eight
// of about this one's cost.
__device__ __forceinline__ void select_row(const uint64_t* keys, int nb, int kept, uint32_t* hist,
                                           int lane, uint64_t* from, int* upto) {
  if (kept == nb) {
    *from = 0;
    *upto = nb;
    return;
  }
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll 8
  for (int j = lane; j < nb; j += 32) {
    const float s = key_score(keys[j]);
    lo = fminf(lo, s);
    hi = fmaxf(hi, s);
  }
#pragma unroll
  for (int x = 0; x < 8; ++x) hist[x * 32 + lane] = 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float width = 256.f / (hi - lo);
  if (width > 0.f && width < INFINITY && hi - lo < INFINITY) {
    auto bin = [&](uint64_t key) { return min(255, (int)((key_score(key) - lo) * width)); };
    __syncwarp();
    // (eight loads ahead of what is written: nothing else hides their time)
    for (int j0 = 0; j0 < nb; j0 += 256) {
      uint64_t key[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) key[x] = keys[min(j0 + 32 * x + lane, nb - 1)];
#pragma unroll
      for (int x = 0; x < 8; ++x)
        if (j0 + 32 * x + lane < nb) atomicAdd(&hist[bin(key[x])], 1u);
    }
    __syncwarp();
    int left;
    const int border = top_bin(hist, kept, lane, &left);
    const int crowd = hist[border];
    __syncwarp();
    if (crowd <= 32) {
      // the border bin's keys, ascending by index, into lanes; the bins'
      // memory holds their indices
      int n = 0;
      for (int j0 = 0; j0 < nb; j0 += 256) {
        uint64_t key[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) key[x] = keys[min(j0 + 32 * x + lane, nb - 1)];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int j = j0 + 32 * x + lane;
          const bool in = j < nb && bin(key[x]) == border;
          const uint32_t m = __ballot_sync(0xffffffffu, in);
          if (in) hist[n + __popc(m & ((1u << lane) - 1u))] = j;
          n += __popc(m);
        }
      }
      __syncwarp();
      const uint64_t mine = lane < n ? keys[hist[lane]] : 0;
      const int want = left < 0 ? n : left;
      int ahead = 0;  // keys of the bin before mine
      for (int x = 0; x < n; ++x) {
        const uint64_t other = __shfl_sync(0xffffffffu, mine, x);
        ahead += other > mine || (other == mine && x < lane);
      }
      const int src =
          __ffs(__ballot_sync(0xffffffffu, lane < n && ahead == want - 1)) - 1;
      *from = __shfl_sync(0xffffffffu, mine, src);
      *upto = hist[src];
      __syncwarp();
      return;
    }
  }
  __syncwarp();
  select_radix(keys, nb, kept, hist, lane, from, upto);
}

// 64-bit words of the keys of R rows: even, so that 16-byte reads may follow.
__host__ __device__ __forceinline__ int64_t key_words(int R, int NB) {
  return ((int64_t)R * NB + 1) / 2 * 2;
}

// Dynamic shared memory: the phases' region (phase_bytes), the union of the
// kept blocks [NB] u32 (the block, and from bit 16 the rows that keep it),
// the rows that keep each block [NB] u16.
template <typename T, int D, int kUnits>
__global__ void __launch_bounds__(kThreads, 1)
    query_attn_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                      const float* __restrict__ k_pool, int heads, int rows_per_head, int tiles,
                      int R, int N, int NB, int block, int k_keep,
                      const int32_t* __restrict__ lengths, float scale_log2, int phase_bytes,
                      T* __restrict__ out, int32_t* __restrict__ idx, float* __restrict__ lse,
                      int32_t* __restrict__ status) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  uint64_t* keys = reinterpret_cast<uint64_t*>(smem_raw);
  // behind the keys, 16-byte aligned
  uint32_t* front = reinterpret_cast<uint32_t*>(keys + key_words(R, NB));
  uint32_t* hist = front + (threadIdx.x / 32) * 256;
  float* qs = reinterpret_cast<float*>(front + kWarps * 256);  // [R][D]
  float* part = reinterpret_cast<float*>(smem_raw);                            // [kWarps][R][D + 2]
  uint32_t* list = reinterpret_cast<uint32_t*>(smem_raw + phase_bytes);
  uint16_t* flags = reinterpret_cast<uint16_t*>(list + NB);
  __shared__ uint64_t row_from[kRows<T>];
  __shared__ int row_upto[kRows<T>];
  __shared__ int warp_n[kWarps];
  __shared__ float joined[kSlots<T>][D + 2];  // states received from the cluster

  const uint32_t C = cluster_size(), rank = cluster_rank();
  const int64_t tile = blockIdx.x / C;
  const int64_t bh = tile / tiles;  // b * heads + key head
  const int row_in = (int)(tile - bh * tiles) * R;
  const int64_t row0 = bh * rows_per_head + row_in;  // first query row
  const int nr = min(R, rows_per_head - row_in);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int len = lengths != nullptr ? __ldg(lengths + bh / heads) : N;
  if (len < 0 || len > N) {  // the cluster's CTAs alike
    if (rank == 0 && threadIdx.x == 0) report(status, PA_ERR_DEVICE_CHECK);
    return;
  }
  const int nb = (len + block - 1) / block;
  const int kept = min(k_keep, nb);
  if (kept == 0) {
    if (rank == 0) {
      for (int e = threadIdx.x; e < nr * D; e += kThreads) out[row0 * D + e] = from_float<T>(0.f);
      for (int e = threadIdx.x; e < nr * k_keep; e += kThreads) idx[row0 * k_keep + e] = -1;
      if (threadIdx.x < nr && lse != nullptr) lse[row0 + threadIdx.x] = -INFINITY;
    }
    return;
  }

  // ---- scores of the blocks j = rank, rank + C, ...: a warp four blocks,
  // their means read once for all rows.  The sums over the lanes are halved
  // as they are added (a lane keeps the half its bit selects), so that each
  // value ends in one lane group; every sum has the same order
  cluster_arrive();
  {
    constexpr int F = D / 32;  // elements of a lane
    const float* pool = k_pool + bh * (int64_t)NB * D + lane * F;
    const int step = (int)C * kWarps;
    bool ready = false;
    for (int j0 = (int)rank + (int)C * warp; j0 < nb || !ready; j0 += step * 4) {
      float f[4][F];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = min(j0 + u * step, nb - 1);
        if constexpr (F == 4) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(pool + (int64_t)j * D));
          f[u][0] = x.x, f[u][1] = x.y, f[u][2] = x.z, f[u][3] = x.w;
        } else {
          const float2 x = __ldg(reinterpret_cast<const float2*>(pool + (int64_t)j * D));
          f[u][0] = x.x, f[u][1] = x.y;
        }
      }
      if (!ready) {  // the query rows, behind the first means on their way
        for (int e = threadIdx.x; e < nr * D; e += kThreads) qs[e] = to_float(q[row0 * D + e]);
        __syncthreads();
        cluster_wait();  // every CTA runs: its shared memory may be written
        ready = true;
      }
      if (j0 >= nb) break;
      auto rows = [&](int r0, auto rb) {
        constexpr int RB = decltype(rb)::value;  // rows at once
        constexpr int kValues = 4 * RB, kLanes = 32 / kValues;
        float hi[kValues], lo[kValues];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          const float* row = qs + min(r0 + r, nr - 1) * D + lane * F;
          float2 nh[2], l2[2];  // minus the sum, and its rest, of two blocks each
          nh[0] = nh[1] = l2[0] = l2[1] = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < F; ++e) {
            const float2 x = make_float2(row[e], row[e]), nx = make_float2(-row[e], -row[e]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float2 y = make_float2(f[2 * u][e], f[2 * u + 1][e]);
              const float2 np = fmul2(nx, y), pe = ffma2(x, y, np);  // x y = pe - np exactly
              const float2 s = fadd2(nh[u], np), t = sub2(s, nh[u]);
              const float2 err = fadd2(sub2(nh[u], sub2(s, t)), sub2(np, t));
              l2[u] = fadd2(l2[u], sub2(pe, err));
              nh[u] = s;
            }
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            hi[4 * r + 2 * u] = -nh[u].x;
            hi[4 * r + 2 * u + 1] = -nh[u].y;
            lo[4 * r + 2 * u] = l2[u].x;
            lo[4 * r + 2 * u + 1] = l2[u].y;
          }
        }
        int held = kValues;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          auto add = [&](int x, float gh, float gl, float kh, float kl) {
            const float oh = __shfl_xor_sync(0xffffffffu, gh, o);
            const float ol = __shfl_xor_sync(0xffffffffu, gl, o);
            float e;
            hi[x] = two_sum(kh, oh, e);
            lo[x] = kl + ol + e;
          };
          if (held > 1) {
            held /= 2;
            const bool up = lane & o;
#pragma unroll
            for (int x = 0; x < kValues / 2; ++x)
              if (x < held)
                add(x, up ? hi[x] : hi[x + held], up ? lo[x] : lo[x + held],
                    up ? hi[x + held] : hi[x], up ? lo[x + held] : lo[x]);
          } else {
            add(0, hi[0], lo[0], hi[0], lo[0]);
          }
        }
        // value i = 4 r + u is in the lanes whose top bits are i
        const int i = lane / kLanes;
        const int r = r0 + i / 4, j = j0 + (i % 4) * step;
        if (r < nr && j < nb) {
          const uint64_t key = score_key(hi[0], lo[0]);
          for (int c = lane % kLanes; c < (int)C; c += kLanes)
            st_cluster(map_rank(keys + (int64_t)r * NB + j, c), key);
        }
      };
      if (nr == 1) {
        rows(0, std::integral_constant<int, 1>{});
      } else {
#pragma unroll 1
        for (int r0 = 0; r0 < nr; r0 += 4) rows(r0, std::integral_constant<int, 4>{});
      }
    }
  }
  cluster_arrive();
  cluster_wait();

  // ---- selection, a warp a row; then which rows keep each block, and the
  // list of the blocks that any keeps, each warp a run of blocks
  for (int r = warp; r < nr; r += kWarps) {
    uint64_t from;
    int upto;
    select_row(keys + (int64_t)r * NB, nb, kept, hist, lane, &from, &upto);
    if (lane == 0) {
      row_from[r] = from;
      row_upto[r] = upto;
    }
  }
  __syncthreads();
  int total = 0;
  {
    const int per = ((nb + kThreads - 1) / kThreads) * 32;
    const int lo = warp * per, hi = min(nb, lo + per);
    int n = 0;
    for (int j0 = lo; j0 < hi; j0 += 32) {
      const int j = j0 + lane;
      uint32_t f = 0;
      if (j < hi) {
        for (int r = 0; r < nr; ++r) {
          const uint64_t key = keys[(int64_t)r * NB + j], from = row_from[r];
          f |= (uint32_t)(key > from || (key == from && j <= row_upto[r])) << r;
        }
        flags[j] = (uint16_t)f;
      }
      n += __popc(__ballot_sync(0xffffffffu, f != 0));
    }
    if (lane == 0) warp_n[warp] = n;
    __syncthreads();
    int at = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += warp_n[w];
      total += warp_n[w];
    }
    for (int j0 = lo; j0 < hi; j0 += 32) {
      const int j = j0 + lane;
      const uint32_t f = j < hi ? flags[j] : 0u;
      const uint32_t ub = __ballot_sync(0xffffffffu, f != 0);
      if (f != 0) list[at + __popc(ub & ((1u << lane) - 1u))] = (uint32_t)j | (f << 16);
      at += __popc(ub);
    }
    __syncthreads();
  }

  // ---- attention over this CTA's share, in batches of 16 keys
  const int shift_block = block == 64 ? 2 : 3;
  const int items = total << shift_block;
  const int first = (int)((int64_t)items * rank / C), last = (int)((int64_t)items * (rank + 1) / C);
  const int64_t base = bh * (int64_t)NB * block;
  auto entry = [&](int it) { return list[it >> shift_block]; };
  auto position = [&](int it) {
    return (int)(entry(it) & 0xffffu) * block + (it & ((1 << shift_block) - 1)) * 16;
  };

  // the warps' states of rows lo .. hi-1 -> this CTA's, sent to the CTA that
  // ends the row: r % C, slot (r / C) C + rank
  auto send = [&](int lo, int hi) {
    for (int x = threadIdx.x; x < (hi - lo) * D; x += kThreads) {
      const int r = lo + x / D, e = x % D;
      const float* from = part + r * (D + 2);
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, from[w * R * (D + 2) + D]);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float os = 0.f, ls = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* f = from + w * R * (D + 2);
        const float wt = sm100::ex2(f[D] - ref);
        os += f[e] * wt;
        ls += f[D + 1] * wt;
      }
      const uint32_t dst = map_rank(joined[(r / C) * C + rank], r % C);
      st_cluster(dst + e * 4, os);
      if (e == 0) {
        st_cluster(dst + D * 4, mm);
        st_cluster(dst + (D + 1) * 4, ls);
      }
    }
  };

  if constexpr (sizeof(T) == 2) {
    constexpr int VPR = D / 8;  // 16-byte chunks of a row
    const int g = lane >> 2, jq = lane & 3;  // this lane's tile row, its columns 2 jq, 2 jq + 1
    const uint32_t ring = sm100::smem_u32(smem_raw) + (uint32_t)warp * kUnits * kUnitBytes<D>;
    // unit n of this warp: K (n even) or V (odd) of its batch n / 2, its
    // chunks swizzled by the row; rows behind the clip's end are zero,
    // whatever the cache holds there
    auto fetch = [&](int n, int slot) {
      const int it = first + warp + (n >> 1) * kWarps;
      if (it < last) {
        const int p0 = position(it);
        const T* src = (n & 1 ? v : k) + (base + p0) * D;
        const uint32_t to = ring + (uint32_t)slot * kUnitBytes<D>;
#pragma unroll
        for (int u = 0; u < VPR / 2; ++u) {
          const int e = u * 32 + lane, r = e / VPR, c = e % VPR;
          sm100::cp_async16(to + (r * VPR + (c ^ (r & 7))) * 16, src + e * 8,
                            p0 + r < len ? 16u : 0u);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // The rows of `set` over the blocks that one of them keeps; whether their
    // states are finite.  kPacked (at most 8 rows): row g + 8 of the tile
    // holds the rests of row g's P; otherwise it is a query row of its own.
    auto attend = [&](uint32_t set, auto packed) -> bool {
      constexpr bool kPacked = decltype(packed)::value;
      constexpr int kHalves = kPacked ? 1 : 2;  // query rows of a lane: g (and g + 8)
      uint32_t qa[D / 16][4];
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = g + 8 * h;
          const uint32_t* src =
              reinterpret_cast<const uint32_t*>(q + (row0 + r) * D + ks * 16 + 2 * jq);
          const bool in = h < kHalves && r < nr;
          qa[ks][h] = in ? __ldg(src) : 0u;
          qa[ks][2 + h] = in ? __ldg(src + 4) : 0u;
        }
      float o[D / 8][4], m[kHalves], l[kHalves];
#pragma unroll
      for (int t = 0; t < D / 8; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) m[h] = -INFINITY, l[h] = 0.f;
#pragma unroll
      for (int n = 0; n < kUnits - 1; ++n) fetch(n, n);
      int n = 0, slot = 0;  // of K's unit
      auto next = [](int s) { return s == kUnits - 1 ? 0 : s + 1; };
      auto before = [](int s) { return s == 0 ? kUnits - 1 : s - 1; };
#pragma unroll 1
      for (int it = first + warp; it < last; it += kWarps, n += 2) {
        fetch(n + kUnits - 1, before(slot));
        asm volatile("cp.async.wait_group %0;" ::"n"(kUnits - 1) : "memory");
        __syncwarp();
        const uint32_t who = (entry(it) >> 16) & set;  // warp-uniform
        const int p0 = position(it);
        float s[2][4];
        if (who != 0) {
          const uint32_t kt = ring + (uint32_t)slot * kUnitBytes<D>;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
          for (int ks = 0; ks < D / 16; ks += 2)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              const int r = nt * 8 + (lane & 7);
              uint32_t b[4];
              ldsm4(kt + (r * VPR + ((ks * 2 + (lane >> 3)) ^ (r & 7))) * 16, b);
              mma16816(s[nt], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b[0], b[1]);
              mma16816(s[nt], qa[ks + 1][0], qa[ks + 1][1], qa[ks + 1][2], qa[ks + 1][3], b[2],
                       b[3]);
            }
        }
        __syncwarp();  // K's unit is consumed
        fetch(n + kUnits, slot);
        uint32_t a[4], rest[4];
        if (who != 0) {
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            const bool mine = (who >> (g + 8 * h)) & 1u;
            float mx = m[h];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float& x = s[nt][2 * h + e];
                x = mine && p0 + nt * 8 + 2 * jq + e < len ? x * scale_log2 : -INFINITY;
                mx = fmaxf(mx, x);
              }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float ref = mx == -INFINITY ? 0.f : mx;
            if (__any_sync(0xffffffffu, mx != m[h])) {
              const float alpha = sm100::ex2(m[h] - ref);
              l[h] *= alpha;
#pragma unroll
              for (int t = 0; t < D / 8; ++t)
#pragma unroll
                for (int e = 0; e < (kPacked ? 4 : 2); ++e) o[t][2 * h + e] *= alpha;
              m[h] = mx;
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              const float x = sm100::ex2(s[nt][2 * h] - ref);
              const float y = sm100::ex2(s[nt][2 * h + 1] - ref);
              l[h] += x + y;
              const uint32_t top = sm100::pack_bf16(x, y);
              const uint32_t low = sm100::pack_bf16(x - __uint_as_float(top << 16),
                                                    y - __uint_as_float(top & 0xffff0000u));
              a[2 * nt + h] = top;
              if (kPacked)
                a[2 * nt + 1] = low;
              else
                rest[2 * nt + h] = low;
            }
          }
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kUnits - 1) : "memory");
        __syncwarp();
        slot = next(slot);
        if (who != 0) {
          const uint32_t vt = ring + (uint32_t)slot * kUnitBytes<D>;
          const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
          for (int t = 0; t < D / 8; t += 2) {
            uint32_t b[4];
            ldsm4t(vt + (r * VPR + ((t + (lane >> 4)) ^ (r & 7))) * 16, b);
            mma16816(o[t], a[0], a[1], a[2], a[3], b[0], b[1]);
            mma16816(o[t + 1], a[0], a[1], a[2], a[3], b[2], b[3]);
            if constexpr (!kPacked) {
              mma16816(o[t], rest[0], rest[1], rest[2], rest[3], b[0], b[1]);
              mma16816(o[t + 1], rest[0], rest[1], rest[2], rest[3], b[2], b[3]);
            }
          }
        }
        __syncwarp();  // V's unit is consumed
        slot = next(slot);
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();  // every warp has left its ring: the states go over it
      bool fine = true;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (!((set >> (g + 8 * h)) & 1u)) continue;
        float* to = part + (warp * R + g + 8 * h) * (D + 2);
#pragma unroll
        for (int t = 0; t < D / 8; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = kPacked ? o[t][e] + o[t][2 + e] : o[t][2 * h + e];
            to[t * 8 + 2 * jq + e] = x;
            fine = fine && fabsf(x) < INFINITY;
          }
        if (jq == 0) {
          to[D] = m[h];
          to[D + 1] = l[h];
        }
      }
      return fine;
    };
    auto pass = [&](uint32_t set) {
      return R <= 8 ? attend(set, std::true_type{}) : attend(set, std::false_type{});
    };
    // A row that does not keep a block has weight 0 there, and 0 times an
    // infinite or NaN value of that block would be NaN: where a state is not
    // finite, the rows go over their blocks one by one.
    const bool fine = __syncthreads_and(pass((1u << nr) - 1u));
    if (fine || nr == 1) {
      send(0, nr);
    } else {
      for (int r = 0; r < nr; ++r) {
        __syncthreads();
        pass(1u << r);
        __syncthreads();
        send(r, r + 1);
      }
    }
  } else {
    constexpr int E = 4, LPR = D / E, RPL = 32 / LPR;  // a row's chunks, lanes and rows of a load
    constexpr int kLoads = 8;                          // 16-byte loads of K, and of V, in flight
    constexpr int RPB = RPL * kLoads;                  // rows of a batch: 8 or 16
    const int c = lane % LPR;
    float qf[E];
    Chunk<T>::unpack(__ldg(reinterpret_cast<const uint4*>(q + row0 * D) + c), qf);
#pragma unroll
    for (int e = 0; e < E; ++e) qf[e] *= scale_log2;
    float o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int it = first + warp; it < last; it += kWarps) {
#pragma unroll 1
      for (int sub = 0; sub < 16; sub += RPB) {
        const int p0 = position(it) + sub + lane / LPR;
        const uint4* ks = reinterpret_cast<const uint4*>(k + (base + p0) * D) + c;
        const uint4* vs = reinterpret_cast<const uint4*>(v + (base + p0) * D) + c;
        uint4 kr[kLoads], vr[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) kr[u] = __ldg(ks + u * RPL * LPR);
#pragma unroll
        for (int u = 0; u < kLoads; ++u) vr[u] = __ldg(vs + u * RPL * LPR);
        float s[kLoads], mx = m;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          float f[E];
          Chunk<T>::unpack(kr[u], f);
          s[u] = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) s[u] = fmaf(qf[e], f[e], s[u]);
        }
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1)
#pragma unroll
          for (int u = 0; u < kLoads; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], off);
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          if (p0 + u * RPL >= len) s[u] = -INFINITY;  // behind the clip's end
          mx = fmaxf(mx, s[u]);
        }
        const float ref = mx == -INFINITY ? 0.f : mx;
        const float alpha = sm100::ex2(m - ref);
        m = mx;
        l *= alpha;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= alpha;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const float p = sm100::ex2(s[u] - ref);
          l += p;
          float f[E];
          Chunk<T>::unpack(vr[u], f);
#pragma unroll
          for (int e = 0; e < E; ++e)
            // a row behind the end has weight 0 whatever its bits are
            o[e] = p0 + u * RPL < len ? fmaf(p, f[e], o[e]) : o[e];
        }
      }
    }
    // join the row groups of the warp
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, off);
      const float l2 = __shfl_xor_sync(0xffffffffu, l, off);
      const float mm = fmaxf(m, m2), ref = mm == -INFINITY ? 0.f : mm;
      const float w1 = sm100::ex2(m - ref), w2 = sm100::ex2(m2 - ref);
      l = l * w1 + l2 * w2;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * w1 + __shfl_xor_sync(0xffffffffu, o[e], off) * w2;
      m = mm;
    }
    if (lane < LPR) {
      float* to = part + warp * (D + 2);
#pragma unroll
      for (int e = 0; e < E; ++e) to[c * E + e] = o[e];
      if (lane == 0) {
        to[D] = m;
        to[D + 1] = l;
      }
    }
    __syncthreads();
    send(0, 1);
  }
  cluster_arrive();
  // the rows' lists, ascending: row r by the CTA behind the one that ends it
  for (int r = (int)((rank + C - 1) % C); r < nr; r += (int)C)
    if ((r / (int)C) % kWarps == warp) {
      int32_t* to = idx + (row0 + r) * k_keep;
      int at = 0;
#pragma unroll 4
      for (int j0 = 0; j0 < nb; j0 += 32) {
        const bool in = j0 + lane < nb && ((flags[j0 + lane] >> r) & 1u);
        const uint32_t m = __ballot_sync(0xffffffffu, in);
        if (in) to[at + __popc(m & ((1u << lane) - 1u))] = j0 + lane;
        at += __popc(m);
      }
      for (int e = kept + lane; e < k_keep; e += 32) to[e] = -1;
    }
  __syncwarp();
  cluster_wait();
  // ---- the rows this CTA ends
  for (int r = (int)rank; r < nr; r += (int)C) {
    const float(*from)[D + 2] = joined + (r / C) * C;
    if (threadIdx.x < D) {
      const int e = threadIdx.x;
      float mm = -INFINITY;
      for (uint32_t w = 0; w < C; ++w) mm = fmaxf(mm, from[w][D]);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float os = 0.f, ls = 0.f;
      for (uint32_t w = 0; w < C; ++w) {
        const float wt = sm100::ex2(from[w][D] - ref);
        os += from[w][e] * wt;
        ls += from[w][D + 1] * wt;
      }
      // no sum: every kept key scored -inf
      out[(row0 + r) * D + e] = from_float<T>(ls == 0.f ? 0.f : os / ls);
      if (e == 0 && lse != nullptr) lse[row0 + r] = (mm + log2f(ls)) * kLn2;
    }
  }
}

// How many clusters of n[C] CTAs, one CTA an SM, the current device runs at
// once (0: such a cluster does not fit): the driver's answer, asked for once a
// device.  It depends on which SMs of the part are in use; one B200 of 148 SMs
// runs 148, 74, 45, 33, 26, 22, 15, 15, 15, 11 and, from C = 11 on, 7.
struct ClusterFit {
  int n[kMaxCluster + 1];
};
template <auto Kern>
cudaError_t cluster_fit(const ClusterFit** out) {
  constexpr int kDevices = 64;
  static std::atomic<const ClusterFit*> known[kDevices];
  static ClusterFit fits[kDevices];
  static std::mutex mutex;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kDevices) return cudaErrorInvalidDevice;
  if ((*out = known[dev].load(std::memory_order_acquire)) != nullptr) return cudaSuccess;
  const std::lock_guard<std::mutex> lock(mutex);
  if ((*out = known[dev].load(std::memory_order_relaxed)) != nullptr) return cudaSuccess;
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, Kern)) != cudaSuccess) return e;
  const int smem = kSmemOptIn - (int)fa.sharedSizeBytes;
  if ((e = opt_in_smem<Kern, true>(smem)) != cudaSuccess) return e;
  ClusterFit& fit = fits[dev];
  for (int c = 1; c <= kMaxCluster; ++c) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&fit.n[c], Kern, &cfg) != cudaSuccess) {
      fit.n[c] = 0;
      (void)cudaGetLastError();  // a size that does not fit is no error of the call
    }
  }
  known[dev].store(&fit, std::memory_order_release);
  *out = &fit;
  return cudaSuccess;
}

template <typename T, int D, int kUnits>
cudaError_t launch_units(const void* q, const void* k, const void* v, const float* k_pool,
                         const Grid& g, int per_head, int R, int C, int phase, int smem, int k_keep,
                         const int32_t* lengths, void* out, int32_t* idx, float* lse,
                         int32_t* status, cudaStream_t s) {
  auto kern = query_attn_kernel<T, D, kUnits>;
  const int tiles = (per_head + R - 1) / R;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)g.B * g.heads * tiles * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const T*>(q), static_cast<const T*>(k),
                            static_cast<const T*>(v), k_pool, g.heads, per_head, tiles, R, g.N, g.NB,
                            g.block, k_keep, lengths, (float)(kLog2e / sqrt((double)D)), phase,
                            static_cast<T*>(out), idx, lse, status);
}

template <typename T, int D>
cudaError_t launch_typed(const void* q, const void* k, const void* v, const float* k_pool,
                         const Grid& g, int group, int M, int k_keep, const int32_t* lengths,
                         void* out, int32_t* idx, float* lse, int32_t* status, cudaStream_t s) {
  const int per_head = group * M;
  const int64_t heads = (int64_t)g.B * g.heads;
  // shared memory: the rings with six units in flight a warp, or three where
  // the lists of very many blocks need the room; the keys of R rows
  const int lists = (g.NB * 6 + 127) / 128 * 128;
  constexpr int kStatic = kSlots<T> * (D + 2) * 4 + 1024;
  const bool deep = kRingBytes<T, D, 6> + lists + kStatic <= kSmemOptIn;
  const int ring = deep ? kRingBytes<T, D, 6> : kRingBytes<T, D, 3>;
  const int room = kSmemOptIn - kStatic - lists;
  const ClusterFit* fit = nullptr;
  const cudaError_t e = deep ? cluster_fit<query_attn_kernel<T, D, 6>>(&fit)
                             : cluster_fit<query_attn_kernel<T, D, 3>>(&fit);
  if (e != cudaSuccess) return e;
  // rows of a cluster: as many as there are, but enough clusters for the SMs
  int R = per_head < kRows<T> ? per_head : kRows<T>;
  auto tiles = [&] { return (per_head + R - 1) / R; };
  auto front = [&] { return key_words(R, g.NB) * 8 + R * D * 4 + kWarps * 256 * 4; };
  while (R > 1 && (heads * tiles() * kMaxCluster < fit->n[1] || front() > room)) R = (R + 1) / 2;
  // CTAs of a cluster: as many as let all clusters run at once, one CTA an
  // SM (12 clusters of 12 CTAs, of which 7 fit, took 29 us, of 9 CTAs 18 us),
  // but four means or a batch of 16 keys for each of their warps
  const int64_t items = (int64_t)k_keep * (g.block / 16);
  const int64_t useful = items / kWarps > g.NB / (4 * kWarps) ? items / kWarps : g.NB / (4 * kWarps);
  int C = 1;
  for (int c = 2; c <= kMaxCluster; ++c)
    if (fit->n[c] >= heads * tiles() && c <= useful) C = c;
  int phase = (int)((front() + 127) / 128 * 128);
  if (phase < ring) phase = ring;
  const int smem = phase + lists;
  if (deep)
    return launch_units<T, D, 6>(q, k, v, k_pool, g, per_head, R, C, phase, smem, k_keep,
                                 lengths, out, idx, lse, status, s);
  return launch_units<T, D, 3>(q, k, v, k_pool, g, per_head, R, C, phase, smem, k_keep, lengths,
                               out, idx, lse, status, s);
}

}  // namespace

cudaError_t launch_query_attn(const void* q, const void* k, const void* v, const float* k_pool,
                              pa_dtype dt, const Grid& g, int group, int M, int k_keep,
                              const int32_t* lengths, void* out, int32_t* idx, float* lse,
                              int32_t* status, cudaStream_t s) {
#define PARO_Q(CODE, T, D)                                                                       \
  if (dt == CODE && g.d == D)                                                                    \
    return launch_typed<T, D>(q, k, v, k_pool, g, group, M, k_keep, lengths, out, idx, lse,      \
                              status, s);
  PARO_Q(PA_BF16, __nv_bfloat16, 64)
  PARO_Q(PA_BF16, __nv_bfloat16, 128)
  PARO_Q(PA_F32, float, 64)
  PARO_Q(PA_F32, float, 128)
#undef PARO_Q
  return cudaErrorInvalidValue;
}

}  // namespace paro
