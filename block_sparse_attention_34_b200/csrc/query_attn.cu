// Block-sparse attention of single query tokens over a stored clip: each
// query row scores the clip's blocks by q . kbar_j (kbar_j the block's mean
// key), keeps the k best and attends to their tokens,
//   out = sum_c softmax_c(q . k_c / sqrt(d)) v_c  over the kept blocks' keys.
//
// A row reads NB block means and k blocks of keys and values and does two
// flops a byte: it is bound by HBM, and by latency where a call has few
// rows.  So the whole row is one launch: a cluster of CTAs splits the means
// (scores exchanged through distributed shared memory), each CTA repeats
// the cheap selection, takes an equal share of the kept rows, and the
// partial softmax states (maximum, sum, weighted values) join in the first
// CTA's shared memory.  No workspace, no atomics, one order of every sum.
//
// The scores are summed in 64 bits: a row keeps or drops whole blocks by
// them, and the order of a 32-bit sum would decide near ties.  Keys, values
// and the softmax are 32-bit sums.
#include "common.cuh"

namespace paro {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLoads = 8;  // 16-byte loads of K, and of V, in flight per thread
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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

// Order-preserving map of a score to 64 bits (NaN as -inf, -0 as +0).
__device__ __forceinline__ uint64_t score_key(double s) {
  if (s != s) s = -INFINITY;
  const uint64_t b = (uint64_t)__double_as_longlong(s + 0.0);
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The selection's threshold so far.
struct Select {
  uint64_t prefix;  // its leading bits
  int need;         // how many of the keys that share them are kept (< 0: all)
};

// Dynamic shared memory: keys [NB] u64, list [NB] int32.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2)
    query_attn_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                      const float* __restrict__ k_pool, int heads, int group, int M, int N, int NB,
                      int block, int k_keep, const int32_t* __restrict__ lengths, float scale_log2,
                      T* __restrict__ out, int32_t* __restrict__ idx, float* __restrict__ lse,
                      int32_t* __restrict__ status) {
  constexpr int E = Chunk<T>::n;       // elements of a 16-byte chunk
  constexpr int LPR = D / E;           // lanes of a row
  constexpr int RPL = 32 / LPR;        // rows of one warp load
  constexpr int RPB = RPL * kLoads;    // rows of a batch: divides the block (64 or 128)
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint64_t* keys = reinterpret_cast<uint64_t*>(smem_raw);
  int32_t* list = reinterpret_cast<int32_t*>(keys + NB);
  __shared__ uint32_t hist[256];
  __shared__ int warp_gt[kWarps], warp_eq[kWarps];
  __shared__ Select sel;
  __shared__ float part[kWarps][D + 2];          // the warps' states
  __shared__ float joined[kMaxCluster][D + 2];   // rank 0: the CTAs' states

  const uint32_t C = cluster_size(), rank = cluster_rank();
  const int64_t row = blockIdx.x / C;  // (b * heads * group + hq) * M + m
  const int64_t bh = row / M / group;  // b * heads + key head
  const int b = (int)(bh / heads);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int len = lengths != nullptr ? __ldg(lengths + b) : N;
  if (len < 0 || len > N) {  // the cluster's CTAs alike
    if (rank == 0 && threadIdx.x == 0) report(status, PA_ERR_DEVICE_CHECK);
    return;
  }
  const int nb = (len + block - 1) / block;
  const int kept = min(k_keep, nb);
  if (kept == 0) {
    if (rank == 0) {
      for (int e = threadIdx.x; e < D; e += kThreads) out[row * D + e] = from_float<T>(0.f);
      for (int e = threadIdx.x; e < k_keep; e += kThreads) idx[row * k_keep + e] = -1;
      if (threadIdx.x == 0 && lse != nullptr) lse[row] = -INFINITY;
    }
    return;
  }

  // ---- scores of the blocks j = rank, rank + C, ...: a warp a block
  cluster_arrive();
  {
    constexpr int F = D / 32;  // elements of a lane
    double qd[F];
#pragma unroll
    for (int e = 0; e < F; ++e) qd[e] = (double)to_float(q[row * D + lane * F + e]);
    const float* pool = k_pool + bh * (int64_t)NB * D + lane * F;
    const int step = (int)C * kWarps;
    constexpr int kAhead = 4;
    cluster_wait();  // every CTA runs: its shared memory may be written
    for (int j0 = (int)rank + (int)C * warp; j0 < nb; j0 += step * kAhead) {
      float f[kAhead][F];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int j = min(j0 + u * step, nb - 1);
        if constexpr (F == 4) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(pool + (int64_t)j * D));
          f[u][0] = x.x;
          f[u][1] = x.y;
          f[u][2] = x.z;
          f[u][3] = x.w;
        } else {
          const float2 x = __ldg(reinterpret_cast<const float2*>(pool + (int64_t)j * D));
          f[u][0] = x.x;
          f[u][1] = x.y;
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int j = j0 + u * step;
        double s = 0.0;
#pragma unroll
        for (int e = 0; e < F; ++e) s = fma(qd[e], (double)f[u][e], s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (j < nb && lane < (int)C) st_cluster(map_rank(keys + j, lane), score_key(s));
      }
    }
  }
  cluster_arrive();
  cluster_wait();

  // ---- the kept-th largest key, eight bits at a time from the top; done
  // early once every key that shares the prefix is kept
  if (threadIdx.x == 0) sel = Select{0, kept};
  uint64_t prefix = 0;
  int need = kept, shift = 56;
  bool whole = kept == nb;  // every key is kept
  for (; !whole && shift >= 0; shift -= 8) {
    hist[threadIdx.x] = 0;
    __syncthreads();
    const uint64_t top = shift == 56 ? 0 : ~0ull << (shift + 8);
    for (int j = threadIdx.x; j < nb; j += kThreads)
      if ((keys[j] & top) == prefix) atomicAdd(&hist[(keys[j] >> shift) & 255], 1u);
    __syncthreads();
    if (warp == 0) {
      // lane l holds the bins 255 - 8l .. 248 - 8l; the bin where the count
      // from the top reaches need
      uint32_t n[8], total = 0;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        n[x] = hist[255 - 8 * lane - x];
        total += n[x];
      }
      uint32_t upto = total;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += t;
      }
      uint32_t above = upto - total;
      if (above < (uint32_t)need && upto >= (uint32_t)need) {  // one lane
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          if (above < (uint32_t)need && above + n[x] >= (uint32_t)need) {
            sel.prefix = prefix | ((uint64_t)(255 - 8 * lane - x) << shift);
            // negative: all n[x] keys of this bin are kept
            sel.need = above + n[x] == (uint32_t)need ? -1 : need - (int)above;
            above = 0x7fffffffu;  // found
          } else if (above < (uint32_t)need) {
            above += n[x];
          }
        }
      }
    }
    __syncthreads();
    prefix = sel.prefix;
    if (sel.need < 0) {
      whole = true;
      break;
    }
    need = sel.need;
    __syncthreads();  // hist and sel are reused
  }
  // kept: keys >= prefix when whole (with shift at the prefix's last digit),
  // else keys > prefix and the first `need` keys equal to it
  {
    const int per = ((nb + kThreads - 1) / kThreads) * 32;  // a warp's run of blocks
    const int lo = warp * per, hi = min(nb, lo + per);
    const uint64_t from = prefix;
    int gt = 0, eq = 0;
    for (int j0 = lo; j0 < hi; j0 += 32) {
      const int j = j0 + lane;
      const uint64_t key = j < hi ? keys[j] : 0;
      gt += __popc(__ballot_sync(0xffffffffu, j < hi && (whole ? key >= from : key > from)));
      eq += __popc(__ballot_sync(0xffffffffu, j < hi && !whole && key == from));
    }
    if (lane == 0) {
      warp_gt[warp] = gt;
      warp_eq[warp] = eq;
    }
    __syncthreads();
    int ties = 0, at = 0;
    for (int w = 0; w < warp; ++w) {
      at += warp_gt[w] + min(warp_eq[w], max(0, need - ties));
      ties += warp_eq[w];
    }
    for (int j0 = lo; j0 < hi; j0 += 32) {
      const int j = j0 + lane;
      const uint64_t key = j < hi ? keys[j] : 0;
      const bool tie = j < hi && !whole && key == from;
      const uint32_t tb = __ballot_sync(0xffffffffu, tie);
      const uint32_t before = (1u << lane) - 1u;
      const bool use = j < hi && ((whole ? key >= from : key > from) ||
                                  (tie && ties + __popc(tb & before) < need));
      const uint32_t ub = __ballot_sync(0xffffffffu, use);
      if (use) list[at + __popc(ub & before)] = j;
      at += __popc(ub);
      ties += __popc(tb);
    }
    __syncthreads();
  }
  if (rank == 0)
    for (int e = threadIdx.x; e < k_keep; e += kThreads)
      idx[row * k_keep + e] = e < kept ? list[e] : -1;

  // ---- attention over this CTA's share of the batches of RPB kept rows.
  // LPR lanes hold a row's chunks; every row group keeps its own softmax
  // state, so nothing is exchanged until the end
  const int c = lane % LPR;
  float qf[E];
  {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(q + row * D) + c);
    Chunk<T>::unpack(u, qf);
#pragma unroll
    for (int e = 0; e < E; ++e) qf[e] *= scale_log2;
  }
  const int per_block = block / RPB;
  const int items = kept * per_block;
  const int first = (int)((int64_t)items * rank / C), last = (int)((int64_t)items * (rank + 1) / C);
  const int64_t base = bh * (int64_t)NB * block;
  float o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int it = first + warp; it < last; it += kWarps) {
    const int p0 = list[it / per_block] * block + (it % per_block) * RPB + lane / LPR;
    const uint4* ks = reinterpret_cast<const uint4*>(k + (base + p0) * D) + c;
    const uint4* vs = reinterpret_cast<const uint4*>(v + (base + p0) * D) + c;
    uint4 kr[kLoads], vr[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) kr[u] = __ldg(ks + u * RPL * LPR);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) vr[u] = __ldg(vs + u * RPL * LPR);
    float s[kLoads];
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
    float mx = m;
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      if (p0 + u * RPL >= len) s[u] = -INFINITY;  // behind the clip's end
      mx = fmaxf(mx, s[u]);
    }
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float alpha = ex2f(m - ref);
    m = mx;
    l *= alpha;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= alpha;
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const float p = ex2f(s[u] - ref);
      l += p;
      float f[E];
      Chunk<T>::unpack(vr[u], f);
#pragma unroll
      for (int e = 0; e < E; ++e)
        // a row behind the end has weight 0 whatever its bits are
        o[e] = p > 0.f ? fmaf(p, f[e], o[e]) : o[e];
    }
  }

  // ---- join the row groups of a warp, the warps, the CTAs
#pragma unroll
  for (int off = LPR; off < 32; off <<= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, off);
    const float l2 = __shfl_xor_sync(0xffffffffu, l, off);
    const float mm = fmaxf(m, m2), ref = mm == -INFINITY ? 0.f : mm;
    const float w1 = ex2f(m - ref), w2 = ex2f(m2 - ref);
    l = l * w1 + l2 * w2;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * w1 + __shfl_xor_sync(0xffffffffu, o[e], off) * w2;
    m = mm;
  }
  if (lane < LPR) {
#pragma unroll
    for (int e = 0; e < E; ++e) part[warp][c * E + e] = o[e];
    if (lane == 0) {
      part[warp][D] = m;
      part[warp][D + 1] = l;
    }
  }
  __syncthreads();
  if (threadIdx.x < D) {
    const int e = threadIdx.x;
    float mm = -INFINITY;
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, part[w][D]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float os = 0.f, ls = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float wt = ex2f(part[w][D] - ref);
      os += part[w][e] * wt;
      ls += part[w][D + 1] * wt;
    }
    const uint32_t dst = map_rank(joined[rank], 0);
    st_cluster(dst + e * 4, os);
    if (e == 0) {
      st_cluster(dst + D * 4, mm);
      st_cluster(dst + (D + 1) * 4, ls);
    }
  }
  cluster_arrive();
  cluster_wait();
  if (rank == 0 && threadIdx.x < D) {
    const int e = threadIdx.x;
    float mm = -INFINITY;
    for (uint32_t w = 0; w < C; ++w) mm = fmaxf(mm, joined[w][D]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float os = 0.f, ls = 0.f;
    for (uint32_t w = 0; w < C; ++w) {
      const float wt = ex2f(joined[w][D] - ref);
      os += joined[w][e] * wt;
      ls += joined[w][D + 1] * wt;
    }
    // no sum: every kept key scored -inf
    out[row * D + e] = from_float<T>(ls == 0.f ? 0.f : os / ls);
    if (e == 0 && lse != nullptr) lse[row] = (mm + log2f(ls)) * kLn2;
  }
}

template <typename T, int D>
cudaError_t launch_typed(const void* q, const void* k, const void* v, const float* k_pool,
                         const Grid& g, int group, int M, int k_keep, const int32_t* lengths,
                         void* out, int32_t* idx, float* lse, int32_t* status, cudaStream_t s) {
  auto kern = query_attn_kernel<T, D>;
  const size_t smem = (size_t)g.NB * 12;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)g.B * g.heads * group * M;
  int cluster = 1;
  while (cluster < kMaxCluster && rows * cluster < 2 * 148) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const T*>(q), static_cast<const T*>(k),
                            static_cast<const T*>(v), k_pool, g.heads, group, M, g.N, g.NB, g.block,
                            k_keep, lengths, (float)(kLog2e / sqrt((double)D)),
                            static_cast<T*>(out), idx, lse, status);
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
