// The forward pass of training attention (with its log-sum-exp) at block 64 on
// the warp-level tensor-core path (mma.sync m16n8k16, bf16 operands, fp32
// sums).  (A tcgen05 tile has 128 rows, or 64 in half of the lanes, where the
// softmax then takes as long.)
//
// A CTA owns a block of 64 rows and goes over the 64-column tiles of its
// list, the next tiles on their way (cp.async) while it works on this one.
// Eight warps: warp w owns rows 16 (w % 4) .. +15 and the columns
// 32 (w / 4) .. +31 of every tile; the two column halves keep their own sums
// and join once at the end.  Long lists are bound by mma.sync (307200 tiles
// at d = 64: 1.43 ms, 1275 cycles of an SM a tile, 1024 of them products);
// short ones by latency: 1280 tiles of 128 lists take 12.4 us, 33 us with one
// tile in flight and four warps a CTA.
#include "bwd.cuh"
#include "sm100.cuh"

namespace paro {
namespace {

constexpr int kBlock = 64;
constexpr int kThreads = 256;
// tiles of a list on their way or in use: their loads take longer than a
// tile's work
template <int D>
constexpr int kStages = D == 64 ? 4 : 3;

__device__ __forceinline__ void ldsm4(const void* p, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(sm100::smem_u32(p)));
}
__device__ __forceinline__ void ldsm4t(const void* p, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(sm100::smem_u32(p)));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A tile of 64 rows of D elements, padded against bank conflicts.
template <int D>
constexpr int kLd = D + 8;
template <int D>
constexpr int kTileElems = kBlock * kLd<D>;

template <int D>
__device__ __forceinline__ void fetch_tile(__nv_bfloat16* dst, const __nv_bfloat16* src) {
  constexpr int VPR = D / 8;
#pragma unroll
  for (int e = threadIdx.x; e < kBlock * VPR; e += kThreads)
    sm100::cp_async16(sm100::smem_u32(dst + (e / VPR) * kLd<D> + (e % VPR) * 8), src + e * 8, 16u);
}
__device__ __forceinline__ void fetch_end() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int D>
__device__ __forceinline__ int next_stage(int s) {
  return s == kStages<D> - 1 ? 0 : s + 1;
}

// The A fragments of a warp's 16 rows (row0 on) at k-step ks of a tile.
template <int D>
__device__ __forceinline__ void a_frag(const __nv_bfloat16* tile, int row0, int ks, int lane,
                                       uint32_t (&f)[4]) {
  ldsm4(tile + (row0 + lane % 16) * kLd<D> + ks * 16 + (lane / 16) * 8, f);
}
// B fragments (two k-steps from ks) of the 8 columns from tile row c0.
template <int D>
__device__ __forceinline__ void b_frag(const __nv_bfloat16* tile, int c0, int ks, int lane,
                                       uint32_t (&f)[4]) {
  ldsm4(tile + (c0 + lane % 8) * kLd<D> + ks * 16 + (lane / 8) * 8, f);
}
// B fragments of the 16 tile rows from r0 as the k dimension: columns n0
// (f[0], f[1]) and n0 + 8 (f[2], f[3]).
template <int D>
__device__ __forceinline__ void bt_frag(const __nv_bfloat16* tile, int r0, int n0, int lane,
                                        uint32_t (&f)[4]) {
  ldsm4t(tile + (r0 + (lane % 8) + ((lane / 8) % 2) * 8) * kLd<D> + n0 + (lane / 16) * 8, f);
}

// 16 x D sums of a warp, times mul, as bf16 rows of a padded tile.
template <int D>
__device__ __forceinline__ void stage_rows(__nv_bfloat16* stage, const float (&acc)[D / 8][4],
                                           int row0, int lane, float mul) {
#pragma unroll
  for (int n = 0; n < D / 8; ++n) {
    const int c = n * 8 + 2 * (lane % 4), r = row0 + lane / 4;
    *reinterpret_cast<uint32_t*>(stage + r * kLd<D> + c) =
        sm100::pack_bf16(acc[n][0] * mul, acc[n][1] * mul);
    *reinterpret_cast<uint32_t*>(stage + (r + 8) * kLd<D> + c) =
        sm100::pack_bf16(acc[n][2] * mul, acc[n][3] * mul);
  }
}
// The staged rows of block t to their tokens' natural positions.
template <int D>
__device__ __forceinline__ void store_rows(const __nv_bfloat16* stage, __nv_bfloat16* dst,
                                           const Grid& g, int order, int64_t bh, int t) {
  constexpr int VPR = D / 8;
  for (int e = threadIdx.x; e < kBlock * VPR; e += kThreads) {
    const int r = e / VPR, c = e % VPR, p = t * kBlock + r;
    if (p >= g.N) continue;
    reinterpret_cast<uint4*>(dst + (bh * g.N + natural_index(g, order, p)) * D)[c] =
        *reinterpret_cast<const uint4*>(stage + r * kLd<D> + c * 8);
  }
}
// The second column half's sums, handed to the first through shared memory
// (one float per thread and element).
template <int D>
__device__ __forceinline__ void join(float (&acc)[D / 8][4], float* pass, int half) {
  float* mine = pass + (threadIdx.x & 127);
  if (half == 1)
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) mine[(n * 4 + e) * 128] = acc[n][e];
  __syncthreads();
  if (half == 0)
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] += mine[(n * 4 + e) * 128];
  __syncthreads();
}

template <int D>
constexpr int kFwdSmem = (1 + 2 * kStages<D>) * kTileElems<D> * 2;
static_assert(kFwdSmem<64> - kTileElems<64> * 2 >= 128 * (64 / 2) * 4, "join");
static_assert(kFwdSmem<128> - kTileElems<128> * 2 >= 128 * (128 / 2) * 4, "join");

template <int D>
__global__ void __launch_bounds__(kThreads)
    fwd_lse_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                   const __nv_bfloat16* __restrict__ v, const __grid_constant__ Grid g,
                   const int32_t* __restrict__ idx, const int32_t* __restrict__ counts, int k_max,
                   float scale_log2, __nv_bfloat16* __restrict__ out, float* __restrict__ lse,
                   int32_t* __restrict__ status) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __nv_bfloat16* Qs = reinterpret_cast<__nv_bfloat16*>(smem_raw);
  __nv_bfloat16* KV = Qs + kTileElems<D>;  // the stages of K, V
  __shared__ float maxima[2][kBlock], sums[2][kBlock];  // of the column halves
  const int t = blockIdx.x;
  const int64_t bh = blockIdx.y;
  const int order = g.perm[(int)(bh % g.heads)];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int half = warp / 4, row_w = (warp % 4) * 16, c0 = half * 32;
  const int64_t head = bh * g.Np, row = bh * g.NB + t;
  const int cnt = counts != nullptr ? __ldg(counts + row) : k_max;
  const int32_t* ids = idx + row * k_max;
  fetch_tile<D>(Qs, q + (head + t * kBlock) * D);
  if (!list_ok(ids, cnt, k_max, g.NB, lane)) {  // every warp alike
    if (threadIdx.x == 0) report(status, PA_ERR_DEVICE_CHECK);
    fetch_end();
    fetch_wait<0>();
    return;
  }
  auto fetch = [&](int e, int stage) {
    if (e < cnt) {
      const int64_t at = (head + (int64_t)__ldg(ids + e) * kBlock) * D;
      __nv_bfloat16* to = KV + stage * 2 * kTileElems<D>;
      fetch_tile<D>(to, k + at);
      fetch_tile<D>(to + kTileElems<D>, v + at);
    }
    fetch_end();
  };
#pragma unroll
  for (int e = 0; e < kStages<D> - 1; ++e) fetch(e, e);  // the first with Q
  float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  int stage = 0;
  for (int e = 0; e < cnt; ++e) {
    fetch_wait<kStages<D> - 2>();
    // this tile is here for every warp, and the one before it is consumed
    __syncthreads();
    fetch(e + kStages<D> - 1, stage == 0 ? kStages<D> - 1 : stage - 1);
    const __nv_bfloat16* Ks = KV + stage * 2 * kTileElems<D>;
    stage = next_stage<D>(stage);
    const __nv_bfloat16* Vs = Ks + kTileElems<D>;
    float s[4][4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ks += 2) {
      uint32_t a0[4], a1[4];
      a_frag<D>(Qs, row_w, ks, lane, a0);
      a_frag<D>(Qs, row_w, ks + 1, lane, a1);
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        uint32_t b[4];
        b_frag<D>(Ks, c0 + nt * 8, ks, lane, b);
        mma16816(s[nt], a0, b[0], b[1]);
        mma16816(s[nt], a1, b[2], b[3]);
      }
    }
    const int first = __ldg(ids + e) * kBlock + c0 + 2 * (lane % 4);
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        // pad keys get no weight
        s[nt][x] = first + nt * 8 + (x & 1) < g.N ? s[nt][x] * scale_log2 : -INFINITY;
        mx[x >> 1] = fmaxf(mx[x >> 1], s[nt][x]);
      }
    float ref[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
      mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
      ref[u] = mx[u] == -INFINITY ? 0.f : mx[u];
      const float alpha = sm100::ex2(m[u] - ref[u]);
      m[u] = mx[u];
      l[u] *= alpha;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][2 * u] *= alpha;
        o[n][2 * u + 1] *= alpha;
      }
    }
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        s[nt][x] = sm100::ex2(s[nt][x] - ref[x >> 1]);
        l[x >> 1] += s[nt][x];
      }
    // P rounded to bf16 for its product (2^-8 of each weight, as the
    // rounding of the result); the sums l are of the unrounded weights
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      uint32_t a[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        a[u] = sm100::pack_bf16(s[2 * ks + (u >> 1)][2 * (u & 1)],
                                s[2 * ks + (u >> 1)][2 * (u & 1) + 1]);
#pragma unroll
      for (int n = 0; n < D / 8; n += 2) {
        uint32_t b[4];
        bt_frag<D>(Vs, c0 + ks * 16, n * 8, lane, b);
        mma16816(o[n], a, b[0], b[1]);
        mma16816(o[n + 1], a, b[2], b[3]);
      }
    }
  }
  fetch_wait<0>();
  // ---- join the column halves, normalise, store
  const int r = row_w + lane / 4;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
    l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
    if (lane % 4 == 0) {
      maxima[half][r + 8 * u] = m[u];
      sums[half][r + 8 * u] = l[u];
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int x = r + 8 * u;
    const float mm = fmaxf(maxima[0][x], maxima[1][x]), ref = mm == -INFINITY ? 0.f : mm;
    const float sum =
        sums[0][x] * sm100::ex2(maxima[0][x] - ref) + sums[1][x] * sm100::ex2(maxima[1][x] - ref);
    const float weight = sum == 0.f ? 0.f : sm100::ex2(m[u] - ref) / sum;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      o[n][2 * u] *= weight;
      o[n][2 * u + 1] *= weight;
    }
    const int p = t * kBlock + x;
    if (half == 0 && lane % 4 == 0 && p < g.N)
      lse[bh * g.N + natural_index(g, order, p)] = row_lse(mm, sum);
  }
  join<D>(o, reinterpret_cast<float*>(KV), half);
  if (half == 0) stage_rows<D>(Qs, o, row_w, lane, 1.f);
  __syncthreads();
  store_rows<D>(Qs, out, g, order, bh, t);
}

template <int D>
cudaError_t launch_fwd(const BwdArgs& a, const Grid& g, void* out, float* lse, cudaStream_t s) {
  const cudaError_t e = opt_in_smem<fwd_lse_kernel<D>>(kFwdSmem<D>);
  if (e != cudaSuccess) return e;
  fwd_lse_kernel<D><<<dim3(g.NB, g.B * g.heads), kThreads, kFwdSmem<D>, s>>>(
      a.q, a.k, a.v, g, a.idx, a.counts, a.k_max, (float)(1.4426950408889634 / sqrt((double)D)),
      static_cast<__nv_bfloat16*>(out), lse, a.status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fwd_lse_mma(const BwdArgs& a, const Grid& g, void* out, float* lse,
                               cudaStream_t s) {
  return g.d == 64 ? launch_fwd<64>(a, g, out, lse, s) : launch_fwd<128>(a, g, out, lse, s);
}

}  // namespace paro
