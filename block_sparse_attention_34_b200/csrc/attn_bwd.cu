// Backward pass of block-sparse attention: its preparation (for every shape)
// and the two gradient kernels on the warp-level tensor-core path.
//
// With S = Q K^T / sqrt(d), P = exp(S - lse) over the kept tiles, O = P V,
// and the gradients dO of O and dlse of lse:
//   D_r  = sum_c dO_rc O_rc - dlse_r
//   dP   = dO V^T,  dS = P o (dP - D)
//   dQ   = dS K / sqrt(d),  dK = dS^T Q / sqrt(d),  dV = P^T dO.
// P needs no running maximum here: lse is known from the forward pass.
//
// dQ sums over a query block's kept key blocks, dK and dV over the query
// blocks that keep a key block, so two kernels, each the owner of its sums:
// no atomics, the same bits on every run, at the price of computing S and dP
// twice (7 products a tile instead of 5; an fp32 dQ of 64 KB a tile added
// through L2 would cost about as much as the two products).
//
// Preparation: dO is copied to the permuted order with each row's -lse (log2
// units) and -D beside it, pad rows as (-inf, 0) so that they drop out of
// every sum as P = 0; the kept lists are transposed to one bit per (key
// block, query block).
#include "bwd.cuh"

namespace paro {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

// One group of d/8 lanes per permuted row: reads O and dO at the row's
// natural position (16 bytes a lane), writes dO permuted and the row's
// statistics.  Bound by HBM: two reads and a write of the tensor.
template <int D>
__global__ void __launch_bounds__(kThreads)
    bwd_prep_kernel(const __nv_bfloat16* __restrict__ out, const __nv_bfloat16* __restrict__ dout,
                    const float* __restrict__ lse, const float* __restrict__ dlse,
                    const __grid_constant__ Grid g, __nv_bfloat16* __restrict__ dop,
                    float* __restrict__ nlse, float* __restrict__ ndel) {
  constexpr int VPR = D / 8;
  const int c = threadIdx.x % VPR;
  const int64_t bh = blockIdx.y;
  const int order = g.perm[(int)(bh % g.heads)];
  const int p = blockIdx.x * (kThreads / VPR) + threadIdx.x / VPR;
  if (p >= g.Np) return;  // Np is a multiple of a CTA's rows: uniform
  uint4 o = make_uint4(0, 0, 0, 0), d = o;
  int64_t row = -1;
  if (p < g.N) {
    row = bh * g.N + natural_index(g, order, p);
    o = __ldg(reinterpret_cast<const uint4*>(out + row * D) + c);
    d = __ldg(reinterpret_cast<const uint4*>(dout + row * D) + c);
  }
  float fo[8], fd[8], s = 0.f;
  Chunk<__nv_bfloat16>::unpack(o, fo);
  Chunk<__nv_bfloat16>::unpack(d, fd);
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fmaf(fo[e], fd[e], s);
#pragma unroll
  for (int off = VPR / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  const int64_t prow = bh * g.Np + p;
  reinterpret_cast<uint4*>(dop + prow * D)[c] = d;
  if (c == 0) {
    nlse[prow] = row >= 0 ? -__ldg(lse + row) * kLog2e : -INFINITY;
    ndel[prow] = row >= 0 ? (dlse != nullptr ? __ldg(dlse + row) : 0.f) - s : 0.f;
  }
}

// One warp per query block's kept list: checks it, then sets bit i of row j
// of the transposed mask for every kept j (zeroed before).  A malformed list
// is reported and sets nothing.
__global__ void __launch_bounds__(kThreads)
    transpose_lists_kernel(const int32_t* __restrict__ idx, const int32_t* __restrict__ counts,
                           int k_max, int NB, int words, int64_t rows,
                           uint32_t* __restrict__ mask, int32_t* __restrict__ status) {
  const int lane = threadIdx.x % 32;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (row >= rows) return;
  const int cnt = counts != nullptr ? __ldg(counts + row) : k_max;
  const int32_t* ids = idx + row * k_max;
  if (!list_ok(ids, cnt, k_max, NB, lane)) {
    if (lane == 0) report(status, PA_ERR_DEVICE_CHECK);
    return;
  }
  const int64_t bh = row / NB;
  const int i = (int)(row - bh * NB);
  for (int e = lane; e < cnt; e += 32)
    atomicOr(mask + (bh * NB + __ldg(ids + e)) * words + (i >> 5), 1u << (i & 31));
}

// ------------------------------------------------- warp-level kernels -----

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void ldsm4(const void* p, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(p)));
}
__device__ __forceinline__ void ldsm4t(const void* p, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(p)));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&t);
}

// BLOCK contiguous rows of a permuted tensor into a padded tile.
template <int D, int LD, int BLOCK>
__device__ __forceinline__ void load_tile(__nv_bfloat16* dst, const __nv_bfloat16* __restrict__ src) {
  constexpr int VPR = D / 8;
  for (int e = threadIdx.x; e < BLOCK * VPR; e += blockDim.x)
    *reinterpret_cast<uint4*>(dst + (e / VPR) * LD + (e % VPR) * 8) =
        __ldg(reinterpret_cast<const uint4*>(src) + e);
}

// kKeys: one CTA per key block, dK and dV (rows are keys: A1 = K, A2 = V;
// streamed query blocks: B1 = Q, B2 = dO).  Otherwise one CTA per query
// block, dQ (A1 = Q, A2 = dO; streamed key blocks: B1 = K, B2 = V).  Either
// way X = A1 B1^T are the scores and Y = A2 B2^T is dP, rows by columns of
// the tile, G1 += dS B1 and (kKeys) G2 += P B2.  A warp owns 16 rows and
// goes over the tile 32 columns at a time, so only the sums stay in
// registers.  P and dS are rounded to bf16 for their products (relative
// 2^-8, as the rounding of the results).
template <int D, int BLOCK, bool kKeys>
__global__ void __launch_bounds__(BLOCK * 2)
    bwd_mma_kernel(const __nv_bfloat16* __restrict__ a1, const __nv_bfloat16* __restrict__ a2,
                   const __nv_bfloat16* __restrict__ b1, const __nv_bfloat16* __restrict__ b2,
                   const float* __restrict__ nlse, const float* __restrict__ ndel, const __grid_constant__ Grid g,
                   const int32_t* __restrict__ idx, const int32_t* __restrict__ counts, int k_max,
                   const uint32_t* __restrict__ mask, int words, float scale,
                   __nv_bfloat16* __restrict__ g1, __nv_bfloat16* __restrict__ g2,
                   int32_t* __restrict__ status) {
  constexpr int LD = D + 8;  // padded row: conflict-free ldmatrix
  constexpr int DT = D / 8;
  constexpr int kTileElems = BLOCK * LD;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __nv_bfloat16* A1 = reinterpret_cast<__nv_bfloat16*>(smem_raw);
  __nv_bfloat16* A2 = A1 + kTileElems;
  __nv_bfloat16* B1 = A2 + kTileElems;
  __nv_bfloat16* B2 = B1 + kTileElems;
  float2* st = reinterpret_cast<float2*>(B2 + kTileElems);  // the query rows' (-lse, -D)

  const int t = blockIdx.x;  // this CTA's block
  const int64_t bh = blockIdx.y;
  const int order = g.perm[(int)(bh % g.heads)];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t head = bh * g.Np;
  const int64_t row = bh * g.NB + t;
  const float scale_log2 = scale * kLog2e;

  const int32_t* ids = nullptr;
  int cnt = 0;
  if constexpr (!kKeys) {
    cnt = counts != nullptr ? __ldg(counts + row) : k_max;
    ids = idx + row * k_max;
    if (!list_ok(ids, cnt, k_max, g.NB, lane)) {  // every warp alike
      if (threadIdx.x == 0) report(status, PA_ERR_DEVICE_CHECK);
      return;
    }
  }
  load_tile<D, LD, BLOCK>(A1, a1 + (head + t * BLOCK) * D);
  load_tile<D, LD, BLOCK>(A2, a2 + (head + t * BLOCK) * D);
  float lse_r[2], d_r[2];
  if constexpr (!kKeys) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t at = head + t * BLOCK + warp * 16 + lane / 4 + 8 * u;
      lse_r[u] = __ldg(nlse + at);
      d_r[u] = __ldg(ndel + at);
    }
  }
  float acc1[DT][4], acc2[kKeys ? DT : 1][4];
#pragma unroll
  for (int x = 0; x < DT; ++x)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc1[x][e] = 0.f;
      if constexpr (kKeys) acc2[x][e] = 0.f;
    }

  auto tile = [&](int j) {
    __syncthreads();  // the previous tile is consumed
    load_tile<D, LD, BLOCK>(B1, b1 + (head + (int64_t)j * BLOCK) * D);
    load_tile<D, LD, BLOCK>(B2, b2 + (head + (int64_t)j * BLOCK) * D);
    if constexpr (kKeys)
      for (int e = threadIdx.x; e < BLOCK; e += blockDim.x)
        st[e] = make_float2(__ldg(nlse + head + (int64_t)j * BLOCK + e),
                            __ldg(ndel + head + (int64_t)j * BLOCK + e));
    __syncthreads();
#pragma unroll 1
    for (int c0 = 0; c0 < BLOCK; c0 += 32) {
      float x[4][4], y[4][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][e] = y[nt][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; kk += 2) {
        uint32_t f1[2][4], f2[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int at = (warp * 16 + lane % 16) * LD + (kk + u) * 16 + (lane / 16) * 8;
          ldsm4(A1 + at, f1[u]);
          ldsm4(A2 + at, f2[u]);
        }
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const int at = (c0 + nt * 8 + lane % 8) * LD + kk * 16 + (lane / 8) * 8;
          uint32_t b[4];
          ldsm4(B1 + at, b);
          mma16816(x[nt], f1[0], b[0], b[1]);
          mma16816(x[nt], f1[1], b[2], b[3]);
          ldsm4(B2 + at, b);
          mma16816(y[nt], f2[0], b[0], b[1]);
          mma16816(y[nt], f2[1], b[2], b[3]);
        }
      }
      // x -> P, y -> dS; element e of an n-tile: row lane/4 + 8 (e / 2),
      // column 2 (lane % 4) + e % 2
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = c0 + nt * 8 + 2 * (lane % 4) + (e & 1);
          float l, dd;
          if constexpr (kKeys) {
            const float2 s = st[col];
            l = s.x;
            dd = s.y;
          } else {
            l = lse_r[e >> 1];
            dd = d_r[e >> 1];
          }
          float p = exp2f(fmaf(x[nt][e], scale_log2, l));
          if constexpr (!kKeys)
            if (j * BLOCK + col >= g.N) p = 0.f;  // pad keys
          x[nt][e] = p;
          y[nt][e] = p * (y[nt][e] + dd);
        }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        uint32_t pa[4], sa[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int nt = 2 * ks + (u >> 1), e = 2 * (u & 1);
          sa[u] = pack2(y[nt][e], y[nt][e + 1]);
          if constexpr (kKeys) pa[u] = pack2(x[nt][e], x[nt][e + 1]);
        }
#pragma unroll
        for (int n = 0; n < DT; n += 2) {
          const int at = (c0 + ks * 16 + (lane % 8) + ((lane / 8) % 2) * 8) * LD + n * 8 +
                         (lane / 16) * 8;
          uint32_t b[4];
          ldsm4t(B1 + at, b);
          mma16816(acc1[n], sa, b[0], b[1]);
          mma16816(acc1[n + 1], sa, b[2], b[3]);
          if constexpr (kKeys) {
            ldsm4t(B2 + at, b);
            mma16816(acc2[n], pa, b[0], b[1]);
            mma16816(acc2[n + 1], pa, b[2], b[3]);
          }
        }
      }
    }
  };
  if constexpr (kKeys) {
    const uint32_t* bits = mask + row * words;
    for (int w = 0; w < words; ++w)
      for (uint32_t m = __ldg(bits + w); m != 0; m &= m - 1) tile(w * 32 + __ffs(m) - 1);
  } else {
    for (int e = 0; e < cnt; ++e) tile(__ldg(ids + e));
  }

  // through shared memory to the rows' natural positions
  auto store = [&](const float (&acc)[DT][4], float mul, __nv_bfloat16* dst) {
    __syncthreads();
    __nv_bfloat16* stage = B1;  // [BLOCK][LD]
    const int r0 = warp * 16 + lane / 4;
#pragma unroll
    for (int n = 0; n < DT; ++n) {
      const int c = n * 8 + 2 * (lane % 4);
      *reinterpret_cast<uint32_t*>(stage + r0 * LD + c) = pack2(acc[n][0] * mul, acc[n][1] * mul);
      *reinterpret_cast<uint32_t*>(stage + (r0 + 8) * LD + c) =
          pack2(acc[n][2] * mul, acc[n][3] * mul);
    }
    __syncthreads();
    constexpr int VPR = D / 8;
    for (int e = threadIdx.x; e < BLOCK * VPR; e += blockDim.x) {
      const int r = e / VPR, c = e % VPR, p = t * BLOCK + r;
      if (p >= g.N) continue;
      reinterpret_cast<uint4*>(dst + (bh * g.N + natural_index(g, order, p)) * D)[c] =
          *reinterpret_cast<const uint4*>(stage + r * LD + c * 8);
    }
  };
  store(acc1, scale, g1);
  if constexpr (kKeys) store(acc2, 1.f, g2);
}

template <int D, int BLOCK>
cudaError_t launch_mma(const BwdArgs& a, const Grid& g, cudaStream_t s) {
  const size_t smem = (size_t)4 * BLOCK * (D + 8) * 2 + BLOCK * sizeof(float2);
  const float scale = (float)(1.0 / sqrt((double)D));
  const dim3 grid(g.NB, g.B * g.heads);
  auto kv = bwd_mma_kernel<D, BLOCK, true>;
  auto kq = bwd_mma_kernel<D, BLOCK, false>;
  cudaError_t e = cudaFuncSetAttribute(kv, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kv<<<grid, BLOCK * 2, smem, s>>>(a.k, a.v, a.q, a.dop, a.nlse, a.ndel, g, nullptr, nullptr, 0, a.mask,
                                   a.words, scale, a.dk, a.dv, a.status);
  kq<<<grid, BLOCK * 2, smem, s>>>(a.q, a.dop, a.k, a.v, a.nlse, a.ndel, g, a.idx, a.counts, a.k_max,
                                   nullptr, 0, scale, a.dq, nullptr, a.status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bwd_prep(const void* out, const void* dout, const float* lse,
                            const float* dlse, const BwdArgs& a, const Grid& g, cudaStream_t s) {
  const int64_t rows = (int64_t)g.B * g.heads * g.NB;
  cudaError_t e = cudaMemsetAsync(a.mask, 0, (size_t)rows * a.words * sizeof(uint32_t), s);
  if (e != cudaSuccess) return e;
  if (a.k_max > 0)
    transpose_lists_kernel<<<(unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0,
                             s>>>(a.idx, a.counts, a.k_max, g.NB, a.words, rows, a.mask, a.status);
  const int per = kThreads / (g.d / 8);
  const dim3 grid((g.Np + per - 1) / per, g.B * g.heads);
  auto* o = static_cast<const __nv_bfloat16*>(out);
  auto* d = static_cast<const __nv_bfloat16*>(dout);
  if (g.d == 64)
    bwd_prep_kernel<64><<<grid, kThreads, 0, s>>>(o, d, lse, dlse, g, a.dop, a.nlse, a.ndel);
  else
    bwd_prep_kernel<128><<<grid, kThreads, 0, s>>>(o, d, lse, dlse, g, a.dop, a.nlse, a.ndel);
  return cudaGetLastError();
}

cudaError_t launch_bwd_mma(const BwdArgs& a, const Grid& g, cudaStream_t s) {
  if (g.d == 64) return g.block == 64 ? launch_mma<64, 64>(a, g, s) : launch_mma<64, 128>(a, g, s);
  return g.block == 64 ? launch_mma<128, 64>(a, g, s) : launch_mma<128, 128>(a, g, s);
}

}  // namespace paro
