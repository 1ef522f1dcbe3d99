// Backward pass of block-sparse attention: its formulas and its preparation.
//
// With S = Q K^T / sqrt(d), P = exp(S - lse) over the kept tiles, O = P V,
// and the gradients dO of O and dlse of lse:
//   D_r  = sum_c dO_rc O_rc - dlse_r
//   dP   = dO V^T,  dS = P o (dP - D)
//   dQ   = dS K / sqrt(d),  dK = dS^T Q / sqrt(d),  dV = P^T dO.
// P needs no running maximum here: lse is known from the forward pass.
//
// dQ sums over a query block's kept key blocks, dK and dV over the query
// blocks that keep a key block, so two kernels (attn_bwd_sm100.cu for block
// 128, attn_train_mma.cu for block 64), each the owner of its sums:
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

}  // namespace paro
