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
// blocks that keep a key block, so each is computed by the owner of its sums
// (attn_bwd_sm100.cu for block 128, attn_bwd64_sm100.cu for block 64):
// no atomics, the same bits on every run, at the price of computing S and dP
// twice (7 products a tile instead of 5; an fp32 dQ of 64 KB a tile added
// through L2 would cost about as much as the two products).
//
// Preparation: dO is copied to the permuted order with each row's -lse (log2
// units) and -D beside it, pad rows and rows whose log-sum-exp is -inf with
// -inf, so that they drop out of every sum as P = 0; the kept lists are
// transposed to one bit per (key block, query block).  One launch, and one for
// both gradient kernels: a small call is bound by its launches.
#include "bwd.cuh"

namespace paro {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

constexpr int kBits = 4096;  // key blocks whose bits a CTA collects at a time

// CTAs x < words: 32 query blocks' kept lists of one head (a warp a list, in
// turn) -> word x of every key block's row of the transposed mask, collected
// in shared memory, so the mask needs no clearing, and how many entries each
// list has (-1: malformed, which is reported and sets nothing).  The other
// CTAs: a group of d/8 lanes per permuted row reads O and dO at the row's
// natural position (16 bytes a lane), writes dO permuted and the row's
// statistics; bound by HBM, two reads and a write of the tensor (12 heads of
// 32,760 rows at d = 128: 56 us, 5.4 TB/s).
template <int D>
__global__ void __launch_bounds__(kThreads)
    bwd_prep_kernel(const __nv_bfloat16* __restrict__ out, const __nv_bfloat16* __restrict__ dout,
                    const float* __restrict__ lse, const float* __restrict__ dlse,
                    const __grid_constant__ Grid g, const int32_t* __restrict__ idx,
                    const int32_t* __restrict__ counts, int k_max, int words,
                    __nv_bfloat16* __restrict__ dop, float* __restrict__ nlse,
                    float* __restrict__ ndel, uint32_t* __restrict__ mask,
                    int32_t* __restrict__ checked, int32_t* __restrict__ counters,
                    int32_t* __restrict__ status) {
  const int64_t bh = blockIdx.y;
  if (blockIdx.x == 0 && bh == 0 && threadIdx.x < 2) counters[threadIdx.x] = 0;
  if ((int)blockIdx.x < words) {
    __shared__ uint32_t bits[kBits];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int i0 = blockIdx.x * 32;
    for (int j0 = 0; j0 < g.NB; j0 += kBits) {
      const int n = min(kBits, g.NB - j0);
      for (int j = threadIdx.x; j < n; j += kThreads) bits[j] = 0u;
      __syncthreads();
      for (int i = i0 + warp; i < min(g.NB, i0 + 32); i += kThreads / 32) {
        const int64_t row = bh * g.NB + i;
        const int cnt = counts != nullptr ? __ldg(counts + row) : k_max;
        const int32_t* ids = idx + row * k_max;
        const bool fine = list_ok(ids, cnt, k_max, g.NB, lane);
        if (lane == 0) {
          checked[row] = fine ? cnt : -1;
          if (!fine) report(status, PA_ERR_DEVICE_CHECK);
        }
        if (!fine) continue;
        for (int e = lane; e < cnt; e += 32) {
          const int j = __ldg(ids + e) - j0;
          if (j >= 0 && j < n) atomicOr(bits + j, 1u << (i & 31));
        }
      }
      __syncthreads();
      for (int j = threadIdx.x; j < n; j += kThreads)
        mask[(bh * g.NB + j0 + j) * words + blockIdx.x] = bits[j];
      __syncthreads();
    }
    return;
  }
  constexpr int VPR = D / 8;
  const int c = threadIdx.x % VPR;
  const int order = g.perm[(int)(bh % g.heads)];
  const int p = (blockIdx.x - words) * (kThreads / VPR) + threadIdx.x / VPR;
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
    // a row whose keys all scored -inf has no weights either
    const float x = row >= 0 ? __ldg(lse + row) : -INFINITY;
    nlse[prow] = x == -INFINITY ? -INFINITY : -x * kLog2e;
    ndel[prow] = row >= 0 ? (dlse != nullptr ? __ldg(dlse + row) : 0.f) - s : 0.f;
  }
}

}  // namespace

cudaError_t launch_bwd_prep(const void* out, const void* dout, const float* lse,
                            const float* dlse, const BwdArgs& a, const Grid& g, cudaStream_t s) {
  const int per = kThreads / (g.d / 8);
  const dim3 grid(a.words + (g.Np + per - 1) / per, g.B * g.heads);
  auto* o = static_cast<const __nv_bfloat16*>(out);
  auto* d = static_cast<const __nv_bfloat16*>(dout);
  auto kern = g.d == 64 ? bwd_prep_kernel<64> : bwd_prep_kernel<128>;
  kern<<<grid, kThreads, 0, s>>>(o, d, lse, dlse, g, a.idx, a.counts, a.k_max, a.words, a.dop, a.nlse,
                                 a.ndel, a.mask, a.checked, a.counters, a.status);
  return cudaGetLastError();
}

}  // namespace paro
