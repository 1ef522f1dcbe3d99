// The forward pass of training attention (with its log-sum-exp) at block 64 on
// the 5th-generation tensor cores (bf16, d = 64 or 128).
//
// A CTA owns a block of 64 query rows and streams its list two key blocks (128
// rows) a step.  As in the backward pass (attn_bwd64_sm100.cu) the streamed
// rows are the rows of the score product, whichever blocks they come from:
//   X = K Q^T              128 x 64
//   P = 2^(X c - ref)      ref: a reference of the query (X's column)
//   O += P^T V             64 x d, P from shared memory (M-major)
// A thread has one key and 32 queries, so a query's maximum and sum run over
// threads.  The sums are kept per thread and joined once at the end.  The
// maximum is not kept: a query's reference is its maximum over the first step,
// and moves only when some score passes it by more than 2^8, which the threads
// vote on every step; then the columns' maxima are taken over the lanes and
// O and the sums are rescaled.  O and the sums are relative to the same
// reference, so the result does not depend on where it lies.
//
// 10 warps: 0-7 elementwise (warp w: the streamed rows 32 (w % 4) .. +31, the
// queries 32 (w / 4) .. +31; at the end the rows of O), 8 tensor memory and
// MMAs, 9 loads.  Tensor memory: X in two buffers at 0 and
// 64, O at 128, its row r in lane 32 (r / 16) + r % 16.
// Issue order: X0 X1, then for every t: O(t) once P(t) is written, X(t+2).
//
// Bounded by the elementwise work (a score's share of the exponentials is half
// of it) and, with short lists, by a CTA's start and its first step, which
// sets the references.  Measured, d = 64: 307200 tiles 1.03 ms (mma.sync
// 1.43), 1280 tiles of 128 lists 13.0 us (12.4); the same at d = 128 13.1 us
// (19.7).  Two load warps, which leave 80 registers: 1.39 ms.
#include <type_traits>

#include "bwd.cuh"
#include "sm100.cuh"

namespace paro {

namespace {

using namespace sm100;

constexpr int kBlock = 64;
constexpr int kStep = 128;
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kThreads = 10 * 32;  // 96 registers a thread with two CTAs on an SM
constexpr int kAluThreads = 256;
constexpr int kKStages = 3, kVStages = 2;
constexpr uint32_t kOwnHalf = kBlock * 128;
constexpr uint32_t kHalf = kStep * 128;
constexpr uint32_t kTmemCols = 256;
constexpr float kFar = 8.f;  // how far (log2) a score may pass its reference

enum : uint32_t {
  BQ = 0,   // Q loaded
  BK = 1,   // K stage full (3)
  BV = 4,   // V stage full (2)
  BX = 6,   // X(t) complete (ring of 3)
  BO = 9,   // O(t) complete: its K and V stages and P are free (ring of 3)
  BP = 12,  // P(t) written by every elementwise thread
  BDRAIN = 13,
  NBAR = 14
};

template <int D>
struct Lay {
  static constexpr uint32_t kOwn = kBlock * D * 2, kTile = kStep * D * 2;
  static constexpr uint32_t kQ = 0, kK = kOwn, kV = kK + kKStages * kTile,
                            kP = kV + kVStages * kTile, kBar = kP + kHalf,
                            kSlot = kBar + NBAR * 8,   // tensor memory's base, the abort flag
      kIds = kSlot + 8,                                // [stage][2]: the blocks of a step
      kRef = kIds + kKStages * 8,                      // -ref of each query
      kAlpha = kRef + kBlock * 4,                      // its rescaling; at the end its sum
      kPart = kAlpha + kBlock * 4,                     // [lane quarter][query]
      kBytes = kPart + 4 * kBlock * 4;
};
static_assert(2 * (Lay<64>::kBytes + 1024) <= 228 * 1024, "two CTAs on an SM at d = 64");
static_assert(Lay<128>::kBytes <= kSmemOptIn, "shared memory, d = 128");
static_assert(Lay<64>::kRef % 16 == 0, "float4 reads");

// Barriers of the elementwise warps alone.
__device__ __forceinline__ void alu_sync() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(kAluThreads) : "memory");
}
__device__ __forceinline__ bool alu_any(bool x) {
  uint32_t any;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\n"
      "barrier.cta.red.or.pred q, 1, %2, p;\nselp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(any)
      : "r"((uint32_t)x), "n"(kAluThreads)
      : "memory");
  return any != 0;
}

// Lane l: the combination over the warp's lanes of v[l].
template <class F>
__device__ __forceinline__ float over_lanes(float (&v)[32], int lane, F f) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + o], o);
      v[i] = f(up ? v[i + o] : v[i], got);
    }
  return v[0];
}

template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1)
    fwd64_sm100_kernel(const __grid_constant__ CUtensorMap map_q,
                       const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v,
                       const __grid_constant__ Grid g, const int32_t* __restrict__ idx,
                       const int32_t* __restrict__ counts, int k_max, float scale_log2,
                       __nv_bfloat16* __restrict__ out, float* __restrict__ lse,
                       int32_t* __restrict__ status) {
  using L = Lay<D>;
  constexpr uint32_t kColO = 128;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = smem_u32(smem);
  if ((base & 1023u) != 0) {
    if (threadIdx.x == 0) report(status, PA_ERR_UNSUPPORTED);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t bh = blockIdx.y;
  const int blk = blockIdx.x;
  const int head = (int)bh * g.Np;  // first row of the head (all rows: < 2^31)
  const int64_t list = bh * g.NB + blk;
  const int cnt = counts != nullptr ? __ldg(counts + list) : k_max;
  const int32_t* ids = idx + list * k_max;
  const bool fine = list_ok(ids, cnt, k_max, g.NB, lane);
  const bool expired =
      status != nullptr && *reinterpret_cast<volatile int32_t*>(status) == PA_ERR_TIMEOUT;
  // one answer for the CTA: the status may change between its threads' reads
  if (__syncthreads_or(!fine || expired)) {
    if (threadIdx.x == 0 && !fine) report(status, PA_ERR_DEVICE_CHECK);
    return;
  }
  const int n = (cnt + 1) / 2;  // steps
  auto bar = [&](uint32_t slot) { return base + L::kBar + slot * 8u; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kSlot);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  volatile int32_t* step_ids = reinterpret_cast<int32_t*>(smem + L::kIds);
  if (threadIdx.x == 0) {
    for (uint32_t b = 0; b < NBAR; ++b) mbar_init(bar(b), b == BP ? kAluThreads / 32 : 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  float* neg_ref = reinterpret_cast<float*>(smem + L::kRef);
  float* alpha = reinterpret_cast<float*>(smem + L::kAlpha);
  float* part = reinterpret_cast<float*>(smem + L::kPart);
  if (threadIdx.x < kBlock) neg_ref[threadIdx.x] = INFINITY;
  if (warp == kMmaWarp) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Ctl ctl{abort_flag, status, kTimeoutNs};

  if (warp == kLoadWarp) {
    // -------------------------------------------------------- copies ----
    if (lane == 0) {
      mbar_arrive_tx(bar(BQ), L::kOwn);
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
        tma_load_2d(base + L::kQ + h * kOwnHalf, &map_q, 64 * h, head + blk * kBlock, bar(BQ));
    }
    int issued_k = 0, issued_v = 0, id_lane = 0;  // id_lane: entry 32 (e / 32) + lane
    const int end = (int)gridDim.y * g.Np;  // rows behind it read as zero
    auto load = [&](const CUtensorMap* map, uint32_t to, int j0, int j1, uint32_t b) {
      mbar_arrive_tx(b, L::kTile);  // release: the ids are visible behind the barrier
      const int y0 = head + j0 * kBlock, y1 = j1 < 0 ? end : head + j1 * kBlock;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        tma_load_2d(to + h * kHalf, map, 64 * h, y0, b);
        tma_load_2d(to + h * kHalf + kOwnHalf, map, 64 * h, y1, b);
      }
    };
    // the step that had a stage is over: nothing of it is read any more
    auto over = [&](int t) { return t < 0 || warp_wait(bar(BO + t % 3), (t / 3) & 1, ctl); };
    for (int t = 0; t < n; ++t) {
      if ((t & 15) == 0) id_lane = 2 * t + lane < cnt ? __ldg(ids + 2 * t + lane) : -1;
      const int j0 = __shfl_sync(0xffffffffu, id_lane, 2 * t & 31);
      const int j1 = __shfl_sync(0xffffffffu, id_lane, (2 * t & 31) + 1);
      const int sk = t % kKStages, sv = t % kVStages;
      if (!over(t - kKStages)) break;
      if (lane == 0) {
        step_ids[2 * sk] = j0;
        step_ids[2 * sk + 1] = j1;  // -1: an odd list's end, whose second place is zero
        load(&map_k, base + L::kK + sk * L::kTile, j0, j1, bar(BK + sk));
      }
      issued_k = t + 1;
      if (!over(t - kVStages)) break;
      if (lane == 0) load(&map_v, base + L::kV + sv * L::kTile, j0, j1, bar(BV + sv));
      issued_v = t + 1;
    }
    // on every path this warp's copies have landed before it leaves
    if (lane == 0) {
      drain_phase(bar(BQ), 0);
      for (int t = issued_k > kKStages ? issued_k - kKStages : 0; t < issued_k; ++t)
        drain_phase(bar(BK + t % kKStages), (t / kKStages) & 1);
      for (int t = issued_v > kVStages ? issued_v - kVStages : 0; t < issued_v; ++t)
        drain_phase(bar(BV + t % kVStages), (t / kVStages) & 1);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------------- MMA ----
    if (elect_one()) {
      constexpr uint32_t id_x = idesc_bf16(kStep, kBlock, false);
      constexpr uint32_t id_o = idesc_bf16(kBlock, D, true) | (1u << 15);  // A M-major too
      const uint64_t dq = sw128_desc(base + L::kQ, 16, 1024);
      const uint64_t dk = sw128_desc(base + L::kK, 16, 1024);
      const uint64_t dv = sw128_desc(base + L::kV, kHalf, 1024);  // MN-major
      const uint64_t dp = sw128_desc(base + L::kP, kHalf, 1024);
      auto issue_x = [&](int t) -> bool {
        if (!wait_phase(bar(BK + t % kKStages), (t / kKStages) & 1, ctl)) return false;
        tc_fence_after();
        const uint64_t b = dk + (uint64_t)(t % kKStages * (L::kTile >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_f16_ss(tmem + (t & 1) * 64, b + (((kk >> 2) * kHalf + (kk & 3) * 32) >> 4),
                     dq + (((kk >> 2) * kOwnHalf + (kk & 3) * 32) >> 4), id_x, kk > 0 ? 1u : 0u);
        mma_commit(bar(BX + t % kKStages));
        return true;
      };
      bool ok = n > 0 && wait_phase(bar(BQ), 0, ctl) && issue_x(0) && (n < 2 || issue_x(1));
      for (int t = 0; ok && t < n; ++t) {
        ok = wait_phase(bar(BP), t & 1, ctl) &&
             wait_phase(bar(BV + t % kVStages), (t / kVStages) & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        const uint64_t b = dv + (uint64_t)(t % kVStages * (L::kTile >> 4));
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk)
          mma_f16_ss(tmem + kColO, dp + (uint64_t)(kk * 128), b + (uint64_t)(kk * 128), id_o,
                     (t > 0 || kk > 0) ? 1u : 0u);
        mma_commit(bar(BO + t % 3));
        if (t + 2 < n) ok = issue_x(t + 2);
      }
      // every MMA issued above has completed once this commit fires
      mma_commit(bar(BDRAIN));
      drain_phase(bar(BDRAIN), 0);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------- elementwise ----
    // Every thread passes the same barriers: a wait that ran out is known to
    // all of them before one leaves.
    const int quarter = warp & 3, half = warp >> 2;
    const int r = quarter * 32 + lane;  // streamed row of a step
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const float2 sc2 = make_float2(scale_log2, scale_log2);
    const float4* refs = reinterpret_cast<const float4*>(neg_ref) + 8 * half;
    const float4* scales = reinterpret_cast<const float4*>(alpha) + 8 * half;
    uint4* p_row = reinterpret_cast<uint4*>(smem + L::kP + r * 128);
    const int row = 16 * quarter + lane;  // of O, lanes 0-15
    float2 l[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) l[c] = make_float2(0.f, 0.f);
    bool ok = true;
    for (int t = 0; t < n; ++t) {
      ok = all_wait(bar(BK + t % kKStages), (t / kKStages) & 1, ctl);
      const int j = step_ids[2 * (t % kKStages) + (r >> 6)];
      const bool valid = j >= 0 && j * kBlock + (r & 63) < g.N;
      ok = ok && warp_wait(bar(BX + t % kKStages), (t / kKStages) & 1, ctl);
      tc_fence_after();
      uint32_t x[32];
      tmem_ld32(lanes + (t & 1) * 64 + 32 * half, x);
      // scores relative to their references, two queries at a time
      auto score = [&](int c, float2 nr) {
        return ffma2(make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), sc2, nr);
      };
      float top = -INFINITY;
      if (t > 0) {
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          const float4 v = refs[c / 2];
          const float2 a = score(c, make_float2(v.x, v.y)), b = score(c + 1, make_float2(v.z, v.w));
          top = fmax3(top, fmaxf(a.x, a.y), fmaxf(b.x, b.y));
        }
      }
      // P's buffer is free, and O(t - 1) may be rescaled
      if (t > 0) ok = ok && warp_wait(bar(BO + (t - 1) % 3), ((t - 1) / 3) & 1, ctl);
      if (alu_any(t == 0 || !ok || (valid && top > kFar))) {
        if (alu_any(!ok)) {
          ok = false;
          break;
        }
        float m[32];
#pragma unroll
        for (int c = 0; c < 32; ++c)
          m[c] = valid ? __uint_as_float(x[c]) * scale_log2 : -INFINITY;
        part[quarter * kBlock + 32 * half + lane] =
            over_lanes(m, lane, [](float a, float b) { return fmaxf(a, b); });
        alu_sync();
        if (threadIdx.x < kBlock) {
          const int c = threadIdx.x;
          const float mm = fmaxf(fmaxf(part[c], part[kBlock + c]),
                                 fmaxf(part[2 * kBlock + c], part[3 * kBlock + c]));
          // (a reference of -inf, which no score has passed yet, counts as 0)
          const float old = neg_ref[c], now = mm == -INFINITY ? old : fminf(old, -mm);
          alpha[c] = old == INFINITY ? 1.f : ex2(now - old);
          neg_ref[c] = now;
        }
        alu_sync();
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          const float4 v = scales[c / 2];
          l[c] = fmul2(l[c], make_float2(v.x, v.y));
          l[c + 1] = fmul2(l[c + 1], make_float2(v.z, v.w));
        }
        if (t > 0) {
          tc_fence_after();
          const float a = lane < 16 ? alpha[row] : 1.f;
#pragma unroll 1
          for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 32) {
            uint32_t o[32];
            tmem_ld32(lanes + kColO + c0, o);
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * a);
            tmem_st32(lanes + kColO + c0, o);
          }
        }
      }
      // P, rounded to bf16 for its product (2^-8 of each weight at most, as
      // the result is); the sums are of the unrounded weights
#pragma unroll
      for (int c = 0; c < 16; c += 4) {
        const float4 v = refs[c / 2], w = refs[c / 2 + 1];
        const float n0 = v.x == INFINITY ? 0.f : v.x, n1 = v.y == INFINITY ? 0.f : v.y,
                    n2 = v.z == INFINITY ? 0.f : v.z, n3 = v.w == INFINITY ? 0.f : v.w,
                    n4 = w.x == INFINITY ? 0.f : w.x, n5 = w.y == INFINITY ? 0.f : w.y,
                    n6 = w.z == INFINITY ? 0.f : w.z, n7 = w.w == INFINITY ? 0.f : w.w;
        const float2 e[4] = {score(c, make_float2(n0, n1)), score(c + 1, make_float2(n2, n3)),
                             score(c + 2, make_float2(n4, n5)), score(c + 3, make_float2(n6, n7))};
        uint32_t pk[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 p = valid ? make_float2(ex2(e[u].x), ex2(e[u].y)) : make_float2(0.f, 0.f);
          l[c + u] = fadd2(l[c + u], p);
          pk[u] = pack_bf16(p.x, p.y);
        }
        p_row[(4 * half + c / 4) ^ (r & 7)] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BP));
    }
    // ---- the sums over the lanes, then the rows of O
    if (n > 0) {
      ok = ok && warp_wait(bar(BO + (n - 1) % 3), ((n - 1) / 3) & 1, ctl);
      ok = !alu_any(!ok);
    }
    if (ok) {
      float s[32];
#pragma unroll
      for (int c = 0; c < 16; ++c) s[2 * c] = l[c].x, s[2 * c + 1] = l[c].y;
      part[quarter * kBlock + 32 * half + lane] =
          over_lanes(s, lane, [](float a, float b) { return a + b; });
      alu_sync();
      tc_fence_after();
      const int pos = blk * kBlock + row;
      const bool mine = lane < 16 && pos < g.N;
      float sum = 0.f;
      if (mine)
        sum = (part[row] + part[kBlock + row]) + (part[2 * kBlock + row] + part[3 * kBlock + row]);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int64_t nat =
          mine ? bh * g.N + natural_index(g, g.perm[(int)(bh % g.heads)], pos) : 0;
      if (mine && half == 0) lse[nat] = row_lse(-neg_ref[row], sum);
      uint4* to = reinterpret_cast<uint4*>(out + nat * D);
#pragma unroll
      for (int c = 0; c < D / 2; c += 32) {
        const int c0 = half * (D / 2) + c;
        uint32_t f[32], o[16];
        if (n > 0) {
          tmem_ld32(lanes + kColO + c0, f);
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) f[x] = 0u;
        }
#pragma unroll
        for (int x = 0; x < 16; ++x)
          o[x] = pack_bf16(__uint_as_float(f[2 * x]) * inv, __uint_as_float(f[2 * x + 1]) * inv);
        if (mine)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            to[c0 / 8 + x] = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch_typed(const BwdArgs& a, const Grid& g, void* out, float* lse, cudaStream_t s) {
  const cudaError_t e = opt_in_smem<fwd64_sm100_kernel<D>>(Lay<D>::kBytes);
  if (e != cudaSuccess) return e;
  const uint64_t rows = (uint64_t)g.B * g.heads * g.Np;
  CUtensorMap mq{}, mk{}, mv{};
  if (!encode_tile_map(&mq, a.q, rows, D, 2, 64, kBlock) ||
      !encode_tile_map(&mk, a.k, rows, D, 2, 64, kBlock) ||
      !encode_tile_map(&mv, a.v, rows, D, 2, 64, kBlock))
    return cudaErrorInvalidValue;
  fwd64_sm100_kernel<D><<<dim3(g.NB, g.B * g.heads), kThreads, Lay<D>::kBytes, s>>>(
      mq, mk, mv, g, a.idx, a.counts, a.k_max, (float)(1.4426950408889634 / sqrt((double)D)),
      static_cast<__nv_bfloat16*>(out), lse, a.status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fwd64_sm100(const BwdArgs& a, const Grid& g, void* out, float* lse,
                               cudaStream_t s) {
  return g.d == 64 ? launch_typed<64>(a, g, out, lse, s) : launch_typed<128>(a, g, out, lse, s);
}

}  // namespace paro
