// Backward pass of block-sparse attention on the 5th-generation tensor cores
// (block = 128, bf16, d = 64 or 128); the formulas are at the head of
// attn_bwd.cu, whose preparation runs first.
//
// One kernel template, two uses.  A CTA owns a block of 128 rows with two
// resident operand tiles A1, A2 and streams the column tiles t = 0, 1, ...
// of its list, B1(t) and B2(t):
//   kKeys   rows = keys:    A1 = K, A2 = V; columns = queries: B1 = Q,
//           B2 = dO; the list is the transposed one (bits of the mask)
//   else    rows = queries: A1 = Q, A2 = dO; columns = keys: B1 = K, B2 = V
//   X = A1 B1^T (scores),  Y = A2 B2^T (dP),  P = 2^(X c - lse),
//   dS = P o (Y - D),  G1 += dS B1 (dK or dQ),  kKeys: G2 += P B2 (dV).
// With the rows in the tensor-memory lanes either way, P and dS are the A
// operands of the second products straight from tensor memory; B1 and B2
// serve K-major for the first products and MN-major for the second.  No
// value crosses a thread: lse and D come with the row (dQ) or, from shared
// memory, with the column (dK, dV).
//
// 12 warps:
//   0-7    elementwise; warp w holds lanes 32 (w % 4) .. +31 (a row a
//          thread) and the tile's columns 64 (w / 4) .. +63, so that two
//          warps share each scheduler and the exponentials of one hide the
//          tensor-memory loads of the other;
//   8      tensor memory, and one lane that issues every MMA;
//   9, 10  TMA loads of A1, A2, B1 and of B2;
//   11     checks the kept list (dQ).
// Tensor memory, 512 columns: kKeys X 0, Y 128, G1 256, G2 384; dQ X0 0,
// X1 128, Y 256, G1 384.  A thread writes its P (or dS) as bf16 pairs over
// the columns of X (or Y) that it read itself: 32 columns from column 64 g
// of the buffer, g the column half.
// Issue order, kKeys: X0 Y0, then for every t: G2(t) X(t+1) G1(t) Y(t+1):
// P(t+1) has the time of G1(t) and Y(t+1), dS(t) that of G2(t) and X(t+1).
// dQ: X0 Y0 X1, then G1(t) Y(t+1) X(t+2).  X(t+1) overwrites the P(t) that
// G2(t) reads, and Y(t+1) the dS(t) of G1(t): MMAs that one thread issues
// run in order in the tensor pipe.
//
// Bounded by the MMA stream (4 products a tile with kKeys, 3 for dQ); the
// exponentials take 16384 / 16 = 1024 cycles a tile of the 3000.  Waits are
// bounded as in the forward kernel.
#include "bwd.cuh"
#include "sm100.cuh"

namespace paro {

namespace {

using namespace sm100;

constexpr int kBlock = 128;
constexpr int kMmaWarp = 8, kB1Warp = 9, kB2Warp = 10, kCheckWarp = 11;
constexpr int kThreads = 12 * 32;
constexpr int kAluThreads = 256;
constexpr uint32_t kHalf = kBlock * 128;  // 64 columns of a tile: 16 KB
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOffBar = 0;
constexpr uint32_t kOffSlot = 256;
constexpr uint32_t kOffStats = 512;  // kKeys: [2 stages][-lse, -D][128] float
constexpr uint32_t kStatBytes = kBlock * 4;
constexpr uint32_t kSmall = 3072;  // operand tiles from here, 1024-aligned

enum : uint32_t {
  BA = 0,     // A1, A2 loaded
  BB1 = 1,    // B1 stage full (3)
  BB2 = 4,    // B2 stage full (2)
  BX = 6,     // X(t) complete (ring of 2)
  BY = 8,     // Y(t) complete (ring of 2)
  BG1 = 10,   // G1(t) complete: its B1 stage is free (3)
  BG2 = 13,   // G2(t) complete: its B2 stage is free (2)
  BP = 15,    // P(t) written by every elementwise thread
  BS = 16,    // dS(t) written
  BDRAIN = 17,
  NBAR = 18
};
static_assert(NBAR * 8 <= kOffSlot, "barrier region");
static_assert(kOffStats + 4 * kStatBytes <= kSmall, "statistics region");

template <bool kKeys>
constexpr int kB1Stages = kKeys ? 2 : 3;
constexpr int kB2Stages = 2;

// Untiled copy of `bytes` (a multiple of 16, both addresses 16-byte aligned).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
          dst),
      "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
      : "memory");
}

template <bool kKeys, int D>
__device__ __forceinline__ void bwd_block(const CUtensorMap& map_a1, const CUtensorMap& map_a2,
                                          const CUtensorMap& map_b1, const CUtensorMap& map_b2,
                                          const BwdArgs& args, const Grid& g, float scale,
                                          float scale_log2) {
  const float* __restrict__ nlse = args.nlse;
  const float* __restrict__ ndel = args.ndel;
  const int words = args.words, k_max = args.k_max;
  const int32_t *idx = args.idx, *counts = args.counts;
  const uint32_t* __restrict__ mask = args.mask;
  __nv_bfloat16* __restrict__ g1 = kKeys ? args.dk : args.dq;
  __nv_bfloat16* __restrict__ g2 = args.dv;  // kKeys only
  int32_t* status = args.status;
  constexpr uint32_t kTile = kBlock * D * 2;
  constexpr int kS1 = kB1Stages<kKeys>;
  constexpr uint32_t kOffA1 = kSmall, kOffA2 = kOffA1 + kTile, kOffB1 = kOffA2 + kTile,
                     kOffB2 = kOffB1 + kS1 * kTile;
  constexpr uint32_t kColX = 0, kColY = kKeys ? 128 : 256, kColG1 = kKeys ? 256 : 384,
                     kColG2 = 384;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t base = smem_u32(smem_raw);
  if ((base & 1023u) != 0) {
    if (threadIdx.x == 0) report(status, PA_ERR_UNSUPPORTED);
    return;
  }
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + kOffSlot);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  volatile uint32_t* bad_flag = tmem_slot + 2;
  auto bar = [&](uint32_t slot) { return base + kOffBar + slot * 8u; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blk = blockIdx.x;  // this CTA's block of rows
  const int64_t bh = blockIdx.y;
  const int order = g.perm[(int)(bh % g.heads)];
  const int64_t row = bh * g.NB + blk;
  const int row0 = (int)(bh * g.Np);  // first row of the head
  const int32_t* ids = kKeys ? nullptr : idx + row * k_max;
  const uint32_t* bits = kKeys ? mask + row * words : nullptr;
  const Ctl ctl{abort_flag, status, kTimeoutNs};
  const bool expired =
      status != nullptr && *reinterpret_cast<volatile int32_t*>(status) == PA_ERR_TIMEOUT;

  // tiles of the list: kKeys counts the bits of the row of the mask
  int cnt;
  if constexpr (kKeys) {
    cnt = 0;
    for (int w = lane; w < words; w += 32) cnt += __popc(__ldg(bits + w));
    cnt = __reduce_add_sync(0xffffffffu, cnt);
  } else {
    cnt = counts != nullptr ? __ldg(counts + row) : k_max;
  }

  if (threadIdx.x == 0) {
    mbar_init(bar(BA), 1);
    for (int s = 0; s < 3; ++s) {
      mbar_init(bar(BB1 + s), 1);
      mbar_init(bar(BG1 + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(BB2 + s), 1);
      mbar_init(bar(BX + s), 1);
      mbar_init(bar(BY + s), 1);
      mbar_init(bar(BG2 + s), 1);
    }
    mbar_init(bar(BP), kAluThreads);
    mbar_init(bar(BS), kAluThreads);
    mbar_init(bar(BDRAIN), 1);
    *abort_flag = 0;
    *bad_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  if (!kKeys && warp == kCheckWarp && !list_ok(ids, cnt, k_max, g.NB, lane) && lane == 0) {
    *bad_flag = 1;
    report(status, PA_ERR_DEVICE_CHECK);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool run = *bad_flag == 0 && !expired;
  const int n = run ? cnt : 0;

  if (warp >= 8) {
    if ((warp == kB1Warp || warp == kB2Warp) && n > 0) {
      // ---------------------------------------------------- copies ----
      const bool first = warp == kB1Warp;
      const int stages = first ? kS1 : kB2Stages;
      const uint32_t ring = base + (first ? kOffB1 : kOffB2);
      const CUtensorMap* map = first ? &map_b1 : &map_b2;
      // a stage is free once the last product that reads it completed: B1's
      // is G1; B2's is G2, or Y where there is no G2
      const uint32_t full0 = first ? BB1 : BB2, free0 = first ? BG1 : kKeys ? BG2 : BY;
      if (first && lane == 0) {
        mbar_arrive_tx(bar(BA), 2 * kTile);
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          tma_load_2d(base + kOffA1 + h * kHalf, &map_a1, 64 * h, row0 + blk * kBlock, bar(BA));
          tma_load_2d(base + kOffA2 + h * kHalf, &map_a2, 64 * h, row0 + blk * kBlock, bar(BA));
        }
      }
      int issued = 0;
      int word = -1;          // kKeys: the current word of the mask
      uint32_t left = 0, chunk = 0;  // its bits left; words 32 (word / 32) + lane
      int id_lane = 0;        // dQ: entry 32 (t / 32) + lane
      for (int t = 0; t < n; ++t) {
        int j;
        if constexpr (kKeys) {
          while (left == 0) {  // warp-uniform; ends: n bits are set
            ++word;
            if ((word & 31) == 0) chunk = word + lane < words ? __ldg(bits + word + lane) : 0u;
            left = __shfl_sync(0xffffffffu, chunk, word & 31);
          }
          j = word * 32 + __ffs(left) - 1;
          left &= left - 1;
        } else {
          if ((t & 31) == 0) id_lane = t + lane < n ? __ldg(ids + t + lane) : 0;
          j = __shfl_sync(0xffffffffu, id_lane, t & 31);
        }
        const int s = t % stages, round = t / stages;
        if (round > 0 && !warp_wait(bar(free0 + s), (round - 1) & 1, ctl)) break;
        if (lane == 0) {
          const uint32_t full = bar(full0 + s);
          const bool stats = kKeys && first;
          mbar_arrive_tx(full, kTile + (stats ? 2 * kStatBytes : 0));
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_2d(ring + s * kTile + h * kHalf, map, 64 * h, row0 + j * kBlock, full);
          if (stats) {
            const uint32_t dst = base + kOffStats + s * 2 * kStatBytes;
            const int64_t at = (int64_t)row0 + j * kBlock;
            bulk_load(dst, nlse + at, kStatBytes, full);
            bulk_load(dst + kStatBytes, ndel + at, kStatBytes, full);
          }
        }
        issued = t + 1;
      }
      // on every path this warp's copies have landed before it leaves
      if (lane == 0) {
        if (first) drain_phase(bar(BA), 0);
        for (int t = issued > stages ? issued - stages : 0; t < issued; ++t)
          drain_phase(bar(full0 + t % stages), (t / stages) & 1);
      }
    } else if (warp == kMmaWarp && lane == 0 && n > 0) {
      // -------------------------------------------------------- MMA ----
      constexpr uint32_t id_x = idesc_bf16(kBlock, kBlock, false);
      constexpr uint32_t id_g = idesc_bf16(kBlock, D, true);
      const uint64_t da1 = sw128_desc(base + kOffA1, 16, 1024);
      const uint64_t da2 = sw128_desc(base + kOffA2, 16, 1024);
      const uint64_t db1 = sw128_desc(base + kOffB1, 16, 1024);
      const uint64_t db2 = sw128_desc(base + kOffB2, 16, 1024);
      const uint64_t dm1 = sw128_desc(base + kOffB1, kHalf, 1024);  // MN-major
      const uint64_t dm2 = sw128_desc(base + kOffB2, kHalf, 1024);
      auto product = [&](uint32_t d, uint64_t a, uint64_t b) {  // d = A B^T over d
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
          mma_f16_ss(d, a + off, b + off, id_x, kk > 0 ? 1u : 0u);
        }
      };
      // d += A B over the tile's 128 columns, A from the elementwise
      // threads' pairs: columns 0-31 and 64-95 of the buffer at a
      auto gather = [&](uint32_t d, uint32_t a, uint64_t b, bool acc) {
#pragma unroll
        for (int kk = 0; kk < kBlock / 16; ++kk)
          mma_f16_ts(d, a + (kk >> 2) * 64 + (kk & 3) * 8, b + (uint64_t)(kk * 128), id_g,
                     (acc || kk > 0) ? 1u : 0u);
      };
      auto b1_off = [&](int t) { return (uint64_t)((t % kS1) * (kTile >> 4)); };
      auto b2_off = [&](int t) { return (uint64_t)((t % kB2Stages) * (kTile >> 4)); };
      auto issue_x = [&](int t) {
        product(tmem + kColX + (kKeys ? 0 : (t & 1) * 128), da1, db1 + b1_off(t));
        mma_commit(bar(BX + (t & 1)));
      };
      auto issue_y = [&](int t) {
        product(tmem + kColY, da2, db2 + b2_off(t));
        mma_commit(bar(BY + (t & 1)));
      };
      auto wait_b1 = [&](int t) { return wait_phase(bar(BB1 + t % kS1), (t / kS1) & 1, ctl); };
      auto wait_b2 = [&](int t) {
        return wait_phase(bar(BB2 + t % kB2Stages), (t / kB2Stages) & 1, ctl);
      };
      bool ok = wait_phase(bar(BA), 0, ctl) && wait_b1(0);
      if (ok) issue_x(0);
      ok = ok && wait_b2(0);
      if (ok) issue_y(0);
      if (!kKeys && n > 1) {
        ok = ok && wait_b1(1);
        if (ok) issue_x(1);
      }
      for (int t = 0; ok && t < n; ++t) {
        if constexpr (kKeys) {
          if (!wait_phase(bar(BP), t & 1, ctl)) break;
          tc_fence_after();
          gather(tmem + kColG2, tmem + kColX, dm2 + b2_off(t), t > 0);
          mma_commit(bar(BG2 + t % kB2Stages));
          if (t + 1 < n) {
            if (!wait_b1(t + 1)) break;
            issue_x(t + 1);
          }
        }
        if (!wait_phase(bar(BS), t & 1, ctl)) break;
        tc_fence_after();
        gather(tmem + kColG1, tmem + kColY, dm1 + b1_off(t), t > 0);
        mma_commit(bar(BG1 + t % kS1));
        if (t + 1 < n) {
          if (!wait_b2(t + 1)) break;
          issue_y(t + 1);
        }
        if (!kKeys && t + 2 < n) {
          if (!wait_b1(t + 2)) break;
          issue_x(t + 2);
        }
      }
      // every MMA issued above has completed once this commit fires
      mma_commit(bar(BDRAIN));
      drain_phase(bar(BDRAIN), 0);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------- elementwise ----
    const int half = warp >> 2;  // columns 64 half .. +63 of a tile
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16) + half * 64;
    const float2 sc2 = make_float2(scale_log2, scale_log2);
    float2 nl2 = make_float2(0.f, 0.f), nd2 = nl2;  // dQ: this row's -lse, -D
    int tail = kBlock;                              // dQ: valid keys of the last listed tile
    if constexpr (!kKeys) {
      const int64_t at = (int64_t)row0 + blk * kBlock + r;
      nl2.x = nl2.y = __ldg(nlse + at);
      nd2.x = nd2.y = __ldg(ndel + at);
      // the list ascends: only its last entry can be the head's last block
      if (n > 0 && __ldg(ids + n - 1) == g.NB - 1) tail = g.N - (g.NB - 1) * kBlock;
    }
    bool ok = true;
    for (int t = 0; t < n; ++t) {
      const float4* stat =
          reinterpret_cast<const float4*>(smem_raw + kOffStats + (t & 1) * 2 * kStatBytes) +
          half * 16;
      if constexpr (kKeys)  // the statistics came with B1(t)
        if (!all_wait(bar(BB1 + t % kS1), (t / kS1) & 1, ctl)) { ok = false; break; }
      if (!warp_wait(bar(BX + (t & 1)), (t >> 1) & 1, ctl)) { ok = false; break; }
      tc_fence_after();
      uint32_t x[64], pk[32];
      tmem_ld64(lane_addr + kColX + (kKeys ? 0 : (t & 1) * 128), x);
      float2 p[32];
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        float2 n0 = nl2, n1 = nl2;
        if constexpr (kKeys) {
          const float4 v = stat[c / 2];
          n0 = make_float2(v.x, v.y);
          n1 = make_float2(v.z, v.w);
        }
        const float2 e0 = ffma2(make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])),
                                sc2, n0);
        const float2 e1 = ffma2(
            make_float2(__uint_as_float(x[2 * c + 2]), __uint_as_float(x[2 * c + 3])), sc2, n1);
        p[c] = make_float2(ex2(e0.x), ex2(e0.y));
        p[c + 1] = make_float2(ex2(e1.x), ex2(e1.y));
      }
      if constexpr (kKeys) {
#pragma unroll
        for (int c = 0; c < 32; ++c) pk[c] = pack_bf16(p[c].x, p[c].y);
        tmem_st32_async(lane_addr + kColX, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(BP));
      } else if (tail < kBlock && t == n - 1) {  // warp-uniform: pad keys
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          if (half * 64 + 2 * c >= tail) p[c].x = 0.f;
          if (half * 64 + 2 * c + 1 >= tail) p[c].y = 0.f;
        }
      }
      if (!warp_wait(bar(BY + (t & 1)), (t >> 1) & 1, ctl)) { ok = false; break; }
      tc_fence_after();
      tmem_ld64(lane_addr + kColY, x);
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        float2 n0 = nd2, n1 = nd2;
        if constexpr (kKeys) {
          const float4 v = stat[kBlock / 4 + c / 2];
          n0 = make_float2(v.x, v.y);
          n1 = make_float2(v.z, v.w);
        }
        const float2 s0 = fmul2(
            p[c], fadd2(make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), n0));
        const float2 s1 = fmul2(
            p[c + 1],
            fadd2(make_float2(__uint_as_float(x[2 * c + 2]), __uint_as_float(x[2 * c + 3])), n1));
        pk[c] = pack_bf16(s0.x, s0.y);
        pk[c + 1] = pack_bf16(s1.x, s1.y);
      }
      tmem_st32_async(lane_addr + kColY, pk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(BS));
    }
    // ---- epilogue: column half `half` of the row's sums, to the natural
    // position of its token
    if (run && ok) {
      const int p = blk * kBlock + r;
      const int64_t at =
          p < g.N ? (bh * g.N + natural_index(g, order, p)) * D + half * (D / 2) : -1;
      if (n > 0) {
        const int last = n - 1;
        ok = warp_wait(bar(BG1 + last % kS1), (last / kS1) & 1, ctl);
        if (kKeys && ok) ok = warp_wait(bar(BG2 + last % kB2Stages), (last / kB2Stages) & 1, ctl);
        tc_fence_after();
      }
      auto store = [&](uint32_t col, float mul, __nv_bfloat16* dst) {
#pragma unroll 1
        for (int c0 = 0; c0 < D / 2; c0 += 32) {
          uint32_t o[32];
          if (n > 0) {
            // lane_addr already holds 64 * half: d = 64's halves are 32 wide
            tmem_ld32(lane_addr + col - half * (64 - D / 2) + c0, o);
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = 0u;
          }
          if (at >= 0) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint4 w;
              w.x = pack_bf16(__uint_as_float(o[8 * c + 0]) * mul, __uint_as_float(o[8 * c + 1]) * mul);
              w.y = pack_bf16(__uint_as_float(o[8 * c + 2]) * mul, __uint_as_float(o[8 * c + 3]) * mul);
              w.z = pack_bf16(__uint_as_float(o[8 * c + 4]) * mul, __uint_as_float(o[8 * c + 5]) * mul);
              w.w = pack_bf16(__uint_as_float(o[8 * c + 6]) * mul, __uint_as_float(o[8 * c + 7]) * mul);
              reinterpret_cast<uint4*>(dst + at + c0)[c] = w;
            }
          }
        }
      };
      if (ok) {
        store(kColG1, scale, g1);
        if constexpr (kKeys) store(kColG2, 1.f, g2);
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

// z = 0: the key blocks' CTAs, z = 1 the query blocks', which fill the SMs as
// the first run out.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_sm100_kernel(const __grid_constant__ CUtensorMap map_q,
                     const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ CUtensorMap map_do,
                     const __grid_constant__ BwdArgs args, const __grid_constant__ Grid g,
                     float scale, float scale_log2) {
  if (blockIdx.z == 0)
    bwd_block<true, D>(map_k, map_v, map_q, map_do, args, g, scale, scale_log2);
  else
    bwd_block<false, D>(map_q, map_do, map_k, map_v, args, g, scale, scale_log2);
}

template <int D>
cudaError_t launch_typed(const BwdArgs& a, const Grid& g, cudaStream_t s) {
  constexpr uint32_t kTile = kBlock * D * 2;
  constexpr int kSmem = kSmall + (2 + kB1Stages<false> + kB2Stages) * kTile;
  static_assert(kSmem <= kSmemOptIn && kB1Stages<true> <= kB1Stages<false>, "shared memory");
  const cudaError_t e = opt_in_smem<bwd_sm100_kernel<D>>(kSmem);
  if (e != cudaSuccess) return e;
  const uint64_t rows = (uint64_t)g.B * g.heads * g.Np;
  CUtensorMap mq{}, mk{}, mv{}, md{};
  if (!encode_tile_map(&mq, a.q, rows, D, 2, 64, kBlock) ||
      !encode_tile_map(&mk, a.k, rows, D, 2, 64, kBlock) ||
      !encode_tile_map(&mv, a.v, rows, D, 2, 64, kBlock) ||
      !encode_tile_map(&md, a.dop, rows, D, 2, 64, kBlock))
    return cudaErrorInvalidValue;
  bwd_sm100_kernel<D><<<dim3(g.NB, g.B * g.heads, 2), kThreads, kSmem, s>>>(
      mq, mk, mv, md, a, g, (float)(1.0 / sqrt((double)D)),
      (float)(1.4426950408889634 / sqrt((double)D)));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bwd_sm100(const BwdArgs& a, const Grid& g, cudaStream_t s) {
  return g.d == 64 ? launch_typed<64>(a, g, s) : launch_typed<128>(a, g, s);
}

}  // namespace paro
