// Backward pass of block-sparse attention on the 5th-generation tensor cores
// for block = 64 (bf16, d = 64 or 128); the formulas are at the head of
// attn_bwd.cu, whose preparation runs first.
//
// A CTA owns one block of 64 rows, with operand tiles A1, A2, and streams its
// list two blocks (128 rows) a step, B1(t) and B2(t):
//   kKeys   own = keys:    A1 = K, A2 = V; streamed = queries: B1 = Q,
//           B2 = dO; the list is the transposed one (bits of the mask)
//   else    own = queries: A1 = Q, A2 = dO; streamed = keys: B1 = K, B2 = V
// The products that fill 128 rows of a matrix instruction have the streamed
// rows as their rows, whichever blocks they come from:
//   X = B1 A1^T (scores),  Y = B2 A2^T (dP)         128 x 64, from shared memory
//   P = 2^(X c - lse),  dS = P o (Y - D)
//   G1 += dS^T B1 (dK or dQ),  kKeys: G2 += P^T B2 (dV)   64 x d
// P and dS go to shared memory as bf16, one after the other into one buffer, a
// row a thread, and are the (M-major) A operand of the second products.  The
// second place of an odd list's last step is loaded from behind the tensors'
// end, as zeros, with P = dS = 0 whatever the own block holds: nothing but the
// block's own kept tiles meets its sums, so what other rows hold (infinities,
// NaN) stays there, and an infinity of its own meets no weight of zero.
//
// 10 warps:
//   0-7  elementwise: warp w holds the streamed rows 32 (w % 4) .. +31 (a row
//        a thread) and the columns 32 (w / 4) .. +31 of X and Y; at the end
//        the sums' rows;
//   8    tensor memory, and one lane that issues every MMA;
//   9    TMA loads, and which blocks a step holds.
// Tensor memory: X 0, Y 64, G1 128, G2 128 + d.  The 64 rows of a sum are in
// lanes 32 w + 0..15, w = 0..3.
// Issue order: X0 Y0, then for every t: X(t+1), (kKeys) G2(t) once P(t) is
// written, Y(t+1), G1(t) once dS(t) is.
//
// Bounded by the chain X, P, Y, dS of a step; at d = 64 two CTAs share an SM
// and fill each other's gaps.  Measured, d = 64: 307200 tiles in each use
// 1.94 ms (mma.sync, which takes 4 times the tensor pipe's cycles: 4.72 ms;
// two load warps, which leave 80 registers: 2.00; with a buffer each for P and
// dS and so only two stages of B1 2.23); 1280 tiles of 128 + 128 lists 21.3 us
// (29.4); the same at d = 128 30.9 us (51), where one CTA fits an SM.
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
constexpr uint32_t kOwnHalf = kBlock * 128;  // 64 columns of an own tile
constexpr uint32_t kHalf = kStep * 128;      // of a streamed one; P and dS

constexpr int kB1Stages = 3;  // X(t+1) is issued before G1(t), and G1(t) frees a stage

enum : uint32_t {
  BA = 0,    // A1, A2 loaded
  BB1 = 1,   // B1 stage full (3)
  BB2 = 4,   // B2 stage full (2)
  BX = 6,    // X(t) complete (ring of 2)
  BY = 8,    // Y(t) complete (ring of 2)
  BG1 = 10,  // G1(t) complete: its B1 stage (dQ: and B2 stage) and dS are free (3)
  BG2 = 13,  // G2(t) complete: its B2 stage and P are free (2)
  BP = 15,   // P(t) written by every elementwise thread (dQ: X(t) read)
  BS = 16,   // dS(t) written
  BDRAIN = 17,
  NBAR = 18
};

template <int D>
struct Lay {
  static constexpr uint32_t kOwn = kBlock * D * 2, kTile = kStep * D * 2;
  static constexpr uint32_t kA1 = 0, kA2 = kOwn, kB1 = 2 * kOwn, kB2 = kB1 + kB1Stages * kTile,
                            kP = kB2 + 2 * kTile,  // P, then dS
                            kBar = kP + kHalf,
                            kSlot = kBar + NBAR * 8,  // tensor memory's base, the abort flag
      kIds = kSlot + 8,                               // [stage][2]: the blocks of a step
      kStats = kIds + 24,                             // dQ: -lse, -D of the own rows
      kBytes = kStats + 2 * kBlock * 4;
};
// two CTAs on an SM at d = 64, each with a kilobyte of the system's
static_assert(2 * (Lay<64>::kBytes + 1024) <= 228 * 1024, "shared memory, d = 64");
static_assert(Lay<128>::kBytes <= kSmemOptIn, "shared memory, d = 128");
static_assert(Lay<64>::kStats % 16 == 0, "float4 reads");

// The CTA's block.  Returns with none of its copies or MMAs in flight,
// whatever happened.
template <bool kKeys, int D>
__device__ __forceinline__ void bwd_block(const CUtensorMap& map_a1, const CUtensorMap& map_a2,
                                          const CUtensorMap& map_b1, const CUtensorMap& map_b2,
                                          const BwdArgs& args, const Grid& g, float scale,
                                          float scale_log2, unsigned char* smem, uint32_t base,
                                          uint32_t tmem, int cnt, Ctl ctl) {
  using L = Lay<D>;
  constexpr uint32_t kColX = 0, kColY = 64, kColG1 = 128, kColG2 = 128 + D;
  auto bar = [&](uint32_t slot) { return base + L::kBar + slot * 8u; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t bh = blockIdx.y;
  const int blk = blockIdx.x;
  const int head = (int)bh * g.Np;  // first row of the head (all rows: < 2^31)
  const int64_t row = bh * g.NB + blk;
  const int n = (cnt + 1) / 2;  // steps
  volatile int32_t* step_ids = reinterpret_cast<int32_t*>(smem + L::kIds);

  if (warp == kLoadWarp) {
    // -------------------------------------------------------- copies ----
    if (lane == 0) {
      mbar_arrive_tx(bar(BA), 2 * L::kOwn);
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        tma_load_2d(base + L::kA1 + h * kOwnHalf, &map_a1, 64 * h, head + blk * kBlock, bar(BA));
        tma_load_2d(base + L::kA2 + h * kOwnHalf, &map_a2, 64 * h, head + blk * kBlock, bar(BA));
      }
    }
    const uint32_t* bits = args.mask + row * args.words;
    const int32_t* ids = args.idx + row * args.k_max;
    int word = -1;                 // kKeys: the current word of the mask
    uint32_t left = 0, chunk = 0;  // its bits left; words 32 (word / 32) + lane
    int id_lane = 0;               // dQ: entry 32 (e / 32) + lane
    auto entry = [&](int e) -> int {
      if constexpr (kKeys) {
        while (left == 0) {  // warp-uniform; ends: cnt bits are set
          ++word;
          if ((word & 31) == 0) chunk = word + lane < args.words ? __ldg(bits + word + lane) : 0u;
          left = __shfl_sync(0xffffffffu, chunk, word & 31);
        }
        const int j = word * 32 + __ffs(left) - 1;
        left &= left - 1;
        return j;
      } else {
        if ((e & 31) == 0) id_lane = e + lane < cnt ? __ldg(ids + e + lane) : 0;
        return __shfl_sync(0xffffffffu, id_lane, e & 31);
      }
    };
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
    auto g1_done = [&](int t) {
      return t < 0 || warp_wait(bar(BG1 + t % kB1Stages), (t / kB1Stages) & 1, ctl);
    };
    int issued1 = 0, issued2 = 0;
    for (int t = 0; t < n; ++t) {
      const int s1 = t % kB1Stages, s2 = t & 1;
      const bool two = 2 * t + 1 < cnt;
      const int j0 = entry(2 * t), j1 = two ? entry(2 * t + 1) : -1;
      if (!g1_done(t - kB1Stages)) break;
      if (lane == 0) {
        step_ids[2 * s1] = j0;
        step_ids[2 * s1 + 1] = j1;
        load(&map_b1, base + L::kB1 + s1 * L::kTile, j0, j1, bar(BB1 + s1));
      }
      issued1 = t + 1;
      const int last = t - 2;  // the step that had the B2 stage
      if (!(kKeys ? last < 0 || warp_wait(bar(BG2 + (last & 1)), (last >> 1) & 1, ctl)
                  : g1_done(last)))
        break;
      if (lane == 0) load(&map_b2, base + L::kB2 + s2 * L::kTile, j0, j1, bar(BB2 + s2));
      issued2 = t + 1;
    }
    // on every path this warp's copies have landed before it leaves
    if (lane == 0) {
      drain_phase(bar(BA), 0);
      for (int t = issued1 > kB1Stages ? issued1 - kB1Stages : 0; t < issued1; ++t)
        drain_phase(bar(BB1 + t % kB1Stages), (t / kB1Stages) & 1);
      for (int t = issued2 > 2 ? issued2 - 2 : 0; t < issued2; ++t)
        drain_phase(bar(BB2 + (t & 1)), (t >> 1) & 1);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------------- MMA ----
    if (elect_one()) {
      constexpr uint32_t id_x = idesc_bf16(kStep, kBlock, false);
      constexpr uint32_t id_g = idesc_bf16(kBlock, D, true) | (1u << 15);  // A M-major too
      const uint64_t da1 = sw128_desc(base + L::kA1, 16, 1024);
      const uint64_t da2 = sw128_desc(base + L::kA2, 16, 1024);
      const uint64_t db1 = sw128_desc(base + L::kB1, 16, 1024);
      const uint64_t db2 = sw128_desc(base + L::kB2, 16, 1024);
      const uint64_t dm1 = sw128_desc(base + L::kB1, kHalf, 1024);  // MN-major
      const uint64_t dm2 = sw128_desc(base + L::kB2, kHalf, 1024);
      const uint64_t dp = sw128_desc(base + L::kP, kHalf, 1024);
      auto stage1 = [](int t) { return (uint64_t)(t % kB1Stages * (L::kTile >> 4)); };
      auto stage2 = [](int t) { return (uint64_t)((t & 1) * (L::kTile >> 4)); };
      auto product = [&](uint32_t d, uint64_t b, uint64_t a) {  // d = B A^T over d
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_f16_ss(d, b + (((kk >> 2) * kHalf + (kk & 3) * 32) >> 4),
                     a + (((kk >> 2) * kOwnHalf + (kk & 3) * 32) >> 4), id_x, kk > 0 ? 1u : 0u);
      };
      auto gather = [&](uint32_t d, uint64_t p, uint64_t b, bool acc) {  // d += p^T b
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk)
          mma_f16_ss(d, p + (uint64_t)(kk * 128), b + (uint64_t)(kk * 128), id_g,
                     (acc || kk > 0) ? 1u : 0u);
      };
      auto issue_x = [&](int t) -> bool {
        if (!wait_phase(bar(BB1 + t % kB1Stages), (t / kB1Stages) & 1, ctl)) return false;
        tc_fence_after();
        product(tmem + kColX, db1 + stage1(t), da1);
        mma_commit(bar(BX + (t & 1)));
        return true;
      };
      auto issue_y = [&](int t) -> bool {
        if (!wait_phase(bar(BB2 + (t & 1)), (t >> 1) & 1, ctl)) return false;
        tc_fence_after();
        product(tmem + kColY, db2 + stage2(t), da2);
        mma_commit(bar(BY + (t & 1)));
        return true;
      };
      bool ok = n > 0 && wait_phase(bar(BA), 0, ctl) && issue_x(0) && issue_y(0);
      for (int t = 0; ok && t < n; ++t) {
        ok = wait_phase(bar(BP), t & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        if (t + 1 < n && !(ok = issue_x(t + 1))) break;
        if constexpr (kKeys) {
          gather(tmem + kColG2, dp, dm2 + stage2(t), t > 0);
          mma_commit(bar(BG2 + (t & 1)));
        }
        ok = wait_phase(bar(BS), t & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        if (t + 1 < n && !(ok = issue_y(t + 1))) break;
        gather(tmem + kColG1, dp, dm1 + stage1(t), t > 0);
        mma_commit(bar(BG1 + t % kB1Stages));
      }
      // every MMA issued above has completed once this commit fires
      mma_commit(bar(BDRAIN));
      drain_phase(bar(BDRAIN), 0);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------- elementwise ----
    const int quarter = warp & 3, half = warp >> 2;
    const int r = quarter * 32 + lane;  // streamed row of a step
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t lane_addr = lanes + 32 * half;
    const float2 sc2 = make_float2(scale_log2, scale_log2);
    const float4* own = reinterpret_cast<const float4*>(smem + L::kStats) + 8 * half;
    uint4* p_row = reinterpret_cast<uint4*>(smem + L::kP + r * 128);
    // the streamed row of step t: whether there is one, and (kKeys) its -lse, -D
    bool valid = false;
    float nl = 0.f, nd = 0.f;
    auto ahead = [&](int t) -> bool {
      if (!all_wait(bar(BB1 + t % kB1Stages), (t / kB1Stages) & 1, ctl)) return false;
      const int j = step_ids[2 * (t % kB1Stages) + (r >> 6)];
      const int pos = j * kBlock + (r & 63);
      valid = j >= 0 && pos < g.N;
      if constexpr (kKeys) {
        nl = valid ? __ldg(args.nlse + (int64_t)head + pos) : -INFINITY;
        nd = valid ? __ldg(args.ndel + (int64_t)head + pos) : 0.f;
      }
      return true;
    };
    bool ok = n == 0 || ahead(0);
    for (int t = 0; ok && t < n; ++t) {
      const bool was_valid = valid;
      const float2 nd2 = make_float2(nd, nd), nl2 = make_float2(nl, nl);
      if (!(ok = warp_wait(bar(BX + (t & 1)), (t >> 1) & 1, ctl))) break;
      tc_fence_after();
      uint32_t x[32];
      tmem_ld32(lane_addr + kColX, x);
      float2 p[16];
#pragma unroll
      for (int c = 0; c < 16; c += 2) {
        float2 n0 = nl2, n1 = nl2;
        if constexpr (!kKeys) {
          const float4 v = own[c / 2];
          n0 = make_float2(v.x, v.y);
          n1 = make_float2(v.z, v.w);
        }
        const float2 e0 =
            ffma2(make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), sc2, n0);
        const float2 e1 = ffma2(
            make_float2(__uint_as_float(x[2 * c + 2]), __uint_as_float(x[2 * c + 3])), sc2, n1);
        p[c] = make_float2(ex2(e0.x), ex2(e0.y));
        p[c + 1] = make_float2(ex2(e1.x), ex2(e1.y));
      }
      if constexpr (kKeys) {
        if (t > 0 && !(ok = warp_wait(bar(BG1 + (t - 1) % kB1Stages), ((t - 1) / kB1Stages) & 1, ctl))) break;
        // (0 where there is no row: 0 times an infinite key is NaN)
        auto pair = [&](float2 f) { return was_valid ? pack_bf16(f.x, f.y) : 0u; };
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2* f = p + 4 * c;
          p_row[(4 * half + c) ^ (r & 7)] =
              make_uint4(pair(f[0]), pair(f[1]), pair(f[2]), pair(f[3]));
        }
      }
      if constexpr (kKeys) fence_async_smem();
      tc_fence_before();
      mbar_arrive(bar(BP));
      if (t + 1 < n && !(ok = ahead(t + 1))) break;
      if (!(ok = warp_wait(bar(BY + (t & 1)), (t >> 1) & 1, ctl))) break;
      tc_fence_after();
      tmem_ld32(lane_addr + kColY, x);
      uint32_t pk[16];
#pragma unroll
      for (int c = 0; c < 16; c += 2) {
        float2 n0 = nd2, n1 = nd2;
        if constexpr (!kKeys) {
          const float4 v = own[kBlock / 4 + c / 2];
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
        if (!was_valid) pk[c] = pk[c + 1] = 0u;
      }
      // the buffer is free once the product of P(t), or of dS(t - 1), is done
      if (kKeys ? !(ok = warp_wait(bar(BG2 + (t & 1)), (t >> 1) & 1, ctl))
                : t > 0 && !(ok = warp_wait(bar(BG1 + (t - 1) % kB1Stages), ((t - 1) / kB1Stages) & 1, ctl)))
        break;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        p_row[(4 * half + c) ^ (r & 7)] =
            make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(bar(BS));
    }
    // ---- the block's sums: row 16 (w % 4) + lane in lanes 0-15, column half w / 4
    if (ok && n > 0) {
      ok = warp_wait(bar(BG1 + (n - 1) % kB1Stages), ((n - 1) / kB1Stages) & 1, ctl);
      if (kKeys && ok) ok = warp_wait(bar(BG2 + ((n - 1) & 1)), ((n - 1) >> 1) & 1, ctl);
      tc_fence_after();
    }
    if (ok) {
      const int pos = blk * kBlock + 16 * quarter + lane;
      const bool mine = lane < 16 && pos < g.N;
      const int64_t at =
          mine ? (bh * g.N + natural_index(g, g.perm[(int)(bh % g.heads)], pos)) * D : 0;
#pragma unroll
      for (int s = 0; s < (kKeys ? 2 : 1); ++s) {
        uint4* to = reinterpret_cast<uint4*>((s ? args.dv : kKeys ? args.dk : args.dq) + at);
        const float mul = s ? 1.f : scale;
#pragma unroll
        for (int c = 0; c < D / 2; c += 32) {
          const int c0 = half * (D / 2) + c;
          uint32_t f[32];
          if (n > 0) {
            tmem_ld32(lanes + (s ? kColG2 : kColG1) + c0, f);
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) f[c] = 0u;
          }
          uint32_t o[16];
#pragma unroll
          for (int c = 0; c < 16; ++c)
            o[c] = pack_bf16(__uint_as_float(f[2 * c]) * mul, __uint_as_float(f[2 * c + 1]) * mul);
          if (mine)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              to[c0 / 8 + c] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
      }
    }
    __syncwarp();
  }
}

// z = 0: the key blocks' CTAs, z = 1 the query blocks'.
template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1)
    bwd64_sm100_kernel(const __grid_constant__ CUtensorMap map_q,
                       const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v,
                       const __grid_constant__ CUtensorMap map_do,
                       const __grid_constant__ BwdArgs args, const __grid_constant__ Grid g,
                       float scale, float scale_log2) {
  using L = Lay<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t base = smem_u32(smem_raw);
  int32_t* status = args.status;
  if ((base & 1023u) != 0) {
    if (threadIdx.x == 0) report(status, PA_ERR_UNSUPPORTED);
    return;
  }
  const bool keys = blockIdx.z == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.y * g.NB + blockIdx.x;
  int cnt = 0;
  if (keys) {
    for (int w = lane; w < args.words; w += 32) cnt += __popc(__ldg(args.mask + row * args.words + w));
    cnt = __reduce_add_sync(0xffffffffu, cnt);
  } else {
    cnt = __ldg(args.checked + row);
  }
  // a malformed list: nothing is written; and where a wait of an earlier
  // launch already expired, end quickly
  if (cnt < 0 || (status != nullptr && *reinterpret_cast<volatile int32_t*>(status) == PA_ERR_TIMEOUT))
    cnt = -1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + L::kSlot);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  // one answer for the CTA: the status may change between its threads' reads
  if (__syncthreads_or(cnt < 0)) return;
  constexpr uint32_t kColsKeys = 128 + 2 * D <= 256 ? 256 : 512;
  const uint32_t cols = keys ? kColsKeys : 256;
  if (threadIdx.x == 0) {
    for (uint32_t b = 0; b < NBAR; ++b)
      mbar_init(base + L::kBar + b * 8u, b == BP || b == BS ? kAluThreads : 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (!keys && threadIdx.x < 2 * kBlock) {
    const float* from = threadIdx.x < kBlock ? args.nlse : args.ndel;
    reinterpret_cast<float*>(smem_raw + L::kStats)[threadIdx.x] =
        __ldg(from + (int64_t)blockIdx.y * g.Np + blockIdx.x * kBlock + threadIdx.x % kBlock);
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(tmem_slot), cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Ctl ctl{abort_flag, status, kTimeoutNs};
  if (keys)
    bwd_block<true, D>(map_k, map_v, map_q, map_do, args, g, scale, scale_log2, smem_raw, base,
                       tmem, cnt, ctl);
  else
    bwd_block<false, D>(map_q, map_do, map_k, map_v, args, g, scale, scale_log2, smem_raw, base,
                        tmem, cnt, ctl);
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, cols);
  }
}

template <int D>
cudaError_t launch_typed(const BwdArgs& a, const Grid& g, cudaStream_t s) {
  const cudaError_t e = opt_in_smem<bwd64_sm100_kernel<D>>(Lay<D>::kBytes);
  if (e != cudaSuccess) return e;
  const uint64_t rows = (uint64_t)g.B * g.heads * g.Np;
  CUtensorMap mq{}, mk{}, mv{}, md{};
  if (!encode_tile_map(&mq, a.q, rows, D, 2, 64, kBlock) ||
      !encode_tile_map(&mk, a.k, rows, D, 2, 64, kBlock) ||
      !encode_tile_map(&mv, a.v, rows, D, 2, 64, kBlock) ||
      !encode_tile_map(&md, a.dop, rows, D, 2, 64, kBlock))
    return cudaErrorInvalidValue;
  bwd64_sm100_kernel<D><<<dim3(g.NB, g.B * g.heads, 2), kThreads, Lay<D>::kBytes, s>>>(
      mq, mk, mv, md, a, g, (float)(1.0 / sqrt((double)D)),
      (float)(1.4426950408889634 / sqrt((double)D)));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bwd64_sm100(const BwdArgs& a, const Grid& g, cudaStream_t s) {
  return g.d == 64 ? launch_typed<64>(a, g, s) : launch_typed<128>(a, g, s);
}

}  // namespace paro
