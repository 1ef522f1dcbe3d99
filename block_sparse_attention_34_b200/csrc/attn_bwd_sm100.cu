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
// The grid is one CTA per SM, which takes the key blocks, then the query
// blocks, from a counter each: a block's loads start while the last one's
// sums are stored, and its first products follow the last one's without a
// pause.  (A CTA per block, which starts and ends 7 us around its tiles,
// took 4 to 7% longer.)
//
// 20 warps:
//   0-15    elementwise; warp w holds lanes 32 (w % 4) .. +31 (a row a
//           thread) and the tile's columns 32 (w / 4) .. +31: four warps
//           share a scheduler, and the exponentials of one hide the
//           tensor-memory loads of the others; at a block's end they read
//           its sums and store them;
//   16      tensor memory, and one lane that issues every MMA;
//   17, 18  TMA loads of A1, A2, B1 and of B2;
//   19      takes the blocks and hands them to the other warps, two ahead.
// The tiles of a CTA's blocks are numbered through (T below): stages and
// barrier phases go on from block to block.
// Tensor memory, 512 columns: kKeys at d = 128: X 0, Y 128, G1 256, G2 384;
// otherwise three buffers at 0, 128, 256 that X and Y go round, G1 384 (and
// kKeys, d = 64, G2 448).  A thread writes its P (or dS) as bf16 pairs over
// the columns of X (or Y) that it read itself: 16 columns from column 32 g
// of the buffer, g its part of the columns.
// Issue order with one X and one Y (kKeys, d = 128): X0 Y0, then for every t:
// G2(t) X(t+1) G1(t) Y(t+1): P(t+1) has the time of G1(t) and Y(t+1), dS(t)
// that of G2(t) and X(t+1).  With three buffers: X0 Y0 X1, then (kKeys G2(t))
// Y(t+1) G1(t) X(t+2).  A product overwrites a P or dS that an earlier one
// reads, MMAs that one thread issues run in order in the tensor pipe, or an X
// that the elementwise threads have read (dQ: they say so in place of P).
//
// P and dS are rounded to bf16 (2^-8 of their value at most) for the second
// products, as P is in the forward kernel; the sums stay in 32 bits.  The
// rounding of dS is what dq and dk carry most of: 0.0025 relative in the
// norm, against 0.0017 of rounding the result alone.  (dS as two bf16 halves
// would bring it to the latter, for one more product a tile in each use.)
//
// Measured, d = 128: 196608 tiles in each use 4.16 ms, 1.39 PFLOP/s with the
// products computed twice, at the clock that the power limit leaves (some
// 1.7 GHz); 740 blocks of 12 tiles 235 us; d = 64, 2556 tiles 70 us.  Bounded
// by the MMA stream and the power limit; with short lists by the gap between
// two blocks (6000 cycles, of which the sums' way out is half; four warps of
// their own for it gained 8 us of 240 there and lost 2% on long lists).  With
// 8 elementwise warps of 64 columns 4.23 ms, 236 us, 77 us; then with X in two
// buffers and one Y 4.24 ms, 241 us, 78 us.
// Waits are bounded as in the forward kernel.
#include "bwd.cuh"
#include "sm100.cuh"

namespace paro {

namespace {

using namespace sm100;

constexpr int kBlock = 128;
constexpr int kSms = 148;
constexpr int kParts = 4;               // column parts of a tile, four elementwise warps each
constexpr int kCols = 128 / kParts;     // a thread's columns of a tile
constexpr int kAluWarps = 4 * kParts;
constexpr int kMmaWarp = kAluWarps, kB1Warp = kAluWarps + 1, kB2Warp = kAluWarps + 2,
              kItemWarp = kAluWarps + 3;
constexpr int kThreads = (kAluWarps + 4) * 32;
constexpr uint32_t kHalf = kBlock * 128;  // 64 columns of a tile: 16 KB
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOffBar = 0;      // two sets of NBAR barriers: kKeys, dQ
constexpr uint32_t kOffSlot = 512;   // tensor memory's base, the abort flag
constexpr uint32_t kOffItems = 528;  // [2 sets][2] of (block of the grid, tiles)
constexpr uint32_t kOffStats = 1024;  // kKeys: [B1 stage][-lse, -D][128] float
constexpr uint32_t kStatBytes = kBlock * 4;

enum : uint32_t {
  BA = 0,      // A1, A2 of the block loaded
  BB1 = 1,     // B1 stage full (3)
  BB2 = 4,     // B2 stage full (2)
  BX = 6,      // X(T) complete (ring of 2)
  BY = 8,      // Y(T) complete (ring of 2)
  BG1 = 10,    // G1(T) complete: its B1 stage is free (3)
  BG2 = 13,    // G2(T) complete: its B2 stage is free (2)
  BP = 15,     // P(T) written by every elementwise thread (dQ: X(T) read; ring of 2:
  BS = 17,     // dS(T) written (2)         they may be a tile ahead of the MMA thread)
  BFREE = 19,  // the block's sums read by every elementwise thread
  BAFREE = 20,  // the block's last product that reads A1 or A2 (Y) complete
  BDRAIN = 21,
  BITEM = 22,   // a block handed out (ring of 2)
  BTAKEN = 24,  // and taken by every warp (2)
  NBAR = 26
};
static_assert(2 * NBAR * 8 <= kOffSlot, "barrier region");
constexpr uint32_t kTakers = kAluWarps + 2 + 1;  // elementwise warps, loaders, MMA

// X and Y in three buffers that go round (X(T), Y(T), X(T + 1), Y(T + 1), ...)
// for dQ, and for dK, dV at d = 64, where tensor memory has the room: the
// elementwise threads find the next X and the next Y done.  X(T + 2) is then
// issued with G1(T), and B1 takes three stages.
template <bool kKeys, int D>
constexpr bool kRound = !kKeys || D == 64;
template <bool kKeys, int D>
constexpr int kB1Stages = kRound<kKeys, D> ? 3 : 2;
// operand tiles from here, 1024-aligned
template <int D>
constexpr uint32_t kSmall =
    (kOffStats + kB1Stages<true, D> * 2 * kStatBytes + 1023) / 1024 * 1024;
constexpr int kB2Stages = 2;

// 32 or 16 columns of a thread's lane.
__device__ __forceinline__ void tmem_cols(uint32_t at, uint32_t (&x)[32]) { tmem_ld32(at, x); }
__device__ __forceinline__ void tmem_cols(uint32_t at, uint32_t (&x)[16]) { tmem_ld16(at, x); }

// Untiled copy of `bytes` (a multiple of 16, both addresses 16-byte aligned).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
          dst),
      "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// All blocks of one use that this CTA takes.  Returns with none of its
// copies or MMAs in flight, whatever happened.
template <bool kKeys, int D>
__device__ __forceinline__ void bwd_blocks(const CUtensorMap& map_a1, const CUtensorMap& map_a2,
                                           const CUtensorMap& map_b1, const CUtensorMap& map_b2,
                                           const BwdArgs& args, const Grid& g, float scale,
                                           float scale_log2, unsigned char* smem, uint32_t base,
                                           uint32_t tmem, Ctl ctl) {
  constexpr uint32_t kTile = kBlock * D * 2;
  constexpr int kS1 = kB1Stages<kKeys, D>;
  constexpr bool kThree = kRound<kKeys, D>;
  constexpr uint32_t kOffA1 = kSmall<D>, kOffA2 = kOffA1 + kTile, kOffB1 = kOffA2 + kTile,
                     kOffB2 = kOffB1 + kS1 * kTile;
  constexpr uint32_t kColG1 = kThree ? 384 : 256, kColG2 = kColG1 + D;
  auto col_x = [](uint32_t x) { return kThree ? 2 * x % 3 * 128 : 0; };
  auto col_y = [](uint32_t x) { return kThree ? (2 * x + 1) % 3 * 128 : 128; };
  auto bar = [&](uint32_t slot) {
    return base + kOffBar + ((kKeys ? 0u : (uint32_t)NBAR) + slot) * 8u;
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)g.B * g.heads * g.NB;
  volatile int32_t* items = reinterpret_cast<int32_t*>(smem + kOffItems) + (kKeys ? 0 : 4);
  const int words = args.words;

  // The next block handed out: its row of the grid (< 0: none is left, or a
  // wait ran out) and its tiles (< 0: a malformed list).  One warp.
  int handed = 0;
  auto take = [&](int& n) -> int {
    const int s = handed & 1;
    if (!all_wait(bar(BITEM + s), (handed >> 1) & 1, ctl)) return -1;
    const int row = items[2 * s];
    n = items[2 * s + 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(BTAKEN + s));
    ++handed;
    return row;
  };

  int n = 0;
  uint32_t T = 0;     // tiles of the blocks before this one
  uint32_t full = 0;  // blocks with tiles before this one
  if (warp == kItemWarp) {
    // -------------------------------------------------------- blocks ----
    // Hands out a block, then loads its A1, A2 once the last block's products
    // have read theirs: a block is known to the other warps, and its first
    // column tiles are on their way, while the one before it is worked on.
    for (int i = 0;; ++i) {
      const int s = i & 1;
      if (i >= 2 && !warp_wait(bar(BTAKEN + s), ((i >> 1) - 1) & 1, ctl)) break;
      int row = 0;
      if (lane == 0) row = atomicAdd(args.counters + (kKeys ? 0 : 1), 1);
      row = __shfl_sync(0xffffffffu, row, 0);
      int cnt = 0;
      if (row < rows) {
        if constexpr (kKeys) {
          const uint32_t* bits = args.mask + (int64_t)row * words;
          for (int w = lane; w < words; w += 32) cnt += __popc(__ldg(bits + w));
          cnt = __reduce_add_sync(0xffffffffu, cnt);
        } else {
          cnt = __ldg(args.checked + row);
        }
      } else {
        row = -1;
      }
      if (lane == 0) {
        items[2 * s] = row;
        items[2 * s + 1] = cnt;
        mbar_arrive(bar(BITEM + s));  // release: the stores above are visible to the takers
      }
      if (row < 0) break;
      if (cnt <= 0) continue;
      if (full > 0 && !warp_wait(bar(BAFREE), (full - 1) & 1, ctl)) break;
      if (lane == 0) {
        const int bh = row / g.NB, at = bh * g.Np + (row - bh * g.NB) * kBlock;
        mbar_arrive_tx(bar(BA), 2 * kTile);
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          tma_load_2d(base + kOffA1 + h * kHalf, &map_a1, 64 * h, at, bar(BA));
          tma_load_2d(base + kOffA2 + h * kHalf, &map_a2, 64 * h, at, bar(BA));
        }
      }
      ++full;
    }
    // on every path this warp's copies have landed before it leaves
    if (lane == 0 && full > 0) drain_phase(bar(BA), (full - 1) & 1);
    __syncwarp();
  } else if (warp == kB1Warp || warp == kB2Warp) {
    // -------------------------------------------------------- copies ----
    const bool first = warp == kB1Warp;
    const int stages = first ? kS1 : kB2Stages;
    const uint32_t ring = base + (first ? kOffB1 : kOffB2);
    const CUtensorMap* map = first ? &map_b1 : &map_b2;
    // a stage is free once the last product that reads it completed: B1's
    // is G1; B2's is G2, or Y where there is no G2
    const uint32_t full0 = first ? BB1 : BB2, free0 = first ? BG1 : kKeys ? BG2 : BY;
    uint32_t issued = 0;  // tiles copied
    for (bool ok = true; ok;) {
      const int row = take(n);
      if (row < 0) break;
      if (n <= 0) continue;
      const int row0 = row / g.NB * g.Np;  // first row of the head
      const uint32_t* bits = args.mask + (int64_t)row * words;
      const int32_t* ids = args.idx + (int64_t)row * args.k_max;
      int word = -1;                 // kKeys: the current word of the mask
      uint32_t left = 0, chunk = 0;  // its bits left; words 32 (word / 32) + lane
      int id_lane = 0;               // dQ: entry 32 (t / 32) + lane
      for (int t = 0; t < n; ++t, ++T) {
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
        const uint32_t s = T % stages, round = T / stages;
        if (round > 0 && !warp_wait(bar(free0 + s), (round - 1) & 1, ctl)) { ok = false; break; }
        if (lane == 0) {
          const uint32_t b = bar(full0 + s);
          const bool stats = kKeys && first;
          mbar_arrive_tx(b, kTile + (stats ? 2 * kStatBytes : 0));
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_2d(ring + s * kTile + h * kHalf, map, 64 * h, row0 + j * kBlock, b);
          if (stats) {
            const uint32_t dst = base + kOffStats + s * 2 * kStatBytes;
            const int64_t at = (int64_t)row0 + j * kBlock;
            bulk_load(dst, args.nlse + at, kStatBytes, b);
            bulk_load(dst + kStatBytes, args.ndel + at, kStatBytes, b);
          }
        }
        issued = T + 1;
      }
    }
    // on every path this warp's copies have landed before it leaves
    if (lane == 0) {
      for (uint32_t x = issued > (uint32_t)stages ? issued - stages : 0; x < issued; ++x)
        drain_phase(bar(full0 + x % stages), (x / stages) & 1);
    }
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------------- MMA ----
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
    // d += A B over the tile's 128 columns, A from the elementwise threads'
    // pairs: the first half of each part's columns of the buffer at a
    auto gather = [&](uint32_t d, uint32_t a, uint64_t b, bool acc) {
#pragma unroll
      for (int kk = 0; kk < kBlock / 16; ++kk)
        mma_f16_ts(d, a + (16 * kk / kCols) * kCols + (16 * kk % kCols) / 2,
                   b + (uint64_t)(kk * 128), id_g, (acc || kk > 0) ? 1u : 0u);
    };
    auto b1_off = [&](uint32_t x) { return (uint64_t)((x % kS1) * (kTile >> 4)); };
    auto b2_off = [&](uint32_t x) { return (uint64_t)((x % kB2Stages) * (kTile >> 4)); };
    auto issue_x = [&](uint32_t x) {
      product(tmem + col_x(x), da1, db1 + b1_off(x));
      mma_commit(bar(BX + (x & 1)));
    };
    auto issue_y = [&](uint32_t x) {
      product(tmem + col_y(x), da2, db2 + b2_off(x));
      mma_commit(bar(BY + (x & 1)));
    };
    auto wait_b1 = [&](uint32_t x) { return wait_phase(bar(BB1 + x % kS1), (x / kS1) & 1, ctl); };
    auto wait_b2 = [&](uint32_t x) {
      return wait_phase(bar(BB2 + x % kB2Stages), (x / kB2Stages) & 1, ctl);
    };
    // the products of one block; false when a wait ran out
    auto block = [&]() -> bool {
      if (!wait_phase(bar(BA), full & 1, ctl) || !wait_b1(T)) return false;
      tc_fence_after();
      issue_x(T);
      if (!wait_b2(T)) return false;
      issue_y(T);
      if (n == 1) mma_commit(bar(BAFREE));
      if (kThree && n > 1) {
        if (!wait_b1(T + 1)) return false;
        issue_x(T + 1);
      }
      // Y(x), and whether it was the block's last product with A1 or A2
      auto next_y = [&](uint32_t x) {
        if (!wait_b2(x)) return false;
        issue_y(x);
        if (x + 1 == T + n) mma_commit(bar(BAFREE));
        return true;
      };
      for (int t = 0; t < n; ++t) {
        const uint32_t x = T + t;
        if (!wait_phase(bar(BP + (x & 1)), (x >> 1) & 1, ctl)) return false;
        // the last block's sums are out of tensor memory
        if (t == 0 && full > 0 && !wait_phase(bar(BFREE), (full - 1) & 1, ctl)) return false;
        tc_fence_after();
        if constexpr (kKeys) {
          gather(tmem + kColG2, tmem + col_x(x), dm2 + b2_off(x), t > 0);
          mma_commit(bar(BG2 + x % kB2Stages));
        }
        if (t + 1 < n) {
          if constexpr (kThree) {
            if (!next_y(x + 1)) return false;
          } else {
            if (!wait_b1(x + 1)) return false;
            issue_x(x + 1);
          }
        }
        if (!wait_phase(bar(BS + (x & 1)), (x >> 1) & 1, ctl)) return false;
        tc_fence_after();
        gather(tmem + kColG1, tmem + col_y(x), dm1 + b1_off(x), t > 0);
        mma_commit(bar(BG1 + x % kS1));
        if constexpr (kThree) {
          if (t + 2 < n) {
            if (!wait_b1(x + 2)) return false;
            issue_x(x + 2);
          }
        } else if (t + 1 < n) {
          if (!next_y(x + 1)) return false;
        }
      }
      return true;
    };
    for (bool ok = true; ok;) {
      if (take(n) < 0) break;
      if (n <= 0) continue;
      ok = !elect_one() || block();
      ok = __all_sync(0xffffffffu, ok);
      T += n;
      ++full;
    }
    if (elect_one()) {  // (the same lane every time)
      // every MMA issued above has completed once this commit fires
      mma_commit(bar(BDRAIN));
      drain_phase(bar(BDRAIN), 0);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------- elementwise ----
    const int part = warp >> 2;  // columns kCols part .. + kCols - 1 of a tile
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t lane_addr = lanes + part * kCols;
    // all lanes' tensor-memory writes and reads are behind the arrival
    auto arrive = [&](uint32_t slot) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(slot));
    };
    const float2 sc2 = make_float2(scale_log2, scale_log2);
    // the next block and, dQ, this thread's -lse and -D of it
    int row, next_n = 0;
    float next_nl = 0.f, next_nd = 0.f;
    auto ahead = [&]() {
      row = take(next_n);
      if (!kKeys && row >= 0 && next_n > 0) {
        const int bh = row / g.NB;
        const int64_t at = (int64_t)bh * g.Np + (row - bh * g.NB) * kBlock + r;
        next_nl = __ldg(args.nlse + at);
        next_nd = __ldg(args.ndel + at);
      }
    };
    ahead();
    for (bool ok = true; ok && row >= 0;) {
      n = next_n;
      const int this_row = row, bh = row / g.NB, blk = row - bh * g.NB;
      const float2 nl2 = make_float2(next_nl, next_nl), nd2 = make_float2(next_nd, next_nd);
      if (n < 0) {  // a malformed list: nothing is written
        ahead();
        continue;
      }
      int tail = kBlock;  // dQ: valid keys of the last listed tile
      // the list ascends: only its last entry can be the head's last block
      if (!kKeys && n > 0 &&
          __ldg(args.idx + (int64_t)this_row * args.k_max + n - 1) == g.NB - 1)
        tail = g.N - (g.NB - 1) * kBlock;
      for (int t = 0; t < n; ++t, ++T) {
        const float4* stat =
            reinterpret_cast<const float4*>(smem + kOffStats + (T % kS1) * 2 * kStatBytes) +
            part * (kCols / 4);
        if constexpr (kKeys)  // the statistics came with B1(T)
          if (!all_wait(bar(BB1 + T % kS1), (T / kS1) & 1, ctl)) { ok = false; break; }
        if (!warp_wait(bar(BX + (T & 1)), (T >> 1) & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        uint32_t x[kCols], pk[kCols / 2];
        const uint32_t x_col = lane_addr + col_x(T), y_col = lane_addr + col_y(T);
        tmem_ld32(x_col, x);
        if constexpr (!kKeys) arrive(BP + (T & 1));  // X is read: its buffer is free
        float2 p[kCols / 2];
#pragma unroll
        for (int c = 0; c < kCols / 2; c += 2) {
          float2 n0 = nl2, n1 = nl2;
          if constexpr (kKeys) {
            const float4 v = stat[c / 2];
            n0 = make_float2(v.x, v.y);
            n1 = make_float2(v.z, v.w);
          }
          const float2 e0 = ffma2(
              make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), sc2, n0);
          const float2 e1 = ffma2(
              make_float2(__uint_as_float(x[2 * c + 2]), __uint_as_float(x[2 * c + 3])), sc2, n1);
          p[c] = make_float2(ex2(e0.x), ex2(e0.y));
          p[c + 1] = make_float2(ex2(e1.x), ex2(e1.y));
        }
        if constexpr (kKeys) {
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) pk[c] = pack_bf16(p[c].x, p[c].y);
          tmem_st16_async(x_col, pk);
          tmem_wait_st();
          arrive(BP + (T & 1));
        } else if (tail < kBlock && t == n - 1) {  // warp-uniform: pad keys
#pragma unroll
          for (int c = 0; c < kCols / 2; ++c) {
            if (part * kCols + 2 * c >= tail) p[c].x = 0.f;
            if (part * kCols + 2 * c + 1 >= tail) p[c].y = 0.f;
          }
        }
        if (!warp_wait(bar(BY + (T & 1)), (T >> 1) & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        tmem_ld32(y_col, x);
#pragma unroll
        for (int c = 0; c < kCols / 2; c += 2) {
          float2 n0 = nd2, n1 = nd2;
          if constexpr (kKeys) {
            const float4 v = stat[kBlock / 4 + c / 2];
            n0 = make_float2(v.x, v.y);
            n1 = make_float2(v.z, v.w);
          }
          const float2 s0 = fmul2(
              p[c],
              fadd2(make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), n0));
          const float2 s1 = fmul2(
              p[c + 1],
              fadd2(make_float2(__uint_as_float(x[2 * c + 2]), __uint_as_float(x[2 * c + 3])), n1));
          pk[c] = pack_bf16(s0.x, s0.y);
          pk[c + 1] = pack_bf16(s1.x, s1.y);
        }
        tmem_st16_async(y_col, pk);
        tmem_wait_st();
        arrive(BS + (T & 1));
      }
      if (!ok) break;
      ahead();
      // ---- the block's sums: this part's columns of the thread's row, as bf16
      // pairs in registers, then to the natural position of its token
      constexpr int kOut = D / kParts, kPairs = kOut / 2;
      constexpr int kChunk = kOut < 32 ? kOut : 32;
      const int pos = blk * kBlock + r;
      const int64_t at =
          pos < g.N ? ((int64_t)bh * g.N + natural_index(g, g.perm[bh % g.heads], pos)) * D +
                          part * kOut
                    : -1;
      uint32_t o1[kPairs], o2[kKeys ? kPairs : 1];
      auto sums = [&](uint32_t col, float mul, uint32_t (&o)[kPairs]) {
#pragma unroll
        for (int c0 = 0; c0 < kOut; c0 += kChunk) {
          uint32_t f[kChunk];
          tmem_cols(lanes + col + part * kOut + c0, f);
#pragma unroll
          for (int c = 0; c < kChunk / 2; ++c)
            o[c0 / 2 + c] =
                pack_bf16(__uint_as_float(f[2 * c]) * mul, __uint_as_float(f[2 * c + 1]) * mul);
        }
      };
      if (n > 0) {
        const uint32_t last = T - 1;
        ok = warp_wait(bar(BG1 + last % kS1), (last / kS1) & 1, ctl);
        if (kKeys && ok) ok = warp_wait(bar(BG2 + last % kB2Stages), (last / kB2Stages) & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        sums(kColG1, scale, o1);
        if constexpr (kKeys) sums(kColG2, 1.f, o2);
        arrive(BFREE);
      } else {
#pragma unroll
        for (int c = 0; c < kPairs; ++c) {
          o1[c] = 0u;
          if constexpr (kKeys) o2[c] = 0u;
        }
      }
      if (at >= 0) {
#pragma unroll
        for (int c = 0; c < kPairs / 4; ++c) {
          reinterpret_cast<uint4*>((kKeys ? args.dk : args.dq) + at)[c] =
              make_uint4(o1[4 * c], o1[4 * c + 1], o1[4 * c + 2], o1[4 * c + 3]);
          if constexpr (kKeys)
            reinterpret_cast<uint4*>(args.dv + at)[c] =
                make_uint4(o2[4 * c], o2[4 * c + 1], o2[4 * c + 2], o2[4 * c + 3]);
        }
      }
    }
    __syncwarp();
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_sm100_kernel(const __grid_constant__ CUtensorMap map_q,
                     const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ CUtensorMap map_do,
                     const __grid_constant__ BwdArgs args, const __grid_constant__ Grid g,
                     float scale, float scale_log2) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t base = smem_u32(smem_raw);
  int32_t* status = args.status;
  if ((base & 1023u) != 0) {
    if (threadIdx.x == 0) report(status, PA_ERR_UNSUPPORTED);
    return;
  }
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + kOffSlot);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const int warp = threadIdx.x >> 5;
  const Ctl ctl{abort_flag, status, kTimeoutNs};
  // a wait of an earlier launch already expired: end quickly, with one answer
  // for the CTA: the status may change between its threads' reads
  if (__syncthreads_or(status != nullptr &&
                       *reinterpret_cast<volatile int32_t*>(status) == PA_ERR_TIMEOUT))
    return;
  if (threadIdx.x == 0) {
    for (uint32_t set = 0; set < 2; ++set)
      for (uint32_t b = 0; b < NBAR; ++b)
        mbar_init(base + kOffBar + (set * NBAR + b) * 8u,
                  b >= BP && b <= BFREE ? kAluWarps
                  : b == BTAKEN || b == BTAKEN + 1u ? kTakers
                                                    : 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bwd_blocks<true, D>(map_k, map_v, map_q, map_do, args, g, scale, scale_log2, smem_raw, base, tmem,
                      ctl);
  tc_fence_before();
  const bool aborted = __syncthreads_or(*abort_flag != 0);
  tc_fence_after();
  if (!aborted)
    bwd_blocks<false, D>(map_q, map_do, map_k, map_v, args, g, scale, scale_log2, smem_raw, base,
                         tmem, ctl);
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch_typed(const BwdArgs& a, const Grid& g, cudaStream_t s) {
  constexpr uint32_t kTile = kBlock * D * 2;
  constexpr int kSmem = kSmall<D> + (2 + kB1Stages<false, D> + kB2Stages) * kTile;
  static_assert(kSmem <= kSmemOptIn && kB1Stages<true, D> <= kB1Stages<false, D>, "shared memory");
  const cudaError_t e = opt_in_smem<bwd_sm100_kernel<D>>(kSmem);
  if (e != cudaSuccess) return e;
  const uint64_t rows = (uint64_t)g.B * g.heads * g.Np;
  CUtensorMap mq{}, mk{}, mv{}, md{};
  if (!encode_tile_map(&mq, a.q, rows, D, 2, 64, kBlock) ||
      !encode_tile_map(&mk, a.k, rows, D, 2, 64, kBlock) ||
      !encode_tile_map(&mv, a.v, rows, D, 2, 64, kBlock) ||
      !encode_tile_map(&md, a.dop, rows, D, 2, 64, kBlock))
    return cudaErrorInvalidValue;
  const int64_t blocks = (int64_t)g.B * g.heads * g.NB;
  bwd_sm100_kernel<D><<<(unsigned)(blocks < kSms ? blocks : kSms), kThreads, kSmem, s>>>(
      mq, mk, mv, md, a, g, (float)(1.0 / sqrt((double)D)),
      (float)(1.4426950408889634 / sqrt((double)D)));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bwd_sm100(const BwdArgs& a, const Grid& g, cudaStream_t s) {
  return g.d == 64 ? launch_typed<64>(a, g, s) : launch_typed<128>(a, g, s);
}

}  // namespace paro
