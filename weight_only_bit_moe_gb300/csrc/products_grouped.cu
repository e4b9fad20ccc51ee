// 16-bit products grouped by expert on tcgen05 tensor cores (sm_103a).
//
//   forward  out[r, j]    = sum_t x[r, t]  W[e][j, t]     j over N, t over K
//   dx       out[r, j]    = sum_t dy[r, t] W[e][t, j]     j over K, t over N
//   dW       out[e][i, j] = sum_{r in e} dy[r, i] x[r, j]
//
// One kernel for the three.  A pair of CTAs (cluster of two, cta_group::2)
// computes 256 x n output values: P, 256 rows on the MMA's M side, 128 in each
// CTA; Q, n <= 256 rows on its N side, half in each CTA's shared memory.
//   forward, dx: P = output features j, Q = rows of one expert.  The ragged
//     dimension sits on the N side because n is a field of the instruction: a
//     tile of m rows costs round_up(m, 32) / 256 of a full one, and a group's
//     rows are cut into equal tiles.
//   dW: P = dy's columns, Q = x's columns; the ragged dimension is the sum.
// The operand order is the bank's own: forward reads both operands with the sum
// innermost, dx reads W with j innermost and dW both operands so, through the
// MN-major descriptors -- nothing is transposed in memory.  Results leave through
// shared memory: dW's by TMA, added to what is there when it accumulates, the others
// as stores of 256 bytes of a row.
//
// A stage is 64 terms of the sum (128-byte lines, 128-byte swizzle), 32 KB per
// CTA, six in flight (dW: five).  Roles: three producer warps per CTA issue TMA,
// one for P and two for Q, counted by the leader's barrier; the leader's MMA warp
// issues; eight epilogue warps per CTA drain one of two TMEM accumulators while the
// MMAs fill the other.  Row tiles are fetched in boxes as large as they are, so a
// decode step moves the weights and little else.  dW's last stage of a group fetches
// its rows past whole sixteens by index, those past the group's end as zeros.
//
// When there are fewer tiles than CTA pairs the sum is cut into S slices, each a
// work item; the last pair to finish a tile adds the slices in their order, so
// results do not depend on timing.
//
// Bounds and measurements (GB300; copy rate 6.8 TB/s, bf16 1880 TFLOP/s):
//   8192 rows x 4096 x 4096, one expert: MMAs, 140 to 144 us = 1910 to 1960 TFLOP/s
//     (library 1980 to 2050 at 8192^3); dx the same, dW in 16 bits 164 us.
//   128 rows over 128 experts of 4096 x 1536: weights from memory, 95 us = 6.5 TB/s.
//   128 experts of 256 rows, 4096 x 1536: memory, 292 to 296 us (floor 292); of
//     2048 x 768, 91 us (floor 86).
//   32 experts of 256 and of 270 rows, 2880 x 2880: 114 and 136 us; past 256 rows the
//     weights pass from L2 twice, once for each row tile.
//   A stage takes at least 0.20 us whatever its rows (issue of its copies and MMAs).
#include <atomic>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "gemm.cuh"
#include "products_tc.cuh"

namespace moe {

constexpr int kGtThreads = 384;       // three producer warps, MMA, eight epilogue warps
constexpr int kGtEpiWarp0 = 4, kGtEpiWarps = 8, kGtEpiThreads = 256;
constexpr int kGtP = 256;             // P rows per pair
constexpr int kGtN = 256;             // Q rows per pair, at most
constexpr int kGtGran = 32;           // n is a multiple of this for cta_group::2, M = 256
constexpr int kGtSorted = 512;        // dW: experts that are taken by falling size, at most
constexpr int kGtOperandBytes = 128 * 128;              // 128 rows x 64 terms of 16 bits
constexpr int kGtStageBytes = 2 * kGtOperandBytes;      // P and Q

struct GroupedTcArgs {
  CUtensorMap map_p;
  CUtensorMap map_out;   // dW: boxes of 32 rows x 128 bytes of the output
  union {
    CUtensorMap map_q[4];     // by row: boxes of 128, 64, 32 and 16 rows of Q
    CUtensorMap map_tail[4];  // dW: boxes of 16 rows and of one, of P and of Q
  };
  CUtensorMap map_dw_q;       // dW: boxes of Q
  ProdArgs g;
  int pairs;             // CTA pairs of the launch
  int wide_store;        // fp32 dW: 32-byte stores are aligned
  int blocked;           // operands stored MN-major have whole blocks of 64 columns: one box brings two
};

template <int MODE>
struct GtSmem {
  static constexpr int kStages = MODE == kProdDw ? 5 : 6;
  static constexpr int kOut = kStages * kGtStageBytes;  // two 4 KB buffers per epilogue warp (dW) or four of them
  static constexpr int kOutBytes = MODE == kProdDw ? kGtEpiWarps * 2 * 4096 : 2 * 2 * 4096;
  static constexpr int kBar = kOut + kOutBytes;
  static constexpr int kNumBars = 2 * kStages + 4 + 1;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kBytes = kMisc + 32;
  static constexpr int kAlloc = kBytes + 1024;
  static constexpr int kStatic = (MODE == kProdDw ? kGtSorted * 2 : (kProdGroups + 1) * 4) + 64;
  static_assert(kAlloc + kStatic <= 227 * 1024, "shared memory over the per-CTA limit");
};

// Items of dW: a regular grid of tiles, x's columns fastest, each cut into S
// slices, the experts by falling size (order; none: in their own order).  Pairs take
// items in turn, and then those of a turn cost about the same: experts drawn by
// Zipf's law, 71 of 1160 x 1400, 459 rows on average, take 147 us by size and 159 by
// number.  A role steps from item to item with carries instead of divisions.
struct DwWalk {
  int p_tiles, q_tiles, S;
  int e, p, q, s;          // the item's expert, tile and slice
  int de, dp, dq, ds;      // the step
  __device__ __forceinline__ void split(int w, int& e, int& p, int& q, int& s) const {
    s = w % S;
    w /= S;
    q = w % q_tiles;
    w /= q_tiles;
    p = w % p_tiles;
    e = w / p_tiles;
  }
  __device__ __forceinline__ void init(int p_tiles_, int q_tiles_, int S_, int first, int step) {
    p_tiles = p_tiles_, q_tiles = q_tiles_, S = S_;
    split(first, e, p, q, s);
    split(step, de, dp, dq, ds);
  }
  __device__ __forceinline__ void next() {
    s += ds, q += dq, p += dp, e += de;
    if (s >= S) s -= S, ++q;
    if (q >= q_tiles) q -= q_tiles, ++p;
    if (p >= p_tiles) p -= p_tiles, ++e;
  }
  __device__ __forceinline__ ProdItem item(const ProdArgs& g, const uint16_t* order) const {
    ProdItem it;
    it.tile = (e * p_tiles + p) * q_tiles + q;
    it.split = s;
    it.e = order ? order[e] : e;
    it.p0 = p * kGtP;
    it.q0 = q * kGtN;
    it.n = min(kGtN, g.K - it.q0);
    int r0, r1;
    group_rows(g, it.e, r0, r1);
    const int stages = (r1 - r0 + 63) / 64;
    it.t0 = 0;
    it.t1 = stages;
    if (S > 1) {
      it.t0 = (int)((int64_t)s * stages / S);
      it.t1 = (int)((int64_t)(s + 1) * stages / S);
    }
    return it;
  }
};

// A role's position among the items of a launch.
template <int MODE>
struct GtWalk {
  DwWalk dw;
  int w, e, step;
  __device__ __forceinline__ GtWalk(const RowPlan& pl, int q_tiles, int pair, int pairs) : w(pair), e(0), step(pairs) {
    if (MODE == kProdDw) dw.init(pl.p_tiles, q_tiles, pl.S, pair, pairs);
  }
  __device__ __forceinline__ ProdItem item(const ProdArgs& g, const RowPlan& pl, const int* start, const uint16_t* order) {
    return MODE == kProdDw ? dw.item(g, order) : row_item<kGtN, kGtGran, kGtP>(g, pl, start, w, e);
  }
  __device__ __forceinline__ void next() {
    w += step;
    if (MODE == kProdDw) dw.next();
  }
};

// The last rows [row, r1) of a group, fewer than 64, of a block of 64 columns: whole
// sixteens as boxes, the rest by index in fours, rows at or past r1 as zeros (row
// `none` lies outside the tensor).
__device__ __forceinline__ void gt_tail(const CUtensorMap* sixteen, const CUtensorMap* single, int col, int row, int r1,
                                        int none, uint32_t slot, uint32_t bar) {
  int b = row;
  for (; b + 16 <= r1; b += 16, slot += 2048) tma2_2d(slot, sixteen, col, b, bar);
  if (b == r1) return;
#pragma unroll
  for (int i = 0; i < 4; ++i, b += 4, slot += 512) {
    const int4 r = make_int4(b < r1 ? b : none, b + 1 < r1 ? b + 1 : none, b + 2 < r1 ? b + 2 : none,
                             b + 3 < r1 ? b + 3 : none);
    tma2_gather4(slot, single, col, r, bar);
  }
}

// One CTA's share of a stage of P and of Q.
template <int MODE>
__device__ __forceinline__ void gt_load_p(const GroupedTcArgs& a, const ProdItem& it, int t, int p, int row, int r1,
                                          uint32_t slot, uint32_t bar) {
  if (MODE == kProdFwd) {
    tma2_3d(slot, &a.map_p, 64 * t, p, it.e, bar);
  } else if (MODE == kProdDx) {
    if (a.blocked) {
      tma2_4d(slot, &a.map_p, 0, 64 * t, p / 64, it.e, bar);
    } else {
      tma2_3d(slot, &a.map_p, p, 64 * t, it.e, bar);
      tma2_3d(slot + 8192, &a.map_p, p + 64, 64 * t, it.e, bar);
    }
  } else if (r1 - row < 64) {
    gt_tail(&a.map_tail[0], &a.map_tail[1], p, row, r1, a.g.rows, slot, bar);
    gt_tail(&a.map_tail[0], &a.map_tail[1], p + 64, row, r1, a.g.rows, slot + 8192, bar);
  } else if (a.blocked) {
    tma2_3d(slot, &a.map_p, 0, row, p / 64, bar);
  } else {
    tma2_2d(slot, &a.map_p, p, row, bar);
    tma2_2d(slot + 8192, &a.map_p, p + 64, row, bar);
  }
}
// Q has two producers: by row the boxes of 128 and 64 rows and those of 32 and 16
// (a stage with three boxes took longer than its MMAs from one warp); dW's tail by
// column block.
template <int MODE>
__device__ __forceinline__ void gt_load_q(const GroupedTcArgs& a, int which, int t, int q, int half, int row, int r1,
                                          uint32_t slot, uint32_t bar) {
  if (MODE != kProdDw) {
    int at = which == 0 ? 0 : half & ~63;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int box = (which == 0 ? 128 : 32) >> i;
      if (half & box) {
        tma2_2d(slot + 128 * at, &a.map_q[2 * which + i], 64 * t, q + at, bar);
        at += box;
      }
    }
  } else if (r1 - row < 64) {
    gt_tail(&a.map_tail[2], &a.map_tail[3], q + 64 * which, row, r1, a.g.rows, slot + 8192 * which, bar);
  } else if (a.blocked) {
    if (which == 0) tma2_3d(slot, &a.map_dw_q, 0, row, q / 64, bar);
  } else {
    tma2_2d(slot + 8192 * which, &a.map_dw_q, q + 64 * which, row, bar);
  }
}

// Q rows per CTA of a tile of n rows; whole 64-column blocks where Q is stored MN-major.
template <int MODE>
__device__ __forceinline__ int gt_half(int n) {
  if (MODE == kProdDw) return n > 128 ? 128 : 64;
  return (n + kGtGran - 1) / kGtGran * (kGtGran / 2);
}

// Bytes that both CTAs' loads of stage t bring.
template <int MODE>
__device__ __forceinline__ uint32_t gt_stage_bytes(int half, int v) {
  if (MODE == kProdDw) return 2u * (uint32_t)(v == 64 ? 64 : (v + 15) / 16 * 16) * 128u * 4u;
  return 2u * (uint32_t)(kGtOperandBytes + half * 128);
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGtThreads, 1)
    grouped_tc_kernel(const __grid_constant__ GroupedTcArgs a) {
  using SM = GtSmem<MODE>;
  constexpr int kStages = SM::kStages;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ int start[MODE == kProdDw ? 1 : kProdGroups + 1];  // first tile of each group
  __shared__ uint16_t sorted[MODE == kProdDw ? kGtSorted : 1];  // dW: experts by falling size
  const uint16_t* order = nullptr;
  __shared__ int warp_tot[kGtThreads / 32];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem_s = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM::kBar);
  uint64_t* full = bars;                    // the leader's count both CTAs' copies
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + 2;       // the leader's
  uint64_t* drain_bar = acc_empty + 2;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + SM::kMisc);  // [0] tmem base, [1] abort, [2] last
  volatile int* abort_flag = reinterpret_cast<volatile int*>(&misc[1]);
  const ProdArgs& g = a.g;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x >> 1;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], 2 * kGtEpiWarps); }
    mbar_init(drain_bar, 1);
    misc[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc2(&misc[0], 512);
    tmem_relinquish2();
  }

  if (warp == 0 && lane < 6) prefetch_map(lane < 4 ? &a.map_q[lane] : lane == 4 ? &a.map_p : &a.map_out);
  // (launched early: everything before this line touches nothing that an earlier kernel writes)
  grid_dependents_launch();
  grid_dependency_wait();
  // --- the plan: tiles per group (rows), or a regular grid of tiles (dW)
  RowPlan pl;
  const int j_dim = MODE == kProdDx ? g.K : g.N;
  pl.p_tiles = (j_dim + kGtP - 1) / kGtP;
  pl.stages = ((MODE == kProdDx ? g.N : g.K) + 63) / 64;
  const int q_tiles = (g.K + kGtN - 1) / kGtN;  // dW
  if (MODE == kProdDw) {
    if (blockIdx.x == 0)
      for (int e = tid; e < g.E; e += kGtThreads)
        if (group_bad(g, e)) atomicOr(g.status, kStatusRouting);
    // (With at most one tile to a pair the order does not matter, and with more than
    // three tiles to four pairs two to four slices take as many rounds: there the sizes
    // would cost 0.9 us for nothing.)
    pl.tiles = g.E * pl.p_tiles * q_tiles;
    if (g.E <= kGtSorted && (pl.tiles > a.pairs || 4 * pl.tiles <= 3 * a.pairs)) {
      order = sorted;
      int* size = reinterpret_cast<int*>(smem);  // (the ring, before its first copy)
      for (int e = tid; e < g.E; e += kGtThreads) {
        int r0, r1;
        group_rows(g, e, r0, r1);
        size[e] = r1 - r0;
      }
      __syncthreads();
      for (int e = tid; e < g.E; e += kGtThreads) {
        const int mine = size[e];
        int larger = 0;
#pragma unroll 8
        for (int j = 0; j < g.E; ++j) larger += size[j] > mine || (size[j] == mine && j < e);
        sorted[larger] = (uint16_t)e;
      }
      fence_async_proxy();
    }
  } else {
    plan_groups<kGtN, kGtThreads>(g, pl.p_tiles, start, warp_tot);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before either signals them
  tc_fence_after();
  const uint32_t tmem = misc[0];
  if (MODE == kProdDw) {  // slices for the longest sum, or the average one
    int r0 = 0, r1 = g.rows / g.E;
    if (order) group_rows(g, order[0], r0, r1);
    pl.stages = (r1 - r0 + 63) / 64;
  } else {
    pl.tiles = min(start[g.E], kProdItems);
  }
  pl.S = plan_slices(pl, a.pairs, 2, MODE == kProdDw ? 1 << 30 : g.rows, kGtN);
  const int items = pl.tiles * pl.S;
  const uint32_t full_s = map_to_rank(smem_u32(full), 0);

  if (warp == 0 || (warp >= 2 && warp < kGtEpiWarp0)) {
    // ------------------------------------------------------------ producers of P (warp 0) and Q (warps 2, 3)
    Ring<kStages> slot;
    uint32_t filled = 0;
    for (GtWalk<MODE> at(pl, q_tiles, pair, a.pairs); at.w < items; at.next()) {
      const ProdItem it = at.item(g, pl, start, order);
      const int half = gt_half<MODE>(it.n);
      int r0 = 0, r1 = 0;
      if (MODE == kProdDw) group_rows(g, it.e, r0, r1);
      const int p = it.p0 + rank * 128, q = it.q0 + rank * half;
      for (int t = it.t0; t < it.t1; ++t) {
        const int row = r0 + 64 * t;
        if (!warp_wait(&empty[slot.i], slot.phase ^ 1, abort_flag, g.status)) break;
        const uint32_t dst = smem_s + slot.i * kGtStageBytes, bar = full_s + 8 * slot.i;
        if (warp == 0) {
          if (rank == 0) expect_tx_elect(&full[slot.i], gt_stage_bytes<MODE>(half, min(64, r1 - row)));
          gt_load_p<MODE>(a, it, t, p, row, r1, dst, bar);
        } else {
          gt_load_q<MODE>(a, warp - 2, t, q, half, row, r1, dst + kGtOperandBytes, bar);
        }
        slot.next();
        ++filled;
      }
      if (*abort_flag) break;
    }
    // leave no copy in flight (the leader's barriers count the peer's copies too)
    if (rank == 0 && warp == 0)
      for (uint32_t i = 0; i < (uint32_t)kStages && i < filled; ++i) {
        const uint32_t u = filled - 1 - i;
        mbar_drain(&full[u % kStages], (u / kStages) & 1, g.status);
      }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (rank == 0) {
      constexpr uint32_t kMajors = MODE == kProdFwd ? 0u : (MODE == kProdDx ? kIdescMajorA : (kIdescMajorA | kIdescMajorB));
      constexpr int kStepA = MODE == kProdFwd ? 2 : 128, kStepB = MODE == kProdDw ? 128 : 2;  // 16 terms, 16-byte units
      const uint32_t bf = g.in_type == kBf16 ? 1u : 0u;
      const uint64_t pd0 = MODE == kProdFwd ? smem_desc_sw128(smem_s) : smem_desc_sw128_mn(smem_s, 8192);
      const uint64_t qd0 = MODE == kProdDw ? smem_desc_sw128_mn(smem_s + kGtOperandBytes, 8192)
                                           : smem_desc_sw128(smem_s + kGtOperandBytes);
      Ring<kStages> slot;
      Ring<2> acc;
      for (GtWalk<MODE> at(pl, q_tiles, pair, a.pairs); at.w < items; at.next()) {
        const ProdItem it = at.item(g, pl, start, order);
        if (it.t0 >= it.t1) continue;  // (dW: no rows; the epilogue takes zeros)
        int r0 = 0, r1 = 0;
        if (MODE == kProdDw) group_rows(g, it.e, r0, r1);
        const uint32_t idesc = idesc_f16_f32(256, 2 * gt_half<MODE>(it.n), bf) | kMajors;
        warp_wait(&acc_empty[acc.i], acc.phase ^ 1, abort_flag, g.status);
        const uint32_t d = tmem + acc.i * kGtN;
        for (int t = it.t0; t < it.t1; ++t) {
          if (!warp_wait(&full[slot.i], slot.phase, abort_flag, g.status)) break;
          tc_fence_after();
          const uint32_t at_slot = slot.i * (kGtStageBytes >> 4);  // (descriptor addresses count 16 bytes and do not carry)
          const uint64_t pd = pd0 + at_slot, qd = qd0 + at_slot;
          const int rows = MODE == kProdDw ? r1 - (r0 + 64 * t) : 64;
          if (rows > 48) {
            umma2_f16_stage_elect<kStepA, kStepB>(d, pd, qd, idesc, t > it.t0 ? 1u : 0u);
          } else {
            for (int i = 0; 16 * i < rows; ++i)
              umma2_f16_elect(d, pd + i * kStepA, qd + i * kStepB, idesc, (t > it.t0 || i > 0) ? 1u : 0u);
          }
          umma2_commit_elect(&empty[slot.i]);
          slot.next();
        }
        umma2_commit_elect(&acc_full[acc.i]);
        acc.next();
      }
      umma2_commit_elect(drain_bar);
      mbar_drain(drain_bar, 0, g.status);
      __syncwarp();
    }
  } else if (warp >= kGtEpiWarp0) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, sub = (warp - kGtEpiWarp0) >> 2;  // TMEM lanes; which 32-column chunks
    const int et = tid - kGtEpiWarp0 * 32;
    const uint32_t acc_empty_s = map_to_rank(smem_u32(acc_empty), 0);
    const uint32_t boxes = smem_s + SM::kOut + (warp - kGtEpiWarp0) * 8192;  // dW: this warp's output boxes
    const uint32_t rows16 = smem_s + SM::kOut + sub * 8192;  // fwd, dx: buffers of sixteen rows of these four warps
    int32_t* counters = reinterpret_cast<int32_t*>(g.scratch);
    uint4* partial = reinterpret_cast<uint4*>(g.scratch + kProdCounterBytes);
    uint32_t ic = 0, box = 0;
    for (GtWalk<MODE> at(pl, q_tiles, pair, a.pairs); at.w < items; at.next()) {
      const ProdItem it = at.item(g, pl, start, order);
      if (MODE == kProdDw && g.accumulate) {  // nothing is added for an expert without rows: its part keeps its bits
        int r0, r1;
        group_rows(g, it.e, r0, r1);
        if (r0 == r1) continue;  // (in every warp and slice: no accumulator or counter moves)
      }
      const int p = it.p0 + rank * 128 + quarter * 32;  // this warp's first P row
      const bool none = it.t0 >= it.t1;                 // no terms: the sums are zeros
      const int acc = ic & 1;
      if (!none) {
        warp_wait(&acc_full[acc], (ic >> 1) & 1, abort_flag, g.status);
        tc_fence_after();
      }
      const uint32_t tb = tmem + ((uint32_t)(quarter * 32) << 16) + acc * kGtN;
      const int chunks = (it.n + 31) / 32;
      // A thread's sums of a partial tile, 16 bytes per thread and step, in its own order.
      const int64_t slice = 128 * kGtN / 4;
      uint4* mine = partial + ((int64_t)it.tile * pl.S * 2 + rank) * slice + quarter * 32 + lane;
      bool finish = true;
      if (pl.S > 1) {
        for (int c = sub; c < chunks; c += 2) {
          uint32_t v[32];
          if (none) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
          } else {
            tmem_ld32(tb + 32 * c, v);
            tmem_ld_wait();
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            __stcg(mine + it.split * 2 * slice + (c * 8 + i) * 128, make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
        }
        named_bar_sync(1, kGtEpiThreads);
        if (et == 0) misc[2] = slice_arrive_last(&counters[it.tile * 2 + rank], pl.S) ? 1u : 0u;
        named_bar_sync(1, kGtEpiThreads);
        finish = misc[2] != 0;
      }
      // 32 columns of the tile: from the slices, from tensor memory, or zeros
      auto columns = [&](int c, uint32_t (&v)[32]) {
        if (pl.S > 1) {
          float f[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) f[i] = 0.0f;
          const uint4* src = mine + c * 8 * 128;
#pragma unroll 4
          for (int s = 0; s < pl.S; ++s, src += 2 * slice) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 u = __ldcg(reinterpret_cast<const float4*>(src) + i * 128);
              f[4 * i] += u.x, f[4 * i + 1] += u.y, f[4 * i + 2] += u.z, f[4 * i + 3] += u.w;
            }
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(f[i]);
        } else if (!none) {
          tmem_ld32(tb + 32 * c, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
      };
      if (finish && MODE == kProdDw) {
        // lane = row of dW[e], registers = 32 consecutive columns, 128 bytes of the row (two halves of
        // them when the output has 16 bits): into the warp's box, swizzled, and on by TMA, which writes
        // whole lines and cuts the box at the matrix's edges.  Of fp32 output half the warps store their
        // rows' columns themselves, 32 bytes a lane: boxes alone load the shared memory that the MMAs
        // read from (171 us for 32 empty experts of 2880 x 2880, but 223 to 232 with 230 or 250 rows
        // each), stores alone the L1's line rate (191, and 223 to 226); halved, 171 and 205 to 207.
        const bool wide = g.out_type == kFp32;
        const int per_warp = kGtN / 2 / (wide ? 32 : 64);
        for (int i = 0; i < per_warp; ++i) {
          const int c = sub * 4 + (wide ? i : 2 * i);  // first 32-column chunk of the box
          if (32 * c >= it.n || p >= g.N) continue;
          if (a.wide_store && !g.accumulate && wide && sub == 1) {
            uint32_t v[32];
            columns(c, v);
            const int row = p + lane, col = it.q0 + 32 * c;
            if (row < g.N) {
              float* dst = static_cast<float*>(g.out) + it.e * g.out_se + (int64_t)row * g.out_ld + col;
#pragma unroll
              for (int b = 0; b < 32; b += 8) {
                const uint32_t o[8] = {v[b], v[b + 1], v[b + 2], v[b + 3], v[b + 4], v[b + 5], v[b + 6], v[b + 7]};
                if (col + b < g.K) stg256(dst + b, o);  // (K is a multiple of 8)
              }
            }
            __syncwarp();  // whole warps read tensor memory
            continue;
          }
          const uint32_t dst = boxes + (box & 1) * 4096;
          if (lane == 0) tma_store_wait_read<1>();  // the box before last has been read
          __syncwarp();
          const uint32_t row = dst + lane * 128;
          uint32_t v[32];
          columns(c, v);
          if (wide) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              sts128(row + ((j ^ (lane & 7)) << 4), make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (h == 1) {
                if (32 * (c + 1) >= it.n) break;  // (columns past the edge are cut)
                columns(c + 1, v);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t o[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  const float lo = __uint_as_float(v[8 * j + 2 * u]), hi = __uint_as_float(v[8 * j + 2 * u + 1]);
                  o[u] = g.out_type == kBf16 ? pack_bf16x2(lo, hi) : pack_half2(lo, hi);
                }
                sts128(row + (((4 * h + j) ^ (lane & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
              }
            }
          }
          fence_async_proxy();
          __syncwarp();
          if (lane == 0) {
            if (g.accumulate) tma_store_3d<true>(&a.map_out, it.q0 + 32 * c, p, it.e, dst);
            else tma_store_3d<false>(&a.map_out, it.q0 + 32 * c, p, it.e, dst);
          }
          ++box;
        }
      } else if (finish) {
        for (int c = sub; c < chunks; c += 2) {
          uint32_t v[32];
          columns(c, v);
          // lane = feature, registers = 32 rows.  Sixteen at a time go through shared memory, where the four
          // warps' features come together: a store then writes 256 bytes of a row.  (Transposed by shuffles,
          // 64 bytes of a row per warp and store: 10 experts of 1408 rows, 6656 x 512, 105 us; this way 78.)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (32 * c + 16 * h >= it.n) break;
            const uint32_t buf = rows16 + (box++ & 1) * 4096;
            const uint32_t col = buf + (quarter * 32 + lane) * 2;
#pragma unroll
            for (int u = 0; u < 16; u += 2) {
              const float lo = __uint_as_float(v[16 * h + u]), hi = __uint_as_float(v[16 * h + u + 1]);
              const uint32_t two = g.out_type == kBf16 ? pack_bf16x2(lo, hi) : pack_half2(lo, hi);
              sts16(col + 256 * u, two);
              sts16(col + 256 * u + 256, two >> 16);
            }
            named_bar_sync(2 + sub, kGtEpiThreads / 2);  // (a buffer's readers are past the barrier after theirs)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int r = quarter * 4 + 2 * b + (lane >> 4), row = 32 * c + 16 * h + r;
              const int j = it.p0 + rank * 128 + (lane & 15) * 8;
              const uint4 o = lds128(buf + r * 256 + ((lane & 15) << 4));
              if (row < it.n && j < j_dim)
                stg128(static_cast<uint16_t*>(g.out) + (int64_t)(it.q0 + row) * g.out_ld + j, o);
            }
          }
          __syncwarp();  // whole warps read tensor memory
        }
      }
      if (!none) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty_s + 8 * acc);
        ++ic;
      }
    }
    if (MODE == kProdDw && lane == 0) tma_store_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the other may signal or read it
  tc_fence_after();
  if (warp == 1) tmem_dealloc2(tmem, 512);
}

// ---------------------------------------------------------------- host
static PFN_cuTensorMapEncodeTiled_v12000 prod_map_encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> cached{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 fn = cached.load(std::memory_order_acquire);
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    cached.store(fn, std::memory_order_release);
  }
  return fn;
}

bool make_prod_map(CUtensorMap* m, int elem_type, const void* base, int nd, const uint64_t* dims,
                   const uint64_t* strides, const uint32_t* box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = prod_map_encoder();
  if (!enc) return false;
  cuuint64_t d[4], s[3];
  cuuint32_t b[4], es[4] = {1u, 1u, 1u, 1u};
  for (int i = 0; i < nd; ++i) d[i] = dims[i], b[i] = box[i];
  for (int i = 0; i + 1 < nd; ++i) s[i] = strides[i];
  const CUtensorMapDataType t = elem_type == kBf16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                : elem_type == kFp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                : elem_type == kFp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                     : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  return enc(m, t, (cuuint32_t)nd, const_cast<void*>(base), d, s, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int prod_sm_count() {
  static std::atomic<int> cache[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = cache[dev].load(std::memory_order_acquire);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cache[dev].store(n, std::memory_order_release);
  }
  return n;
}

template <int MODE>
static cudaError_t launch_mode(GroupedTcArgs& a, cudaStream_t st) {
  static std::atomic<bool> ready[64] = {};
  int dev = 0;
  cudaError_t rc = cudaGetDevice(&dev);
  if (rc != cudaSuccess) return rc;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    rc = cudaFuncSetAttribute(grouped_tc_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, GtSmem<MODE>::kAlloc);
    if (rc != cudaSuccess) return rc;
    ready[dev].store(true, std::memory_order_release);
  }
  return launch_dependent(grouped_tc_kernel<MODE>, dim3(2 * a.pairs), dim3(kGtThreads), GtSmem<MODE>::kAlloc, st, a);
}

static bool grid16(const void* p, int64_t stride) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0 && stride < ((int64_t)1 << 38);
}

cudaError_t launch_grouped_tc(const ProdArgs& g, int mode, cudaStream_t st, bool* done) {
  *done = false;
  const int out_cols = mode == kProdFwd ? g.N : g.K;
  // stores and descriptors work on 8 elements: the contiguous dimensions must be whole eights
  if (g.rows == 0 || out_cols % 8 || !grid16(g.a, g.a_ld) || !grid16(g.w, g.w_ld) || !grid16(g.out, g.out_ld)) return cudaSuccess;
  if (mode == kProdDw ? (g.out_se % 8 != 0) : (g.w_se % 8 != 0 || (g.w_se <= 0 && g.E > 1))) return cudaSuccess;
  // tile numbers are 32-bit
  const double tiles = (mode == kProdDw ? (double)g.E * ((g.N + kGtP - 1) / kGtP) : (double)g.rows / kGtN + g.E) *
                       ((out_cols + 255) / 256);
  if (tiles > 1e9) return cudaSuccess;
  GroupedTcArgs a;
  a.g = g;
  const uint64_t ald = (uint64_t)g.a_ld * 2, wld = (uint64_t)g.w_ld * 2;
  const uint64_t N = (uint64_t)g.N, K = (uint64_t)g.K, rows = (uint64_t)g.rows, E = (uint64_t)g.E;
  const int ty = g.in_type;
  bool ok;
  if (mode == kProdDw) {
    a.blocked = g.N % 64 == 0 && g.K % 64 == 0;
    const uint64_t dp[2] = {N, rows}, dq[2] = {K, rows};
    const uint32_t box[2] = {64, 64}, sixteen[2] = {64, 16}, one[2] = {64, 1};
    ok = make_prod_map(&a.map_tail[0], ty, g.a, 2, dp, &ald, sixteen) && make_prod_map(&a.map_tail[1], ty, g.a, 2, dp, &ald, one) &&
         make_prod_map(&a.map_tail[2], ty, g.w, 2, dq, &wld, sixteen) && make_prod_map(&a.map_tail[3], ty, g.w, 2, dq, &wld, one);
    if (a.blocked) {
      const uint64_t bp[3] = {64, rows, N / 64}, bq[3] = {64, rows, K / 64}, sp[2] = {ald, 128}, sq[2] = {wld, 128};
      const uint32_t two[3] = {64, 64, 2};
      ok = ok && make_prod_map(&a.map_p, ty, g.a, 3, bp, sp, two) && make_prod_map(&a.map_dw_q, ty, g.w, 3, bq, sq, two);
    } else {
      ok = ok && make_prod_map(&a.map_p, ty, g.a, 2, dp, &ald, box) && make_prod_map(&a.map_dw_q, ty, g.w, 2, dq, &wld, box);
    }
    const uint64_t each = g.out_type == kFp32 ? 4 : 2, od[3] = {K, N, E};
    const uint64_t os[2] = {(uint64_t)g.out_ld * each, (uint64_t)(g.E > 1 ? g.out_se : g.out_ld) * each};
    const uint32_t obox[3] = {128 / (uint32_t)each, 32, 1};
    ok = ok && make_prod_map(&a.map_out, g.out_type, g.out, 3, od, os, obox);
  } else {
    a.blocked = mode == kProdDx && g.K % 64 == 0;
    const uint64_t we = g.E > 1 ? (uint64_t)g.w_se * 2 : wld;
    if (a.blocked) {
      const uint64_t d[4] = {64, N, K / 64, E}, st4[3] = {wld, 128, we};
      const uint32_t two[4] = {64, 64, 2, 1};
      ok = make_prod_map(&a.map_p, ty, g.w, 4, d, st4, two);
    } else {
      const uint64_t d[3] = {K, N, E}, st3[2] = {wld, we};
      const uint32_t box[3] = {64, mode == kProdFwd ? 128u : 64u, 1};
      ok = make_prod_map(&a.map_p, ty, g.w, 3, d, st3, box);
    }
    const uint64_t da[2] = {mode == kProdFwd ? K : N, rows};
    for (int i = 0; i < 4 && ok; ++i) {
      const uint32_t box[2] = {64, 128u >> i};
      ok = make_prod_map(&a.map_q[i], ty, g.a, 2, da, &ald, box);
    }
  }
  if (mode != kProdDw) a.map_out = a.map_dw_q = a.map_p;
  if (!ok) return cudaSuccess;  // (the plain kernel takes what a tensor map cannot describe)
  const int sms = prod_sm_count();
  if (sms < 2 || sms > kProdWidth) return cudaErrorInvalidDevice;
  a.pairs = sms / 2;
  a.wide_store = (reinterpret_cast<uintptr_t>(g.out) & 31) == 0 && g.out_ld % 8 == 0 && g.out_se % 8 == 0;
  *done = true;
  if (mode == kProdFwd) return launch_mode<kProdFwd>(a, st);
  if (mode == kProdDx) return launch_mode<kProdDx>(a, st);
  return launch_mode<kProdDw>(a, st);
}

}  // namespace moe
