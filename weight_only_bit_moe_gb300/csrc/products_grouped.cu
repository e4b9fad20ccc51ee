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
// MN-major descriptors -- nothing is transposed in memory.
//
// A stage is 64 terms of the sum (128-byte lines, 128-byte swizzle), 32 KB per
// CTA, six in flight.  Roles: one producer thread per CTA issues TMA, counted
// by the leader's barrier; the leader's MMA warp issues; eight epilogue warps
// per CTA drain one of two TMEM accumulators while the MMAs fill the other.
// Row tiles are fetched in boxes as large as they are, so a decode step moves the
// weights and little else.  dW's last stage of a group fetches
// its rows by index (gather), rows past the group's end as zeros.
//
// When there are fewer tiles than CTA pairs the sum is cut into S slices, each a
// work item; the last pair to finish a tile adds the slices in their order, so
// results do not depend on timing.
#include <atomic>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "gemm.cuh"
#include "products_tc.cuh"

namespace moe {

constexpr int kGtThreads = 384;       // producer, MMA, two idle warps, eight epilogue warps
constexpr int kGtEpiWarp0 = 4, kGtEpiWarps = 8, kGtEpiThreads = 256;
constexpr int kGtP = 256;             // P rows per pair
constexpr int kGtN = 256;             // Q rows per pair, at most
constexpr int kGtGran = 32;           // n is a multiple of this for cta_group::2, M = 256
constexpr int kGtStages = 6;
constexpr int kGtOperandBytes = 128 * 128;              // 128 rows x 64 terms of 16 bits
constexpr int kGtStageBytes = 2 * kGtOperandBytes;      // P and Q

struct GroupedTcArgs {
  CUtensorMap map_p;
  CUtensorMap map_q[4];  // by row: boxes of 128, 64, 32 and 16 rows of Q; dW: [0] boxes of both, and
                         // single rows for gathers, [1] of P and [2] of Q
  ProdArgs g;
  int pairs;             // CTA pairs of the launch
  int blocked;           // operands stored MN-major have whole blocks of 64 columns: one box brings two
  int wide_store;              // 32-byte stores are aligned
};

struct GtSmem {
  static constexpr int kBar = kGtStages * kGtStageBytes;
  static constexpr int kNumBars = 2 * kGtStages + 4 + 1;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kBytes = kMisc + 32;
  static constexpr int kAlloc = kBytes + 1024;
};
static_assert(GtSmem::kAlloc + (kProdGroups + 1) * 4 + 64 <= 227 * 1024, "shared memory over the per-CTA limit");

// Item w of dW: a regular grid of tiles, x's columns fastest.
struct DwPlan {
  int p_tiles, q_tiles;
};
__device__ __forceinline__ ProdItem dw_item(const ProdArgs& g, const DwPlan& pl, int w) {
  ProdItem it;
  const int per = pl.p_tiles * pl.q_tiles;
  it.tile = w;
  it.split = 0;
  it.e = w / per;
  const int l = w - it.e * per;
  it.p0 = (l / pl.q_tiles) * kGtP;
  it.q0 = (l % pl.q_tiles) * kGtN;
  it.n = min(kGtN, g.K - it.q0);
  int r0, r1;
  group_rows(g, it.e, r0, r1);
  it.t0 = 0;
  it.t1 = (r1 - r0 + 63) / 64;
  return it;
}

// The last rows [row, r1) of a group, fewer than 64, of `blocks` blocks of 64
// columns: rows up to a multiple of 16 are fetched, those at or past r1 as zeros
// (row `none` lies outside the tensor).
__device__ __forceinline__ void gt_gather(const CUtensorMap* map, int col, int blocks, int row, int r1, int none,
                                          uint32_t slot, uint32_t bar) {
  const int fours = (r1 - row + 15) / 16 * 4;
  for (int i = 0; i < fours; ++i) {
    const int b = row + 4 * i;
    const int4 r = make_int4(b < r1 ? b : none, b + 1 < r1 ? b + 1 : none, b + 2 < r1 ? b + 2 : none,
                             b + 3 < r1 ? b + 3 : none);
    for (int c = 0; c < blocks; ++c) tma2_gather4(slot + 8192 * c + 512 * i, map, col + 64 * c, r, bar);
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
    gt_gather(&a.map_q[1], p, 2, row, r1, a.g.rows, slot, bar);
  } else if (a.blocked) {
    tma2_3d(slot, &a.map_p, 0, row, p / 64, bar);
  } else {
    tma2_2d(slot, &a.map_p, p, row, bar);
    tma2_2d(slot + 8192, &a.map_p, p + 64, row, bar);
  }
}
template <int MODE>
__device__ __forceinline__ void gt_load_q(const GroupedTcArgs& a, int t, int q, int half, int row, int r1,
                                          uint32_t slot, uint32_t bar) {
  if (MODE != kProdDw) {
    // rows in boxes of 128, or of 64, 32 and 16
    int at = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int box = 128 >> i;
      if (half & box) {
        tma2_2d(slot + 128 * at, &a.map_q[i], 64 * t, q + at, bar);
        at += box;
      }
    }
  } else if (r1 - row < 64) {
    gt_gather(&a.map_q[2], q, 2, row, r1, a.g.rows, slot, bar);
  } else if (a.blocked) {
    tma2_3d(slot, &a.map_q[0], 0, row, q / 64, bar);
  } else {
    tma2_2d(slot, &a.map_q[0], q, row, bar);
    tma2_2d(slot + 8192, &a.map_q[0], q + 64, row, bar);
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
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ int start[kProdGroups + 1];  // first tile of each group
  __shared__ int warp_tot[kGtThreads / 32];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem_s = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + GtSmem::kBar);
  uint64_t* full = bars;                    // the leader's count both CTAs' copies
  uint64_t* empty = full + kGtStages;
  uint64_t* acc_full = empty + kGtStages;
  uint64_t* acc_empty = acc_full + 2;       // the leader's
  uint64_t* drain_bar = acc_empty + 2;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + GtSmem::kMisc);  // [0] tmem base, [1] abort, [2] last
  volatile int* abort_flag = reinterpret_cast<volatile int*>(&misc[1]);
  const ProdArgs& g = a.g;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x >> 1;

  if (tid == 0) {
    for (int i = 0; i < kGtStages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], 2 * kGtEpiWarps); }
    mbar_init(drain_bar, 1);
    misc[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc2(&misc[0], 512);
    tmem_relinquish2();
  }

  if (warp == 0 && lane < 5) prefetch_map(lane < 4 ? &a.map_q[lane] : &a.map_p);
  // --- the plan: tiles per group (rows), or a regular grid of tiles (dW)
  RowPlan pl;
  DwPlan dw;
  const int j_dim = MODE == kProdDx ? g.K : g.N;
  pl.p_tiles = (j_dim + kGtP - 1) / kGtP;
  pl.stages = ((MODE == kProdDx ? g.N : g.K) + 63) / 64;
  dw.p_tiles = pl.p_tiles;
  dw.q_tiles = (g.K + kGtN - 1) / kGtN;
  if (MODE == kProdDw) {
    if (blockIdx.x == 0)
      for (int e = tid; e < g.E; e += kGtThreads)
        if (group_bad(g, e)) atomicOr(g.status, kStatusRouting);
  } else {
    plan_groups<kGtN, kGtThreads>(g, pl.p_tiles, start, warp_tot);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before either signals them
  tc_fence_after();
  const uint32_t tmem = misc[0];
  pl.tiles = MODE == kProdDw ? g.E * dw.p_tiles * dw.q_tiles : start[g.E];
  pl.S = MODE == kProdDw ? 1 : plan_slices(pl, a.pairs, 2, g.rows, kGtN);
  auto item = [&](int w) { return MODE == kProdDw ? dw_item(g, dw, w) : row_item<kGtN, kGtGran, kGtP>(g, pl, start, w); };
  const int items = pl.tiles * pl.S;
  const uint32_t full_s = map_to_rank(smem_u32(full), 0);

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ producers of P (warp 0) and Q (warp 2)
    uint32_t k = 0;
    for (int w = pair; w < items; w += a.pairs) {
      const ProdItem it = item(w);
      const int half = gt_half<MODE>(it.n);
      int r0 = 0, r1 = 0;
      if (MODE == kProdDw) group_rows(g, it.e, r0, r1);
      const int p = it.p0 + rank * 128, q = it.q0 + rank * half;
      for (int t = it.t0; t < it.t1; ++t, ++k) {
        const int s = k % kGtStages, row = r0 + 64 * t;
        mbar_wait(&empty[s], ((k / kGtStages) + 1) & 1, abort_flag, g.status);
        if (*abort_flag) break;
        __syncwarp();
        const uint32_t slot = smem_s + s * kGtStageBytes, bar = full_s + 8 * s;
        if (warp == 0) {
          if (rank == 0) expect_tx_elect(&full[s], gt_stage_bytes<MODE>(half, min(64, r1 - row)));
          gt_load_p<MODE>(a, it, t, p, row, r1, slot, bar);
        } else {
          gt_load_q<MODE>(a, t, q, half, row, r1, slot + kGtOperandBytes, bar);
        }
      }
      if (*abort_flag) break;
    }
    // leave no copy in flight (the leader's barriers count the peer's copies too)
    if (rank == 0 && warp == 0)
      for (uint32_t i = 0; i < (uint32_t)kGtStages && i < k; ++i) {
        const uint32_t u = k - 1 - i;
        mbar_drain(&full[u % kGtStages], (u / kGtStages) & 1, g.status);
      }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (rank == 0) {
      constexpr uint32_t kMajors = MODE == kProdFwd ? 0u : (MODE == kProdDx ? kIdescMajorA : (kIdescMajorA | kIdescMajorB));
      constexpr uint32_t kStepA = MODE == kProdFwd ? 2 : 128, kStepB = MODE == kProdDw ? 128 : 2;  // 16 terms, 16-byte units
      const uint32_t bf = g.in_type == kBf16 ? 1u : 0u;
      uint32_t k = 0, ic = 0;
      for (int w = pair; w < items; w += a.pairs) {
        const ProdItem it = item(w);
        if (it.t0 >= it.t1) continue;  // (dW: a group without rows; the epilogue writes zeros)
        int r0 = 0, r1 = 0;
        if (MODE == kProdDw) group_rows(g, it.e, r0, r1);
        const uint32_t idesc = idesc_f16_f32(256, 2 * gt_half<MODE>(it.n), bf) | kMajors;
        const int acc = ic & 1;
        mbar_wait(&acc_empty[acc], ((ic >> 1) + 1) & 1, abort_flag, g.status);
        __syncwarp();
        tc_fence_after();
        const uint32_t d = tmem + acc * kGtN;
        for (int t = it.t0; t < it.t1; ++t, ++k) {
          const int s = k % kGtStages;
          mbar_wait(&full[s], (k / kGtStages) & 1, abort_flag, g.status);
          __syncwarp();
          tc_fence_after();
          const uint32_t slot = smem_s + s * kGtStageBytes;
          const uint64_t pd = MODE == kProdFwd ? smem_desc_sw128(slot) : smem_desc_sw128_mn(slot, 8192);
          const uint64_t qd = MODE == kProdDw ? smem_desc_sw128_mn(slot + kGtOperandBytes, 8192)
                                              : smem_desc_sw128(slot + kGtOperandBytes);
          const int steps = MODE == kProdDw ? (min(64, r1 - (r0 + 64 * t)) + 15) / 16 : 4;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < steps) umma2_f16_elect(d, pd + i * kStepA, qd + i * kStepB, idesc, (t > it.t0 || i > 0) ? 1u : 0u);
          umma2_commit_elect(&empty[s]);
        }
        umma2_commit_elect(&acc_full[acc]);
        ++ic;
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
    int32_t* counters = reinterpret_cast<int32_t*>(g.scratch);
    float* partial = reinterpret_cast<float*>(g.scratch + kProdCounterBytes);
    uint32_t ic = 0;
    for (int w = pair; w < items; w += a.pairs) {
      const ProdItem it = item(w);
      const int p = it.p0 + rank * 128 + quarter * 32;  // this warp's first P row
      const bool none = it.t0 >= it.t1;
      const int acc = ic & 1;
      if (!none) {
        mbar_wait(&acc_full[acc], (ic >> 1) & 1, abort_flag, g.status);
        tc_fence_after();
      }
      const uint32_t tb = tmem + ((uint32_t)(quarter * 32) << 16) + acc * kGtN;
      bool finish = true;
      const int chunks = (it.n + 31) / 32;
      if (MODE != kProdDw && pl.S > 1) {
        // this thread's values of the slice, 16 bytes per thread and step, in its own order
        float* mine = partial + ((int64_t)((it.tile * pl.S + it.split) * 2 + rank) * 128) * kGtN;
        for (int c = sub; c < chunks; c += 2) {
          uint32_t v[32];
          tmem_ld32(tb + 32 * c, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            __stcg(reinterpret_cast<uint4*>(mine) + (c * 8 + i) * 128 + quarter * 32 + lane,
                   make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
        }
        named_bar_sync(1, kGtEpiThreads);
        if (et == 0) {
          misc[2] = slice_arrive_last(&counters[it.tile * 2 + rank], pl.S) ? 1u : 0u;
        }
        named_bar_sync(1, kGtEpiThreads);
        finish = misc[2] != 0;
      }
      if (finish) {
        for (int c = sub; c < chunks; c += 2) {
          uint32_t v[32];
          if (MODE != kProdDw && pl.S > 1) {
            float f[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = 0.0f;
            const float4* src = reinterpret_cast<const float4*>(partial + ((int64_t)it.tile * pl.S * 2 + rank) * 128 * kGtN) +
                                c * 8 * 128 + quarter * 32 + lane;
#pragma unroll 4
            for (int s = 0; s < pl.S; ++s, src += 2 * 128 * kGtN / 4) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 u = __ldcg(src + i * 128);
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
          if (MODE == kProdDw) {
            // lane = row i of dW[e], registers = 32 consecutive columns
            const int i = p + lane, j = it.q0 + 32 * c;
            if (i < g.N) {
              const int64_t at = it.e * g.out_se + (int64_t)i * g.out_ld + j;
              const int cols = min(32, g.K - j);  // a multiple of 8
              if (g.out_type == kFp32) {
                float* dst = static_cast<float*>(g.out) + at;
                if (g.accumulate) {
                  for (int b = 0; b < cols; b += 4) {
#pragma unroll
                    for (int u = 0; u < 32; u += 4)
                      if (u == b) {
                        const float4 o = *reinterpret_cast<const float4*>(dst + u);
                        v[u] = __float_as_uint(__uint_as_float(v[u]) + o.x);
                        v[u + 1] = __float_as_uint(__uint_as_float(v[u + 1]) + o.y);
                        v[u + 2] = __float_as_uint(__uint_as_float(v[u + 2]) + o.z);
                        v[u + 3] = __float_as_uint(__uint_as_float(v[u + 3]) + o.w);
                      }
                  }
                }
#pragma unroll
                for (int b = 0; b < 32; b += 8) {
                  if (b < cols) {
                    const uint32_t o[8] = {v[b], v[b + 1], v[b + 2], v[b + 3], v[b + 4], v[b + 5], v[b + 6], v[b + 7]};
                    if (a.wide_store) {
                      stg256(dst + b, o);
                    } else {
                      stg128(dst + b, make_uint4(o[0], o[1], o[2], o[3]));
                      stg128(dst + b + 4, make_uint4(o[4], o[5], o[6], o[7]));
                    }
                  }
                }
              } else {
                uint16_t* dst = static_cast<uint16_t*>(g.out) + at;
                uint32_t h[16];
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                  const float lo = __uint_as_float(v[2 * u]), hi = __uint_as_float(v[2 * u + 1]);
                  h[u] = g.out_type == kBf16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
                }
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  const uint32_t o[8] = {h[8 * b], h[8 * b + 1], h[8 * b + 2], h[8 * b + 3],
                                         h[8 * b + 4], h[8 * b + 5], h[8 * b + 6], h[8 * b + 7]};
                  if (a.wide_store && 16 * b + 16 <= cols) {
                    stg256(dst + 16 * b, o);
                  } else {
                    if (16 * b < cols) stg128(dst + 16 * b, make_uint4(o[0], o[1], o[2], o[3]));
                    if (16 * b + 8 < cols) stg128(dst + 16 * b + 8, make_uint4(o[4], o[5], o[6], o[7]));
                  }
                }
              }
            }
          } else {
            // lane = feature, registers = 32 rows: eight rows at a time, transposed
            // inside groups of eight lanes, so that a lane stores 16 bytes of one row
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              uint32_t wd[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const float lo = __uint_as_float(v[8 * b + 2 * u]), hi = __uint_as_float(v[8 * b + 2 * u + 1]);
                wd[u] = g.out_type == kBf16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
              }
              const uint4 o = transpose8x8_u16(wd, lane);
              const int row = 32 * c + 8 * b + (lane & 7), j = p + (lane & 24);
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
    rc = cudaFuncSetAttribute(grouped_tc_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, GtSmem::kAlloc);
    if (rc != cudaSuccess) return rc;
    ready[dev].store(true, std::memory_order_release);
  }
  grouped_tc_kernel<MODE><<<2 * a.pairs, kGtThreads, GtSmem::kAlloc, st>>>(a);
  return cudaPeekAtLastError();
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
    const uint32_t box[2] = {64, 64}, one[2] = {64, 1};
    ok = make_prod_map(&a.map_q[1], ty, g.a, 2, dp, &ald, one) && make_prod_map(&a.map_q[2], ty, g.w, 2, dq, &wld, one);
    if (a.blocked) {
      const uint64_t bp[3] = {64, rows, N / 64}, bq[3] = {64, rows, K / 64}, sp[2] = {ald, 128}, sq[2] = {wld, 128};
      const uint32_t two[3] = {64, 64, 2};
      ok = ok && make_prod_map(&a.map_p, ty, g.a, 3, bp, sp, two) && make_prod_map(&a.map_q[0], ty, g.w, 3, bq, sq, two);
    } else {
      ok = ok && make_prod_map(&a.map_p, ty, g.a, 2, dp, &ald, box) && make_prod_map(&a.map_q[0], ty, g.w, 2, dq, &wld, box);
    }
    a.map_q[3] = a.map_q[2];
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
  if (!ok) return cudaSuccess;  // (the plain kernel takes what a tensor map cannot describe)
  const int sms = prod_sm_count();
  if (sms < 2) return cudaErrorInvalidDevice;
  a.pairs = sms / 2;
  const int per32 = g.out_type == kFp32 ? 8 : 16;  // elements of 32 bytes
  a.wide_store = (reinterpret_cast<uintptr_t>(g.out) & 31) == 0 && g.out_ld % per32 == 0 && g.out_se % per32 == 0;
  *done = true;
  if (mode == kProdFwd) return launch_mode<kProdFwd>(a, st);
  if (mode == kProdDx) return launch_mode<kProdDx>(a, st);
  return launch_mode<kProdDw>(a, st);
}

}  // namespace moe
