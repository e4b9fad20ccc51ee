// Tensor-core helpers of the products: clusters of two CTAs that share one
// tcgen05 MMA (cta_group::2), TMA loads that complete on the leader's barrier,
// and shared-memory descriptors of both operand orders.
#pragma once

#include <cuda.h>

#include "products.cuh"

namespace moe {

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ---------------------------------------------------------------- cluster of two
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared-memory object in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// ---------------------------------------------------------------- TMA into this CTA, counted by the barrier at
// `bar` (a shared::cluster address: the leader's).  Called by a whole converged
// warp, issued by its elected lane: loops and operands then stay warp-uniform,
// without which each issue costs its thread some hundred cycles.
__device__ __forceinline__ void expect_tx_elect(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void tma2_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma2_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma2_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                        uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
// Four rows r.x .. r.w, 128 bytes each from column c0; rows outside the tensor arrive as zeros.
__device__ __forceinline__ void tma2_gather4(uint32_t dst, const CUtensorMap* map, int c0, int4 r, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar)
      : "memory");
}

// The same within one CTA.
__device__ __forceinline__ void tma1_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma1_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// ---------------------------------------------------------------- tcgen05 over the CTA pair
__device__ __forceinline__ void tmem_alloc2(uint32_t* smem_dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_dst)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// One MMA of 32 bytes along the sum (16 terms of 16 bits), issued by the converged warp's elected lane.
__device__ __forceinline__ void umma2_f16_elect(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Four such MMAs, 64 terms; the descriptors advance by DA and DB (16-byte units)
// a step.  One election for the four: the issuing warp's time per stage bounds
// narrow tiles.
template <int DA, int DB>
__device__ __forceinline__ void umma2_f16_stage_elect(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "add.u64 a1, %1, %3;\n\tadd.u64 a2, a1, %3;\n\tadd.u64 a3, a2, %3;\n\t"
      "add.u64 b1, %2, %4;\n\tadd.u64 b2, b1, %4;\n\tadd.u64 b3, b2, %4;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %5, p;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %5, 1;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %5, 1;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %5, 1;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "n"(DA), "n"(DB), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrive on the barrier at this offset in both CTAs once the MMAs issued so far are done.
__device__ __forceinline__ void umma2_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "mov.b16 m, 3;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}
// One CTA, 128 E4M3 terms (four MMAs of 32) of operands stored with the terms
// innermost: D = A B, nothing accumulated from before.
__device__ __forceinline__ void umma1_f8_block_elect(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
      "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc)
      : "memory");
}
// 32 TMEM lanes x 32 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// 32 TMEM lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Two fp32 sums in a 64-bit register pair.
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, uint32_t& lo, uint32_t& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
}
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}

// Operand whose rows run along the sum's other dimension (contiguous along rows
// of the tile, "MN-major"), 128-byte swizzle: blocks of 64 16-bit columns, each
// block one 128-byte line per term of the sum, eight lines an atom of 1024
// bytes (stride-dimension offset), the next 64 columns `block_bytes` further
// (leading-dimension offset).
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t saddr, uint32_t block_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(block_bytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kIdescMajorA = 1u << 15, kIdescMajorB = 1u << 16;  // operand stored MN-major

// ---------------------------------------------------------------- stores
// A box from shared memory, by one thread after fence_async_proxy and a warp
// barrier; ADD: added to what is there (fp32).
template <bool ADD>
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int c0, int c1, int c2, uint32_t src) {
  if (ADD)
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(src)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(src)
                 : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the newest `N` boxes of this thread have been read from shared memory.
template <int N>
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tma_store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"((uint16_t)v) : "memory");
}
__device__ __forceinline__ void stg256(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t v;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
  return v;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t v;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
  return v;
}

// Position in a ring of N slots and the parity of the pass through it.
template <int N>
struct Ring {
  uint32_t i = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      phase ^= 1;
    }
  }
};

// mbar_wait by a whole warp, with one answer for all its lanes: false once the CTA
// has given up, and the role then leaves its loop.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status));
}

// ---------------------------------------------------------------- work items
// The tiles of a product by rows: a group of m rows has ceil(m / ROWS) row tiles,
// each times the tiles of output features; with few tiles the sum is cut into S
// slices.
constexpr int kProdGroups = 1024;       // groups, at most
constexpr int kProdTokenChunk = 8;      // row tiles that run next to each other through a group's features
constexpr int kProdPartials = 320;      // partial tiles of 128 x 256 sums that the scratch holds
constexpr int kProdCounterBytes = 4096; // scratch: arrival counters, then partial tiles
// Items of a launch, at most.  Offsets that do not overlap give 1e9 of them (the host's limit); others can count up
// to 2^31, and a role's position, which passes the last item by up to a launch's width, must not wrap to numbers
// below 0 that would be taken for items again.
constexpr int kProdWidth = 65536;       // CTAs of a launch, at most
constexpr int kProdItems = 0x7FFFFFFF - kProdWidth;
static_assert(kProdItems > 1000000000, "offsets that keep the rule would lose tiles");

struct RowPlan {
  int tiles, S, stages, p_tiles;
};
struct ProdItem {
  int e, p0, q0, n;  // expert, first feature (dW: column of dy), first row (dW: column of x), rows
  int t0, t1;        // stages of the slice
  int split, tile;
};

// First tile of each group into start[0 .. E]; all THREADS threads of the CTA.
template <int ROWS, int THREADS>
__device__ __forceinline__ void plan_groups(const ProdArgs& g, int p_tiles, int* start, int* warp_tot) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kPer = (kProdGroups + THREADS - 1) / THREADS;
  int cnt[kPer], run = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    cnt[i] = 0;
    if (e < g.E) {
      int r0, r1;
      group_rows(g, e, r0, r1);
      cnt[i] = (r1 - r0 + ROWS - 1) / ROWS * p_tiles;
      if (blockIdx.x == 0 && group_bad(g, e)) atomicOr(g.status, kStatusRouting);
    }
    run += cnt[i];
  }
  int incl = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) warp_tot[warp] = incl;
  __syncthreads();
  int pos = incl - run;
  for (int w = 0; w < warp; ++w) pos += warp_tot[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e < g.E) start[e] = pos;
    pos += cnt[i];
    if (e == g.E - 1) start[g.E] = pos;
  }
}

// Slices of the sum, when there are fewer tiles than workers (CTAs or pairs, each
// with `partials` partial tiles to an item): the S that minimises, in stages,
//   rounds * (stages / S + 6) + (S > 1 ? 4 + S * (0.5 + 3.5 cols / 256) : 0),
// six stages for what an item costs besides its stages, and the second term for
// storing, signalling and adding partial tiles of `cols` columns (fitted to S = 1 ..
// 12 at sums of 8 to 64 stages: 1 x 256 x 7168 in FP8 takes 20.5, 14.8, 11.6 and 10.7 us
// at S = 1, 2, 4 and 8; 300 x 512 x 4096 takes 23.0, 20.8 and 23.7 at 1, 4 and 8).
// Up to ten stages a second slice cannot save what it costs.  The columns
// are those of an average tile, at most `most`.  A lane per S;
// called by whole warps.
__device__ __forceinline__ int plan_slices(const RowPlan& pl, int workers, int partials, int rows, int most) {
  if (pl.tiles >= workers || pl.tiles == 0 || pl.stages <= 10) return 1;
  const int cols = min(most, (int)__fdividef((float)rows * pl.p_tiles, (float)pl.tiles));
  const int s = (threadIdx.x & 31) + 1;
  uint32_t cost = 0xFFFFFFu;
  if (s <= pl.stages && s * pl.tiles <= kProdPartials / partials) {
    const int rounds = (pl.tiles * s + workers - 1) / workers;
    cost = 4 * rounds * ((pl.stages + s - 1) / s + 6) + (s > 1 ? 16 + s * (2 + 14 * cols / 256) : 0);
  }
  return (int)(__reduce_min_sync(0xffffffffu, min(cost, 0xFFFFFFu) * 64 + s) & 63);
}

// Item w: its slice, then row tiles in chunks of kProdTokenChunk -- inside a chunk
// row tiles fastest, then features, so that the tiles which run at one time share
// rows and weights in L2.  A group's rows are cut into equal tiles, rounded to GRAN.
// A role walks its items in ascending order, so the search for the group goes on
// from the last one's (`e`, 0 at first), and the divisions are skipped where the
// quotient is known: every item costs each role this code before its first copy.
template <int ROWS, int GRAN, int FEATURES>
__device__ __forceinline__ ProdItem row_item(const ProdArgs& g, const RowPlan& pl, const int* start, int w, int& e) {
  ProdItem it;
  it.tile = w;
  it.split = 0;
  it.t0 = 0;
  it.t1 = pl.stages;
  if (pl.S > 1) {
    it.tile = w / pl.S;
    it.split = w - it.tile * pl.S;
    it.t0 = it.split * pl.stages / pl.S;
    it.t1 = (it.split + 1) * pl.stages / pl.S;
  }
  while (start[e + 1] <= it.tile) ++e;  // (ends: tile < start[E], and the last such group is not empty)
  it.e = e;
  int l = it.tile - start[e];
  int r0, r1;
  group_rows(g, e, r0, r1);
  const int m = r1 - r0, nt = (m + ROWS - 1) / ROWS;
  if (nt == 1) {
    it.p0 = l * FEATURES;
    it.q0 = r0;
    it.n = m;
    return it;
  }
  int c = 0;
  if (nt > kProdTokenChunk) {
    c = l / (kProdTokenChunk * pl.p_tiles);
    l -= c * kProdTokenChunk * pl.p_tiles;
  }
  const int width = min(kProdTokenChunk, nt - c * kProdTokenChunk), f = l / width;
  it.p0 = f * FEATURES;
  const int q = ((m + nt - 1) / nt + GRAN - 1) / GRAN * GRAN;
  it.q0 = r0 + (c * kProdTokenChunk + l - f * width) * q;
  it.n = min(q, r1 - it.q0);
  return it;
}

// Arrival of one slice of a tile whose partial sums the CTA's threads have stored,
// called by one of them after a barrier of all: true for the last of `S` arrivals,
// whose CTA may then (after another barrier) read every slice's.  The counter
// starts at 0 and is back at 0 after the last.
__device__ __forceinline__ bool slice_arrive_last(int32_t* counter, int S) {
  uint32_t old;
  asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(old) : "l"(counter), "r"(S - 1) : "memory");
  return old == (uint32_t)(S - 1);
}

// ---------------------------------------------------------------- host
// A tensor map of 2 to 4 dimensions (innermost first), 128-byte swizzle; strides in bytes of the outer ones.
bool make_prod_map(CUtensorMap* m, int elem_type, const void* base, int nd, const uint64_t* dims,
                   const uint64_t* strides, const uint32_t* box);

// The tensor-core kernels; *done stays false for operands that they cannot address (16-byte rules).
cudaError_t launch_fp8_tc(const ProdArgs& g, cudaStream_t st, bool* done);
cudaError_t launch_grouped_tc(const ProdArgs& g, int mode, cudaStream_t st, bool* done);

}  // namespace moe
