// The adapters of many rows: each adapter's positions in tiles of 128, in two launches.
//
//   mid[i, j] = sum_p in[r, p] F[l](j, p)                       adapter_mid_kernel
//   out[r, q] = base[r, q] + scale[l] sum_j mid[i, j] S[l](q, j)  adapter_out_kernel
//
// (forward: F = A, S = B; gradient by the rows: F = B^T, S = A^T, read where they lie.)
// Both are streams: 2 P bytes a row in, then 2 Q in and out, against 2 R (P + 2 Q)
// operations, R of 8 to 256.
//
// This one: 16384 rows of 7168 (one adapter, rank 16) take 43 us, 5.5 TB/s (floor 35);
// 8191 rows of 4096 of 23 requests, rank 64, 23 us (floor 10): the plan of the tiles,
// the pipeline's filling and the last tiles' sums cost about 8 us whatever the rows.
// With the sum cut into slices of equal number instead of equal CTAs: 21 and, for 8188
// rows of 32 experts of 2880, 19.4 instead of 16.
#include "adapters.cuh"

namespace moe {

// A persistent CTA per SM on tcgen05: 128 rows on the MMA's M side, the ranks on its N
// side, a stage of 64 terms of the sum in 128-byte swizzled lines.  Eight loader warps
// gather the rows (and F) with 16-byte asynchronous copies, which take any order of
// the rows and leave zeros past the ends; an MMA warp; four epilogue warps.  F enters
// as it lies: terms innermost (A) or ranks innermost (B^T) through MN-major
// descriptors.  The tiles' stages are cut evenly over the CTAs; what several CTAs have
// of a tile the second launch adds in their order.
constexpr int kMdThreads = 416, kMdLoaders = 256;  // warps 0-7; 8-11 epilogue, 12 MMA

template <int RB>  // blocks of 64 ranks
struct MidCfg {
  static constexpr int kStages = RB == 1 ? 8 : RB == 2 ? 6 : 4;
  static constexpr int kLag = RB == 1 ? 6 : RB == 2 ? 4 : 3;  // stages of copies in flight
  static constexpr int kFBytes = RB * 8192;
  static constexpr int kStageBytes = 16384 + kFBytes;
  static constexpr int kAlloc = kStages * kStageBytes + 1024;
  static_assert(kLag < kStages, "a loader would wait for a stage that it has not signalled");
  static_assert(kAlloc + (kAdAdapters + 1) * 4 + 512 <= 227 * 1024, "shared memory over the per-CTA limit");
};

// A role's position among the CTA's pieces of tiles.
struct MidItem {
  int l, pos, n;  // adapter, first position, rows
  int t0, t1;     // stages
  float* out;     // of the first row
};
struct MidWalk {
  const AdapterArgs& a;
  const int* start;
  MidSplit split;
  int64_t unit, end;
  int l = 0;
  __device__ __forceinline__ MidWalk(const AdapterArgs& a_, const int* start_, int tiles)
      : a(a_), start(start_), split(a_, tiles) {
    if (a.mid_ctas > 0) {
      unit = (int)blockIdx.x < split.ctas ? split.begin(blockIdx.x) : 0;
      end = (int)blockIdx.x < split.ctas ? split.begin(blockIdx.x + 1) : 0;
    } else {  // whole tiles, spread evenly
      unit = (int64_t)tiles * blockIdx.x / gridDim.x * split.stages;
      end = (int64_t)tiles * (blockIdx.x + 1) / gridDim.x * split.stages;
    }
  }
  __device__ __forceinline__ bool next(MidItem& it) {
    if (unit >= end) return false;
    const int tile = (int)(unit / split.stages);
    while (start[l + 1] <= tile) ++l;
    it.l = l;
    int i0, i1;
    adapter_rows(a.offsets, a.rows, l, i0, i1);
    it.pos = i0 + (tile - start[l]) * kAtRows;
    it.n = min(kAtRows, i1 - it.pos);
    it.t0 = (int)(unit - (int64_t)tile * split.stages);
    it.t1 = (int)min((int64_t)split.stages, it.t0 + end - unit);
    unit += it.t1 - it.t0;
    it.out = it.t1 - it.t0 == split.stages ? a.mid + (int64_t)it.pos * a.R
                                           : a.part + (int64_t)(blockIdx.x + tile) * kAtRows * a.R;
    return true;
  }
};

template <int RB, bool FWD>
__global__ void __launch_bounds__(kMdThreads, 1) adapter_mid_kernel(const __grid_constant__ AdapterArgs a) {
  using C = MidCfg<RB>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ int start[kAdAdapters + 1];
  __shared__ int warp_tot[kMdThreads / 32];
  __shared__ uint64_t full[C::kStages], empty[C::kStages], acc_full[2], acc_empty[2], drain_bar;
  __shared__ uint32_t misc[2];  // tensor memory, abort
  volatile int* abort_flag = reinterpret_cast<volatile int*>(&misc[1]);
  const uint32_t smem_s = (smem_u32(smem_raw) + 1023) & ~1023u;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t ranks = (a.R + 15) / 16 * 16, columns = tmem_columns(2 * ranks);
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) { mbar_init(&full[i], kMdLoaders); mbar_init(&empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], 4); }
    mbar_init(&drain_bar, 1);
    misc[1] = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(&misc[0], columns);
    tmem_relinquish();
  }
  grid_dependency_wait();
  grid_dependents_launch();  // (after the wait: the second launch reads operands before its own)
  plan_adapters<kAtRows, kMdThreads>(a.offsets, a.rows, a.L, start, warp_tot, a.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const int tiles = start[a.L];

  if (warp < 8) {
    // ------------------------------------------------------------ loaders
    const int c = tid & 7, line0 = tid >> 3;               // 16-byte column, first line (others 32 apart)
    const uint32_t sw = (uint32_t)((c ^ (line0 & 7)) << 4);  // (lines 32 apart share it)
    const uint16_t* in = static_cast<const uint16_t*>(a.in);
    int filled = 0, signalled = 0;
    Ring<C::kStages> slot, done;
    bool ok = true;
    MidItem it;
    for (MidWalk at(a, start, tiles); ok && at.next(it);) {
      const uint16_t* row[4];
      int there[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = line0 + 32 * i;
        const int r = n < it.n ? row_of(a.order, a.rows, it.pos + n, a.status) : -1;
        row[i] = in + (int64_t)max(r, 0) * a.in_ld + 8 * c;
        there[i] = r >= 0 ? 16 : 0;
      }
      const uint16_t* const f = static_cast<const uint16_t*>(a.f) + it.l * a.f_l;
      for (int t = it.t0; t < it.t1; ++t) {
        if (!mbar_wait(&empty[slot.i], slot.phase ^ 1, abort_flag, a.status)) {
          ok = false;
          break;
        }
        const uint32_t dst = smem_s + slot.i * C::kStageBytes + line0 * 128 + sw;
        const bool whole = 64 * t + 8 * c < a.P;
        const int q = whole ? 64 * t : -8 * c;  // (past the sum's end: the row's start, of which nothing is copied)
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async16(dst + i * 4096, row[i] + q, whole ? there[i] : 0);
        if (FWD) {
#pragma unroll
          for (int i = 0; i < 2 * RB; ++i) {
            const int j = line0 + 32 * i;
            if (j < a.R) cp_async16(dst + 16384 + i * 4096, f + j * a.f_r + 8 * c + q, whole ? 16 : 0);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int term = 64 * t + line0 + 32 * i;
            const uint16_t* line = f + (int64_t)(term < a.P ? term : 0) * a.f_r;
#pragma unroll
            for (int b = 0; b < RB; ++b)
              if (64 * b + 8 * c < a.R)
                cp_async16(dst + 16384 + b * 8192 + i * 4096, line + 64 * b + 8 * c, term < a.P ? 16 : 0);
          }
        }
        cp_async_commit();
        slot.next();
        if (++filled > C::kLag) {
          cp_async_wait<C::kLag>();
          fence_async_proxy();
          mbar_arrive(&full[done.i]);
          done.next();
          ++signalled;
        }
      }
    }
    cp_async_wait<0>();
    fence_async_proxy();
    for (; signalled < filled; ++signalled) {
      mbar_arrive(&full[done.i]);
      done.next();
    }
  } else if (warp == 12) {
    // ------------------------------------------------------------ MMA
    const uint32_t idesc = idesc_f16_f32(kAtRows, ranks, a.type == kBf16 ? 1u : 0u) | (FWD ? 0u : kIdescMajorB);
    const uint64_t xd0 = smem_desc_sw128(smem_s);
    const uint64_t fd0 = FWD ? smem_desc_sw128(smem_s + 16384) : smem_desc_sw128_mn(smem_s + 16384, 8192);
    Ring<C::kStages> slot;
    Ring<2> acc;
    bool ok = true;
    MidItem it;
    for (MidWalk at(a, start, tiles); ok && at.next(it);) {
      if (!warp_wait(&acc_empty[acc.i], acc.phase ^ 1, abort_flag, a.status)) break;
      tc_fence_after();
      for (int t = it.t0; t < it.t1; ++t) {
        if (!(ok = warp_wait(&full[slot.i], slot.phase, abort_flag, a.status))) break;
        tc_fence_after();
        const uint32_t by = slot.i * (C::kStageBytes >> 4);
        umma1_f16_stage_elect<2, FWD ? 2 : 128>(tmem + acc.i * ranks, xd0 + by, fd0 + by, idesc, t > it.t0 ? 1u : 0u);
        umma_commit_elect(&empty[slot.i]);
        slot.next();
      }
      umma_commit_elect(&acc_full[acc.i]);
      acc.next();
    }
    umma_commit_elect(&drain_bar);
    mbar_drain(&drain_bar, 0, a.status);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue: a row to a thread
    Ring<2> acc;
    MidItem it;
    for (MidWalk walk(a, start, tiles); walk.next(it);) {
      if (!warp_wait(&acc_full[acc.i], acc.phase, abort_flag, a.status)) break;
      tc_fence_after();
      const int at = (warp & 3) * 32 + lane;
      float* out = it.out + (int64_t)at * a.R;
      const uint32_t src = tmem + ((uint32_t)((warp & 3) * 32) << 16) + acc.i * ranks;
      for (int j = 0; j < a.R; j += 16) {
        uint32_t v[16];
        tmem_ld16(src + j, v);
        tmem_ld_wait();
        if (at < it.n) {
#pragma unroll
          for (int u = 0; u < 16; u += 4)
            if (j + u < a.R) *reinterpret_cast<uint4*>(out + j + u) = make_uint4(v[u], v[u + 1], v[u + 2], v[u + 3]);
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[acc.i]);
      acc.next();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, columns);
}

// ---------------------------------------------------------------- host
template <int RB, bool FWD>
static cudaError_t launch_mid(const AdapterArgs& a, int sms, cudaStream_t st) {
  static std::atomic<bool> ready[64] = {};
  const cudaError_t rc = allow_smem(adapter_mid_kernel<RB, FWD>, MidCfg<RB>::kAlloc, ready);
  if (rc != cudaSuccess) return rc;
  return launch_dependent(adapter_mid_kernel<RB, FWD>, dim3(sms), dim3(kMdThreads), MidCfg<RB>::kAlloc, st, a);
}

template <bool FWD>
static cudaError_t launch_mid(const AdapterArgs& a, int sms, cudaStream_t st) {
  return a.R <= 64 ? launch_mid<1, FWD>(a, sms, st) : a.R <= 128 ? launch_mid<2, FWD>(a, sms, st) : launch_mid<4, FWD>(a, sms, st);
}

cudaError_t launch_adapter_tc(AdapterArgs& a, bool fwd, bool mid_wanted, int64_t part_values, cudaStream_t st) {
  const int sms = prod_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  a.want_mid = mid_wanted;
  // parts of tiles, where they are added up and the workspace holds them
  const int64_t tiles = (int64_t)a.rows / kAtRows + a.L;
  a.mid_ctas = a.out && (sms + tiles) * kAtRows * a.R <= part_values ? sms : 0;
  const cudaError_t rc = fwd ? launch_mid<true>(a, sms, st) : launch_mid<false>(a, sms, st);
  if (rc != cudaSuccess || !a.out) return rc;
  return fwd ? launch_adapter_out_fwd(a, sms, st) : launch_adapter_out_dx(a, sms, st);
}

}  // namespace moe
