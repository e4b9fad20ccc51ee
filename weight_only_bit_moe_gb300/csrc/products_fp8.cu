// Block-scaled FP8 product on tcgen05 tensor cores (sm_103a):
//
//   y[r, n] = sum_b xs[r, b] ws[n / 128, b] D_b[r, n],   D_b[r, n] = sum_{k in b} x[r, k] w[n, k]
//
// over blocks b of 128 terms, dense or grouped by expert.  A pair of CTAs
// (cta_group::2) computes each D_b of its tile into tensor memory -- a stage of
// the pipeline is one block, 128 bytes of every row -- and eight epilogue warps
// per CTA add it, times its scale, to fp32 sums in registers while the MMAs fill
// the next buffer.  Scales are arbitrary fp32, so D_b cannot stay in the tensor
// core's accumulator over blocks; reading it back once per block is what bounds
// the product where it is not memory.
//
// Two orientations:
//   rows on M (prompts): 256 rows x 256 features, a thread owns one row and the
//     128 features of one weight block: one scale per thread and block, taken as
//     a scalar into packed fp32 multiply-adds.
//   rows on N (decode): 256 features x up to 64 rows, a thread owns one feature
//     and 32 rows, whose scales it reads from shared memory.  The tile moves the
//     weights once and costs the MMA round_up(rows, 32) / 256 of a full one.
// With rows on N a 256-row tile would read 32 scales from shared memory for 128
// sums, more than the shared memory delivers in the time of the block's MMAs;
// with rows on M a tile of few rows would run the MMA nearly empty.
#include <atomic>

#include "gemm.cuh"
#include "products_tc.cuh"

namespace moe {

constexpr int kF8Threads = 320;  // eight epilogue warps, producer, MMA
constexpr int kF8EpiWarps = 8, kF8EpiThreads = 256, kF8Producer = 8, kF8Mma = 9;
constexpr int kF8FactorStages = 64;  // blocks whose scales are staged at a time (rows on N)

template <bool ROWS_M>
struct Fp8Cfg {
  static constexpr int kRows = ROWS_M ? 256 : 64;  // rows of a tile
  static constexpr int kGran = ROWS_M ? 16 : 32;
  static constexpr int kAcc = ROWS_M ? 128 : 32;   // sums per thread
  static constexpr int kBufCols = ROWS_M ? 256 : 64, kBufs = ROWS_M ? 2 : 4;
  static constexpr int kPBytes = 128 * 128;
  static constexpr int kQBytes = ROWS_M ? 128 * 128 : 32 * 128;
  static constexpr int kSlot = kPBytes + kQBytes;
  static constexpr int kStages = ROWS_M ? 6 : 9;
  static constexpr int kBar = kStages * kSlot;
  static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 1;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kFactors = (kMisc + 32 + 15) / 16 * 16;
  static constexpr int kBytes = kFactors + (ROWS_M ? 0 : kF8FactorStages * 64 * 4);
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc + (kProdGroups + 1) * 4 + 64 <= 227 * 1024, "shared memory over the per-CTA limit");
};

struct Fp8TcArgs {
  CUtensorMap map_x, map_xs;  // 128- and 16-row boxes of x
  CUtensorMap map_w;          // 128-row boxes of a bank's expert
  ProdArgs g;
  int pairs;
  int wide_store;
};

// Rows of CTA `rank` of a tile with rows on M: valid ones, and those copied (whole boxes of 16).
__device__ __forceinline__ int f8_rows(int n, int rank) { return min(max(n - rank * 128, 0), 128); }

template <bool ROWS_M>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kF8Threads, 1)
    fp8_tc_kernel(const __grid_constant__ Fp8TcArgs a) {
  using C = Fp8Cfg<ROWS_M>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ int start[kProdGroups + 1];
  __shared__ int warp_tot[kF8Threads / 32];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem_s = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBar);  // the leader's count both CTAs' copies
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + C::kBufs;  // the leader's
  uint64_t* drain_bar = acc_empty + C::kBufs;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kMisc);  // [0] tmem base, [1] abort, [2] last
  volatile int* abort_flag = reinterpret_cast<volatile int*>(&misc[1]);
  const ProdArgs& g = a.g;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x >> 1;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < C::kBufs; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], 2 * kF8EpiWarps); }
    mbar_init(drain_bar, 1);
    misc[1] = 0;
    fence_mbar_init();
  }
  if (warp == kF8Mma) {
    tmem_alloc2(&misc[0], 512);
    tmem_relinquish2();
  }
  RowPlan pl;
  pl.p_tiles = (g.N + kProdFeatures - 1) / kProdFeatures;
  pl.stages = (g.K + 127) / 128;
  plan_groups<C::kRows, kF8Threads>(g, pl.p_tiles, start, warp_tot);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before either signals them
  tc_fence_after();
  const uint32_t tmem = misc[0];
  pl.tiles = start[g.E];
  pl.S = plan_slices(pl.tiles, pl.stages, a.pairs);
  const int items = pl.tiles * pl.S;

  if (warp == kF8Producer) {
    // ------------------------------------------------------------ producer
    const uint32_t full_s = map_to_rank(smem_u32(full), 0);
    uint32_t k = 0;
    for (int w = pair; w < items; w += a.pairs) {
      const ProdItem it = row_item<C::kRows, C::kGran>(g, pl, start, w);
      // boxes of 16 rows of x per CTA, and their rows' first
      const int half = (it.n + 31) / 32 * 16;  // rows on N: rows per CTA
      const int boxes = ROWS_M ? (f8_rows(it.n, rank) + 15) / 16 : half / 16;
      const int both = ROWS_M ? (f8_rows(it.n, 0) + 15) / 16 + (f8_rows(it.n, 1) + 15) / 16 : 2 * boxes;
      const int x0 = it.q0 + rank * (ROWS_M ? 128 : half);
      const int w0 = it.p0 + rank * 128;
      for (int t = it.t0; t < it.t1; ++t, ++k) {
        const int s = k % C::kStages;
        mbar_wait(&empty[s], ((k / C::kStages) + 1) & 1, abort_flag, g.status);
        if (*abort_flag) break;
        __syncwarp();
        const uint32_t bar = full_s + 8 * s;
        if (rank == 0) expect_tx_elect(&full[s], 2 * 128 * 128 + both * 2048);
        const uint32_t ps = smem_s + s * C::kSlot, qs = ps + C::kPBytes;
        tma2_3d(ROWS_M ? qs : ps, &a.map_w, 128 * t, w0, it.e, bar);
        const uint32_t xd = ROWS_M ? ps : qs;
        if (ROWS_M && boxes == 8) {
          tma2_2d(xd, &a.map_x, 128 * t, x0, bar);
        } else {
          for (int b = 0; b < boxes; ++b) tma2_2d(xd + 2048 * b, &a.map_xs, 128 * t, x0 + 16 * b, bar);
        }
      }
      if (*abort_flag) break;
    }
    // leave no copy in flight (the leader's barriers count the peer's copies too)
    if (rank == 0)
      for (uint32_t i = 0; i < (uint32_t)C::kStages && i < k; ++i) {
        const uint32_t u = k - 1 - i;
        mbar_drain(&full[u % C::kStages], (u / C::kStages) & 1, g.status);
      }
  } else if (warp == kF8Mma) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (rank == 0) {
      uint32_t k = 0;
      for (int w = pair; w < items; w += a.pairs) {
        const ProdItem it = row_item<C::kRows, C::kGran>(g, pl, start, w);
        // E4M3 operands and fp32 sums have the fields of fp16 operands and fp32 sums
        const uint32_t idesc = idesc_f16_f32(256, ROWS_M ? 256 : (it.n + 31) / 32 * 32, 0u);
        for (int t = it.t0; t < it.t1; ++t, ++k) {
          const int s = k % C::kStages, b = k % C::kBufs;
          mbar_wait(&acc_empty[b], ((k / C::kBufs) + 1) & 1, abort_flag, g.status);
          mbar_wait(&full[s], (k / C::kStages) & 1, abort_flag, g.status);
          __syncwarp();
          tc_fence_after();
          const uint64_t pd = smem_desc_sw128(smem_s + s * C::kSlot);
          const uint64_t qd = smem_desc_sw128(smem_s + s * C::kSlot + C::kPBytes);
#pragma unroll
          for (int i = 0; i < 4; ++i) umma2_f8_elect(tmem + b * C::kBufCols, pd + 2 * i, qd + 2 * i, idesc, i > 0);
          umma2_commit_elect(&empty[s]);
          umma2_commit_elect(&acc_full[b]);
        }
      }
      umma2_commit_elect(drain_bar);
      mbar_drain(drain_bar, 0, g.status);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, sub = warp >> 2;  // TMEM lanes; half of the tile's columns
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t acc_empty_s = map_to_rank(smem_u32(acc_empty), 0);
    float* factors = reinterpret_cast<float*>(smem + C::kFactors);
    int32_t* counters = reinterpret_cast<int32_t*>(g.scratch);
    float4* partial = reinterpret_cast<float4*>(g.scratch + kProdCounterBytes);
    const int n_blocks = (g.N + 127) / 128;
    uint32_t k = 0;
    for (int w = pair; w < items; w += a.pairs) {
      const ProdItem it = row_item<C::kRows, C::kGran>(g, pl, start, w);
      uint64_t sum[C::kAcc / 2];
#pragma unroll
      for (int i = 0; i < C::kAcc / 2; ++i) sum[i] = 0;
      if (ROWS_M) {
        // one row, the 128 features of one weight block: one scale a block, fetched two blocks ahead
        const int r = rank * 128 + quarter * 32 + lane;
        const int nb = min(it.p0 / 128 + sub, n_blocks - 1);
        const float* xs = g.xs + (int64_t)(it.q0 + min(r, it.n - 1)) * g.xs_m;
        const float* ws = g.ws + it.e * g.ws_e + nb * g.ws_n;
        auto scale = [&](int t) { return t < it.t1 ? __ldg(xs + t * g.xs_g) * __ldg(ws + t * g.ws_k) : 0.0f; };
        float s0 = scale(it.t0), s1 = scale(it.t0 + 1);
        for (int t = it.t0; t < it.t1; ++t, ++k) {
          const int b = k % C::kBufs;
          const float s2 = scale(t + 2);
          const uint64_t ss = pack2(__float_as_uint(s0), __float_as_uint(s0));
          mbar_wait(&acc_full[b], (k / C::kBufs) & 1, abort_flag, g.status);
          tc_fence_after();
          const uint32_t tb = lanes + b * C::kBufCols + sub * 128;
          uint32_t v[2][16];
          tmem_ld16(tb, v[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            tmem_ld_wait();
            if (c < 7) {
              tmem_ld16(tb + 16 * (c + 1), v[(c + 1) & 1]);  // arrives while this chunk is added
            } else {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(acc_empty_s + 8 * b);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) fma2(sum[8 * c + i], pack2(v[c & 1][2 * i], v[c & 1][2 * i + 1]), ss);
          }
          s0 = s1;
          s1 = s2;
        }
      } else {
        // one feature, 32 rows
        const int half = (it.n + 31) / 32 * 16;
        const int nb = min((it.p0 + rank * 128) / 128, n_blocks - 1);
        for (int t = it.t0; t < it.t1; ++t, ++k) {
          const int in = (t - it.t0) % kF8FactorStages;
          if (in == 0) {
            named_bar_sync(2, kF8EpiThreads);  // the readers of the last scales are done
            const int count = min(kF8FactorStages, it.t1 - t);
            for (int u = tid; u < count * 64; u += kF8EpiThreads) {
              const int row = u % 64, tt = t + u / 64;
              factors[u] = row < it.n ? __ldg(g.xs + (int64_t)(it.q0 + row) * g.xs_m + tt * g.xs_g) *
                                            __ldg(g.ws + it.e * g.ws_e + nb * g.ws_n + tt * g.ws_k)
                                      : 0.0f;
            }
            named_bar_sync(2, kF8EpiThreads);
          }
          const int b = k % C::kBufs;
          mbar_wait(&acc_full[b], (k / C::kBufs) & 1, abort_flag, g.status);
          tc_fence_after();
          uint32_t v[32];
          const bool live = 32 * sub < 2 * half;
          if (live) {
            tmem_ld32(lanes + b * C::kBufCols + 32 * sub, v);
            tmem_ld_wait();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(acc_empty_s + 8 * b);
          if (live) {
            const uint32_t fs = smem_u32(factors) + (in * 64 + 32 * sub) * 4;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 f = lds128(fs + 16 * i);
              fma2(sum[2 * i], pack2(v[4 * i], v[4 * i + 1]), pack2(f.x, f.y));
              fma2(sum[2 * i + 1], pack2(v[4 * i + 2], v[4 * i + 3]), pack2(f.z, f.w));
            }
          }
        }
      }
      bool finish = true;
      if (pl.S > 1) {
        // this thread's sums of the slice, in its own order
        float4* mine = partial + (int64_t)((it.tile * pl.S + it.split) * 2 + rank) * (128 * 256 / 4) + tid;
#pragma unroll
        for (int i = 0; i < C::kAcc / 4; ++i) {
          uint4 u;
          unpack2(sum[2 * i], u.x, u.y);
          unpack2(sum[2 * i + 1], u.z, u.w);
          __stcg(reinterpret_cast<uint4*>(mine) + i * kF8EpiThreads, u);
        }
        named_bar_sync(1, kF8EpiThreads);
        if (tid == 0) {
          __threadfence();
          const unsigned old = atomicInc(reinterpret_cast<unsigned*>(&counters[it.tile * 2 + rank]), (unsigned)(pl.S - 1));
          misc[2] = old == (unsigned)(pl.S - 1) ? 1u : 0u;
          __threadfence();
        }
        named_bar_sync(1, kF8EpiThreads);
        finish = misc[2] != 0;
        if (finish) {
#pragma unroll
          for (int i = 0; i < C::kAcc / 2; ++i) sum[i] = 0;
          const uint64_t one = pack2(0x3F800000u, 0x3F800000u);
          for (int s = 0; s < pl.S; ++s) {
            const float4* src = partial + (int64_t)((it.tile * pl.S + s) * 2 + rank) * (128 * 256 / 4) + tid;
#pragma unroll
            for (int i = 0; i < C::kAcc / 4; ++i) {
              const uint4 u = __ldcg(reinterpret_cast<const uint4*>(src) + i * kF8EpiThreads);
              fma2(sum[2 * i], pack2(u.x, u.y), one);
              fma2(sum[2 * i + 1], pack2(u.z, u.w), one);
            }
          }
        }
      }
      if (!finish) continue;
      if (ROWS_M) {
        const int r = rank * 128 + quarter * 32 + lane;
        const int j0 = it.p0 + sub * 128;
        const int64_t at = (int64_t)(it.q0 + r) * g.out_ld + j0;
#pragma unroll
        for (int c = 0; c < C::kAcc / 16; ++c) {  // sixteen features at a time
          const int left = r < it.n ? g.N - j0 - 16 * c : 0;
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) unpack2(sum[8 * c + i], v[2 * i], v[2 * i + 1]);
          if (left >= 16) {
            if (g.out_type == kFp32) {
              float* dst = static_cast<float*>(g.out) + at + 16 * c;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t o[8] = {v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3],
                                       v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]};
                if (a.wide_store) {
                  stg256(dst + 8 * h, o);
                } else {
                  stg128(dst + 8 * h, make_uint4(o[0], o[1], o[2], o[3]));
                  stg128(dst + 8 * h + 4, make_uint4(o[4], o[5], o[6], o[7]));
                }
              }
            } else {
              uint16_t* dst = static_cast<uint16_t*>(g.out) + at + 16 * c;
              uint32_t o[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float lo = __uint_as_float(v[2 * i]), hi = __uint_as_float(v[2 * i + 1]);
                o[i] = g.out_type == kBf16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
              }
              if (a.wide_store) {
                stg256(dst, o);
              } else {
                stg128(dst, make_uint4(o[0], o[1], o[2], o[3]));
                stg128(dst + 8, make_uint4(o[4], o[5], o[6], o[7]));
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i < left) store_elem(g.out, at + 16 * c + i, g.out_type, __uint_as_float(v[i]));
          }
        }
      } else {
        // 32 consecutive features of a row per store
        const int j = it.p0 + rank * 128 + quarter * 32 + lane;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint32_t lo, hi;
          unpack2(sum[i], lo, hi);
          const int r = 32 * sub + 2 * i;
          if (j < g.N && r < it.n) store_elem(g.out, (int64_t)(it.q0 + r) * g.out_ld + j, g.out_type, __uint_as_float(lo));
          if (j < g.N && r + 1 < it.n)
            store_elem(g.out, (int64_t)(it.q0 + r + 1) * g.out_ld + j, g.out_type, __uint_as_float(hi));
        }
      }
      __syncwarp();  // whole warps read tensor memory
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the other may signal or read it
  tc_fence_after();
  if (warp == kF8Mma) tmem_dealloc2(tmem, 512);
}

template <bool ROWS_M>
static cudaError_t launch_orientation(const Fp8TcArgs& a, cudaStream_t st) {
  static std::atomic<bool> ready[64] = {};
  int dev = 0;
  cudaError_t rc = cudaGetDevice(&dev);
  if (rc != cudaSuccess) return rc;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  constexpr int bytes = Fp8Cfg<ROWS_M>::kAlloc;
  if (!ready[dev].load(std::memory_order_acquire)) {
    rc = cudaFuncSetAttribute(fp8_tc_kernel<ROWS_M>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (rc != cudaSuccess) return rc;
    ready[dev].store(true, std::memory_order_release);
  }
  fp8_tc_kernel<ROWS_M><<<2 * a.pairs, kF8Threads, bytes, st>>>(a);
  return cudaPeekAtLastError();
}

static bool grid16b(const void* p, int64_t stride) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 16 == 0 && stride < ((int64_t)1 << 39);
}

cudaError_t launch_fp8_tc(const ProdArgs& g, cudaStream_t st, bool* done) {
  *done = false;
  const int out_bytes = g.out_type == kFp32 ? 4 : 2;
  if (!grid16b(g.a, g.a_ld) || !grid16b(g.w, g.w_ld) || !grid16b(g.out, g.out_ld * out_bytes)) return cudaSuccess;
  if (g.E > 1 && (g.w_se % 16 != 0 || g.w_se <= 0)) return cudaSuccess;
  if (((double)g.rows / 64 + g.E) * ((g.N + 255) / 256) > 1e9) return cudaSuccess;  // tile numbers are 32-bit
  Fp8TcArgs a;
  a.g = g;
  const uint64_t xd[2] = {(uint64_t)g.K, (uint64_t)g.rows}, xl = (uint64_t)g.a_ld;
  const uint64_t wd[3] = {(uint64_t)g.K, (uint64_t)g.N, (uint64_t)g.E};
  const uint64_t wl[2] = {(uint64_t)g.w_ld, g.E > 1 ? (uint64_t)g.w_se : (uint64_t)g.w_ld};
  const uint32_t box[2] = {128, 128}, small[2] = {128, 16}, wbox[3] = {128, 128, 1};
  if (!make_prod_map(&a.map_x, kE4m3, g.a, 2, xd, &xl, box) || !make_prod_map(&a.map_xs, kE4m3, g.a, 2, xd, &xl, small) ||
      !make_prod_map(&a.map_w, kE4m3, g.w, 3, wd, wl, wbox))
    return cudaSuccess;  // (the plain kernel takes what a tensor map cannot describe)
  const int sms = prod_sm_count();
  if (sms < 2) return cudaErrorInvalidDevice;
  a.pairs = sms / 2;
  a.wide_store = (reinterpret_cast<uintptr_t>(g.out) & 31) == 0 && g.out_ld * out_bytes % 32 == 0;
  *done = true;
  // 64 rows an expert on average: up to there one or two tiles of 64 rows stream the weights at the
  // memory's rate, above it the row tiles of the other orientation do not run emptier than the memory
  return g.rows <= (int64_t)64 * g.E ? launch_orientation<false>(a, st) : launch_orientation<true>(a, st);
}

}  // namespace moe
