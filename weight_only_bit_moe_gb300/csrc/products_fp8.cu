// Block-scaled FP8 product on tcgen05 tensor cores (sm_103a):
//
//   y[r, n] = sum_b xs[r, b] ws[n / 128, b] D_b[r, n],   D_b[r, n] = sum_{k in b} x[r, k] w[n, k]
//
// over blocks b of 128 terms, dense or grouped by expert.  A CTA computes each D_b
// of its tile into tensor memory -- a stage of the pipeline is one block, 128
// bytes of every row -- and eight epilogue warps add it, times its scale, to fp32
// sums in registers while the MMAs fill another buffer.  Scales are arbitrary
// fp32, so D_b cannot stay in the tensor core's accumulator over blocks; the
// hand-over of a buffer and the multiply-adds, 128 x 256 a block, are what bounds
// the product where memory does not.
//
// Two orientations:
//   rows on M (many tiles): 128 rows x 256 features, a thread owns one row and the
//     128 features of one weight block: one scale per thread and block.
//   rows on N (few tiles): 128 features x up to 64 rows, a thread owns one feature
//     and 32 rows, whose scales it reads from shared memory.
// With rows on N a 256-row tile would read 32 scales from shared memory for 128
// sums, more than the shared memory delivers in the time of the block's MMAs;
// with rows on M a tile of few rows would run the MMA nearly empty.
//
// Single CTAs, not the pairs of the 16-bit products: a buffer passes from the MMA
// to the epilogue and back once a block, and across two CTAs that round trip took
// longer than the block's MMAs (0.63 us a block and tile, here 0.44, of which the
// MMAs alone take 0.34).  The 128 sums of a thread leave 40 registers for the rest:
// 16 columns of tensor memory at a time and plain multiply-adds fit, packed ones or
// 32 columns spill inside the loop (293 us when the prompt below took 188).
//
// Measured on GB300: 8191 x 4096 x 7168 184 us, 2615 TFLOP/s (the bf16 product of
// these sizes at the measured peak takes 256); 32 experts of 225 to 285 rows, 4096 x
// 4096, 157 us; 5 rows x 4096 x 7168 11.4 us with the weights in L2 and 13.0 from memory,
// 38912 x 7168 47 us, 6.0 TB/s.
#include <atomic>

#include "gemm.cuh"
#include "products_tc.cuh"

namespace moe {

constexpr int kF8Threads = 320;  // eight epilogue warps, producer, MMA
constexpr int kF8EpiWarps = 8, kF8EpiThreads = 256, kF8Producer = 8, kF8Mma = 9;
static_assert(kF8Threads == (kF8EpiWarps + 2) * 32, "every other warp would run the epilogue");
constexpr int kF8FactorStages = 64;  // blocks whose scales are staged at a time (rows on N)

template <bool ROWS_M>
struct Fp8Cfg {
  static constexpr int kRows = ROWS_M ? 128 : 64;       // rows of a tile
  static constexpr int kFeatures = ROWS_M ? 256 : 128;  // features of a tile
  static constexpr int kGran = 16;
  static constexpr int kAcc = ROWS_M ? 128 : 32;   // sums per thread
  static constexpr int kBufCols = ROWS_M ? 256 : 64, kBufs = ROWS_M ? 2 : 4;
  static constexpr int kPBytes = 128 * 128;
  static constexpr int kQBytes = ROWS_M ? 256 * 128 : 64 * 128;
  static constexpr int kSlot = kPBytes + kQBytes;
  static constexpr int kStages = ROWS_M ? 4 : 8;
  static constexpr int kBar = kStages * kSlot;
  static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 1;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kFactors = (kMisc + 32 + 15) / 16 * 16;
  static constexpr int kBytes = kFactors + (ROWS_M ? 0 : kF8FactorStages * 64 * 4);
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc + (kProdGroups + 1) * 4 + 64 <= 227 * 1024, "shared memory over the per-CTA limit");
};

struct Fp8TcArgs {
  CUtensorMap map_x[4];  // boxes of 128, 64, 32 and 16 rows of x
  CUtensorMap map_w;     // boxes of a tile's features
  ProdArgs g;
  int wide_store;        // 32-byte stores are aligned
};

template <bool ROWS_M>
__global__ void __launch_bounds__(kF8Threads, 1) fp8_tc_kernel(const __grid_constant__ Fp8TcArgs a) {
  using C = Fp8Cfg<ROWS_M>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ int start[kProdGroups + 1];
  __shared__ int warp_tot[kF8Threads / 32];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem_s = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBar);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + C::kBufs;
  uint64_t* drain_bar = acc_empty + C::kBufs;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kMisc);  // [0] tmem base, [1] abort, [2] last
  volatile int* abort_flag = reinterpret_cast<volatile int*>(&misc[1]);
  const ProdArgs& g = a.g;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < C::kBufs; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], kF8EpiWarps); }
    mbar_init(drain_bar, 1);
    misc[1] = 0;
    fence_mbar_init();
  }
  if (warp == kF8Mma) {
    tmem_alloc(&misc[0], 512);
    tmem_relinquish();
  }
  if (warp == kF8Producer && lane < 5) prefetch_map(lane < 4 ? &a.map_x[lane] : &a.map_w);
  // (launched early: everything before this line touches nothing that an earlier kernel writes)
  grid_dependents_launch();
  grid_dependency_wait();
  RowPlan pl;
  pl.p_tiles = (g.N + C::kFeatures - 1) / C::kFeatures;
  pl.stages = (g.K + 127) / 128;
  plan_groups<C::kRows, kF8Threads>(g, pl.p_tiles, start, warp_tot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  pl.tiles = min(start[g.E], kProdItems);
  pl.S = plan_slices(pl, gridDim.x, 1, ROWS_M ? 1 << 30 : 0, 256);
  const int items = pl.tiles * pl.S;

  if (warp == kF8Producer) {
    // ------------------------------------------------------------ producer
    Ring<C::kStages> at_slot;
    uint32_t filled = 0;
    for (int w = blockIdx.x, e = 0; w < items; w += gridDim.x) {
      const ProdItem it = row_item<C::kRows, C::kGran, C::kFeatures>(g, pl, start, w, e);
      const int rows = (it.n + 15) / 16 * 16;  // copied
      for (int t = it.t0; t < it.t1; ++t) {
        const int s = at_slot.i;
        if (!warp_wait(&empty[s], at_slot.phase ^ 1, abort_flag, g.status)) break;
        const uint32_t bar = smem_u32(&full[s]), ps = smem_s + s * C::kSlot, qs = ps + C::kPBytes;
        expect_tx_elect(&full[s], (C::kFeatures + rows) * 128);
        tma1_3d(ROWS_M ? qs : ps, &a.map_w, 128 * t, it.p0, it.e, bar);
        const uint32_t xd = ROWS_M ? ps : qs;
        if (rows == C::kRows) {
          tma1_2d(xd, &a.map_x[ROWS_M ? 0 : 1], 128 * t, it.q0, bar);
        } else {
          int at = 0;
#pragma unroll
          for (int i = ROWS_M ? 1 : 2; i < 4; ++i) {
            const int box = 128 >> i;
            if (rows & box) {
              tma1_2d(xd + 128 * at, &a.map_x[i], 128 * t, it.q0 + at, bar);
              at += box;
            }
          }
        }
        at_slot.next();
        ++filled;
      }
      if (*abort_flag) break;
    }
    // leave no copy in flight
    for (uint32_t i = 0; i < (uint32_t)C::kStages && i < filled; ++i) {
      const uint32_t u = filled - 1 - i;
      mbar_drain(&full[u % C::kStages], (u / C::kStages) & 1, g.status);
    }
  } else if (warp == kF8Mma) {
    // ------------------------------------------------------------ MMA issuer
    Ring<C::kStages> at_slot;
    Ring<C::kBufs> at_buf;
    const uint64_t pd = smem_desc_sw128(smem_s), qd = smem_desc_sw128(smem_s + C::kPBytes);
    for (int w = blockIdx.x, e = 0; w < items; w += gridDim.x) {
      const ProdItem it = row_item<C::kRows, C::kGran, C::kFeatures>(g, pl, start, w, e);
      // E4M3 operands and fp32 sums have the fields of fp16 operands and fp32 sums
      const uint32_t idesc = idesc_f16_f32(128, ROWS_M ? 256 : (it.n + 15) / 16 * 16, 0u);
      for (int t = it.t0; t < it.t1; ++t) {
        const uint32_t s = at_slot.i, b = at_buf.i;
        if (!warp_wait(&full[s], at_slot.phase, abort_flag, g.status) ||
            !warp_wait(&acc_empty[b], at_buf.phase ^ 1, abort_flag, g.status))
          break;
        tc_fence_after();
        const uint32_t slot = s * (C::kSlot >> 4);  // (descriptor addresses count 16 bytes and do not carry)
        umma1_f8_block_elect(tmem + b * C::kBufCols, pd + slot, qd + slot, idesc);
        umma_commit_elect(&acc_full[b]);
        umma_commit_elect(&empty[s]);
        at_slot.next();
        at_buf.next();
      }
    }
    umma_commit_elect(drain_bar);
    mbar_drain(drain_bar, 0, g.status);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, sub = warp >> 2;  // TMEM lanes; half of the tile's columns
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    float* factors = reinterpret_cast<float*>(smem + C::kFactors);
    int32_t* counters = reinterpret_cast<int32_t*>(g.scratch);
    float4* partial = reinterpret_cast<float4*>(g.scratch + kProdCounterBytes);
    const int n_blocks = (g.N + 127) / 128;
    Ring<C::kBufs> at_buf;
    for (int w = blockIdx.x, e = 0; w < items; w += gridDim.x) {
      const ProdItem it = row_item<C::kRows, C::kGran, C::kFeatures>(g, pl, start, w, e);
      float sum[C::kAcc];
#pragma unroll
      for (int i = 0; i < C::kAcc; ++i) sum[i] = 0.0f;
      if (ROWS_M) {
        // one row, the 128 features of one weight block: one scale a block.  Its two factors are
        // fetched two blocks ahead, two blocks at a time, and first touched when they are due.
        const int r = quarter * 32 + lane;
        const int nb = min(it.p0 / 128 + sub, n_blocks - 1);
        const float* xs = g.xs + (int64_t)(it.q0 + min(r, it.n - 1)) * g.xs_m + it.t0 * g.xs_g;
        const float* ws = g.ws + it.e * g.ws_e + nb * g.ws_n + it.t0 * g.ws_k;
        float x[2], y[2];
        int ahead = it.t0;
        auto fetch = [&](int i) {
          x[i] = __ldg(xs), y[i] = __ldg(ws);
          if (++ahead < it.t1) xs += g.xs_g, ws += g.ws_k;
        };
        fetch(0);
        fetch(1);
        for (int t = it.t0; t < it.t1; t += 2) {
          const float s0 = x[0] * y[0], s1 = x[1] * y[1];
          fetch(0);
          fetch(1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (t + h < it.t1) {
              const uint32_t b = at_buf.i;
              const float sc = h ? s1 : s0;
              warp_wait(&acc_full[b], at_buf.phase, abort_flag, g.status);
              tc_fence_after();
              const uint32_t tb = lanes + b * C::kBufCols + sub * 128;
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                uint32_t v[16];
                tmem_ld16(tb + 16 * c, v);
                tmem_ld_wait();
                if (c == 7) {
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) mbar_arrive(&acc_empty[b]);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[16 * c + i] = fmaf(__uint_as_float(v[i]), sc, sum[16 * c + i]);
              }
              at_buf.next();
            }
          }
        }
      } else {
        // one feature, 32 rows
        const int nb = it.p0 / 128;
        for (int t = it.t0; t < it.t1; ++t, at_buf.next()) {
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
          const uint32_t b = at_buf.i;
          warp_wait(&acc_full[b], at_buf.phase, abort_flag, g.status);
          tc_fence_after();
          uint32_t v[32];
          const bool live = 32 * sub < it.n;
          if (live) {
            tmem_ld32(lanes + b * C::kBufCols + 32 * sub, v);
            tmem_ld_wait();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[b]);
          if (live) {
            const uint32_t fs = smem_u32(factors) + (in * 64 + 32 * sub) * 4;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 f = lds128(fs + 16 * i);
              sum[4 * i] = fmaf(__uint_as_float(v[4 * i]), __uint_as_float(f.x), sum[4 * i]);
              sum[4 * i + 1] = fmaf(__uint_as_float(v[4 * i + 1]), __uint_as_float(f.y), sum[4 * i + 1]);
              sum[4 * i + 2] = fmaf(__uint_as_float(v[4 * i + 2]), __uint_as_float(f.z), sum[4 * i + 2]);
              sum[4 * i + 3] = fmaf(__uint_as_float(v[4 * i + 3]), __uint_as_float(f.w), sum[4 * i + 3]);
            }
          }
        }
      }
      bool finish = true;
      if (pl.S > 1) {
        // this thread's sums of the slice, in its own order
        float4* mine = partial + (int64_t)(it.tile * pl.S + it.split) * (128 * 256 / 4) + tid;
#pragma unroll
        for (int i = 0; i < C::kAcc / 4; ++i) {
          __stcg(mine + i * kF8EpiThreads, make_float4(sum[4 * i], sum[4 * i + 1], sum[4 * i + 2], sum[4 * i + 3]));
        }
        named_bar_sync(1, kF8EpiThreads);
        if (tid == 0) {
          misc[2] = slice_arrive_last(&counters[it.tile], pl.S) ? 1u : 0u;
        }
        named_bar_sync(1, kF8EpiThreads);
        finish = misc[2] != 0;
        if (finish) {
#pragma unroll
          for (int i = 0; i < C::kAcc; ++i) sum[i] = 0.0f;
          // (rows on N: four slices' loads in flight, as they are few)
          const float4* src = partial + (int64_t)it.tile * pl.S * (128 * 256 / 4) + tid;
#pragma unroll(ROWS_M ? 1 : 4)
          for (int s = 0; s < pl.S; ++s, src += 128 * 256 / 4) {
#pragma unroll
            for (int i = 0; i < C::kAcc / 4; ++i) {
              const float4 u = __ldcg(src + i * kF8EpiThreads);
              sum[4 * i] += u.x, sum[4 * i + 1] += u.y, sum[4 * i + 2] += u.z, sum[4 * i + 3] += u.w;
            }
          }
        }
      }
      if (!finish) continue;
      if (ROWS_M && a.wide_store) {
        // A lane holds a row, but a store of 32 bytes to each of 32 lines takes longer than one of 8 whole
        // lines: four lanes trade chunks, so that they write 128 consecutive bytes of a row (32 experts of
        // 256 rows, 4096 x 4096: 132 us, with each lane's own rows 136; 10 of 1408, 6656 x 1024: 119 and 127).
        const int size = g.out_type == kFp32 ? 4 : 2, per = 32 / size;  // bytes and features of a chunk
        const int j0 = it.p0 + sub * 128 + (lane & 3) * per, r0 = quarter * 32 + (lane & ~3);
        unsigned char* dst = static_cast<unsigned char*>(g.out) + ((int64_t)(it.q0 + r0) * g.out_ld + j0) * size;
        auto send = [&](uint32_t (&v)[4][8], int step) {  // the chunks of step * 128 bytes on
#pragma unroll
          for (int b = 1; b <= 2; b <<= 1) {
            const bool up = lane & b;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (c & b) continue;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? v[c][i] : v[c + b][i], b);
                if (up) v[c][i] = got; else v[c + b][i] = got;
              }
            }
          }
          const int left = g.N - j0 - 4 * per * step;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (r0 + c >= it.n) continue;
            unsigned char* d = dst + (int64_t)c * g.out_ld * size + 128 * step;
            if (left >= per) {
              stg256(d, v[c]);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                if (size == 4) {
                  if (i < left) reinterpret_cast<uint32_t*>(d)[i] = v[c][i];
                } else {
                  if (2 * i < left) reinterpret_cast<uint16_t*>(d)[2 * i] = (uint16_t)v[c][i];
                  if (2 * i + 1 < left) reinterpret_cast<uint16_t*>(d)[2 * i + 1] = (uint16_t)(v[c][i] >> 16);
                }
              }
            }
          }
        };
        uint32_t v[4][8];
        if (size == 4) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i / 8][i % 8] = __float_as_uint(sum[32 * t + i]);
            send(v, t);
          }
        } else {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float lo = sum[64 * t + 2 * i], hi = sum[64 * t + 2 * i + 1];
              v[i / 8][i % 8] = g.out_type == kBf16 ? pack_bf16x2(lo, hi) : pack_half2(lo, hi);
            }
            send(v, t);
          }
        }
      } else if (ROWS_M) {
        // Rows whose sectors do not start with a chunk: each lane its own, as whole sectors (traded chunks of
        // 16 bytes: 10 experts of 1408 rows, 6648 x 128 78 us instead of 68).
        const int r = quarter * 32 + lane;
        const int j0 = it.p0 + sub * 128;
        const int64_t at = (int64_t)(it.q0 + r) * g.out_ld + j0;
        const bool f32 = g.out_type == kFp32, bf = g.out_type == kBf16;
        unsigned char* dst = static_cast<unsigned char*>(g.out) + at * (f32 ? 4 : 2);
        const bool sector = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;  // (else 16 past one)
        auto pack8 = [&](int f, uint32_t* o) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[i] = bf ? pack_bf16x2(sum[f + 2 * i], sum[f + 2 * i + 1]) : pack_half2(sum[f + 2 * i], sum[f + 2 * i + 1]);
        };
#pragma unroll
        for (int c = 0; c < C::kAcc / 16; ++c) {  // sixteen features at a time
          const int left = r < it.n ? g.N - j0 - 16 * c : 0;
          if (left >= 16) {
            uint32_t o[8];
            if (f32) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(sum[16 * c + 8 * h + i]);
                if (sector) {
                  stg256(dst + 64 * c + 32 * h, o);
                } else {
                  stg128(dst + 64 * c + 32 * h, make_uint4(o[0], o[1], o[2], o[3]));
                  stg128(dst + 64 * c + 32 * h + 16, make_uint4(o[4], o[5], o[6], o[7]));
                }
              }
            } else if (sector) {
              pack8(16 * c, o);
              pack8(16 * c + 8, o + 4);
              stg256(dst + 32 * c, o);
            } else {  // eight features further, so that whole sectors are written here too
              if (c == 0) {
                pack8(0, o);
                stg128(dst, make_uint4(o[0], o[1], o[2], o[3]));
              }
              pack8(16 * c + 8, o);
              if (c + 1 < C::kAcc / 16 && left >= 32) {
                pack8((16 * c + 16) % C::kAcc, o + 4);
                stg256(dst + 32 * c + 16, o);
              } else {
                stg128(dst + 32 * c + 16, make_uint4(o[0], o[1], o[2], o[3]));
              }
            }
          } else if (left > 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i < left) store_elem(g.out, at + 16 * c + i, g.out_type, sum[16 * c + i]);
          }
        }
      } else {
        // 32 consecutive features of a row per store
        const int j = it.p0 + quarter * 32 + lane;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int r = 32 * sub + i;
          if (j < g.N && r < it.n) store_elem(g.out, (int64_t)(it.q0 + r) * g.out_ld + j, g.out_type, sum[i]);
        }
      }
      __syncwarp();  // whole warps read tensor memory
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kF8Mma) tmem_dealloc(tmem, 512);
}

template <bool ROWS_M>
static cudaError_t launch_orientation(const Fp8TcArgs& a, int sms, cudaStream_t st) {
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
  return launch_dependent(fp8_tc_kernel<ROWS_M>, dim3(sms), dim3(kF8Threads), bytes, st, a);
}

static bool grid16b(const void* p, int64_t stride) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 16 == 0 && stride < ((int64_t)1 << 39);
}

cudaError_t launch_fp8_tc(const ProdArgs& g, cudaStream_t st, bool* done) {
  *done = false;
  const int out_bytes = g.out_type == kFp32 ? 4 : 2;
  if (!grid16b(g.a, g.a_ld) || !grid16b(g.w, g.w_ld) || !grid16b(g.out, g.out_ld * out_bytes)) return cudaSuccess;
  if (g.E > 1 && (g.w_se % 16 != 0 || g.w_se <= 0)) return cudaSuccess;
  if (((double)g.rows / 64 + g.E) * ((g.N + 127) / 128) > 1e9) return cudaSuccess;  // tile numbers are 32-bit
  // Rows on N where its tiles, of half the rows and half the features, all run at one time: 1024 x 4096 (N x K),
  // 256 rows 11.5 and 17.0 us with rows on M; 16384 x 4096, 16 rows 15.2 and 19.5; 4 experts of 100 rows, 2048 x
  // 2048 11.9 and 12.3.  With more tiles rows on M are ahead for any rows: 24576 x 4096, 16 rows 28.6 and 21.3; 128
  // experts of one row, 4096 x 4096 340 and 316.  Where rows on N are too many tiles for two slices and rows on M few
  // enough for four, a long sum is faster in those: 8192 x 7168, 128 rows 25.7 and 23.2, 5120 x 16384 45.8 and 32.1;
  // up to 40 blocks it is not (8192 x 5120 19.8 and 20.6).
  const int sms = prod_sm_count();
  if (sms <= 0 || sms > kProdWidth) return cudaErrorInvalidDevice;
  const int64_t groups = g.E < g.rows ? g.E : g.rows, each = (g.rows + groups - 1) / groups;  // (rows > 0)
  const int64_t tiles_n = groups * ((each + 63) / 64) * ((g.N + 127) / 128);
  const int64_t tiles_m = groups * ((each + 127) / 128) * ((g.N + 255) / 256);
  const bool rows_m = tiles_n > sms || (2 * tiles_n > sms && 4 * tiles_m <= sms && g.K > 40 * 128);
  Fp8TcArgs a;
  a.g = g;
  const uint64_t xd[2] = {(uint64_t)g.K, (uint64_t)g.rows}, xl = (uint64_t)g.a_ld;
  const uint64_t wd[3] = {(uint64_t)g.K, (uint64_t)g.N, (uint64_t)g.E};
  const uint64_t wl[2] = {(uint64_t)g.w_ld, g.E > 1 ? (uint64_t)g.w_se : (uint64_t)g.w_ld};
  const uint32_t wbox[3] = {128, rows_m ? 256u : 128u, 1};
  bool ok = make_prod_map(&a.map_w, kE4m3, g.w, 3, wd, wl, wbox);
  for (int i = 0; i < 4 && ok; ++i) {
    const uint32_t box[2] = {128, 128u >> i};
    ok = make_prod_map(&a.map_x[i], kE4m3, g.a, 2, xd, &xl, box);
  }
  if (!ok) return cudaSuccess;  // (the plain kernel takes what a tensor map cannot describe)
  a.wide_store = (reinterpret_cast<uintptr_t>(g.out) & 31) == 0 && g.out_ld * out_bytes % 32 == 0;
  *done = true;
  return rows_m ? launch_orientation<true>(a, sms, st) : launch_orientation<false>(a, sms, st);
}

}  // namespace moe
