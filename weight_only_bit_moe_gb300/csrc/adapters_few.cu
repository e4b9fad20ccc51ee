// The adapters of a decode batch: few rows, each adapter's factors read once for one
// or a few of them.
//
//   mid[i, j] = sum_p x[r, p] A[l][j, p],   out[r, q] = base[r, q] + scale[l] sum_j mid[i, j] B[l][q, j]
//
// One launch.  A cluster of two to eight CTAs, as many as run at one time, has up to
// eight positions of one adapter: the tiles are numbered by a scan over all adapters.
//   first product: ranks on the MMA's M side, rows on its N side (8), the sum cut over
//     the cluster's warps.  Both operands go from memory straight into registers, 16
//     bytes a lane: the terms of the sum are dealt to the MMA's slots in the order in
//     which they arrive, the same for both.  B's rows are on their way to L2 meanwhile.
//   Every CTA adds up the cluster's parts of mid, in their order, over distributed
//     shared memory.
//   second: the columns are cut over the cluster; a thread holds two and multiplies in
//     fp32, mid read from shared memory by all threads alike.
//
// Bound by the chain of one latency after the other -- offsets, the rows' numbers, rows
// and A, the cluster, B -- not by memory: one row of 8 adapters of rank 16, 1024 x 512,
// takes 4.4 us of GPU time (floor 0.01), 64 rows with an adapter each of 4096 x 4096
// 10.8 (12.3 MB, floor 1.8), 246 rows of 8 adapters of rank 8, 1024 x 512, 5.1.  As two
// launches over global memory: 5.3, 12.5 and 6.4.
#include "adapters.cuh"

namespace moe {

constexpr int kFwThreads = 256, kFwWarps = kFwThreads / 32, kFwRows = 8;
constexpr int kFwCtas = 8;  // of a cluster, at most

struct FewSpan {
  int l, i, n;  // adapter (-1: none), first position, positions; n = 0: no such tile
};

// Tile k: the adapters' come first, then those of the rows without one.  All threads; `found` and `warp_tot` shared.
__device__ __forceinline__ FewSpan few_span(const AdapterArgs& a, int k, FewSpan* found, int* warp_tot) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.L + kFwThreads - 1) / kFwThreads;
  int run = 0, bad = 0;
  for (int u = 0; u < per; ++u) {
    const int l = tid * per + u;
    if (l >= a.L) break;
    const int i0 = __ldg(a.offsets + l), i1 = __ldg(a.offsets + l + 1);
    bad |= i0 < 0 || i1 < i0 || i1 > a.rows;
    run += (i1 - i0 + kFwRows - 1) / kFwRows;
  }
  int incl = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) warp_tot[warp] = incl;
  if (tid == 0) found->n = 0;
  if (__syncthreads_or(bad)) {
    if (bad && blockIdx.x == 0) atomicOr(a.status, kStatusRouting);
    FewSpan none;
    none.l = -1, none.i = 0, none.n = 0;
    return none;
  }
  int at = incl - run, all = 0;
#pragma unroll
  for (int w = 0; w < kFwWarps; ++w) {
    at += w < warp ? warp_tot[w] : 0;
    all += warp_tot[w];
  }
  if (k >= at && k < at + run) {
    int l = tid * per, i0, i1;
    for (;; ++l) {
      i0 = __ldg(a.offsets + l), i1 = __ldg(a.offsets + l + 1);
      const int tiles = (i1 - i0 + kFwRows - 1) / kFwRows;
      if (k < at + tiles) break;
      at += tiles;
    }
    found->l = l;
    found->i = i0 + (k - at) * kFwRows;
    found->n = min(kFwRows, i1 - found->i);
  } else if (tid == 0 && k >= all && a.out && a.base != a.out) {
    const int before = __ldg(a.offsets), from = __ldg(a.offsets + a.L);
    const int first = (before + kFwRows - 1) / kFwRows, k1 = k - all;
    const int i = k1 < first ? k1 * kFwRows : from + (k1 - first) * kFwRows;
    found->l = -1;
    found->i = i;
    found->n = max(0, min(kFwRows, (k1 < first ? before : a.rows) - i));
  }
  __syncthreads();
  return *found;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <int TYPE, int MT>  // MT: groups of 16 ranks at a time
__global__ void __launch_bounds__(kFwThreads) adapter_few_kernel(const __grid_constant__ AdapterArgs a) {
  __shared__ float red[kFwWarps][16 * MT][kFwRows + 1];
  __shared__ __align__(16) float part[kFwRows][kAdRank], mid[kFwRows][kAdRank];
  __shared__ int warp_tot[kFwWarps];
  __shared__ FewSpan found;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = (int)cluster_rank(), ctas = a.few_ctas;
  grid_dependents_launch();
  grid_dependency_wait();
  const FewSpan s = few_span(a, blockIdx.x / ctas, &found, warp_tot);
  if (s.n == 0) return;  // (the whole cluster)
  const int i = s.i;
  const uint16_t* base = static_cast<const uint16_t*>(a.base);
  uint16_t* out = static_cast<uint16_t*>(a.out);
  // columns of this CTA
  const int each = ((a.Q + ctas - 1) / ctas + 7) / 8 * 8;
  const int q0 = rank * each, q1 = min(a.Q, q0 + each);
  if (s.l < 0) {  // no adapter
    for (int n = 0; n < s.n; ++n) {
      const int r = row_of(a.order, a.rows, i + n, a.status);
      if (r >= 0)
        for (int q = q0 + 2 * tid; q < q1; q += 2 * kFwThreads)
          *reinterpret_cast<uint32_t*>(out + r * a.out_ld + q) =
              base ? *reinterpret_cast<const uint32_t*>(base + r * a.base_ld + q) : 0u;
    }
    return;
  }
  const uint16_t* const second = static_cast<const uint16_t*>(a.s) + s.l * a.s_l;
  if (out)
    for (int q = q0 + tid; q < q1; q += kFwThreads)
      for (int j = 0; j < a.R; j += 64) prefetch_l2(second + q * a.s_r + j);

  {  // ------------------------------------------------------------ mid
    const int row = g < s.n ? row_of(a.order, a.rows, i + g, a.status) : -1;
    const uint16_t* const x = static_cast<const uint16_t*>(a.in) + (int64_t)max(row, 0) * a.in_ld + 8 * t;
    const uint16_t* const f = static_cast<const uint16_t*>(a.f) + s.l * a.f_l + 8 * t;
    const int units = (a.P + 31) / 32, w = rank * kFwWarps + warp;  // 32 terms a unit
    const int u0 = (int)((int64_t)w * units / (ctas * kFwWarps)), u1 = (int)((int64_t)(w + 1) * units / (ctas * kFwWarps));
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int j0 = 0; j0 < a.R; j0 += 16 * MT) {
      float acc[MT][4] = {};
#pragma unroll 2
      for (int u = u0; u < u1; ++u) {
        const int p = 32 * u;
        const bool in = p + 8 * t < a.P;
        const uint4 xv = in && row >= 0 ? __ldg(reinterpret_cast<const uint4*>(x + p)) : zero;
        uint4 lo[MT], hi[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int j = j0 + 16 * m + g;
          lo[m] = in && j < a.R ? __ldg(reinterpret_cast<const uint4*>(f + j * a.f_r + p)) : zero;
          hi[m] = in && j + 8 < a.R ? __ldg(reinterpret_cast<const uint4*>(f + (j + 8) * a.f_r + p)) : zero;
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mma_type<TYPE>(acc[m], lo[m].x, hi[m].x, lo[m].y, hi[m].y, xv.x, xv.y);
          mma_type<TYPE>(acc[m], lo[m].z, hi[m].z, lo[m].w, hi[m].w, xv.z, xv.w);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[warp][16 * m + g + 8 * (v >> 1)][2 * t + (v & 1)] = acc[m][v];
      __syncthreads();
      for (int u = tid; u < 16 * MT * kFwRows; u += kFwThreads) {
        const int r = u / (16 * MT), j = u % (16 * MT);
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kFwWarps; ++k) sum += red[k][j][r];
        part[r][j0 + j] = sum;
      }
      __syncthreads();
    }
  }
  cluster_sync_all();
  for (int u = tid; u < s.n * a.R; u += kFwThreads) {
    const int r = u / a.R, j = u - r * a.R;
    float v[kFwCtas], sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kFwCtas; ++c) {
      v[c] = 0.0f;
      if (c < ctas)
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[c]) : "r"(map_to_rank(smem_u32(&part[r][j]), c)) : "memory");
    }
#pragma unroll
    for (int c = 0; c < kFwCtas; ++c) sum += v[c];
    mid[r][j] = sum;
    if (a.want_mid && rank == 0) a.mid[(int64_t)(i + r) * a.R + j] = sum;
  }
  // ------------------------------------------------------------ out
  const float scale = a.scale ? __ldg(a.scale + s.l) : 1.0f;
  int row[kFwRows];
#pragma unroll
  for (int r = 0; r < kFwRows; ++r) row[r] = out && r < s.n ? row_of(a.order, a.rows, i + r, a.status) : -1;
  __syncthreads();
  for (int q = q0 + 2 * tid; out && q < q1; q += 2 * kFwThreads) {
    uint32_t was[kFwRows];
#pragma unroll
    for (int r = 0; r < kFwRows; ++r)
      was[r] = row[r] >= 0 && base ? *reinterpret_cast<const uint32_t*>(base + row[r] * a.base_ld + q) : 0u;
    const uint16_t* const f = second + q * a.s_r;
    float acc[kFwRows][2] = {};
#pragma unroll 2
    for (int j = 0; j < a.R; j += 8) {
      const uint4 u0 = __ldg(reinterpret_cast<const uint4*>(f + j)), u1 = __ldg(reinterpret_cast<const uint4*>(f + a.s_r + j));
      const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
      float2 v0[4], v1[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v0[c] = unpack_type<TYPE>(w0[c]);
        v1[c] = unpack_type<TYPE>(w1[c]);
      }
#pragma unroll
      for (int r = 0; r < kFwRows; ++r) {
        if (r >= s.n) break;
        const float4 m0 = *reinterpret_cast<const float4*>(&mid[r][j]), m1 = *reinterpret_cast<const float4*>(&mid[r][j + 4]);
        const float m[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          acc[r][0] = fmaf(m[2 * c], v0[c].x, fmaf(m[2 * c + 1], v0[c].y, acc[r][0]));
          acc[r][1] = fmaf(m[2 * c], v1[c].x, fmaf(m[2 * c + 1], v1[c].y, acc[r][1]));
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kFwRows; ++r) {
      if (row[r] < 0) continue;
      const float2 b = unpack_type<TYPE>(was[r]);
      *reinterpret_cast<uint32_t*>(out + row[r] * a.out_ld + q) =
          pack_type<TYPE>(fmaf(scale, acc[r][0], b.x), fmaf(scale, acc[r][1], b.y));
    }
  }
  cluster_sync_all();  // (nobody leaves while its part is read)
}

template <int TYPE, int MT>
static cudaError_t launch_few(const AdapterArgs& a, int tiles, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * a.few_ctas));
  cfg.blockDim = dim3(kFwThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.few_ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, adapter_few_kernel<TYPE, MT>, a);
}

cudaError_t launch_adapter_few(AdapterArgs& a, bool mid_wanted, cudaStream_t st) {
  const int sms = prod_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  a.want_mid = mid_wanted;
  // Tiles, at most: one for each row, or for each eight and one more for each adapter and both ends.  Two CTAs fit an
  // SM (64 requests with an adapter each take 11.6 us in clusters of eight, which run in two rounds, 10.8 in those of four).
  const int tiles = min(a.rows, a.rows / kFwRows + a.L + 2);
  a.few_ctas = kFwCtas;
  while (a.few_ctas > 2 && tiles * a.few_ctas > 2 * sms) a.few_ctas /= 2;
  if (a.R <= 16) return a.type == kBf16 ? launch_few<kBf16, 1>(a, tiles, st) : launch_few<kFp16, 1>(a, tiles, st);
  return a.type == kBf16 ? launch_few<kBf16, 2>(a, tiles, st) : launch_few<kFp16, 2>(a, tiles, st);
}

}  // namespace moe
