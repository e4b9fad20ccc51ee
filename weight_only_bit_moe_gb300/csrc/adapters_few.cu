// The adapters of a decode batch: few rows, each adapter's factors read once for one
// or a few of them.
//
//   mid[i, j] = sum_p x[r, p] A[l][j, p],   out[r, q] = base[r, q] + scale[l] sum_j mid[i, j] B[l][q, j]
//
// Two launches.  A CTA belongs to a position: to up to eight of one adapter where it
// is the first of eight, else it leaves.  It finds its adapter by comparing all
// offsets at one time.
//   first: ranks on the MMA's M side, rows on its N side (8).  Both operands go from
//     memory straight into registers, 16 bytes a lane: the terms of the sum are dealt
//     to the MMA's slots in the order in which they arrive, the same for both.  K is
//     cut into slices over CTAs and warps.
//   second: a thread holds two output columns and multiplies in fp32; mid, the sum of
//     its slices in their order, is read from shared memory by all threads alike.
#include "adapters.cuh"

namespace moe {

constexpr int kFwThreads = 256, kFwWarps = kFwThreads / 32, kFwRows = 8;
constexpr int kFwStep = kFwWarps * 32;  // terms of the sum that a CTA takes at a time
constexpr int kFwCols = 2 * kFwThreads;

struct FewSpan {
  int l, n;  // adapter (-1: none) and rows; n = 0: another CTA has the position
};

// What the CTA of position i does; all threads.
__device__ __forceinline__ FewSpan few_span(const AdapterArgs& a, int i, int* warp_tot) {
  int below = 0;
  for (int l = threadIdx.x; l <= a.L; l += kFwThreads) below += min(max(__ldg(a.offsets + l), 0), a.rows) <= i;
  below = __reduce_add_sync(0xffffffffu, below);
  if ((threadIdx.x & 31) == 0) warp_tot[threadIdx.x >> 5] = below;
  __syncthreads();
  below = 0;
#pragma unroll
  for (int w = 0; w < kFwWarps; ++w) below += warp_tot[w];
  FewSpan s;
  s.l = below - 1;
  s.n = 1;
  if (s.l < 0 || s.l >= a.L) {
    s.l = -1;
    return s;
  }
  int i0, i1;
  adapter_rows(a.offsets, a.rows, s.l, i0, i1);
  s.n = i < i0 || i >= i1 || (i - i0) % kFwRows ? 0 : min(kFwRows, i1 - i);
  return s;
}

template <int TYPE, int MT>
__global__ void __launch_bounds__(kFwThreads) adapter_few_mid_kernel(const __grid_constant__ AdapterArgs a) {
  __shared__ float red[kFwWarps][16 * MT][kFwRows];
  __shared__ int warp_tot[kFwWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int i = blockIdx.x, j0 = blockIdx.z * 16 * MT;
  grid_dependents_launch();
  grid_dependency_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
    for (int l = tid; l < a.L; l += kFwThreads)
      if (adapter_bad(a.offsets, a.rows, l)) atomicOr(a.status, kStatusRouting);
  const FewSpan s = few_span(a, i, warp_tot);
  if (s.l < 0 || s.n == 0) return;
  const int row = g < s.n ? row_of(a.order, a.rows, i + g, a.status) : -1;
  const uint16_t* x = static_cast<const uint16_t*>(a.in) + (int64_t)max(row, 0) * a.in_ld;
  const uint16_t* f = static_cast<const uint16_t*>(a.f) + s.l * a.f_l;
  const int steps = (a.P + kFwStep - 1) / kFwStep;
  const int s0 = (int)((int64_t)blockIdx.y * steps / gridDim.y), s1 = (int)((int64_t)(blockIdx.y + 1) * steps / gridDim.y);
  float acc[MT][4] = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 4
  for (int step = s0; step < s1; ++step) {
    const int p = step * kFwStep + warp * 32 + t * 8;
    const bool in = p < a.P;
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
  for (int m = 0; m < MT; ++m) {
    red[warp][16 * m + g][2 * t] = acc[m][0];
    red[warp][16 * m + g][2 * t + 1] = acc[m][1];
    red[warp][16 * m + g + 8][2 * t] = acc[m][2];
    red[warp][16 * m + g + 8][2 * t + 1] = acc[m][3];
  }
  __syncthreads();
  float* out = a.part + (int64_t)blockIdx.y * a.rows * a.R;
  for (int u = tid; u < 16 * MT * kFwRows; u += kFwThreads) {
    const int r = u / (16 * MT), j = u % (16 * MT);
    if (r >= s.n || j0 + j >= a.R) continue;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kFwWarps; ++w) sum += red[w][j][r];
    out[(int64_t)(i + r) * a.R + j0 + j] = sum;
  }
}

template <int TYPE>
__global__ void __launch_bounds__(kFwThreads) adapter_few_out_kernel(const __grid_constant__ AdapterArgs a) {
  __shared__ float mid[kFwRows][kAdRank];
  __shared__ int warp_tot[kFwWarps];
  const int tid = threadIdx.x, i = blockIdx.x, q = blockIdx.y * kFwCols + 2 * tid;
  grid_dependents_launch();
  grid_dependency_wait();
  const FewSpan s = few_span(a, i, warp_tot);
  if (s.n == 0) return;
  const uint16_t* base = static_cast<const uint16_t*>(a.base);
  uint16_t* out = static_cast<uint16_t*>(a.out);
  if (s.l < 0) {  // no adapter
    const int r = a.base == a.out ? -1 : row_of(a.order, a.rows, i, a.status);
    if (r >= 0 && q < a.Q)
      *reinterpret_cast<uint32_t*>(out + r * a.out_ld + q) =
          base ? *reinterpret_cast<const uint32_t*>(base + r * a.base_ld + q) : 0u;
    return;
  }
  for (int u = tid; u < s.n * a.R; u += kFwThreads) {
    const int r = u / a.R, j = u % a.R;
    const float* part = a.part + (int64_t)(i + r) * a.R + j;
    float sum = part[0];
    for (int k = 1; k < a.slices; ++k) sum += part[(int64_t)k * a.rows * a.R];
    mid[r][j] = sum;
    if (a.mid && blockIdx.y == 0) a.mid[(int64_t)(i + r) * a.R + j] = sum;
  }
  int row[kFwRows];
  uint32_t was[kFwRows];
#pragma unroll
  for (int r = 0; r < kFwRows; ++r) {
    row[r] = r < s.n && q < a.Q ? row_of(a.order, a.rows, i + r, a.status) : -1;
    was[r] = row[r] >= 0 && base ? *reinterpret_cast<const uint32_t*>(base + row[r] * a.base_ld + q) : 0u;
  }
  const float scale = a.scale ? a.scale[s.l] : 1.0f;
  __syncthreads();
  if (q >= a.Q) return;
  const uint16_t* f = static_cast<const uint16_t*>(a.s) + s.l * a.s_l + q * a.s_r;
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

// mid_wanted: a.mid is the caller's; the partial sums lie in a.part in any case.
cudaError_t launch_adapter_few(AdapterArgs& a, bool mid_wanted, cudaStream_t st) {
  const int steps = (a.P + kFwStep - 1) / kFwStep;
  a.slices = min((steps + 3) / 4, a.slices);
  if (a.slices < 1) a.slices = 1;
  if (!a.out) a.slices = 1;
  if (a.slices == 1 && mid_wanted) a.part = a.mid;
  if (a.slices == 1 || !mid_wanted) a.mid = nullptr;
  const bool bf = a.type == kBf16;
  const int mt = a.R <= 16 ? 1 : 2;
  const dim3 grid(a.rows, a.slices, (a.R + 16 * mt - 1) / (16 * mt));
  cudaError_t rc;
  if (mt == 1)
    rc = bf ? launch_dependent(adapter_few_mid_kernel<kBf16, 1>, grid, dim3(kFwThreads), 0, st, a)
            : launch_dependent(adapter_few_mid_kernel<kFp16, 1>, grid, dim3(kFwThreads), 0, st, a);
  else
    rc = bf ? launch_dependent(adapter_few_mid_kernel<kBf16, 2>, grid, dim3(kFwThreads), 0, st, a)
            : launch_dependent(adapter_few_mid_kernel<kFp16, 2>, grid, dim3(kFwThreads), 0, st, a);
  if (rc != cudaSuccess || !a.out) return rc;
  const dim3 cols(a.rows, (a.Q + kFwCols - 1) / kFwCols);
  return bf ? launch_dependent(adapter_few_out_kernel<kBf16>, cols, dim3(kFwThreads), 0, st, a)
            : launch_dependent(adapter_few_out_kernel<kFp16>, cols, dim3(kFwThreads), 0, st, a);
}

}  // namespace moe
