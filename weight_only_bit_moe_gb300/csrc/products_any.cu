// The products of moe_products.h for any size, stride and alignment.
//
//   forward, FP8:  out[r, n]    = sum_k rows[r, k] W[e][n, k]
//   dx:            out[r, k]    = sum_n rows[r, n] W[e][n, k]
//   dW:            out[e][n, k] = sum_{r in e} dy[r, n] x[r, k]
//
// A 64 x 64 output tile per CTA, 4 x 4 sums per thread in fp32, operands
// converted to fp32 on their way into shared memory, 16 terms of the sum at a
// time.  FP8: each block's sum is multiplied by xs ws, as on the tensor cores; the
// elements times their scales could leave fp32's range where the product of the
// scales does not.  Plain loads of single elements: this
// kernel takes the operands that TMA cannot address, and is bound by its fp32
// multiply-adds and these loads.
#include "products.cuh"

namespace moe {

constexpr int kAnyTile = 64, kAnyK = 16, kAnyThreads = 256;

struct AnyTiles {
  float a[kAnyK][kAnyTile + 4];
  float b[kAnyK][kAnyTile + 4];
};

// One value of the two operands of the sum's term t: A(i, t), B(j, t).
template <int MODE>
__device__ __forceinline__ float any_a(const ProdArgs& g, int64_t i, int t) {
  if (MODE == kProdDw) return load_elem(g.a, (int64_t)t * g.a_ld + i, g.in_type);
  return load_elem(g.a, i * g.a_ld + t, g.in_type);
}
template <int MODE>
__device__ __forceinline__ float any_b(const ProdArgs& g, int e, int64_t j, int t) {
  if (MODE == kProdDw) return load_elem(g.w, (int64_t)t * g.w_ld + j, g.in_type);
  if (MODE == kProdDx) return load_elem(g.w, e * g.w_se + (int64_t)t * g.w_ld + j, g.in_type);
  return load_elem(g.w, e * g.w_se + j * g.w_ld + t, g.in_type);
}

// acc[y][x] += sum over t in [t0, t1) of A(i0 + 4 ty + y, t) B(j0 + 4 tx + x, t); rows at or
// past i1, columns at or past j1 count as zeros.
template <int MODE>
__device__ void any_tile(const ProdArgs& g, int e, int i0, int i1, int j0, int j1, int t0, int t1, AnyTiles& s,
                         float (&acc)[4][4]) {
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  for (int t = t0; t < t1; t += kAnyK) {
    __syncthreads();
    for (int u = tid; u < kAnyTile * kAnyK; u += kAnyThreads) {
      // consecutive threads read consecutive addresses of each operand
      const int ia = MODE == kProdDw ? u % kAnyTile : u / kAnyK, ta = MODE == kProdDw ? u / kAnyTile : u % kAnyK;
      s.a[ta][ia] = (i0 + ia < i1 && t + ta < t1) ? any_a<MODE>(g, i0 + ia, t + ta) : 0.0f;
      const int jb = MODE == kProdFwd ? u / kAnyK : u % kAnyTile, tb = MODE == kProdFwd ? u % kAnyK : u / kAnyTile;
      s.b[tb][jb] = (j0 + jb < j1 && t + tb < t1) ? any_b<MODE>(g, e, j0 + jb, t + tb) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kAnyK; ++k)
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[y][x] = fmaf(s.a[k][4 * ty + y], s.b[k][4 * tx + x], acc[y][x]);
  }
}

// Products by row: a CTA owns 64 rows whatever their groups and runs each group
// that has some of them.
template <int MODE>
__global__ void __launch_bounds__(kAnyThreads) products_any_rows_kernel(const __grid_constant__ ProdArgs g) {
  __shared__ AnyTiles s;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int cols = MODE == kProdDx ? g.K : g.N, terms = MODE == kProdDx ? g.N : g.K;
  const int j0 = blockIdx.y * kAnyTile;
  const int row0 = blockIdx.x * kAnyTile, row1 = min(row0 + kAnyTile, g.rows);
  for (int e = 0; e < g.E; ++e) {
    int r0, r1;
    group_rows(g, e, r0, r1);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && group_bad(g, e)) atomicOr(g.status, kStatusRouting);
    const int i0 = max(row0, r0), i1 = min(row1, r1);
    if (i0 >= i1) continue;
    float acc[4][4] = {};
    if (MODE == kProdFwd && g.in_type == kE4m3) {
      for (int b = 0; 128 * b < terms; ++b) {
        float part[4][4] = {};
        any_tile<MODE>(g, e, i0, i1, j0, cols, 128 * b, min(128 * b + 128, terms), s, part);
        const float ws = g.ws[e * g.ws_e + (int64_t)(j0 >> 7) * g.ws_n + (int64_t)b * g.ws_k];  // (64 columns: one block)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int i = i0 + 4 * ty + y;
          const float scale = i < i1 ? g.xs[i * g.xs_m + (int64_t)b * g.xs_g] * ws : 0.0f;
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[y][x] = fmaf(part[y][x], scale, acc[y][x]);
        }
      }
    } else {
      any_tile<MODE>(g, e, i0, i1, j0, cols, 0, terms, s, acc);
    }
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = i0 + 4 * ty + y, j = j0 + 4 * tx + x;
        if (i < i1 && j < cols) store_elem(g.out, (int64_t)i * g.out_ld + j, g.out_type, acc[y][x]);
      }
  }
}

__global__ void __launch_bounds__(kAnyThreads) products_any_dw_kernel(const __grid_constant__ ProdArgs g) {
  __shared__ AnyTiles s;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int e = blockIdx.z, i0 = blockIdx.y * kAnyTile, j0 = blockIdx.x * kAnyTile;
  int r0, r1;
  group_rows(g, e, r0, r1);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && group_bad(g, e)) atomicOr(g.status, kStatusRouting);
  if (g.accumulate && r0 == r1) return;  // nothing is added: the expert's part keeps its bits
  float acc[4][4] = {};
  any_tile<kProdDw>(g, e, i0, g.N, j0, g.K, r0, r1, s, acc);
#pragma unroll
  for (int y = 0; y < 4; ++y)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int i = i0 + 4 * ty + y, j = j0 + 4 * tx + x;
      if (i >= g.N || j >= g.K) continue;
      const int64_t at = e * g.out_se + (int64_t)i * g.out_ld + j;
      float v = acc[y][x];
      if (g.accumulate) v += static_cast<const float*>(g.out)[at];
      store_elem(g.out, at, g.out_type, v);
    }
}

cudaError_t launch_products_any(const ProdArgs& g, int mode, cudaStream_t st) {
  auto tiles = [](int n) { return (unsigned)((n + kAnyTile - 1) / kAnyTile); };
  if (mode == kProdDw) {
    products_any_dw_kernel<<<dim3(tiles(g.K), tiles(g.N), g.E), kAnyThreads, 0, st>>>(g);
  } else if (mode == kProdDx) {
    products_any_rows_kernel<kProdDx><<<dim3(tiles(g.rows), tiles(g.K)), kAnyThreads, 0, st>>>(g);
  } else {
    products_any_rows_kernel<kProdFwd><<<dim3(tiles(g.rows), tiles(g.N)), kAnyThreads, 0, st>>>(g);
  }
  return cudaPeekAtLastError();
}

}  // namespace moe
