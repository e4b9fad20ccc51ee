// What the kernels of moe_adapters.h share: the arguments and the rows of an adapter.
#pragma once

#include "../../include/moe_adapters.h"
#include "products_tc.cuh"

namespace moe {

constexpr int kAdAdapters = MOE_MAX_ADAPTERS, kAdRank = MOE_MAX_RANK;

// mid[i, j] = sum_p in[r, p] F[l](j, p), out[r, q] = base[r, q] + scale[l] sum_j mid[i, j] S[l](q, j):
// the forward product with F = A, S = B, the gradient by the rows with F = B^T, S = A^T.
struct AdapterArgs {
  const void* in;
  int64_t in_ld;
  const void* f;             // F[l](j, p) at l f_l + (FWD: j f_r + p; gradient: p f_r + j)
  int64_t f_l, f_r;
  const void* s;             // S[l](q, j) at l s_l + (FWD: q s_r + j; gradient: j s_r + q)
  int64_t s_l, s_r;
  const int32_t* offsets;
  const int32_t* order;
  const float* scale;
  int L, rows, P, Q, R, type;
  const void* base;
  int64_t base_ld;
  void* out;
  int64_t out_ld;
  float* mid;                // [rows, R]
  unsigned* status;
};

// dF[l](j, p) = scale[l] sum_i mid[i, j] in[r, p]: dA with in = x, dB with in = dy.
struct AdapterGradSide {
  const void* in;            // NULL: this side is left out
  int64_t in_ld;
  const float* mid;
  int P;
  void* out;
  int64_t out_l, out_j, out_p;  // strides
};
struct AdapterGradArgs {
  AdapterGradSide side[2];
  const int32_t* offsets;
  const int32_t* order;
  const float* scale;
  int L, rows, R, type, out_type, accumulate;
  unsigned* status;
};

// Positions [i0, i1) of adapter l, inside [0, rows] whatever the offsets hold.
__device__ __forceinline__ void adapter_rows(const int32_t* offsets, int rows, int l, int& i0, int& i1) {
  i0 = min(max(__ldg(offsets + l), 0), rows);
  i1 = max(i0, min(max(__ldg(offsets + l + 1), 0), rows));
}
__device__ __forceinline__ bool adapter_bad(const int32_t* offsets, int rows, int l) {
  const int a = __ldg(offsets + l), b = __ldg(offsets + l + 1);
  return a < 0 || b < a || b > rows;
}
// The row of position i, -1 (reported) where order leaves the rows.
__device__ __forceinline__ int row_of(const int32_t* order, int rows, int i, unsigned* status) {
  if (!order) return i;
  const int r = __ldg(order + i);
  if (r >= 0 && r < rows) return r;
  atomicOr(status, kStatusRouting);
  return -1;
}

cudaError_t launch_adapter_any(const AdapterArgs& a, bool fwd, cudaStream_t st);
cudaError_t launch_adapter_grad_any(const AdapterGradArgs& a, int side, cudaStream_t st);
cudaError_t launch_adapter_rest(const AdapterArgs& a, cudaStream_t st);

}  // namespace moe
