// What the grouped and block-scaled products share: the arguments of a product,
// the rows of a group and the element conversions.
#pragma once

#include <cuda_fp8.h>

#include "../../include/moe_products.h"
#include "common.cuh"

namespace moe {

// The operand type of a product (fp8 only as the E4M3 operands of the scaled product).
enum ProdType : int { kBf16 = MOE_BF16, kFp16 = MOE_FP16, kFp32 = MOE_FP32, kE4m3 = 3 };

// The three products of a bank W[e] (N x K).
enum ProdMode : int {
  kProdFwd = 0,  // out[r, n] = sum_k rows[r, k] W[e][n, k]
  kProdDx = 1,   // out[r, k] = sum_n rows[r, n] W[e][n, k]
  kProdDw = 2,   // out[e][n, k] = sum_r rows[r, n] x[r, k]
};

struct ProdArgs {
  const void* a;            // rows: x (forward, fp8), dy (both gradients)
  int64_t a_ld;
  const void* w;            // the bank; dW: x
  int64_t w_se, w_ld;       // dW: w_ld is x's row stride
  const float* xs;          // fp8: scales of the rows and of the bank
  int64_t xs_m, xs_g;
  const float* ws;
  int64_t ws_e, ws_n, ws_k;
  const int32_t* offsets;   // NULL: one group of all rows
  int E, rows, N, K;
  int in_type, out_type;
  int accumulate;
  void* out;
  int64_t out_se, out_ld;
  unsigned* status;         // workspace
  uint8_t* scratch;
};

// Rows [r0, r1) of group e, inside [0, rows] whatever the offsets hold.
__device__ __forceinline__ void group_rows(const ProdArgs& g, int e, int& r0, int& r1) {
  if (!g.offsets) {
    r0 = 0;
    r1 = g.rows;
    return;
  }
  r0 = min(max(__ldg(g.offsets + e), 0), g.rows);
  r1 = max(r0, min(max(__ldg(g.offsets + e + 1), 0), g.rows));
}
// Offsets of group e that break the rule (reported, never followed).
__device__ __forceinline__ bool group_bad(const ProdArgs& g, int e) {
  if (!g.offsets) return false;
  const int a = __ldg(g.offsets + e), b = __ldg(g.offsets + e + 1);
  return a < 0 || b < a || b > g.rows;
}

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int type) {
  if (type == kBf16) return bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
  if (type == kFp16) return __half2float(__ushort_as_half(static_cast<const uint16_t*>(p)[i]));
  if (type == kE4m3) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(p)[i], __NV_E4M3);  // exact
    return __half2float(*reinterpret_cast<const __half*>(&h));
  }
  return static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store_elem(void* p, int64_t i, int type, float v) {
  if (type == kBf16) static_cast<uint16_t*>(p)[i] = float_to_bf16_bits(v);
  else if (type == kFp16) static_cast<uint16_t*>(p)[i] = __half_as_ushort(__float2half_rn(v));
  else static_cast<float*>(p)[i] = v;
}

int prod_sm_count();  // of the current device; 0 on an error

cudaError_t launch_products_any(const ProdArgs& g, int mode, cudaStream_t st);

}  // namespace moe
