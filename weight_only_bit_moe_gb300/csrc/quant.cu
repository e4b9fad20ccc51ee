// FP8 quantisation of activation rows in blocks of 1 x 128 (moe_products.h):
//   v = x[row]  or  silu(gate) * up,   s = max(max |v| / 448, 2^-126),
//   q = e4m3_rn(v * (1 / s)).
// One warp per block of 128 columns, four columns per lane, one pass: the
// values stay in registers between the maximum and the rounding.
#include "products.cuh"

namespace moe {

constexpr int kQuThreads = 256;

struct QuantArgs {
  const void* x;
  int64_t x_ld;
  int x_rows;
  const int32_t* row_index;
  int rows, K, type;
  uint8_t* q;
  int64_t q_ld;
  float* scale;
  int64_t s_m, s_g;
};

template <bool GATED>
__global__ void __launch_bounds__(kQuThreads) quant_block_kernel(const __grid_constant__ QuantArgs a) {
  const int lane = threadIdx.x & 31;
  const int blocks = (a.K + 127) / 128;
  const int64_t total = (int64_t)a.rows * blocks;
  const int64_t step = (int64_t)gridDim.x * (kQuThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kQuThreads / 32) + (threadIdx.x >> 5); u < total; u += step) {
    const int row = (int)(u / blocks), b = (int)(u % blocks);
    const int src = a.row_index ? a.row_index[row] : row;
    const bool live = (unsigned)src < (unsigned)a.x_rows;
    float v[4], top = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = b * 128 + 4 * lane + i;
      v[i] = 0.0f;
      if (live && c < a.K) {
        const int64_t at = (int64_t)src * a.x_ld + c;
        v[i] = load_elem(a.x, at, a.type);
        if (GATED) v[i] = __fmul_rn(__fdiv_rn(v[i], __fadd_rn(1.0f, expf(-v[i]))), load_elem(a.x, at + a.K, a.type));
      }
      top = fmax_nan(top, fabsf(v[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float s = fmax_nan(__fdiv_rn(top, 448.0f), 1.17549435e-38f), r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = b * 128 + 4 * lane + i;
      if (c < a.K)
        a.q[(int64_t)row * a.q_ld + c] = __nv_cvt_float_to_fp8(__fmul_rn(v[i], r), __NV_SATFINITE, __NV_E4M3);
    }
    if (lane == 0) a.scale[row * a.s_m + b * a.s_g] = s;
  }
}

}  // namespace moe

using namespace moe;

extern "C" int moe_quant_fp8_block(int dtype, const void* x, int64_t x_stride, int x_rows, const int32_t* row_index,
                                   int rows, int K, int gated, void* q, int64_t q_stride, float* scale,
                                   int64_t scale_stride_m, int64_t scale_stride_g, void* stream) {
  if ((dtype != MOE_BF16 && dtype != MOE_FP16) || x_rows < 0 || rows < 0 || K < 1 || K > (1 << 30) || gated < 0 || gated > 1)
    return MOE_ERR_INVALID;
  if (x_stride < (int64_t)K * (gated ? 2 : 1) || q_stride < K || (!row_index && rows != x_rows)) return MOE_ERR_INVALID;
  if (rows == 0) return MOE_OK;
  if ((!x && x_rows > 0) || !q || !scale || (reinterpret_cast<uintptr_t>(x) & 1)) return MOE_ERR_INVALID;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return MOE_ERR_CUDA;
  QuantArgs a{x, x_stride, x_rows, row_index, rows, K, dtype, static_cast<uint8_t*>(q), q_stride, scale,
              scale_stride_m, scale_stride_g};
  const int64_t blocks = (int64_t)rows * ((K + 127) / 128);
  const int64_t want = (blocks + kQuThreads / 32 - 1) / (kQuThreads / 32);
  const int ctas = (int)(want < sms * 8 ? want : sms * 8);
  if (gated) quant_block_kernel<true><<<ctas, kQuThreads, 0, (cudaStream_t)stream>>>(a);
  else quant_block_kernel<false><<<ctas, kQuThreads, 0, (cudaStream_t)stream>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
