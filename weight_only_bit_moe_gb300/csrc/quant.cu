// FP8 quantisation of activation rows in blocks of 1 x 128 (moe_products.h):
//   v = x[row]  or  silu(gate) * up,   s = max(max |v| / 448, 2^-126),
//   q = e4m3_rn(v * (1 / s)).
// A stream: two bytes in (four when gated), one out, a scale per 128.  Sixteen
// lanes hold a block, eight values each, so every load is 16 bytes and every
// store 8; a warp takes up to 1024 columns of a row at a time with all their
// loads in flight before the first maximum.  The values stay in registers
// between the maximum and the rounding.  Operands off the 16-byte grid run a
// form of the same with single elements.
//
// Gathered rows are bound by instructions (16384 rows of 4096 from 2048: 17.5 us with
// the tokens in L2, 19.9 from memory, 201 MB moved, ALU 65 % busy; floor by memory
// 12.7): each token is quantised as often as it is gathered.  Gated rows fill no unit
// (4093 rows of 2880: 10.9 us in L2, 13.3 from memory, where ALU 36 %, FMA 47 % and
// DRAM 37 % are busy; floor 8.7): a warp's loads, arithmetic and stores follow one
// another.
#include "products_tc.cuh"

namespace moe {

constexpr int kQuThreads = 256;
constexpr int kQuWarps = kQuThreads / 32;
constexpr int kQuCtas = 5;  // resident on an SM

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

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t both(float v) { return pack2(__float_as_uint(v), __float_as_uint(v)); }

// silu(g) * u = g / (1 + exp(-g)) * u of two values, each operation rounded to
// fp32.  The quotient is one Newton step in the form that Markstein gives for
// division: r = 1 / d to within an ulp, q = g r, q + (g - q d) r with the residual
// exact in a fused multiply-add, which rounds like the quotient itself.  Both sides
// are taken times 1/4 (exact: a 16-bit g / 4 is one in fp32), so that 1 / d stays in
// the normal range for every finite d.  Where exp(-g) is infinite (g below -88.72)
// r is flushed to 0, and so is the result.
//
// A cheaper exponential as well (2^t on the special-function unit with a
// correction) took 11.4 instead of 12.6 us for 4093 rows of 2880, but moved more
// values across the boundary between two codes: 2.5e-4 relative error of the codes
// against 64 bits instead of at most 8e-5 (10 of the 11.8 million codes differ; of
// separate fp32 operations as many).
__device__ __forceinline__ void silu_mul2(float& g0, float& g1, float u0, float u1) {
  const float d0 = fmin_nan(fmaf(expf(-g0), 0.25f, 0.25f), 1.7014118e38f);
  const float d1 = fmin_nan(fmaf(expf(-g1), 0.25f, 0.25f), 1.7014118e38f);
  float r0, r1;  // -1 / d
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(-d0));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(-d1));
  const uint64_t n = mul2(pack2(__float_as_uint(g0), __float_as_uint(g1)), both(-0.25f));
  const uint64_t d = pack2(__float_as_uint(d0), __float_as_uint(d1)), r = pack2(__float_as_uint(r0), __float_as_uint(r1));
  uint64_t q = mul2(n, r), m = n;
  fma2(m, q, d);  // q d - g
  fma2(q, m, r);
  uint32_t v0, v1;
  unpack2(mul2(q, pack2(__float_as_uint(u0), __float_as_uint(u1))), v0, v1);
  g0 = __uint_as_float(v0);
  g1 = __uint_as_float(v1);
}

// Scale of a block whose largest magnitude is `top`.
__device__ __forceinline__ float block_scale(float top) { return fmax_nan(__fdiv_rn(top, 448.0f), 1.17549435e-38f); }

template <int TYPE>
__device__ __forceinline__ void widen8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (TYPE == kBf16) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The largest magnitude of each block, for a warp whose lanes 0-15 and 16-31 hold
// eight values of a block of each chunk.  Lanes trade chunks as they reduce, so a
// lane ends up with the maximum of chunk mine(lane) of its half: half the
// exchanges, and one division per lane for all chunks.
//
// Plain rows: the magnitudes' bits order like the values (NaN above infinity), so
// 16-bit integer maxima do, two chunks in one register.  Four chunks: lanes with
// bit 3 take chunks 2 and 3; bit 2 tells which of the two the lane answers for.
__device__ __forceinline__ int mine4(int lane) { return ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1); }
template <int TYPE>
__device__ __forceinline__ float block_max4(const uint4 (&in)[4], int lane) {
  uint32_t m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    const uint32_t p = max_u16x2(max_u16x2(in[i].x & kAbs, in[i].y & kAbs), max_u16x2(in[i].z & kAbs, in[i].w & kAbs));
    m[i] = max(p & 0xFFFFu, p >> 16);
  }
  const uint32_t lo = m[0] | (m[1] << 16), hi = m[2] | (m[3] << 16);
  const bool up = lane & 8;
  uint32_t v = max_u16x2(up ? hi : lo, __shfl_xor_sync(0xffffffffu, up ? lo : hi, 8));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v = max_u16x2(v, __shfl_xor_sync(0xffffffffu, v, o));
  v = lane & 4 ? v >> 16 : v & 0xFFFFu;
  return TYPE == kBf16 ? __uint_as_float(v << 16) : __half2float(__ushort_as_half((uint16_t)v));
}
// Gated rows: fp32 values, two chunks; lanes with bit 3 answer for chunk 1.
__device__ __forceinline__ int mine2(int lane) { return (lane >> 3) & 1; }
__device__ __forceinline__ float block_max2(const float (&v)[2][8], int lane) {
  float m[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m[i] = fmax_nan(m[i], fabsf(v[i][j]));
  }
  const bool up = lane & 8;
  float t = fmax_nan(up ? m[1] : m[0], __shfl_xor_sync(0xffffffffu, up ? m[0] : m[1], 8));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) t = fmax_nan(t, __shfl_xor_sync(0xffffffffu, t, o));
  return t;
}

__device__ __forceinline__ uint32_t codes4(const float (&v)[8], int i, uint64_t rr) {
  uint32_t a, b, c, d, o;
  unpack2(mul2(pack2(__float_as_uint(v[i]), __float_as_uint(v[i + 1])), rr), a, b);
  unpack2(mul2(pack2(__float_as_uint(v[i + 2]), __float_as_uint(v[i + 3])), rr), c, d);
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(o)
      : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)), "f"(__uint_as_float(d)));
  return o;
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float r) {
  const uint64_t rr = both(r);
  return make_uint2(codes4(v, 0, rr), codes4(v, 4, rr));
}

// One warp, kChunks chunks of 256 columns of one row from column c0 on: enough
// 16-byte loads in flight to stream, few enough registers for five CTAs on an SM.
// WHOLE: every lane's columns lie inside the row and the row exists.
template <bool GATED, int TYPE, bool WHOLE>
__device__ __forceinline__ void quant_unit(const QuantArgs& a, int row, int src, int c0, int lane) {
  constexpr int kChunks = GATED ? 2 : 4;
  const bool live = WHOLE || (unsigned)src < (unsigned)a.x_rows;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + (int64_t)(live ? src : 0) * a.x_ld + c0 + 8 * lane;
  const int left = WHOLE ? 256 * kChunks : a.K - c0 - 8 * lane;  // columns from this lane's first on
  uint4 in[kChunks], up[GATED ? kChunks : 1];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    if (WHOLE || (live && left > 256 * i)) {
      in[i] = __ldg(reinterpret_cast<const uint4*>(x + 256 * i));
      if (GATED) up[i] = __ldg(reinterpret_cast<const uint4*>(x + a.K + 256 * i));
    } else {
      in[i] = make_uint4(0, 0, 0, 0);
      if (GATED) up[i] = make_uint4(0, 0, 0, 0);
    }
  }
  float v[GATED ? 2 : 1][8], top;
  int mine;
  if constexpr (GATED) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float w[8];
      widen8<TYPE>(in[i], v[i]);
      widen8<TYPE>(up[i], w);
#pragma unroll
      for (int j = 0; j < 8; j += 2) silu_mul2(v[i][j], v[i][j + 1], w[j], w[j + 1]);
    }
    top = block_max2(v, lane);
    mine = mine2(lane);
  } else {
    top = block_max4<TYPE>(in, lane);
    mine = mine4(lane);
  }
  const float s = block_scale(top), r = __frcp_rn(s);
  // one lane of those that hold the block's scale stores it
  const int block = (c0 >> 7) + 2 * mine + (lane >> 4);
  if ((lane & (GATED ? 7 : 3)) == 0 && (WHOLE || 128 * block < a.K)) a.scale[row * a.s_m + block * a.s_g] = s;
  uint8_t* q = a.q + (int64_t)row * a.q_ld + c0 + 8 * lane;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    // chunk i's reciprocal from the first lane of this half that holds it
    const int from = (lane & 16) + (GATED ? 8 * i : 8 * (i >> 1) + 4 * (i & 1));
    const float ri = __shfl_sync(0xffffffffu, r, from);
    if constexpr (!GATED) widen8<TYPE>(in[i], v[0]);
    if (WHOLE || left > 256 * i) *reinterpret_cast<uint2*>(q + 256 * i) = codes8(v[GATED ? i : 0], ri);
  }
}

// A warp per unit: rows along x, the units of a row along y (no division, and the
// hardware balances the CTAs).
template <bool GATED, int TYPE>
__global__ void __launch_bounds__(kQuThreads, kQuCtas) quant_rows_kernel(const __grid_constant__ QuantArgs a) {
  constexpr int kCols = GATED ? 512 : 1024;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kQuWarps + (threadIdx.x >> 5), c0 = blockIdx.y * kCols;
  grid_dependents_launch();
  grid_dependency_wait();
  if (row >= a.rows) return;
  const int src = a.row_index ? __ldg(a.row_index + row) : row;
  if (c0 + kCols <= a.K && (unsigned)src < (unsigned)a.x_rows) quant_unit<GATED, TYPE, true>(a, row, src, c0, lane);
  else quant_unit<GATED, TYPE, false>(a, row, src, c0, lane);
}

// Any alignment: a warp per block, four columns per lane.
template <bool GATED>
__global__ void __launch_bounds__(kQuThreads) quant_any_kernel(const __grid_constant__ QuantArgs a) {
  const int lane = threadIdx.x & 31;
  const int blocks = (a.K + 127) / 128;
  const int64_t total = (int64_t)a.rows * blocks;
  const int64_t step = (int64_t)gridDim.x * kQuWarps;
  for (int64_t u = (int64_t)blockIdx.x * kQuWarps + (threadIdx.x >> 5); u < total; u += step) {
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
        if (GATED) {
          float unused = 0.0f;
          silu_mul2(v[i], unused, load_elem(a.x, at + a.K, a.type), 0.0f);
        }
      }
      top = fmax_nan(top, fabsf(v[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float s = block_scale(top), r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = b * 128 + 4 * lane + i;
      if (c < a.K)
        a.q[(int64_t)row * a.q_ld + c] = __nv_cvt_float_to_fp8(__fmul_rn(v[i], r), __NV_SATFINITE, __NV_E4M3);
    }
    if (lane == 0) a.scale[row * a.s_m + b * a.s_g] = s;
  }
}

template <bool GATED>
static cudaError_t launch_quant(const QuantArgs& a, int sms, cudaStream_t st) {
  const int cols = GATED ? 512 : 1024;  // columns a warp takes
  const int per_row = (a.K + cols - 1) / cols;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.x) & 15) | (reinterpret_cast<uintptr_t>(a.q) & 7)) == 0 &&
                    a.x_ld % 8 == 0 && a.q_ld % 8 == 0 && a.K % 8 == 0 && per_row <= 65535;
  if (wide) {
    const dim3 grid((unsigned)(((int64_t)a.rows + kQuWarps - 1) / kQuWarps), (unsigned)per_row);
    return launch_dependent(a.type == kBf16 ? quant_rows_kernel<GATED, kBf16> : quant_rows_kernel<GATED, kFp16>, grid,
                            dim3(kQuThreads), 0, st, a);
  }
  const int64_t ctas = ((int64_t)a.rows * ((a.K + 127) / 128) + kQuWarps - 1) / kQuWarps;
  quant_any_kernel<GATED><<<(int)(ctas < sms * 8 ? ctas : sms * 8), kQuThreads, 0, st>>>(a);
  return cudaPeekAtLastError();
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
  const int sms = prod_sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  const QuantArgs a{x, x_stride, x_rows, row_index, rows, K, dtype, static_cast<uint8_t*>(q), q_stride, scale,
                    scale_stride_m, scale_stride_g};
  const cudaError_t rc = gated ? launch_quant<true>(a, sms, (cudaStream_t)stream)
                               : launch_quant<false>(a, sms, (cudaStream_t)stream);
  return rc == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
