// Entry points of moe_products.h: argument rules and the choice of the kernel.
#include <new>

#include "products_tc.cuh"

using namespace moe;

namespace moe {

constexpr int kMaxGroups = 1024;
constexpr int kMaxRows = 0x7FFFFFFF - 1024;  // row numbers may run past the last one by a tile
// gridDim.y of the plain kernel counts 64-column tiles
constexpr int kMaxDim = 65535 * 64;

static int check_products(const ProdArgs& g, const void* workspace, int64_t workspace_bytes) {
  if (g.E < 1 || g.E > kMaxGroups || g.rows < 0 || g.rows > kMaxRows || g.N < 1 || g.K < 1 || g.N > kMaxDim || g.K > kMaxDim)
    return MOE_ERR_INVALID;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)) return MOE_ERR_INVALID;
  if (workspace_bytes < MOE_PRODUCTS_WORKSPACE_BYTES) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

// Every pointer on a boundary of its element.
static bool on_elements(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

static int run(const ProdArgs& g, int mode, void* stream) {
  bool done = false;
  const cudaError_t rc = g.in_type == kE4m3 ? launch_fp8_tc(g, (cudaStream_t)stream, &done)
                                            : launch_grouped_tc(g, mode, (cudaStream_t)stream, &done);
  if (rc != cudaSuccess) return MOE_ERR_CUDA;
  if (done) return MOE_OK;
  return launch_products_any(g, mode, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// 256 bytes of status, the scratch's counters, its partial tiles.
static void set_workspace(ProdArgs& g, void* workspace) {
  static_assert(256 + kProdCounterBytes <= MOE_PRODUCTS_WORKSPACE_HEAD_BYTES, "counters outside the zeroed part");
  static_assert(256 + kProdCounterBytes + (int64_t)kProdPartials * 128 * 256 * 4 <= MOE_PRODUCTS_WORKSPACE_BYTES,
                "partial tiles outside the workspace");
  g.status = static_cast<unsigned*>(workspace);
  g.scratch = static_cast<uint8_t*>(workspace) + 256;
}

}  // namespace moe

extern "C" int moe_grouped_mm(int dtype, const void* x, int64_t x_stride, const void* w, int64_t w_stride_e,
                              int64_t w_stride_n, const int32_t* offsets, int num_experts, int rows, int N, int K,
                              void* out, int64_t out_stride, void* workspace, int64_t workspace_bytes,
                              void* stream) {
  ProdArgs g{};
  g.E = num_experts, g.rows = rows, g.N = N, g.K = K;
  const int rc = check_products(g, workspace, workspace_bytes);
  if (rc != MOE_OK) return rc;
  if ((dtype != MOE_BF16 && dtype != MOE_FP16) || x_stride < K || w_stride_n < K || out_stride < N || w_stride_e < 0)
    return MOE_ERR_INVALID;
  if (rows == 0) return MOE_OK;
  if (!x || !w || !offsets || !out || !on_elements(x, 2) || !on_elements(w, 2) || !on_elements(out, 2))
    return MOE_ERR_INVALID;
  g.a = x, g.a_ld = x_stride, g.w = w, g.w_se = w_stride_e, g.w_ld = w_stride_n;
  g.offsets = offsets, g.in_type = g.out_type = dtype, g.out = out, g.out_ld = out_stride;
  set_workspace(g, workspace);
  return run(g, kProdFwd, stream);
}

extern "C" int moe_grouped_mm_dx(int dtype, const void* dy, int64_t dy_stride, const void* w, int64_t w_stride_e,
                                 int64_t w_stride_n, const int32_t* offsets, int num_experts, int rows, int N, int K,
                                 void* dx, int64_t dx_stride, void* workspace, int64_t workspace_bytes,
                                 void* stream) {
  ProdArgs g{};
  g.E = num_experts, g.rows = rows, g.N = N, g.K = K;
  const int rc = check_products(g, workspace, workspace_bytes);
  if (rc != MOE_OK) return rc;
  if ((dtype != MOE_BF16 && dtype != MOE_FP16) || dy_stride < N || w_stride_n < K || dx_stride < K || w_stride_e < 0)
    return MOE_ERR_INVALID;
  if (rows == 0) return MOE_OK;
  if (!dy || !w || !offsets || !dx || !on_elements(dy, 2) || !on_elements(w, 2) || !on_elements(dx, 2))
    return MOE_ERR_INVALID;
  g.a = dy, g.a_ld = dy_stride, g.w = w, g.w_se = w_stride_e, g.w_ld = w_stride_n;
  g.offsets = offsets, g.in_type = g.out_type = dtype, g.out = dx, g.out_ld = dx_stride;
  set_workspace(g, workspace);
  return run(g, kProdDx, stream);
}

extern "C" int moe_grouped_mm_dw(int dtype, const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                 const int32_t* offsets, int num_experts, int rows, int N, int K, int dw_dtype,
                                 int accumulate, void* dw, int64_t dw_stride_e, int64_t dw_stride_n,
                                 void* workspace, int64_t workspace_bytes, void* stream) {
  ProdArgs g{};
  g.E = num_experts, g.rows = rows, g.N = N, g.K = K;
  const int rc = check_products(g, workspace, workspace_bytes);
  if (rc != MOE_OK) return rc;
  if ((dtype != MOE_BF16 && dtype != MOE_FP16) || dy_stride < N || x_stride < K || dw_stride_n < K) return MOE_ERR_INVALID;
  if (num_experts > 1 && dw_stride_e < (N - 1) * dw_stride_n + K) return MOE_ERR_INVALID;  // experts would overlap
  if ((dw_dtype != dtype && dw_dtype != MOE_FP32) || accumulate < 0 || accumulate > 1) return MOE_ERR_INVALID;
  if (accumulate && dw_dtype != MOE_FP32) return MOE_ERR_INVALID;
  if (!offsets || !dw || !on_elements(dw, dw_dtype == MOE_FP32 ? 4 : 2)) return MOE_ERR_INVALID;
  if (rows > 0 && (!dy || !x || !on_elements(dy, 2) || !on_elements(x, 2))) return MOE_ERR_INVALID;
  g.a = dy, g.a_ld = dy_stride, g.w = x, g.w_ld = x_stride;
  g.offsets = offsets, g.in_type = dtype, g.out_type = dw_dtype, g.accumulate = accumulate;
  g.out = dw, g.out_se = dw_stride_e, g.out_ld = dw_stride_n;
  set_workspace(g, workspace);
  return run(g, kProdDw, stream);
}

extern "C" int moe_gemm_fp8_block(const void* x, int64_t x_stride, const float* x_scale, int64_t xs_stride_m,
                                  int64_t xs_stride_g, const void* w, int64_t w_stride_e, int64_t w_stride_n,
                                  const float* w_scale, int64_t ws_stride_e, int64_t ws_stride_n,
                                  int64_t ws_stride_k, const int32_t* offsets, int num_experts, int rows, int N,
                                  int K, int out_dtype, void* out, int64_t out_stride, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
  ProdArgs g{};
  g.E = num_experts, g.rows = rows, g.N = N, g.K = K;
  const int rc = check_products(g, workspace, workspace_bytes);
  if (rc != MOE_OK) return rc;
  if (out_dtype < MOE_BF16 || out_dtype > MOE_FP32 || x_stride < K || w_stride_n < K || out_stride < N || w_stride_e < 0)
    return MOE_ERR_INVALID;
  if (!offsets && num_experts != 1) return MOE_ERR_INVALID;
  if (rows == 0) return MOE_OK;
  if (!x || !x_scale || !w || !w_scale || !out || !on_elements(out, out_dtype == MOE_FP32 ? 4 : 2))
    return MOE_ERR_INVALID;
  g.a = x, g.a_ld = x_stride, g.xs = x_scale, g.xs_m = xs_stride_m, g.xs_g = xs_stride_g;
  g.w = w, g.w_se = w_stride_e, g.w_ld = w_stride_n;
  g.ws = w_scale, g.ws_e = ws_stride_e, g.ws_n = ws_stride_n, g.ws_k = ws_stride_k;
  g.offsets = offsets, g.in_type = kE4m3, g.out_type = out_dtype, g.out = out, g.out_ld = out_stride;
  set_workspace(g, workspace);
  return run(g, kProdFwd, stream);
}

// ---------------------------------------------------------------- captured calls
namespace moe {

// The capture's number (0: none) and graph.
static bool capture_of(void* stream, unsigned long long* id, cudaGraph_t* graph) {
  cudaStreamCaptureStatus status;
  if (cudaStreamGetCaptureInfo((cudaStream_t)stream, &status, id, graph) != cudaSuccess) return false;
  if (status == cudaStreamCaptureStatusInvalidated) return false;
  if (status == cudaStreamCaptureStatusNone) *id = 0;
  return true;
}

}  // namespace moe

extern "C" int moe_capture_id(void* stream, uint64_t* id) {
  unsigned long long n = 0;
  if (!id) return MOE_ERR_INVALID;
  if (!capture_of(stream, &n, nullptr)) return MOE_ERR_CUDA;
  *id = n;
  return MOE_OK;
}

extern "C" int moe_capture_mode(int* mode) {
  if (!mode || *mode < 0 || *mode > 2) return MOE_ERR_INVALID;
  static_assert(cudaStreamCaptureModeRelaxed == 2, "the header names this value");
  cudaStreamCaptureMode m = (cudaStreamCaptureMode)*mode;
  if (cudaThreadExchangeStreamCaptureMode(&m) != cudaSuccess) return MOE_ERR_CUDA;
  *mode = (int)m;
  return MOE_OK;
}

extern "C" int moe_capture_watch(void* stream, const int32_t** gone) {
  if (!gone) return MOE_ERR_INVALID;
  unsigned long long id = 0;
  cudaGraph_t graph = nullptr;
  if (!capture_of(stream, &id, &graph)) return MOE_ERR_CUDA;
  if (id == 0) return MOE_ERR_INVALID;
  int32_t* word = new (std::nothrow) int32_t(0);
  if (!word) return MOE_ERR_CUDA;
  cudaUserObject_t object;
  const cudaHostFn_t set = [](void* p) { __atomic_store_n(static_cast<int32_t*>(p), 1, __ATOMIC_RELEASE); };
  if (cudaUserObjectCreate(&object, word, set, 1, cudaUserObjectNoDestructorSync) != cudaSuccess) {
    delete word;
    return MOE_ERR_CUDA;
  }
  if (cudaGraphRetainUserObject(graph, object, 1, cudaGraphUserObjectMove) != cudaSuccess) {
    cudaUserObjectRelease(object, 1);  // (sets the word some time from now: it stays)
    return MOE_ERR_CUDA;
  }
  *gone = word;
  return MOE_OK;
}
