#include "adapters_out.cuh"

namespace moe {

cudaError_t launch_adapter_out_fwd(const AdapterArgs& a, int sms, cudaStream_t st) {
  return a.type == kBf16 ? launch_out<kBf16, true>(a, sms, st) : launch_out<kFp16, true>(a, sms, st);
}

}  // namespace moe
