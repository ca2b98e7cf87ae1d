// prefix_d64.cu — the prefix kernel of pa_decode_shared (prefix_kernel.cuh) at head_dim 64.
#include "prefix_kernel.cuh"

namespace pa {

int launch_prefix_d64(const DecodeSharedArgs& a, const DeviceInfo& info, cudaStream_t stream) {
  return a.f16 ? launch_prefix_t<64, true>(a, info, stream)
               : launch_prefix_t<64, false>(a, info, stream);
}

}  // namespace pa
