// prefix_d128.cu — the prefix kernel of pa_decode_shared (prefix_kernel.cuh) at head_dim 128.
#include "prefix_kernel.cuh"

namespace pa {

int launch_prefix_d128(const DecodeSharedArgs& a, const DeviceInfo& info, cudaStream_t stream) {
  return a.f16 ? launch_prefix_t<128, true>(a, info, stream)
               : launch_prefix_t<128, false>(a, info, stream);
}

}  // namespace pa
