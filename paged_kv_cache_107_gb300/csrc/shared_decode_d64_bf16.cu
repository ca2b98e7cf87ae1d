// shared_decode_d64_bf16.cu — pa_decode_shared (shared_decode.cuh) at head_dim 64 with bf16
// elements, in its own translation unit so the variants compile in parallel.
#include "shared_decode.cuh"

namespace pa {

int launch_shared_d64_bf16(const DecodeSharedArgs& a, const DeviceInfo& info,
                         cudaStream_t stream) {
  return dispatch_shared<64, false>(a, info, stream);
}

}  // namespace pa
