// shared_decode_d64_f16.cu — pa_decode_shared (shared_decode.cuh) at head_dim 64 with IEEE fp16
// elements, in its own translation unit so the variants compile in parallel.
#include "shared_decode.cuh"

namespace pa {

int launch_shared_d64_f16(const DecodeSharedArgs& a, const DeviceInfo& info,
                         cudaStream_t stream) {
  return dispatch_shared<64, true>(a, info, stream);
}

}  // namespace pa
