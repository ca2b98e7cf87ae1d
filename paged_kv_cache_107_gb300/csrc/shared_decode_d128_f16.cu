// shared_decode_d128_f16.cu — pa_decode_shared (shared_decode.cuh) at head_dim 128 with IEEE fp16
// elements, in its own translation unit so the variants compile in parallel.
#include "shared_decode.cuh"

namespace pa {

int launch_shared_d128_f16(const DecodeSharedArgs& a, const DeviceInfo& info,
                         cudaStream_t stream) {
  return dispatch_shared<128, true>(a, info, stream);
}

}  // namespace pa
