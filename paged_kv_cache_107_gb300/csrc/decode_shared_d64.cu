// decode_shared_d64.cu — the decode behind shared prefixes at head_dim 64 (decode_shared.cu).
#include "decode_tc.cuh"

namespace pa {

int launch_decode_shared_rest_d64(const DecodeSharedArgs& a, const DeviceInfo& info,
                                  cudaStream_t stream) {
  return a.f16 ? dispatch_slab_tc<false, 64, true, kTcShared>(a, info, stream)
               : dispatch_slab_tc<false, 64, false, kTcShared>(a, info, stream);
}

}  // namespace pa
