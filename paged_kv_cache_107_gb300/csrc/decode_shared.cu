// decode_shared.cu — pa_decode_shared: the prefix kernel (prefix_d*.cu), then the tensor-core
// decode of what lies behind the prefixes (decode_tc.cuh, kTcShared), launched as its
// programmatic dependent; head_dim 128 here, 64 in decode_shared_d64.cu.
#include "decode_tc.cuh"

namespace pa {

int launch_decode_shared(const DecodeSharedArgs& a, const DeviceInfo& info, cudaStream_t stream) {
  if (a.head_dim != 64 && a.head_dim != 128) return PA_ERR_UNSUPPORTED;
  const int rc = a.head_dim == 64 ? launch_prefix_d64(a, info, stream)
                                  : launch_prefix_d128(a, info, stream);
  if (rc != PA_OK) return rc;
  if (a.head_dim == 64) return launch_decode_shared_rest_d64(a, info, stream);
  return a.f16 ? dispatch_slab_tc<false, 128, true, kTcShared>(a, info, stream)
               : dispatch_slab_tc<false, 128, false, kTcShared>(a, info, stream);
}

}  // namespace pa
