// decode_shared.cu — pa_decode_shared: the prefix kernel (prefix_d*.cu), the tensor-core decode
// of what lies behind the prefixes (decode_tc.cuh, kTcShared; head_dim 128 here, 64 in
// decode_shared_d64.cu) and the join (shared_join.cu), each a programmatic dependent of the
// one before.
#include "decode_tc.cuh"

namespace pa {

int launch_decode_shared(const DecodeSharedArgs& a, const DeviceInfo& info, cudaStream_t stream) {
  if (a.head_dim != 64 && a.head_dim != 128) return PA_ERR_UNSUPPORTED;
  const int rc = a.head_dim == 64 ? launch_prefix_d64(a, info, stream)
                                  : launch_prefix_d128(a, info, stream);
  if (rc != PA_OK) return rc;
  const int rc2 = a.head_dim == 64 ? launch_decode_shared_rest_d64(a, info, stream)
                  : a.f16 ? dispatch_slab_tc<false, 128, true, kTcShared>(a, info, stream)
                          : dispatch_slab_tc<false, 128, false, kTcShared>(a, info, stream);
  return rc2 != PA_OK ? rc2 : launch_shared_join(a, info, stream);
}

}  // namespace pa
