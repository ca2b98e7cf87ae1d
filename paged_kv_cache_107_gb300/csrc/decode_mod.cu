// decode_mod.cu — pa_decode_mod on the tensor-core decode (decode_tc.cuh) at head_dim 128:
// every group size, bf16 or IEEE fp16 elements. head_dim 64 is in decode_mod_d64.cu.
#include "decode_tc.cuh"

namespace pa {

int launch_decode_mod(const DecodeModArgs& a, const DeviceInfo& info, cudaStream_t stream) {
  if (a.head_dim == 64) return launch_decode_mod_d64(a, info, stream);
  if (a.head_dim != 128) return PA_ERR_UNSUPPORTED;
  return a.f16 ? dispatch_slab_tc<false, 128, true, kTcMod>(a, info, stream)
               : dispatch_slab_tc<false, 128, false, kTcMod>(a, info, stream);
}

}  // namespace pa
