// decode_mod_d64.cu — pa_decode_mod at head_dim 64 (decode_mod.cu), in its own translation
// unit so the variants compile in parallel.
#include "decode_tc.cuh"

namespace pa {

int launch_decode_mod_d64(const DecodeModArgs& a, const DeviceInfo& info, cudaStream_t stream) {
  return a.f16 ? dispatch_slab_tc<false, 64, true, kTcMod>(a, info, stream)
               : dispatch_slab_tc<false, 64, false, kTcMod>(a, info, stream);
}

}  // namespace pa
