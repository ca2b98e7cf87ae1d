// decode_mod.cu — pa_decode_mod on the tensor-core decode (decode_tc.cuh) at head_dim 128:
// every group size, bf16 or IEEE fp16 elements. head_dim 64 is in decode_mod_d64.cu.
//
// The rules act on the score accumulators: x = cap tanh(scale q.k / cap) - slope (p - t), then
// the masks. Bound by memory like the plain form, whatever the rules (where the block size
// allows TMA boxes; decode_tc.cuh gives the time where it does not): 256 sequences of 100 to
// 2,048 positions under a cap take 169 us against 168 (1.03 of the copy rate), 8 of 32k to
// 131k with slopes 327 (1.00), so the tanh is the exact one. Hidden key tiles are not walked:
// 200 sequences of 500 to 32k with a window of 1,000 take 71 us, 897 without it.
#include "decode_tc.cuh"

namespace pa {

int launch_decode_mod(const DecodeModArgs& a, const DeviceInfo& info, cudaStream_t stream) {
  if (a.head_dim == 64) return launch_decode_mod_d64(a, info, stream);
  if (a.head_dim != 128) return PA_ERR_UNSUPPORTED;
  return a.f16 ? dispatch_slab_tc<false, 128, true, kTcMod>(a, info, stream)
               : dispatch_slab_tc<false, 128, false, kTcMod>(a, info, stream);
}

}  // namespace pa
