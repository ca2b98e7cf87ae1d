// decode_q8_e4m3_d128_bf16.cu — pa_decode_q8 (decode_q8.cuh) with e4m3 codes at head_dim 128, bf16 queries.
#include "decode_q8.cuh"

namespace pa {

int launch_decode_q8_e4m3_d128_bf16(const DecodeQ8Args& a, const DeviceInfo& info, cudaStream_t stream) {
  return dispatch_slab_q8<128, PA_Q8_E4M3, false>(a, info, stream);
}

}  // namespace pa
