// decode_q8_int8_d64_bf16.cu — pa_decode_q8 (decode_q8.cuh) with int8 codes at head_dim 64, bf16 queries.
#include "decode_q8.cuh"

namespace pa {

int launch_decode_q8_int8_d64_bf16(const DecodeQ8Args& a, const DeviceInfo& info, cudaStream_t stream) {
  return dispatch_slab_q8<64, PA_Q8_INT8, false>(a, info, stream);
}

}  // namespace pa
