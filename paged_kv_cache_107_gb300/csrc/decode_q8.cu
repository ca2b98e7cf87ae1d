// decode_q8.cu — pa_decode_q8 (decode_q8.cuh) with e4m3 codes at head_dim 128; the other forms
// are in decode_q8_*.cu.
#include "decode_q8.cuh"

namespace pa {

int launch_decode_q8_e4m3_d64(const DecodeQ8Args& a, const DeviceInfo& info, cudaStream_t stream);
int launch_decode_q8_int8_d128(const DecodeQ8Args& a, const DeviceInfo& info, cudaStream_t stream);
int launch_decode_q8_int8_d64(const DecodeQ8Args& a, const DeviceInfo& info, cudaStream_t stream);

int launch_decode_q8(const DecodeQ8Args& a, int fmt, const DeviceInfo& info, cudaStream_t stream) {
  if (fmt == PA_Q8_E4M3)
    return a.head_dim == 128 ? dispatch_slab_q8<128, PA_Q8_E4M3>(a, info, stream)
                             : launch_decode_q8_e4m3_d64(a, info, stream);
  return a.head_dim == 128 ? launch_decode_q8_int8_d128(a, info, stream)
                           : launch_decode_q8_int8_d64(a, info, stream);
}

}  // namespace pa
