// decode_q8.cu — the forms of pa_decode_q8 (decode_q8.cuh), one translation unit each.
#include "pa_launch.h"

namespace pa {

int launch_decode_q8_e4m3_d64_bf16(const DecodeQ8Args& a, const DeviceInfo& info, cudaStream_t stream);
int launch_decode_q8_e4m3_d64_f16(const DecodeQ8Args& a, const DeviceInfo& info, cudaStream_t stream);
int launch_decode_q8_e4m3_d128_bf16(const DecodeQ8Args& a, const DeviceInfo& info, cudaStream_t stream);
int launch_decode_q8_e4m3_d128_f16(const DecodeQ8Args& a, const DeviceInfo& info, cudaStream_t stream);
int launch_decode_q8_int8_d64_bf16(const DecodeQ8Args& a, const DeviceInfo& info, cudaStream_t stream);
int launch_decode_q8_int8_d64_f16(const DecodeQ8Args& a, const DeviceInfo& info, cudaStream_t stream);
int launch_decode_q8_int8_d128_bf16(const DecodeQ8Args& a, const DeviceInfo& info, cudaStream_t stream);
int launch_decode_q8_int8_d128_f16(const DecodeQ8Args& a, const DeviceInfo& info, cudaStream_t stream);

int launch_decode_q8(const DecodeQ8Args& a, int fmt, const DeviceInfo& info, cudaStream_t stream) {
  if (fmt == PA_Q8_E4M3) {
    if (a.head_dim == 128)
      return a.f16 ? launch_decode_q8_e4m3_d128_f16(a, info, stream)
                   : launch_decode_q8_e4m3_d128_bf16(a, info, stream);
    return a.f16 ? launch_decode_q8_e4m3_d64_f16(a, info, stream)
                 : launch_decode_q8_e4m3_d64_bf16(a, info, stream);
  }
  if (a.head_dim == 128)
    return a.f16 ? launch_decode_q8_int8_d128_f16(a, info, stream)
                 : launch_decode_q8_int8_d128_bf16(a, info, stream);
  return a.f16 ? launch_decode_q8_int8_d64_f16(a, info, stream)
               : launch_decode_q8_int8_d64_bf16(a, info, stream);
}

}  // namespace pa
