// rotary_store_d64_bf16.cu — pa_rotary_store and pa_rotary_store_q8 (kv_rows.cuh) at head_dim 64
// with bf16 elements.
#include "kv_rows.cuh"

namespace pa {

int launch_rotary_d64_bf16(const RowsArgs& a, int fmt, const DeviceInfo& info, cudaStream_t stream) {
  return launch_rotary_rows_t<64, false>(a, fmt, info, stream);
}

}  // namespace pa
