// prefill_cap_d64_bf16.cu — pa_prefill_mod on the prefill kernel (prefill_kernel.cuh, kFormCap)
// for head_dim 64 with bf16 elements, in its own translation unit so the variants
// compile in parallel.
#include "prefill_form.cuh"

namespace pa {

template int launch_prefill_form<64, false, kFormCap>(const PrefillModArgs&, const DeviceInfo&,
                                                  cudaStream_t, const CUtensorMap&,
                                                  const CUtensorMap&);

}  // namespace pa
