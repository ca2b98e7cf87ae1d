// prefill_form.cuh — definition of launch_prefill_form, for the translation units that
// instantiate one (head_dim, element type, form) each.
#pragma once

#include "prefill_kernel.cuh"

namespace pa {

template <int D, bool F16, int FORM>
int launch_prefill_form(const PrefillModArgs& a, const DeviceInfo& info, cudaStream_t stream,
                        const CUtensorMap& mk, const CUtensorMap& mv) {
  return dispatch_prefill<D, F16, FORM>(a, info, stream, mk, mv);
}

}  // namespace pa
