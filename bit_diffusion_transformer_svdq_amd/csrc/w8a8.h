// Internal to the 8-bit linear's kernels: the few-token form.
#pragma once

#include "svdq_internal.h"

namespace svdq {

// up to 64 tokens run on the weight-streaming kernel
inline bool w8a8_few_tokens(int64_t M) { return M <= 64; }
hipError_t launch_w8a8_skinny(const W8a8Args& a, hipStream_t stream);

}  // namespace svdq
