// Internal to the 8-bit linear's kernels: the few-token form.
#pragma once

#include "svdq_internal.h"

namespace svdq {

hipError_t launch_w8a8_skinny(const W8a8Args& a, hipStream_t stream);

}  // namespace svdq
