// pa_flags.cuh -- faults that depend on device data, for the kernels of the rotary append and of
// the windowed decode.
#pragma once

#include "pa_internal.h"

namespace pa {

namespace {

// Adds PA_DEV_ERR_* bits to the caller's flag, if there is one.
__device__ __forceinline__ void raise_flag(int32_t* err, int bits) {
    if (err) atomicOr(err, bits);
}

}  // namespace

}  // namespace pa
