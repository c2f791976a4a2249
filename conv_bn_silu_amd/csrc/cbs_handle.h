// cbs_handle.h -- the library handle and the checks that every entry point of
// the C ABI makes on it (defined in cbs_api.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/conv_bn_silu.h"

struct conv_bn_silu_handle {
    // Fixed at create and only read afterwards, so one handle may serve
    // concurrent calls from any number of threads and streams.
    int device;
    int num_cu;
    // Device address of the allocation-free entry point's scratch on this
    // device (NULL if the lookup failed; that entry point then reports it).
    void *noalloc_scratch;
};

namespace cbs {

// Whether h is a live handle of this library (never dereferences a foreign pointer).
bool handle_live(const conv_bn_silu_handle *h);
// CBS_OK if the current device is the handle's, else the status to return.
int check_device(const conv_bn_silu_handle *h);
// The status of a HIP call; keeps a failure's code for conv_bn_silu_last_hip_error.
int record_hip(hipError_t e);

}  // namespace cbs
