// Host helpers shared by the C-ABI entry files.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "../../include/okls.h"

namespace okls {

// Keep the message for okls_last_error() and return the status.
okls_status host_fail(okls_status s, const char* fmt, ...);

// SM count of the current device; fails on anything but an sm_103 GPU.
okls_status host_device_sms(int* sms);

// cuTensorMapEncodeTiled of the driver, or null.
PFN_cuTensorMapEncodeTiled_v12000 host_encode_fn();

}  // namespace okls
