// fa_host.h -- host-side helpers of fa_api.cu that the other files of the C
// ABI use: the current device's set-up and the tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace fa {

// Checks that the current device is an sm_100 GPU; its error word and SM count.
int host_device(int **err, int *sm_count);

// The driver's cuTensorMapEncodeTiled.
int host_encoder(PFN_cuTensorMapEncodeTiled_v12000 *fn);

// Limit of every device-side wait, in nanoseconds.
unsigned long long host_wait_limit_ns();

}  // namespace fa
