// The driver's tensor-map encoder, looked up once per process.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace pkd {
// null when the driver has none
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
}  // namespace pkd
