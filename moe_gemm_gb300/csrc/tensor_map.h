// The driver's tensor-map encoder, resolved once (null when the driver lacks it).
#pragma once

#include <cudaTypedefs.h>

namespace w8a8 {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode_fn();

}  // namespace w8a8
