// gdn_tensor_map.cuh -- host side: the driver's tensor map encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace gdn {

// looked up once (the library links the runtime alone); nullptr where the driver has none
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(e == cudaSuccess && found == cudaDriverEntryPointSuccess ? f : nullptr);
    }();
    return encode;
}

}  // namespace gdn
