// tensor_map.cuh -- cuTensorMapEncodeTiled from the driver, looked up once through the runtime (the
// library does not link the driver).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace stq {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Null where the driver has no such entry point.
inline EncodeTiled encode_tiled()
{
    // a function-local static: initialised once, safely across host threads
    static const EncodeTiled fn = []() -> EncodeTiled {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiled>(f);
        return nullptr;
    }();
    return fn;
}

}  // namespace stq
