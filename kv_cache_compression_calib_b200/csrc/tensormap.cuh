// Tensor maps for TMA copies, encoded through the runtime's driver entry point (no
// link to libcuda).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "tri_internal.cuh"

namespace tri {

inline PFN_cuTensorMapEncodeTiled_v12000 tensormap_encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }
    return fn;
}

}  // namespace tri
