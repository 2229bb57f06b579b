// Errors of the CUDA runtime's host calls.
#pragma once

#include <cuda_runtime.h>

namespace vc {

// The result of a runtime call, which the entry point returns as its own: it is not left
// behind as the runtime's last error, where the program's next call that asks for that
// would find it and take it for its own.
inline cudaError_t reported(cudaError_t e) {
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

}  // namespace vc
