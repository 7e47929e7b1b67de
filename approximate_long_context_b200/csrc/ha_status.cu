// ha_status.cu -- the status word of the serving kernels is read and cleared in one step: kernels of graphs that were captured on
// the handle may set bits in it from other streams at any time, and a bit set between a copy and a clear would be lost.
#include "ha_internal.h"

namespace ha {
namespace {

__global__ void take_status_kernel(int *status, int *taken) { *taken = atomicExch(status, 0); }

}  // namespace

bool launch_take_status(int *status, int *taken, cudaStream_t st) {
    void *args[] = {&status, &taken};
    return cudaLaunchKernel(reinterpret_cast<const void *>(take_status_kernel), dim3(1), dim3(1), args, 0, st) == cudaSuccess;
}

}  // namespace ha
