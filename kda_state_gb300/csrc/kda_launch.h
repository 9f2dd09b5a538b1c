// What launches share.  Host-side only.
#pragma once

#include <atomic>
#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

// Lets a kernel use `bytes` of dynamic shared memory on the current device: asked for once a device (a call costs as
// much as a launch's arguments do), `done` has a bit for each of the first 64.
inline cudaError_t allow_shared(const void *kernel, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

// A launch that may come in before the end of the one ahead of it in the stream, if that one allows it
// (let_later_kernels_in).  The kernel calls wait_for_earlier_kernels before it reads or writes anything, whatever is ahead of
// it: another thread may launch in between, and caches may hold what was there before.
template <typename... A>
cudaError_t launch_early(void (*kernel)(A...), dim3 grid, dim3 block, size_t shared, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = grid, c.blockDim = block, c.dynamicSmemBytes = shared, c.stream = s;
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &early, c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

}  // namespace kda
