// Host side of the library that its C entry points and launchers share.
#pragma once
#include <cuda_runtime.h>

#include <atomic>

namespace lola {

// Sets the text of lola_last_error_string and returns code; adds to lola_launch_count.
int report(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
void count_launches(int kernels);

// Lets a kernel use up to `bytes` of dynamic shared memory (0: all that a block may have, 227 KB), asked of the
// driver once on each device (bit i of *done).  The limit belongs to the device: a launch that asked for its own
// size could lower it under a larger launch of another thread, so `bytes` is the most that any launch takes.
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<unsigned long long>* done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (done->load(std::memory_order_relaxed) & bit) return cudaSuccess;
    if (bytes == 0) {
        cudaFuncAttributes at;
        if ((e = cudaFuncGetAttributes(&at, kernel)) != cudaSuccess) return e;
        bytes = 227 * 1024 - (int)at.sharedSizeBytes;
    }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace lola
