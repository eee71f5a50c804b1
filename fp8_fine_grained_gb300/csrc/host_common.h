// Host-side helpers shared by the library's translation units: per-device
// status word, SM count, wait limit and argument checks.
#pragma once

#include <atomic>

#include <cuda_runtime.h>
#include <stdint.h>

#include "fp8fg.h"

namespace fp8fg {

// Device address of the current device's status word (a __device__ int in
// capi.cu), or nullptr when CUDA is unavailable.
int *status_word_ptr();

// Number of SMs of the current device (cached per device), 0 on error.
int sm_count();

// Wait limit of the device-side bounded waits, in nanoseconds.
uint64_t wait_limit_ns();

// One-shot test hook consumed by the next GEMM launch on the current device.
bool take_skip_first_load();

// Schedule of the grouped GEMM with rows in expert order: the skinny-tile
// row threshold (0: off) and a skinny tile's SM time relative to a full
// tile, in percent.
int grouped_skinny_rows();
int grouped_skinny_cost_pct();

// Current device is a Blackwell sm_103 part (cached per device).
bool device_supported();

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int launch_status()
{
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? FP8FG_OK : FP8FG_ECUDA;
}

// Allow `bytes` of dynamic shared memory, once per kernel and device: `done`
// holds a bit per device and belongs to the kernel. (The call costs about as
// much as the rest of a launch's preparation.)
template <typename K>
bool allow_smem(K k, size_t bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return false;
    }
    const uint64_t bit = 1ull << dev;
    if (done.load() & bit)
        return true;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    done.fetch_or(bit);
    return true;
}

// Launch with programmatic stream serialization: the grid may start while the
// previous kernel's last CTAs run, so the kernel waits (griddep_wait) before
// it touches memory that an earlier kernel of the stream reads or writes.
template <typename... KArgs, typename... Args>
int launch_pss(void (*k)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t s, const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k, KArgs(args)...) != cudaSuccess) {
        cudaGetLastError();
        return FP8FG_ECUDA;
    }
    return launch_status();
}

}  // namespace fp8fg
