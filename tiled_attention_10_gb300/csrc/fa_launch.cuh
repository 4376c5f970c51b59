/*
 * fa_launch.cuh -- launch of a kernel as a programmatic dependent of the work
 * before it on the stream: its blocks may be placed while that work ends.  The
 * kernel has to call wait_for_stream() before it reads or writes memory, in
 * every thread (one that did not would let the kernel after it start early),
 * and then lets the next kernel's blocks be placed too, as its own end.
 */
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

namespace fa {

// The calling thread's current context (fa_api.cu).
CUcontext current_context(int* dev_out);

// Raises a kernel's limit of dynamic shared memory: once per device and context,
// not at every call.
template <auto KERNEL>
cudaError_t allow_smem(int bytes) {
  static std::atomic<CUcontext> known[64];
  int dev = 0;
  const CUcontext ctx = current_context(&dev);
  const bool kept = ctx && dev >= 0 && dev < 64;
  if (kept && known[dev].load(std::memory_order_acquire) == ctx) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && kept) known[dev].store(ctx, std::memory_order_release);
  return e;
}

struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  Launch(dim3 grid, int threads, size_t smem, cudaStream_t stream) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  Launch(const Launch&) = delete;
};

// Dynamic shared memory that a kernel gets without asking: 48 KB less what it
// declares itself (1 KB is kept for that here).
constexpr size_t kFreeSmem = 47 * 1024;

__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The next kernel on the stream may be placed once all blocks have come here (so
// only into room that none of them still needs); it waits for this one's end.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace fa
