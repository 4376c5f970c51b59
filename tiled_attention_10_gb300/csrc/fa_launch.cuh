/*
 * fa_launch.cuh -- launch of a kernel as a programmatic dependent of the work
 * before it on the stream: its blocks may be placed while that work ends.  The
 * kernel has to call wait_for_stream() before it reads or writes memory, in
 * every thread (one that did not would let the kernel after it start early).
 */
#pragma once
#include <cuda_runtime.h>

namespace fa {

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

__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace fa
