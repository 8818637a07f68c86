// tk_launch.cuh -- launches that overlap the end of the launch before them.
//
// The serving calls follow one another on a stream and take a few microseconds
// each, of which getting a grid going is a good part.  They are launched with
// programmatic stream serialization: a grid's blocks may become resident while
// the grid before still runs, and every thread waits (grid_wait) before it
// reads or writes device memory, for all of that grid to have ended and its
// writes to be visible.  A grid that was launched the plain way ends before, as
// ever; and one that calls grid_launch_dependents lets the next begin once all its
// own blocks have.  Every block waits, whatever it then does: a grid's end so
// implies the end of all grids before it.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace tkattn {

__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_launch_dependents_if(int on) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %0, 0;\n\t"
               "@p griddepcontrol.launch_dependents;\n\t}" ::"r"(on)
               : "memory");
}
__device__ __forceinline__ void grid_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Whether a grid's blocks (of 64 or 128 threads) can all be resident at once.  One
// that is not leaves the next alone: begun beside the last of many waves, that ran
// slower than one behind the other (norm with rotation, then its gradients, 4 x 4096
// tokens, 40 heads of 128: 166 us for 146).
inline int one_wave(long long blocks, int num_sms) { return blocks <= 16LL * num_sms; }

template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, Args &&...args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(std::forward<Args>(args))...);
}

}  // namespace tkattn
