// kvq_around.cuh -- the launches of the calls around the cache: rotation with several
// axes, attention over prompts, selection over beams, caches reordered.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

cudaError_t launch_rotate(const kvq_rotate_args& args, cudaStream_t st);

cudaError_t launch_prompt_attention(const kvq_prompt_args& args, cudaStream_t st);

size_t beam_workspace_bytes(int batch, int beams, int vocab, int n);
cudaError_t launch_beam_select(const kvq_beam_args& args, cudaStream_t st);

cudaError_t launch_reorder(const Dims& d, const kvq_cache_view& dv, const Dims& s, const kvq_cache_view& sv,
                           const int32_t* index, bool share, cudaStream_t st);

// A launch that may begin while the kernel before it ends (and waits for it).
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                              const Args&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Nothing is read or written before the kernel before this one is done.  What is read then
// changed while this kernel ran, so it is no read-only data (__ldg), which may be loaded at
// any time.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
}

}  // namespace kvq
