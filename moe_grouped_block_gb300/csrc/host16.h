// host16.h -- host-side helpers of the 16-bit operators' launchers.
#pragma once

#include "mxg_host.h"

namespace mxg {

// 3-D tensor map with the 128-byte swizzle: dims[0] innermost (16-bit elements),
// byte strides of dims 1 and 2, box extents per dimension.  Returns false if the
// driver entry point is missing or rejects the description.
bool make_tmap_3d_swizzled(CUtensorMap* m, const void* base, const uint64_t dims[3],
                           const uint64_t strides_bytes[2], const uint32_t box[3]);

// Launches `kern`; with `early`, as soon as the kernel before it on the stream
// allows (grid_launch_dependents), so that its launch overlaps that kernel.  Such
// a kernel calls grid_wait_for_previous before it touches anything.
template <typename Kern, typename... Args>
cudaError_t launch_after(bool early, Kern kern, unsigned grid, int threads, size_t smem,
                         cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace mxg
