// mxg_host.h -- host-side helpers shared by the launchers.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mxg {

// 2-D tensor map over a row-major [rows, inner] matrix of `dtype` elements
// with `row_bytes` between rows; box [box_rows, box_inner]; the given
// swizzle.  Returns false if the driver entry point is missing or rejects
// the description.
bool make_tmap_2d(CUtensorMap* m, CUtensorMapDataType dtype, const void* base, uint64_t inner,
                  uint64_t rows, uint64_t row_bytes, uint32_t box_inner, uint32_t box_rows,
                  CUtensorMapSwizzle swizzle);

// 3-D tensor map: dims[0] innermost (elements), byte strides of dims 1 and 2,
// box extents per dimension, the given swizzle (none by default).
bool make_tmap_3d(CUtensorMap* m, CUtensorMapDataType dtype, const void* base, const uint64_t dims[3],
                  const uint64_t strides_bytes[2], const uint32_t box[3],
                  CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_NONE);

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
