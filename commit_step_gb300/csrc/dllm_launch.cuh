// dllm_launch.cuh -- host-side launch helpers shared by the cache, attention
// and scoring entry points.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/dllmcommit.h"

namespace dllm {

// Programmatic dependent launch of `kernel` (see the header's conventions),
// as clusters of `cluster` CTAs when cluster > 1.
inline dllm_status launch_pdl(const void* kernel, dim3 grid, dim3 block, size_t smem, dllm_stream_t stream, void** args,
                              int cluster = 1) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelExC(&cfg, kernel, args) == cudaSuccess ? DLLM_OK : DLLM_ERR_CUDA;
}

// a * b for a, b >= 0, or -1 when the product exceeds 2^62 (no such buffer).
inline int64_t mul_or_neg(int64_t a, int64_t b) {
  constexpr int64_t lim = static_cast<int64_t>(1) << 62;
  if (a < 0 || b < 0) return -1;
  if (a == 0 || b == 0) return 0;
  return a > lim / b ? -1 : a * b;
}

// The current device's fault word (dllm_fault_word), or null.
int32_t* fault_word();

// The bytes of rows x cols elements of `size` bytes, rows `stride` elements apart.
struct Extent {
  const void* at;
  int64_t bytes;
};
inline Extent extent(const void* at, int64_t rows, int64_t cols, int64_t stride, int64_t size) {
  return {at, at && rows > 0 ? ((rows - 1) * stride + cols) * size : 0};
}
inline bool overlap(Extent a, Extent b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.bytes > 0 && b.bytes > 0 && x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}
// Whether an output overlaps an input, or another output.
template <size_t N, size_t M>
inline bool overlapping(const Extent (&outs)[N], const Extent (&ins)[M]) {
  for (size_t i = 0; i < N; ++i) {
    for (const Extent& in : ins)
      if (overlap(outs[i], in)) return true;
    for (size_t j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace dllm
