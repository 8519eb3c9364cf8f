// internal.h -- what the library's translation units share on the host side.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace afd {

// Launch a kernel that may start while the stream's kernel before it ends (ptx.cuh: wait_dependency): about a
// microsecond less between two small kernels.
template <typename... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s,
                             const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Record the error of a call without a handle (afd_ffn_last_cuda_error(NULL)); AFD_ERR_CUDA.
int rows_cuda_fail(cudaError_t e);

// The current device's error word of the calls without a handle (afd_ffn_rows_error).
int rows_err_word(int** out);

// Descriptor of a matrix of `rows` rows of row_bytes bytes (16-byte aligned), boxes of box_rows rows x
// box_bytes (64 or 128) bytes with the swizzle of that many bytes, zero fill outside.
bool encode_byte_rows(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows, uint32_t box_bytes,
                      uint32_t box_rows);

}  // namespace afd
