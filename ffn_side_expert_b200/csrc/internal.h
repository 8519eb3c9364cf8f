// internal.h -- what the library's translation units share on the host side.
#pragma once

#include <cuda_runtime.h>

namespace afd {

// Record the error of a call without a handle (afd_ffn_last_cuda_error(NULL)); AFD_ERR_CUDA.
int rows_cuda_fail(cudaError_t e);

// The current device's error word of the calls without a handle (afd_ffn_rows_error).
int rows_err_word(int** out);

}  // namespace afd
