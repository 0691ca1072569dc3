// ds_host.h -- error reporting shared by the library's host code.
#pragma once

#include <cuda_runtime.h>

namespace ds {

// Message of the calling thread's most recent failure (ds_last_error_detail).
extern thread_local char g_detail[512];

// Records a message and returns `status`.
int fail(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int fail_cuda(cudaError_t e, const char *what);

// The current device's ordinal and its SM count, asked of CUDA once a device.
int current_device(int *dev, int *sms);

}  // namespace ds
