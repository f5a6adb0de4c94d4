// Shared by the library's entry points: per-thread errors, counters, device facts and
// the workspace pool (defined in gemv_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gemv.h"

namespace gemv {

void record_cuda_error(int e);
void count_launches(int n);
int launch_overlap();  // the calling thread's gemv_set_launch_overlap mode

// record_cuda_error, as a status.
gemv_status_t fail(int cuda_error);
// SMs of the current device.
gemv_status_t device_sms(int *out);
// Status word of the current device, for kernels with bounded waits or checks of their own.
gemv_status_t device_status_word(int **out);
// Limit of a bounded wait, and the test switch that withholds an MMA.
int64_t wait_limit(int *stall);
// [p, p + n) and [q, q + m) share a byte.
bool overlaps(const void *p, int64_t n, const void *q, int64_t m);
// Tensor map of a row-major matrix of bytes, in boxes of box_rows x box_cols (128-byte
// swizzle), zeros outside.
bool map_bytes(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int box_rows, int box_cols);
// Stream-ordered memory from the library's own pool of the current device, which keeps
// what it has mapped (the device's default pool gives it back at each synchronisation,
// and mapping it again costs more than these kernels take).  Free with cudaFreeAsync.
cudaError_t workspace(void **p, size_t bytes, cudaStream_t s);

}  // namespace gemv
