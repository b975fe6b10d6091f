// The word in which the kernels of one source file that keep no handle record a
// wait that gave up (svdq_operator_status reads and clears them all).
#pragma once

#include "common.cuh"

namespace svdq {

static __device__ int g_status;

static cudaError_t take_status(int* status, cudaStream_t st) {
  const int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(status, g_status, 4, 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && *status) {
    e = cudaMemcpyToSymbolAsync(g_status, &zero, 4, 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  return e;
}

}  // namespace svdq
