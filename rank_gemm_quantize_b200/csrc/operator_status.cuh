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

// Self-test: one lane waits for an arrival that never comes, the others for one that
// has. All of them have to give up; a lane that went on would clear the word again.
static __global__ void give_up_kernel() {
  __shared__ uint64_t bars[2];
  __shared__ int abort_word;
  if (threadIdx.x == 0) {
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    abort_word = 0;
    fence_barrier_init();
    mbar_arrive(&bars[1]);
  }
  __syncthreads();
  const bool ok = warp_wait(&bars[lane_id() > 0], 0, &abort_word, &g_status);
  __syncwarp();
  if (ok) atomicExch(&g_status, kDevOk);
}

static cudaError_t give_up(cudaStream_t st) {
  give_up_kernel<<<1, 32, 0, st>>>();
  return cudaGetLastError();
}

}  // namespace svdq
