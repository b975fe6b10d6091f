// The norms around a transformer block, fused with the block's gate and the
// scale of its residual. Per token (row) r of sequence b:
//   x' = a x + gate[b] * N_post(y)
//   h  = N_pre(x') * (1 + scale[b]) + shift[b]
// N is a layer norm (mean and variance), an RMS norm or absent, each with its
// own weight and bias vectors. One pass: x and y are read once, x' and h
// written once, and h is computed from the unrounded float x'.
//
// Both statistics are centred sums taken over values that stay in registers
// (the mean first, then the squares of the differences), so a large mean
// costs no digits. Memory bounds the kernel: (2 sizeof(x) + 4) bytes a value.
#include <algorithm>
#include <cstdint>
#include <string>

#include "common.cuh"
#include "kernels.h"

namespace svdq {
void set_last_error(const std::string& msg);
}

using namespace svdq;

namespace {

svdq_status fail(svdq_status st, const std::string& msg) {
  set_last_error(msg);
  return st;
}

struct NormParams {
  const void *x, *y;
  void *x_out, *h_out;
  const void *gate, *post_weight, *post_bias;   // gate [seqs, dim]
  const void *weight, *bias, *scale, *shift;    // scale, shift [seqs, dim]
  const int* offsets;                           // [seqs + 1] or NULL (one sequence)
  int rows, dim, seqs;
  float residual_scale, eps;
  int post_norm, norm;
};

template <class T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

// VEC consecutive values, as wide loads where VEC is 8.
template <class T, int VEC>
__device__ __forceinline__ void load(const void* base, size_t at, float (&v)[VEC]) {
  const T* p = static_cast<const T*>(base) + at;
  if constexpr (VEC == 8) {
    constexpr int kWords = sizeof(T) / 2;
    uint4 w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    const T* t = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f(t[i]);
  } else {
    v[0] = to_f(p[0]);
  }
}
template <class T, int VEC>
__device__ __forceinline__ void store(void* base, size_t at, const float (&v)[VEC]) {
  T* p = static_cast<T*>(base) + at;
  if constexpr (VEC == 8) {
    constexpr int kWords = sizeof(T) / 2;
    uint4 w[kWords];
    T* t = reinterpret_cast<T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = from_f<T>(v[i]);
#pragma unroll
    for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
  } else {
    p[0] = from_f<T>(v[0]);
  }
}

// Sum over the WARPS warps of a row, the same in every thread. `turn` picks
// one of two scratch lines, so one barrier a sum is enough.
template <int WARPS>
__device__ __forceinline__ float row_sum(float v, float (*scratch)[WARPS], int& turn) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (WARPS > 1) {
    if (lane_id() == 0) scratch[turn][warp_id()] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v += scratch[turn][w];
    turn ^= 1;
  }
  return v;
}

constexpr int kRowsPerBlock1 = 4;  // rows of a block where one warp takes a row

// T: type of y, h and the vectors; X: type of x and x'. A row belongs to WARPS
// warps, each thread holds NV groups of VEC values.
template <class T, class X, int VEC, int NV, int WARPS>
__global__ void __launch_bounds__(WARPS == 1 ? kRowsPerBlock1 * 32 : WARPS * 32) residual_norm_kernel(const NormParams p) {
  __shared__ float scratch[2][WARPS];
  const int row = WARPS == 1 ? static_cast<int>(blockIdx.x) * kRowsPerBlock1 + static_cast<int>(warp_id()) : blockIdx.x;
  if (row >= p.rows) return;
  const int t = WARPS == 1 ? lane_id() : threadIdx.x;
  constexpr int kStep = WARPS * 32 * VEC;
  const size_t base = static_cast<size_t>(row) * p.dim;
  const float inv_dim = 1.0f / static_cast<float>(p.dim);
  int turn = 0;

  float v[NV][VEC], u[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = t * VEC + i * kStep;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[i][e] = u[i][e] = 0.f;
    if (c < p.dim) {
      load<X, VEC>(p.x, base + c, v[i]);
      if (p.y) load<T, VEC>(p.y, base + c, u[i]);
    }
  }
  // the row's sequence: the number of sequence ends at or before it; every
  // warp counts for itself
  int seq = 0;
  if (p.offsets) {
    if (row < p.offsets[0]) return;
    for (int b0 = 0; b0 < p.seqs; b0 += 32) {
      const int b = b0 + lane_id();
      seq += __popc(__ballot_sync(0xffffffffu, b < p.seqs && p.offsets[b + 1 <= p.seqs ? b + 1 : p.seqs] <= row));
    }
    if (seq >= p.seqs) return;  // behind the last sequence: the row is left alone
  }
  const size_t mod = static_cast<size_t>(seq) * p.dim;

  // 1 / deviation, after centring the values where the norm does
  auto normalise = [&](float (&a)[NV][VEC], int kind) {
    if (kind == SVDQ_NORM_LAYER) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += a[i][e];
      const float mean = row_sum<WARPS>(s, scratch, turn) * inv_dim;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (t * VEC + i * kStep < p.dim)
#pragma unroll
          for (int e = 0; e < VEC; ++e) a[i][e] -= mean;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s = fmaf(a[i][e], a[i][e], s);
    const float r = 1.0f / sqrtf(row_sum<WARPS>(s, scratch, turn) * inv_dim + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) a[i][e] *= r;
  };

  if (p.y) {
    if (p.post_norm != SVDQ_NORM_NONE) normalise(u, p.post_norm);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t * VEC + i * kStep;
      if (c < p.dim) {
        float w[VEC];
        if (p.post_weight) {
          load<T, VEC>(p.post_weight, c, w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) u[i][e] *= w[e];
        }
        if (p.post_bias) {
          load<T, VEC>(p.post_bias, c, w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) u[i][e] += w[e];
        }
        if (p.gate) {
          load<T, VEC>(p.gate, mod + c, w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) u[i][e] *= w[e];
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] = fmaf(p.residual_scale, v[i][e], u[i][e]);
        store<X, VEC>(p.x_out, base + c, v[i]);
      }
    }
  }
  if (p.norm == SVDQ_NORM_NONE) return;
  normalise(v, p.norm);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = t * VEC + i * kStep;
    if (c < p.dim) {
      float w[VEC];
      if (p.weight) {
        load<T, VEC>(p.weight, c, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] *= w[e];
      }
      if (p.bias) {
        load<T, VEC>(p.bias, c, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] += w[e];
      }
      if (p.scale) {
        load<T, VEC>(p.scale, mod + c, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] *= 1.0f + w[e];
      }
      if (p.shift) {
        load<T, VEC>(p.shift, mod + c, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] += w[e];
      }
      store<T, VEC>(p.h_out, base + c, v[i]);
    }
  }
}

template <class T, class X, int VEC, int NV, int WARPS>
cudaError_t start(const NormParams& p, cudaStream_t st) {
  if (WARPS == 1)
    residual_norm_kernel<T, X, VEC, NV, WARPS><<<(p.rows + kRowsPerBlock1 - 1) / kRowsPerBlock1, kRowsPerBlock1 * 32, 0, st>>>(p);
  else
    residual_norm_kernel<T, X, VEC, NV, WARPS><<<p.rows, WARPS * 32, 0, st>>>(p);
  return cudaGetLastError();
}

// The fewest warps that hold the row at SHORT groups of VEC values a thread,
// and LONG groups where even 16 warps need them (32 values of x and 32 of y a
// thread: 512 threads still have the registers for that, 1024 would not).
template <class T, class X, int VEC, int SHORT, int LONG>
cudaError_t pick_warps(const NormParams& p, cudaStream_t st) {
  const int groups = (p.dim + 32 * VEC - 1) / (32 * VEC);  // groups of VEC per lane of one warp
  if (groups <= SHORT) return start<T, X, VEC, SHORT, 1>(p, st);
  if (groups <= 4 * SHORT) return start<T, X, VEC, SHORT, 4>(p, st);
  if (groups <= 8 * SHORT) return start<T, X, VEC, SHORT, 8>(p, st);
  if (groups <= 16 * SHORT) return start<T, X, VEC, SHORT, 16>(p, st);
  return start<T, X, VEC, LONG, 16>(p, st);
}

template <class T, class X>
cudaError_t pick_vector(const NormParams& p, bool wide, cudaStream_t st) {
  return wide ? pick_warps<T, X, 8, 2, 4>(p, st) : pick_warps<T, X, 1, 8, 32>(p, st);
}

template <class T>
cudaError_t pick_stream(const NormParams& p, bool x_float, bool wide, cudaStream_t st) {
  return x_float ? pick_vector<T, float>(p, wide, st) : pick_vector<T, T>(p, wide, st);
}

constexpr int kMaxDim = 16384;  // 16 warps, 32 values a thread

}  // namespace

extern "C" svdq_status svdq_residual_norm(const svdq_residual_norm_args* a, void* stream) {
  if (!a) return fail(SVDQ_ERR_INVALID_ARG, "args is NULL");
  if (a->dtype != SVDQ_BF16 && a->dtype != SVDQ_F16) return fail(SVDQ_ERR_INVALID_ARG, "unknown dtype");
  if (a->x_dtype != a->dtype && a->x_dtype != SVDQ_F32)
    return fail(SVDQ_ERR_INVALID_ARG, "x_dtype must be dtype or SVDQ_F32");
  if (a->rows < 0 || a->dim < 1 || a->seqs < 1) return fail(SVDQ_ERR_INVALID_ARG, "bad rows, dim or seqs");
  if (a->dim > kMaxDim) return fail(SVDQ_ERR_UNSUPPORTED, "dim exceeds 16384");
  auto kind = [](int k) { return k == SVDQ_NORM_NONE || k == SVDQ_NORM_LAYER || k == SVDQ_NORM_RMS; };
  if (!kind(a->norm) || !kind(a->post_norm)) return fail(SVDQ_ERR_INVALID_ARG, "unknown norm");
  if (!(a->eps >= 0.f) || a->eps > 1e30f) return fail(SVDQ_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (!(a->residual_scale >= -1e30f && a->residual_scale <= 1e30f))
    return fail(SVDQ_ERR_INVALID_ARG, "residual_scale must be finite");
  if (!a->offsets && a->seqs != 1) return fail(SVDQ_ERR_INVALID_ARG, "several sequences need offsets");
  if (a->rows == 0) return SVDQ_OK;  // empty tensors may have no address
  if (!a->y && (a->x_out || a->gate || a->post_weight || a->post_bias || a->post_norm != SVDQ_NORM_NONE ||
                a->residual_scale != 1.f))
    return fail(SVDQ_ERR_INVALID_ARG, "without y there is no x_out, gate, post norm or residual scale");
  if (a->post_norm == SVDQ_NORM_NONE && (a->post_weight || a->post_bias))
    return fail(SVDQ_ERR_INVALID_ARG, "post_weight and post_bias belong to a post norm");
  if (a->norm == SVDQ_NORM_NONE && (a->h_out || a->weight || a->bias || a->scale || a->shift))
    return fail(SVDQ_ERR_INVALID_ARG, "without a norm there is no h_out, weight, bias, scale or shift");
  if (!a->y && a->norm == SVDQ_NORM_NONE) return fail(SVDQ_ERR_INVALID_ARG, "neither y nor a norm: nothing to do");
  if (!a->x || (a->y && !a->x_out) || (a->norm != SVDQ_NORM_NONE && !a->h_out))
    return fail(SVDQ_ERR_INVALID_ARG, "x, x_out or h_out is NULL");
  const void* all[] = {a->x, a->y, a->x_out, a->h_out, a->gate, a->post_weight, a->post_bias, a->weight, a->bias, a->scale, a->shift};
  uintptr_t bits = 0;
  for (const void* q : all) bits |= reinterpret_cast<uintptr_t>(q);
  if (bits & 15) return fail(SVDQ_ERR_INVALID_ARG, "device pointers must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(a->offsets) & 3) return fail(SVDQ_ERR_INVALID_ARG, "offsets must be 4-byte aligned");
  NormParams p{a->x, a->y, a->x_out, a->h_out, a->gate, a->post_weight, a->post_bias, a->weight, a->bias,
               a->scale, a->shift, a->offsets, a->rows, a->dim, a->seqs, a->residual_scale, a->eps, a->post_norm, a->norm};
  // rows of a multiple of 8 values keep every row 16-byte aligned: wide loads
  const bool wide = a->dim % 8 == 0, x_float = a->x_dtype == SVDQ_F32;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == SVDQ_BF16 ? pick_stream<__nv_bfloat16>(p, x_float, wide, st)
                                              : pick_stream<__half>(p, x_float, wide, st);
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, std::string("residual norm: ") + cudaGetErrorString(e));
  return SVDQ_OK;
}
