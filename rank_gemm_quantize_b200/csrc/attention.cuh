// What the attention kernels share: the call's parameters, the packed
// sequences' extents, 16-bit conversions.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace svdq {

struct AttnParams {
  const void *q, *v;  // v for the values that a product with 0 would spoil; tiles come by TMA
  void* out;          // [q_rows, q_heads, dim]
  const int *q_offsets, *k_offsets;
  int batch, q_rows, k_rows, q_heads, kv_heads, group, dim, causal;
  float scale_log2;   // scale * log2(e): softmax in base 2
  long long q_row, q_head, v_row, v_head;  // strides in elements
  // keys split over CTAs (few queries)
  int chunk;          // keys of a share, a multiple of the key tile
  int max_slots;      // partial results the workspace holds
  float *part, *part_ml;
};
struct AttnMaps {
  CUtensorMap k, v;   // [k_rows][kv_heads][dim], box {64, 1, key tile}, 128-byte swizzle, zero fill
};

__device__ __forceinline__ void seq_extent(const int* offsets, int b, int rows, int& start, int& len) {
  if (!offsets) {
    start = 0;
    len = rows;
    return;
  }
  start = min(max(offsets[b], 0), rows);
  len = min(max(offsets[b + 1], start), rows) - start;
}

template <class T>
struct Half16;
template <>
struct Half16<__nv_bfloat16> {
  static constexpr uint32_t kExp = 0x7F80;  // all exponent bits: infinities and NaN
  static constexpr uint32_t kFmt = 1;       // operand format code of kind::f16
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ float to_float(uint32_t bits) { return __uint_as_float(bits << 16); }
};
template <>
struct Half16<__half> {
  static constexpr uint32_t kExp = 0x7C00;
  static constexpr uint32_t kFmt = 0;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ float to_float(uint32_t bits) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
  }
};

// Zeroes the infinities and NaN of eight 16-bit values; true if there were any.
template <class T>
__device__ __forceinline__ bool drop_non_finite(uint4& v) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    constexpr uint32_t e = Half16<T>::kExp;
    if ((w[i] & e) == e) w[i] &= 0xFFFF0000u, any = true;
    if ((w[i] >> 16 & e) == e) w[i] &= 0x0000FFFFu, any = true;
  }
  return any;
}

// 2^x in one instruction (results under the normal range become 0).
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Keys and rows of the split kernel's tiles.
constexpr int kStepKeys = 64;
constexpr int kStepRows = 16;
// Sequences of at most this many row tiles have their keys split over CTAs.
constexpr int kSplitTiles = 4;

cudaError_t take_status_attention_step(int* status, cudaStream_t st);
cudaError_t launch_attention_step(const AttnParams& p, const AttnMaps& maps, bool bf16, int sms, cudaStream_t st);

}  // namespace svdq
