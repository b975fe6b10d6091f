// The norms around a transformer block, fused with the block's gate and the
// scale of its residual. Per token (row) r of sequence b:
//   x' = a x + gate[b] * N_post(y)
//   h  = N_pre(x') * (1 + scale[b]) + shift[b]
// N is a layer norm (mean and variance), an RMS norm or absent, each with its
// own weight and bias vectors. One pass: x and y are read once, x' and h
// written once, and h is computed from the unrounded float x'.
//
// Both statistics are centred sums taken over values that stay in registers
// (the mean first, then the squares of the differences), so a large mean costs
// no digits. Memory bounds a call of many rows: 2 (sizeof(x) + 2) bytes a value.
// What decides how near it comes is how many rows an SM has under way, so the
// layouts below keep the registers low and the blocks small (at 16384 x 4096 with
// a float stream, norms on both sides, gate, scale and shift: 133 us, 92% of a copy's
// rate; the vectors asked for earlier, with twice the registers: 152 us; a
// persistent kernel fed by bulk copies through shared memory: 187 to 348 us). A call
// of few rows takes one row's latency, 2.6 us.
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

// VEC consecutive values as they lie in memory: words of 16, 4 or 2 bytes.
template <int BYTES>
struct WordOf;
template <>
struct WordOf<16> {
  using type = uint4;
};
template <>
struct WordOf<8> {
  using type = uint2;
};
template <>
struct WordOf<4> {
  using type = uint32_t;
};
template <>
struct WordOf<2> {
  using type = uint16_t;
};
template <class T, int VEC>
struct Raw {
  static constexpr int kWord = VEC * sizeof(T) < 16 ? VEC * sizeof(T) : 16;
  static constexpr int kWords = VEC * sizeof(T) / kWord;
  typename WordOf<kWord>::type w[kWords];
  __device__ __forceinline__ void load(const void* base, size_t at) {  // never an output of the call
    const auto* p = reinterpret_cast<const typename WordOf<kWord>::type*>(static_cast<const T*>(base) + at);
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldg(p + i);
  }
  __device__ __forceinline__ void load_once(const void* base, size_t at) {  // read by no other row
    const auto* p = reinterpret_cast<const typename WordOf<kWord>::type*>(static_cast<const T*>(base) + at);
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldcs(p + i);
  }
  __device__ __forceinline__ void store(void* base, size_t at) const {
    auto* p = reinterpret_cast<typename WordOf<kWord>::type*>(static_cast<T*>(base) + at);
#pragma unroll
    for (int i = 0; i < kWords; ++i) p[i] = w[i];
  }
  __device__ __forceinline__ float get(int e) const { return to_f(reinterpret_cast<const T*>(w)[e]); }
  __device__ __forceinline__ void set(int e, float v) { reinterpret_cast<T*>(w)[e] = from_f<T>(v); }
};

// a *= b, a += b, a = s b + a on VEC values, two at a time.
template <int VEC>
__device__ __forceinline__ void mul(float (&a)[VEC], const float (&b)[VEC]) {
#pragma unroll
  for (int e = 0; e + 1 < VEC; e += 2) {
    const float2 v = __fmul2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
    a[e] = v.x, a[e + 1] = v.y;
  }
  if constexpr (VEC == 1) a[0] *= b[0];
}
template <int VEC>
__device__ __forceinline__ void add(float (&a)[VEC], const float (&b)[VEC]) {
#pragma unroll
  for (int e = 0; e + 1 < VEC; e += 2) {
    const float2 v = __fadd2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
    a[e] = v.x, a[e + 1] = v.y;
  }
  if constexpr (VEC == 1) a[0] += b[0];
}
template <int VEC>
__device__ __forceinline__ void add_scaled(float (&a)[VEC], float s, const float (&b)[VEC]) {
#pragma unroll
  for (int e = 0; e + 1 < VEC; e += 2) {
    const float2 v = __ffma2_rn(make_float2(s, s), make_float2(b[e], b[e + 1]), make_float2(a[e], a[e + 1]));
    a[e] = v.x, a[e + 1] = v.y;
  }
  if constexpr (VEC == 1) a[0] = fmaf(s, b[0], a[0]);
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

// When a thread asks for the vectors (gate, weights, biases, scale, shift):
// kAtOnce along with the row (a call of few rows: the time is one row's latency);
// kBySum those of each norm before its sums; kByUse where they are used, which
// leaves the registers for more rows at a time.
enum When { kAtOnce, kBySum, kByUse };

constexpr int kRowsPerBlock1 = 4;  // rows of a block where one warp takes a row

// T: type of y, h and the vectors; X: type of x and x'. A row belongs to WARPS
// warps, each thread holds NV groups of VEC values.
template <class T, class X, int VEC, int NV, int WARPS, When WHEN>
__global__ void __launch_bounds__(WARPS == 1 ? kRowsPerBlock1 * 32 : WARPS * 32) residual_norm_kernel(const NormParams p) {
  __shared__ float scratch[2][WARPS];
  const int row = WARPS == 1 ? static_cast<int>(blockIdx.x) * kRowsPerBlock1 + static_cast<int>(warp_id()) : blockIdx.x;
  if (row >= p.rows) return;
  const int t = WARPS == 1 ? lane_id() : threadIdx.x;
  constexpr int kStep = WARPS * 32 * VEC;
  const size_t base = static_cast<size_t>(row) * p.dim;
  const float inv_dim = 1.0f / static_cast<float>(p.dim);
  int turn = 0;
  auto column = [&](int i) { return t * VEC + i * kStep; };

  Raw<X, VEC> xr[NV];
  Raw<T, VEC> yr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (column(i) < p.dim) {
      xr[i].load_once(p.x, base + column(i));
      if (p.y) yr[i].load_once(p.y, base + column(i));
    }
  // the row's sequence: the number of sequence ends at or before it; every
  // warp counts for itself
  int seq = 0;
  if (p.offsets) {
    if (row < p.offsets[0]) return;
    for (int b0 = 0; b0 < p.seqs; b0 += 32) {
      const int b = b0 + lane_id();
      seq += __popc(__ballot_sync(0xffffffffu, b < p.seqs && p.offsets[min(b + 1, p.seqs)] <= row));
    }
    if (seq >= p.seqs) return;  // behind the last sequence: the row is left alone
  }
  const size_t mod = static_cast<size_t>(seq) * p.dim;

  Raw<T, VEC> gate[NV], post_weight[NV], post_bias[NV], weight[NV], bias[NV], scale[NV], shift[NV];
  auto ask = [&](Raw<T, VEC>(&v)[NV], const void* from, size_t at) {
    if (from)
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (column(i) < p.dim) v[i].load(from, at + column(i));
  };
  auto ask_post = [&] {
    ask(post_weight, p.post_weight, 0);
    ask(post_bias, p.post_bias, 0);
    ask(gate, p.gate, mod);
  };
  auto ask_rest = [&] {
    ask(weight, p.weight, 0);
    ask(bias, p.bias, 0);
    ask(scale, p.scale, mod);
    ask(shift, p.shift, mod);
  };
  if constexpr (WHEN != kByUse) ask_post();
  if constexpr (WHEN == kAtOnce) ask_rest();

  float v[NV][VEC];
  // group i of v times (1 + a vector) or plus a vector
  auto times = [&](int i, Raw<T, VEC>(&w)[NV], const void* from, size_t at, float plus) {
    if (!from) return;
    if constexpr (WHEN == kByUse) w[i].load(from, at + column(i));
    float f[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = plus + w[i].get(e);
    mul(v[i], f);
  };
  auto plus = [&](int i, Raw<T, VEC>(&w)[NV], const void* from, size_t at) {
    if (!from) return;
    if constexpr (WHEN == kByUse) w[i].load(from, at + column(i));
    float f[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = w[i].get(e);
    add(v[i], f);
  };
  // centres the values where the norm does; returns 1 / deviation
  auto deviation = [&](int kind) {
    if (kind == SVDQ_NORM_LAYER) {
      float part[VEC] = {};
#pragma unroll
      for (int i = 0; i < NV; ++i) add(part, v[i]);
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += part[e];
      const float mean = row_sum<WARPS>(s, scratch, turn) * inv_dim;
      float minus[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) minus[e] = -mean;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (column(i) < p.dim) add(v[i], minus);
    }
    float part[VEC] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) part[e] = fmaf(v[i][e], v[i][e], part[e]);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) s += part[e];
    return 1.0f / sqrtf(row_sum<WARPS>(s, scratch, turn) * inv_dim + p.eps);
  };
  auto scaled = [&](int i, float r) {
    float f[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = r;
    mul(v[i], f);
  };

  if (p.y) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = column(i) < p.dim ? yr[i].get(e) : 0.f;
    const float r = p.post_norm != SVDQ_NORM_NONE ? deviation(p.post_norm) : 1.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = column(i);
      if (c < p.dim) {
        if (p.post_norm != SVDQ_NORM_NONE) scaled(i, r);
        times(i, post_weight, p.post_weight, 0, 0.f);
        plus(i, post_bias, p.post_bias, 0);
        times(i, gate, p.gate, mod, 0.f);
        float x[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] = xr[i].get(e);
        add_scaled(v[i], p.residual_scale, x);
        Raw<X, VEC> out;
#pragma unroll
        for (int e = 0; e < VEC; ++e) out.set(e, v[i][e]);
        out.store(p.x_out, base + c);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = column(i) < p.dim ? xr[i].get(e) : 0.f;
  }
  if (p.norm == SVDQ_NORM_NONE) return;
  if constexpr (WHEN == kBySum) ask_rest();
  const float r = deviation(p.norm);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = column(i);
    if (c < p.dim) {
      scaled(i, r);
      times(i, weight, p.weight, 0, 0.f);
      plus(i, bias, p.bias, 0);
      times(i, scale, p.scale, mod, 1.f);
      plus(i, shift, p.shift, mod);
      Raw<T, VEC> out;
#pragma unroll
      for (int e = 0; e < VEC; ++e) out.set(e, v[i][e]);
      out.store(p.h_out, base + c);
    }
  }
}

template <class T, class X, int VEC, int NV, int WARPS, When WHEN>
cudaError_t start(const NormParams& p, cudaStream_t st) {
  const int blocks = WARPS == 1 ? (p.rows + kRowsPerBlock1 - 1) / kRowsPerBlock1 : p.rows;
  residual_norm_kernel<T, X, VEC, NV, WARPS, WHEN><<<blocks, WARPS == 1 ? kRowsPerBlock1 * 32 : WARPS * 32, 0, st>>>(p);
  return cudaGetLastError();
}

// Rows of a multiple of 8 values (every row 16-byte aligned). Many rows: 2 to 4
// groups a thread, and as few warps a row as that takes; few rows: as many warps
// as the row has work for.
template <class T, class X>
cudaError_t pick_wide(const NormParams& p, bool many, cudaStream_t st) {
  const int groups = (p.dim + 255) / 256;  // groups of 8 a lane, for one warp
  if (many) {
    if (groups <= 2) return start<T, X, 8, 2, 1, kBySum>(p, st);
    if (groups <= 4) return start<T, X, 8, 2, 2, kBySum>(p, st);
    if (groups <= 6) return start<T, X, 8, 3, 2, kBySum>(p, st);
    if (groups <= 8) return start<T, X, 8, 2, 4, kBySum>(p, st);
    if (groups <= 12) return start<T, X, 8, 3, 4, kBySum>(p, st);
    if (groups <= 16) return start<T, X, 8, 2, 8, kByUse>(p, st);
    if (groups <= 24) return start<T, X, 8, 3, 8, kBySum>(p, st);
    if (groups <= 32) return start<T, X, 8, 4, 8, kByUse>(p, st);
    return start<T, X, 8, 4, 16, kByUse>(p, st);
  }
  if (groups <= 1) return start<T, X, 8, 1, 1, kAtOnce>(p, st);
  if (groups <= 4) return start<T, X, 8, 1, 4, kAtOnce>(p, st);
  if (groups <= 8) return start<T, X, 8, 1, 8, kAtOnce>(p, st);
  if (groups <= 16) return start<T, X, 8, 1, 16, kAtOnce>(p, st);
  if (groups <= 32) return start<T, X, 8, 2, 16, kAtOnce>(p, st);
  return start<T, X, 8, 4, 16, kByUse>(p, st);
}

// Other widths, by the same rule: pairs (an even dim) or single values.
template <class T, class X, int VEC>
cudaError_t pick_narrow(const NormParams& p, bool many, cudaStream_t st) {
  const int groups = (p.dim + 32 * VEC - 1) / (32 * VEC);
  constexpr When kWhen = VEC == 2 ? kBySum : kByUse;
  if (many) {
    if (groups <= 8) return start<T, X, VEC, 8, 1, kWhen>(p, st);
    if (groups <= 32) return start<T, X, VEC, 8, 4, kWhen>(p, st);
    if (groups <= 48) return start<T, X, VEC, 12, 4, kWhen>(p, st);
    if (groups <= 96) return start<T, X, VEC, 12, 8, kWhen>(p, st);
  } else {
    if (groups <= 2) return start<T, X, VEC, 2, 1, kAtOnce>(p, st);
    if (groups <= 8) return start<T, X, VEC, 2, 4, kAtOnce>(p, st);
    if (groups <= 32) return start<T, X, VEC, 2, 16, kAtOnce>(p, st);
    if (groups <= 64) return start<T, X, VEC, 4, 16, kAtOnce>(p, st);
  }
  return start<T, X, VEC, 32 / VEC, 16, kByUse>(p, st);
}

template <class T, class X>
cudaError_t pick_vector(const NormParams& p, cudaStream_t st) {
  const bool many = p.rows >= 200;  // at 3072: 600 rows 5.8 us so, 7.6 with the layout for few; 148 rows 3.1 with that
  if (p.dim % 8 == 0) return pick_wide<T, X>(p, many, st);
  return p.dim % 2 == 0 ? pick_narrow<T, X, 2>(p, many, st) : pick_narrow<T, X, 1>(p, many, st);
}

template <class T>
cudaError_t pick_stream(const NormParams& p, bool x_float, cudaStream_t st) {
  return x_float ? pick_vector<T, float>(p, st) : pick_vector<T, T>(p, st);
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
  const bool x_float = a->x_dtype == SVDQ_F32;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == SVDQ_BF16 ? pick_stream<__nv_bfloat16>(p, x_float, st)
                                              : pick_stream<__half>(p, x_float, st);
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, std::string("residual norm: ") + cudaGetErrorString(e));
  return SVDQ_OK;
}
