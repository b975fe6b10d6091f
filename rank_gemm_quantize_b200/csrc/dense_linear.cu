// The linear layer whose weight stays in 16 bits, with bias, activation and
// residual in the product's epilogue:
//   Y = residual + act(X W + bias),  X [M, K], W [K, N] (read in place)
//
// Rows kernel (few tiles): a CTA computes Y^T for 128 columns of W and RB
// rows of X. W^T is the tensor core's A operand (the tile [64 k, 128 n] lands by
// TMA as it lies in memory: M-major), X its B operand, so a product with few
// rows costs few tensor-core columns and the kernel streams W at memory speed.
// Where the tiles leave SMs free, the CTAs of a cluster take shares of K: each
// sends its float partial sums of a slice of the rows to the CTA that owns the
// slice (distributed shared memory), and the owner adds them in a fixed order.
// No workspace, no atomics, one launch. W's bytes bound it (1 x 3072 x 18432,
// 113 MB: 21.4 us, 81% of a copy's rate), and where W is small the latency of one
// load, one product and the join (37 x 2056 x 1000: 6.7 us on the device).
//
// Pair kernel (many tiles): two SMs work as one (tcgen05 .cta_group::2) on a
// tile of 256 rows and 256 or 128 columns, each holding its own 128 rows of X and
// half of W's columns: an SM then loads 32 KB per 512 cycles of products (a
// tile of its own, 128 x 128, needs as much for 256; an SM takes in 50 to 60 bytes a
// cycle). Persistent; two accumulators in tensor memory, so the epilogue of a tile
// runs under the next tile's products. The tensor core bounds it (4608 x 3072 x
// 12288: single calls 222 to 229 us, 1519 to 1568 TFLOP/s, and 260 us, 1336 TFLOP/s,
// in a long run under the power cap; a library's plain product 235 to 243 and 255 us).
#include <algorithm>
#include <cstdint>
#include <string>

#include "attention.cuh"
#include "common.cuh"
#include "kernels.h"
#include "operator_status.cuh"

namespace svdq {
void set_last_error(const std::string& msg);
}

using namespace svdq;

namespace {

svdq_status fail(svdq_status st, const std::string& msg) {
  set_last_error(msg);
  return st;
}

struct DenseParams {
  const void *bias, *residual;  // may be NULL
  void* Y;
  int M, N, K, act;
};
struct DenseMaps {
  CUtensorMap x;  // X [M, K], box {64, rows of a tile}, 128-byte swizzle, zero fill
  CUtensorMap w;  // W [K, N], box {64, 64}, 128-byte swizzle, zero fill
  CUtensorMap y;  // pair kernel: Y [M, N], box {32, 32}, 64-byte swizzle
};

// GELU of two values, t Phi(t) = t / (1 + 2^-g(t)) with g = log2(Phi(t) / Phi(-t)):
// this form keeps the digits of the negative side, where 1 + erf loses them.
// g(t) / t is even and smooth; P is a polynomial in t^2 fitted to it on [0, 30] by
// weighted minimax (Lawson's iteration), the weight making the result's error at
// most 2^-21 + 2^-18 |t Phi(t)| over 7. Behind the fit's end, where -t Phi(t)
// < 2e-7, t^2 stays at 30. Seven packed multiply-adds, one ex2, one division.
__device__ __forceinline__ float2 gelu2(float2 t) {
  const float2 t2 = __fmul2_rn(t, t);
  const float2 s = make_float2(fminf(t2.x, 30.f), fminf(t2.y, 30.f));
  auto both = [](float c) { return make_float2(c, c); };
  float2 q = both(5.11132959e-09f);
  q = __ffma2_rn(q, s, both(-3.80040715e-07f));
  q = __ffma2_rn(q, s, both(1.13597776e-05f));
  q = __ffma2_rn(q, s, both(-0.000158607879f));
  q = __ffma2_rn(q, s, both(-9.8645113e-05f));
  q = __ffma2_rn(q, s, both(0.104843492f));
  q = __ffma2_rn(q, s, both(2.30220498f));
  const float2 g = __fmul2_rn(q, t);
  return make_float2(__fdividef(t.x, 1.f + exp2_fast(-g.x)), __fdividef(t.y, 1.f + exp2_fast(-g.y)));
}

// In float, by the hardware's exponential and an approximate division, whose documented
// errors are a few 2^-22 of the result near 0 and up to 2^-16 of one at t = -80; the
// output keeps 2^-8 or 2^-11. Where the divisor passes 2^126 (t under -87) the division
// gives 0 for less than 2e-36.
template <int N>
__device__ __forceinline__ void activate(float2 (&v)[N], int act) {
  switch (act) {
    case SVDQ_ACT_RELU:
#pragma unroll
      for (float2& t : v) t = make_float2(t.x < 0.f ? 0.f : t.x, t.y < 0.f ? 0.f : t.y);  // NaN stays
      break;
    case SVDQ_ACT_SILU:
#pragma unroll
      for (float2& t : v) t = make_float2(__fdividef(t.x, 1.f + __expf(-t.x)), __fdividef(t.y, 1.f + __expf(-t.y)));
      break;
    case SVDQ_ACT_GELU:
#pragma unroll
      for (float2& t : v) t = gelu2(t);
      break;
    case SVDQ_ACT_GELU_TANH:
      // (1 + tanh(z)) / 2 = 1 / (1 + exp(-2 z)); 2 log2(e) sqrt(2 / pi) = 2.302208198
#pragma unroll
      for (float2& t : v) {
        const float2 t2 = __fmul2_rn(t, t);
        const float2 z = __fmul2_rn(__ffma2_rn(t2, make_float2(0.10294324f, 0.10294324f), make_float2(2.3022082f, 2.3022082f)), t);
        t = make_float2(__fdividef(t.x, 1.f + exp2_fast(-z.x)), __fdividef(t.y, 1.f + exp2_fast(-z.y)));
      }
      break;
  }
}

template <class T>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  return make_float2(Half16<T>::to_float(w & 0xFFFFu), Half16<T>::to_float(w >> 16));
}

// Eight columns of a row: bias, activation, residual (what p has of them), one rounding.
template <class T>
__device__ __forceinline__ uint4 finish8(const DenseParams& p, const uint4& bias, const float (&a)[8], const uint4& residual) {
  float2 v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = make_float2(a[2 * e], a[2 * e + 1]);
  if (p.bias) {
    const uint32_t w[4] = {bias.x, bias.y, bias.z, bias.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __fadd2_rn(v[e], unpack<T>(w[e]));
  }
  activate(v, p.act);
  if (p.residual) {
    const uint32_t w[4] = {residual.x, residual.y, residual.z, residual.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __fadd2_rn(v[e], unpack<T>(w[e]));
  }
  return make_uint4(Half16<T>::pack(v[0].x, v[0].y), Half16<T>::pack(v[1].x, v[1].y), Half16<T>::pack(v[2].x, v[2].y),
                    Half16<T>::pack(v[3].x, v[3].y));
}

constexpr int kBK = 64;

// ---------------------------------------------------------------- rows kernel
constexpr int kRowsN = 128;  // columns of W of a CTA
constexpr int kRowsThreads = 256, kRowsWarps = 8;

template <int RB>
struct RowsSmem {
  static constexpr int kW = kRowsN * kBK * 2;  // 16 KB
  static constexpr int kX = RB * kBK * 2;
  static constexpr int kStage = kW + kX;
  static constexpr int kPitch = kRowsN + 4;  // floats of a row of partial sums
  static constexpr int kSums = RB * kPitch * 4;
  static constexpr int kRoom = (RB == 128 ? 200 : 110) * 1024;  // up to 64 rows: two CTAs an SM
  static constexpr int kStages = (kRoom - kSums) / kStage;
  static constexpr int kSumsOff = kStages * kStage;
  static constexpr int kBars = kSumsOff + kSums;
  static constexpr int kTotal = kBars + 256 + 1024;
};

// The shared::cluster address of `addr` in CTA `rank`.
__device__ __forceinline__ uint32_t map_cluster(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// That the barriers of this CTA are there, which fence_barrier_init has published (a
// releasing arrival: 37 x 2056 x 1000 7.2 us for 6.7).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <class T, int RB>
__global__ void __launch_bounds__(kRowsThreads) dense_rows_kernel(const DenseParams p, const __grid_constant__ DenseMaps maps, int share_bits) {
  using L = RowsSmem<RB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* empty = full + L::kStages;
  uint64_t* acc_full = empty + L::kStages;
  uint64_t* sums_full = acc_full + 1;  // the shares' sums of this CTA's rows have arrived
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sums_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t kCols = RB < 32 ? 32 : RB;

  const int warp = warp_id(), lane = lane_id();
  const int shares = 1 << share_bits;
  const int share = blockIdx.x & (shares - 1);  // also the rank in the cluster
  const int n0 = (blockIdx.x >> share_bits) * kRowsN;
  const int m0 = blockIdx.y * RB;
  const int blocks = (p.K + kBK - 1) / kBK;
  const int first = static_cast<int>(static_cast<long long>(blocks) * share / shares);
  const int last = static_cast<int>(static_cast<long long>(blocks) * (share + 1) / shares);

  constexpr int kRowBits = RB == 16 ? 4 : RB == 32 ? 5 : RB == 64 ? 6 : 7;
  const int slice_bits = kRowBits - share_bits, slice = 1 << slice_bits;  // rows that each CTA of the cluster finishes
  const int mine = max(0, min(slice, p.M - m0 - share * slice));

  // The first loads need no one but the barriers: they start before tensor
  // memory is there.
  const int ahead = min(last - first, L::kStages);
  auto load = [&](int n) {
    const int s = n % L::kStages;
    uint8_t* st = smem + s * L::kStage;
    mbar_arrive_expect_tx(&full[s], L::kStage);
    tma_load_2d(st, &maps.w, &full[s], n0, (first + n) * kBK);
    tma_load_2d(st + 8192, &maps.w, &full[s], n0 + 64, (first + n) * kBK);
    tma_load_2d(st + L::kW, &maps.x, &full[s], (first + n) * kBK, m0);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(sums_full, shares * kRowsWarps);
    *abort_flag = 0;
    fence_barrier_init();
    for (int n = 0; n < ahead; ++n) load(n);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (shares > 1) cluster_arrive();  // this CTA's barriers are ready for the others
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int n = ahead;
      for (; n < last - first; ++n)
        if (mbar_wait(&empty[n % L::kStages], ((n / L::kStages) & 1) ^ 1, abort_flag, &g_status))
          load(n);
        else
          break;
      if (n < last - first) {  // gave up: the copies in flight land before the CTA ends
        volatile int no_abort = 0;
        for (int e = std::max(0, n - L::kStages); e < n; ++e)
          mbar_wait(&full[e % L::kStages], (e / L::kStages) & 1, &no_abort, nullptr);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      // A: W^T, 128 columns of W, M-major (bit 15); B: X, RB rows, K-major
      const uint32_t idesc = idesc_dense(kFmtF32, Half16<T>::kFmt, Half16<T>::kFmt, kRowsN, RB) | (1u << 15);
      for (int n = 0; n < last - first; ++n) {
        const int s = n % L::kStages;
        if (!mbar_wait(&full[s], (n / L::kStages) & 1, abort_flag, &g_status)) break;
        tc_fence_after();
        const uint32_t wa = smem_u32(smem + s * L::kStage), xb = wa + L::kW;
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k)
          mma_f16(tmem, smem_desc(wa + 2048 * k, 8192, 1024, kSw128), smem_desc(xb + 32 * k, 16, 1024, kSw128), idesc,
                  (n > 0 || k > 0) ? 1u : 0u);
        tc_commit(&empty[s]);
      }
      tc_commit(acc_full);
    }
    __syncwarp();
  }
  // Thread t finishes columns 8 (t % 16) .. of rows t / 16, t / 16 + 16, .. of the
  // slice; the bias and the first row's residual are asked for ahead. The
  // loops below are kept rolled: their code runs once, and fetching it costs.
  const int c8 = threadIdx.x % (kRowsN / 8) * 8, r0 = threadIdx.x / (kRowsN / 8), n8 = n0 + c8;
  uint4 bias = make_uint4(0, 0, 0, 0);
  if (p.bias && n8 < p.N) bias = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.bias) + n8));
  auto at = [&](int r) { return static_cast<size_t>(m0 + share * slice + r) * p.N + n8; };
  auto residual = [&](int r) {
    if (!p.residual || r >= mine || n8 >= p.N) return make_uint4(0, 0, 0, 0);
    return *reinterpret_cast<const uint4*>(static_cast<const T*>(p.residual) + at(r));
  };
  uint4 res = residual(r0);
  volatile int no_abort = 0;
  warp_wait(acc_full, 0, &no_abort, &g_status);
  tc_fence_after();

  // The partial sums go to the owners of the rows, [share][row of the slice][column];
  // two warps a quarter of the lanes, each with every other 16 rows.
  if (shares > 1) cluster_wait();
  const uint32_t column = 32 * (warp & 3) + lane;
  const uint32_t here = smem_u32(smem + L::kSumsOff) + (share * slice * L::kPitch + column) * 4;
#pragma unroll 1
  for (int c = 16 * (warp >> 2); c < RB; c += 32) {
    if (m0 + c >= p.M) break;  // rows behind the last one are not read below
    uint32_t r[16];
    tmem_ld16(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + c, r);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 16; e += 2) {  // a slice has two rows or more
      const uint32_t to = map_cluster(here + ((c + e) & (slice - 1)) * (L::kPitch * 4), (c + e) >> slice_bits);
      store_cluster(to, __uint_as_float(r[e]));
      store_cluster(to + L::kPitch * 4, __uint_as_float(r[e + 1]));
    }
  }
  tc_fence_before();
  __syncwarp();
  if (lane < shares) arrive_cluster(map_cluster(smem_u32(sums_full), lane));
  mbar_wait_cluster(sums_full, 0, &no_abort, &g_status);
  const uint8_t* sums = smem + L::kSumsOff;
#pragma unroll 1
  for (int r = r0; r < mine; r += kRowsThreads / (kRowsN / 8)) {
    const uint4 now = res;
    res = residual(r + kRowsThreads / (kRowsN / 8));
    if (n8 >= p.N) continue;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < shares; ++s) {
      const float4* src = reinterpret_cast<const float4*>(sums + ((s * slice + r) * L::kPitch + c8) * 4);
      const float4 a = src[0], b = src[1];
      v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
      v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    }
    *reinterpret_cast<uint4*>(static_cast<T*>(p.Y) + at(r)) = finish8<T>(p, bias, v, now);
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

template <class T, int RB>
cudaError_t start_rows(const DenseParams& p, const DenseMaps& maps, int sms, cudaStream_t st) {
  using L = RowsSmem<RB>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(dense_rows_kernel<T, RB>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
  });
  if (e != cudaSuccess) return e;
  const int tiles_n = (p.N + kRowsN - 1) / kRowsN, tiles_m = (p.M + RB - 1) / RB;
  // shares of K while they find free SMs and keep four blocks of K each
  const int room = (RB == 128 ? 1 : 2) * sms, blocks = (p.K + kBK - 1) / kBK;
  int share_bits = 0;
  while (share_bits < 3 && (2ll << share_bits) * tiles_n * tiles_m <= room && blocks >= 8 << share_bits) ++share_bits;
  const int shares = 1 << share_bits;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(tiles_n * shares, tiles_m);
  cfg.blockDim = dim3(kRowsThreads);
  cfg.dynamicSmemBytes = L::kTotal;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = shares;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dense_rows_kernel<T, RB>, p, maps, share_bits);
}

// ---------------------------------------------------------------- pair kernel
constexpr int kPairM = 256;                // rows of a pair's tile; it has NT columns, 256 or 128
constexpr int kEpiWarps = 8;               // two per quarter of the lanes, half the columns each
constexpr int kPairThreads = (2 + kEpiWarps) * 32;
constexpr int kGroupM = 16;                // row blocks that share the column blocks of W in L2

template <int NT>
struct PairSmem {
  static constexpr int kX = 128 * kBK * 2;  // this CTA's rows
  static constexpr int kW = kBK * NT;       // this CTA's columns, half of the tile's
  static constexpr int kStage = kX + kW;
  static constexpr int kStages = NT == 256 ? 6 : 8;
  static constexpr int kBox = 32 * 64;      // Y on its way out: 32 rows, 32 columns
  static constexpr int kBoxes = kStages * kStage;
  static constexpr int kBars = kBoxes + kEpiWarps * 2 * kBox;
  static constexpr int kTotal = kBars + 512 + 1024;
};
static_assert(PairSmem<256>::kTotal <= 232448 && PairSmem<128>::kTotal <= 232448, "shared memory budget");

// The CTAs of a pair meet. Nothing is published here: the releasing form waits for
// all that the thread has written, 1100 cycles where this takes 300.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}
// An arrival that publishes nothing either (accumulators that have been read):
// 1500 cycles less than the releasing form.
__device__ __forceinline__ void arrive_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void pair_tile(int tile, int m_blocks, int n_blocks, int& mb, int& nb) {
  const int group = tile / (kGroupM * n_blocks), first = group * kGroupM, in = tile % (kGroupM * n_blocks);
  const int size = min(kGroupM, m_blocks - first);
  mb = first + in % size;
  nb = in / size;
}

template <class T, int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    dense_pair_kernel(const DenseParams p, const __grid_constant__ DenseMaps maps) {
  using L = PairSmem<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);  // [kStages] (leader) both CTAs' loads have landed
  uint64_t* empty = full + L::kStages;                            // [kStages] (both) the MMAs are done with the stage
  uint64_t* acc_full = empty + L::kStages;                        // [2] (both) a tile's sums are complete
  uint64_t* acc_empty = acc_full + 2;                             // [2] (leader) both CTAs have read them
  uint64_t* drain = acc_empty + 2;                                // (both) every MMA has completed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = warp_id(), lane = lane_id();
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int m_blocks = (p.M + kPairM - 1) / kPairM, n_blocks = (p.N + NT - 1) / NT;
  const int tiles = m_blocks * n_blocks, pairs = gridDim.x >> 1;
  const int blocks = (p.K + kBK - 1) / kBK;
  int mb, nb;  // of the first tile, before there is anything to wait for
  pair_tile(blockIdx.x >> 1, m_blocks, n_blocks, mb, nb);

  if (warp == 2 && lane < 3) prefetch_tensormap(lane == 0 ? &maps.x : lane == 1 ? &maps.w : &maps.y);
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 2 * NT);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_meet();  // the barriers are there: fence_barrier_init has published them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // -------------------------------------------------------------- loads (both CTAs)
    if (lane == 0) {
      bool ok = true;
      uint32_t it = 0;
      for (int tile = blockIdx.x >> 1; tile < tiles && ok; tile += pairs) {
        if (it > 0) pair_tile(tile, m_blocks, n_blocks, mb, nb);
        const int m = mb * kPairM + static_cast<int>(rank) * 128, n = nb * NT + static_cast<int>(rank) * (NT / 2);
        for (int k = 0; k < blocks; ++k, ++it) {
          const int s = it % L::kStages;
          ok = mbar_wait(&empty[s], ((it / L::kStages) & 1) ^ 1, abort_flag, &g_status);
          if (!ok) break;
          uint8_t* st = smem + s * L::kStage;
          const uint32_t bar = leader_addr(&full[s]);
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * L::kStage);
          tma_load_2d_pair(st, &maps.x, bar, k * kBK, m);
          tma_load_2d_pair(st + L::kX, &maps.w, bar, n, k * kBK);
          if (NT == 256) tma_load_2d_pair(st + L::kX + 8192, &maps.w, bar, n + 64, k * kBK);
        }
      }
      if (!ok && leader) {  // gave up: the pair's copies in flight land before it ends
        volatile int no_abort = 0;
        for (uint32_t e = it > L::kStages ? it - L::kStages : 0; e < it; ++e)
          mbar_wait(&full[e % L::kStages], (e / L::kStages) & 1, &no_abort, nullptr);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMAs (leader)
    // The whole warp goes through the loops, one lane issues: what an MMA reads then
    // stays in uniform registers.
    if (leader) {
      // B: W, NT columns over the pair, N-major (bit 16)
      const uint32_t idesc = idesc_dense(kFmtF32, Half16<T>::kFmt, Half16<T>::kFmt, kPairM, NT) | (1u << 16);
      const bool issues = elect_one();
      const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0), ring = smem_u32(smem);
      auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, abort_flag, &g_status); };
      bool ok = true;
      uint32_t it = 0;
      int ti = 0;
      for (int tile = blockIdx.x >> 1; tile < tiles && ok; tile += pairs, ++ti) {
        const int b = ti & 1;
        ok = wait(&acc_empty[b], ((ti >> 1) & 1) ^ 1);
        if (!ok) break;
        tc_fence_after();
        for (int k = 0; k < blocks; ++k, ++it) {
          const int s = it % L::kStages;
          ok = wait(&full[s], (it / L::kStages) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t xa = ring + s * L::kStage, wb = xa + L::kX;
          if (issues) {
#pragma unroll
            for (int e = 0; e < kBK / 16; ++e)
              mma_f16_pair(base + b * NT, smem_desc(xa + 32 * e, 16, 1024, kSw128), smem_desc(wb + 2048 * e, 8192, 1024, kSw128),
                           idesc, (k > 0 || e > 0) ? 1u : 0u);
            tc_commit_pair_mc(&empty[s], 0x3);
          }
        }
        if (ok && issues) tc_commit_pair_mc(&acc_full[b], 0x3);
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- epilogue (both CTAs)
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* box = smem + L::kBoxes + (warp - 2) * 2 * L::kBox;
    const T *bias = static_cast<const T*>(p.bias), *residual = static_cast<const T*>(p.residual);
    int ti = 0;
    for (int tile = blockIdx.x >> 1; tile < tiles; tile += pairs, ++ti) {
      if (ti > 0) pair_tile(tile, m_blocks, n_blocks, mb, nb);
      const int buf = ti & 1, row0 = mb * kPairM + static_cast<int>(rank) * 128 + 32 * q, row = row0 + lane;
      const int col0 = nb * NT + half * (NT / 2);
      const uint32_t acc = tmem + (static_cast<uint32_t>(32 * q) << 16) + buf * NT + half * (NT / 2);
      // a lane holds the bias of NT / 64 columns; shuffles bring them where they are added
      constexpr int kWords = NT / 128;
      uint32_t bias_words[kWords] = {};
      const int bias_col = col0 + 2 * kWords * lane;
      if (bias && bias_col < p.N) {
        if constexpr (kWords == 2) {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(bias + bias_col));
          bias_words[0] = w.x, bias_words[1] = w.y;
        } else {
          bias_words[0] = __ldg(reinterpret_cast<const uint32_t*>(bias + bias_col));
        }
      }
      uint4 r4[4] = {};  // the residual of the next 32 columns
      auto fetch = [&](int c) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int n = col0 + c + 8 * v;
          if (residual && row < p.M && n < p.N) r4[v] = __ldcs(reinterpret_cast<const uint4*>(residual + static_cast<size_t>(row) * p.N + n));
        }
      };
      fetch(0);
      if (!warp_wait(&acc_full[buf], (ti >> 1) & 1, abort_flag, &g_status)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < NT / 2; c += 32) {
        uint32_t a[32];
        tmem_ld32(acc + c, a);
        const uint4 r[4] = {r4[0], r4[1], r4[2], r4[3]};
        if (c + 32 < NT / 2) fetch(c + 32);
        tmem_ld_wait();
        if (c + 32 == NT / 2 && tile + 2 * pairs < tiles) {  // the sums are in registers: the next tile but one may start
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_relaxed(leader_addr(&acc_empty[buf]));
        }
        float2 v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = make_float2(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1]));
        if (bias) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            v[e] = __fadd2_rn(v[e], unpack<T>(__shfl_sync(0xffffffffu, bias_words[e % kWords], c / (2 * kWords) + e / kWords)));
        }
        activate(v, p.act);
        if (residual) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint4 w = r[e >> 2];
            v[e] = __fadd2_rn(v[e], unpack<T>((e & 3) == 0 ? w.x : (e & 3) == 1 ? w.y : (e & 3) == 2 ? w.z : w.w));
          }
        }
        uint8_t* out = box + ((c >> 5) & 1) * L::kBox + lane * 64;
        if (lane == 0) bulk_wait_group_read<1>();  // the store before the last has read this box
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(out + ((e ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(Half16<T>::pack(v[4 * e].x, v[4 * e].y), Half16<T>::pack(v[4 * e + 1].x, v[4 * e + 1].y),
                         Half16<T>::pack(v[4 * e + 2].x, v[4 * e + 2].y), Half16<T>::pack(v[4 * e + 3].x, v[4 * e + 3].y));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (row0 < p.M && col0 + c < p.N) tma_store_2d(&maps.y, box + ((c >> 5) & 1) * L::kBox, col0 + c, row0);
          bulk_commit_group();  // an empty one too: the waits above count groups
        }
      }
    }
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
  }

  // Neither CTA leaves, or frees its tensor memory, while the other can still be
  // signalled or read by the pair's MMAs. What one CTA signals to the other is waited
  // for there before it comes here, unless a wait was given up.
  if (warp == 1 && leader && lane == 0) tc_commit_pair_mc(drain, 0x3);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    volatile int no_abort = 0;
    warp_wait(drain, 0, &no_abort, nullptr);
  }
  tc_fence_before();
  if (*abort_flag) asm volatile("fence.acq_rel.cluster;" ::: "memory");
  cluster_meet();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * NT);
  }
}

template <class T, int NT>
cudaError_t start_pair(const DenseParams& p, const DenseMaps& maps, int sms, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(dense_pair_kernel<T, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, PairSmem<NT>::kTotal);
  });
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>((p.M + kPairM - 1) / kPairM) * ((p.N + NT - 1) / NT);
  dense_pair_kernel<T, NT><<<2 * static_cast<int>(std::min<long long>(tiles, sms / 2)), kPairThreads, PairSmem<NT>::kTotal, st>>>(p, maps);
  return cudaGetLastError();
}

template <class T>
svdq_status run(const DenseParams& p, const void* X, const void* W, cudaStream_t st) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return fail(SVDQ_ERR_CUDA, "no usable current device");
  const CUtensorMapDataType dt = Half16<T>::kFmt == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  // The rows kernel where its 128 x 128 tiles leave so many SMs free that it can cut
  // K (256 x 3072 x 3072: 15.0 us, a pair's tiles 16); then tiles of 128 columns
  // while all pairs' tiles run at once (256 x 3072 x 9216: 17 us, 256 columns 21, the
  // rows kernel 24), of 256 when not (256 x 3072 x 12288: 22 us, 128 columns 28; rows 43).
  const long long tiles = static_cast<long long>((p.M + kPairM - 1) / kPairM) * ((p.N + 127) / 128);
  const bool pair = p.M > 128 && 4 * tiles > sms, wide = tiles > sms / 2;
  const int rb = pair ? 128 : p.M <= 16 ? 16 : p.M <= 32 ? 32 : p.M <= 64 ? 64 : 128;
  DenseMaps maps{};
  if (!make_map(&maps.x, dt, X, p.K, p.M, static_cast<uint64_t>(p.K) * 2, kBK, rb, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&maps.w, dt, W, p.N, p.K, static_cast<uint64_t>(p.N) * 2, 64, kBK, CU_TENSOR_MAP_SWIZZLE_128B) ||
      (pair && !make_map(&maps.y, dt, p.Y, p.N, p.M, static_cast<uint64_t>(p.N) * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B)))
    return fail(SVDQ_ERR_CUDA, "cuTensorMapEncodeTiled (dense linear) failed");
  const cudaError_t e = pair       ? wide ? start_pair<T, 256>(p, maps, sms, st) : start_pair<T, 128>(p, maps, sms, st)
                        : rb == 16 ? start_rows<T, 16>(p, maps, sms, st)
                        : rb == 32 ? start_rows<T, 32>(p, maps, sms, st)
                        : rb == 64 ? start_rows<T, 64>(p, maps, sms, st)
                                   : start_rows<T, 128>(p, maps, sms, st);
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, std::string("dense linear kernel: ") + cudaGetErrorString(e));
  return SVDQ_OK;
}

}  // namespace

namespace svdq {
cudaError_t take_status_dense(int* status, cudaStream_t st) { return take_status(status, st); }
cudaError_t give_up_dense(cudaStream_t st) { return give_up(st); }
}  // namespace svdq

extern "C" svdq_status svdq_dense_linear_forward(const svdq_dense_linear_args* a, void* stream) {
  if (!a) return fail(SVDQ_ERR_INVALID_ARG, "args is NULL");
  if (a->dtype != SVDQ_BF16 && a->dtype != SVDQ_F16) return fail(SVDQ_ERR_INVALID_ARG, "unknown dtype");
  if (a->activation < SVDQ_ACT_NONE || a->activation > SVDQ_ACT_GELU_TANH) return fail(SVDQ_ERR_INVALID_ARG, "unknown activation");
  if (a->M < 0 || a->K <= 0 || a->N <= 0 || a->K % 8 || a->N % 8)
    return fail(SVDQ_ERR_INVALID_ARG, "M must not be negative, K and N positive multiples of 8");
  if (a->M > 1 << 22 || a->K > 1 << 22 || a->N > 1 << 22) return fail(SVDQ_ERR_UNSUPPORTED, "M, K or N exceeds 4194304");
  if (a->M == 0) return SVDQ_OK;
  if (!a->X || !a->W || !a->Y) return fail(SVDQ_ERR_INVALID_ARG, "X, W or Y is NULL");
  uintptr_t bits = 0;
  for (const void* q : {a->X, a->W, a->bias, a->residual, static_cast<const void*>(a->Y)}) bits |= reinterpret_cast<uintptr_t>(q);
  if (bits & 15) return fail(SVDQ_ERR_INVALID_ARG, "device pointers must be 16-byte aligned");
  const DenseParams p{a->bias, a->residual, a->Y, a->M, a->N, a->K, a->activation};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a->dtype == SVDQ_BF16 ? run<__nv_bfloat16>(p, a->X, a->W, st) : run<__half>(p, a->X, a->W, st);
}
