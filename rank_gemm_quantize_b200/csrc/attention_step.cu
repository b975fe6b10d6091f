// Attention of few queries per sequence (single new tokens, short pieces): the
// keys and values are read once at memory speed, split over the SMs along the
// sequence and joined by a second kernel.
//
// The query heads of a key head and the queries of a sequence form one list of
// rows (row = query * group + head), cut into tiles of 16. A CTA of four warps
// takes parts of 16 rows, one key head and some of the keys, one after another: an
// equal stretch of the call's work (Line).
// TMA brings 64 keys and values at a time into a ring of stages; each warp
// takes 16 of them: scores by mma.m16n8k16, softmax statistics and the product
// with V in registers, with no exchange between warps until the part's end. The
// parts' results (unnormalised float sums, maximum, sum) go to the workspace, or
// straight to the output where a row tile is one part. The probabilities are rounded
// to 16 bits for the product with V, which takes nothing wider; the sums take them
// unrounded, and in fp16 one under 2^-25 of the warp's largest becomes 0. A call of so few and
// short sequences that eight CTAs an item are all there is to gain takes one
// launch: the eight are a cluster, cut the keys evenly and join their results
// through distributed shared memory.
//
// Memory bounds it: 4 dim bytes a key and key head (64 sequences of 200 to 16000
// keys, 8 key heads of 128, 973 MB: 156 us with the join, 6.2 TB/s, 95% of a copy's
// rate); 16 rows cost a fraction of the tensor pipe, which is why the narrow mma is
// used here and a 128-row tensor-memory tile would only add latency. A lone
// token is latency (777 keys, 4 key heads of 128: 6.1 us on the device; as stretches
// and a join, two launches, 11.4 us).
#include <string>

#include "attention.cuh"
#include "operator_status.cuh"

using namespace svdq;

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;

template <int DP>
struct StepSmem {
  static constexpr int kTile = kStepKeys * DP * 2;  // keys, or values
  static constexpr int kStage = 2 * kTile;
  static constexpr int kStages = 96 * 1024 / kStage;  // 96 KB of loads: two CTAs an SM
  static constexpr int kPitch = DP + 4;               // floats of a row when the warps' sums are joined
  // results of the cluster's CTAs for the two rows that this one finishes
  static constexpr int kOwnRows = kStepRows / kStepCluster;
  static constexpr int kSums = kStages * kStage;
  static constexpr int kBars = kSums + kStepCluster * kOwnRows * kPitch * 4;
  static constexpr int kTotal = kBars + 256 + 1024;
  static_assert(kWarps * kStepRows * kPitch * 4 <= kStages * kStage, "the join reuses the stages");
};

__device__ __forceinline__ void ldsm(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <class T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (Half16<T>::kFmt == 1)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte piece `piece` of row `key` in a swizzled tile of 64
// rows: columns of 64 values (128 bytes) side by side.
__device__ __forceinline__ uint32_t tile_at(int key, int piece) {
  return (piece >> 3) * (kStepKeys * 128) + key * 128 + (((piece & 7) ^ (key & 7)) << 4);
}

__device__ __forceinline__ uint32_t map_cluster(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

template <class T, int DP, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2) attention_step_kernel(const AttnParams p, const __grid_constant__ AttnMaps maps) {
  using L = StepSmem<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* empty = full + L::kStages;
  __shared__ int sums[kWarps];
  __shared__ Found found;
  __shared__ long long line_sums[kWarps][2];
  __shared__ Part line_part;
  __shared__ int spoiled;
  __shared__ int abort_word;
  __shared__ float warp_ml[kWarps][kStepRows][2];
  __shared__ float2 share_ml[kStepCluster][L::kOwnRows];
  volatile int* abort_flag = &abort_word;

  const int tid = threadIdx.x, warp = warp_id(), lane = lane_id();
  const int g = lane >> 2, t = lane & 3;
  const int hk = blockIdx.y;
  if (tid == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    abort_word = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (CLUSTER) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  // the thread that notes for the join what this CTA has the second part of
  const bool notes = !CLUSTER && p.max_slots && hk == 0 && tid == kThreads - 32;
  Line line{};
  LineSearch along{0, 0};
  long long x = 0, x_end = 0;  // this CTA's stretch of the line
  if (!CLUSTER) {
    line = line_of<kWarps>(p, line_sums);
    if (notes) p.cuts[blockIdx.x] = Cut{};
    if (static_cast<int>(blockIdx.x) >= line.ctas) return;
    x = line.begin(blockIdx.x), x_end = line.begin(blockIdx.x + 1);
  }
  uint32_t used = 0;    // key tiles since the kernel's start
  uint32_t issued = 0;  // ... and how many of them thread 0 has asked for
  Search at{0, 0, p.chunk};
  for (int item = blockIdx.x / kStepCluster;; item += gridDim.x) {
    Found f{};
    Part part{};
    int first = 0, length = 0;  // key tiles of this part
    if (CLUSTER) {
      if (!find_item<kWarps>(p, at, item, &found, sums, &f)) {  // a cluster's CTAs alike
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        return;
      }
    } else {
      if (x >= x_end) return;
      part = part_at<kWarps>(p, along, x, &line_part, line_sums);
      const int end = static_cast<int>(min(static_cast<long long>(part.tiles + Line::kEnds), part.place + x_end - x));
      x += end - part.place;
      first = max(0, part.place - Line::kEnds);
      length = end - Line::kEnds - first;
      if (length <= 0) continue;  // the unit's key tiles are the next CTA's
      f.b = part.b;
      f.tile = part.unit;
    }
    int qs, ql, ks, kl;
    seq_extent(p.q_offsets, f.b, p.q_rows, qs, ql);
    seq_extent(p.k_offsets, f.b, p.k_rows, ks, kl);
    const int rows = ql * p.group;
    const int row0 = f.tile * kStepRows;
    // keys [k_begin, k_end) of this share; row r sees keys <= limit(r)
    auto limit = [&](int row) {
      return row < rows ? last_key(p, row, ql, kl) : -1;
    };
    const int seen = limit(min(row0 + kStepRows, rows) - 1) + 1;  // keys that some row sees
    int k_begin, k_end;
    if (CLUSTER) {
      const int all = (max(seen, 0) + kStepKeys - 1) / kStepKeys, share = blockIdx.x % kStepCluster;
      k_begin = all * share / kStepCluster * kStepKeys;
      k_end = min(all * (share + 1) / kStepCluster * kStepKeys, seen);
    } else {
      k_begin = first * kStepKeys;
      k_end = min((first + length) * kStepKeys, seen);
    }
    const int first_limit = limit(row0);
    const int tiles = k_end > k_begin ? (k_end - k_begin + kStepKeys - 1) / kStepKeys : 0;

    auto issue = [&](int i) {  // one thread: key tile i of this item
      const int s = (used + i) % L::kStages;
      uint8_t* st = smem + s * L::kStage;
      mbar_arrive_expect_tx(&full[s], L::kStage);
      const int key = ks + k_begin + i * kStepKeys;
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        tma_load_3d(st + c * kStepKeys * 128, &maps.k, &full[s], c * 64, hk, key);
        tma_load_3d(st + L::kTile + c * kStepKeys * 128, &maps.v, &full[s], c * 64, hk, key);
      }
    };
    if (tid == 0) {
      spoiled = 0;
      // every stage is free: the last item's tiles were all used
      for (int i = 0; i < min(tiles, L::kStages); ++i) issue(i);
    }
    issued = used + min(tiles, L::kStages);
    if (notes && first > 0) {
      const long long begin = line.begin(blockIdx.x) - first;  // of the unit's key tiles
      const int cta = line.cta_of(begin);
      if (cta + 1 == static_cast<int>(blockIdx.x))
        p.cuts[blockIdx.x] = {part.unit, cta, line.cta_of(begin + part.tiles - 1) - cta + 1, part.b, qs, ql, kl, 0};
    }

    // the rows' queries as mma operands
    uint32_t qf[DP / 16][4];
    {
      const T* qb = static_cast<const T*>(p.q);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = row0 + g + 8 * h;
        const bool in = row < rows;
        const T* src = qb + static_cast<long long>(qs + (in ? row / p.group : 0)) * p.q_row +
                       (hk * p.group + (in ? row % p.group : 0)) * p.q_head;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int col = 16 * k + 8 * w + 2 * t;
            qf[k][h + 2 * w] = in && col < p.dim ? *reinterpret_cast<const uint32_t*>(src + col) : 0u;
          }
      }
    }
    const int lim[2] = {limit(row0 + g), limit(row0 + g + 8)};
    float o[DP / 8][4];
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    int i = 0;
    for (; i < tiles; ++i) {
      const uint32_t n = used + i;
      const int s = n % L::kStages;
      if (!warp_wait(&full[s], (n / L::kStages) & 1, abort_flag, &g_status)) break;
      uint8_t* st = smem + s * L::kStage;
      const uint32_t kt = smem_u32(st), vt = kt + L::kTile;
      const int key0 = k_begin + i * kStepKeys + 16 * warp;  // the warp's 16 keys
      // Values of keys that no row sees, or not every row, must not meet the
      // product (0 times infinity): keys behind the sequence become 0;
      // infinities and NaN of the others become 0 here and are put back into
      // the rows that do see them at the end.
      if (key0 + 15 > first_limit) {
        bool any = false;
        for (int e = lane; e < 16 * (DP / 8); e += 32) {
          const int r = e / (DP / 8), key = key0 + r;
          if (key <= first_limit) continue;
          uint4* at16 = reinterpret_cast<uint4*>(st + L::kTile + tile_at(16 * warp + r, e % (DP / 8)));
          uint4 v = *at16;
          if (key >= kl)
            *at16 = make_uint4(0, 0, 0, 0);
          else if (has_non_finite<T>(v)) {
            drop_non_finite<T>(v);
            *at16 = v, any = true;
          }
        }
        if (any) spoiled = 1;
        fence_proxy_async_smem();  // the stage is loaded again by TMA
        __syncwarp();
      }
      float sc[2][4];
#pragma unroll
      for (int a = 0; a < 2; ++a) sc[a][0] = sc[a][1] = sc[a][2] = sc[a][3] = 0.f;
      {
        const int mtx = lane >> 3, key = 16 * warp + (mtx >> 1) * 8 + (lane & 7);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          uint32_t b[4];
          ldsm(kt + tile_at(key, 2 * k + (mtx & 1)), b);
          mma16816<T>(sc[0], qf[k], b[0], b[1]);
          mma16816<T>(sc[1], qf[k], b[2], b[3]);
        }
      }
      float corr[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float top = m[h];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = sc[a][2 * h + e];
            if (key0 + 8 * a + 2 * t + e > lim[h]) x = -INFINITY;
            top = fmaxf(top, x);
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float base = (top == -INFINITY ? 0.f : top) * p.scale_log2;
        corr[h] = exp2_fast(fmaf(m[h], p.scale_log2, -base));
        m[h] = top;
        float sum = 0.f;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = sc[a][2 * h + e];
            x = exp2_fast(fmaf(x, p.scale_log2, -base));
            sum += x;
          }
        l[h] = fmaf(l[h], corr[h], sum);
      }
#pragma unroll
      for (int n8 = 0; n8 < DP / 8; ++n8) {
        o[n8][0] *= corr[0];
        o[n8][1] *= corr[0];
        o[n8][2] *= corr[1];
        o[n8][3] *= corr[1];
      }
      const uint32_t pf[4] = {Half16<T>::pack(sc[0][0], sc[0][1]), Half16<T>::pack(sc[0][2], sc[0][3]),
                              Half16<T>::pack(sc[1][0], sc[1][1]), Half16<T>::pack(sc[1][2], sc[1][3])};
      {
        const int mtx = lane >> 3, key = 16 * warp + (mtx & 1) * 8 + (lane & 7);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          uint32_t b[4];
          ldsm_t(vt + tile_at(key, 2 * k + (mtx >> 1)), b);
          mma16816<T>(o[2 * k], pf, b[0], b[1]);
          mma16816<T>(o[2 * k + 1], pf, b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      if (tid == 0 && i + L::kStages < tiles && mbar_wait(&empty[s], (n / L::kStages) & 1, abort_flag, &g_status)) {
        issue(i + L::kStages);
        ++issued;
      }
    }
    __syncwarp();
    // the row sums over the four threads of a row
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    __syncthreads();  // every warp is done with the stages
    if (*abort_flag) {  // a wait gave up: let the copies in flight land, then leave
      if (tid == 0) {
        volatile int no_abort = 0;
        for (uint32_t n = issued > L::kStages ? issued - L::kStages : 0; n < issued; ++n)
          mbar_wait(&full[n % L::kStages], (n / L::kStages) & 1, &no_abort, nullptr);
      }
      if (!CLUSTER) return;  // a cluster's CTAs meet below, whatever their results are worth
      __syncthreads();
    }
    used += tiles;
    // join the warps: each row's maximum, sum and products
    float* join = reinterpret_cast<float*>(smem);
    if (t == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        warp_ml[warp][g + 8 * h][0] = m[h];
        warp_ml[warp][g + 8 * h][1] = l[h];
      }
    }
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(join + (warp * kStepRows + g + 8 * h) * L::kPitch + 8 * n + 2 * t) =
            make_float2(o[n][2 * h], o[n][2 * h + 1]);
    __syncthreads();
    const int r = tid >> 3, row = row0 + r;
    if (CLUSTER) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the cluster runs
    if (row < rows) {
      float top = -INFINITY, total = 0.f, w[kWarps];
#pragma unroll
      for (int a = 0; a < kWarps; ++a) top = fmaxf(top, warp_ml[a][r][0]);
      const float base = (top == -INFINITY ? 0.f : top) * p.scale_log2;
#pragma unroll
      for (int a = 0; a < kWarps; ++a) {
        w[a] = exp2_fast(fmaf(warp_ml[a][r][0], p.scale_log2, -base));
        total = fmaf(warp_ml[a][r][1], w[a], total);
      }
      const bool split = CLUSTER || length < part.tiles;
      const int row_limit = limit(row);
      const float norm = split ? 1.f : row_norm(total, [&] { return row_limit; });
      const int share = 2 * blockIdx.x + (first == 0);
      const size_t slot = (static_cast<size_t>(share) * p.kv_heads + hk) * kStepRows + r;
      const bool fits = share < p.max_slots;
      const int owner = r / L::kOwnRows, slot_row = blockIdx.x % kStepCluster * L::kOwnRows + r % L::kOwnRows;
      const uint32_t to = CLUSTER ? map_cluster(smem_u32(smem + L::kSums) + slot_row * (L::kPitch * 4), owner) : 0;
#pragma unroll
      for (int c0 = 0; c0 < DP; c0 += 32) {
        const int c = c0 + (tid & 7) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int a = 0; a < kWarps; ++a) {
          const float4 v = *reinterpret_cast<const float4*>(join + (a * kStepRows + r) * L::kPitch + c);
          acc.x = fmaf(v.x, w[a], acc.x);
          acc.y = fmaf(v.y, w[a], acc.y);
          acc.z = fmaf(v.z, w[a], acc.z);
          acc.w = fmaf(v.w, w[a], acc.w);
        }
        if (spoiled && c < p.dim) {
          for (int key = max(k_begin, first_limit + 1); key < min(k_end, row_limit + 1); ++key) {
            const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const T*>(p.v) + static_cast<long long>(ks + key) * p.v_row +
                                                            hk * p.v_head + c);
            const uint32_t e[4] = {v.x & 0xFFFFu, v.x >> 16, v.y & 0xFFFFu, v.y >> 16};
            float* x = &acc.x;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if ((e[j] & Half16<T>::kExp) == Half16<T>::kExp) x[j] += Half16<T>::to_float(e[j]);
          }
        }
        if (CLUSTER) {
          asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to + c * 4), "f"(acc.x), "f"(acc.y), "f"(acc.z), "f"(acc.w)
                       : "memory");
        } else if (split) {
          if (fits) *reinterpret_cast<float4*>(p.part + slot * DP + c) = acc;
        } else if (c < p.dim) {
          uint2 v;
          v.x = Half16<T>::pack(acc.x * norm, acc.y * norm);
          v.y = Half16<T>::pack(acc.z * norm, acc.w * norm);
          *reinterpret_cast<uint2*>(static_cast<T*>(p.out) +
                                    (static_cast<size_t>(qs + row / p.group) * p.q_heads + hk * p.group + row % p.group) * p.dim + c) = v;
        }
      }
      if (CLUSTER) {
        if ((tid & 7) == 0)
          asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(map_cluster(smem_u32(&share_ml[0][0]) + slot_row * 8, owner)),
                       "f"(top), "f"(total)
                       : "memory");
      } else if (split && fits && (tid & 7) == 0) {
        *reinterpret_cast<float2*>(p.part_ml + 2 * slot) = make_float2(top, total);
      }
    }
    if (CLUSTER) {
      cluster_sync_all();  // the rows of this CTA have arrived from all eight
      constexpr int kThreadsRow = kThreads / L::kOwnRows, kCols = DP / kThreadsRow;
      const int own = tid / kThreadsRow, c = tid % kThreadsRow * kCols, mine = row0 + blockIdx.x % kStepCluster * L::kOwnRows + own;
      if (mine < rows && c < p.dim) {
        float top = -INFINITY, total = 0.f, o[kCols] = {};
#pragma unroll
        for (int s = 0; s < kStepCluster; ++s) top = fmaxf(top, share_ml[s][own].x);
        const float base = (top == -INFINITY ? 0.f : top) * p.scale_log2;
#pragma unroll
        for (int s = 0; s < kStepCluster; ++s) {
          const float2 ml = share_ml[s][own];
          const float w = exp2_fast(fmaf(ml.x, p.scale_log2, -base));
          total = fmaf(ml.y, w, total);
#pragma unroll
          for (int e = 0; e < kCols; ++e)
            o[e] = fmaf(reinterpret_cast<const float*>(smem + L::kSums)[(s * L::kOwnRows + own) * L::kPitch + c + e], w, o[e]);
        }
        const float norm = row_norm(total, [&] { return limit(mine); });
        T* out = static_cast<T*>(p.out) + (static_cast<size_t>(qs + mine / p.group) * p.q_heads + hk * p.group + mine % p.group) * p.dim + c;
        if constexpr (kCols == 2)
          *reinterpret_cast<uint32_t*>(out) = Half16<T>::pack(o[0] * norm, o[1] * norm);
        else
          *reinterpret_cast<uint16_t*>(out) = static_cast<uint16_t>(Half16<T>::pack(o[0] * norm, 0.f));
      }
      return;
    }
    fence_proxy_async_smem();  // the stages are loaded again by TMA
    __syncthreads();
  }
}

// A warp's part of a row's softmax over partial results: every STEP-th of them from
// `from` on, the slot of each by slot_of. A lane holds DP / 32 columns.
template <int DP>
struct Joined {
  static constexpr int kPer = DP / 32;
  float top = -INFINITY, total = 0.f, o[kPer] = {};
  __device__ __forceinline__ void add(float ml_top, float ml_total, const float (&v)[kPer], float scale_log2) {
    const float now = fmaxf(top, ml_top), base = (now == -INFINITY ? 0.f : now) * scale_log2;
    const float was = exp2_fast(fmaf(top, scale_log2, -base)), w = exp2_fast(fmaf(ml_top, scale_log2, -base));
    top = now;
    total = fmaf(total, was, ml_total * w);
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = fmaf(o[e], was, v[e] * w);
  }
  template <int STEP, class SlotOf>
  __device__ __forceinline__ void gather(const AttnParams& p, int from, int shares, SlotOf slot_of) {
#pragma unroll 8
    for (int c = from; c < shares; c += STEP) {
      const size_t slot = slot_of(c);
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * slot);
      float v[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[e] = p.part[slot * DP + kPer * lane_id() + e];
      add(ml.x, ml.y, v, p.scale_log2);
    }
  }
  // row of a sequence of ql queries, which start at qs, and kl keys
  template <class T>
  __device__ __forceinline__ void store(const AttnParams& p, int qs, int ql, int kl, int hk, int row) const {
    const float norm = row_norm(total, [&] { return last_key(p, row, ql, kl); });
    const int c = kPer * lane_id();
    if (c >= p.dim) return;
    T* out = static_cast<T*>(p.out) + (static_cast<size_t>(qs + row / p.group) * p.q_heads + hk * p.group + row % p.group) * p.dim + c;
    if constexpr (kPer == 4)
      *reinterpret_cast<uint2*>(out) = make_uint2(Half16<T>::pack(o[0] * norm, o[1] * norm), Half16<T>::pack(o[2] * norm, o[3] * norm));
    else
      *reinterpret_cast<uint32_t*>(out) = Half16<T>::pack(o[0] * norm, o[1] * norm);
  }
};

// Joins the shares of attention_prompt.cu, of up to 32 sequences (key_chunk). CTA (b, key
// head, z) takes four rows at a time, 4 z .., 4 (z + gridDim.z) .., a warp each.
template <class T, int DP>
__global__ void __launch_bounds__(128) attention_join_kernel(const AttnParams p) {
  __shared__ Shares own;
  __shared__ int own_before;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the kernel before has ended
  const int b = blockIdx.x, hk = blockIdx.y, warp = warp_id(), lane = lane_id();
  int qs, ql, ks, kl;
  seq_extent(p.q_offsets, b, p.q_rows, qs, ql);
  seq_extent(p.k_offsets, b, p.k_rows, ks, kl);
  // the sequence's shares and the slots before its own: by the first warp, since the
  // others have the same to find
  if (warp == 0) {
    const int chunk = key_chunk(p);
    const Shares s = shares_of(p, b, chunk);
    const int before = __reduce_add_sync(0xffffffffu, lane < b ? shares_of(p, lane, chunk).slots : 0);
    if (lane == 0) own = s, own_before = before;
  }
  __syncthreads();
  const Shares s = own;
  if (!s.slots || own_before + s.slots > p.max_slots) return;
  for (int row = 4 * blockIdx.z + warp; row < ql * p.group; row += 4 * gridDim.z) {
    const int first = own_before + row / p.tile_rows * s.chunks;
    Joined<DP> joined;
    joined.template gather<1>(p, 0, s.chunks, [&](int c) {
      return (static_cast<size_t>(first + c) * p.kv_heads + hk) * p.tile_rows + row % p.tile_rows;
    });
    joined.template store<T>(p, qs, ql, kl, hk, row);
  }
}

// Joins the parts of attention_step_kernel's units: CTA (x, key head, z) those that CTA
// x + 1 there has noted, ROWS rows at a time, ROWS z .., ROWS (z + gridDim.z) .., each by
// 16 / ROWS warps. (A CTA for each sequence and row, which all look for their unit: 4000
// tokens on 200 keys, 8 key heads, 1790 us for 820; one CTA a beginning of a stretch
// that looks for the unit there: 16 tokens 14.7 us.)
constexpr int kJoinWarps = 16;
template <class T, int DP, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32) attention_line_join_kernel(const AttnParams p) {
  constexpr int kSplit = kJoinWarps / ROWS;
  __shared__ float2 warp_ml[kJoinWarps];
  __shared__ float warp_o[kJoinWarps][DP];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the kernel before has ended
  const int hk = blockIdx.y, warp = warp_id(), lane = lane_id();
  const Cut cut = p.cuts[blockIdx.x + 1];
  if (!cut.shares) return;
  const int row0 = cut.unit * kStepRows, rows = min(kStepRows, cut.ql * p.group - row0);
  constexpr int kPer = Joined<DP>::kPer;
  for (int r0 = ROWS * blockIdx.z; r0 < rows; r0 += ROWS * gridDim.z) {
    const int r = r0 + warp / kSplit;
    Joined<DP> joined;
    if (r < rows)
      joined.template gather<kSplit>(p, warp % kSplit, cut.shares, [&](int c) {
        return (static_cast<size_t>(2 * (cut.first + c) + (c == 0)) * p.kv_heads + hk) * kStepRows + r;
      });
    if (lane == 0) warp_ml[warp] = make_float2(joined.top, joined.total);
#pragma unroll
    for (int e = 0; e < kPer; ++e) warp_o[warp][kPer * lane + e] = joined.o[e];
    __syncthreads();
    if (warp % kSplit == 0 && r < rows) {
#pragma unroll
      for (int a = 1; a < kSplit; ++a) {
        const float2 ml = warp_ml[warp + a];
        float v[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[e] = warp_o[warp + a][kPer * lane + e];
        joined.add(ml.x, ml.y, v, p.scale_log2);
      }
      joined.template store<T>(p, cut.qs, cut.ql, cut.kl, hk, row0 + r);
    }
    __syncthreads();
  }
}

template <class T, int DP, bool CLUSTER>
cudaError_t start(const AttnParams& p, const AttnMaps& maps, cudaStream_t st) {
  using L = StepSmem<DP>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(attention_step_kernel<T, DP, CLUSTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kTotal;
  cfg.stream = st;
  if (CLUSTER) {
    const long long items = static_cast<long long>(p.q_rows) * p.group / kStepRows + p.batch;
    cfg.gridDim = dim3(static_cast<unsigned>(items) * kStepCluster, p.kv_heads);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kStepCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  } else {
    cfg.gridDim = dim3(p.ctas, p.kv_heads);
  }
  return cudaLaunchKernelEx(&cfg, attention_step_kernel<T, DP, CLUSTER>, p, maps);
}

template <class T, int DP>
cudaError_t join(const AttnParams& p, cudaStream_t st) {
  const long long rows = (static_cast<long long>(p.q_rows) * p.group + p.batch - 1) / p.batch;
  const bool prompt = p.tile_rows > kStepRows;
  // Few sequences have many parts a row: 16 warps a row (one token on 64000 keys, one key
  // head: 15.8 us, with four warps 25.4); else four rows a CTA (16 tokens on 1000 keys, 8
  // key heads: 16.2 us, with 16 warps a row 18.7).
  const bool many = !prompt && p.ctas > 16 * p.batch;
  // the launch is prepared while the parts are computed, and waits for them at its
  // start (a call takes 0.1 us less than with an ordinary launch)
  cudaLaunchConfig_t cfg{};
  if (prompt)
    cfg.gridDim = dim3(p.batch, p.kv_heads, static_cast<unsigned>(std::min<long long>((rows + 3) / 4, 4096)));
  else
    cfg.gridDim = dim3(p.ctas - 1, p.kv_heads, static_cast<unsigned>(std::min<long long>(many ? rows : (rows + 3) / 4, kStepRows)));
  cfg.blockDim = dim3(prompt ? 128 : kJoinWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return prompt ? cudaLaunchKernelEx(&cfg, attention_join_kernel<T, DP>, p)
         : many ? cudaLaunchKernelEx(&cfg, attention_line_join_kernel<T, DP, 1>, p)
                : cudaLaunchKernelEx(&cfg, attention_line_join_kernel<T, DP, 4>, p);
}

}  // namespace

namespace svdq {

cudaError_t take_status_attention_step(int* status, cudaStream_t st) { return take_status(status, st); }
cudaError_t give_up_attention_step(cudaStream_t st) { return give_up(st); }

template <class T>
static cudaError_t start_dim(const AttnParams& p, const AttnMaps& maps, bool cluster, cudaStream_t st) {
  if (p.dim <= 64) return cluster ? start<T, 64, true>(p, maps, st) : start<T, 64, false>(p, maps, st);
  return cluster ? start<T, 128, true>(p, maps, st) : start<T, 128, false>(p, maps, st);
}

cudaError_t launch_attention_step(const AttnParams& p, const AttnMaps& maps, bool bf16, bool cluster, cudaStream_t st) {
  return bf16 ? start_dim<__nv_bfloat16>(p, maps, cluster, st) : start_dim<__half>(p, maps, cluster, st);
}

cudaError_t launch_attention_join(const AttnParams& p, bool bf16, cudaStream_t st) {
  if (p.dim <= 64) return bf16 ? join<__nv_bfloat16, 64>(p, st) : join<__half, 64>(p, st);
  return bf16 ? join<__nv_bfloat16, 128>(p, st) : join<__half, 128>(p, st);
}

}  // namespace svdq
