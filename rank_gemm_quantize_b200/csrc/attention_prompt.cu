// Attention of many queries per sequence (whole prompts, long pieces) on the
// tensor cores, scores and results in tensor memory.
//
// The query heads of a key head and the queries of a sequence form one list of
// rows (row = query * group + head), so grouped heads fill the tiles and read
// each key once. A CTA takes 256 rows of one key head: two tiles of 128
// rows. Per 128 keys
//   S = Q K^T     (both operands in shared memory, S float in tensor memory)
//   P = 2^(c S - c m), rounded to 16 bits over S in tensor memory
//   O += P V      (P from tensor memory, V from shared memory as it lies there)
// with m the row's running maximum and the row's sum kept in registers: one thread
// owns a row, so neither needs an exchange. While the threads of one tile work on
// their scores, the tensor core multiplies for the other tile; P goes to it in
// two halves, so that the first is multiplied while the second is computed.
//
// A tile's chain of S, softmax and P V bounds it: the two tiles' products take
// 2048 cycles per 128 keys, a chain 3300 (the softmax 2100 of them, whether the
// other tile's runs beside it or not). The exponential unit alone would need 1024
// cycles a tile, so two of eight pairs of exponentials are computed with
// multiply-adds (exp2_pair). 4608 x 4608 keys, 24 heads of 128: 221 to 236 us for a few
// calls (1105 to 1180 TFLOP/s), 259 us and 1007 TFLOP/s in a long run under the power
// cap, 73% of a library product's rate there; 8192 x 8192, 16 heads of 64: 402 to 436 us,
// where the exponentials alone take 240 us. Each step loads five spilled values again
// (by the counters; they are stored outside the loop). What was slower than 230 us:
// steps of 64 keys with two S a tile (302 us: an MMA of 64 columns takes as long as
// one of 128), two threads a row (260), P handed over in parts of 32 and 96 keys
// (232) or 96 and 32 (238), the second half of S loaded under the first's maximum
// (247), and for heads of 64 P in columns of its own with S issued ahead (463 for 406).
//
// P is rounded to the operands' 16 bits: the tensor core multiplies V, which has 16,
// by nothing wider. That adds up to half a step of the type to a value's error; in fp16
// a probability under 2^-25 of the one at m becomes 0. The row's sum takes P unrounded.
//
// O is not rescaled whenever m grows, only when it grew by more than 2^8 since
// the last time: P may then be up to 2^8 instead of 1, which costs no digits
// (its relative rounding is the same), and the final division puts it right.
//
// Warps: 0-3 and 4-7 the softmax of the two tiles, 8 issues the MMAs, 9 the TMA loads, 10 and
// 11 keep values that a query must not see out of the product (below). K and V tiles
// share one ring of stages in the order K0 V0 K1 V1 ..
#include <string>

#include "attention.cuh"
#include "operator_status.cuh"

using namespace svdq;

namespace {

constexpr int kThreads = 384;
constexpr int kTileRows = 128;
constexpr int kRegsSoftmax = 216, kRegsOther = 72;  // registers a thread: 256 threads and 128
constexpr int kStepN = 128;       // keys of one S
constexpr float kGrow = 8.f;  // log2 of how far the maximum may grow before O is rescaled

template <int DP>
struct PromptSmem {
  static constexpr int kQTile = kTileRows * DP * 2;
  static constexpr int kStage = kPromptKeys * DP * 2;  // one K or V tile
  static constexpr int kStages = DP == 128 ? 5 : 8;
  static constexpr int kRing = 2 * kQTile;
  static constexpr int kBars = kRing + kStages * kStage;
  static constexpr int kTotal = kBars + 512 + 1024;
};
static_assert(PromptSmem<128>::kTotal <= 232448, "shared memory budget");

// Byte offset of 16-byte piece `piece` of a row in a swizzled tile of 128 rows.
__device__ __forceinline__ uint32_t tile_at(int row, int piece) {
  return (piece >> 3) * (128 * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}

// Operand descriptors of 128-byte-swizzled tiles as two words: the upper is the
// same for all (8 rows of 128 bytes are 1024 apart), the lower holds the address
// and the step between columns of 64 values, so a step along a tile is one
// addition. One thread issues every MMA, and what it does between two of them
// bounds the kernel (descriptors built anew for each: 135 cycles an MMA).
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | static_cast<uint32_t>(kSw128) << 29;
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t column_step) { return saddr >> 4 | (column_step >> 4) << 16; }

// D[tmem] (+)= A B, A and B in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc)), "r"(kDescHigh)
      : "memory");
}
// D[tmem] (+)= A[tmem] B: A is 16-bit pairs, one row a lane, 8 columns a k-step of 16.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc)), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 2^x of two values without the exponential unit: x = i + f, f in [-1/2, 1/2]; the
// polynomial (minimax in the relative error by Lawson's iteration, 2.6e-6) gives
// 2^f, and i goes into its exponent. 0 below 2^-126, as a hidden key needs. Of NaN it
// makes some number: the row's sum is NaN then, whatever is added (largest3).
__device__ __forceinline__ float2 exp2_pair(float2 x) {
  auto both = [](float c) { return make_float2(c, c); };
  const float2 t = __fadd2_rn(x, both(12582912.f));  // 3 2^22: i in the low bits
  const float2 f = __ffma2_rn(__fadd2_rn(t, both(-12582912.f)), both(-1.f), x);
  float2 q = both(0.00957007046f);
  q = __ffma2_rn(q, f, both(0.0559178127f));
  q = __ffma2_rn(q, f, both(0.240247451f));
  q = __ffma2_rn(q, f, both(0.693121821f));
  q = __ffma2_rn(q, f, both(0.999999262f));
  const float a = __uint_as_float(__float_as_uint(q.x) + (__float_as_uint(t.x) << 23));
  const float b = __uint_as_float(__float_as_uint(q.y) + (__float_as_uint(t.y) << 23));
  return make_float2(x.x < -126.f ? 0.f : a, x.y < -126.f ? 0.f : b);
}

// The largest of three values, NaN if one of them is.
__device__ __forceinline__ float largest3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Tensor memory: S (and, over it, P) of the two tiles, then the two results.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScoreCol = 0, kResultCol = 256;

template <class T, int DP>
__global__ void __launch_bounds__(kThreads, 1) attention_prompt_kernel(const AttnParams p, const __grid_constant__ AttnMaps maps) {
  using L = PromptSmem<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);  // [kStages] a K or V tile can be used
  uint64_t* empty = full + L::kStages;                            // [kStages] the MMAs are done with it
  uint64_t* s_full = empty + L::kStages;                          // [2 tiles] the scores are complete
  uint64_t* p_full = s_full + 2;                                  // [2 tiles][2] a half of the probabilities is written
  uint64_t* o_done = p_full + 4;                                  // [2 tiles] the last product with V is complete
  uint64_t* dirty = o_done + 2;                                   // [kStages] a V tile with hidden keys has landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dirty + L::kStages);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* spoiled = abort_flag + 1;
  __shared__ int sums[kThreads / 32];
  __shared__ Found found;

  const int tid = threadIdx.x, lane = lane_id();
  const int warp = __shfl_sync(0xffffffffu, warp_id(), 0);  // known to be the same for the warp
  const int hk = blockIdx.x % p.kv_heads;  // heads side by side: the heaviest tiles of all of them start first
  Search at{0, 0, key_chunk(p)};
  Found f;
  if (!find_item<kThreads / 32>(p, at, blockIdx.x / p.kv_heads, &found, sums, &f)) return;
  int qs, ql, ks, kl;
  seq_extent(p.q_offsets, f.b, p.q_rows, qs, ql);
  seq_extent(p.k_offsets, f.b, p.k_rows, ks, kl);
  const int rows = ql * p.group;
  // the tiles that see most keys first
  const int tile = f.tiles - 1 - f.tile, row0 = tile * kPromptRows;
  const int k_begin = f.chunks > 1 ? f.chunk * at.chunk : 0;
  auto limit = [&](int row) { return last_key(p, row, ql, kl); };
  auto key_steps = [&](int t) {
    const int first = row0 + t * kTileRows, last = min(first + kTileRows, rows) - 1;
    if (first >= rows) return 0;
    const int end = min(f.chunks > 1 ? k_begin + at.chunk : kl, limit(last) + 1);
    return end > k_begin ? (end - k_begin + kStepN - 1) / kStepN : 0;
  };
  const int n0 = key_steps(0), n1 = key_steps(1), steps = max(n0, n1);
  const int n = (steps * kStepN + kPromptKeys - 1) / kPromptKeys;  // key tiles to load
  const int first_limit = limit(row0);
  // key tiles from this one on hold keys that some row does not see
  const int first_hidden = max(0, first_limit + 1 - k_begin) / kPromptKeys;
  // parity of the barrier on which such a V tile lands; its stage is that of every kPeriod-th V tile
  constexpr int kPeriod = L::kStages % 2 ? L::kStages : L::kStages / 2;
  auto hidden_parity = [&](int j) { return static_cast<uint32_t>((j - first_hidden) / kPeriod & 1); };

  // loads: K of key tile i / 2, then its V
  auto hidden = [&](int i) { return (i & 1) && (i >> 1) >= first_hidden; };
  auto load = [&](int i) {
    const int s = i % L::kStages;
    uint8_t* st = smem + L::kRing + s * L::kStage;
    const CUtensorMap* map = i & 1 ? &maps.v : &maps.k;
    uint64_t* bar = hidden(i) ? &dirty[s] : &full[s];
    if (!hidden(i)) mbar_arrive(&full[s]);
    mbar_arrive_expect_tx(bar, L::kStage);
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) tma_load_3d(st + c * 128 * 128, map, bar, c * 64, hk, ks + k_begin + (i >> 1) * kPromptKeys);
  };
  const int ahead = min(2 * n, L::kStages);
  if (warp == 9) {  // the load warp: the first loads wait for nothing but the barriers
    constexpr int kBarriers = 3 * L::kStages + 8;
    static_assert(kBarriers <= 32, "a lane a barrier");
    // two arrivals on `full`: by this warp, or one of each of the two that clean the tile; four warps on p_full
    if (lane < kBarriers) mbar_init(&full[lane], lane < L::kStages ? 2 : &full[lane] >= p_full && &full[lane] < p_full + 4 ? 4 : 1);
    if (lane == 0) {
      *abort_flag = 0;
      *spoiled = 0;
    }
    fence_barrier_init();
    __syncwarp();
    if (lane == 0)
      for (int i = 0; i < ahead; ++i) load(i);
    __syncwarp();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  // The rows' queries, zeros behind the last row and column: a lane of the softmax
  // warps finds its row's place, then a warp copies whole rows, all asked for at once.
  constexpr int kLanes = DP / 8, kAtOnce = 32 / kLanes;  // lanes of a row, rows of a load
  const int own_row = row0 + 32 * warp + lane;
  if (warp < 8) {
    const long long place = own_row < rows ? static_cast<long long>(qs + own_row / p.group) * p.q_row + (hk * p.group + own_row % p.group) * p.q_head : -1;
    uint4 v[32 / kAtOnce];
#pragma unroll
    for (int i = 0; i < 32 / kAtOnce; ++i) {
      const long long from = __shfl_sync(0xffffffffu, place, i * kAtOnce + lane / kLanes);
      const int c = lane % kLanes;
      v[i] = from >= 0 && 8 * c < p.dim ? *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + from + 8 * c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 32 / kAtOnce; ++i) {
      const int r = 32 * warp + i * kAtOnce + lane / kLanes;
      store_shared(smem_u32(smem) + (r / kTileRows) * L::kQTile + tile_at(r % kTileRows, lane % kLanes), v[i]);
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 9) {
      // ------------------------------------------------------------ loads
      if (lane == 0) {
        int i = ahead;
        for (; i < 2 * n; ++i) {
          if (!mbar_wait(&empty[i % L::kStages], ((i / L::kStages) & 1) ^ 1, abort_flag, &g_status)) break;
          load(i);
        }
        if (i < 2 * n) {  // gave up: the copies in flight land before the CTA ends
          volatile int no_abort = 0;
          for (int e = max(0, i - L::kStages); e < i; ++e)
            if (hidden(e))
              mbar_wait(&dirty[e % L::kStages], hidden_parity(e >> 1), &no_abort, nullptr);
            else
              mbar_wait(&full[e % L::kStages], (e / L::kStages) & 1, &no_abort, nullptr);
        }
      }
    } else if (warp == 8) {
      // ------------------------------------------------------------ MMAs
      // The whole warp goes through the loops, one lane issues: what an MMA reads is
      // then the same for the warp and stays in uniform registers (a lone lane's
      // values are moved there for each MMA, 70 cycles of it).
      if (n > 0) {
        constexpr uint32_t kFmt = Half16<T>::kFmt;
        const uint32_t idesc_s = idesc_dense(kFmtF32, kFmt, kFmt, kTileRows, kStepN);
        const uint32_t idesc_o = idesc_dense(kFmtF32, kFmt, kFmt, kTileRows, DP) | (1u << 16);  // V: columns contiguous
        const bool issues = elect_one();
        const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
        const int m0 = __shfl_sync(0xffffffffu, n0, 0), m1 = __shfl_sync(0xffffffffu, n1, 0), all = max(m0, m1);
        const uint32_t q = smem_u32(smem), ring = q + L::kRing;
        auto wait_full = [&](int i) { return warp_wait(&full[i % L::kStages], (i / L::kStages) & 1, abort_flag, &g_status); };
        auto commit = [&](uint64_t* bar) {
          if (issues) tc_commit(bar);
        };
        auto scores = [&](int t, int j) {
          const uint32_t a = desc_low(q + t * L::kQTile, 16), b = desc_low(ring + (2 * j) % L::kStages * L::kStage, 16);
          const uint32_t d = base + kScoreCol + t * kStepN;
          if (issues) {
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
              const uint32_t at16 = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
              mma_ss(d, a + at16, b + at16, idesc_s, k > 0);
            }
            tc_commit(&s_full[t]);
          }
        };
        auto products = [&](int t, int j, int half) {  // 64 of the tile's keys
          const uint32_t b = desc_low(ring + (2 * j + 1) % L::kStages * L::kStage + half * (64 * 128), 128 * 128);
          const uint32_t d = base + kResultCol + t * DP, a = base + kScoreCol + t * kStepN + half * 32;
          if (issues) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_ts(d, a + 8 * k, b + (2048 >> 4) * k, idesc_o, j > 0 || half > 0 || k > 0);
          }
        };
        bool ok = wait_full(0);
        if (ok) {
          tc_fence_after();
          if (m0 > 0) scores(0, 0);
          if (m1 > 0) scores(1, 0);
          commit(&empty[0]);
        }
        for (int j = 0; j < all && ok; ++j) {
          const int iv = 2 * j + 1, ik = iv + 1;  // V tile of this step, K tile of the next
          ok = wait_full(iv);
          if (ok && j + 1 < all) ok = wait_full(ik);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int nt = t ? m1 : m0;
            if (!ok || j >= nt) continue;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (ok) ok = warp_wait(&p_full[2 * t + half], j & 1, abort_flag, &g_status);
              if (!ok) continue;
              tc_fence_after();
              products(t, j, half);
            }
            if (!ok) continue;
            if (j + 1 < nt)
              scores(t, j + 1);  // over P: MMAs of one thread run in order
            else
              commit(&o_done[t]);
          }
          if (!ok) break;
          commit(&empty[iv % L::kStages]);
          if (j + 1 < all) commit(&empty[ik % L::kStages]);
        }
        if (!ok) {  // gave up: the MMAs in flight end before the CTA does
          commit(&o_done[0]);
          commit(&o_done[1]);
        }
      }
    } else {
      // ------------------------------------------------------------ hidden values
      // A key that a row does not see has probability 0, but 0 times infinity is
      // NaN: in tiles that hold hidden keys, values behind the sequence become 0;
      // infinities and NaN of other keys that not every row sees become 0 too,
      // and are put back into the rows that do see them at the end.
      for (int j = first_hidden; j < n; ++j) {
        const int stage = (2 * j + 1) % L::kStages;
        if (!warp_wait(&dirty[stage], hidden_parity(j), abort_flag, &g_status)) break;
        uint8_t* st = smem + L::kRing + stage * L::kStage;
        const int key0 = k_begin + j * kPromptKeys;
        bool any = false;
        // a thread's 16-byte pieces lie in the same place of every kApart-th row
        constexpr int kApart = 64 / (DP / 8), kBatch = 8;
        const int piece = ((warp - 10) * 32 + lane) % (DP / 8), r0 = ((warp - 10) * 32 + lane) / (DP / 8);
        const uint32_t tile = smem_u32(st);
#pragma unroll 1
        for (int r = r0; r < kPromptKeys; r += kBatch * kApart) {
          uint4 v[kBatch];
          bool odd = false;
#pragma unroll
          for (int i = 0; i < kBatch; ++i) v[i] = load_shared(tile + tile_at(r + i * kApart, piece));
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int key = key0 + r + i * kApart;
            odd |= (key >= kl) | ((key > first_limit) & has_non_finite<T>(v[i]));
          }
          if (!odd) continue;
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int key = key0 + r + i * kApart;
            if (key >= kl) {
              v[i] = make_uint4(0, 0, 0, 0);
            } else if (key > first_limit && has_non_finite<T>(v[i])) {
              drop_non_finite<T>(v[i]);
              any = true;
            }
            store_shared(tile + tile_at(r + i * kApart, piece), v[i]);
          }
        }
        if (any) *spoiled = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[stage]);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // -------------------------------------------------------------- softmax
    const int t = warp >> 2, nt = t ? n1 : n0;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t result = tmem + lanes + kResultCol + t * DP;
    const int row = row0 + t * kTileRows + 32 * (warp & 3) + lane;
    const int lim = row < rows ? limit(row) : -1;
    const int warp_limit = limit(row - lane);  // its first row sees least
    const float c = p.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    const uint32_t scores = tmem + lanes + kScoreCol + t * kStepN;
    for (int j = 0; j < nt; ++j) {
      ok = warp_wait(&s_full[t], j & 1, abort_flag, &g_status);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int b = 0; b < 4; ++b) tmem_ld32(scores + 32 * b, s[b]);
      tmem_ld_wait();
      const int key0 = k_begin + j * kStepN;
      if (key0 + kStepN - 1 > warp_limit) {  // some row does not see some key
        const int seen = lim - key0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * b + e > seen) s[b][e] = 0xFF800000u;  // minus infinity
      }
      const float2 c2 = make_float2(c, c);
      float2 base2, sum[4];  // a packed sum takes long: several chains of them
      uint32_t pk[2][16];
      // 64 of the scores to probabilities, two of eight pairs by multiply-adds
      auto half = [&](int h) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * h + b][2 * e]), __uint_as_float(s[2 * h + b][2 * e + 1])), c2, base2);
            if ((3 * e) % 8 < 2) {
              x = exp2_pair(x);
            } else {
              x.x = exp2_fast(x.x);
              x.y = exp2_fast(x.y);
            }
            sum[e % 4] = __fadd2_rn(sum[e % 4], x);
            pk[b][e] = Half16<T>::pack(x.x, x.y);
          }
      };
      auto hand_over = [&](int h) {
        tmem_st16(scores + 32 * h, pk[0]);
        tmem_st16(scores + 32 * h + 16, pk[1]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * t + h]);
      };
      float top[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        top[b] = largest3(__uint_as_float(s[b][0]), __uint_as_float(s[b][1]), __uint_as_float(s[b][1]));
#pragma unroll
        for (int e = 2; e < 32; e += 2) top[b] = largest3(top[b], __uint_as_float(s[b][e]), __uint_as_float(s[b][e + 1]));
      }
      const float now = largest3(largest3(top[0], top[1], top[2]), top[3], top[3]);
      const bool grew = (now - m) * c > kGrow;  // also the first time; false while nothing was seen, and for NaN
      if (__any_sync(0xffffffffu, grew)) {
        const float factor = grew ? exp2_fast((m - now) * c) : 1.f;
        if (grew) m = now;
        l *= factor;
        if (j > 0) {  // the last product is complete: these scores were issued after it
#pragma unroll 1
          for (int b = 0; b < DP; b += 16) {
            uint32_t o[16];
            tmem_ld16(result + b, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
            tmem_st16(result + b, o);
          }
        }
      }
      const float base = (m == -INFINITY ? 0.f : m) * c;
      base2 = make_float2(-base, -base);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = make_float2(0.f, 0.f);
      half(0);
      hand_over(0);
      half(1);
      hand_over(1);
#pragma unroll
      for (int i = 1; i < 4; ++i) sum[0] = __fadd2_rn(sum[0], sum[i]);
      l += sum[0].x + sum[0].y;
      // a score of NaN or infinity (infinity less itself is NaN) that the row sees: the row
      // is NaN (kept by each value's exponential instead, 4608 x 4608: 247 us for 236)
      if (!(now < INFINITY)) l = __uint_as_float(0x7FFFFFFFu);
    }
    if (nt > 0) {
      volatile int no_abort = 0;
      ok = warp_wait(&o_done[t], 0, &no_abort, &g_status) && ok && __all_sync(0xffffffffu, !*abort_flag);
      tc_fence_after();
    }
    // ---------------------------------------------------------------- result
    if (ok) {
      const bool split = f.chunks > 1;
      // as row_norm; its branch in the code costs spills here (40 prompts of 200: 112 us for 110)
      const float norm = split || lim < 0 ? 1.f : l == 0.f ? __uint_as_float(0x7FFFFFFFu) : 1.f / l;
      const int share = f.slots + tile * f.chunks + f.chunk;
      const size_t slot = (static_cast<size_t>(share) * p.kv_heads + hk) * kPromptRows + row - row0;
      const bool write = row < rows && (!split || share < p.max_slots);
      const int spoil_end = *spoiled ? min(lim + 1, k_begin + nt * kStepN) : 0;
      // a row's place in the output (or its slot), as the lanes that write it need it
      const long long place = !write ? -1
                              : split ? static_cast<long long>(slot) * DP
                                      : (static_cast<long long>(qs + row / p.group) * p.q_heads + hk * p.group + row % p.group) * p.dim;
      const uint32_t stage = smem_u32(smem) + t * L::kQTile;  // the tile's queries are used up; each warp keeps to its rows
#pragma unroll 1
      for (int b = 0; b < DP; b += 32) {
        uint32_t o[32];
        if (nt > 0) {
          tmem_ld32(result + b, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        for (int key = max(k_begin, first_limit + 1); key < spoil_end; ++key) {
          const T* v = static_cast<const T*>(p.v) + static_cast<long long>(ks + key) * p.v_row + hk * p.v_head + b;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t bits = b + e < p.dim ? reinterpret_cast<const uint16_t*>(v)[e] : 0u;
            if ((bits & Half16<T>::kExp) == Half16<T>::kExp) o[e] = __float_as_uint(__uint_as_float(o[e]) + Half16<T>::to_float(bits));
          }
        }
        __syncwarp();
        if (split) {  // 32 float columns a row at a time: 128 bytes
#pragma unroll
          for (int e = 0; e < 8; ++e)
            store_shared(stage + tile_at(32 * (warp & 3) + lane, e), o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + lane / 8;
            const long long to = __shfl_sync(0xffffffffu, place, r);
            const uint4 v = load_shared(stage + tile_at(32 * (warp & 3) + r, lane % 8));
            if (to >= 0) *reinterpret_cast<uint4*>(p.part + to + b + 4 * (lane % 8)) = v;
          }
          __syncwarp();
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t w[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) w[h] = Half16<T>::pack(__uint_as_float(o[e + 2 * h]) * norm, __uint_as_float(o[e + 2 * h + 1]) * norm);
            store_shared(stage + tile_at(32 * (warp & 3) + lane, (b + e) / 8), w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (!split) {
        __syncwarp();
        const int c = lane % kLanes;
        uint4 v[32 / kAtOnce];
#pragma unroll
        for (int i = 0; i < 32 / kAtOnce; ++i)
          v[i] = load_shared(stage + tile_at(32 * (warp & 3) + i * kAtOnce + lane / kLanes, c));
#pragma unroll
        for (int i = 0; i < 32 / kAtOnce; ++i) {
          const long long to = __shfl_sync(0xffffffffu, place, i * kAtOnce + lane / kLanes);
          if (to >= 0 && 8 * c < p.dim) *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + to + 8 * c) = v[i];
        }
      }
      if (split && write) *reinterpret_cast<float2*>(p.part_ml + 2 * slot) = make_float2(m, l);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <class T, int DP>
cudaError_t start(const AttnParams& p, const AttnMaps& maps, cudaStream_t st) {
  using L = PromptSmem<DP>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = once_per_device(done, [] {
    // the softmax warps' registers come out of what the block starts with
    cudaFuncAttributes a;
    const cudaError_t r = cudaFuncGetAttributes(&a, attention_prompt_kernel<T, DP>);
    if (r != cudaSuccess) return r;
    if (a.numRegs * kThreads < kRegsSoftmax * 256 + kRegsOther * 128) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(attention_prompt_kernel<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
  });
  if (e != cudaSuccess) return e;
  // CTAs behind the last item leave at once
  const long long items = p.max_slots + static_cast<long long>(p.q_rows) * p.group / kPromptRows + p.batch;
  attention_prompt_kernel<T, DP><<<static_cast<unsigned>(items * p.kv_heads), kThreads, L::kTotal, st>>>(p, maps);
  return cudaGetLastError();
}

}  // namespace

namespace svdq {

cudaError_t take_status_attention_prompt(int* status, cudaStream_t st) { return take_status(status, st); }
cudaError_t give_up_attention_prompt(cudaStream_t st) { return give_up(st); }

cudaError_t launch_attention_prompt(const AttnParams& p, const AttnMaps& maps, bool bf16, cudaStream_t st) {
  if (p.dim <= 64) return bf16 ? start<__nv_bfloat16, 64>(p, maps, st) : start<__half, 64>(p, maps, st);
  return bf16 ? start<__nv_bfloat16, 128>(p, maps, st) : start<__half, 128>(p, maps, st);
}

}  // namespace svdq
