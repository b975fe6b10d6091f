// What the attention kernels share: the call's parameters, the packed
// sequences' extents, 16-bit conversions.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace svdq {

struct Cut;
struct AttnParams {
  const void *q, *v;  // v for the values that a product with 0 would spoil; tiles come by TMA
  void* out;          // [q_rows, q_heads, dim]
  const int *q_offsets, *k_offsets;
  int batch, q_rows, k_rows, q_heads, kv_heads, group, dim, causal;
  float scale_log2;   // scale * log2(e): softmax in base 2
  long long q_row, q_head, v_row, v_head;  // strides in elements
  // A sequence's rows (query * group + head in the group) are cut into tiles of
  // tile_rows, for attention_prompt.cu its keys into shares of `chunk` (a multiple of
  // the key tile; 0: see key_chunk).
  int tile_rows, chunk;
  int fill;           // with chunk 0: CTAs a key head that run at once
  int ctas;           // attention_step.cu: CTAs a key head
  int max_slots;      // partial results (tile_rows rows each) the workspace holds
  float *part, *part_ml;
  Cut* cuts;   // attention_step.cu: [ctas]
};
// A row tile that is in parts, as the second CTA that works on it notes it for the join.
struct Cut {
  int unit, first, shares, b;  // row tile, the first CTA, how many CTAs (0: none is noted), sequence
  int qs, ql, kl, none;        // the sequence's first query, its queries and keys
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
  static constexpr uint32_t kExp = 0x7F80;  // the exponent's bits (all of them: infinities and NaN)
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

// Whether any of eight 16-bit values is an infinity or NaN (all exponent bits
// set: one more in the exponent's last place carries into the sign's).
template <class T>
__device__ __forceinline__ bool has_non_finite(const uint4& v) {
  constexpr uint32_t e = Half16<T>::kExp * 0x10001u, one = (Half16<T>::kExp & -Half16<T>::kExp) * 0x10001u;
  return (((v.x & e) + one) | ((v.y & e) + one) | ((v.z & e) + one) | ((v.w & e) + one)) & 0x80008000u;
}
// Those values become 0.
template <class T>
__device__ __forceinline__ void drop_non_finite(uint4& v) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    constexpr uint32_t e = Half16<T>::kExp;
    if ((w[i] & e) == e) w[i] &= 0xFFFF0000u;
    if ((w[i] >> 16 & e) == e) w[i] &= 0x0000FFFFu;
  }
}

__device__ __forceinline__ uint4 load_shared(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void store_shared(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void store_shared(uint32_t addr, const uint4& v) { store_shared(addr, v.x, v.y, v.z, v.w); }

// The last key that a row (query * group + head) of a sequence of ql queries and kl keys
// sees, below 0 if it sees none.
__device__ __forceinline__ int last_key(const AttnParams& p, int row, int ql, int kl) {
  return p.causal ? min(row / p.group + kl - ql, kl - 1) : kl - 1;
}
// What a row's products with V are multiplied by. A sum of 0: the row sees no key (last()
// is below 0) and its result is 0, or every key that it sees has a score of minus
// infinity, and its result is NaN.
template <class Last>
__device__ __forceinline__ float row_norm(float sum, Last last) {
  if (sum == 0.f) return last() < 0 ? 1.f : __uint_as_float(0x7FFFFFFFu);
  return 1.f / sum;
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

// Row tiles, key shares and workspace slots of a sequence.
struct Shares {
  int tiles, chunks, slots;
};
__device__ __forceinline__ Shares shares_of(const AttnParams& p, int b, int chunk) {
  int qs, ql, ks, kl;
  seq_extent(p.q_offsets, b, p.q_rows, qs, ql);
  seq_extent(p.k_offsets, b, p.k_rows, ks, kl);
  Shares s;
  s.tiles = (ql * p.group + p.tile_rows - 1) / p.tile_rows;
  s.chunks = kl > chunk ? (kl + chunk - 1) / chunk : 1;
  s.slots = s.chunks > 1 ? s.tiles * s.chunks : 0;
  return s;
}

__device__ __forceinline__ int warp_inclusive(int v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (static_cast<int>(lane_id()) >= o) v += u;
  }
  return v;
}

// The keys of a share where the host left it open (few row tiles, up to 32
// sequences): the longest sequence's keys cut into as many shares as still run at
// once, each of 512 keys or more; a warp's lanes try 1 to 31 (a lone sequence of 64000
// keys, one key head, 32 rows: 43 us, with 16 at most 62). The lengths are on the
// device, so every CTA works it out for itself, and all come to the same.
__device__ __forceinline__ int key_chunk(const AttnParams& p) {
  if (p.chunk) return p.chunk;
  const int lane = lane_id();
  int tiles = 0, keys = 0;
  if (lane < p.batch) {
    int start, ql;
    seq_extent(p.q_offsets, lane, p.q_rows, start, ql);
    seq_extent(p.k_offsets, lane, p.k_rows, start, keys);
    tiles = (ql * p.group + p.tile_rows - 1) / p.tile_rows;
    if (!tiles) keys = 0;
  }
  int longest = keys;
#pragma unroll
  for (int o = 16; o; o >>= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
  // lane n tries n + 1 shares of the longest sequence; the last before the first that fails
  const int c = ((longest + lane) / (lane + 1) + 127) & ~127;
  int ctas = 0;
  for (int b = 0; b < p.batch; ++b) {
    const int k = __shfl_sync(0xffffffffu, keys, b);
    ctas += __shfl_sync(0xffffffffu, tiles, b) * (k > c ? (k + c - 1) / c : 1);
  }
  const unsigned fails = __ballot_sync(0xffffffffu, lane > 0 && (c < 512 || ctas > p.fill || lane == 31));
  const int chunk = fails & 2u ? longest + 1 : __shfl_sync(0xffffffffu, c, __ffs(fails) - 2);
  return chunk;
}

struct Found {
  int b, tile, tiles, chunk, chunks;
  int slots;  // workspace slots before the sequence's; it has slot tile * chunks + chunk of its own
};
struct Search {  // where the search for an item stands: sequences before b0 hold `items` items
  int b0, items;
  int chunk;  // key_chunk
};

// The sequence, row tile and key share of item `idx`: false behind the last.
// Called by the whole CTA of WARPS warps with idx that never decreases; `shared`
// and `sums` are in shared memory. The keys of more than 32 sequences are not cut.
template <int WARPS>
__device__ bool find_item(const AttnParams& p, Search& at, int idx, Found* shared, int* sums, Found* found) {
  if (p.batch <= 32) {  // each warp for itself, no barrier
    const int lane = lane_id();
    Shares s{0, 0, 0};
    if (lane < p.batch) s = shares_of(p, lane, at.chunk);
    const int own = s.tiles * s.chunks, items = warp_inclusive(own), slots = warp_inclusive(s.slots);
    const unsigned here = __ballot_sync(0xffffffffu, idx >= items - own && idx < items);
    if (!here) return false;
    const int b = __ffs(here) - 1, i = idx - (__shfl_sync(0xffffffffu, items - own, b));
    found->b = b;
    found->tiles = __shfl_sync(0xffffffffu, s.tiles, b);
    found->chunks = __shfl_sync(0xffffffffu, s.chunks, b);
    found->slots = __shfl_sync(0xffffffffu, slots - s.slots, b);
    found->tile = i / found->chunks;
    found->chunk = i % found->chunks;
    return true;
  }
  for (; at.b0 < p.batch; at.b0 += WARPS * 32) {
    const int b = at.b0 + static_cast<int>(threadIdx.x);
    const int own = b < p.batch ? shares_of(p, b, at.chunk).tiles : 0;
    int items = warp_inclusive(own);
    __syncthreads();  // the previous use of sums and found is over
    if (lane_id() == 31) sums[warp_id()] = items;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w == static_cast<int>(warp_id())) items += total;
      total += sums[w];
    }
    if (idx < at.items + total) {
      const int first = at.items + items - own;
      if (idx >= first && idx < first + own) *shared = {b, idx - first, own, 0, 1, 0};
      __syncthreads();
      *found = *shared;
      return true;
    }
    at.items += total;
  }
  return false;
}

// Few queries (attention_step.cu): row and key tiles.
constexpr int kStepRows = 16;
constexpr int kStepKeys = 64;
constexpr int kStepCluster = 8;  // CTAs of an item that join within a cluster
// Many queries (attention_prompt.cu): rows of a CTA (two tensor-memory tiles), key tile.
constexpr int kPromptRows = 256;
constexpr int kPromptKeys = 128;

// The work of attention_step.cu as a line: each row tile of each sequence is a unit of
// kEnds places, for what it costs to begin and end one, and one for each of its key tiles
// (one at least); unit after unit. Each CTA takes an equal stretch, so that they end
// together whatever the lengths are, and only the units at a stretch's ends are in
// parts: the part that begins a unit goes to slot 2 cta + 1, any other to slot 2 cta.
// (64 tokens on 200 to 16000 keys, 8 key heads: 156 us; shares of equal length dealt
// out in turn 166. 16 on 4000 keys each: 50 and 58. Short sequences of one length lose by
// it: 16 on 1000 each 16.1 and 15.1, 16 on 200 each 12.6 and 10.7; no cuts where a unit
// has kLeast tiles or fewer on average would help those, but 12 tokens on 20 to 700 keys
// then take 2.4 us more. kEnds 2: 20 tokens on 30 to 12000 keys, 4 key heads, 21.2 us, 4:
// 18.2; 8: the 64 tokens 160. kLeast 8: 6 tokens, 8 key heads, 13.9 us, 5: 11.5; 3: the 20
// tokens 18.4.)
struct Line {
  long long places;  // of all units
  int ctas;          // that share it: one a unit and one per kLeast key tiles, as far as they go
  static constexpr int kLeast = 5, kEnds = 4;
  __device__ __forceinline__ long long begin(int cta) const { return places * cta / ctas; }
  __device__ __forceinline__ int cta_of(long long place) const { return static_cast<int>(((place + 1) * ctas - 1) / places); }
};
struct Units {
  int units;        // row tiles of a sequence
  int tiles;        // key tiles of each
};
__device__ __forceinline__ Units units_of(const AttnParams& p, int b) {
  int start, ql, kl;
  seq_extent(p.q_offsets, b, p.q_rows, start, ql);
  seq_extent(p.k_offsets, b, p.k_rows, start, kl);
  return {(ql * p.group + kStepRows - 1) / kStepRows, max(1, (kl + kStepKeys - 1) / kStepKeys)};
}
// Sum over the warp of values from 0 up, together 2^52 at most, in two parts of 24 and 28 bits.
__device__ __forceinline__ long long warp_sum(long long v) {
  const unsigned low = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v & 0xFFFFFF));
  const unsigned high = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v >> 24));
  return (static_cast<long long>(high) << 24) + low;
}
// Called by the whole CTA; `sums` is in shared memory.
template <int WARPS>
__device__ __forceinline__ Line line_of(const AttnParams& p, long long (*sums)[2]) {
  long long v[2] = {0, 0};  // places, units
  const bool alone = p.batch <= 32;  // each warp for itself, no barrier
  for (int j = alone ? lane_id() : threadIdx.x; j < p.batch; j += alone ? 32 : WARPS * 32) {
    const Units u = units_of(p, j);
    v[0] += static_cast<long long>(u.units) * (u.tiles + Line::kEnds);
    v[1] += u.units;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) v[i] = warp_sum(v[i]);
  if (!alone) {
    if (lane_id() == 0)
      for (int i = 0; i < 2; ++i) sums[warp_id()][i] = v[i];
    __syncthreads();
    v[0] = v[1] = 0;
    for (int w = 0; w < WARPS; ++w)
      for (int i = 0; i < 2; ++i) v[i] += sums[w][i];
    __syncthreads();
  }
  return {v[0], static_cast<int>(min(static_cast<long long>(p.ctas), v[1] + (v[0] - v[1] * Line::kEnds) / Line::kLeast))};
}
struct Part {
  int b, unit;       // sequence, row tile
  int place, tiles;  // the place in the unit, and its key tiles
};
struct LineSearch {  // sequences before b0 hold `places` places
  int b0;
  long long places;
};
// The unit that place `x` of the line belongs to, x less than the line's places. Called
// by the whole CTA with x that never decreases; `shared` and `sums` are in shared memory.
template <int WARPS>
__device__ __forceinline__ Part part_at(const AttnParams& p, LineSearch& at, long long x, Part* shared, long long (*sums)[2]) {
  const int per = p.batch <= 32 ? 32 : WARPS * 32;
  for (;; at.b0 += per) {
    const int b = at.b0 + (per == 32 ? static_cast<int>(lane_id()) : static_cast<int>(threadIdx.x));
    Units u{0, 1};
    if (b < p.batch) u = units_of(p, b);
    const int length = u.tiles + Line::kEnds;
    const long long own = static_cast<long long>(u.units) * length;
    long long total = warp_sum(own), end = own;
    if (total < 1ll << 31) {
      end = warp_inclusive(static_cast<int>(own));
    } else {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, end, o);
        if (static_cast<int>(lane_id()) >= o) end += v;
      }
    }
    if (per > 32) {
      __syncthreads();  // the previous use of sums and shared is over
      if (lane_id() == 31) sums[warp_id()][0] = end;
      __syncthreads();
      total = 0;
      for (int w = 0; w < WARPS; ++w) {
        if (w == static_cast<int>(warp_id())) end += total;
        total += sums[w][0];
      }
    }
    if (x < at.places + total || at.b0 + per >= p.batch) {
      const long long i = x - at.places - (end - own);
      const bool here = i >= 0 && i < own;
      Part part{b, 0, 0, u.tiles};
      if (here) {
        part.unit = own < 1ll << 31 ? static_cast<int>(i) / length : static_cast<int>(i / length);
        part.place = static_cast<int>(i - static_cast<long long>(part.unit) * length);
      }
      if (per == 32) {
        const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        return {__shfl_sync(0xffffffffu, part.b, from), __shfl_sync(0xffffffffu, part.unit, from),
                __shfl_sync(0xffffffffu, part.place, from), __shfl_sync(0xffffffffu, part.tiles, from)};
      }
      if (here) *shared = part;
      __syncthreads();
      return *shared;
    }
    at.places += total;
  }
}

cudaError_t take_status_attention_prompt(int* status, cudaStream_t st);
cudaError_t give_up_attention_prompt(cudaStream_t st);
cudaError_t launch_attention_prompt(const AttnParams& p, const AttnMaps& maps, bool bf16, cudaStream_t st);
// Joins the parts of the row tiles that have several (after either kernel).
cudaError_t launch_attention_join(const AttnParams& p, bool bf16, cudaStream_t st);
cudaError_t take_status_attention_step(int* status, cudaStream_t st);
cudaError_t give_up_attention_step(cudaStream_t st);
cudaError_t launch_attention_step(const AttnParams& p, const AttnMaps& maps, bool bf16, bool cluster, cudaStream_t st);

}  // namespace svdq
