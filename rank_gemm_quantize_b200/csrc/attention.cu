// Host side of the attention calls: argument checks, tensor maps, the choice
// of the kernel and of the shares the keys are cut into.
#include <algorithm>
#include <string>

#include "attention.cuh"

namespace svdq {
void set_last_error(const std::string& msg);
cudaError_t take_status_dense(int* status, cudaStream_t st);
cudaError_t give_up_dense(cudaStream_t st);
}  // namespace svdq

using namespace svdq;

namespace {

svdq_status fail(svdq_status st, const std::string& msg) {
  set_last_error(msg);
  return st;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

svdq_status check(const svdq_attention_args* c) {
  if (!c) return fail(SVDQ_ERR_INVALID_ARG, "args is NULL");
  if (c->dtype != SVDQ_BF16 && c->dtype != SVDQ_F16) return fail(SVDQ_ERR_INVALID_ARG, "unknown dtype");
  if (c->batch < 1 || c->q_rows < 0 || c->k_rows < 0) return fail(SVDQ_ERR_INVALID_ARG, "bad batch, q_rows or k_rows");
  if (c->batch > 65535) return fail(SVDQ_ERR_UNSUPPORTED, "batch exceeds 65535");
  if (c->q_heads < 1 || c->kv_heads < 1 || c->q_heads % c->kv_heads || c->q_heads / c->kv_heads > 128)
    return fail(SVDQ_ERR_INVALID_ARG, "q_heads must be 1 to 128 times kv_heads");
  if (c->kv_heads > 65535) return fail(SVDQ_ERR_UNSUPPORTED, "kv_heads exceeds 65535");
  if (c->head_dim < 8 || c->head_dim > 128 || c->head_dim % 8)
    return fail(SVDQ_ERR_INVALID_ARG, "head_dim must be a multiple of 8, 8 to 128");
  if (c->causal != 0 && c->causal != 1) return fail(SVDQ_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (!(c->scale > 0.f) || c->scale > 1e30f) return fail(SVDQ_ERR_INVALID_ARG, "scale must be positive, at most 1e30");
  // rows and row-head pairs are counted in int
  if (static_cast<long long>(c->q_rows) * c->q_heads > 1ll << 30 || c->k_rows > 1 << 30)
    return fail(SVDQ_ERR_UNSUPPORTED, "q_rows x q_heads or k_rows exceeds 2^30");
  // The places of the line of work (Line) times its CTAs are counted in 64 bits. Offsets
  // that overlap can give each sequence all rows and all keys.
  const double rows = static_cast<double>(c->q_rows) * (c->q_heads / c->kv_heads);
  if (rows <= static_cast<double>(kStepRows) * c->batch &&
      c->batch * (rows / kStepRows + 1) * (c->k_rows / kStepKeys + 1. + Line::kEnds) > static_cast<double>(1ll << 52))
    return fail(SVDQ_ERR_UNSUPPORTED, "batch x q_rows x k_rows is too large");
  const long long strides[] = {c->q_row_stride, c->q_head_stride, c->k_row_stride, c->k_head_stride, c->v_row_stride, c->v_head_stride};
  const int extent[] = {c->q_rows, c->q_heads, c->k_rows, c->kv_heads, c->k_rows, c->kv_heads};
  for (int i = 0; i < 6; ++i)  // the stride of a single row or head is not used
    if (extent[i] > 1 && (strides[i] < 8 || strides[i] % 8 || strides[i] >= 1ll << 38))
      return fail(SVDQ_ERR_INVALID_ARG, "strides must be positive multiples of 8 under 2^38");
  return SVDQ_OK;
}

struct Plan {
  int sms, chunk, max_slots, ctas;
  bool prompt;   // attention_prompt.cu, or attention_step.cu
  bool cluster;  // attention_step.cu: an item's shares are a cluster
  bool open;     // attention_prompt.cu: the kernel sets `chunk`
  int fill;
  size_t ml, cuts, total;  // bytes of the partial results, of their maxima and sums too, and of all
};

// Which kernel, and the shares the keys are cut into. The lengths of the
// sequences are on the device: the rules go by the totals, and both kernels are
// right for any lengths.
svdq_status plan(const svdq_attention_args* c, Plan* out) {
  int dev = 0;
  Plan p{};
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&p.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return fail(SVDQ_ERR_CUDA, "no usable current device");
  }
  const long long rows = static_cast<long long>(c->q_rows) * (c->q_heads / c->kv_heads);
  // Eight CTAs an item where all of those run at once, up to 768 keys each (a lone
  // token, 4 key heads: of 777 keys 6.1 us, as stretches and a join 11.4; of 5000 11.2
  // and 12.4; of 7000 13.5 and 12.1). Else the kernel for many queries where a sequence
  // has more than one tile of rows on average, since each reads the keys again (32
  // rows, 4000 keys, 64 sequences of 8 key heads: 229 us, the kernel for few 334; 24 rows
  // of 1000 keys 84 and 96; 24 rows, 4 sequences of 4000: 28 and 24).
  p.cluster = (rows / kStepRows + c->batch) * c->kv_heads * kStepCluster <= 2 * p.sms &&
              c->k_rows <= static_cast<long long>(768) * kStepCluster * c->batch;
  p.prompt = !p.cluster && rows > static_cast<long long>(kStepRows) * c->batch;
  const int key_tile = p.prompt ? kPromptKeys : kStepKeys, tile_rows = p.prompt ? kPromptRows : kStepRows;
  long long slots = 0;  // partial results
  if (p.prompt) {
    // where the row tiles alone leave SMs idle, the kernel cuts the keys (key_chunk); its
    // shares are no more than the CTAs that run at once. One warp finds them, a lane a
    // sequence, hence 32 (32 rows on 16000 keys, one key head: 32 sequences 75 us, 33,
    // whose keys are not cut, 199)
    const long long tiles = rows / kPromptRows;
    p.fill = p.sms / c->kv_heads;
    p.open = c->batch <= 32 && tiles < p.fill && c->k_rows > 768;  // of fewer keys no share would have 512
    slots = p.open ? p.fill : 0;
  } else if (!p.cluster) {
    // two CTAs an SM, no more than there are stretches (Line) that are worth one
    const long long units = rows / kStepRows + c->batch;
    p.ctas = static_cast<int>(std::min(std::max(1ll, 2ll * p.sms / c->kv_heads), units + c->k_rows / (Line::kLeast * kStepKeys)));
    slots = p.ctas > 1 ? 2ll * p.ctas : 0;
  }
  p.chunk = std::max(1, (c->k_rows + key_tile - 1) / key_tile) * key_tile;
  if ((slots + rows / tile_rows + c->batch) * c->kv_heads > 0x7fffffffll) return fail(SVDQ_ERR_UNSUPPORTED, "too many sequences times heads");
  p.max_slots = static_cast<int>(slots);
  const size_t slot_rows = static_cast<size_t>(slots) * c->kv_heads * tile_rows;
  p.ml = slot_rows * (c->head_dim <= 64 ? 64 : 128) * 4;
  p.cuts = p.ml + slot_rows * 8;
  p.total = p.cuts + (p.prompt || !slots ? 0 : p.ctas * sizeof(Cut));
  *out = p;
  return SVDQ_OK;
}

bool make_kv_map(CUtensorMap* m, const svdq_attention_args* c, const void* base, long long row, long long head, int keys) {
  const uint64_t dims[3] = {static_cast<uint64_t>(c->head_dim), static_cast<uint64_t>(c->kv_heads), static_cast<uint64_t>(c->k_rows)};
  // a single head or row has no stride of its own: any legal one
  const uint64_t strides[2] = {static_cast<uint64_t>(c->kv_heads > 1 ? head : c->head_dim) * 2,
                               static_cast<uint64_t>(c->k_rows > 1 ? row : c->head_dim) * 2};
  const uint32_t box[3] = {64, 1, static_cast<uint32_t>(keys)};
  return make_map_3d(m, c->dtype == SVDQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

extern "C" {

svdq_status svdq_attention_workspace_size(const svdq_attention_args* args, size_t* bytes) {
  if (svdq_status e = check(args)) return e;
  if (!bytes) return fail(SVDQ_ERR_INVALID_ARG, "bytes is NULL");
  Plan p;
  if (svdq_status e = plan(args, &p)) return e;
  *bytes = p.total;
  return SVDQ_OK;
}

svdq_status svdq_attention_forward(const svdq_attention_args* a, void* stream) {
  if (svdq_status e = check(a)) return e;
  if (a->q_rows == 0) return SVDQ_OK;
  if (!a->q || !a->out || (a->k_rows > 0 && (!a->k || !a->v))) return fail(SVDQ_ERR_INVALID_ARG, "q, k, v or out is NULL");
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->out, 16))
    return fail(SVDQ_ERR_INVALID_ARG, "q, k, v and out must be 16-byte aligned");
  if ((!a->q_offsets || !a->k_offsets) && a->batch != 1) return fail(SVDQ_ERR_INVALID_ARG, "several sequences need offsets");
  if (!aligned(a->q_offsets, 4) || !aligned(a->k_offsets, 4)) return fail(SVDQ_ERR_INVALID_ARG, "offsets must be 4-byte aligned");
  Plan pl;
  if (svdq_status e = plan(a, &pl)) return e;
  if (pl.total && (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < pl.total))
    return fail(SVDQ_ERR_INVALID_ARG, "workspace missing, misaligned or too small");
  AttnParams p{};
  p.q = a->q;
  p.v = a->v;
  p.out = a->out;
  p.q_offsets = a->q_offsets;
  p.k_offsets = a->k_offsets;
  p.batch = a->batch;
  p.q_rows = a->q_rows;
  p.k_rows = a->k_rows;
  p.q_heads = a->q_heads;
  p.kv_heads = a->kv_heads;
  p.group = a->q_heads / a->kv_heads;
  p.dim = a->head_dim;
  p.causal = a->causal;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.q_row = a->q_row_stride;
  p.q_head = a->q_head_stride;
  p.v_row = a->v_row_stride;
  p.v_head = a->v_head_stride;
  p.tile_rows = pl.prompt ? kPromptRows : kStepRows;
  p.chunk = pl.open ? 0 : pl.chunk;
  p.fill = pl.fill;
  p.ctas = pl.ctas;
  p.max_slots = pl.max_slots;
  p.part = static_cast<float*>(a->workspace);
  p.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(a->workspace) + pl.ml);
  p.cuts = reinterpret_cast<Cut*>(static_cast<uint8_t*>(a->workspace) + pl.cuts);
  AttnMaps maps{};
  const int key_tile = pl.prompt ? kPromptKeys : kStepKeys;
  if (a->k_rows > 0 && (!make_kv_map(&maps.k, a, a->k, a->k_row_stride, a->k_head_stride, key_tile) ||
                          !make_kv_map(&maps.v, a, a->v, a->v_row_stride, a->v_head_stride, key_tile)))
    return fail(SVDQ_ERR_CUDA, "cuTensorMapEncodeTiled (keys or values) failed");
  const bool bf16 = a->dtype == SVDQ_BF16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = pl.prompt ? launch_attention_prompt(p, maps, bf16, st) : launch_attention_step(p, maps, bf16, pl.cluster, st);
  if (e == cudaSuccess && pl.max_slots > 0) e = launch_attention_join(p, bf16, st);
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, std::string("attention kernel: ") + cudaGetErrorString(e));
  return SVDQ_OK;
}

svdq_status svdq_operator_status(void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  bool timeout = false;
  for (auto take : {take_status_attention_step, take_status_attention_prompt, take_status_dense}) {
    int status = 0;
    const cudaError_t e = take(&status, st);
    if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, std::string("operator status: ") + cudaGetErrorString(e));
    timeout |= status == kDevTimeout;
  }
  if (timeout) return fail(SVDQ_ERR_DEVICE_TIMEOUT, "a kernel gave up a pipeline wait");
  return SVDQ_OK;
}

svdq_status svdq_selftest_operator_wait(int kernels, void* stream) {
  constexpr cudaError_t (*start[])(cudaStream_t) = {give_up_attention_step, give_up_attention_prompt, give_up_dense};
  if (kernels < 0 || kernels > 2) return fail(SVDQ_ERR_INVALID_ARG, "kernels must be 0, 1 or 2");
  const cudaError_t e = start[kernels](static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, std::string("self-test kernel: ") + cudaGetErrorString(e));
  return SVDQ_OK;
}

}  // extern "C"
