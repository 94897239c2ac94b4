// The part of the C ABI between two decode steps (declared in
// include/mla_decode.h): argument checks and dispatch of the draft
// verification, the request lists and the row moves.  Nothing here allocates or
// synchronises; nothing throws across the boundary.
#include <cstdint>

#include "mla_launch.h"
#include "mla_serving.h"

using namespace mla;

namespace {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool ready(const void* p, uintptr_t n = 16) { return p && aligned(p, n); }
// A stride in elements of an input that is only read: 0 (the same for all) included.
inline bool stride_ok(int64_t s) { return s >= 0 && s < (1ll << 40); }
inline bool slots_ok(int64_t n) { return n >= 1 && n <= 0x7FFFFFFFll; }

// Rows [layers, layer_rows, row_bytes] and their scales [layers, layer_rows].
bool rows_ok(const void* cache, const float* scales, int64_t num_slots, int64_t layer_rows, int32_t layers,
             int32_t row_bytes) {
  if (!ready(cache) || !slots_ok(num_slots)) return false;
  if (layers > 1 && (layer_rows < num_slots || layer_rows > (1ll << 40))) return false;
  return !scales || (row_bytes == kRow && aligned(scales, 4));
}

}  // namespace

extern "C" {

int mla_verify_drafts(const float* target_probs, int64_t target_batch_stride, int64_t target_row_stride,
                      const float* draft_probs, int64_t draft_batch_stride, int64_t draft_row_stride,
                      const int32_t* tokens, const int32_t* tree_parents, const float* uniforms, int32_t batch,
                      int32_t q_len, int32_t vocab, int32_t* path, int32_t* accepted, int32_t* next_token,
                      void* workspace, void* stream) {
  if (batch < 0 || q_len < 1 || vocab < 1) return MLA_ERR_INVALID_ARG;
  if (q_len > kMaxDrafts || vocab > kMaxVocab || (draft_probs && tree_parents)) return MLA_ERR_UNSUPPORTED;
  if (!stride_ok(target_batch_stride) || !stride_ok(target_row_stride)) return MLA_ERR_INVALID_ARG;
  if (draft_probs && (!stride_ok(draft_batch_stride) || !stride_ok(draft_row_stride))) return MLA_ERR_INVALID_ARG;
  if (batch == 0) return MLA_OK;
  if (!ready(target_probs, 4) || !ready(tokens, 4) || !ready(uniforms, 4) || !ready(path, 4) || !ready(accepted, 4) ||
      !ready(next_token, 4) || !aligned(draft_probs, 4) || !aligned(tree_parents, 4) || !aligned(workspace, 16))
    return MLA_ERR_INVALID_ARG;
  VerifyParams p{};
  p.target = target_probs;
  p.draft = draft_probs;
  p.tokens = tokens;
  p.parents = tree_parents;
  p.uniforms = uniforms;
  p.path = path;
  p.accepted = accepted;
  p.next = next_token;
  p.status = static_cast<int*>(workspace);
  p.t_bs = target_batch_stride;
  p.t_rs = target_row_stride;
  p.d_bs = draft_batch_stride;
  p.d_rs = draft_row_stride;
  p.batch = batch;
  p.width = q_len;
  p.vocab = vocab;
  return launch_verify(p, reinterpret_cast<cudaStream_t>(stream));
}

size_t mla_slots_workspace_bytes(int64_t num_slots) { return slots_ok(num_slots) ? slots_ws(num_slots).total : 0; }

int mla_repack_requests(const int32_t* kv_indptr, const int32_t* kv_indices, int64_t entries, int32_t batch,
                        const int32_t* sources, int32_t new_batch, const int32_t* path, const int32_t* accepted,
                        int32_t q_len, int32_t* new_indptr, int32_t* new_indices, int64_t capacity, int64_t num_slots,
                        int32_t* freed, int64_t freed_capacity, int32_t* freed_count, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (batch < 0 || new_batch < 0 || entries < 0 || entries > 0x7FFFFFFFll || capacity < 0 || capacity > kMaxCapacity ||
      freed_capacity < 0 || !slots_ok(num_slots))
    return MLA_ERR_INVALID_ARG;
  if ((path == nullptr) != (accepted == nullptr) || (freed == nullptr) != (freed_count == nullptr))
    return MLA_ERR_INVALID_ARG;
  if (path && q_len < 1) return MLA_ERR_INVALID_ARG;
  if ((path && q_len > kMaxDrafts) || (freed && batch > kMaxRequests) || new_batch > kMaxNew) return MLA_ERR_UNSUPPORTED;
  if (!ready(workspace)) return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < slots_ws(num_slots).total) return MLA_ERR_WORKSPACE;
  if (!ready(kv_indptr, 4) || !ready(new_indptr, 4) || (new_batch > 0 && !ready(sources, 4)) ||
      (entries > 0 && !ready(kv_indices, 4)) || (capacity > 0 && !ready(new_indices, 4)) || !aligned(path, 4) ||
      !aligned(accepted, 4) || !aligned(freed, 4) || !aligned(freed_count, 4))
    return MLA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  RepackParams p{};
  p.indptr = kv_indptr;
  p.indices = kv_indices;
  p.sources = sources;
  p.path = path;
  p.accepted = accepted;
  p.new_indptr = new_indptr;
  p.new_indices = new_indices;
  p.freed = freed;
  p.freed_count = freed_count;
  p.bits = reinterpret_cast<uint32_t*>(ws + slots_ws(num_slots).bits);
  p.status = reinterpret_cast<int*>(ws);
  p.entries = entries;
  p.capacity = capacity;
  p.freed_capacity = freed_capacity;
  p.num_slots = num_slots;
  p.batch = batch;
  p.new_batch = new_batch;
  p.width = path ? q_len : 0;
  return launch_repack(p, reinterpret_cast<cudaStream_t>(stream));
}

int mla_copy_rows(const void* src_cache, const float* src_scales, int64_t src_num_slots, int64_t src_layer_rows,
                  const int32_t* src_slots, void* dst_cache, float* dst_scales, int64_t dst_num_slots,
                  int64_t dst_layer_rows, const int32_t* dst_slots, int32_t rows, int32_t layers, int32_t row_bytes,
                  void* workspace, void* stream) {
  if (rows < 0 || layers < 0) return MLA_ERR_INVALID_ARG;
  if (row_bytes != kRow && row_bytes != 2 * kRow) return MLA_ERR_UNSUPPORTED;
  if ((src_scales == nullptr) != (dst_scales == nullptr) || !aligned(workspace, 16)) return MLA_ERR_INVALID_ARG;
  if (rows == 0 || layers == 0) return MLA_OK;
  if (!rows_ok(src_cache, src_scales, src_num_slots, src_layer_rows, layers, row_bytes) ||
      !rows_ok(dst_cache, dst_scales, dst_num_slots, dst_layer_rows, layers, row_bytes) || !ready(src_slots, 4) ||
      !ready(dst_slots, 4))
    return MLA_ERR_INVALID_ARG;
  MoveParams m{};
  m.src = static_cast<const uint8_t*>(src_cache);
  m.dst = static_cast<uint8_t*>(dst_cache);
  m.src_scales = src_scales;
  m.dst_scales = dst_scales;
  m.from = src_slots;
  m.to = dst_slots;
  m.status = static_cast<int*>(workspace);
  m.src_rows = src_layer_rows;
  m.dst_rows = dst_layer_rows;
  m.src_slots = src_num_slots;
  m.dst_slots = dst_num_slots;
  m.count = rows;
  m.layers = layers;
  m.row_bytes = row_bytes;
  return launch_move(m, rows, reinterpret_cast<cudaStream_t>(stream));
}

int mla_compact_cache(void* kv_cache, float* kv_scales, int64_t num_slots, int64_t layer_rows, int32_t layers,
                      int32_t row_bytes, const int32_t* kv_indptr, int32_t batch, const int32_t* kv_indices,
                      int64_t entries, int32_t* new_indices, int32_t* live_count, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (layers < 1 || batch < 0 || entries < 0 || entries > 0x7FFFFFFFll) return MLA_ERR_INVALID_ARG;
  if (row_bytes != kRow && row_bytes != 2 * kRow) return MLA_ERR_UNSUPPORTED;
  if (!rows_ok(kv_cache, kv_scales, num_slots, layer_rows, layers, row_bytes) || !ready(kv_indptr, 4) ||
      !ready(live_count, 4) || (entries > 0 && (!ready(kv_indices, 4) || !ready(new_indices, 4))) || !ready(workspace))
    return MLA_ERR_INVALID_ARG;
  const SlotsWs w = slots_ws(num_slots, workspace_bytes);
  if (workspace_bytes < w.total) return MLA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  CompactParams c{};
  c.indptr = kv_indptr;
  c.indices = kv_indices;
  c.new_indices = new_indices;
  c.live_count = live_count;
  c.bits = reinterpret_cast<uint32_t*>(ws + w.bits);
  c.live = reinterpret_cast<uint2*>(ws + w.live);
  c.holes = reinterpret_cast<int32_t*>(ws + w.holes);
  c.away = reinterpret_cast<int32_t*>(ws + w.away);
  c.counts = reinterpret_cast<int32_t*>(ws + w.counts);
  c.status = reinterpret_cast<int*>(ws);
  c.entries = entries;
  c.num_slots = num_slots;
  c.batch = batch;
  MoveParams m{};
  m.src = static_cast<const uint8_t*>(kv_cache);
  m.dst = static_cast<uint8_t*>(kv_cache);
  m.src_scales = kv_scales;
  m.dst_scales = kv_scales;
  m.from = c.away;
  m.to = c.holes;
  m.count_dev = c.counts + 1;
  m.status = c.status;
  m.src_rows = m.dst_rows = layer_rows;
  m.src_slots = m.dst_slots = num_slots;
  m.layers = layers;
  m.row_bytes = row_bytes;
  return launch_compact(c, m, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
