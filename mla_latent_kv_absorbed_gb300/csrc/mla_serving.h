// Shared by the entry points between two decode steps (mla_serving_api.cpp)
// and their kernels: verification of drafts, request lists, row moves.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "mla_internal.h"

namespace mla {

constexpr int kMaxDrafts = 64;        // drafts of a request (a 64-bit set of them)
constexpr int kMaxVocab = 1 << 30;    // (four elements to a block, and those of the last one are counted in 32 bits)
constexpr int kMaxRequests = 65536;   // requests of a batch whose lists are rewritten with their freed slots
constexpr int kMaxNew = 1 << 20;      // new requests: every block adds up the lengths of all before its own
constexpr long long kMaxCapacity = 0x7FFFFFFEll;   // entries of the new lists: a sum of lengths ends at 2^31 - 1, and is past it

struct VerifyParams {
  const float* target;        // row n of request b at target + b*t_bs + n*t_rs
  const float* draft;         // row c of request b at draft + b*d_bs + c*d_rs, or null
  const int32_t* tokens;      // [batch, width]
  const int32_t* parents;     // [batch, width], or null: a chain
  const float* uniforms;      // [batch, width]
  int32_t* path;              // [batch, width]
  int32_t* accepted;          // [batch]
  int32_t* next;              // [batch]
  int* status;                // status word, or null
  long long t_bs, t_rs, d_bs, d_rs;
  int batch, width, vocab;
};

int launch_verify(const VerifyParams& p, cudaStream_t stream);

// ---- workspace of the calls that keep sets of slots --------------------------
// A set of slots is a bitmap, 32 to a word; `bits` is all zero between calls.  It
// lies at the front and the rest at the end, so that the rest of a small pool's
// call leaves the words of a larger pool's set alone.
struct SlotsWs {
  size_t bits;                // uint32 [words]
  size_t live;                // uint2 [words]: a word of the live slots, and how many live ones are in the words before
  size_t holes;               // int32 [slots / 2]: free slots among the lowest n, ascending
  size_t away;                // int32 [slots / 2]: live slots past them, descending (the k-th of them in ascending
                              // order, which goes to holes[k], is entry count - 1 - k)
  size_t counts;              // int32 [2]: live slots, and those of them past the lowest n
  size_t total;
};
inline SlotsWs slots_ws(int64_t num_slots, size_t bytes = 0) {
  const size_t n = static_cast<size_t>(num_slots), words = (n + 31) / 32;
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t live = up(8 * words), list = up(4 * (n / 2)), rest = live + 2 * list + 256;
  SlotsWs w{};
  w.bits = kWsHeaderBytes;
  w.total = up(w.bits + 4 * words) + rest;
  w.live = (bytes > w.total ? bytes & ~size_t(255) : w.total) - rest;
  w.holes = w.live + live;
  w.away = w.holes + list;
  w.counts = w.away + list;
  return w;
}

struct RepackParams {
  const int32_t* indptr;      // [batch + 1]
  const int32_t* indices;     // [entries]
  const int32_t* sources;     // [new_batch]
  const int32_t* path;        // [batch, width], or null
  const int32_t* accepted;    // [batch], or null
  int32_t* new_indptr;        // [new_batch + 1]
  int32_t* new_indices;       // [capacity]
  int32_t* freed;             // [freed_capacity], or null: nothing is kept track of
  int32_t* freed_count;       // [1]
  uint32_t* bits;             // [words], zero
  int* status;
  long long entries, capacity, freed_capacity, num_slots;
  int batch, new_batch, width;
  bool marked;                // (launch_repack: the marking kernel runs before the others)
};

int launch_repack(const RepackParams& p, cudaStream_t stream);

struct MoveParams {
  const uint8_t* src;         // row s of layer l at src + (l * src_rows + s) * row_bytes
  uint8_t* dst;
  const float* src_scales;    // [layers, src_rows], or null
  float* dst_scales;
  const int32_t* from;        // [count]
  const int32_t* to;          // [count]
  const int32_t* count_dev;   // device count in the place of `count`, or null
  int* status;                // status word, or null
  long long src_rows, dst_rows, src_slots, dst_slots;
  int count, layers, row_bytes;
};

int launch_move(const MoveParams& p, long long most, cudaStream_t stream);

struct CompactParams {
  const int32_t* indptr;      // [batch + 1]; entry `batch` counts the entries of indices
  const int32_t* indices;     // [entries at most]
  int32_t* new_indices;
  int32_t* live_count;        // [1]
  uint32_t* bits;             // [words], zero
  uint2* live;                // [words]
  int32_t *holes, *away;      // [num_slots / 2], as in SlotsWs
  int32_t* counts;            // [2]
  int* status;
  long long entries, num_slots;
  int batch;
};

int launch_compact(const CompactParams& c, const MoveParams& m, cudaStream_t stream);

}  // namespace mla
