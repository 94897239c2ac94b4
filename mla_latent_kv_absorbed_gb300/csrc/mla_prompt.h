// Shared by the prompt-side entry points (mla_prompt_api.cpp) and their
// kernels: rotary positions, latent expansion and the expanded attention.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <vector>

#include "mla_internal.h"

namespace mla {

constexpr int kPairs = kRope / 2;     // rotated pairs of a head
constexpr int kNope = 128;            // per-head key width beside the rope part, and value width
constexpr int kQk = kNope + kRope;    // 192

// Frequencies of the 32 pairs as 64-bit fractions of a turn per position
// (passed by value: they are constants of the model), and the factor on cos
// and sin.
struct RopeFreqs {
  uint64_t f[kPairs];
  float amplitude;
  int interleaved;            // pairs (2i, 2i+1), else (i, i + 32)
};

struct RopeQueryParams {
  const uint16_t* q;          // head h of token t at q + t*q_ts + h*q_hs: nope then rope
  const int32_t* positions;   // [tokens]
  uint16_t* q_rope;           // rope part of (t, h) at q_rope + t*r_ts + h*r_hs
  uint16_t* q_nope;           // dense [tokens, heads, nope], or null
  long long q_ts, q_hs, r_ts, r_hs;
  int tokens, heads, nope;
};

struct RopeAppendParams {
  void* kv_cache;             // [num_slots, 576] bf16 or E4M3
  const uint16_t* rows;       // row t at rows + t*row_stride
  const int32_t* positions;   // [tokens]
  const int32_t* slots;       // [tokens]
  const uint16_t* weight;     // bf16 [512] norm weight, or null: latents unchanged
  int* status;                // status word, or null
  long long num_slots, row_stride;
  int tokens;
  float eps;
  float kv_scale;             // FP8 cache only
  float kv_recip;             // 1 / kv_scale where a product with it is the quotient exactly, else 0
};

struct ExpandParams {
  const uint8_t* kv_cache;    // [num_slots, 576] bf16 or E4M3
  const int32_t* kv_indices;  // [tokens]
  uint16_t *k_nope, *v;       // [tokens, heads, 128]
  uint16_t* k_rope;           // [tokens, 64]
  int* status;                // status word, or null
  long long num_slots;
  int tokens, heads;
  float kv_scale;             // FP8 cache only
};

// ---- prefill plan words --------------------------------------------------
constexpr int32_t kPfMagic = 0x4D4C4150;
constexpr int32_t kPfVersion = 1;
constexpr int kPfHeaderWords = 16;
enum PfHeader : int {
  kPMagic = 0, kPVersion, kPBatch, kPHeads, kPCausal, kPQTokens, kPKvTokens, kPItems, kPPartials, kPMerges,
  kPHeadGroup /* heads whose items are launched together */, kPTotalWords, kPNumSms,
  kPRows /* query rows of an item, at most: 256, or 512 for CTA pairs */,
  kPSolo /* no item has more than 128 */,
  kPTail /* of the items, the last so many wait until all heads' others have been handed out */
};
constexpr int kPfItemWords = 8;       // request, q0, nq, k0, nk, off, partial (or -1), 0
constexpr int kPfMergeWords = 4;      // q0, nq, first partial, last partial + 1
constexpr int kPfRows = 256;          // query rows of one CTA's item, at most
constexpr int kPfKeys = 128;          // keys of a tile
constexpr long long kPfMaxBlocks = 0x7FFF0000;   // items x heads: every block of the launch counts one past them
constexpr int32_t kPfNoLimit = 0x3FFFFFFF;   // off of an item without a causal limit

// Words of the workspace's status header that the prefill kernel counts in
// (zero between launches): items handed out, blocks that have finished, items
// worked on.
constexpr int kWsCounter = 16, kWsDone = 17, kWsWorked = 18;

inline int pf_items_off(const int32_t*) { return kPfHeaderWords; }
inline int pf_merge_off(const int32_t* h) { return kPfHeaderWords + kPfItemWords * h[kPItems]; }
// Workspace: status header, partial outputs [partials][heads][rows][128] fp32,
// partial log-sum-exps [partials][heads][rows].
inline size_t pf_part_lse_off(const int32_t* h) {
  return kWsHeaderBytes + static_cast<size_t>(h[kPPartials]) * h[kPHeads] * h[kPRows] * kNope * 4;
}
inline size_t pf_workspace_bytes(const int32_t* h) {
  return pf_part_lse_off(h) + static_cast<size_t>(h[kPPartials]) * h[kPHeads] * h[kPRows] * 4;
}

int build_prefill_plan(const int32_t* q_indptr, const int32_t* kv_indptr, int batch, int heads, int causal,
                       int num_sms, std::vector<int32_t>& words);

struct PrefillParams {
  const int32_t* items;       // device plan items
  const int32_t* merges;      // device plan merge entries
  const uint16_t *q, *k_nope, *k_rope, *v;
  long long q_ts, q_hs, k_ts, k_hs, kr_ts, v_ts, v_hs;   // strides in elements
  uint16_t* out;              // [q_tokens, heads, 128] bf16
  float* lse;                 // [q_tokens, heads] or null
  float* part_o;
  float* part_lse;
  int* status;
  int n_items, n_tail, n_merges, heads, head_group, partials, rows;
  bool solo;                  // no item has more than 128 rows
  int q_tokens, kv_tokens;
  float scale_log2;           // |sm_scale| * log2(e), > 0
  int negate;                 // sm_scale < 0: the scores are those of -q
};

int launch_rope_query(const RopeQueryParams& p, const RopeFreqs& f, cudaStream_t stream);
int launch_rope_append(const RopeAppendParams& p, const RopeFreqs& f, bool fp8, cudaStream_t stream);
// How the expansion is tiled: columns of a tile, and whether CTA pairs share
// one.  Maps: w_kc as [heads * 128, 512] (box: 128 rows x 64), w_vc as [heads *
// 512, 128] (box 64 x 64).
struct ExpandTiling {
  int cols;
  bool pair;
};
ExpandTiling expand_tiling(int tokens, int heads, int sms);
int launch_expand(const ExpandParams& p, const CUtensorMap (&tm)[2], ExpandTiling tiling, int sms, bool fp8,
                  cudaStream_t stream);
// tm_q over q as [rows, heads, 192] (box 128 rows x 64), tm_k and tm_v over
// [keys, heads, 128] (boxes of 128 - for CTA pairs 64 - and 64 keys x 64), tm_kr
// over [keys, 64] (box as tm_k's).
int launch_prefill(const PrefillParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_kr,
                   const CUtensorMap& tm_v, cudaStream_t stream);

}  // namespace mla
