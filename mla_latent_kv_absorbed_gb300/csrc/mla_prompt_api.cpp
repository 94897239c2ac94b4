// The prompt side of the C ABI (declared in include/mla_decode.h): argument
// checks and dispatch of the rotary, expansion and expanded-attention
// kernels.  Nothing here allocates device memory or synchronises; nothing
// throws across the boundary.
#include <cmath>
#include <cstring>
#include <limits>
#include <new>
#include <vector>

#include "mla_launch.h"
#include "mla_prompt.h"

using namespace mla;

namespace {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool ready(const void* p, uintptr_t n = 16) { return p && aligned(p, n); }

// A stride in elements that keeps 16-byte pieces aligned (bf16) and, in bytes,
// below a tensor map's 2^40; the `n` rows of `width` must not overlap.  That of a
// dimension of one is not used: anything.
inline bool stride_ok(int64_t s, int64_t n, int64_t width = 0) {
  return n <= 1 || (s >= width && s < (1ll << 38) && s % 8 == 0);
}

// Whether `n` rotary parts, `step` apart, lie apart and end before the next of
// `outer` such groups, `stride` apart (by division: (n - 1) * step may pass 64 bits).
inline bool inside(int64_t n, int64_t step, int64_t outer, int64_t stride) {
  if (n > 1 && step < kRope) return false;
  return outer <= 1 || (stride >= kRope && (n <= 1 || n - 1 <= (stride - kRope) / step));
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(p);
    return nullptr;
  }();
  return fn;
}

// bf16 [rows, heads, width] with strides in elements (heads 0: [rows, width]),
// boxes of `box_rows` (<= 256) rows of one head x 64 values in the 128-byte
// swizzle; reads past the last row give zeros.  The stride of a dimension of one is not used.
bool make_map(CUtensorMap* m, const void* base, int64_t rows, int64_t row_stride, int64_t heads, int64_t head_stride,
              int width, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t rs = static_cast<cuuint64_t>(rows > 1 ? row_stride : width) * 2;
  const cuuint64_t hs = static_cast<cuuint64_t>(heads > 1 ? head_stride : width) * 2;
  const int rank = heads > 0 ? 3 : 2;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {hs, rs};
  cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(box_rows)}, step[3] = {1, 1, 1};
  if (rank == 2) {
    dims[1] = dims[2];
    strides[0] = rs;
    box[1] = box[2];
  }
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool rope_args(const uint64_t* freqs, float amplitude, int32_t interleaved, RopeFreqs* f) {
  if (!freqs || !std::isfinite(amplitude) || (interleaved != 0 && interleaved != 1)) return false;
  std::memcpy(f->f, freqs, sizeof f->f);
  f->amplitude = amplitude;
  f->interleaved = interleaved;
  return true;
}

}  // namespace

extern "C" {

int mla_rope_frequencies(double theta, int32_t scaling, double factor, int32_t original_positions, double beta_fast,
                         double beta_slow, uint64_t* freqs) {
  if (!freqs || !std::isfinite(theta) || !(theta > 1.0)) return MLA_ERR_INVALID_ARG;
  if (scaling < 0 || scaling > 2) return MLA_ERR_UNSUPPORTED;
  if (scaling != 0 && (!std::isfinite(factor) || !(factor >= 1.0))) return MLA_ERR_INVALID_ARG;
  const double pi = 3.14159265358979323846;
  double low = 0.0, high = 0.0;
  if (scaling == 2) {
    if (original_positions < 1 || !std::isfinite(beta_fast) || !(beta_slow > 0.0) || !(beta_fast >= beta_slow))
      return MLA_ERR_INVALID_ARG;
    // the pair that makes `beta` turns over the original context
    auto pair_of = [&](double beta) { return kRope * std::log(original_positions / (beta * 2.0 * pi)) / (2.0 * std::log(theta)); };
    low = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
    high = std::fmin(std::ceil(pair_of(beta_slow)), kRope - 1.0);
  }
  for (int i = 0; i < kPairs; ++i) {
    const double inv = std::pow(theta, -2.0 * i / kRope);
    double f = inv;
    if (scaling == 1) f = inv / factor;
    if (scaling == 2) {
      const double ramp = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
      f = inv / factor * ramp + inv * (1.0 - ramp);
    }
    freqs[i] = static_cast<uint64_t>(std::nearbyint(std::ldexp(f / (2.0 * pi), 64)));   // f / 2 pi < 0.16: fits
  }
  return MLA_OK;
}

int mla_rope_query(const void* q, int64_t q_token_stride, int64_t q_head_stride, const int32_t* positions,
                   int32_t tokens, int32_t num_heads, int32_t nope_dim, const uint64_t* freqs, float amplitude,
                   int32_t interleaved, void* q_rope, int64_t rope_token_stride, int64_t rope_head_stride,
                   void* q_nope, void* stream) {
  RopeFreqs f;
  if (!rope_args(freqs, amplitude, interleaved, &f)) return MLA_ERR_INVALID_ARG;
  if (tokens < 0 || num_heads < 1 || num_heads > 65535 || nope_dim < 0) return MLA_ERR_INVALID_ARG;
  if (nope_dim % 8 != 0 || nope_dim > 65536) return MLA_ERR_UNSUPPORTED;
  if (!stride_ok(q_token_stride, tokens) || !stride_ok(q_head_stride, num_heads) ||
      !stride_ok(rope_token_stride, tokens) || !stride_ok(rope_head_stride, num_heads))
    return MLA_ERR_INVALID_ARG;
  // rows of the output must not overlap, whichever of tokens and heads is outer
  const int64_t T = tokens, H = num_heads;
  const bool heads_inner = inside(H, rope_head_stride, T, rope_token_stride);
  const bool tokens_inner = inside(T, rope_token_stride, H, rope_head_stride);
  if (!heads_inner && !tokens_inner) return MLA_ERR_INVALID_ARG;
  if (tokens == 0) return MLA_OK;
  if (!ready(q) || !ready(positions, 4) || !ready(q_rope) || (q_nope && !aligned(q_nope, 16)))
    return MLA_ERR_INVALID_ARG;
  RopeQueryParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.positions = positions;
  p.q_rope = static_cast<uint16_t*>(q_rope);
  p.q_nope = nope_dim > 0 ? static_cast<uint16_t*>(q_nope) : nullptr;
  p.q_ts = q_token_stride;
  p.q_hs = q_head_stride;
  p.r_ts = rope_token_stride;
  p.r_hs = rope_head_stride;
  p.tokens = tokens;
  p.heads = num_heads;
  p.nope = nope_dim;
  return launch_rope_query(p, f, reinterpret_cast<cudaStream_t>(stream));
}

namespace {
int rope_append(void* kv_cache, int64_t num_slots, const int32_t* slots, const void* rows, int64_t row_stride,
                const int32_t* positions, int32_t tokens, const void* norm_weight, float eps, const uint64_t* freqs,
                float amplitude, int32_t interleaved, bool fp8, float kv_scale, void* workspace, void* stream) {
  RopeFreqs f;
  if (!rope_args(freqs, amplitude, interleaved, &f)) return MLA_ERR_INVALID_ARG;
  if (tokens < 0 || num_slots < 1 || num_slots > 0x7FFFFFFFll || !std::isfinite(eps) || !(eps >= 0.f))
    return MLA_ERR_INVALID_ARG;
  if (fp8 && (!std::isfinite(kv_scale) || !(kv_scale > 0.f))) return MLA_ERR_INVALID_ARG;
  if (!stride_ok(row_stride, tokens, kRow)) return MLA_ERR_INVALID_ARG;
  if (tokens == 0) return MLA_OK;
  if (!ready(kv_cache) || !ready(slots, 4) || !ready(rows) || !ready(positions, 4) ||
      (norm_weight && !aligned(norm_weight, 16)) || (workspace && !aligned(workspace, 16)))
    return MLA_ERR_INVALID_ARG;
  RopeAppendParams p{};
  p.kv_cache = kv_cache;
  p.rows = static_cast<const uint16_t*>(rows);
  p.positions = positions;
  p.slots = slots;
  p.weight = static_cast<const uint16_t*>(norm_weight);
  p.status = static_cast<int*>(workspace);
  p.num_slots = num_slots;
  p.row_stride = row_stride;
  p.tokens = tokens;
  p.eps = eps;
  p.kv_scale = kv_scale;
  int exponent = 0;
  if (std::frexp(kv_scale, &exponent) == 0.5f && std::isnormal(kv_scale) && std::isnormal(1.f / kv_scale))
    p.kv_recip = 1.f / kv_scale;
  return launch_rope_append(p, f, fp8, reinterpret_cast<cudaStream_t>(stream));
}
}  // namespace

int mla_rope_append_kv(void* kv_cache, int64_t num_slots, const int32_t* slots, const void* rows, int64_t row_stride,
                       const int32_t* positions, int32_t tokens, const void* norm_weight, float eps,
                       const uint64_t* freqs, float amplitude, int32_t interleaved, void* workspace, void* stream) {
  return rope_append(kv_cache, num_slots, slots, rows, row_stride, positions, tokens, norm_weight, eps, freqs,
                     amplitude, interleaved, false, 1.f, workspace, stream);
}

int mla_rope_append_kv_fp8(void* kv_cache, int64_t num_slots, const int32_t* slots, const void* rows,
                           int64_t row_stride, const int32_t* positions, int32_t tokens, const void* norm_weight,
                           float eps, const uint64_t* freqs, float amplitude, int32_t interleaved, float kv_scale,
                           void* workspace, void* stream) {
  return rope_append(kv_cache, num_slots, slots, rows, row_stride, positions, tokens, norm_weight, eps, freqs,
                     amplitude, interleaved, true, kv_scale, workspace, stream);
}

namespace {
int expand(const void* kv_cache, int64_t num_slots, const int32_t* kv_indices, int32_t tokens, const void* w_kc,
           const void* w_vc, int32_t num_heads, bool fp8, float kv_scale, void* k_nope, void* k_rope, void* v,
           void* workspace, void* stream) {
  if (tokens < 0 || num_heads < 1 || num_heads > 65535 || num_slots < 1 || num_slots > 0x7FFFFFFFll)
    return MLA_ERR_INVALID_ARG;
  if (fp8 && (!std::isfinite(kv_scale) || !(kv_scale > 0.f))) return MLA_ERR_INVALID_ARG;
  if (tokens == 0) return MLA_OK;
  if (!ready(kv_cache) || !ready(kv_indices, 4) || !ready(w_kc) || !ready(w_vc) || !ready(k_nope) || !ready(k_rope) ||
      !ready(v) || (workspace && !aligned(workspace, 16)))
    return MLA_ERR_INVALID_ARG;
  ExpandParams p{};
  p.kv_cache = static_cast<const uint8_t*>(kv_cache);
  p.kv_indices = kv_indices;
  p.k_nope = static_cast<uint16_t*>(k_nope);
  p.v = static_cast<uint16_t*>(v);
  p.k_rope = static_cast<uint16_t*>(k_rope);
  p.status = static_cast<int*>(workspace);
  p.num_slots = num_slots;
  p.tokens = tokens;
  p.heads = num_heads;
  p.kv_scale = kv_scale;
  const int sms = device_sm_count();
  if (sms < 1) return MLA_ERR_CUDA;
  const int64_t H = num_heads;
  CUtensorMap tm[2];
  if (!make_map(&tm[0], w_kc, H * kNope, kLatent, 0, 0, kLatent, 128) ||
      !make_map(&tm[1], w_vc, H * kLatent, kNope, 0, 0, kNope, 64))
    return MLA_ERR_CUDA;
  return launch_expand(p, tm, expand_tiling(tokens, num_heads, sms), sms, fp8, reinterpret_cast<cudaStream_t>(stream));
}
}  // namespace

int mla_expand_kv(const void* kv_cache, int64_t num_slots, const int32_t* kv_indices, int32_t tokens,
                  const void* w_kc, const void* w_vc, int32_t num_heads, void* k_nope, void* k_rope, void* v,
                  void* workspace, void* stream) {
  return expand(kv_cache, num_slots, kv_indices, tokens, w_kc, w_vc, num_heads, false, 1.f, k_nope, k_rope, v,
                workspace, stream);
}

int mla_expand_kv_fp8(const void* kv_cache, int64_t num_slots, float kv_scale, const int32_t* kv_indices,
                      int32_t tokens, const void* w_kc, const void* w_vc, int32_t num_heads, void* k_nope,
                      void* k_rope, void* v, void* workspace, void* stream) {
  return expand(kv_cache, num_slots, kv_indices, tokens, w_kc, w_vc, num_heads, true, kv_scale, k_nope, k_rope, v,
                workspace, stream);
}

int mla_prefill_plan(const int32_t* q_indptr, const int32_t* kv_indptr, int32_t batch, int32_t num_heads,
                     int32_t causal, int32_t num_sms, int32_t* plan, size_t plan_words, size_t* plan_words_needed,
                     size_t* workspace_bytes) {
  if (batch < 0 || !q_indptr || !kv_indptr || q_indptr[0] != 0 || kv_indptr[0] != 0) return MLA_ERR_INVALID_ARG;
  for (int b = 0; b < batch; ++b)
    if (q_indptr[b + 1] < q_indptr[b] || kv_indptr[b + 1] < kv_indptr[b]) return MLA_ERR_INVALID_ARG;
  if (num_heads < 1 || num_heads > 65535 || (causal != 0 && causal != 1) || num_sms < 0) return MLA_ERR_INVALID_ARG;
  // lengths whose causal limits, as relative key numbers, stay below the "no limit" mark
  if (q_indptr[batch] >= kPfNoLimit || kv_indptr[batch] >= kPfNoLimit) return MLA_ERR_UNSUPPORTED;
  if (num_sms == 0) {
    num_sms = device_sm_count();
    if (num_sms < 1) return MLA_ERR_CUDA;
  }
  try {
    std::vector<int32_t> words;
    const int st = build_prefill_plan(q_indptr, kv_indptr, batch, num_heads, causal, num_sms, words);
    if (st != MLA_OK) return st;
    if (plan_words_needed) *plan_words_needed = words.size();
    if (workspace_bytes) *workspace_bytes = pf_workspace_bytes(words.data());
    if (!plan) return MLA_OK;
    if (plan_words < words.size()) return MLA_ERR_WORKSPACE;
    std::memcpy(plan, words.data(), words.size() * sizeof(int32_t));
    return MLA_OK;
  } catch (const std::bad_alloc&) {
    return MLA_ERR_WORKSPACE;               // host memory for the plan
  } catch (...) {
    return MLA_ERR_INVALID_ARG;
  }
}

namespace {
bool prefill_header_ok(const int32_t* h) {
  if (!h || h[kPMagic] != kPfMagic || h[kPVersion] != kPfVersion) return false;
  if (h[kPBatch] < 0 || h[kPHeads] < 1 || h[kPHeads] > 65535 || h[kPQTokens] < 0 || h[kPKvTokens] < 0 ||
      h[kPItems] < 0 || h[kPPartials] < 0 || h[kPMerges] < 0 || h[kPMerges] > 65535 || h[kPHeadGroup] < 1 ||
      h[kPHeadGroup] > h[kPHeads] || (h[kPRows] != kPfRows && h[kPRows] != 2 * kPfRows) ||
      (h[kPSolo] != 0 && h[kPSolo] != 1) || h[kPTail] < 0 || h[kPTail] > h[kPItems])
    return false;
  if (static_cast<long long>(h[kPItems]) * h[kPHeads] > kPfMaxBlocks) return false;
  const long long words = kPfHeaderWords + static_cast<long long>(kPfItemWords) * h[kPItems] +
                          static_cast<long long>(kPfMergeWords) * h[kPMerges];
  return words == h[kPTotalWords];
}
}  // namespace

int mla_prefill_run(const int32_t* plan_host, const int32_t* plan_dev, const void* q, int64_t q_token_stride,
                    int64_t q_head_stride, const void* k_nope, int64_t k_token_stride, int64_t k_head_stride,
                    const void* k_rope, int64_t k_rope_stride, const void* v, int64_t v_token_stride,
                    int64_t v_head_stride, float sm_scale, void* out, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!prefill_header_ok(plan_host) || !ready(plan_dev)) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(sm_scale)) return MLA_ERR_INVALID_ARG;
  if (!ready(workspace)) return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < pf_workspace_bytes(plan_host)) return MLA_ERR_WORKSPACE;
  if (plan_host[kPQTokens] == 0) return MLA_OK;
  const int H = plan_host[kPHeads];
  const int64_t nq = plan_host[kPQTokens], nk = plan_host[kPKvTokens];
  if (!stride_ok(q_token_stride, nq, kQk) || !stride_ok(q_head_stride, H, kQk)) return MLA_ERR_INVALID_ARG;
  if (nk > 0 && (!stride_ok(k_token_stride, nk, kNope) || !stride_ok(k_head_stride, H, kNope) ||
                 !stride_ok(k_rope_stride, nk, kRope) || !stride_ok(v_token_stride, nk, kNope) ||
                 !stride_ok(v_head_stride, H, kNope)))
    return MLA_ERR_INVALID_ARG;
  if (!ready(q) || !ready(out) || (lse && !aligned(lse, 4))) return MLA_ERR_INVALID_ARG;
  if (plan_host[kPKvTokens] > 0 && (!ready(k_nope) || !ready(k_rope) || !ready(v))) return MLA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PrefillParams p{};
  p.items = plan_dev + pf_items_off(plan_host);
  p.merges = plan_dev + pf_merge_off(plan_host);
  p.q = static_cast<const uint16_t*>(q);
  p.k_nope = static_cast<const uint16_t*>(k_nope);
  p.k_rope = static_cast<const uint16_t*>(k_rope);
  p.v = static_cast<const uint16_t*>(v);
  p.q_ts = q_token_stride;
  p.q_hs = q_head_stride;
  p.k_ts = k_token_stride;
  p.k_hs = k_head_stride;
  p.kr_ts = k_rope_stride;
  p.v_ts = v_token_stride;
  p.v_hs = v_head_stride;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.part_o = reinterpret_cast<float*>(ws + kWsHeaderBytes);
  p.part_lse = reinterpret_cast<float*>(ws + pf_part_lse_off(plan_host));
  p.status = reinterpret_cast<int*>(ws);
  p.n_items = plan_host[kPItems];
  p.n_tail = plan_host[kPTail];
  p.n_merges = plan_host[kPMerges];
  p.heads = H;
  p.head_group = plan_host[kPHeadGroup];
  p.partials = plan_host[kPPartials];
  p.rows = plan_host[kPRows];
  p.solo = plan_host[kPSolo] != 0;
  const int key_box = p.rows > kPfRows ? kPfKeys / 2 : kPfKeys;
  p.q_tokens = plan_host[kPQTokens];
  p.kv_tokens = plan_host[kPKvTokens];
  // the kernel takes maxima of the products before it scales them, and masks
  // them by -inf: a positive scale.  0 becomes the smallest number, 2^-149,
  // which leaves every finite fp32 score (below 2^128) under 2^-21.
  p.scale_log2 = std::fmax(std::fabs(sm_scale) * 1.4426950408889634f, std::numeric_limits<float>::denorm_min());
  p.negate = sm_scale < 0.f;
  if (!std::isfinite(p.scale_log2)) return MLA_ERR_INVALID_ARG;
  CUtensorMap tm_q, tm_k, tm_kr, tm_v;
  if (!make_map(&tm_q, q, nq, q_token_stride, H, q_head_stride, kQk, 128)) return MLA_ERR_CUDA;
  if (nk == 0) {
    tm_k = tm_kr = tm_v = tm_q;                 // nothing is loaded through them
  } else if (!make_map(&tm_k, k_nope, nk, k_token_stride, H, k_head_stride, kNope, key_box) ||
             !make_map(&tm_kr, k_rope, nk, k_rope_stride, 0, 0, kRope, key_box) ||
             !make_map(&tm_v, v, nk, v_token_stride, H, v_head_stride, kNope, 64)) {
    return MLA_ERR_CUDA;
  }
  return launch_prefill(p, tm_q, tm_k, tm_kr, tm_v, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
