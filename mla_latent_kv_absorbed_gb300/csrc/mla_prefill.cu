// Attention of ragged sequences over expanded keys and values:
//   s_ij = sm_scale (q_i . [k_nope_j, k_rope_j]),  out_i = softmax_j(s_ij) v_j,
//   lse_i = ln sum_j exp(s_ij),
// j up to the causal limit of row i (the sequences' ends aligned).  One pass
// over the keys with the running maximum and sum.
#include "mla_device.cuh"
#include "mla_prompt.h"

namespace mla {
namespace {

constexpr int kThreads = kPfRows;      // one thread a query row
constexpr int kTile = 32;              // keys in shared memory at a time

struct Item {
  int q0, nq, k0, nk, off, part;
};

// The item's words, or false (and MLA_ERR_PLAN_MISMATCH) when it does not lie
// inside the arrays of this launch.
__device__ __forceinline__ bool load_item(const PrefillParams& p, int i, Item& it) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(p.items) + 2 * i);
  const int4 b = __ldg(reinterpret_cast<const int4*>(p.items) + 2 * i + 1);
  it = Item{a.y, a.z, a.w, b.x, b.y, b.z};
  return it.q0 >= 0 && it.nq >= 1 && it.nq <= kPfRows && it.q0 <= p.q_tokens - it.nq && it.k0 >= 0 && it.nk >= 0 &&
         it.k0 <= p.kv_tokens - it.nk && it.part >= -1 && it.part < p.partials && it.off >= -kPfNoLimit &&
         it.off <= kPfNoLimit;
}

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// Simple form: a thread keeps its row's query and output in registers and
// reads the keys and values of a tile from shared memory, one key at a time.
__global__ void __launch_bounds__(kThreads) prefill_kernel(const PrefillParams p) {
  __shared__ __align__(16) float ks[kTile][kQk];
  __shared__ __align__(16) float vs[kTile][kNope];
  const int h = blockIdx.y;
  Item it;
  if (!load_item(p, blockIdx.x, it)) {
    if (threadIdx.x == 0) record_status(p.status, MLA_ERR_PLAN_MISMATCH);
    return;
  }
  const int r = threadIdx.x;
  const bool live = r < it.nq;
  const uint16_t* qs = p.q + (it.q0 + (live ? r : 0)) * p.q_ts + h * p.q_hs;
  float o[kNope];
#pragma unroll
  for (int d = 0; d < kNope; ++d) o[d] = 0.f;
  float m = -INFINITY, l = 0.f;
  const int lim = min(it.nk, max(0, it.off + r + 1));       // keys this row sees
  for (int t0 = 0; t0 < it.nk; t0 += kTile) {
    const int n = min(kTile, it.nk - t0);
    __syncthreads();
    for (int i = r; i < n * kQk; i += kThreads) {
      const int j = i / kQk, d = i - j * kQk;
      const long long key = it.k0 + t0 + j;
      ks[j][d] = bf(d < kNope ? __ldg(p.k_nope + key * p.k_ts + h * p.k_hs + d)
                              : __ldg(p.k_rope + key * p.kr_ts + d - kNope));
    }
    for (int i = r; i < n * kNope; i += kThreads) {
      const int j = i / kNope, d = i - j * kNope;
      vs[j][d] = bf(__ldg(p.v + (it.k0 + t0 + j) * p.v_ts + h * p.v_hs + d));
    }
    __syncthreads();
    const int n_row = live ? min(n, lim - t0) : 0;
    for (int j = 0; j < n_row; ++j) {
      float s = 0.f;
#pragma unroll 4
      for (int d = 0; d < kQk; d += 4) {
        const float4 k = *reinterpret_cast<const float4*>(&ks[j][d]);
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(qs + d));
        s = fmaf(__uint_as_float(w.x << 16), k.x, s);
        s = fmaf(__uint_as_float(w.x & 0xFFFF0000u), k.y, s);
        s = fmaf(__uint_as_float(w.y << 16), k.z, s);
        s = fmaf(__uint_as_float(w.y & 0xFFFF0000u), k.w, s);
      }
      s *= p.scale_log2;
      if (s > m) {
        const float f = exp2f(m - s);
        l *= f;
#pragma unroll
        for (int d = 0; d < kNope; ++d) o[d] *= f;
        m = s;
      }
      const float e = s == -INFINITY ? 0.f : exp2f(s - m);
      l += e;
#pragma unroll
      for (int d = 0; d < kNope; ++d) o[d] = fmaf(e, vs[j][d], o[d]);
    }
  }
  if (!live) return;
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  const float lse = l > 0.f || l != l ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
  if (it.part >= 0) {
    const size_t row = (static_cast<size_t>(it.part) * p.heads + h) * kPfRows + r;
    p.part_lse[row] = lse;
    for (int d = 0; d < kNope; ++d) p.part_o[row * kNope + d] = o[d] * inv;
    return;
  }
  const size_t row = static_cast<size_t>(it.q0 + r) * p.heads + h;
  if (p.lse) p.lse[row] = lse;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + row * kNope);
#pragma unroll
  for (int d = 0; d < kNope; d += 2) out[d / 2] = pack_bf16x2(o[d] * inv, o[d + 1] * inv);
}

// Joins the pieces of a cut tile: one warp a (row, head), 4 values a lane.
__global__ void __launch_bounds__(256) prefill_merge_kernel(const PrefillParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int4 e = __ldg(reinterpret_cast<const int4*>(p.merges) + blockIdx.y);
  const int q0 = e.x, nq = e.y, p0 = e.z, p1 = e.w;
  if (q0 < 0 || nq < 1 || nq > kPfRows || q0 > p.q_tokens - nq || p0 < 0 || p1 <= p0 || p1 > p.partials) {
    if (threadIdx.x == 0) record_status(p.status, MLA_ERR_PLAN_MISMATCH);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int r = i / p.heads, h = i - r * p.heads;
  if (r >= nq) return;
  float m = -INFINITY;
  bool bad = false;
  for (int k = p0; k < p1; ++k) {
    const float s = p.part_lse[(static_cast<size_t>(k) * p.heads + h) * kPfRows + r];
    bad |= s != s;
    m = fmaxf(m, s);
  }
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  for (int k = p0; k < p1; ++k) {
    const size_t row = (static_cast<size_t>(k) * p.heads + h) * kPfRows + r;
    const float s = p.part_lse[row];
    if (s == -INFINITY) continue;                          // nothing seen in this piece
    const float w = expf(s - m);
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + row * kNope + 4 * lane);
    l += w;
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  }
  const bool any = l > 0.f || bad || l != l;
  const float inv = any ? 1.f / l : 0.f;
  const size_t row = static_cast<size_t>(q0 + r) * p.heads + h;
  if (p.lse && lane == 0) p.lse[row] = bad ? NAN : any ? m + logf(l) : -INFINITY;
  reinterpret_cast<uint2*>(p.out + row * kNope)[lane] =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

}  // namespace

int launch_prefill(const PrefillParams& p, cudaStream_t stream) {
  if (p.n_items <= 0) return MLA_OK;
  prefill_kernel<<<dim3(p.n_items, p.heads), kThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return MLA_ERR_CUDA;
  if (p.n_merges > 0) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((kPfRows * p.heads + 7) / 8, p.n_merges, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, prefill_merge_kernel, p) != cudaSuccess) return MLA_ERR_CUDA;
    if (cudaPeekAtLastError() != cudaSuccess) return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

}  // namespace mla
