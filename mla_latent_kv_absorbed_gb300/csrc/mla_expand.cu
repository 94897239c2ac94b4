// Latent expansion: the cached rows named by kv_indices to every head's keys
// and values,
//   k[t, h, n] = sum_r c_t[r] w_kc[h, n, r],   v[t, h, n] = sum_r c_t[r] w_vc[h, r, n],
// and the rope key that all heads share.  c_t is the 512-wide latent of the
// row (an FP8 row's code values times kv_scale); sums in fp32, one rounding.
#include "mla_device.cuh"
#include "mla_prompt.h"

namespace mla {
namespace {

constexpr int kTok = 16;       // rows of a block

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

__device__ __forceinline__ uint16_t to_bf(float x) { return static_cast<uint16_t>(pack_bf16x2(x, 0.f)); }

// One block: 16 rows, one head; thread n < 128 a key column, else a value column.
template <bool kFp8>
__global__ void __launch_bounds__(256) expand_kernel(const ExpandParams p) {
  __shared__ float c[kLatent][kTok];
  const int t0 = blockIdx.x * kTok, h = blockIdx.y;
  for (int i = threadIdx.x; i < kTok * kRow; i += 256) {
    const int k = i / kRow, d = i - k * kRow, t = t0 + k;
    float x = 0.f;
    if (t < p.tokens) {
      long long slot = __ldg(p.kv_indices + t);
      if (slot < 0 || slot >= p.num_slots) {
        record_status(p.status, MLA_ERR_INDEX_OOB);
        slot = 0;
      }
      if constexpr (kFp8) {
        x = e4m3x2_value(p.kv_cache[slot * kRow + d]).x;
      } else {
        x = bf(reinterpret_cast<const uint16_t*>(p.kv_cache)[slot * kRow + d]);
      }
      if (d >= kLatent && h == 0) p.k_rope[static_cast<size_t>(t) * kRope + d - kLatent] = to_bf(kFp8 ? x * p.kv_scale : x);
    }
    if (d < kLatent) c[d][k] = x;
  }
  __syncthreads();
  const int n = threadIdx.x & 127;
  const bool key = threadIdx.x < 128;
  const uint16_t* w = key ? p.w_kc + (static_cast<size_t>(h) * kNope + n) * kLatent
                          : p.w_vc + static_cast<size_t>(h) * kLatent * kNope + n;
  const int step = key ? 1 : kNope;
  float acc[kTok];
#pragma unroll
  for (int k = 0; k < kTok; ++k) acc[k] = 0.f;
  for (int r = 0; r < kLatent; ++r) {
    const float x = bf(__ldg(w + static_cast<size_t>(r) * step));
#pragma unroll
    for (int k = 0; k < kTok; ++k) acc[k] = fmaf(c[r][k], x, acc[k]);
  }
  uint16_t* out = key ? p.k_nope : p.v;
#pragma unroll
  for (int k = 0; k < kTok; ++k)
    if (t0 + k < p.tokens)
      out[(static_cast<size_t>(t0 + k) * p.heads + h) * kNope + n] = to_bf(kFp8 ? acc[k] * p.kv_scale : acc[k]);
}

}  // namespace

int launch_expand(const ExpandParams& p, bool fp8, cudaStream_t stream) {
  const dim3 grid((p.tokens + kTok - 1) / kTok, p.heads, 1);
  if (fp8) expand_kernel<true><<<grid, 256, 0, stream>>>(p);
  else expand_kernel<false><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace mla
