// Rotary positions: the query's 64-wide rotary part, and a row's rotary key
// on its way into the cache together with the RMS norm of its latent.
//
//   turn_i = position * f_i  (turns),  f_i = inv_freq_i / 2 pi
//   (x0, x1) -> a (x0 cos - x1 sin,  x1 cos + x0 sin)
//   latent y = x * rsqrt(mean x^2 + eps) * w
//
// The angle is exact at any position: f_i is a 64-bit fraction of a turn, so
// position * f_i in 64-bit integers drops whole turns by wrapping and leaves
// the phase to 2^-64 * position turns; its upper 32 bits, as a signed fraction
// in [-1/2, 1/2), become the argument of sincospif (error: 2^-25 of a half
// turn from the conversion to 24 bits).  No table is read and no position is
// too large.  Sums and products are fp32, rounded once to the output's type.
#include "mla_device.cuh"
#include "mla_prompt.h"

namespace mla {
namespace {

__device__ __forceinline__ float2 phase_cos_sin(uint64_t freq, int position, float amplitude) {
  const uint64_t turn = freq * static_cast<uint64_t>(static_cast<int64_t>(position));
  const int hi = static_cast<int>(turn >> 32);              // turns * 2^32, wrapped to [-1/2, 1/2)
  float s, c;
  sincospif(static_cast<float>(hi) * 0x1p-31f, &s, &c);     // 2 * turns half turns
  return make_float2(c * amplitude, s * amplitude);
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void rotate(float& a, float& b, float2 cs) {
  const float x = a, y = b;
  a = x * cs.x - y * cs.y;
  b = y * cs.x + x * cs.y;
}

// ------------------------------------------------------------------- query --
// A block takes one token and `heads_per_block` heads.  Eight lanes move a
// head's rotary part, 16 bytes each; the 32 pairs' cos and sin are computed
// once a block, by warp 0, while the other loads are in flight.
constexpr int kQThreads = 256;

__global__ void __launch_bounds__(kQThreads) rope_query_kernel(const RopeQueryParams p,
                                                               const __grid_constant__ RopeFreqs f,
                                                               int heads_per_block) {
  __shared__ float2 cs[kPairs];
  griddep_wait();
  griddep_launch_dependents();
  const int chunks = (p.heads + heads_per_block - 1) / heads_per_block;
  const int t = blockIdx.x / chunks;
  const int h0 = (blockIdx.x % chunks) * heads_per_block;
  const int nh = min(heads_per_block, p.heads - h0);
  if (threadIdx.x < kPairs)
    cs[threadIdx.x] = phase_cos_sin(f.f[threadIdx.x], __ldg(p.positions + t), f.amplitude);
  __syncthreads();
  const uint16_t* src = p.q + t * p.q_ts + h0 * p.q_hs;
  uint16_t* dst = p.q_rope + t * p.r_ts + h0 * p.r_hs;
  if (f.interleaved) {
    for (int i = threadIdx.x; i < nh * 8; i += kQThreads) {
      const int h = i >> 3, d = (i & 7) * 8;
      uint4 v = *reinterpret_cast<const uint4*>(src + h * p.q_hs + p.nope + d);
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float a = bf_lo(w[k]), b = bf_hi(w[k]);
        rotate(a, b, cs[d / 2 + k]);
        w[k] = pack_bf16x2(a, b);
      }
      *reinterpret_cast<uint4*>(dst + h * p.r_hs + d) = v;
    }
  } else {
    for (int i = threadIdx.x; i < nh * 4; i += kQThreads) {
      const int h = i >> 2, d = (i & 3) * 8;
      const uint16_t* s = src + h * p.q_hs + p.nope + d;
      uint4 va = *reinterpret_cast<const uint4*>(s), vb = *reinterpret_cast<const uint4*>(s + 32);
      uint32_t* wa = reinterpret_cast<uint32_t*>(&va);
      uint32_t* wb = reinterpret_cast<uint32_t*>(&vb);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float a0 = bf_lo(wa[k]), b0 = bf_lo(wb[k]), a1 = bf_hi(wa[k]), b1 = bf_hi(wb[k]);
        rotate(a0, b0, cs[d + 2 * k]);
        rotate(a1, b1, cs[d + 2 * k + 1]);
        wa[k] = pack_bf16x2(a0, a1);
        wb[k] = pack_bf16x2(b0, b1);
      }
      *reinterpret_cast<uint4*>(dst + h * p.r_hs + d) = va;
      *reinterpret_cast<uint4*>(dst + h * p.r_hs + d + 32) = vb;
    }
  }
  if (p.q_nope) {
    const int pieces = p.nope / 8;
    uint16_t* out = p.q_nope + (static_cast<long long>(t) * p.heads + h0) * p.nope;
    for (int i = threadIdx.x; i < nh * pieces; i += kQThreads) {
      const int h = i / pieces, d = (i - h * pieces) * 8;
      *reinterpret_cast<uint4*>(out + static_cast<long long>(h) * p.nope + d) =
          *reinterpret_cast<const uint4*>(src + h * p.q_hs + d);
    }
  }
}

// ------------------------------------------------------------------ append --
// One warp a row: a lane holds 16 latent values (two 16-byte pieces) and one
// rotary pair.  A slot outside [0, num_slots) is skipped and recorded.
constexpr int kAThreads = 256;

template <bool kFp8>
__global__ void __launch_bounds__(kAThreads) rope_append_kernel(const RopeAppendParams p,
                                                                const __grid_constant__ RopeFreqs f) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kAThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.tokens) return;
  const long long slot = __ldg(p.slots + t);
  const int pos = __ldg(p.positions + t);
  const uint16_t* src = p.rows + t * p.row_stride;
  const uint4 v0 = __ldg(reinterpret_cast<const uint4*>(src) + lane);
  const uint4 v1 = __ldg(reinterpret_cast<const uint4*>(src) + 32 + lane);
  const uint16_t* rs = src + kLatent;
  const int ia = f.interleaved ? 2 * lane : lane, ib = f.interleaved ? 2 * lane + 1 : lane + kPairs;
  float ra = __uint_as_float(static_cast<uint32_t>(__ldg(rs + ia)) << 16);
  float rb = __uint_as_float(static_cast<uint32_t>(__ldg(rs + ib)) << 16);
  if (slot < 0 || slot >= p.num_slots) {
    if (lane == 0) record_status(p.status, MLA_ERR_INDEX_OOB);
    return;
  }
  rotate(ra, rb, phase_cos_sin(f.f[lane], pos, f.amplitude));
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf_lo(w[i]);
    x[2 * i + 1] = bf_hi(w[i]);
  }
  if (p.weight) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss * (1.f / kLatent) + p.eps);
    const uint4 g0 = __ldg(reinterpret_cast<const uint4*>(p.weight) + lane);
    const uint4 g1 = __ldg(reinterpret_cast<const uint4*>(p.weight) + 32 + lane);
    const uint32_t g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = x[2 * i] * r * bf_lo(g[i]);
      x[2 * i + 1] = x[2 * i + 1] * r * bf_hi(g[i]);
    }
  }
  if constexpr (kFp8) {
    uint8_t* dst = static_cast<uint8_t*>(p.kv_cache) + slot * kRow;
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = e4m3x2(__fdiv_rn(x[4 * i], p.kv_scale), __fdiv_rn(x[4 * i + 1], p.kv_scale)) |
             e4m3x2(__fdiv_rn(x[4 * i + 2], p.kv_scale), __fdiv_rn(x[4 * i + 3], p.kv_scale)) << 16;
    reinterpret_cast<uint2*>(dst)[lane] = make_uint2(c[0], c[1]);
    reinterpret_cast<uint2*>(dst)[32 + lane] = make_uint2(c[2], c[3]);
    const uint32_t r2 = e4m3x2(__fdiv_rn(ra, p.kv_scale), __fdiv_rn(rb, p.kv_scale));
    dst[kLatent + ia] = static_cast<uint8_t>(r2);
    dst[kLatent + ib] = static_cast<uint8_t>(r2 >> 8);
  } else {
    uint16_t* dst = static_cast<uint16_t*>(p.kv_cache) + slot * kRow;
    uint4 o0 = v0, o1 = v1;                       // without a norm the latent's bits pass unchanged
    if (p.weight) {
      o0 = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
      o1 = make_uint4(pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]), pack_bf16x2(x[12], x[13]),
                      pack_bf16x2(x[14], x[15]));
    }
    reinterpret_cast<uint4*>(dst)[lane] = o0;
    reinterpret_cast<uint4*>(dst)[32 + lane] = o1;
    const uint32_t r2 = pack_bf16x2(ra, rb);
    if (f.interleaved) {
      reinterpret_cast<uint32_t*>(dst + kLatent)[lane] = r2;
    } else {
      dst[kLatent + ia] = static_cast<uint16_t>(r2);
      dst[kLatent + ib] = static_cast<uint16_t>(r2 >> 16);
    }
  }
}

template <typename Kernel, typename... Args>
int launch_dependent(Kernel* kernel, int blocks, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return MLA_ERR_CUDA;
  return cudaPeekAtLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace

int launch_rope_query(const RopeQueryParams& p, const RopeFreqs& f, cudaStream_t stream) {
  const int per_block = 32;
  const long long blocks = static_cast<long long>(p.tokens) * ((p.heads + per_block - 1) / per_block);
  if (blocks > 0x7FFFFFFFll) return MLA_ERR_UNSUPPORTED;
  return launch_dependent(rope_query_kernel, static_cast<int>(blocks), kQThreads, stream, p, f, per_block);
}

int launch_rope_append(const RopeAppendParams& p, const RopeFreqs& f, bool fp8, cudaStream_t stream) {
  constexpr int kRows = kAThreads / 32;
  const int blocks = static_cast<int>((p.tokens + static_cast<long long>(kRows) - 1) / kRows);
  return fp8 ? launch_dependent(rope_append_kernel<true>, blocks, kAThreads, stream, p, f)
             : launch_dependent(rope_append_kernel<false>, blocks, kAThreads, stream, p, f);
}

}  // namespace mla
