// Rotary positions: the query's 64-wide rotary part, and a row's rotary key
// on its way into the cache together with the RMS norm of its latent.
//
//   turn_i = position * f_i  (turns),  f_i = inv_freq_i / 2 pi
//   (x0, x1) -> a (x0 cos - x1 sin,  x1 cos + x0 sin)
//   latent y = x * rsqrt(mean x^2 + eps) * w
//
// f_i is a 64-bit fraction of a turn, so position * f_i in 64-bit integers drops
// whole turns by wrapping, without an error of its own; as a signed fraction in
// [-1/2, 1/2) it becomes the argument of sincospif, rounded to 24 bits.  All 64
// bits take part: the slowest pairs turn by 1e-9 of a turn a position, and of the
// upper 32 bits alone their sines would keep few digits.  No table is read and no
// position is too large.  Sums and products are fp32, rounded once to the
// output's type.
#include "mla_device.cuh"
#include "mla_launch.h"
#include "mla_prompt.h"

namespace mla {
namespace {

__device__ __forceinline__ float2 phase_cos_sin(uint64_t freq, int position, float amplitude) {
  const uint64_t turn = freq * static_cast<uint64_t>(static_cast<int64_t>(position));
  float s, c;
  sincospif(__ll2float_rn(static_cast<long long>(turn)) * 0x1p-63f, &s, &c);   // wrapped to [-1, 1) half turns
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
// Work is cut into units of one token and up to 32 J heads; a block walks
// units.  Eight lanes move a head's rotary part, 16 bytes each (half layout:
// four lanes, both halves), and a thread has J heads in flight.  The 32 pairs'
// cos and sin are computed once a unit, by warp 0, while the loads are on
// their way; each of its lanes keeps its pair's frequency in a register (read
// from the parameters by lane it is a replay a lane, once a block).
// Bound: HBM (the rotary part read and written once).  8191 tokens x 128 heads
// take 44.0 us (6.1 TB/s, 0.91 of a plain copy's rate); 64 tokens x 128 heads
// with the copy of the rest 2.9 us, which is a launch and a round trip.
constexpr int kQThreads = 256;

template <int J>
__global__ void __launch_bounds__(kQThreads, 4) rope_query_kernel(const RopeQueryParams p,
                                                               const __grid_constant__ RopeFreqs f, int units) {
  __shared__ __align__(16) float2 cs_of[2][kPairs];
  const int tid = threadIdx.x;
  const uint64_t freq = tid < kPairs ? f.f[tid] : 0;
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kHeads = 32 * J;
  const int chunks = (p.heads + kHeads - 1) / kHeads;
  const int pieces = p.nope / 8;
  // the copy of the rest of the heads: a thread's piece, its first head and the heads a pass covers
  const int span = pieces > 0 && pieces <= kQThreads ? kQThreads / pieces : 0;
  const int ch = span ? tid / pieces : 0, cd = span ? (tid - ch * pieces) * 8 : 0;
  int buf = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x, buf ^= 1) {
    const int t = u / chunks, h0 = (u - t * chunks) * kHeads;
    const int nh = min(kHeads, p.heads - h0);
    const uint16_t* src = p.q + t * p.q_ts + h0 * p.q_hs;
    uint16_t* dst = p.q_rope + t * p.r_ts + h0 * p.r_hs;
    const float4* cs = reinterpret_cast<const float4*>(cs_of[buf]);
    if (f.interleaved) {
      const int h = tid >> 3, d = (tid & 7) * 8;
      uint4 v[J];
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (h + 32 * j < nh) v[j] = *reinterpret_cast<const uint4*>(src + (h + 32 * j) * p.q_hs + p.nope + d);
      if (tid < kPairs) cs_of[buf][tid] = phase_cos_sin(freq, __ldg(p.positions + t), f.amplitude);
      __syncthreads();
      const float4 c01 = cs[d / 4], c23 = cs[d / 4 + 1];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (h + 32 * j >= nh) continue;
        uint32_t* w = reinterpret_cast<uint32_t*>(&v[j]);
        auto turn = [&](uint32_t& x, float c, float sn) {
          float a = bf_lo(x), b = bf_hi(x);
          rotate(a, b, make_float2(c, sn));
          x = pack_bf16x2(a, b);
        };
        turn(w[0], c01.x, c01.y);
        turn(w[1], c01.z, c01.w);
        turn(w[2], c23.x, c23.y);
        turn(w[3], c23.z, c23.w);
        *reinterpret_cast<uint4*>(dst + (h + 32 * j) * p.r_hs + d) = v[j];
      }
    } else {
      constexpr int kN = (J + 1) / 2;
      const int h = tid >> 2, d = (tid & 3) * 8;
      uint4 va[kN], vb[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j)
        if (h + 64 * j < nh) {
          const uint16_t* x = src + (h + 64 * j) * p.q_hs + p.nope + d;
          va[j] = *reinterpret_cast<const uint4*>(x);
          vb[j] = *reinterpret_cast<const uint4*>(x + 32);
        }
      if (tid < kPairs) cs_of[buf][tid] = phase_cos_sin(freq, __ldg(p.positions + t), f.amplitude);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        if (h + 64 * j >= nh) continue;
        uint32_t* wa = reinterpret_cast<uint32_t*>(&va[j]);
        uint32_t* wb = reinterpret_cast<uint32_t*>(&vb[j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 c = cs[d / 2 + k];
          float a0 = bf_lo(wa[k]), b0 = bf_lo(wb[k]), a1 = bf_hi(wa[k]), b1 = bf_hi(wb[k]);
          rotate(a0, b0, make_float2(c.x, c.y));
          rotate(a1, b1, make_float2(c.z, c.w));
          wa[k] = pack_bf16x2(a0, a1);
          wb[k] = pack_bf16x2(b0, b1);
        }
        uint16_t* y = dst + (h + 64 * j) * p.r_hs + d;
        *reinterpret_cast<uint4*>(y) = va[j];
        *reinterpret_cast<uint4*>(y + 32) = vb[j];
      }
    }
    if (p.q_nope) {
      uint16_t* out = p.q_nope + (static_cast<long long>(t) * p.heads + h0) * p.nope;
      if (span) {
        if (ch < span) {
#pragma unroll 4
          for (int h = ch; h < nh; h += span)
            *reinterpret_cast<uint4*>(out + static_cast<long long>(h) * p.nope + cd) =
                *reinterpret_cast<const uint4*>(src + h * p.q_hs + cd);
        }
      } else {
        for (int i = tid; i < nh * pieces; i += kQThreads) {
          const int h = i / pieces, d = (i - h * pieces) * 8;
          *reinterpret_cast<uint4*>(out + static_cast<long long>(h) * p.nope + d) =
              *reinterpret_cast<const uint4*>(src + h * p.q_hs + d);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ append --
// One warp a row: a lane holds 16 latent values (two 16-byte pieces) and one
// rotary pair, and over all rows of the warp its pair's frequency and its part
// of the norm's weight (read from the parameters by lane, a frequency is a
// replay a lane: at one row a warp that took as long as the rows).  A slot
// outside [0, num_slots) is skipped and recorded.  Bound: HBM for long prompts,
// else the launch and the dependent trip to the slot and back: 16384 rows take
// 9.0 us (4.2 TB/s), 5000 rows into an E4M3 cache 4.3 us, 4 rows 2.0 us.
constexpr int kAThreads = 256;

constexpr int kABlocks = 3;      // blocks an SM holds: a row being worked on and the next one on its way a warp

// x / scale in fp32; by its reciprocal where that is exact (a power of two).
__device__ __forceinline__ float unscale(float x, const RopeAppendParams& p) {
  return p.kv_recip != 0.f ? x * p.kv_recip : __fdiv_rn(x, p.kv_scale);
}

template <bool kFp8>
__global__ void __launch_bounds__(kAThreads, kABlocks) rope_append_kernel(const RopeAppendParams p,
                                                                          const __grid_constant__ RopeFreqs f,
                                                                          int warps) {
  const int lane = threadIdx.x & 31;
  const int warp = blockIdx.x * (kAThreads / 32) + (threadIdx.x >> 5);
  const uint64_t freq = f.f[lane];
  const int ia = f.interleaved ? 2 * lane : lane, ib = f.interleaved ? 2 * lane + 1 : lane + kPairs;
  griddep_wait();
  griddep_launch_dependents();
  uint4 g0 = make_uint4(0, 0, 0, 0), g1 = g0;
  if (p.weight) {
    g0 = __ldg(reinterpret_cast<const uint4*>(p.weight) + lane);
    g1 = __ldg(reinterpret_cast<const uint4*>(p.weight) + 32 + lane);
  }
  struct Row {
    int slot, pos;
    uint4 v0, v1;
    uint32_t r;                  // the rotary pair
  };
  auto load = [&](int t) {
    Row x;
    const uint16_t* src = p.rows + t * p.row_stride;
    x.slot = __ldg(p.slots + t);
    x.pos = __ldg(p.positions + t);
    x.v0 = __ldg(reinterpret_cast<const uint4*>(src) + lane);
    x.v1 = __ldg(reinterpret_cast<const uint4*>(src) + 32 + lane);
    if (f.interleaved) x.r = __ldg(reinterpret_cast<const uint32_t*>(src + kLatent) + lane);
    else x.r = static_cast<uint32_t>(__ldg(src + kLatent + ia)) | static_cast<uint32_t>(__ldg(src + kLatent + ib)) << 16;
    return x;
  };
  if (warp >= p.tokens) return;
  Row next = load(warp);
  for (int t = warp; t < p.tokens; t += warps) {
    const Row cur = next;
    if (t + warps < p.tokens) next = load(t + warps);
    const long long slot = cur.slot;
    const uint4 v0 = cur.v0, v1 = cur.v1;
    float ra = bf_lo(cur.r), rb = bf_hi(cur.r);
    if (slot < 0 || slot >= p.num_slots) {
      if (lane == 0) record_status(p.status, MLA_ERR_INDEX_OOB);
      continue;
    }
    rotate(ra, rb, phase_cos_sin(freq, cur.pos, f.amplitude));
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
        c[i] = e4m3x2(unscale(x[4 * i], p), unscale(x[4 * i + 1], p)) |
               e4m3x2(unscale(x[4 * i + 2], p), unscale(x[4 * i + 3], p)) << 16;
      reinterpret_cast<uint2*>(dst)[lane] = make_uint2(c[0], c[1]);
      reinterpret_cast<uint2*>(dst)[32 + lane] = make_uint2(c[2], c[3]);
      const uint32_t r2 = e4m3x2(unscale(ra, p), unscale(rb, p));
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

// Heads of a unit: 128 where the units then still reach half of the SMs, else
// 32.  128 heads, us at 128 and 32 a unit: 64 tokens 2.22 and 2.16, 100 tokens
// 2.21 and 2.52, 300 2.67 and 3.31, 2000 13.0 and 18.3.
int launch_rope_query(const RopeQueryParams& p, const RopeFreqs& f, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms < 1) return MLA_ERR_CUDA;
  const bool wide = static_cast<long long>(p.tokens) * ((p.heads + 127) / 128) >= sms / 2 && p.heads > 32;
  const int per = wide ? 128 : 32;
  const long long units = static_cast<long long>(p.tokens) * ((p.heads + per - 1) / per);
  if (units > 0x3FFFFFFFll) return MLA_ERR_UNSUPPORTED;
  const int grid = static_cast<int>(units < 4ll * sms ? units : 4ll * sms);   // what the SMs hold at once
  return wide ? launch_dependent(rope_query_kernel<4>, grid, kQThreads, stream, p, f, static_cast<int>(units))
              : launch_dependent(rope_query_kernel<1>, grid, kQThreads, stream, p, f, static_cast<int>(units));
}

int launch_rope_append(const RopeAppendParams& p, const RopeFreqs& f, bool fp8, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms < 1) return MLA_ERR_CUDA;
  constexpr int kWarps = kAThreads / 32;
  // as many warps as the SMs hold, each the same number of rows
  const long long held = static_cast<long long>(sms) * kABlocks * kWarps;
  const long long rows = (p.tokens + held - 1) / held;
  const int grid = static_cast<int>((p.tokens + rows * kWarps - 1) / (rows * kWarps));
  return fp8 ? launch_dependent(rope_append_kernel<true>, grid, kAThreads, stream, p, f, grid * kWarps)
             : launch_dependent(rope_append_kernel<false>, grid, kAThreads, stream, p, f, grid * kWarps);
}

}  // namespace mla
