// Verification of drafted tokens against the target's probabilities, from
// given random numbers ("[sglang] EAGLE 트리 검증 어텐션 최적화", section
// "들어가며": the drafts of a tree are verified in one pass of the target).
//
//   node = draft 0;  for the node's children c in their order:
//     accepted  iff  u_c a_c < t_node(x_c);  then node = c and the walk goes on
//     a_c = q_c(x_c) for drafts sampled from q, or what the rejected siblings
//     left of the node's mass, 1 - sum t_node(x), for chosen drafts
//   what is left:  r_v = max(t_v - q_v, 0)  |  t_v off the rejected siblings
//   next token  =  the lowest v with  sum_{w <= v} r_w > u_0 sum_w r_w
//
// (The first form keeps the target's distribution for sampled drafts: the token
// comes with q(x) min(1, t/q) + the rejected rest spread as max(t - q, 0); the
// second walks the inverse of the node's distribution child by child.)
//
// A pick near a border of the running sum is decided by the sum's last bits,
// so sums are held to about 47 bits, as pairs of fp32 numbers: t - q with its
// exact error (t > q >= 0: t - d and the rest are exact), added to a pair with
// the addition's exact error (the published error-free transformations: Knuth's
// sum of two numbers, Dekker's of a larger and a smaller one, a product's error by
// a fused multiply-add).  Two elements go through eleven packed instructions, beside
// the clamping and the minimum.  64-bit arithmetic, at one two-hundredth of fp32's rate, would take longer than the
// element's eight bytes from memory; even for the few sums of sums it took a
// quarter of the kernel's time.  The tests u a < t are those of 64 bits (a product
// of two fp32 numbers is exact in them): in fp32 where the two sides are further
// apart than its roundings, and in 64 bits where they are not.
//
// One cluster of CTAs a request, each a stretch of the row: every CTA walks the
// drafts itself (one warp, a few hundred bytes, the same answer), sums its
// stretch, and hands the sum to all others through distributed shared memory;
// the one whose stretch holds the pick finds the warp's part of it, which the
// CTA's warps sum again in eighths, and one warp scans the right eighth.  The
// second and third reads are of kilobytes that lie in L1 or L2.
#include "mla_device.cuh"
#include "mla_launch.h"
#include "mla_serving.h"

namespace mla {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = kWarps;

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster_f2(uint32_t addr, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}

// A number as the sum x + y of two, |y| at most half a step of x.
using Pair = float2;
__device__ __forceinline__ Pair pair_of(float big, float small) {   // |big| >= |small|, or big = 0
  const float s = __fadd_rn(big, small);
  return make_float2(s, __fsub_rn(small, __fsub_rn(s, big)));
}
// a + b and what rounding left of it
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
  return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z)));
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.x, b.x);
  return pair_of(s.x, __fadd_rn(s.y, __fadd_rn(a.y, b.y)));
}
__device__ __forceinline__ Pair minus(Pair a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ Pair times(Pair a, float b) {
  const float p = __fmul_rn(a.x, b);
  return pair_of(p, __fmaf_rn(a.y, b, __fmaf_rn(a.x, b, -p)));
}
__device__ __forceinline__ bool above(Pair a, Pair b) { return a.x > b.x || (a.x == b.x && a.y > b.y); }
__device__ __forceinline__ Pair shfl_xor(Pair a, int o) {
  return make_float2(__shfl_xor_sync(0xffffffffu, a.x, o), __shfl_xor_sync(0xffffffffu, a.y, o));
}

// A probability: NaN and negative values count as 0, values past 1 as 1.
__device__ __forceinline__ float prob(float x) { return __saturatef(x); }

// What a request's drafts left: the row that the next token is drawn from.
struct Walk {
  int node;                   // the last accepted draft
  int below;                  // the rejected draft whose q is taken off, or -1
  int excluded;               // tokens whose mass is taken out
};

// max(t - q, 0), exactly (0 where q >= t).
__device__ __forceinline__ Pair rest(float t, float q) {
  const float less = fminf(q, t), d = __fsub_rn(t, less);
  return make_float2(d, __fsub_rn(__fsub_rn(t, d), less));
}

// One warp: lane i has drafts i and 32 + i.
__device__ __forceinline__ Walk walk_drafts(const VerifyParams& p, int b, int lane, bool write, int32_t* gone) {
  const int W = p.width;
  int par[2], tok[2];
  float t[2], q[2], u[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    par[k] = -2;
    tok[k] = -1;
    t[k] = q[k] = u[k] = 0.f;
    if (i >= W) continue;
    const long long at = static_cast<long long>(b) * W + i;
    int up = p.parents ? __ldg(p.parents + at) : i - 1;
    tok[k] = __ldg(p.tokens + at);
    u[k] = __ldg(p.uniforms + at);
    if (up < -1 || up >= i) {
      if (write) record_status(p.status, MLA_ERR_TREE);
      up = -1;
    }
    par[k] = i == 0 ? -2 : up;                     // a second child of the context is nobody's child here
    if (i > 0 && (tok[k] < 0 || tok[k] >= p.vocab)) {
      if (write) record_status(p.status, MLA_ERR_INDEX_OOB);
      tok[k] = -1;
    }
    if (par[k] >= 0 && tok[k] >= 0) {
      t[k] = prob(__ldg(p.target + b * p.t_bs + par[k] * p.t_rs + tok[k]));
      if (p.draft) q[k] = prob(__ldg(p.draft + b * p.d_bs + i * p.d_rs + tok[k]));
    }
  }
  auto both = [&](bool lo, bool hi) {
    return static_cast<unsigned long long>(__ballot_sync(0xffffffffu, lo)) |
           static_cast<unsigned long long>(__ballot_sync(0xffffffffu, hi)) << 32;
  };
  auto of = [&](const auto (&v)[2], int c) {
    const auto lo = __shfl_sync(0xffffffffu, v[0], c & 31), hi = __shfl_sync(0xffffffffu, v[1], c & 31);
    return c < 32 ? lo : hi;
  };
  int path[2] = {lane == 0 ? 0 : -1, -1};
  int node = 0, count = 1;
  unsigned long long rejected = 0;
  // a draft's test against the share `left` of its node's mass, or its own probability
  constexpr float kNear = 0x1p-20f;                // of `mass`: fp32 has the product, and a pair above 2^-20 its x, to 2^-22
  auto close = [&](float u, float against, float mass) {
    const float p = __fmul_rn(u, against), slack = kNear * mass;
    return mass > 0.f && (mass < 0x1p-100f || !(p < mass - slack || p > mass + slack));
  };
  auto less = [&](float u, double against, float mass) { return static_cast<double>(u) * against < static_cast<double>(mass); };
#pragma unroll
  for (int k = 0; k < 2; ++k) u[k] = fmaxf(u[k], 0.f);     // (NaN too)
  if (!p.parents) {
    // a chain: every draft at once; those before the first that fails are accepted
    bool a[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float against = p.draft ? q[k] : 1.f;
      a[k] = close(u[k], against, t[k]) ? less(u[k], static_cast<double>(against), t[k]) : __fmul_rn(u[k], against) < t[k];
    }
    const unsigned long long fail = ~(both(a[0], a[1]) | 1ull);
    count = fail ? min(__ffsll(static_cast<long long>(fail)) - 1, W) : W;
    node = count - 1;
    if (count < W) rejected = 1ull << count;
#pragma unroll
    for (int k = 0; k < 2; ++k) path[k] = lane + 32 * k < count ? lane + 32 * k : -1;
  } else {
    float counted[2] = {0.f, 0.f};                 // the mass that a rejected draft took (a repeated token's: none)
    for (bool moved = true; moved;) {              // at most W - 1 children are tried in all
      unsigned long long kids = both(par[0] == node, par[1] == node);
      rejected = 0;
      Pair left = make_float2(1.f, 0.f);
      moved = false;
      while (kids) {
        const int c = __ffsll(static_cast<long long>(kids)) - 1;
        kids &= kids - 1;
        const int x = of(tok, c);
        const bool again = both((rejected >> lane & 1) && tok[0] == x, (rejected >> (32 + lane) & 1) && tok[1] == x) != 0;
        const float mass = again ? 0.f : of(t, c), uc = of(u, c);
        bool taken = __fmul_rn(uc, left.x) < mass;
        if (close(uc, left.x, mass) || left.x < 0x1p-20f) {   // (seldom) what the rejected siblings left, in 64 bits
          double share = 1.0;
          for (unsigned long long r = rejected; r; r &= r - 1)
            share = fmax(share - static_cast<double>(of(counted, __ffsll(static_cast<long long>(r)) - 1)), 0.0);
          taken = less(uc, share, mass);
        }
        if (taken) {
          node = c;
          path[0] = lane == count ? c : path[0];
          path[1] = lane + 32 == count ? c : path[1];
          ++count;
          moved = true;
          break;
        }
        rejected |= 1ull << c;
        counted[0] = lane == c ? mass : counted[0];
        counted[1] = lane + 32 == c ? mass : counted[1];
        left = add(left, make_float2(-mass, 0.f));
        if (!(left.x > 0.f)) left = make_float2(0.f, 0.f);
      }
    }
  }
  if (write) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (lane + 32 * k < W) p.path[static_cast<long long>(b) * W + lane + 32 * k] = path[k];
    if (lane == 0) p.accepted[b] = count;
  }
  Walk w{node, -1, 0};
  if (p.draft) {
    if (rejected) w.below = __ffsll(static_cast<long long>(rejected)) - 1;
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bool mine = (rejected >> (lane + 32 * k) & 1) && tok[k] >= 0;
      const uint32_t m = __ballot_sync(0xffffffffu, mine);
      if (mine) gone[w.excluded + __popc(m & ((1u << lane) - 1))] = tok[k];
      w.excluded += __popc(m);
    }
  }
  return w;
}

// Sums of up to eight parts, a part a lane, and the sums of those up to it.  By a whole warp.
struct Parts {
  Pair sum, upto;
};
__device__ __forceinline__ Pair shfl(Pair a, int lane) {
  return make_float2(__shfl_sync(0xffffffffu, a.x, lane), __shfl_sync(0xffffffffu, a.y, lane));
}
__device__ __forceinline__ Pair shfl_up(Pair a, int o) {
  return make_float2(__shfl_up_sync(0xffffffffu, a.x, o), __shfl_up_sync(0xffffffffu, a.y, o));
}
__device__ __forceinline__ Parts parts_of(const Pair* sum, int n, int lane) {
  Parts p;
  p.sum = lane < n ? sum[lane] : make_float2(0.f, 0.f);
  p.upto = p.sum;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const Pair x = shfl_up(p.upto, o);
    if (lane >= o) p.upto = add(p.upto, x);
  }
  return p;
}
// Which part the running sum passes `thr` in (the last with any mass where
// rounding or a number of 1 leaves it short; 0 without mass), and the sum before
// it.
__device__ __forceinline__ int pick(const Parts& p, Pair thr, Pair& before) {
  const uint32_t some = __ballot_sync(0xffffffffu, p.sum.x > 0.f);
  const uint32_t past = __ballot_sync(0xffffffffu, p.sum.x > 0.f && above(p.upto, thr));
  const int at = past ? __ffs(past) - 1 : some ? 31 - __clz(some) : 0;
  before = shfl(p.upto, max(at - 1, 0));
  if (at == 0) before = make_float2(0.f, 0.f);
  return at;
}

// (Four blocks an SM: 64 requests of eight CTAs are resident at once.  With 77 registers they are not, and the batch
// of 64 x 8 x 129280 takes 4 us more.)
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const VerifyParams p) {
  __shared__ Pair cta_sum[kMaxCluster], warp_sum[kWarps], part_sum[kWarps];
  __shared__ int32_t gone[kMaxDrafts];
  __shared__ Walk walk;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_ctarank());
  const int b = blockIdx.x / C;
  griddep_wait();
  griddep_launch_dependents();
  cluster_arrive();                                // (the other CTAs run: their shared memory may be written)
  if (warp == 0) {
    const Walk w = walk_drafts(p, b, lane, rank == 0, gone);
    if (lane == 0) walk = w;
  }
  __syncthreads();
  const float* P = p.target + b * p.t_bs + walk.node * p.t_rs;
  const float* Q = walk.below >= 0 ? p.draft + b * p.d_bs + walk.below * p.d_rs : nullptr;
  const int n_gone = walk.excluded;
  // the row in blocks of four elements that lie on 16 bytes: element v is in block (v + lead) / 4
  const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(P) >> 2 & 3);
  const bool q_wide = Q && (reinterpret_cast<uintptr_t>(Q) >> 2 & 3) == static_cast<uintptr_t>(lead);
  const int V = p.vocab;
  const int blocks = static_cast<int>((static_cast<long long>(V) + lead + 3) / 4);
  const int per = (blocks + C * kWarps - 1) / (C * kWarps);
  auto first = [&](int part) { return static_cast<int>(min(static_cast<long long>(part) * per, static_cast<long long>(blocks))); };

  // the four t and q of block k; elements outside the row and taken-out tokens are 0
  auto load = [&](int k, float (&t)[4], float (&q)[4]) {
    const int v0 = 4 * k - lead;
    const bool whole = v0 >= 0 && v0 + 4 <= V;
    if (whole) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(P + v0));
      t[0] = x.x, t[1] = x.y, t[2] = x.z, t[3] = x.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = v0 + i >= 0 && v0 + i < V ? __ldg(P + v0 + i) : 0.f;
    }
    if (q_wide && whole) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(Q + v0));
      q[0] = x.x, q[1] = x.y, q[2] = x.z, q[3] = x.w;
    } else if (Q) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = v0 + i >= 0 && v0 + i < V ? __ldg(Q + v0 + i) : 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = 0.f;
    }
  };
  auto clean = [&](int k, float (&t)[4], float (&q)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[i] = prob(t[i]);
      q[i] = prob(q[i]);
    }
    for (int g = 0; g < n_gone; ++g) {
      const int at = gone[g] + lead - 4 * k;
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = at == i ? 0.f : t[i];
    }
  };
  // Sum of max(t - q, 0) over blocks [k0, k1), by a warp; in every lane.  The even and the odd elements have a running
  // sum each, and go through packed instructions together.  (Four blocks a lane on their way: 15.8 us of the batch
  // of 64 x 8 x 129280; two 17.9, three 16.4, six 21.8, and two while two are added up 15.9, all before the parts'
  // sums were scanned by lanes; with that, and the drafts' tests as in 64 bits, 15.2.)
  auto sum_of = [&](int k0, int k1) -> Pair {
    constexpr int kDeep = 4;
    const float2 minus1 = make_float2(-1.f, -1.f);
    float2 s = make_float2(0.f, 0.f), e = s;
    for (int k = k0 + lane; k < k1; k += 32 * kDeep) {
      float t[kDeep][4], q[kDeep][4];
#pragma unroll
      for (int j = 0; j < kDeep; ++j)
        if (k + 32 * j < k1) load(k + 32 * j, t[j], q[j]);
#pragma unroll
      for (int j = 0; j < kDeep; ++j) {
        if (k + 32 * j >= k1) continue;
        clean(k + 32 * j, t[j], q[j]);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float2 x = make_float2(t[j][i], t[j][i + 1]);
          const float2 y = make_float2(fminf(q[j][i], x.x), fminf(q[j][i + 1], x.y));
          const float2 d = f2_fma(y, minus1, x), low = f2_fma(y, minus1, f2_fma(d, minus1, x));   // x - y, exactly
          const float2 n = f2_add(s, d), z = f2_fma(s, minus1, n);                                // s + d and its error
          const float2 off = f2_add(f2_fma(f2_fma(z, minus1, n), minus1, s), f2_fma(z, minus1, d));
          s = n;
          e = f2_add(e, f2_add(off, low));
        }
      }
    }
    Pair all = add(pair_of(s.x, e.x), pair_of(s.y, e.y));
#pragma unroll
    for (int o = 16; o; o >>= 1) all = add(all, shfl_xor(all, o));
    return all;
  };

  const int mine = rank * kWarps + warp;
  const Pair part = sum_of(first(mine), first(mine + 1));
  if (lane == 0) warp_sum[warp] = part;
  __syncwarp();
  cluster_wait();
  __syncthreads();
  if (warp == 0) {
    Pair all = lane < kWarps ? warp_sum[lane] : make_float2(0.f, 0.f);
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) all = add(all, shfl_xor(all, o));
    if (lane < C) st_cluster_f2(mapa_shared(smem_u32(cta_sum + rank), lane), all);   // (C <= kWarps: they have it)
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  const Parts ctas = parts_of(cta_sum, C, lane);
  const Pair total = shfl(ctas.upto, C - 1);
  if (!(total.x > 0.f)) {
    if (rank == 0 && tid == 0) p.next[b] = -1;
    return;
  }
  const float u0 = __ldg(p.uniforms + static_cast<long long>(b) * p.width);
  Pair thr = times(total, u0);
  if (!(u0 < 1.f)) thr.x = __int_as_float(0x7FFFFFFF);   // (NaN: nothing is past it, whatever the parts' roundings)
  Pair before;
  if (pick(ctas, thr, before) != rank) return;
  thr = add(thr, minus(before));
  const int w = pick(parts_of(warp_sum, kWarps, lane), thr, before);
  thr = add(thr, minus(before));
  // the warp's part in eighths
  const int k0 = first(rank * kWarps + w), k1 = first(rank * kWarps + w + 1);
  const int eighth = (k1 - k0 + kWarps - 1) / kWarps;
  const int e0 = min(k0 + warp * eighth, k1), e1 = min(e0 + eighth, k1);
  const Pair sub = sum_of(e0, e1);
  if (lane == 0) part_sum[warp] = sub;
  __syncthreads();
  if (pick(parts_of(part_sum, kWarps, lane), thr, before) != warp) return;
  thr = add(thr, minus(before));
  // 32 blocks at a time, a block a lane
  Pair run = make_float2(0.f, 0.f);
  int last = -1;
  for (int k = e0; k < e1; k += 32) {
    float t[4], q[4];
    Pair r[4], s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = s;
    if (k + lane < e1) {
      load(k + lane, t, q);
      clean(k + lane, t, q);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[i] = rest(t[i], q[i]);
        s = add(s, r[i]);
      }
    }
    Pair upto = s, less = make_float2(0.f, 0.f);   // with, and without this lane's own
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Pair x = shfl_up(upto, o);
      if (lane >= o) upto = add(upto, x);
    }
    less = shfl_up(upto, 1);
    if (lane == 0) less = make_float2(0.f, 0.f);
    const uint32_t some = __ballot_sync(0xffffffffu, s.x > 0.f);
    const uint32_t past = __ballot_sync(0xffffffffu, s.x > 0.f && above(add(run, upto), thr));
    // the first lane past the number, or, to fall back on, the last one with mass
    const int who = past ? __ffs(past) - 1 : some ? 31 - __clz(some) : -1;
    int v = -1;
    if (who == lane) {
      Pair x = add(run, less);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool over = v >= 0 && past && above(x, thr);   // passed at an earlier element
        x = add(x, r[i]);
        if (!over && r[i].x > 0.f) v = 4 * (k + lane) - lead + i;
      }
    }
    if (who >= 0) last = __shfl_sync(0xffffffffu, v, who);
    if (past) break;
    run = add(run, shfl(upto, 31));
  }
  if (lane == 0) p.next[b] = last;
}

}  // namespace

// CTAs a request: as many as give the SMs work, up to the cluster's limit, and
// each warp of them at least a block a lane.
int launch_verify(const VerifyParams& p, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms < 1) return MLA_ERR_CUDA;
  int ctas = 1;
  while (ctas < kMaxCluster && static_cast<long long>(p.batch) * ctas < 8ll * sms && p.vocab / (2 * ctas * kWarps) >= 128) ctas *= 2;
  const long long grid = static_cast<long long>(p.batch) * ctas;
  if (grid > 0x7FFFFFFFll) return MLA_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, verify_kernel, p) != cudaSuccess) return MLA_ERR_CUDA;
  return cudaPeekAtLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace mla
