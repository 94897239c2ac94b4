// Attention of ragged sequences over expanded keys and values:
//   s_ij = sm_scale (q_i . [k_nope_j, k_rope_j]),  out_i = softmax_j(s_ij) v_j,
//   lse_i = ln sum_j exp(s_ij),
// j up to the causal limit of row i (the sequences' ends aligned), in one pass
// over the keys with the running maximum and sum.
//
// One CTA takes one item (up to 256 query rows, their keys) for one head: two
// row tiles A and B of 128, each with its scores and its output in TMEM (4 x
// 128 columns: all of it), so that one tile's softmax runs while the tensor
// core works for the other.  Key tiles of 128:
//   S = Q K^T       M = 128, N = 128, 12 steps of K = 16 (128 + 64 dims), both
//                   operands from shared memory
//   P = exp2(..)    in registers, one row a thread; written back as bf16 over
//                   the scores' own columns
//   O += P V        A from TMEM, V as it lies in memory (N-major), 8 steps
// Bound: the tensor core.  A key tile against both row tiles is 2 x 20 MMAs of
// ~64.4 cycles.  The running maximum is a reference that moves only when a
// tile's maximum exceeds it by 2^8: weights stay below 2^8 (bf16 keeps their 8
// bits at any magnitude, sums are fp32), and O is rescaled in TMEM only then.
//
// Warps: 0-3 softmax and epilogue of tile A, 4-7 of tile B, 8 TMA producer, 9
// MMA issuer, 10-11 the guard.  A tile that some row sees only in part is
// masked by index in the softmax, but a zero weight times a value that is not
// finite is NaN in the matrix product: the guard clears those values (and the
// rows behind the last key) in shared memory before the product reads them,
// notes the keys, and the epilogue adds them to the rows that do see them.
#include "mla_device.cuh"
#include "mla_launch.h"
#include "mla_prompt.h"

namespace mla {
namespace {

constexpr int kThreads = 384;
constexpr int kProducer = 8, kIssuer = 9, kGuard = 10;
constexpr int kSlots = 8;                             // of 16 KB: 5 a tile in turn, 3 of keys, 2 of values
constexpr int kBlock = 16384;
constexpr int kOffQ = 0;                              // 2 row tiles x 3 blocks of 128 rows x 64 dims
// The ring, in the order of use: keys of tile t as blocks 5t .. 5t+2 (128 keys
// x 64 dims), its values as 5t+3, 5t+4 (64 keys x 128 dims, two 64-dim chunks).
constexpr int kOffRing = 6 * kBlock;
constexpr int kOffBar = kOffRing + kSlots * kBlock;
enum Bar : int {
  bQFull = 0,                    // [2]
  bKFull = bQFull + 2,           // [2] key tile t on t & 1
  bVFull = bKFull + 2,           // [2] its values (tiles that every row sees whole)
  bKFree = bVFull + 2,           // [2] key tile t on t & 1: its QK products are done
  bVFree = bKFree + 2,           // [2]
  bSFull = bVFree + 2,           // [2] per row tile
  bPFull = bSFull + 2,           // [2]
  bPvDone = bPFull + 2,          // [2]
  bVMasked = bPvDone + 2,        // [3] the values of the item's masked tiles have landed
  bVClean = bVMasked + 3,        // [3] and the guard has been over them
  bDrain = bVClean + 3,
  kBars
};
constexpr int kOffMisc = kOffBar + 8 * kBars;         // TMEM address, abort flag, then the guard's key masks
constexpr int kOffBad = kOffMisc + 16;                // [3][4] words: bit j = key j of the masked tile
constexpr int kSmemBytes = kOffBad + 48 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr uint32_t kTmemS = 0, kTmemO = 256;          // S_A, S_B, O_A, O_B: 128 columns each
constexpr float kSlack = 8.f;                         // log2 growth of the maximum that moves the reference

struct Item {
  int q0, nq, k0, nk, off, part;
};

// The item's words, or false (and MLA_ERR_PLAN_MISMATCH) when it does not lie
// inside the arrays of this launch or has keys past its last row's limit.
__device__ __forceinline__ bool load_item(const PrefillParams& p, int i, Item& it) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(p.items) + 2 * i);
  const int4 b = __ldg(reinterpret_cast<const int4*>(p.items) + 2 * i + 1);
  it = Item{a.y, a.z, a.w, b.x, b.y, b.z};
  return it.q0 >= 0 && it.nq >= 1 && it.nq <= kPfRows && it.q0 <= p.q_tokens - it.nq && it.k0 >= 0 && it.nk >= 0 &&
         it.k0 <= p.kv_tokens - it.nk && it.part >= -1 && it.part < p.partials && it.off >= -kPfNoLimit &&
         it.off <= kPfNoLimit && (it.nk == 0 || it.nk <= it.off + it.nq);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// 32 lanes x 32 consecutive columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ bool not_finite(uint32_t bf16_bits) { return (bf16_bits & 0x7F80u) == 0x7F80u; }

// The warp waits through its first lane; every lane returns the outcome.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtx& wc, int lane) {
  bool ok = true;
  if (lane == 0) ok = mbar_wait(bar, parity, wc);
  return __shfl_sync(0xffffffffu, ok, 0);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// After a wait has given up: the same bounded wait, blind to the abort flag,
// for copies and products that are still in flight.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > MLA_WAIT_LIMIT_NS) return;
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_kr, const __grid_constant__ CUtensorMap tm_v,
                   const PrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return base + kOffBar + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  uint32_t* bad = reinterpret_cast<uint32_t*>(smem + kOffBad);
  const WaitCtx wc{abort_flag, p.status};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(bar(i), i >= bPFull && i < bPFull + 2 ? 4 : i >= bVClean && i < bVClean + 3 ? 2 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < 12) bad[threadIdx.x] = 0;
  if (warp == kIssuer) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == kProducer && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_kr);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  // blocks are numbered group of heads by group, items (heaviest first) within it, heads innermost
  int h, item;
  {
    const int per_group = p.n_items * p.head_group;
    const int g = blockIdx.x / per_group, rest = blockIdx.x - g * per_group;
    const int in_group = min(p.head_group, p.heads - g * p.head_group);
    item = rest / in_group;
    h = g * p.head_group + rest - item * in_group;
  }
  Item it;
  bool good = load_item(p, item, it);
  if (!good) {
    if (threadIdx.x == 0) record_status(p.status, MLA_ERR_PLAN_MISMATCH);
    it.nk = it.nq = 0;
  }
  // key tiles of each row tile, and the first that some row sees only in part
  auto tiles_of = [&](int w) -> int {
    if (it.nq <= 128 * w) return 0;
    const int last = min(it.nk, it.off + min(it.nq, 128 * w + 128));    // keys that the tile's last row sees
    return last > 0 ? (last + kPfKeys - 1) / kPfKeys : 0;
  };
  const int n_a = tiles_of(0), n_b = tiles_of(1);
  const int n = max(n_a, n_b);
  const int whole = min(max(it.off + 1, 0), it.nk) / kPfKeys;           // tiles that every row sees whole
  // (whole <= n, and at most three tiles follow: nk <= off + 256)

  if (warp == kProducer) {
    // ------------------------------------------------------------- producer
    if (lane == 0 && n > 0) {
      auto load_q = [&](int w) {
        mbar_arrive_expect_tx(bar(bQFull + w), 3 * kBlock);
        for (int i = 0; i < 3; ++i)
          tma_load_3d(base + kOffQ + (3 * w + i) * kBlock, &tm_q, 64 * i, h, it.q0 + 128 * w, bar(bQFull + w));
      };
      bool ok = true;
      int k_armed = 0, v_armed = 0;                           // tiles on their way or landed
      // the place of block c, once the block before in it (c - 8) has been used
      auto place = [&](int c) -> uint32_t {
        if (c >= kSlots) {
          const int u = (c - kSlots) / 5;
          const int b = (c - kSlots) % 5 < 3 ? bKFree : bVFree;
          ok = mbar_wait(bar(b + (u & 1)), (u >> 1) & 1, wc);
        }
        return base + kOffRing + (c % kSlots) * kBlock;
      };
      auto load_k = [&](int t) {
        for (int i = 0; i < 3 && ok; ++i) {
          const uint32_t dst = place(5 * t + i), b = bar(bKFull + (t & 1));
          if (!ok) break;
          if (i == 0) mbar_arrive_expect_tx(b, 3 * kBlock);
          k_armed = t + 1;
          if (i < 2) tma_load_3d(dst, &tm_k, 64 * i, h, it.k0 + t * kPfKeys, b);
          else tma_load_2d(dst, &tm_kr, 0, it.k0 + t * kPfKeys, b);
        }
      };
      auto load_v = [&](int t) {
        for (int i = 0; i < 2 && ok; ++i) {
          const uint32_t dst = place(5 * t + 3 + i);
          if (!ok) break;
          const uint32_t b = t < whole ? bar(bVFull + (t & 1)) : bar(bVMasked + t - whole);
          v_armed = t + 1;
          if (i == 0) mbar_arrive_expect_tx(b, 2 * kBlock);
          for (int k = 0; k < 2; ++k)
            tma_load_3d(dst + k * (kBlock / 2), &tm_v, 64 * k, h, it.k0 + t * kPfKeys + 64 * i, b);
        }
      };
      if (n_a > 0) load_q(0);
      load_k(0);
      if (n_b > 0) load_q(1);
      for (int t = 0; t < n && ok; ++t) {
        load_v(t);
        if (ok && t + 1 < n) load_k(t + 1);
      }
      if (!ok) {                                              // no copy outlives the block
        if (n_a > 0) drain_wait(bar(bQFull), 0);
        if (n_b > 0) drain_wait(bar(bQFull + 1), 0);
        for (int t = max(0, k_armed - 2); t < k_armed; ++t) drain_wait(bar(bKFull + (t & 1)), (t >> 1) & 1);
        for (int t = max(0, v_armed - 2); t < v_armed; ++t)
          drain_wait(t < whole ? bar(bVFull + (t & 1)) : bar(bVMasked + t - whole), t < whole ? (t >> 1) & 1 : 0);
      }
    }
    __syncwarp();
  } else if (warp == kIssuer) {
    // ----------------------------------------------------------- MMA issuer
    // The whole warp runs the loop and one elected lane issues: loop counters
    // and descriptors are then uniform to the compiler, which keeps them in
    // uniform registers.
    if (n > 0) {
      const bool lead = elect_one();
      const uint32_t idesc_s = idesc_bf16(128, 128, false, false) | (p.negate ? 1u << 13 : 0u);   // -Q
      constexpr uint32_t kIdescO = idesc_bf16(128, 128, false, true);
      auto D = [](uint64_t d, uint32_t off) -> uint64_t { return d + (off >> 4); };
      bool ok = true;
      auto block_at = [&](int c) -> uint32_t { return base + kOffRing + (c % kSlots) * kBlock; };
      // scores of key tile t for row tile w
      auto qk = [&](int t, int w) {
        const uint32_t d = tmem + kTmemS + 128 * w;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const uint64_t da = sdesc(base + kOffQ + (3 * w + i) * kBlock, 16, 1024);
          const uint64_t db = sdesc(block_at(5 * t + i), 16, 1024);
          if (lead) {
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_ss(d, D(da, 32 * k), D(db, 32 * k), idesc_s, (i | k) != 0 ? 1u : 0u);
          }
        }
        if (lead) umma_commit(bar(bSFull + w));
      };
      auto pv = [&](int t, int w) {
        const uint32_t a = tmem + kTmemS + 128 * w, d = tmem + kTmemO + 128 * w;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t db = sdesc(block_at(5 * t + 3 + i), kBlock / 2, 1024);
          if (lead) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_ts(d, a + 32 * i + 8 * k, D(db, 2048 * k), kIdescO, t > 0 || (i | k) != 0 ? 1u : 0u);
          }
        }
        if (lead) umma_commit(bar(bPvDone + w));
      };
      // a tile's keys and values are waited for once, before row tile A's products (B's when A has none left)
      auto wait_k = [&](int t) { return mbar_wait(bar(bKFull + (t & 1)), (t >> 1) & 1, wc); };
      auto wait_v = [&](int t) {
        if (t < whole) return mbar_wait(bar(bVFull + (t & 1)), (t >> 1) & 1, wc);
        return mbar_wait(bar(bVMasked + t - whole), 0, wc) && mbar_wait(bar(bVClean + t - whole), 0, wc);
      };
      ok = (n_a == 0 || mbar_wait(bar(bQFull), 0, wc)) && wait_k(0);
      tc_fence_after();
      if (ok && n_a > 0) qk(0, 0);
      if (ok && n_b > 0) {
        ok = mbar_wait(bar(bQFull + 1), 0, wc);
        tc_fence_after();
        if (ok) qk(0, 1);
      }
      if (ok && lead) umma_commit(bar(bKFree));
      for (int t = 0; t < n && ok; ++t) {
        bool have_v = false, have_k = false;
        for (int w = 0; w < 2 && ok; ++w) {
          const int nw = w ? n_b : n_a;
          if (t >= nw) continue;
          if (!have_v) ok = wait_v(t);
          have_v = true;
          ok = ok && mbar_wait(bar(bPFull + w), t & 1, wc);
          if (!ok) break;
          tc_fence_after();
          pv(t, w);
          if (t + 1 >= nw) continue;
          if (!have_k) ok = wait_k(t + 1);
          have_k = true;
          tc_fence_after();
          if (ok) qk(t + 1, w);
        }
        if (ok && lead) {
          umma_commit(bar(bVFree + (t & 1)));
          if (t + 1 < n) umma_commit(bar(bKFree + ((t + 1) & 1)));
        }
      }
      if (lead) umma_commit(bar(bDrain));
      drain_wait(bar(bDrain), 0);              // every MMA has finished before TMEM is given back
    }
    __syncwarp();
  } else if (warp >= kGuard) {
    // ---------------------------------------------------------------- guard
    const int g = warp - kGuard;                              // which half of a tile's keys
    for (int t = whole; t < n; ++t) {
      const int j = t - whole;
      if (!warp_wait(bar(bVMasked + j), 0, wc, lane)) break;
      uint8_t* half = smem + kOffRing + ((5 * t + 3 + g) % kSlots) * kBlock;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int r = 32 * m + lane;                          // key 64 g + r of the tile
        const bool there = t * kPfKeys + 64 * g + r < it.nk;
        // x * 0 is NaN exactly where x is not finite
        __nv_bfloat162 acc = __float2bfloat162_rn(0.f);
        const __nv_bfloat162 zero = acc;
        for (int c = 0; c < 16; ++c) {
          // chunks of 16 bytes in an order that keeps the lanes of a quarter warp on different banks
          uint4* q = reinterpret_cast<uint4*>(half + (c >> 3) * (kBlock / 2) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
          if (there) {
            uint4 v = *q;
            const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc = __hfma2(b[e], zero, acc);
          } else {
            *q = make_uint4(0, 0, 0, 0);
          }
        }
        const float2 sum = __bfloat1622float2(acc);
        const bool found = sum.x != 0.f || sum.y != 0.f;      // NaN compares unequal
        const uint32_t mask = __ballot_sync(0xffffffffu, found);
        if (found) {
          for (int c = 0; c < 16; ++c) {
            uint4* q = reinterpret_cast<uint4*>(half + (c >> 3) * (kBlock / 2) + r * 128 + ((c & 7) << 4));
            uint4 v = *q;
            uint32_t* b = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (not_finite(b[e])) b[e] &= 0xFFFF0000u;
              if (not_finite(b[e] >> 16)) b[e] &= 0x0000FFFFu;
            }
            *q = v;
          }
        }
        if (lane == 0) bad[4 * j + 2 * g + m] = mask;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bVClean + j));
    }
  } else {
    // -------------------------------------------------- softmax and epilogue
    const int w = warp >> 2;                                  // row tile
    const int row = 128 * w + 32 * (warp & 3) + lane;         // row of the item
    const uint32_t quad = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + kTmemS + 128 * w + quad, to = tmem + kTmemO + 128 * w + quad;
    const int nw = w ? n_b : n_a;
    const int seen = min(it.nk, it.off + row + 1);            // keys that this row sees (<= 0: none)
    const int first_masked = min(max(it.off + 128 * w + 1, 0), it.nk) / kPfKeys;   // of this row tile
    float ref = -INFINITY, sum = 0.f;
    bool ok = true;
    for (int t = 0; t < nw; ++t) {
      ok = warp_wait(bar(bSFull + w), t & 1, wc, lane);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, s + 32 * c);
      tmem_wait_ld();
      if (t >= first_masked) {
        const int left = seen - t * kPfKeys;
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= left) s[c] = 0xFF800000u;
      }
      float m0 = __uint_as_float(s[0]), m1 = __uint_as_float(s[1]), m2 = __uint_as_float(s[2]),
            m3 = __uint_as_float(s[3]);
#pragma unroll
      for (int c = 4; c < 124; c += 8) {
        m0 = max3(m0, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        m1 = max3(m1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
        m2 = max3(m2, __uint_as_float(s[c + 4]), __uint_as_float(s[c + 5]));
        m3 = max3(m3, __uint_as_float(s[c + 6]), __uint_as_float(s[c + 7]));
      }
      m0 = max3(m0, __uint_as_float(s[124]), __uint_as_float(s[125]));
      m1 = max3(m1, __uint_as_float(s[126]), __uint_as_float(s[127]));
      const float top = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * p.scale_log2;
      const bool move = top > ref + kSlack || (ref == -INFINITY && top > -INFINITY);
      if (t == 0) {
        if (move) ref = top;
      } else if (__any_sync(0xffffffffu, move)) {
        // the product before this one has finished: O is this warp's to rescale
        ok = warp_wait(bar(bPvDone + w), (t - 1) & 1, wc, lane);
        if (!ok) break;
        tc_fence_after();
        const float f = move ? (ref == -INFINITY ? 0.f : ex2_approx(ref - top)) : 1.f;
        if (move) ref = top;
        sum *= f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t o[16];
          tmem_ld16(to + 16 * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tmem_st16(to + 16 * c, o);
        }
      }
      const float sub = ref == -INFINITY ? 0.f : -ref;
      const float2 sc = make_float2(p.scale_log2, p.scale_log2), sb = make_float2(sub, sub);
      float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w32[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 x = f2_fma(make_float2(__uint_as_float(s[64 * c + 2 * e]), __uint_as_float(s[64 * c + 2 * e + 1])), sc, sb);
          const float2 y = make_float2(ex2_approx(x.x), ex2_approx(x.y));
          if (e & 1) acc1 = f2_add(acc1, y);
          else acc0 = f2_add(acc0, y);
          w32[e] = pack_bf16x2(y.x, y.y);
        }
        tmem_st32(ts + 32 * c, w32);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bPFull + w));
      sum += (acc0.x + acc0.y) + (acc1.x + acc1.y);
    }
    if (ok && nw > 0) {
      ok = warp_wait(bar(bPvDone + w), (nw - 1) & 1, wc, lane);
      tc_fence_after();
      for (int t = whole; t < nw && ok; ++t) ok = warp_wait(bar(bVClean + t - whole), 0, wc, lane);
    }
    if (ok && 128 * w < it.nq) {                              // the whole warp: tcgen05.ld is collective
      const bool any = nw > 0 && !(sum == 0.f);
      const float inv = any ? 1.f / sum : 0.f;
      const float lse = any ? (ref + log2f(sum)) * 0.69314718055994531f : -INFINITY;
      const bool live = row < it.nq;
      const size_t out_row = static_cast<size_t>(it.q0 + row) * p.heads + h;
      const size_t part_row = (static_cast<size_t>(max(it.part, 0)) * p.heads + h) * kPfRows + row;
      if (live) {
        if (it.part >= 0) p.part_lse[part_row] = lse;
        else if (p.lse) p.lse[out_row] = lse;
      }
      uint32_t dirty = 0;
      for (int i = 0; i < 12; ++i) dirty |= bad[i];
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t o[32];
        if (nw > 0) {
          tmem_ld32(to + c, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = any ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
        if (!live) continue;
        if (dirty) {
          // values that the guard took out: a key that this row sees gives its infinity or NaN to the sum
          for (int i = 0; i < 12; ++i)
            for (uint32_t m = bad[i]; m; m &= m - 1) {
              const int key = (whole + (i >> 2)) * kPfKeys + 32 * (i & 3) + __ffs(m) - 1;
              if (key >= seen) continue;
              const uint16_t* v = p.v + (it.k0 + key) * p.v_ts + h * p.v_hs + c;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (not_finite(v[e]))
                  o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(static_cast<uint32_t>(v[e]) << 16));
            }
        }
        if (it.part >= 0) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + part_row * kNope + c);
#pragma unroll
          for (int e = 0; e < 8; ++e) reinterpret_cast<uint4*>(dst)[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(p.out + out_row * kNope + c);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t* x = o + 8 * e;
            dst[e] = make_uint4(pack_bf16x2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                                pack_bf16x2(__uint_as_float(x[2]), __uint_as_float(x[3])),
                                pack_bf16x2(__uint_as_float(x[4]), __uint_as_float(x[5])),
                                pack_bf16x2(__uint_as_float(x[6]), __uint_as_float(x[7])));
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) tmem_dealloc(tmem, 512);
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

int launch_prefill(const PrefillParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_kr,
                   const CUtensorMap& tm_v, cudaStream_t stream) {
  if (p.n_items <= 0) return MLA_OK;
  if (!set_smem_limit(reinterpret_cast<const void*>(&prefill_kernel), kSmemBytes)) return MLA_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(p.n_items * p.heads, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  if (cudaLaunchKernelEx(&cfg, prefill_kernel, tm_q, tm_k, tm_kr, tm_v, p) != cudaSuccess) return MLA_ERR_CUDA;
  if (p.n_merges > 0) {
    cfg.gridDim = dim3((kPfRows * p.heads + 7) / 8, p.n_merges, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, prefill_merge_kernel, p) != cudaSuccess) return MLA_ERR_CUDA;
  }
  return cudaPeekAtLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace mla
