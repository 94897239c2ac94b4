// Attention of ragged sequences over expanded keys and values:
//   s_ij = sm_scale (q_i . [k_nope_j, k_rope_j]),  out_i = softmax_j(s_ij) v_j,
//   lse_i = ln sum_j exp(s_ij),
// j up to the causal limit of row i (the sequences' ends aligned), in one pass
// over the keys with the running maximum and sum.
//
// One CTA an SM works through items (up to 256 query rows, their keys) for one
// head each, taken from a counter in the plan's order (heaviest first): two row
// tiles A and B of 128, each with its scores and its output in TMEM (4 x 128
// columns: all of it), so that one tile's softmax runs while the tensor core
// works for the other.  The next item's loads and first scores overlap the
// item's last product and epilogue.  Key tiles of 128:
//   S = Q K^T       M = 128, N = 128, 12 steps of K = 16 (128 + 64 dims), both
//                   operands from shared memory
//   P = exp2(..)    in registers, four threads a row; written back as bf16 over
//                   the scores' own columns
//   O += P V        A from TMEM, V as it lies in memory (N-major), 8 steps
// Bound: the tensor core.  A key tile against both row tiles is 2 x 20 MMAs of
// ~64.4 cycles.  The running maximum is a reference that moves only when a
// tile's maximum exceeds it by 2^8: weights stay below 2^8 (bf16 keeps their 8
// bits at any magnitude, sums are fp32), and O is rescaled in TMEM only then.
//
// A row tile's scores, weights and product follow one another (the weights lie
// over the scores), so its key tile takes as long as that chain.  Traced, the
// softmax takes 250-300 cycles to load, mask and find the maximum, 130 to vote on
// the reference, 710 for the weights (23 exponentials a cycle), 20 to hand them
// over, and then waits for the other row tile's scores, 380 cycles in a causal
// prompt of 4096 rows, 540 without a causal limit: 3540 for a step of both row
// tiles (fitted over causal and ragged batches), about 4000 without a limit, of
// which 2580 are products.  All softmax warps take one row tile, then
// the other: four threads a row, whose quarter of a tile's scores stays in
// registers.  With half of the warps on each (two threads a row, half a tile)
// the long prompts took as long, but registers spilled and items' ends, which
// fall on one row tile at a time, were slower: 140 us instead of 137 for the chunk
// below, 8.5 instead of 8.0 for four requests of 1 to 100 rows; with one thread a
// row the step took 4000.
// Three forms, chosen by the plan:
//   kPair   two CTAs of a cluster and 512 rows (cta_group::2: products of 256
//           rows, CTA 0 issues).  Each CTA holds half of the keys and values,
//           a step takes 3070 cycles for twice the rows, and the ring holds
//           3.2 key tiles instead of 1.6; but an item's ends (first scores,
//           epilogue, up to five partly seen tiles) cost 11400 cycles instead
//           of 7800, and items are coarser.  us on pairs and on single CTAs:
//             causal     1024 x 128 heads 69 and 60, 2048 x 128 163 and 158,
//                        4096 x 128 502 and 514, 8192 x 64 889 and 949
//             no limit   1024 x 128 91 and 91, 2048 x 128 239 and 270,
//                        4096 x 128 887 and 1020, 8192 x 64 1671 and 1951
//             keys cut   512 rows over 65536 x 16 heads 224 and 268, 1024 over
//                        32768 x 32 466 and 530, 2048 over 16384 x 32 448 and 495
//           (the SM clock between 1.75 and 2.07 GHz under the power cap; the
//           long ones vary by 3% from run to run).
//   kSolo   no item has more than 128 rows: one row tile, whose scores take
//           turns in both score buffers (the next key tile's are formed under
//           the softmax of this one), and the second tile's queries' place is
//           ring (2.2 key tiles).  Bound by HBM: 64 rows over 65536 and 32064
//           keys x 16 heads take 137 us (5.9 TB/s), with the general form 155.
//           From L2 a key tile takes 1930 cycles, the general form's step of one
//           row tile, a chain without a second one beside it, 2740.  (Two score
//           buffers with the general form's ring took 178 us where this took 143.)
//
// Warps: 0-15 softmax and epilogue, 16 TMA producer, 17 MMA issuer, 18-19 the
// guard.  A tile that some row sees only in part is
// masked by index in the softmax, but a zero weight times a value that is not
// finite is NaN in the matrix product: the guard clears those values (and the
// rows behind the last key) in shared memory before the product reads them,
// notes the keys, and the epilogue adds them to the rows that do see them.
#include <algorithm>
#include <type_traits>

#include "mla_device.cuh"
#include "mla_launch.h"
#include "mla_prompt.h"

namespace mla {
namespace {

using TileA = std::integral_constant<int, 0>;
using TileB = std::integral_constant<int, 1>;

constexpr int kThreads = 640;
constexpr int kProducer = 16, kIssuer = 17, kGuard = 18;
constexpr int kBlock = 16384;
constexpr int kOffQ = 0;                              // 2 row tiles x 3 blocks of 128 rows x 64 dims
// The ring, in the order of use: keys of tile t as blocks 5t .. 5t+2 (128 keys
// x 64 dims), its values as 5t+3, 5t+4 (64 keys x 128 dims, two 64-dim chunks).
// A pair's CTA has half of each: blocks of 64 keys x 64 dims.
constexpr int kOffRing = 6 * kBlock;
constexpr int kRingBytes = 8 * kBlock;
constexpr int kOffRingSolo = 3 * kBlock;              // a launch of items with one row tile: from behind its queries on
constexpr int kOffBar = kOffRing + kRingBytes;
constexpr int kDepth = 4;                             // tiles told apart: more than the ring holds
constexpr int kSched = 4;                             // items announced ahead
// Masked tiles told apart.  An item has up to three of them, on pairs five, so that the notes that a tile's overwrite
// are of an item that ended three tiles before it or more.  They have been read by then: the tile's place in the ring
// (3.2 tiles at most) is free only when a tile at most three before it has had its products, that tile is of a later
// item than the notes, and its weights come from warps that are through with the items before.
constexpr int kMasked = 8;
constexpr int kConsumers = 4 + 1 + 2;                 // arrivals that give an announced item back: of the softmax warps one for a
                                                      // row's four, issuer (in CTA 1: producer), guard
enum Bar : int {
  bQFull = 0,                    // [2] per row tile
  bQFree = bQFull + 2,           // [2] the row tile's last scores of the item are done
  bKFull = bQFree + 2,           // [4] key tile T on T & 3, T counting the CTA's tiles over all items
  bVFull = bKFull + kDepth,      // [4] the values of whole tile U (that every row sees whole) on U & 3
  bKFree = bVFull + kDepth,      // [4] its QK products are done
  bVFree = bKFree + kDepth,      // [4]
  bSFull = bVFree + kDepth,           // [2] per row tile
  bSOdd = bSFull + 2,            // odd key tiles of an item, in a launch of items with one row tile
  bPFull = bSOdd + 1,            // [2] per row tile; with one, of even and odd key tiles
  bPvDone = bPFull + 2,          // [2] the same
  bVMasked = bPvDone + 2,         // [8] the values of masked tile M (on M & 7) have landed
  bVClean = bVMasked + kMasked,  // [8] and the guard has been over them
  bSched = bVClean + kMasked,    // [4] an item has been announced
  bSchedFree = bSched + kSched,  // [4] and read by every warp
  bDrain = bSchedFree + kSched,
  kBars
};
constexpr int kOffMisc = (kOffBar + 8 * kBars + 15) / 16 * 16;   // TMEM address, abort flag
constexpr int kOffFound = kOffMisc + 8;               // nonzero once some mask in kOffBad was
constexpr int kOffBad = kOffMisc + 16;                // [8][2][4] words: bit j = key j of masked tile M, by the CTA that saw it
constexpr int kOffSched = kOffBad + 32 * kMasked;     // [4] announced items, 8 words each
constexpr int kOffMeet = kOffSched + 32 * kSched;      // [4][2][32] floats: where a row's four threads meet
constexpr int kSmemBytes = kOffMeet + 1024 + 1024;
static_assert(kOffSched % 16 == 0, "announced items are read as 16-byte words");
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr uint32_t kTmemS = 0, kTmemO = 256;          // S_A, S_B, O_A, O_B: 128 columns each
constexpr float kSlack = 8.f;                         // log2 growth of the maximum that moves the reference

// Rows of a row tile's products: one CTA's 128, or a pair's 256.
template <bool kPair>
constexpr int kTileRows = kPair ? 256 : 128;

struct Item {
  int q0, nq, k0, nk, off, part, h;
};

// The item's words, or false (and MLA_ERR_PLAN_MISMATCH) when it does not lie
// inside the arrays of this launch or has keys past its last row's limit.
template <bool kPair, bool kSolo>
__device__ __forceinline__ bool load_item(const PrefillParams& p, int i, Item& it) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(p.items) + 2 * i);
  const int4 b = __ldg(reinterpret_cast<const int4*>(p.items) + 2 * i + 1);
  it = Item{a.y, a.z, a.w, b.x, b.y, b.z, 0};
  return it.q0 >= 0 && it.nq >= 1 && it.nq <= (kSolo ? 1 : 2) * kTileRows<kPair> && it.q0 <= p.q_tokens - it.nq && it.k0 >= 0 && it.nk >= 0 &&
         it.k0 <= p.kv_tokens - it.nk && it.part >= -1 && it.part < p.partials && it.off >= -kPfNoLimit &&
         it.off <= kPfNoLimit && (it.nk == 0 || it.nk <= it.off + it.nq);
}

// What an item asks of each row tile.
struct Shape {
  int n_a, n_b, n;             // key tiles that some row of A, of B, of either sees
  int whole;                   // the first of them are seen whole by every row; at most three (a pair: five) follow
  Shape() = default;
  __device__ __forceinline__ Shape(const Item& it, int rows) {
    auto tiles = [&](int w) -> int {
      if (it.nq <= rows * w) return 0;
      const int last = min(it.nk, it.off + min(it.nq, rows * w + rows));  // keys that the tile's last row sees
      return last > 0 ? (last + kPfKeys - 1) / kPfKeys : 0;
    };
    n_a = tiles(0);
    n_b = tiles(1);
    n = max(n_a, n_b);
    whole = min(n, min(max(it.off + 1, 0), it.nk) / kPfKeys);
  }
};

__device__ __forceinline__ void tma_prefetch_3d(const void* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// ---- the two-CTA forms: a load counted on a barrier of either CTA, products of
// 256 rows issued by CTA 0, commits to both (mla_device.cuh has the others).
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* map, int x, int y, int z, uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
      : "memory");
}
template <bool kPair>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (kPair) umma_commit2(bar);
  else umma_commit(bar);
}
__device__ __forceinline__ void st_cluster_b32(uint32_t addr_cluster, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr_cluster), "r"(v) : "memory");
}

// 32 lanes x 32 consecutive columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
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
// The products with their shared-memory descriptors in halves: the upper word
// (strides, layout) is a constant, only the lower one (address, leading stride)
// changes from MMA to MMA.
template <uint32_t kHigh, bool kPair>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, bool accumulate) {
  if constexpr (kPair) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(kHigh)
      : "memory");
    return;
  }
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(kHigh)
      : "memory");
}
template <uint32_t kHigh, bool kPair>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc, bool accumulate) {
  if constexpr (kPair) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_low), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(kHigh)
      : "memory");
    return;
  }
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_low), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(kHigh)
      : "memory");
}
// The words of sdesc(addr, lbo, 1024) for 128-byte-swizzled atoms.
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | kLayoutSw128 << 29;
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) { return addr >> 4 | (lbo >> 4) << 16; }

__device__ __forceinline__ bool not_finite(uint32_t bf16_bits) { return (bf16_bits & 0x7F80u) == 0x7F80u; }

// Multiplies 32 columns of the thread's TMEM lane by f.  Rare, and out of line:
// inlined, its registers push values of the loop over the keys into memory.
__device__ __noinline__ void rescale_columns(uint32_t taddr, float f) {
#pragma unroll 1
  for (int c = 0; c < 32; c += 16) {
    uint32_t o[16];
    tmem_ld16(taddr + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
    tmem_st16(taddr + c, o);
  }
  tmem_wait_st();
}

// 32 columns of the output from TMEM, times inv, as bf16 (a piece: fp32) to the
// thread's row.  Four lanes exchange blocks of 16 bytes, so that a store writes
// 64 bytes of a row: `dst` is block lane & 3 of the first of their rows, `rows`
// how many of the four there are.  Out of line for the same reason; with all its
// registers free 64 columns of two threads a row took 1700 cycles where 16 at a
// time in the caller took 4500.
template <typename T>
__device__ __noinline__ void store_columns(uint32_t taddr, float inv, T* dst, size_t stride, int rows) {
  constexpr bool kHalf = sizeof(T) == 2;
  constexpr int kCols = kHalf ? 32 : 16;
  const int lane = threadIdx.x & 31;
  uint32_t o[32];
  tmem_ld32(taddr, o);
  tmem_wait_ld();
#pragma unroll
  for (int y = 0; y < 32; y += kCols) {
    uint32_t b[16];
#pragma unroll
    for (int e = 0; e < 16; ++e)
      b[e] = kHalf ? pack_bf16x2(__uint_as_float(o[(2 * e) & 31]) * inv, __uint_as_float(o[(2 * e + 1) & 31]) * inv)
                   : __float_as_uint(__uint_as_float(o[(y + e) & 31]) * inv);
    transpose4_blocks<4>(b, lane);
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (x < rows)
        *reinterpret_cast<uint4*>(dst + x * stride + y) = make_uint4(b[4 * x], b[4 * x + 1], b[4 * x + 2], b[4 * x + 3]);
  }
}

// The warp waits, every lane for itself (through one lane and a shuffle it took
// 7% of the kernel's time longer); all return the same outcome.
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtx& wc) {
  return __all_sync(0xffffffffu, mbar_wait<kCluster>(bar, parity, wc));
}

template <bool kPair, bool kSolo>
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
  int* sched = reinterpret_cast<int*>(smem + kOffSched);
  const WaitCtx wc{abort_flag, p.status};
  constexpr int kRingBlock = kPair ? kBlock / 2 : kBlock;
  constexpr int kRing = kSolo ? kOffRingSolo : kOffRing, kSlots = (kOffBar - kRing) / kRingBlock;
  constexpr int kCtas = kPair ? 2 : 1;
  const uint32_t rank = kPair ? cluster_ctarank() : 0;
  const uint32_t peer = rank ^ 1u;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) {
      const bool softmax = i >= bPFull && i < bPFull + 2;
      const bool two = i >= bVClean && i < bVClean + kMasked;
      const bool all = i >= bSchedFree && i < bSchedFree + kSched;
      mbar_init(bar(i), softmax ? 16 * kCtas : two ? 2 * kCtas : all ? kConsumers * kCtas : 1);
    }
    *abort_flag = 0;
    *reinterpret_cast<int*>(smem + kOffFound) = 0;
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < 8 * kMasked; i += kThreads) bad[i] = 0;
  if (warp == kIssuer) {
    if constexpr (kPair) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(smem_u32(tmem_slot), 512);
      tmem_relinquish();
    }
  }
  if (warp == kProducer && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_kr);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  if constexpr (kPair) cluster_sync_all();              // both CTAs' barriers exist before any remote use
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  // The k-th item announced to this CTA, for every consumer warp: false when there is none left (or on an abort).
  auto announced = [&](uint32_t k, Item& it) -> bool {
    volatile const int* w = sched + 8 * (k % kSched);
    it = Item{w[0], w[1], w[2], w[3], w[4], w[5], w[6]};
    return w[7] != 0;
  };
  auto release_item = [&](uint32_t k) {
    __syncwarp();
    if (lane == 0) {
      if constexpr (kPair) mbar_arrive_cluster(bar(bSchedFree + k % kSched), 0);
      else mbar_arrive(bar(bSchedFree + k % kSched));
    }
  };
  auto next_item = [&](uint32_t k, Item& it) -> bool {
    if (!warp_wait<kPair>(bar(bSched + k % kSched), (k / kSched) & 1, wc)) return false;
    const bool there = announced(k, it);
    release_item(k);
    return there;
  };

  if (warp == kProducer) {
    // ------------------------------------------------ producer and scheduler
    if (lane == 0) {
      const int total = p.n_items * p.heads;
      bool ok = true;
      // block `w` of the launch: items are numbered group of heads by group, heaviest first within it, heads
      // innermost; behind them the tail's items for all heads at once
      const int body = p.n_items - p.n_tail;
      auto fetch = [&](int w, Item& it) {
        const bool tail = w >= body * p.heads;
        const int per_group = body * p.head_group;
        const int g = tail ? 0 : w / per_group, rest = w - (tail ? body * p.heads : g * per_group);
        const int in_group = tail ? p.heads : min(p.head_group, p.heads - g * p.head_group);
        const int item = (tail ? body : 0) + rest / in_group;
        if (!load_item<kPair, kSolo>(p, item, it)) {
          record_status(p.status, MLA_ERR_PLAN_MISMATCH);
          it.nk = it.nq = 0;
        }
        it.h = g * p.head_group + rest % in_group;
      };
      auto announce = [&](uint32_t k, const Item& it, bool there) {
        const int s = k % kSched;
        if (k >= kSched && !mbar_wait<kPair>(bar(bSchedFree + s), ((k / kSched) - 1) & 1, wc)) { ok = false; return; }
        if constexpr (kPair) {
          // to CTA 1 as stores that its barrier counts (its producer arms it)
          const uint32_t to = mapa_shared(base + kOffSched + 32 * s, 1), tb = mapa_shared(bar(bSched + s), 1);
          st_async_v4(to, it.q0, it.nq, it.k0, it.nk, tb);
          st_async_v4(to + 16, it.off, it.part, it.h, there ? 1 : 0, tb);
        }
        reinterpret_cast<int4*>(sched)[2 * s] = make_int4(it.q0, it.nq, it.k0, it.nk);
        reinterpret_cast<int4*>(sched)[2 * s + 1] = make_int4(it.off, it.part, it.h, there ? 1 : 0);
        mbar_arrive(bar(bSched + s));
      };
      // CTA 1's producer: the k-th item as CTA 0 announces it; false when there is none left (or on an abort)
      auto hear = [&](uint32_t k, Item& it) -> bool {
        mbar_arrive_expect_tx(bar(bSched + k % kSched), 32);
        ok = mbar_wait<kPair>(bar(bSched + k % kSched), (k / kSched) & 1, wc);
        if (!ok) return false;
        const bool there = announced(k, it);
        mbar_arrive_cluster(bar(bSchedFree + k % kSched), 0);
        return there;
      };
      int tbase = 0, ubase = 0, mbase = 0;                    // tiles before this item: all, whole, masked
      uint32_t q_items[2] = {0, 0};                           // items with queries in the row tile
      int k_armed = 0, q_bar[2] = {-1, -1};                   // what may be in flight: key tiles, query tiles,
      int v_new = -1, v_old = -1;                             // the last two tiles' values (barrier * 2 + parity)
      Item it;
      if (rank == 0) {
        fetch(blockIdx.x / kCtas, it);
        announce(0, it, true);
      } else {
        hear(0, it);                                          // (every pair has an item)
      }
      int worked = 0;
      for (uint32_t k = 0; ok; ++k) {
        ++worked;
        const Shape sh(it, kTileRows<kPair>);
        auto load_3d = [&](uint32_t dst, const CUtensorMap* m, int x, int z, int b) {
          if constexpr (kPair) tma_load_3d_pair(dst, m, x, it.h, z, mapa_shared(bar(b), 0));
          else tma_load_3d(dst, m, x, it.h, z, bar(b));
        };
        auto load_q = [&](auto W) {
          constexpr int w = W.value;
          if (q_items[w] > 0) ok = mbar_wait(bar(bQFree + w), (q_items[w] - 1) & 1, wc);   // the last item's queries
          if (!ok) return;
          q_bar[w] = q_items[w] & 1;
          ++q_items[w];
          // (a pair's barriers of landed queries, keys and values are CTA 0's, which counts both halves)
          if (rank == 0) mbar_arrive_expect_tx(bar(bQFull + w), kCtas * 3 * kBlock);
          for (int i = 0; i < 3; ++i)
            load_3d(base + kOffQ + (3 * w + i) * kBlock, &tm_q, 64 * i, it.q0 + kTileRows<kPair> * w + 128 * static_cast<int>(rank),
                    bQFull + w);
        };
        // the place of block c, once the block before in it (c - kSlots) has been used
        auto place = [&](int c) -> uint32_t {
          if (c >= kSlots) {
            const int u = (c - kSlots) / 5;
            const int b = (c - kSlots) % 5 < 3 ? bKFree : bVFree;
            ok = mbar_wait(bar(b + u % kDepth), (u / kDepth) & 1, wc);
          }
          return base + kRing + (c % kSlots) * kRingBlock;
        };
        auto load_k = [&](int t) {
          const int T = tbase + t;
          for (int i = 0; i < 3 && ok; ++i) {
            const uint32_t dst = place(5 * T + i);
            const int b = bKFull + T % kDepth, key = it.k0 + t * kPfKeys + 64 * static_cast<int>(rank);
            if (!ok) break;
            if (i == 0 && rank == 0) mbar_arrive_expect_tx(bar(b), 3 * kBlock);
            k_armed = T + 1;
            if (i < 2) load_3d(dst, &tm_k, 64 * i, key, b);
            else if constexpr (kPair) tma_load_2d_pair(dst, &tm_kr, 0, key, mapa_shared(bar(b), 0));
            else tma_load_2d(dst, &tm_kr, 0, key, bar(b));
          }
        };
        auto load_v = [&](int t) {
          const int T = tbase + t, U = ubase + t, M = mbase + t - sh.whole;
          for (int i = 0; i < 2 && ok; ++i) {
            const uint32_t dst = place(5 * T + 3 + i);
            if (!ok) break;
            // masked tiles' values are counted by the CTA whose guard goes over them
            const bool masked = t >= sh.whole;
            const int b = masked ? bVMasked + M % kMasked : bVFull + U % kDepth;
            if (i == 0) {
              v_old = v_new;
              v_new = 2 * b + (masked ? (M / kMasked) & 1 : (U / kDepth) & 1);
              if (masked) mbar_arrive_expect_tx(bar(b), 2 * kRingBlock);
              else if (rank == 0) mbar_arrive_expect_tx(bar(b), 2 * kBlock);
            }
            const int key = it.k0 + t * kPfKeys + 64 * i;
            if constexpr (kPair) {
              if (masked) tma_load_3d(dst, &tm_v, 64 * static_cast<int>(rank), it.h, key, bar(b));
              else load_3d(dst, &tm_v, 64 * static_cast<int>(rank), key, b);
            } else {
              for (int x = 0; x < 2; ++x) tma_load_3d(dst + x * (kBlock / 2), &tm_v, 64 * x, it.h, key, bar(b));
            }
          }
        };
        Item next{};
        bool more = false;
        auto look_ahead = [&] {
          if (rank != 0) {
            more = hear(k + 1, next);
            return;
          }
          const int w = atomicAdd(p.status + kWsCounter, 1) + static_cast<int>(gridDim.x) / kCtas;
          more = static_cast<uint32_t>(w) < static_cast<uint32_t>(total);   // (a counter that was not zero may be negative)
          if (more) fetch(w, next);
          announce(k + 1, next, more);
        };
        // The next item's queries are asked for when a row tile's last scores of this one are done; from L2 they
        // are there sooner.
        auto prefetch_q = [&] {
          const Shape ns(next, kTileRows<kPair>);
          for (int w = 0; w < 2; ++w)
            for (int i = 0; i < 3 && (w ? ns.n_b : ns.n_a) > 0; ++i)
              tma_prefetch_3d(&tm_q, 64 * i, next.h, next.q0 + kTileRows<kPair> * w + 128 * static_cast<int>(rank));
        };
        if (sh.n_a > 0) load_q(TileA{});
        if (ok && sh.n > 0) load_k(0);
        if (ok && sh.n_b > 0) load_q(TileB{});
        if (ok && sh.n > 0) load_v(0);
        if (ok) look_ahead();                                 // the ring is full: its latency costs nothing here
        if (ok && more) prefetch_q();
        for (int t = 1; t < sh.n && ok; ++t) {
          load_k(t);
          if (ok) load_v(t);
        }
        tbase += sh.n;
        ubase += sh.whole;
        mbase += sh.n - sh.whole;
        if (!more) break;
        it = next;
      }
      if (rank == 0) atomicAdd(p.status + kWsWorked, worked);
      if (!ok) {                                              // no copy outlives the block (a pair: the pair)
        if (rank == 0) {
          if (q_bar[0] >= 0) drain_wait(bar(bQFull), q_bar[0]);
          if (q_bar[1] >= 0) drain_wait(bar(bQFull + 1), q_bar[1]);
          for (int T = max(0, k_armed - kDepth); T < k_armed; ++T) drain_wait(bar(bKFull + T % kDepth), (T / kDepth) & 1);
        }
        for (int x : {v_old, v_new})
          if (x >= 0 && (rank == 0 || (x >> 1) >= bVMasked)) drain_wait(bar(x >> 1), x & 1);
      }
    }
    __syncwarp();
  } else if (warp == kIssuer) {
    // ----------------------------------------------------------- MMA issuer
    // The whole warp runs the loop and one elected lane issues: counters and
    // descriptors are then uniform to the compiler (64 cycles an MMA; run by a
    // single lane, 118).  The loop is kept short: what it does between the
    // products is not hidden, as the tensor core's queue holds about four MMAs.
    auto uwait = [&](int b, uint32_t parity) -> bool { return mbar_wait<kPair>(bar(b), parity, wc); };
    const bool lead = elect_one();
    const uint32_t idesc_s = idesc_bf16(kTileRows<kPair>, 128, false, false) | (p.negate ? 1u << 13 : 0u);   // -Q
    constexpr uint32_t kIdescO = idesc_bf16(kTileRows<kPair>, 128, false, true);
    auto block_at = [&](int c) -> uint32_t { return base + kRing + (c % kSlots) * kRingBlock; };
    // scores of key tile T for row tile w; its last of the item: the queries are free
    auto qk = [&](int T, int w, bool last, int odd = 0) {
      const uint32_t d = tmem + kTmemS + 128 * (w + odd);
      const uint32_t a = desc_low(base + kOffQ + 3 * w * kBlock, 16);
      const uint32_t b0 = desc_low(block_at(5 * T), 16), b1 = desc_low(block_at(5 * T + 1), 16),
                     b2 = desc_low(block_at(5 * T + 2), 16);
      if (lead) {
#pragma unroll
        for (int k = 0; k < 12; ++k)
          mma_ss<kDescHigh, kPair>(d, a + (k >> 2) * (kBlock >> 4) + 2 * (k & 3), (k < 4 ? b0 : k < 8 ? b1 : b2) + 2 * (k & 3),
                            idesc_s, k > 0);
        commit<kPair>(bar(bSFull + w + 2 * odd));
        if (last) commit<kPair>(bar(bQFree + w));
      }
    };
    auto pv = [&](int T, int w, bool first, int odd = 0) {
      const uint32_t a = tmem + kTmemS + 128 * (w + odd), d = tmem + kTmemO + 128 * w;
      const uint32_t b0 = desc_low(block_at(5 * T + 3), kBlock / 2), b1 = desc_low(block_at(5 * T + 4), kBlock / 2);
      if (lead) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ts<kDescHigh, kPair>(d, a + 8 * k, (k < 4 ? b0 : b1) + 128 * (k & 3), kIdescO, !first || k > 0);
        commit<kPair>(bar(bPvDone + w + odd));
      }
    };
    int tbase = 0, ubase = 0, mbase = 0;
    uint32_t items = 0, steps = 0;                            // bit w: parity of row tile w's items begun, of its P barrier
    bool ok = true;
    // A wait that gives up makes `ok` false; what is issued until the check at the end of the step stays inside
    // shared memory and TMEM.
    Shape sh{}, next{};
    bool more = rank == 0, there = false;                     // items may follow; `next` is one, and has keys
    uint32_t k = 0;
    auto look_ahead = [&] {
      Item it;
      more = next_item(k++, it);
      if (more) next = Shape(it, kTileRows<kPair>);
      there = more && next.n > 0;
    };
    int k_landed = -1;                                        // the last key tile waited for
    // One row tile in every item: the scores of the next key tile are formed, in a second buffer, under the softmax
    // of this one.
    while (kSolo && ok) {
      do look_ahead();
      while (more && !there);
      if (!there) break;
      sh = next;
      ok = uwait(bKFull + tbase % kDepth, (tbase / kDepth) & 1) && uwait(bQFull, items & 1);
      items ^= 1u;
      tc_fence_after();
      qk(tbase, 0, sh.n == 1);
      if (lead) commit<kPair>(bar(bKFree + tbase % kDepth));
      for (int t = 0; t < sh.n && ok; ++t) {
        const int T = tbase + t, U = ubase + t, M = mbase + t - sh.whole;
        if (t + 1 < sh.n) {
          ok &= uwait(bKFull + (T + 1) % kDepth, ((T + 1) / kDepth) & 1);
          tc_fence_after();
          qk(T + 1, 0, t + 2 == sh.n, ~t & 1);
          if (lead) commit<kPair>(bar(bKFree + (T + 1) % kDepth));
        }
        ok &= t < sh.whole ? uwait(bVFull + U % kDepth, (U / kDepth) & 1)
                           : uwait(bVClean + M % kMasked, (M / kMasked) & 1);
        // (the softmax may be a tile ahead here: even and odd tiles have barriers of their own)
        ok &= uwait(bPFull + (t & 1), (steps >> (t & 1)) & 1);
        steps ^= 1u << (t & 1);
        tc_fence_after();
        pv(T, 0, t == 0, t & 1);
        if (lead) commit<kPair>(bar(bVFree + T % kDepth));
      }
      tbase += sh.n;
      ubase += sh.whole;
      mbase += sh.n - sh.whole;
    }
    auto free_queries = [&] {
      if (sh.n_a > 0) commit<kPair>(bar(bQFree));
      if (sh.n_b > 0) commit<kPair>(bar(bQFree + 1));
    };
    // A CTA of its own: its chain of products and softmax has no slack, and the pairs' loop, which looks into the next
    // item, takes 4% more there (16% a causal prompt of 4096 rows).
    while (!kPair && !kSolo && ok) {
      do look_ahead();
      while (more && !there);
      if (!there) break;
      sh = next;
      // the first scores: they may run while the epilogue of the item before reads its output
      ok = uwait(bKFull + tbase % kDepth, (tbase / kDepth) & 1);
#pragma unroll 1
      for (int w = 0; w < 2; ++w) {
        if ((w ? sh.n_b : sh.n_a) == 0) {
          if (lead) commit<kPair>(bar(bSFull + w));           // an empty step
          continue;
        }
        ok &= uwait(bQFull + w, (items >> w) & 1);
        items ^= 1u << w;
        tc_fence_after();
        qk(tbase, w, false);
      }
      if (lead) {
        commit<kPair>(bar(bKFree + tbase % kDepth));
        if (sh.n == 1) free_queries();
      }
      for (int t = 0; t < sh.n && ok; ++t) {
        const int T = tbase + t, U = ubase + t, M = mbase + t - sh.whole;
        ok &= t < sh.whole ? uwait(bVFull + U % kDepth, (U / kDepth) & 1)
                           : uwait(bVClean + M % kMasked, (M / kMasked) & 1);
        // P of an item's first tile also tells that its warps have read the output of the item before
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
          const int nw = w ? sh.n_b : sh.n_a;
          if (t < nw) {
            ok &= uwait(bPFull + w, (steps >> w) & 1);
            steps ^= 1u << w;
            tc_fence_after();
            pv(T, w, t == 0);
          }
          if (w == 0 && t + 1 < sh.n) ok &= uwait(bKFull + (T + 1) % kDepth, ((T + 1) / kDepth) & 1);
          if (t + 1 < nw) {
            tc_fence_after();
            qk(T + 1, w, false);
          }
        }
        if (lead) {
          commit<kPair>(bar(bVFree + T % kDepth));
          if (t + 1 < sh.n) commit<kPair>(bar(bKFree + (T + 1) % kDepth));
          if (t + 2 == sh.n) free_queries();
        }
      }
      for (int w = 0; w < 2; ++w)
        if ((w ? sh.n_b : sh.n_a) == 0) {
          ok &= uwait(bPFull + w, (steps >> w) & 1);
          steps ^= 1u << w;
          if (lead) commit<kPair>(bar(bPvDone + w));
        }
      tbase += sh.n;
      ubase += sh.whole;
      mbase += sh.n - sh.whole;
    }
    while (kPair && ok) {
      // Step t of the item: each row tile's product of key tile t and its scores of tile t + 1, or of the next item's
      // first, which then run while the epilogue of this one reads its output.  Step -1, of no item, begins the first
      // item and one behind an item without keys.
      uint32_t begun = 0;                                     // bit w: the next item's first scores of row tile w are issued
      for (int t = sh.n > 0 ? 0 : -1; t < sh.n && ok; ++t) {
        const int T = tbase + t, U = ubase + t, M = mbase + t - sh.whole;
        if (t < 0) {
          while (more && !there) look_ahead();
        } else {
          // (one item only: the announcement of a second may wait for the softmax of this one)
          if (t == max(0, sh.n - 2) && more) look_ahead();
          ok &= t < sh.whole ? uwait(bVFull + U % kDepth, (U / kDepth) & 1)
                             : uwait(bVClean + M % kMasked, (M / kMasked) & 1);
        }
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
          const int nw = w ? sh.n_b : sh.n_a;
          // P of an item's first tile also tells that its warps have finished with the item before (a row tile without
          // keys takes an empty step for that alone)
          if (t >= 0 && t < max(nw, 1)) {
            ok &= uwait(bPFull + w, (steps >> w) & 1);
            steps ^= 1u << w;
            tc_fence_after();
            if (nw > 0) pv(T, w, t == 0);
            else if (lead) commit<kPair>(bar(bPvDone + w));
          }
          int tile = T + 1, left = nw - t - 1;                // row tile's key tiles from there on
          if (left <= 0) {
            // The next item's keys lie in the ring beside what this one still needs: 10 of its 16 blocks one tile
            // before the last.
            if (!there || (begun >> w & 1) || t + 2 < sh.n) continue;
            begun |= 1u << w;
            tile = tbase + sh.n;
            left = w ? next.n_b : next.n_a;
            if (left == 0) {
              if (lead) commit<kPair>(bar(bSFull + w));
              continue;
            }
            ok &= uwait(bQFull + w, (items >> w) & 1);
            items ^= 1u << w;
          }
          if (tile != k_landed) ok &= uwait(bKFull + tile % kDepth, (tile / kDepth) & 1);
          k_landed = tile;
          tc_fence_after();
          qk(tile, w, left == 1);
        }
        if (lead) {
          if (t >= 0) commit<kPair>(bar(bVFree + T % kDepth));
          if (t + 1 < sh.n || there) commit<kPair>(bar(bKFree + (T + 1) % kDepth));
        }
      }
      tbase += sh.n;
      ubase += sh.whole;
      mbase += sh.n - sh.whole;
      if (there) sh = next;
      else if (more) sh = Shape{};
      else break;
      there = false;
    }
    if (rank == 0) {
      if (lead) commit<kPair>(bar(bDrain));
      drain_wait(bar(bDrain), 0);                             // every MMA has finished before TMEM is given back
    }
    __syncwarp();
  } else if (warp >= kGuard) {
    // ---------------------------------------------------------------- guard
    const int g = warp - kGuard;                              // which half of a tile's keys
    int tbase = 0, M = 0;
    Item it;
    bool ok = true;
    for (uint32_t k = 0; ok && next_item(k, it); ++k) {
      const Shape sh(it, kTileRows<kPair>);
      for (int t = sh.whole; t < sh.n; ++t, ++M) {
        ok = warp_wait(bar(bVMasked + M % kMasked), (M / kMasked) & 1, wc);
        if (!ok) break;
        uint8_t* half = smem + kRing + ((5 * (tbase + t) + 3 + g) % kSlots) * kRingBlock;
#pragma unroll 1
        for (int m = 2 * g; m < 2 * g + 2; ++m) {
          const int r = 32 * (m & 1) + lane;                  // row of this half's 64: key 32 m + lane of the tile
          const bool there = t * kPfKeys + 32 * m + lane < it.nk;
          // chunks of 16 bytes in an order that keeps the lanes of a quarter warp on different banks
          auto chunk = [&](int c) {
            return reinterpret_cast<uint4*>(half + (c >> 3) * (kBlock / 2) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
          };
          constexpr int kChunks = kPair ? 8 : 16;             // of a key's values that lie here
          uint4 v[kChunks];
#pragma unroll
          for (int c = 0; c < kChunks; ++c) v[c] = *chunk(c);
          // x * 0 is NaN exactly where x is not finite
          __nv_bfloat162 acc = __float2bfloat162_rn(0.f);
          const __nv_bfloat162 zero = acc;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&v[c]);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc = __hfma2(b[e], zero, acc);
          }
          if (!there) {
            acc = zero;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) *chunk(c) = make_uint4(0, 0, 0, 0);
          }
          const float2 sum = __bfloat1622float2(acc);
          const bool found = sum.x != 0.f || sum.y != 0.f;    // NaN compares unequal
          const uint32_t mask = __ballot_sync(0xffffffffu, found);
          if (found) {
            for (int c = 0; c < kChunks; ++c) {
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
          if (lane == 0) {
            const int at = 8 * (M % kMasked) + 4 * static_cast<int>(rank) + m;
            bad[at] = mask;
            if (mask) *reinterpret_cast<volatile int*>(smem + kOffFound) = 1;
            if constexpr (kPair) {
              st_cluster_b32(mapa_shared(base + kOffBad + 4 * at, peer), mask);
              if (mask) st_cluster_b32(mapa_shared(base + kOffFound, peer), 1);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair) mbar_arrive_cluster(bar(bVClean + M % kMasked), peer);
          mbar_arrive(bar(bVClean + M % kMasked));
        }
      }
      tbase += sh.n;
    }
  } else {
    // -------------------------------------------------- softmax and epilogue
    // All 16 warps work on one row tile, then on the other: four threads a row, in the warps of one TMEM lane
    // quadrant, each with a quarter of a tile's keys and of the output's columns.  They meet at a named barrier of
    // their 128 threads and agree on the reference maximum there.
    const int quarter = warp >> 2, quad = warp & 3;
    const int row_a = 128 * static_cast<int>(rank) + 32 * quad + lane;   // row of the item, in row tile A
    const int quad_bar = 1 + quad;
    float* meet = reinterpret_cast<float*>(smem + kOffMeet) + 64 * quad + lane;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * quad) << 16);
    const uint32_t ts = at + kTmemS + 32 * quarter, tp = at + kTmemS + 16 * quarter, to = at + kTmemO + 32 * quarter;
    // Combines a value of the row's four threads, in a fixed order; all return the result.
    auto all4 = [&](float mine, auto op) -> float {
      if (quarter >= 2) meet[32 * (quarter - 2)] = mine;
      named_bar_sync(quad_bar, 128);
      if (quarter < 2) mine = op(mine, meet[32 * quarter]);
      if (quarter == 1) meet[32] = mine;
      named_bar_sync(quad_bar, 128);
      if (quarter == 0) {
        mine = op(mine, meet[32]);
        meet[0] = mine;
      }
      named_bar_sync(quad_bar, 128);
      return meet[0];                                         // (the next to write it comes through a barrier first)
    };
    auto agree = [&](bool fine) -> bool { return !named_bar_or(quad_bar, 128, !fine); };
    uint32_t scores = 0;                                      // bit b: parity of score barrier b
    auto arrive_p = [&](int b) {
      __syncwarp();
      if (lane == 0) {
        if constexpr (kPair) mbar_arrive_leader_relaxed(bar(bPFull + b));
        else mbar_arrive(bar(bPFull + b));
      }
    };
    int mbase = 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      // (a wait that gives up ends all warps of a row at the same place: none is left at their barrier)
      ok = agree(warp_wait<kPair>(bar(bSched + k % kSched), (k / kSched) & 1, wc));
      if (!ok) break;
      // The item's words are read here for the loop over the keys and again for the epilogue.
      int n_a, n_b, n, seen_a, nk;
      {
        Item it;
        const bool there = announced(k, it);
        if (!there) break;
        const Shape sh(it, kTileRows<kPair>);
        n_a = sh.n_a;
        n_b = sh.n_b;
        n = sh.n;
        nk = it.nk;
        seen_a = it.off + row_a + 1;                          // keys that the row sees, had the item more of them
      }
      float ref = -INFINITY, sum = 0.f, ref_other = -INFINITY, sum_other = 0.f;   // of this row tile, of the other
#pragma unroll 1
      for (int x = 0; x < 2 * (n + 1); ++x) {
        const int t = x >> 1, w = x & 1, nw = w ? n_b : n_a;
        const int b = kSolo ? t & 1 : w;                      // score buffer, and the barriers'
        if (kSolo && w) continue;
        if (t < nw) {
          ok = warp_wait(bar(kSolo && b ? bSOdd : bSFull + w), (scores >> b) & 1, wc);
          scores ^= 1u << b;
          tc_fence_after();
          uint32_t s[32];
          auto load_scores = [&] {
            tmem_ld32(ts + 128 * b, s);
            tmem_wait_ld();
            // of the quarter's keys, those this row sees
            const int left = min(nk, seen_a + kTileRows<kPair> * w) - t * kPfKeys - 32 * quarter;
            if (left < 32) {
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (c >= left) s[c] = 0xFF800000u;
            }
          };
          load_scores();
          float m0 = -INFINITY, m1 = m0;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            m0 = max3(m0, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
            m1 = max3(m1, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
          }
          float top = fmaxf(m0, m1) * p.scale_log2;
          // some row of the four warps has outgrown its reference (a wait that gave up ends all of them here, too)
          auto outgrown = [&] { return top > ref + kSlack || (ref == -INFINITY && top > -INFINITY); };
          tc_fence_before();
          const bool settle = named_bar_or(quad_bar, 128, outgrown() || !ok);
          tc_fence_after();
          if (settle) {
            ok = agree(ok);
            if (ok) {
              top = all4(top, [](float a, float b) { return fmaxf(a, b); });
              const bool move = outgrown();
              if (t == 0) {
                if (move) ref = top;
              } else {
                // the product before this one has finished: O is these warps' to rescale
                if constexpr (kSolo) ok = warp_wait(bar(bPvDone + (b ^ 1)), (~scores >> (b ^ 1)) & 1, wc);
                else ok = warp_wait(bar(bPvDone + w), (scores >> w) & 1, wc);
                tc_fence_after();
                const float f = move ? (ref == -INFINITY ? 0.f : ex2_approx(ref - top)) : 1.f;
                if (move) ref = top;
                sum *= f;
                rescale_columns(to + 128 * w, f);
                load_scores();
                tc_fence_before();
                ok = agree(ok);
                tc_fence_after();
              }
            }
          }
          if (!ok) break;
          const float sub = ref == -INFINITY ? 0.f : -ref;
          const float2 sc = make_float2(p.scale_log2, p.scale_log2), sb = make_float2(sub, sub);
          float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
          // The weights go over columns 0-63 of the tile's scores, which all four warps have read: they have passed
          // the barrier above.
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t* z = s + 16 * c + 2 * e;
              const float2 v = f2_fma(make_float2(__uint_as_float(z[0]), __uint_as_float(z[1])), sc, sb);
              const float2 y = make_float2(ex2_approx(v.x), ex2_approx(v.y));
              if (e & 1) acc1 = f2_add(acc1, y);
              else acc0 = f2_add(acc0, y);
              pk[e] = pack_bf16x2(y.x, y.y);
            }
            tmem_st8(tp + 128 * b + 8 * c, pk);
          }
          tmem_wait_st();
          tc_fence_before();
          arrive_p(b);
          sum += (acc0.x + acc0.y) + (acc1.x + acc1.y);
        } else if (t == nw) {
          // ------ the row tile's end: its output
          Item it;
          announced(k, it);
          const Shape sh(it, kTileRows<kPair>);
          if (!kSolo && nw == 0 && n > 0) {                   // an empty step
            ok = warp_wait(bar(bSFull + w), (scores >> w) & 1, wc);
            scores ^= 1u << w;
            arrive_p(w);
          }
          if (nw > 0) {
            const int last = kSolo ? (nw - 1) & 1 : w;
            ok = warp_wait(bar(bPvDone + last), (~scores >> last) & 1, wc);
            tc_fence_after();
          }
          uint32_t dirty = 0;                                 // some masked tile of this row tile had its values cleared
          if (ok && nw > sh.whole) {                          // the guard's notes up to this row tile's last
            const int M = mbase + nw - 1 - sh.whole;
            ok = warp_wait<kPair>(bar(bVClean + M % kMasked), (M / kMasked) & 1, wc);
            if (*reinterpret_cast<volatile int*>(smem + kOffFound))
              for (int u = sh.whole; u < nw; ++u)
                for (int i = 0; i < 8; ++i) dirty |= bad[8 * ((mbase + u - sh.whole) % kMasked) + i];
          }
          ok = agree(ok);
          if (!ok) break;
          // The words of the item before are given back: the row's four warps have read them.  Across the pair that
          // release waits for the warp's output stores, which are done by now (right behind them it took 5% of the
          // kernel's time).
          if (w == 0 && k > 0 && quarter == 0) release_item(k - 1);
          const int row = row_a + kTileRows<kPair> * w;
          if (row - lane - 32 * quad < it.nq) {               // all warps of this CTA: they meet
            sum = all4(sum, [](float a, float b) { return a + b; });
            const bool any = nw > 0 && !(sum == 0.f);
            const float inv = any ? 1.f / sum : 0.f;
            const float lse = any ? (ref + log2f(sum)) * 0.69314718055994531f : -INFINITY;
            const bool live = row < it.nq;
            const size_t out_row = static_cast<size_t>(it.q0 + row) * p.heads + it.h;
            const size_t part_row = (static_cast<size_t>(max(it.part, 0)) * p.heads + it.h) * (2 * kTileRows<kPair>) + row;
            if (live && quarter == 0) {
              if (it.part >= 0) p.part_lse[part_row] = lse;
              else if (p.lse) p.lse[out_row] = lse;
            }
            // all but rows without a key and tiles of which the guard has taken out values
            const int mate = lane & 3, first = row - mate;    // of the first of four lanes' rows
            const bool plain = __all_sync(0xffffffffu, any) && dirty == 0;
            if (plain && it.part < 0)
              store_columns(to + 128 * w, inv, p.out + (out_row - static_cast<size_t>(mate) * p.heads) * kNope + 32 * quarter + 8 * mate,
                            static_cast<size_t>(p.heads) * kNope, it.nq - first);
            else if (plain)
              store_columns(to + 128 * w, inv, p.part_o + (part_row - mate) * kNope + 32 * quarter + 4 * mate, static_cast<size_t>(kNope),
                            it.nq - first);
#pragma unroll 1
            for (int c = 32 * quarter; c < 32 * quarter + 32 && !plain; c += 16) {
              uint32_t o[16];
              if (nw > 0) {
                tmem_ld16(to + 128 * w + (c & 16), o);
                tmem_wait_ld();
              }
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = any ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
              if (dirty && live && any) {
                // values that the guard took out: a key that this row sees gives its infinity or NaN to the sum (a
                // row without a score above -inf has no sum)
                const int all = min(it.nk, it.off + row + 1);
                for (int u = sh.whole; u < nw; ++u)
                  for (int i = 0; i < 4; ++i)
                    for (uint32_t m = bad[8 * ((mbase + u - sh.whole) % kMasked) + i] |
                                      bad[8 * ((mbase + u - sh.whole) % kMasked) + 4 + i];
                         m; m &= m - 1) {
                      const int key = u * kPfKeys + 32 * i + __ffs(m) - 1;
                      if (key >= all) continue;
                      const uint16_t* v = p.v + (it.k0 + key) * p.v_ts + it.h * p.v_hs + c;
#pragma unroll
                      for (int e = 0; e < 16; ++e)
                        if (not_finite(v[e]))
                          o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(static_cast<uint32_t>(v[e]) << 16));
                    }
              }
              // the same exchange, of 16 columns
              if (it.part >= 0) {
                transpose4_blocks<4>(o, lane);
                float* dst = p.part_o + (part_row - mate) * kNope + c + 4 * mate;
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  if (first + y < it.nq)
                    *reinterpret_cast<uint4*>(dst + y * kNope) = make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
              } else {
                uint32_t h[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = pack_bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
                transpose4_blocks<2>(h, lane);
                uint16_t* dst = p.out + (out_row - static_cast<size_t>(mate) * p.heads) * kNope + c + 4 * mate;
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  if (first + y < it.nq)
                    *reinterpret_cast<uint2*>(dst + static_cast<size_t>(y) * p.heads * kNope) = make_uint2(h[2 * y], h[2 * y + 1]);
              }
            }
          }
        }
        if constexpr (!kSolo) {
          const float r = ref, a = sum;
          ref = ref_other;
          sum = sum_other;
          ref_other = r;
          sum_other = a;
        }
      }
      if (!ok) break;
      {
        Item it;
        announced(k, it);
        const Shape sh(it, kTileRows<kPair>);
        mbase += sh.n - sh.whole;
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  if constexpr (kPair) {
    cluster_sync_all();                                       // no CTA leaves while the other signals it
    if (warp == kIssuer) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  } else {
    __syncthreads();
    if (warp == kIssuer) tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0) {
    // The last block to finish leaves the counters at zero for the next launch.  All items have been worked on by then
    // (unless a wait gave up: its status stands); fewer or more say that the counters were not zero, or that another
    // launch used them.
    __threadfence();
    const int blocks = static_cast<int>(gridDim.x), done = atomicAdd(p.status + kWsDone, 1);
    if (done == blocks - 1) {
      if (atomicExch(p.status + kWsWorked, 0) != p.n_items * p.heads) record_status(p.status, MLA_ERR_WORKSPACE);
      p.status[kWsCounter] = 0;
      p.status[kWsDone] = 0;
    } else if (done < 0 || done >= blocks) {
      record_status(p.status, MLA_ERR_WORKSPACE);
    }
  }
}

// Joins the pieces of a cut tile: one warp a (row, head), 4 values a lane.
// Bound: latency (10 MB of pieces where it was measured); with the pieces' weights
// and rows one after the other the call took 3 us longer.
__global__ void __launch_bounds__(256) prefill_merge_kernel(const PrefillParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int4 e = __ldg(reinterpret_cast<const int4*>(p.merges) + blockIdx.y);
  const int q0 = e.x, nq = e.y, p0 = e.z, p1 = e.w;
  if (q0 < 0 || nq < 1 || nq > p.rows || q0 > p.q_tokens - nq || p0 < 0 || p1 <= p0 || p1 > p.partials) {
    if (threadIdx.x == 0) record_status(p.status, MLA_ERR_PLAN_MISMATCH);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int r = i / p.heads, h = i - r * p.heads;
  if (r >= nq) return;
  // A lane takes a piece's log-sum-exp (32 pieces at a time), then the pieces' rows come four at a time.
  auto lse_of = [&](int k) -> float {
    return k < p1 ? p.part_lse[(static_cast<size_t>(k) * p.heads + h) * p.rows + r] : -INFINITY;
  };
  float m = -INFINITY;
  bool bad = false;
  for (int k = p0; k < p1; k += 32) {
    const float s = lse_of(k + lane);
    bad |= s != s;
    m = fmaxf(m, s);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  bad = __any_sync(0xffffffffu, bad);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  for (int k = p0; k < p1; k += 32) {
    const float s = lse_of(k + lane);
    const float e = s == -INFINITY ? 0.f : expf(s - m);    // 0: nothing seen in this piece
    const int n = min(32, p1 - k);
#pragma unroll 4
    for (int x = 0; x < n; ++x) {
      const float w = __shfl_sync(0xffffffffu, e, x);
      const float4 v = *reinterpret_cast<const float4*>(
          p.part_o + ((static_cast<size_t>(k + x) * p.heads + h) * p.rows + r) * kNope + 4 * lane);
      l += w;
      o.x = fmaf(w, v.x, o.x);
      o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
    }
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
  const bool pair = p.rows > kPfRows;
  const auto kernel = pair ? &prefill_kernel<true, false> : p.solo ? &prefill_kernel<false, true> : &prefill_kernel<false, false>;
  if (!set_smem_limit(reinterpret_cast<const void*>(kernel), kSmemBytes)) return MLA_ERR_CUDA;
  const int sms = device_sm_count();
  if (sms < 1) return MLA_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pair ? 2 : 1;
  const int workers = pair ? std::max(1, sms / 2) : sms;
  cfg.gridDim = dim3(std::min(p.n_items * p.heads, workers) * (pair ? 2 : 1), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  if (cudaLaunchKernelEx(&cfg, kernel, tm_q, tm_k, tm_kr, tm_v, p) != cudaSuccess) return MLA_ERR_CUDA;
  cfg.numAttrs = 1;
  if (p.n_merges > 0) {
    cfg.gridDim = dim3((p.rows * p.heads + 7) / 8, p.n_merges, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, prefill_merge_kernel, p) != cudaSuccess) return MLA_ERR_CUDA;
  }
  return cudaPeekAtLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace mla
