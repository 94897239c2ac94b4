// Latent expansion: the cached rows named by kv_indices to every head's keys
// and values,
//   k[t, h, n] = sum_r c_t[r] w_kc[h, n, r],   v[t, h, n] = sum_r c_t[r] w_vc[h, r, n],
// and the rope key that all heads share.  c_t is the 512-wide latent of the
// row (an FP8 row's code values, kv_scale - or the row's own scale - applied to
// the sums); fp32 sums, one rounding.  With rows' own scales 4095 rows x 128
// heads take 99 us (1.39 PFLOP/s), 257 rows x 16 heads 8.1.
//
// One matrix product [tokens, 512] x [512, 256 heads] whose left side is
// gathered.  A CTA keeps the whole depth of 128 rows in shared memory (128
// KB), so a row is gathered - and an FP8 row widened - once for all the column
// tiles that the CTA walks, by plain loads of four warps, and only weights
// stream.  A column tile is NT columns: the keys, or the values, of NT / 128
// heads; w_kc is K-major as it lies, w_vc N-major.
//   warp 0      TMA producer of the weights, 64-deep chunks in a ring
//   warp 1      TMEM allocator, MMA issuer: two accumulators in turn
//   warps 4-11  epilogue: a TMEM lane is a row; 32 columns at a time, exchanged
//               between four lanes and stored in rows of 64 bytes; two warps
//               share a lane quadrant and take half of the columns each (four
//               warps needed 6500 cycles a tile, the products 4100)
//   warps 12-15 rows: gather, swizzle (128-byte atoms), rope keys
//   warp 2      (CTA 1 of a pair) tells CTA 0 of landed rows
// kPair: two CTAs of a cluster work on one tile of 256 rows x 256 columns
// (cta_group::2): each holds its 128 rows and half of the weights' columns,
// CTA 0 issues for both.  That halves the weights that every SM reads from L2,
// which bounded the single-CTA form (1.07 GB in 134 us at 4096 rows x 128
// heads).  Bound: the weights from L2 still: with them there a tile of 256 x 256
// takes 4200 cycles (32 MMAs of 128), but late, 5500-6100 through most of the
// kernel, as beside the rows there is room for six stages of 16 KB (four: 112 us,
// five: 103, and the output stored through shared memory in the sixth's place).
// 4096 rows x 128 heads take 97 us (1415 TFLOP/s, 0.71 of cuBLAS's rate), 8191
// rows x 32 heads from E4M3 48 us, 257 rows x 16 heads 6.2 us.
#include <type_traits>

#include "mla_device.cuh"
#include "mla_launch.h"
#include "mla_prompt.h"

namespace mla {
namespace ex {

constexpr int kThreads = 512;
constexpr int kEpiWarp0 = 4, kEpiWarps = 8, kRowWarp0 = 12;
constexpr int BM = 128, BK = 64, kChunks = kLatent / BK;

template <int NT_, bool kPair>
struct Cfg {
  static constexpr int NT = NT_;
  static constexpr int kHeads = NT / kNope;                 // heads of a tile
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kABytes = kChunks * BM * 128;        // 128 KB
  static constexpr int kCols = NT / kCtas;                  // of a tile's columns, those this CTA loads
  static constexpr int kBBytes = kCols * BK * 2;
  static constexpr int kStages = (96 * 1024) / kBBytes;
  static constexpr int kOffB = kABytes;
  static constexpr int kOffBar = kOffB + kStages * kBBytes;
  // full[S], empty[S], a_full[8], a_free[8], acc_full[2], acc_empty[2]
  static constexpr int kBars = 2 * kStages + 2 * kChunks + 4;
  static constexpr int kOffMisc = kOffBar + 8 * kBars;
  static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
  static constexpr int kTmemCols = 2 * NT;
  static constexpr uint32_t kIdescK = idesc_bf16(kCtas * BM, NT, false, false);
  static constexpr uint32_t kIdescV = idesc_bf16(kCtas * BM, NT, false, true);
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t codes) {
  const float2 f = e4m3x2_value(codes);
  return pack_bf16x2(f.x, f.y);                             // exact
}

// ---- the two-CTA forms of the tensor core's instructions
__device__ __forceinline__ void tmem_alloc2(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void umma_ss2(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 bytes, or 16 zero bytes with nothing read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N of this thread's committed groups have landed.
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <CacheForm kForm, int NT, bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    expand_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const ExpandParams p) {
  using C = Cfg<NT, kPair>;
  constexpr bool kFp8 = kForm != CacheForm::kBf16, kRows = kForm == CacheForm::kRowScaled;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return base + C::kOffBar + 8u * i; };
  auto full = [&](int s) { return bar(s); };
  auto empty = [&](int s) { return bar(C::kStages + s); };
  auto a_full = [&](int k) { return bar(2 * C::kStages + k); };
  auto a_free = [&](int k) { return bar(2 * C::kStages + kChunks + k); };
  auto acc_full = [&](int i) { return bar(2 * C::kStages + 2 * kChunks + i); };
  auto acc_empty = [&](int i) { return bar(2 * C::kStages + 2 * kChunks + 2 + i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const WaitCtx wc{abort_flag, p.status};

  const uint32_t rank = kPair ? cluster_ctarank() : 0;
  // this CTA's (pair's) tiles: rows outer, columns (keys of the heads, then values) inner
  const int groups = (p.heads + C::kHeads - 1) / C::kHeads;
  const int cols = 2 * groups;
  const int tile_rows = C::kCtas * BM;
  const long long tiles = static_cast<long long>((p.tokens + tile_rows - 1) / tile_rows) * cols;
  const int worker = blockIdx.x / C::kCtas, workers = gridDim.x / C::kCtas;
  const int t0 = static_cast<int>(tiles * worker / workers);
  const int t1 = static_cast<int>(tiles * (worker + 1) / workers);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) { mbar_init(full(s), 1); mbar_init(empty(s), 1); }
    for (int k = 0; k < kChunks; ++k) { mbar_init(a_full(k), kPair && rank == 0 ? 5 : 4); mbar_init(a_free(k), 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(acc_full(i), 1); mbar_init(acc_empty(i), kEpiWarps * C::kCtas); }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc2(smem_u32(tmem_slot), C::kTmemCols);
      tmem_relinquish2();
    } else {
      tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
      tmem_relinquish();
    }
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  if constexpr (kPair) cluster_sync_all();                  // both CTAs' barriers exist before any remote use
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0) {
    // ---------------------------------------------------- weights producer
    if (lane == 0) {
      uint32_t c = 0;
      bool ok = true;
      for (int t = t0; t < t1 && ok; ++t) {
        const int col = t % cols, h = (col % groups) * C::kHeads;
        for (int k = 0; k < kChunks; ++k, ++c) {
          const uint32_t s = c % C::kStages;
          if (c >= C::kStages && !mbar_wait(empty(s), ((c / C::kStages) - 1) & 1, wc)) { ok = false; break; }
          const uint32_t dst = base + C::kOffB + s * C::kBBytes;
          // both halves of a pair's tile are counted on CTA 0's barrier
          if (rank == 0) mbar_arrive_expect_tx(full(s), C::kCtas * C::kBBytes);
          const int hh = h + static_cast<int>(rank) * (C::kCols / kNope);
          const uint32_t fb = kPair ? mapa_shared(full(s), 0) : full(s);
          auto load = [&](uint32_t d, const CUtensorMap* m, int x, int y) {
            if constexpr (kPair) tma_load_2d_pair(d, m, x, y, fb);
            else tma_load_2d(d, m, x, y, fb);
          };
          if (col < groups) {
            load(dst, &tm_k, k * BK, hh * kNope);                             // kCols rows of 64
          } else {
#pragma unroll
            for (int j = 0; j < C::kCols / 64; ++j)                           // 64 rows of 64
              load(dst + j * (BK * 128), &tm_v, 64 * (j & 1), (hh + (j >> 1)) * kLatent + k * BK);
          }
        }
      }
      if (!ok && rank == 0)                                  // no copy outlives the block
        for (uint32_t d = c > C::kStages ? c - C::kStages : 0; d < c; ++d)
          drain_wait(full(d % C::kStages), (d / C::kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer
    // The whole warp runs the loop and one elected lane issues: loop counters
    // and descriptors are then uniform to the compiler, which keeps them in
    // uniform registers.
    if (rank == 0) {
      const bool lead = elect_one();
      auto mma = [](uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
        if constexpr (kPair) umma_ss2(d, a, b, idesc, acc);
        else umma_ss(d, a, b, idesc, acc);
      };
      auto commit = [](uint32_t b) {
        if constexpr (kPair) umma_commit2(b);
        else umma_commit(b);
      };
      auto D = [](uint64_t d, uint32_t off) -> uint64_t { return d + (off >> 4); };
      uint32_t c = 0, i = 0, block = 0;
      bool ok = true;
      for (int t = t0; t < t1 && ok; ++t, ++i) {
        const bool fresh = t == t0 || t % cols == 0;         // the first tile of a block of rows
        const bool last = t + 1 == t1 || (t + 1) % cols == 0;
        const bool key = t % cols < groups;
        const uint32_t buf = i & 1;
        if (i >= 2 && !mbar_wait<kPair>(acc_empty(buf), ((i >> 1) - 1) & 1, wc)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem + buf * NT;
        for (int k = 0; k < kChunks; ++k, ++c) {
          const uint32_t s = c % C::kStages;
          if (fresh && !mbar_wait<kPair>(a_full(k), block & 1, wc)) { ok = false; break; }
          if (!mbar_wait(full(s), (c / C::kStages) & 1, wc)) { ok = false; break; }
          tc_fence_after();
          const uint64_t da = sdesc(base + k * (BM * 128), 16, 1024);
          if (key) {
            const uint64_t db = sdesc(base + C::kOffB + s * C::kBBytes, 16, 1024);
#pragma unroll
            for (int ks = 0; ks < BK / 16; ++ks)
              if (lead) mma(d, D(da, ks * 32), D(db, ks * 32), C::kIdescK, (k | ks) != 0 ? 1u : 0u);
          } else {
            const uint64_t db = sdesc(base + C::kOffB + s * C::kBBytes, BK * 128, 1024);
#pragma unroll
            for (int ks = 0; ks < BK / 16; ++ks)
              if (lead) mma(d, D(da, ks * 32), D(db, ks * 2048), C::kIdescV, (k | ks) != 0 ? 1u : 0u);
          }
          if (lead) {
            commit(empty(s));
            if (last) commit(a_free(k));
          }
        }
        if (!ok) break;
        if (lead) commit(acc_full(buf));
        if (last) ++block;
      }
      if (!ok) {                                             // products in flight end before TMEM is given back
        if (lead) commit(acc_full(i & 1));
        drain_wait(acc_full(i & 1), (i >> 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 2 && rank == 1) {
    // Tells CTA 0 of this CTA's rows.  From a warp of its own: a release at cluster scope waits for what its
    // warp has in flight, and the row warps have the next chunks' copies (1200 cycles a chunk).
    if (lane == 0) {
      uint32_t block = 0;
      bool ok = true;
      for (int t = t0; t < t1 && ok; t = (t / cols + 1) * cols, ++block)
        for (int k = 0; k < kChunks && ok; ++k) {
          ok = mbar_wait(a_full(k), block & 1, wc);
          if (ok) mbar_arrive_cluster(a_full(k), 0);
        }
    }
    __syncwarp();
  } else if (warp >= kRowWarp0) {
    // ------------------------------------------------------------------ rows
    const int rt = threadIdx.x - 32 * kRowWarp0;             // 0..127
    const int sub = rt & 7;                                  // 16-byte piece of a row's chunk
    uint32_t block = 0;
    for (int t = t0; t < t1; t = (t / cols + 1) * cols, ++block) {
      const int m0 = (t / cols) * tile_rows + static_cast<int>(rank) * BM;
      // a thread's rows are 16 i + rt / 8; the rows past the last are zeros, not read (one row read for all of
      // them is 128 reads of the same lines, 6 us)
      long long row[8];
      bool oob = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = m0 + 16 * i + (rt >> 3);
        long long slot = r < p.tokens ? __ldg(p.kv_indices + r) : 0;
        if (slot < 0 || slot >= p.num_slots) { oob = true; slot = 0; }
        row[i] = r < p.tokens ? slot * (kFp8 ? kRow : 2 * kRow) : -1;
      }
      if (oob) record_status(p.status, MLA_ERR_INDEX_OOB);
      bool ok = true;
      // chunk k's place is free once the block before has used it
      auto wait_free = [&](int k) {
        if (block == 0 || !ok) return;
        ok = __all_sync(0xffffffffu, mbar_wait(a_free(k), (block - 1) & 1, wc));
      };
      // 16 bytes a lane and row: an eighth of a bf16 chunk's row; a quarter of an FP8 chunk's, for half the rows
      // each of the chunk's two lane groups (rows 16 i + rt / 8 with i even for lanes of sub < 4, odd for others)
      auto load = [&](int k) {
        const uint32_t chunk = base + k * (BM * 128);
        if constexpr (kFp8) {
          // the codes wait in the chunk's upper half, 64 bytes a row, until they are widened over it
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 16 * i + (rt >> 3);
            if ((i & 1) == (sub >> 2))
              cp_async16(chunk + BM * 64 + r * 64 + (sub & 3) * 16, p.kv_cache + max(row[i], 0ll) + k * 64 + (sub & 3) * 16,
                         row[i] >= 0);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 16 * i + (rt >> 3);
            cp_async16(chunk + r * 128 + ((sub ^ (r & 7)) << 4), p.kv_cache + max(row[i], 0ll) + k * 128 + sub * 16,
                       row[i] >= 0);
          }
        }
      };
      auto landed = [&](int k) {
        if constexpr (kFp8) {
          // each thread widens what it loaded itself, once all have taken theirs into registers
          uint8_t* chunk = smem + k * (BM * 128);
          uint4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 16 * (2 * i + (sub >> 2)) + (rt >> 3);
            x[i] = *reinterpret_cast<const uint4*>(chunk + BM * 64 + r * 64 + (sub & 3) * 16);
          }
          ok = !named_bar_or(1, 128, !ok);                   // (all four warps leave after the same block)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 16 * (2 * i + (sub >> 2)) + (rt >> 3), c = 2 * (sub & 3);
            *reinterpret_cast<uint4*>(chunk + r * 128 + ((c ^ (r & 7)) << 4)) =
                make_uint4(e4m3x2_to_bf16x2(x[i].x), e4m3x2_to_bf16x2(x[i].x >> 16), e4m3x2_to_bf16x2(x[i].y),
                           e4m3x2_to_bf16x2(x[i].y >> 16));
            *reinterpret_cast<uint4*>(chunk + r * 128 + (((c + 1) ^ (r & 7)) << 4)) =
                make_uint4(e4m3x2_to_bf16x2(x[i].z), e4m3x2_to_bf16x2(x[i].z >> 16), e4m3x2_to_bf16x2(x[i].w),
                           e4m3x2_to_bf16x2(x[i].w >> 16));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(a_full(k));
      };
      // four chunks on their way; the first block's all at once, as it has nothing to wait for
      auto run = [&](auto lag) {
        constexpr int kLag = decltype(lag)::value;
#pragma unroll 1                                               // (code run once comes slowly: the loop stays short)
        for (int k = 0; k < kChunks + kLag; ++k) {
          if (k < kChunks) wait_free(k);
          if (k < kChunks && ok) load(k);
          cp_async_commit();                                 // empty groups keep the count
          if (k >= kLag) {
            cp_async_wait<kLag>();
            landed(k - kLag);                                // (after a wait that gave up, of what is there)
          }
        }
      };
      if (block == 0) run(std::integral_constant<int, kChunks - 1>{});
      else run(std::integral_constant<int, 3>{});
      if (!ok) break;
      if (t % cols == 0) {                                   // the CTA with the block's first tile writes its rope keys
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = m0 + 16 * i + (rt >> 3);
          if (r >= p.tokens) continue;
          uint4* dst = reinterpret_cast<uint4*>(p.k_rope + static_cast<size_t>(r) * kRope) + sub;
          if constexpr (kFp8) {
            const uint2 c = __ldg(reinterpret_cast<const uint2*>(p.kv_cache + row[i] + kLatent) + sub);
            float scale = p.kv_scale;
            if constexpr (kRows) scale = row_scale(__ldg(p.kv_scales + row[i] / kRow));
            auto val = [&](uint32_t codes) {
              const float2 f = e4m3x2_value(codes);
              return pack_bf16x2(f.x * scale, f.y * scale);
            };
            *dst = make_uint4(val(c.x), val(c.x >> 16), val(c.y), val(c.y >> 16));
          } else {
            *dst = __ldg(reinterpret_cast<const uint4*>(p.kv_cache + row[i] + 2 * kLatent) + sub);
          }
        }
      }
    }
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - kEpiWarp0) >> 2;
    float scale = kForm == CacheForm::kScaled ? p.kv_scale : 1.f;
    // the output streams through L2 (__stcs); the weights, read by every block of rows, should stay
    const int mate = lane & 3;
    uint32_t i = 0;
    for (int t = t0; t < t1; ++t, ++i) {
      const int col = t % cols, h = (col % groups) * C::kHeads;
      const int r0 = (t / cols) * tile_rows + static_cast<int>(rank) * BM + 32 * q;
      const uint32_t buf = i & 1;
      if constexpr (kRows) {
        // a lane's accumulator row is a token: its scale, once a block of rows, while the products run
        if ((t == t0 || col == 0) && r0 + lane < p.tokens) {
          const int slot = __ldg(p.kv_indices + r0 + lane);
          scale = row_scale(__ldg(p.kv_scales + (slot >= 0 && static_cast<long long>(slot) < p.num_slots ? slot : 0)));
        }
      }
      if (!__all_sync(0xffffffffu, mbar_wait(acc_full(buf), (i >> 1) & 1, wc))) break;
      tc_fence_after();
      const int end = min((half + 1) * (NT / 2), (p.heads - h) * kNope);   // an odd last head: half a tile
#pragma unroll 1
      for (int c = half * (NT / 2); c < end; c += 32) {
        uint32_t a[16], b[16], w[16];
        const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + buf * NT + c;
        tmem_ld16(src, a);
        tmem_ld16(src + 16, b);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          w[e] = pack_bf16x2(__uint_as_float(a[2 * e]) * scale, __uint_as_float(a[2 * e + 1]) * scale);
          w[8 + e] = pack_bf16x2(__uint_as_float(b[2 * e]) * scale, __uint_as_float(b[2 * e + 1]) * scale);
        }
        // four lanes exchange blocks of 16 bytes, so that a store writes 64 bytes of a row
        transpose4_blocks<4>(w, lane);
        uint16_t* dst = (col < groups ? p.k_nope : p.v) +
                        (static_cast<size_t>(r0 + lane - mate) * p.heads + h + (c >> 7)) * kNope + (c & 127) + 8 * mate;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (r0 + lane - mate + x < p.tokens)
            __stcs(reinterpret_cast<uint4*>(dst + static_cast<size_t>(x) * p.heads * kNope),
                   make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        // (with release semantics it waited for the stores before it, about 4800 cycles a tile)
        if constexpr (kPair) mbar_arrive_leader_relaxed(acc_empty(buf));
        else mbar_arrive(acc_empty(buf));
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  if constexpr (kPair) {
    cluster_sync_all();                                     // no CTA leaves while the other signals it or uses its TMEM
    if (warp == 1) tmem_dealloc2(tmem, C::kTmemCols);
  } else {
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <CacheForm kForm, int NT, bool kPair>
int launch(const ExpandParams& p, const CUtensorMap (&tm)[2], int grid, cudaStream_t stream) {
  using C = Cfg<NT, kPair>;
  const auto kernel = &expand_kernel<kForm, NT, kPair>;
  if (!set_smem_limit(reinterpret_cast<const void*>(kernel), C::kSmemBytes)) return MLA_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C::kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kPair ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, tm[0], tm[1], p) != cudaSuccess) return MLA_ERR_CUDA;
  return cudaPeekAtLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace ex

// 256 rows x 256 columns on CTA pairs, or 128 x 128 on single CTAs where there
// are few tiles: the end of the schedule is finer then, and a pair's second half
// may have no rows.  us on pairs and single CTAs: 256 rows x 64 heads 10.1 and
// 8.7, 600 x 64 18.6 and 16.1, 1024 x 64 22.0 and 22.3, 1536 x 64 27.2 and 29.6,
// 1024 x 128 33.2 and 40.5; E4M3 rows 0.5 to 1 us in the pairs' favour beside that.
ExpandTiling expand_tiling(int tokens, int heads, int sms) {
  const long long blocks = (tokens + ex::BM - 1) / ex::BM;
  const long long groups = 2ll * ((heads + 1) / 2);
  if (blocks * groups < 4ll * sms) return {128, false};
  return {256, true};
}

int launch_expand(const ExpandParams& p, const CUtensorMap (&tm)[2], ExpandTiling tiling, int sms, CacheForm form,
                  cudaStream_t stream) {
  const int per = tiling.cols / kNope, rows = tiling.pair ? 2 * ex::BM : ex::BM;
  const long long tiles = (p.tokens + static_cast<long long>(rows) - 1) / rows * 2 * ((p.heads + per - 1) / per);
  if (tiles > 0x3FFFFFFFll) return MLA_ERR_UNSUPPORTED;
  const int workers = tiling.pair ? sms / 2 : sms;
  const int grid = static_cast<int>(tiles < workers ? tiles : workers) * (tiling.pair ? 2 : 1);
  auto go = [&](auto form_of) {
    constexpr CacheForm kForm = decltype(form_of)::value;
    return tiling.pair ? ex::launch<kForm, 256, true>(p, tm, grid, stream)
                       : ex::launch<kForm, 128, false>(p, tm, grid, stream);
  };
  if (form == CacheForm::kBf16) return go(std::integral_constant<CacheForm, CacheForm::kBf16>{});
  if (form == CacheForm::kScaled) return go(std::integral_constant<CacheForm, CacheForm::kScaled>{});
  return go(std::integral_constant<CacheForm, CacheForm::kRowScaled>{});
}

}  // namespace mla
