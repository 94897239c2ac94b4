// Absorbed MLA decode over an FP8 (E4M3) latent cache with a scale for every
// row (H = 16..128, step 16) on sm_103a.  ("MLA and torch.compile: v0.3's two
// sources", section "MLA: starting from a 439-line commit": the FP8 KV cache;
// "实现差距：MLA 与 DeepSeek V3", section 2.4: the latent and rope dot products
// summed and scaled, FA2-style online softmax, the latent rows reused as the
// values.)
//
// Row t has codes x_t and the scale r_t; the exponents carry the scale,
//   e_t = sm_scale log2(e) r_t (q . x_t) + log2 r_t,
// so that w_t = 2^(e_t - m) is the weight of the row's codes, w_t / r_t its
// share of the sum, and the reference m that of the weights which the 8-bit
// parts below have to hold.
//
// Both products are kind::f8f6f4 and take the codes as they lie in shared
// memory.  The query is two E4M3 parts, q 2^a = hi + lo / 32 (a puts the head's
// largest element into [128, 256)), stacked on M of A, in tensor memory: in each
// quadrant of 32 rows the hi parts of 16 heads and then their lo parts, so that
// the two of a head meet by a shuffle.
//   S[128 x 64 rows] = [hi; lo] X^T          16 K-steps from TMEM, 2 of the rope
// The weights are parts that add up in one accumulator.  A part leaves a rest
// below half its step, in the binade under that, and E5M2's steps go on down to
// 2^-16 where E4M3's end at 2^-9:
//   out bf16   2^7 for the reference, at most 431: E4M3 + E5M2, off by 2^-8 of the
//              weight, or 2^-14
//   out fp32   2^10, at most 3445: E5M2 + E4M3 + two of E5M2, off by 2^-16 of the
//              weight (rests 2^-3, 2^-8, 2^-12, 2^-16 of its binade), or 2^-17
//   O^T[512 dims x heads] += X^T W^T         4 blocks of 128 dims, 2 K-steps of
//                                            32 rows a part
// The sum l takes the weights unrounded, so what the second bounds leave out is
// lost: nothing beside the rows that set the reference, but half of the result
// where one row outweighs 2^16 others, each by 2^16.  So the reference also
// goes down: every thread adds up what its rows may have lost at most and the
// largest weights that it had since the last move, and once the former passes
// kEps of the latter and of the reference's own row, a tile that lies below the
// reference takes its place.  (O and l, in fp32, follow a factor of 2^24 upwards
// as they follow one downwards.)  What is lost is then at most 2 kEps of all
// weights, at any number of rows.  (With E4M3 + E4M3 at 2^5 and a reference that
// only went up, 16384 rows of scores N(0, 1) beside one that has 0.8 of the sum
// gave 0.07 off, and 65536 equal ones 0.4, by an emulation; what is measured now is
// a bf16 out's rounding, and 4e-5 for an fp32 out, which is the tensor core's cut
// of its sums.  Moves are few: 2 to 5 an item of 16384 rows with scores N(0, 1.7) to
// N(0, 5), and fewer since an item's first reference stands 3 above its first tile's
// maximum: 152 requests of 8192 rows, 128 heads, fp32 out, scores N(0, 1.7): 398 ->
// 384 us, and 390 with a reference that only went up.)
//
// A worker of 48 or more heads is two CTAs, and each takes half of the HEADS:
// all of the scores, the softmax and the output of a head are one CTA's, and
// nothing passes between the two.  Both gather every row, the second of them
// from L2.  (As a cluster that gathers half of the rows each and multicasts
// them, a gather of four rows took the TMA unit 47 cycles, and 40 of them a tile
// 1900; on its own one takes about 14.)
//
// What bounds it: the products of a tile are 18 of 34 cycles and 16 (fp32: 32)
// of 48 (they read shared memory at its full rate), 1400 cycles (fp32 2150),
// against 1600 for a tile's bytes at the measured bandwidth where one CTA has
// them, 800 where two do.  What is measured is 2000 to 2700 cycles a tile: a
// tile's place in shared memory, of which there are four, is taken for 2500
// cycles of gathers, 1000 of scores, 2500 (fp32 3800) of softmax and 1500 of
// sums.  So the softmax's chain is cut where it can be: two crews of warps have
// every second tile each; rows' numbers arrive with the scores; and O follows a
// moved reference by other warps' hands.  (Two crews instead of one that begins a
// tile's scores before the weights of the one before: 27.5 -> 25.6 us of 64
// requests of 512..4096 rows, 16 heads, bf16 out.  One warp that issues both
// products can keep A of a block's parts in the collector buffer, 35 cycles a
// product: 263 -> 256 us of 256 requests of 16..16384 rows, 128 heads, fp32 out,
// but 24.5 -> 25.6 us of the former, as it has more to wait for at a time.  Five
// places for tiles where they fit: 25.1 us.)
//
// With the kernels before and after, the former batch takes 24.5 us (2.6 TB/s; fp32
// out 27.9) and the latter 258 us (0.66 PFLOP/s of the formula's operations; bf16
// out 210; 64 heads 195).  What was tried above was timed before the reference went
// both ways: with that, and the weights of 2^7 and 2^10, they were 24.0 and 252 us,
// and 24.6 and 263 with 2^5 and 2^8 and a lag of 3.75.
//
// A kernel before this one splits each request's query into its parts, once for
// all items (in here a warp took 20000 cycles an item for it), in the order in
// which the lanes below read them, and this one is its programmatic dependent:
// only the warps that need the query wait for it.
//
// TMEM (512 columns): O^T [0, 256), the query [256, 384), two score buffers.
//
// Warps:
//   0-15   softmax, two crews.  A thread of a head's hi or lo part reads 32 rows'
//          scores, gives half of them to the thread of the other part and goes
//          on with 16 rows (at most 32 heads a CTA: quadrants 2 and 3 hold the
//          heads of 0 and 1 once more, and a thread has half as many)
//   16-23  the next item's query; O into new references' units; and the output
//   24     issuer of the scores     25  TMEM allocator, issuer of the weighted sums
//   26-29  gathers of the latents, an atom each: 16 of four rows a tile (a warp
//          takes some 60 cycles for each of a burst, so they are spread)
//   30     gathers of the rope keys
//   31     the numbers made of the rows' scales
#include "mla_device.cuh"
#include "mla_launch.h"

namespace mla {
namespace rows8 {

constexpr int T = 64;                                // rows of a tile
constexpr int kSoftWarps = 16, kQueryWarps = 8;
constexpr int kQueryWarp0 = 16, kQkWarp = 24, kPvWarp = 25, kLatentWarp0 = 26, kRopeWarp = 30, kScaleWarp = 31;
constexpr int kThreads = 32 * 32;
constexpr int kAtom = T * 128;                       // 64 rows x 128 dims
constexpr int kRopeOff = 4 * kAtom;
constexpr int kUnit = 4 * kAtom + T * 64;            // a tile: 36 KB
constexpr int kQr = 128 * 64;                        // rope query: [hi; lo] x 64 dims (64-byte swizzle)
constexpr int kPPair = 64 * 128;                     // two parts of the weights: 64 heads x (64 + 64) rows
constexpr int kImage = 2 * kRow;                     // bytes of a head's query: hi and lo codes
constexpr int kCrews = 2, kCrewWarps = kSoftWarps / kCrews;   // a crew has every second tile
constexpr int kScSlots = 4;                          // tiles whose rows' numbers are held
constexpr int kScSlot = 3 * T * 4;                   // factors, log2 of the scales, reciprocals
constexpr int kItemCache = 16;                       // this worker's first items, copied to shared memory
constexpr float kLoWeight = 1.f / 32.f;              // value of a query's lo part
constexpr float kLag = 1.75f;                        // weights are 2^(e - m + kTop) with e <= m + kLag
constexpr float kHead = 3.f, kHeadRoom = 0.125f;     // an item's first reference is that far above its first tile's maximum
constexpr float kDepth = 24.f;                       // the reference's deepest under its highest: less is nothing beside that
constexpr int kBarCrew0 = 1, kBarGather = 9;   // named barriers
constexpr int kTmO = 0, kTmQ = 256, kTmS = 384;
constexpr uint32_t kIdescQK = idesc_e4m3(128, T, false, false);

template <bool kFine, bool kFew>
struct Cfg {
  static constexpr int kPairs = kFine ? 2 : 1;       // pairs of weight parts
  static constexpr int kUnits = 4;
  static constexpr int kPSlots = 3;                  // tiles whose weights are held
  static constexpr int kGroups = kFew ? 2 : 4;       // of 16 heads
  static constexpr int kPBuf = kPairs * kPPair;
  static constexpr int kRows = kFew ? 8 : 16;        // rows of a tile that a softmax thread has
  static constexpr float kTop = kFine ? 10.f : 7.f;  // (the first two parts hold up to 2^11.75, or 2^8.75)
  static constexpr float kLost = kFine ? 0x1p-17f : 0x1p-14f;   // what a small weight loses at most
  static constexpr float kEps = kFine ? 0x1p-16f : 0x1p-9f;     // what all weights together may lose of their sum
  // a thread's share of that of the reference's own row (of weight 2^kTop; kCrews T / kRows threads have a head)
  static constexpr float kRoom = kEps * (kFine ? 1024.f : 128.f) * kRows / (kCrews * T);
  static constexpr int kOffQr = kUnits * kUnit;
  static constexpr int kOffP = kOffQr + kQr;
  static constexpr int kOffSc = kOffP + kPSlots * kPBuf;
  static constexpr int kOffRed = kOffSc + kScSlots * kScSlot;   // [kCrews][256] maxima, or sums
  static constexpr int kOffOwe = kOffRed + kCrews * 256 * 4;     // [kCrews][256] what may have been lost
  static constexpr int kOffBc = kOffOwe + kCrews * 256 * 4;      // [kUnits][64] a tile's rescaling factors
  static constexpr int kOffSum = kOffBc + kUnits * 64 * 4;      // [2][kCrews][64] an item's sums, for the output
  static constexpr int kOffRef = kOffSum + 2 * kCrews * 64 * 4; // [2][kCrews][64] and references
  static constexpr int kOffNow = kOffRef + 2 * kCrews * 64 * 4; // [64] the references as the last tile left them
  static constexpr int kOffHigh = kOffNow + 64 * 4;             // [64] the highest references of the item
  static constexpr int kOffSlots = kOffHigh + 64 * 4;           // [5][64] a tile's slots, for each gathering warp
  static constexpr int kOffBar = kOffSlots + 5 * T * 4;
  static constexpr int bFull = 0;                    // [kUnits] a tile's rows have landed
  static constexpr int bEmpty = bFull + kUnits;      // [kUnits]
  static constexpr int bQFull = bEmpty + kUnits;
  static constexpr int bQEmpty = bQFull + 1;
  static constexpr int bSFull = bQEmpty + 1;         // [2] a tile's scores, and its rows' numbers
  static constexpr int bSEmpty = bSFull + 2;         // [2]
  static constexpr int bPFull = bSEmpty + 2;         // [kPSlots]
  static constexpr int bVoted = bPFull + kPSlots;    // [kUnits] a tile's references are settled
  static constexpr int bFixed = bVoted + kUnits;     // [kUnits] and what has been added up is in their units
  static constexpr int bOFull = bFixed + kUnits;
  static constexpr int bSumFull = bOFull + 1;        // [2]
  static constexpr int bSumEmpty = bSumFull + 2;     // [2]
  static constexpr int bDrain = bSumEmpty + 2;
  static constexpr int kNumBars = bDrain + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffMoved = kOffMisc + 8;     // [kUnits][2] heads whose reference a tile moved
  static constexpr int kOffLast = kOffMoved + kUnits * 8;       // [kUnits] last armed use
  static constexpr int kOffItems = (kOffLast + 4 * kUnits + 15) / 16 * 16;
  static constexpr int kSmemBytes = kOffItems + 16 * kItemCache;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static_assert(kUnit % 1024 == 0 && kOffQr % 1024 == 0 && kOffP % 1024 == 0 && kOffBar % 8 == 0,
                "alignment");
};

__device__ __forceinline__ bool item_ok(const DecodeParams& p, int nnz, int b, int s, int e) {
  return b >= 0 && b < p.batch && 0 <= s && s < e && e <= nnz;
}
__device__ __forceinline__ bool item_in_request(const DecodeParams& p, int b, int s, int e) {
  const int lo = __ldg(p.kv_indptr + b), hi = __ldg(p.kv_indptr + b + 1);
  return lo <= s && e <= hi;
}

// ------------------------------------------------------------ query parts --
// One warp a head, eight heads a block: lane l has latent dims 16 l .. and rope
// dims 2 l ..; q' = q 2^a, hi = e4m3(q'), lo = e4m3(32 (q' - hi)).  A CTA's image is 36 pieces of 16 dims, each with the hi and then the lo
// codes of its heads; the block's eight heads of a piece go out together, 128
// bytes (one by one, half sectors, the ragged batch's took 20 us).  Bound: launch
// and a round trip, or for large batches HBM: 32768
// heads take 14.8 us (5.1 TB/s read and written).
constexpr int kPrepWarps = 8, kPrepThreads = 32 * kPrepWarps;
__global__ void __launch_bounds__(kPrepThreads) rows8_prep_kernel(const Fp8PrepParams p, int heads) {
  constexpr int kCodes = 2 * kRow / 16, kPitch = kPrepWarps + 1;               // (a piece of padding: bank conflicts)
  __shared__ uint4 stage[2][kCodes * kPitch];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, Hc = heads > 32 ? heads >> 1 : heads;
  griddep_wait();
  griddep_launch_dependents();
  uint4 v[2];
  uint32_t v_rope = 0;
  auto load = [&](int i) {
    const uint4* qn = reinterpret_cast<const uint4*>(p.q_nope + static_cast<size_t>(i) * kLatent) + 2 * lane;
    v[0] = __ldg(qn);
    v[1] = __ldg(qn + 1);
    v_rope = __ldg(reinterpret_cast<const uint32_t*>(p.q_rope + static_cast<size_t>(i) * kRope) + lane);
  };
  const int step = kPrepWarps * gridDim.x;           // (rows: a multiple of eight, of one CTA's image each)
  int i = blockIdx.x * kPrepWarps + warp, buf = 0;
  if (i < p.rows) load(i);
  for (; i < p.rows; i += step, buf ^= 1) {
    const uint32_t x[9] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w, v_rope};
    if (i + step < p.rows) load(i + step);
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 9; ++k)
      amax = max3(amax, fabsf(__uint_as_float(x[k] << 16)), fabsf(__uint_as_float(x[k] & 0xFFFF0000u)));
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    int a = 0;                                       // amax = m 2^e, m in [0.5, 1): a = 8 - e
    if (amax > 0.f && amax <= 3.0e38f) {
      int e;
      frexpf(amax, &e);
      a = min(126, max(-126, 8 - e));
    }
    const float up = ldexpf(1.f, a);
    uint32_t hi[9], lo[9];                           // two codes each
#pragma unroll
    for (int k = 0; k < 9; ++k) {
      const float u0 = __uint_as_float(x[k] << 16) * up, u1 = __uint_as_float(x[k] & 0xFFFF0000u) * up;
      hi[k] = e4m3x2(u0, u1);
      const float2 hv = e4m3x2_value(hi[k]);
      lo[k] = e4m3x2((u0 - hv.x) * 32.f, (u1 - hv.y) * 32.f);
    }
    auto piece = [](const uint32_t (&c)[9]) {
      return make_uint4(c[0] | c[1] << 16, c[2] | c[3] << 16, c[4] | c[5] << 16, c[6] | c[7] << 16);
    };
    uint4* at = stage[buf] + lane * 2 * kPitch + warp;
    at[0] = piece(hi);
    at[kPitch] = piece(lo);
    uint16_t* at_rope = reinterpret_cast<uint16_t*>(stage[buf] + (32 + (lane >> 3)) * 2 * kPitch + warp) + (lane & 7);
    at_rope[0] = static_cast<uint16_t>(hi[8]);
    at_rope[8 * kPitch] = static_cast<uint16_t>(lo[8]);
    if (lane == 0) p.fac[i] = ldexpf(1.f, -a);
    __syncthreads();                                 // (and the buffer of the round before has been read)
    const int i0 = i - warp, b = i0 / heads, h = i0 - b * heads, c = h >= Hc, hl = c ? h - Hc : h;
    uint4* img = reinterpret_cast<uint4*>(p.img + (static_cast<size_t>(b) * heads + c * Hc) * kImage) + hl;
#pragma unroll
    for (int j = threadIdx.x; j < kCodes * kPrepWarps; j += kPrepThreads) {
      const int row = j / kPrepWarps, k = j % kPrepWarps;
      img[row * Hc + k] = stage[buf][row * kPitch + k];
    }
  }
}

// kFew: at most 32 heads a CTA
template <bool kFine, bool kFew>
__global__ void __launch_bounds__(kThreads, 1)
    rows8_kernel(const __grid_constant__ CUtensorMap tm_lat, const __grid_constant__ CUtensorMap tm_rope,
                 const DecodeParams p, const Fp8Params p8) {
  using C = Cfg<kFine, kFew>;
  const float* __restrict__ kv_scales = p8.kv_scales;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int shift = p.heads > 32 ? 1 : 0;            // a worker's CTAs: two, or one that takes all heads
  const int cta = blockIdx.x & shift;                // which of them
  auto bar = [&](int i) -> uint32_t { return base + C::kOffBar + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  int* last_armed = reinterpret_cast<int*>(smem + C::kOffLast);
  const WaitCtx wc{abort_flag, p.status};
  const int w = blockIdx.x >> shift;
  const int Hc = p.heads >> shift;                   // this CTA's heads: [cta * Hc, (cta + 1) * Hc)

  // the items' loads, one behind another, while barriers and TMEM are set up
  const int nnz = __ldg(p.kv_indptr + p.batch);
  int it0, it1;
  plan_items(p, w, it0, it1);
  const int32_t* items = p.plan + p.items_off;
  int32_t* s_items = reinterpret_cast<int32_t*>(smem + C::kOffItems);
  if (warp == kQueryWarp0) {
    const int n_cached = min(max(it1 - it0, 0), kItemCache);
    for (int i = lane; i < 4 * n_cached; i += 32) s_items[i] = items[4 * it0 + i];
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kUnits; ++i) { mbar_init(bar(C::bFull + i), 1); mbar_init(bar(C::bEmpty + i), 1); }
    mbar_init(bar(C::bQFull), kQueryWarps);
    mbar_init(bar(C::bQEmpty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::bSFull + i), 2); mbar_init(bar(C::bSEmpty + i), kCrewWarps);
      mbar_init(bar(C::bSumFull + i), kCrews * C::kGroups); mbar_init(bar(C::bSumEmpty + i), kQueryWarps);
    }
    for (int i = 0; i < C::kPSlots; ++i) mbar_init(bar(C::bPFull + i), kCrewWarps);
    for (int i = 0; i < C::kUnits; ++i) { mbar_init(bar(C::bVoted + i), C::kGroups); mbar_init(bar(C::bFixed + i), kQueryWarps); }
    mbar_init(bar(C::bOFull), 1);
    mbar_init(bar(C::bDrain), 2);
    for (int i = 0; i < C::kUnits; ++i) last_armed[i] = -1;
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kPvWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == kLatentWarp0 && lane == 0) tma_prefetch_desc(&tm_lat);
  if (warp == kRopeWarp && lane == 0) tma_prefetch_desc(&tm_rope);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto item_w = [&](int it, int k) -> int {
    return it - it0 < kItemCache ? s_items[4 * (it - it0) + k] : items[4 * it + k];
  };
  griddep_launch_dependents();
  bool aborted = false;                              // of the softmax and query warps

  if (warp == kScaleWarp) {
    // --------------------------------------------------- the rows' scales
    // Lane l has rows l and 32 + l of a tile.  Slots are loaded two tiles ahead
    // and scales one (a random 4 bytes from memory), over all items.
    int it = it0, s = 0, n = 0, t0 = 0;
    auto next_slots = [&](int (&slot)[2]) -> bool {
      while (t0 >= n) {                              // the next usable item
        if (it >= it1) return false;
        const int b = item_w(it, 0), s0 = item_w(it, 1), e = item_w(it, 2);
        ++it;
        if (!item_ok(p, nnz, b, s0, e)) {
          if (lane == 0 && cta == 0) record_status(p.status, MLA_ERR_PLAN_MISMATCH);
          continue;
        }
        if (lane == 0 && cta == 0 && !item_in_request(p, b, s0, e)) record_status(p.status, MLA_ERR_PLAN_MISMATCH);
        s = s0;
        n = e - s0;
        t0 = 0;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) slot[i] = __ldg(p.kv_indices + s + min(t0 + lane + 32 * i, n - 1));
      t0 += T;
      return true;
    };
    auto load = [&](const int (&slot)[2], float (&r)[2]) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool in = slot[i] >= 0 && static_cast<long long>(slot[i]) < p.num_slots;
        if (!in) record_status(p.status, MLA_ERR_INDEX_OOB);
        r[i] = __ldg(kv_scales + (in ? slot[i] : 0));
      }
    };
    int slot[2] = {0, 0};
    float next[2] = {1.f, 1.f};
    bool more = next_slots(slot);
    if (more) load(slot, next);
    bool ahead = more && next_slots(slot);
    for (uint32_t g = 0; more; ++g) {
      const float r[2] = {row_scale(next[0]), row_scale(next[1])};
      more = ahead;
      if (more) {
        load(slot, next);
        ahead = next_slots(slot);
      }
      const float f[2] = {r[0] * p.scale_log2, r[1] * p.scale_log2};
      const float lg[2] = {__log2f(r[0]), __log2f(r[1])}, iv[2] = {__frcp_rn(r[0]), __frcp_rn(r[1])};
      // scores of tile g - 2 read: the weights of tile g - 4 have been made
      bool ok = true;
      if (lane == 0 && g >= 2) ok = mbar_wait(bar(C::bSEmpty + (g & 1)), ((g >> 1) - 1) & 1, wc);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      float* out = reinterpret_cast<float*>(smem + C::kOffSc + (g % kScSlots) * kScSlot);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        out[lane + 32 * i] = f[i];
        out[T + lane + 32 * i] = lg[i];
        out[2 * T + lane + 32 * i] = iv[i];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::bSFull + (g & 1)));
    }
  } else if (warp >= kLatentWarp0) {
    // ------------------------------------------------------------- gathers
    // A latent atom of the tile, or the rope keys, by 16 gathers of four rows.
    // The warp loads and checks the slots (a tile ahead; lane l has rows l and 32
    // + l) and leaves them in shared memory, one elected lane issues: the
    // operands of a gather are uniform registers, and lanes that issue with their
    // own make the compiler build them one lane after another (230 cycles each).
    // An out-of-range slot reads row 0 (the scales' warp records it), the ragged
    // tail repeats the last valid slot.
    const bool lead = elect_one();
    const int atom = warp - kLatentWarp0;
    const bool rope = warp == kRopeWarp;
    const int x = rope ? kLatent : 128 * atom;
    const uint32_t dst = base + (rope ? kRopeOff : atom * kAtom), step = rope ? 4 * 64 : 4 * 128;
    const CUtensorMap* map = rope ? &tm_rope : &tm_lat;
    int* slots = reinterpret_cast<int*>(smem + C::kOffSlots) + T * atom;
    const int4* quads = reinterpret_cast<const int4*>(slots);
    const uint64_t pol = l2_policy_evict_first();
    int it = it0, s = 0, n = 0, t0 = 0;
    auto next_item = [&]() {
      for (; it < it1; ++it) {
        const int b = item_w(it, 0), s0 = item_w(it, 1), e = item_w(it, 2);
        if (!item_ok(p, nnz, b, s0, e)) continue;
        s = s0;
        n = e - s0;
        return;
      }
    };
    int next[2] = {0, 0};
    auto load_slots = [&]() {
#pragma unroll
      for (int i = 0; i < 2; ++i) next[i] = __ldg(p.kv_indices + s + min(t0 + lane + 32 * i, n - 1));
    };
    next_item();
    if (it < it1) load_slots();
    uint32_t g = 0;
    while (it < it1) {
      __syncwarp();                                  // (the slots of the tile before have been read)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        slots[lane + 32 * i] = next[i] < 0 || static_cast<long long>(next[i]) >= p.num_slots ? 0 : next[i];
      t0 += T;
      if (t0 >= n) {
        ++it;
        next_item();
        t0 = 0;
      }
      if (it < it1) load_slots();
      const uint32_t slot = g % C::kUnits, use = g / C::kUnits;
      if (!__all_sync(0xffffffffu, use == 0 || mbar_wait(bar(C::bEmpty + slot), (use - 1) & 1, wc))) break;
      const uint32_t full = bar(C::bFull + slot), to = dst + slot * kUnit;
      if (lead) {
        if (atom == 0) {
          mbar_arrive_expect_tx(full, kUnit);
          last_armed[slot] = static_cast<int>(use);
        }
#pragma unroll
        for (int i = 0; i < T / 4; ++i) {
          const int4 y = quads[i];
          tma_gather4(to + i * step, map, x, y.x, y.y, y.z, y.w, full, pol);
        }
      }
      ++g;
    }
    __syncwarp();
    named_bar_sync(kBarGather, 5 * 32);
    if (atom == 0 && lane < C::kUnits) {             // no copy outlives the block
      const int u = last_armed[lane];
      if (u >= 0) drain_wait(bar(C::bFull + lane), u & 1);
    }
    __syncwarp();
  } else if (warp >= kQkWarp) {
    // -------------------------------------------------------------- products
    // The whole warp runs the loop and one elected lane issues, so that
    // descriptors and counters stay in uniform registers.
    const bool lead = elect_one();
    auto D = [](uint64_t d, uint32_t byte_off) -> uint64_t { return d + (byte_off >> 4); };
    const uint64_t dk = sdesc(base, 16, 1024), dv = sdesc(base, kAtom, 1024);
    const uint64_t dr = sdesc(base + kRopeOff, 16, 512, kLayoutSw64);
    const uint64_t dq = sdesc(base + C::kOffQr, 16, 512, kLayoutSw64);
    const uint64_t dp = sdesc(base + C::kOffP, 16, 1024);
    const int cols = (Hc + 15) & ~15;                // columns that hold heads
    const uint32_t idesc4 = idesc_e4m3(128, cols, true, false);
    const uint32_t idesc5 = idesc_f8(kFmtE4M3, kFmtE5M2, 128, cols, true, false);
    uint32_t g = 0, nitem = 0, slot = 0, lap = 0;
    bool ok = true;
    for (int it = it0; it < it1 && ok; ++it) {
      const int b = item_w(it, 0), s = item_w(it, 1), e = item_w(it, 2);
      if (!item_ok(p, nnz, b, s, e)) continue;
      const int nt = (e - s + T - 1) / T;
      if (warp == kQkWarp) ok = mbar_wait(bar(C::bQFull), nitem & 1, wc);
      for (int j = 0; j < nt && ok; ++j, ++g) {
        const uint32_t buf = g & 1;
        if (warp == kQkWarp) {
          ok = (g < 2 || mbar_wait(bar(C::bSEmpty + buf), ((g >> 1) - 1) & 1, wc)) && mbar_wait(bar(C::bFull + slot), lap, wc);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d_s = tmem + kTmS + buf * T;
          const uint64_t bk = D(dk, slot * kUnit), br = D(dr, slot * kUnit);
          if (lead) {
#pragma unroll
            for (int k = 0; k < 16; ++k)             // 512 latent dims, A from TMEM
              umma_ts_f8(d_s, tmem + kTmQ + 8 * k, D(bk, (k >> 2) * kAtom + (k & 3) * 32), kIdescQK, k != 0 ? 1u : 0u);
#pragma unroll
            for (int k = 0; k < 2; ++k) umma_ss_f8(d_s, D(dq, 32 * k), D(br, 32 * k), kIdescQK, 1u);
            umma_commit(bar(C::bSFull + buf));
            if (j == nt - 1) umma_commit(bar(C::bQEmpty));
          }
        } else {
          const uint32_t ps = g % C::kPSlots;
          ok = mbar_wait(bar(C::bFixed + slot), lap, wc) && mbar_wait(bar(C::bPFull + ps), (g / C::kPSlots) & 1, wc);
          if (!ok) break;
          tc_fence_after();
          const uint64_t av = D(dv, slot * kUnit), bp = D(dp, ps * C::kPBuf);
          if (lead) {
#pragma unroll
            for (int mb = 0; mb < 4; ++mb)
#pragma unroll
              for (int ks = 0; ks < 2; ++ks) {       // 32 rows
                const uint64_t a = D(av, mb * kAtom + 4096 * ks);
                const uint32_t d = tmem + kTmO + 64 * mb;
                umma_ss_f8(d, a, D(bp, 32 * ks), kFine ? idesc5 : idesc4, (j == 0 && ks == 0) ? 0u : 1u);
                umma_ss_f8(d, a, D(bp, 64 + 32 * ks), kFine ? idesc4 : idesc5, 1u);
                if constexpr (kFine) {
                  umma_ss_f8(d, a, D(bp, kPPair + 32 * ks), idesc5, 1u);
                  umma_ss_f8(d, a, D(bp, kPPair + 64 + 32 * ks), idesc5, 1u);
                }
              }
            umma_commit(bar(C::bEmpty + slot));
            if (j == nt - 1) umma_commit(bar(C::bOFull));
          }
        }
        if (++slot == static_cast<uint32_t>(C::kUnits)) {
          slot = 0;
          lap ^= 1;
        }
      }
      ++nitem;
    }
    if (lead) {
      umma_commit(bar(C::bDrain));
      drain_wait(bar(C::bDrain), 0);
    }
    __syncwarp();
  } else if (warp >= kQueryWarp0) {
    // ------------------------------------------- the items' queries and outputs
    // Query: of quadrant q of A, rows 0-15 are the hi parts of heads 16 q .. and rows
    // 16-31 their lo parts (kFew: of heads 16 (q % 2) ..); two warps share a
    // quadrant, each 256 latent and 32 rope dims of its rows.  Output: dims 32 q + lane of every block of 128, heads 32 half ..
    // of the CTA's (kFew: of blocks 2 half and 2 half + 1, all heads).
    const int q = warp & 3, half = (warp >> 2) & 1;
    const int row = 32 * q + lane, hl = 16 * (kFew ? q & 1 : q) + (lane & 15);
    const int h0 = kFew ? 0 : 32 * half;
    constexpr int kBlocks = kFew ? 2 : 4;            // of the output's 128 dims
    const int block0 = kFew ? 2 * half : 0;
    const bool lo = lane >= 16, head_ok = hl < Hc;
    auto wait = [&](uint32_t bb, uint32_t par) {
      if (!aborted && !__all_sync(0xffffffffu, mbar_wait(bb, par, wc))) aborted = true;
    };
    griddep_wait();                                  // the queries' parts come from the kernel before
    auto query = [&](int b, uint32_t nitem) {
      // 16 codes of a row are one 16-byte piece, and the pieces of all rows lie together
      const uint4* src = reinterpret_cast<const uint4*>(p8.img + (static_cast<size_t>(b) * p.heads + cta * Hc) * kImage) +
                         (lo ? Hc : 0) + hl;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      uint4 v[8], r[2];
      auto pieces = [&](int c) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = head_ok ? src[(16 * half + c + k) * 2 * Hc] : zero;
      };
      const uint32_t tq = tmem + (static_cast<uint32_t>(32 * q) << 16) + kTmQ + 64 * half;
      auto store = [&](int c) {
        if (aborted) return;
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
          const uint32_t w[16] = {v[k].x,     v[k].y,     v[k].z,     v[k].w,     v[k + 1].x, v[k + 1].y, v[k + 1].z, v[k + 1].w,
                                  v[k + 2].x, v[k + 2].y, v[k + 2].z, v[k + 2].w, v[k + 3].x, v[k + 3].y, v[k + 3].z, v[k + 3].w};
          tmem_st16(tq + 4 * (c + k), w);
        }
      };
#pragma unroll
      for (int k = 0; k < 2; ++k) r[k] = head_ok ? src[(32 + 2 * half + k) * 2 * Hc] : zero;
      pieces(0);
      if (nitem > 0) wait(bar(C::bQEmpty), (nitem - 1) & 1);
      tc_fence_after();
      store(0);
      pieces(8);
      store(8);
      if (!aborted) {
        tmem_wait_st();
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<uint4*>(smem + C::kOffQr + (row >> 3) * 512 + (row & 7) * 64 +
                                    (((2 * half + k) ^ ((row >> 1) & 3)) << 4)) = r[k];
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && !aborted) mbar_arrive(bar(C::bQFull));
    };
    auto output = [&](int b, int dest, uint32_t nitem, uint32_t last) {   // last: the crew of the item's last tile
      const bool part_ok = dest < p.max_partials;    // a device-only plan naming a partial past the workspace
      if (!part_ok && warp == kQueryWarp0 && lane == 0) record_status(p.status, MLA_ERR_PLAN_MISMATCH);
      wait(bar(C::bSumFull + (nitem & 1)), (nitem >> 1) & 1);
      const float* sums = reinterpret_cast<const float*>(smem + C::kOffSum) + 64 * kCrews * (nitem & 1) + h0 + lane;
      const float* refs = reinterpret_cast<const float*>(smem + C::kOffRef) + 64 * kCrews * (nitem & 1) + h0 + lane;
      const float ref = refs[64 * last];             // O's units (the other crew may have seen a higher one before)
      const float l = fmaf(sums[64 * (last ^ 1)], ex2_approx(refs[64 * (last ^ 1)] - ref), sums[64 * last]);
      const float inv = l > 0.f ? 1.f / l : 0.f;     // of head h0 + lane
      __syncwarp();
      if (lane == 0 && !aborted) mbar_arrive(bar(C::bSumEmpty + (nitem & 1)));
      const size_t row0 = static_cast<size_t>(dest < 0 ? b : dest) * p.heads + cta * Hc;
      if (q == 0 && (!kFew || half == 0) && h0 + lane < Hc && !aborted && part_ok) {
        const float lse = l > 0.f ? (ref + __log2f(l) - C::kTop) * 0.69314718055994531f : -INFINITY;
        if (dest >= 0) p.part_lse[row0 + h0 + lane] = lse;
        else if (p.lse) p.lse[row0 + h0 + lane] = lse;
      }
      wait(bar(C::bOFull), nitem & 1);
      tc_fence_after();
      if (!aborted && part_ok) {
        const size_t first = (row0 + h0) * kLatent + 128 * block0 + 32 * q + lane;
        const int n = min(max(Hc - h0, 0), 32);      // heads, a multiple of 8
        const uint32_t from = tmem + (static_cast<uint32_t>(32 * q) << 16) + kTmO + 64 * block0 + h0;
        // (a store's 32 lanes are a head's 128 bytes; the type is looked at once, not at every store)
        auto put = [&](auto* dst, auto as) {
#pragma unroll 1
          for (int c = 0; c < 2 * kBlocks; ++c) {    // block c / 2, 16 heads
            if (16 * (c & 1) >= n) continue;
            uint32_t o[16];
            tmem_ld16(from + 64 * (c >> 1) + 16 * (c & 1), o);
            tmem_wait_ld();
            auto* at = dst + 128 * (c >> 1) + 16 * (c & 1) * kLatent;
            auto eight = [&](int i0) {
              float v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                v[i] = __uint_as_float(o[i0 + i]) * __shfl_sync(0xffffffffu, inv, 16 * (c & 1) + i0 + i);
#pragma unroll
              for (int i = 0; i < 8; ++i) at[(i0 + i) * kLatent] = as(v[i]);
            };
            eight(0);
            if (16 * (c & 1) + 8 < n) eight(8);
          }
        };
        if (dest < 0 && p.out_bf16)
          put(static_cast<__nv_bfloat16*>(p.out) + first, [](float v) { return __float2bfloat16_rn(v); });
        else
          put((dest >= 0 ? p.part_o : static_cast<float*>(p.out)) + first, [](float v) { return v; });
      }
      tc_fence_before();                             // (the next item's first bFixed says that O has been read)
    };
    // O in the units of tile g's references, where those moved
    auto fix = [&](uint32_t g) {
      const uint32_t at = g % C::kUnits;
      wait(bar(C::bVoted + at), (g / C::kUnits) & 1);
      const uint32_t moved = reinterpret_cast<const volatile uint32_t*>(smem + C::kOffMoved)[2 * at + (kFew ? 0 : half)];
      if (moved && !aborted) {
        wait(bar(C::bEmpty + (g - 1) % C::kUnits), ((g - 1) / C::kUnits) & 1);   // the sums of the tiles before are done
        tc_fence_after();
        const float4* bc = reinterpret_cast<const float4*>(smem + C::kOffBc) + 16 * at + h0 / 4;
        const uint32_t to = tmem + (static_cast<uint32_t>(32 * q) << 16) + kTmO + 64 * block0 + h0;
        if (!aborted)
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {              // 8 heads
            if (((moved >> (8 * c)) & 0xffu) == 0) continue;
            uint32_t o[kBlocks][8];
#pragma unroll
            for (int mb = 0; mb < kBlocks; ++mb) tmem_ld8(to + 64 * mb + 8 * c, o[mb]);
            const float4 f0 = bc[2 * c], f1 = bc[2 * c + 1];
            const float2 f[4] = {f2_pack(f0.x, f0.y), f2_pack(f0.z, f0.w), f2_pack(f1.x, f1.y), f2_pack(f1.z, f1.w)};
            tmem_wait_ld();
#pragma unroll
            for (int mb = 0; mb < kBlocks; ++mb) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 v = f2_mul(f2_pack(__uint_as_float(o[mb][2 * i]), __uint_as_float(o[mb][2 * i + 1])), f[i]);
                o[mb][2 * i] = __float_as_uint(v.x);
                o[mb][2 * i + 1] = __float_as_uint(v.y);
              }
              tmem_st8(to + 64 * mb + 8 * c, o[mb]);
            }
          }
        tmem_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0 && !aborted) mbar_arrive(bar(C::bFixed + at));
    };
    uint32_t nitem = 0, g = 0;
    int it = it0;
    auto usable = [&](int i) { return item_ok(p, nnz, item_w(i, 0), item_w(i, 1), item_w(i, 2)); };
    while (it < it1 && !usable(it)) ++it;
    if (it < it1) query(item_w(it, 0), 0);
    while (it < it1) {
      const int b = item_w(it, 0), dest = item_w(it, 3);
      for (int left = (item_w(it, 2) - item_w(it, 1) + T - 1) / T; left > 1; --left) fix(g++);
      do ++it;
      while (it < it1 && !usable(it));
      if (it < it1) query(item_w(it, 0), nitem + 1);
      fix(g++);
      output(b, dest, nitem++, (g - 1) & 1);
    }
  } else {
    // ----------------------------------------------------------------- softmax
    // Two crews, a tile each in turn: a tile is a chain of waits and exchanges,
    // and two of them at once fill each other's.  What passes from a tile to the
    // next is the heads' references.  A group of 16 heads is a quadrant's, and goes
    // on by itself; with kFew quadrants 2 and 3 hold the heads of 0 and 1 once more,
    // and their warps take half of the rows.
    constexpr int kRows = C::kRows, kShare = T / kRows, kHeads = 16 * C::kGroups;  // kShare threads have a head
    constexpr int kMeet = 32 * kCrewWarps / C::kGroups;                            // threads of a group
    const int q = warp & 3, crew = warp >> 3, th = (warp >> 2) & 1, part = lane >> 4;
    const int group = kFew ? q & 1 : q;
    const int hl = 16 * group + (lane & 15);         // head of this CTA
    const int share = kFew ? 4 * th + 2 * (q >> 1) + part : 2 * th + part;         // which kRows rows of a tile
    const bool first = th == 0 && (!kFew || q < 2);  // the warp that speaks for its group (lanes 0-15: share 0)
    const int meet = kBarCrew0 + C::kGroups * crew + group;
    const uint32_t quad = static_cast<uint32_t>(32 * q) << 16;
    float* red = reinterpret_cast<float*>(smem + C::kOffRed) + 256 * crew;
    float* owe = reinterpret_cast<float*>(smem + C::kOffOwe) + 256 * crew;
    volatile float* now = reinterpret_cast<volatile float*>(smem + C::kOffNow);
    volatile float* high = reinterpret_cast<volatile float*>(smem + C::kOffHigh);
    volatile uint16_t* moved_of = reinterpret_cast<volatile uint16_t*>(smem + C::kOffMoved);   // heads to rescale
    auto wait = [&](uint32_t bb, uint32_t par) {     // (every lane for itself: a third of the time of one for all)
      if (!aborted && !__all_sync(0xffffffffu, mbar_wait(bb, par, wc))) aborted = true;
    };
    griddep_wait();                                  // the factors come from the kernel before
    // 2^-a of this head in the next usable item from `it` on, loaded while the item before is worked on
    auto factor = [&](int it) -> float {
      for (; it < it1; ++it) {
        const int b = item_w(it, 0);
        if (item_ok(p, nnz, b, item_w(it, 1), item_w(it, 2)))
          return hl < Hc ? p8.fac[static_cast<size_t>(b) * p.heads + cta * Hc + hl] : 1.f;
      }
      return 1.f;
    };
    const float w_own = part == 0 ? 1.f : kLoWeight, w_other = part == 0 ? kLoWeight : 1.f;
    float fac_next = factor(it0);
    uint32_t g0 = 0, nitem = 0;                      // the item's first tile
    for (int it = it0; it < it1; ++it) {
      const int b = item_w(it, 0), s = item_w(it, 1), e = item_w(it, 2);
      if (!item_ok(p, nnz, b, s, e)) continue;
      const int n = e - s, nt = (n + T - 1) / T;
      const float fac = fac_next;
      fac_next = factor(it + 1);
      float l_sum = 0.f, m_own = -INFINITY;          // this thread's sum, in the units of that reference
      float over = 0.f;                              // by how much its rows since then may have lost too much
      for (int j = (g0 ^ crew) & 1; j < nt; j += kCrews) {
        const uint32_t g = g0 + j;
        // Scores, from TMEM: of 2 kRows rows the thread of the hi part goes on with the first half and gives the
        // second to that of the lo part, 16 lanes on, and gets the lo part's share of its own.
        uint32_t v0[kRows], v1[kRows];
        wait(bar(C::bSFull + (g & 1)), (g >> 1) & 1);
        if (!aborted) {
          tc_fence_after();
          const uint32_t ts = tmem + quad + kTmS + T * (g & 1) + kRows * (share - part);
          if constexpr (kFew) {
            tmem_ld8(ts, v0);
            tmem_ld8(ts + 8, v1);
          } else {
            tmem_ld16(ts, v0);
            tmem_ld16(ts + 16, v1);
          }
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < kRows; ++i) v0[i] = v1[i] = 0;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !aborted) mbar_arrive(bar(C::bSEmpty + (g & 1)));
        // the exponents and their largest
        float2 x[kRows / 2];
        const float4* sc = reinterpret_cast<const float4*>(smem + C::kOffSc + (g % kScSlots) * kScSlot) + kRows / 4 * share;
        const float2 f_own = f2_pack(fac * w_own, fac * w_own), f_other = f2_pack(fac * w_other, fac * w_other);
        auto score = [&](int i) -> float2 {          // rows i and i + 1
          auto own = [&](int k) { return __uint_as_float(part ? v1[k] : v0[k]); };
          auto other = [&](int k) { return __shfl_xor_sync(0xffffffffu, __uint_as_float(part ? v0[k] : v1[k]), 16); };
          const float a = own(i), b = own(i + 1), c = other(i), d = other(i + 1);
          return f2_fma(f2_pack(c, d), f_other, f2_mul(f2_pack(a, b), f_own));
        };
#pragma unroll
        for (int k = 0; k < kRows / 4; ++k) {
          const float4 f = sc[k], lg = sc[T / 4 + k];
          x[2 * k] = f2_fma(score(4 * k), f2_pack(f.x, f.y), f2_pack(lg.x, lg.y));
          x[2 * k + 1] = f2_fma(score(4 * k + 2), f2_pack(f.z, f.w), f2_pack(lg.z, lg.w));
        }
        const int nvalid = n - j * T - kRows * share;
        if (nvalid < kRows) {
#pragma unroll
          for (int i = 0; i < kRows / 2; ++i) {
            if (2 * i >= nvalid) x[i].x = -INFINITY;
            if (2 * i + 1 >= nvalid) x[i].y = -INFINITY;
          }
        }
        float mx = fmaxf(x[0].x, x[0].y);
#pragma unroll
        for (int i = 1; i < kRows / 2; ++i) mx = max3(mx, x[i].x, x[i].y);
        // The references, as the tile before left them.  (This one's are written after its threads have met, and so
        // after the other crew's have read theirs: its own tile before this one waited for that.)
        if (g > 0) wait(bar(C::bVoted + (g - 1) % C::kUnits), ((g - 1) / C::kUnits) & 1);
        const float m_old = j > 0 ? now[hl] : -INFINITY;
        float m_ref = m_old;
        uint32_t which = 0;                          // heads whose O has to follow
        if (named_bar_or(meet, kMeet, j == 0 || mx > m_old + kLag || over > 0.f)) {   // some head's reference may move
          red[share * kHeads + hl] = mx;             // (the last maxima there have been read: all have met since)
          owe[share * kHeads + hl] = over;
          named_bar_sync(meet, kMeet);
          float mt = mx, sum = 0.f;
#pragma unroll
          for (int i = 0; i < kShare; i += 2) {
            mt = max3(mt, red[i * kHeads + hl], red[(i + 1) * kHeads + hl]);
            sum += owe[i * kHeads + hl] + owe[(i + 1) * kHeads + hl];
          }
          over = sum * (1.f / kShare);               // (the crew's threads of a head go on alike)
          if (mt > m_old + kLag) {
            m_ref = j == 0 ? mt + kHead : mt;
          } else if (sum > 0.f && mt < m_old - 1.f) {
            m_ref = fmaxf(mt, high[hl] - kDepth);
            over = -C::kRoom;
          }
          if (first) {
            const float alpha = m_ref == m_old ? 1.f : ex2_approx(m_old - m_ref);
            if (part == 0) {
              reinterpret_cast<float*>(smem + C::kOffBc)[64 * (g % C::kUnits) + hl] = alpha;
              now[hl] = m_ref;
              if (j == 0 || m_ref > m_old) high[hl] = j == 0 ? m_ref : fmaxf(high[hl], m_ref);   // (read above only where it is not written)
            }
            which = __ballot_sync(0xffffffffu, part == 0 && alpha != 1.f && hl < Hc);
          }
        }
        if (first) {
          if (lane == 0) moved_of[4 * (g % C::kUnits) + group] = static_cast<uint16_t>(j > 0 ? which : 0);
          __syncwarp();
          if (lane == 0 && !aborted) mbar_arrive(bar(C::bVoted + g % C::kUnits));
        }
        if (m_ref != m_own) {
          l_sum *= ex2_approx(m_own - m_ref);
          m_own = m_ref;
          over = j < kCrews ? -C::kRoom * kHeadRoom : -C::kRoom;
        }
        const float most = ex2_approx(mx - m_ref + C::kTop);         // this thread's largest weight
        over += fmaf(-C::kEps, most, kRows * fminf(C::kLost, most));
        // weights and their parts
        uint32_t w0[kRows / 4], w1[kRows / 4], w2[kRows / 4], w3[kRows / 4];
        const float2 shift = f2_pack(C::kTop - m_ref, C::kTop - m_ref);
        float2 l2 = f2_pack(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kRows / 4; ++k) {
          const float4 iv = sc[2 * T / 4 + k];
          uint32_t c0[2], c1[2], c2[2], c3[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 e2 = f2_add(x[2 * k + i], shift);
            float2 r = f2_pack(ex2_approx(e2.x), ex2_approx(e2.y));
            l2 = f2_fma(r, i ? f2_pack(iv.z, iv.w) : f2_pack(iv.x, iv.y), l2);
            if constexpr (kFine) {
              const float2 minus = f2_pack(-1.f, -1.f);
              c0[i] = e5m2x2(r.x, r.y);
              r = f2_fma(e5m2x2_value(c0[i]), minus, r);   // (exact, like the next two)
              c1[i] = e4m3x2(r.x, r.y);
              r = f2_fma(e4m3x2_value(c1[i]), minus, r);
              c2[i] = e5m2x2(r.x, r.y);
              r = f2_fma(e5m2x2_value(c2[i]), minus, r);
              c3[i] = e5m2x2(r.x, r.y);
            } else {
              e4m3_e5m2_split(r.x, r.y, c0[i], c1[i]);
            }
          }
          w0[k] = c0[0] | (c0[1] << 16);
          w1[k] = c1[0] | (c1[1] << 16);
          if constexpr (kFine) {
            w2[k] = c2[0] | (c2[1] << 16);
            w3[k] = c3[0] | (c3[1] << 16);
          }
        }
        l_sum += l2.x + l2.y;
        const uint32_t ps = g % C::kPSlots;
        if (g >= C::kPSlots)                         // the sum that used these weights' place
          wait(bar(C::bEmpty + (g - C::kPSlots) % C::kUnits), ((g - C::kPSlots) / C::kUnits) & 1);
        if (!aborted) {
          // byte kRows share of the head's 64 (hi), then the same of the lo part: chunks c at c ^ (head mod 8)
          uint8_t* row = smem + C::kOffP + ps * C::kPBuf + hl * 128 + (kRows * share & 15);
          const int c = kRows * share >> 4, at = (c ^ (hl & 7)) << 4, at_lo = ((4 + c) ^ (hl & 7)) << 4;
          auto put = [&](int to, const uint32_t (&v)[kRows / 4]) {
            if constexpr (kFew) *reinterpret_cast<uint2*>(row + to) = make_uint2(v[0], v[1]);
            else *reinterpret_cast<uint4*>(row + to) = make_uint4(v[0], v[1], v[2], v[3]);
          };
          put(at, w0);
          put(at_lo, w1);
          if constexpr (kFine) {
            put(kPPair + at, w2);
            put(kPPair + at_lo, w3);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !aborted) mbar_arrive(bar(C::bPFull + ps));
      }
      g0 += nt;
      // what the output needs: each crew's sums, in the units of its last reference
      if (nitem >= 2) wait(bar(C::bSumEmpty + (nitem & 1)), ((nitem >> 1) - 1) & 1);
      named_bar_sync(meet, kMeet);
      red[share * kHeads + hl] = l_sum;
      named_bar_sync(meet, kMeet);
      if (first) {
        float l = 0.f;
#pragma unroll
        for (int i = 0; i < kShare; ++i) l += red[i * kHeads + hl];
        if (part == 0) {
          reinterpret_cast<float*>(smem + C::kOffSum)[64 * (kCrews * (nitem & 1) + crew) + hl] = l;
          reinterpret_cast<float*>(smem + C::kOffRef)[64 * (kCrews * (nitem & 1) + crew) + hl] = m_own;
        }
        __syncwarp();
        if (lane == 0 && !aborted) mbar_arrive(bar(C::bSumFull + (nitem & 1)));
      }
      ++nitem;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kPvWarp) tmem_dealloc(tmem, 512);
}

template <typename Kernel, typename... Args>
int launch_after(Kernel* kernel, int grid, int threads, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return MLA_ERR_CUDA;
  return cudaPeekAtLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace rows8

int launch_rows8(const CUtensorMap& tm_lat, const CUtensorMap& tm_rope, const DecodeParams& p, const Fp8Params& p8,
                 const Fp8PrepParams& pp, int workers, cudaStream_t stream) {
  if (p.heads < 16 || p.heads > 128 || p.heads % 16 != 0) return MLA_ERR_UNSUPPORTED;
  const int ctas = p.heads > 32 ? 2 * workers : workers;
  const bool few = p.heads <= 64;                    // heads of a CTA <= 32
  const auto kernel = p.out_bf16 ? (few ? &rows8::rows8_kernel<false, true> : &rows8::rows8_kernel<false, false>)
                                 : (few ? &rows8::rows8_kernel<true, true> : &rows8::rows8_kernel<true, false>);
  const int smem = p.out_bf16 ? (few ? rows8::Cfg<false, true>::kSmemBytes : rows8::Cfg<false, false>::kSmemBytes)
                              : (few ? rows8::Cfg<true, true>::kSmemBytes : rows8::Cfg<true, false>::kSmemBytes);
  if (!set_smem_limit(reinterpret_cast<const void*>(kernel), smem)) return MLA_ERR_CUDA;
  // as many blocks as are resident at once (a block for every eight heads: 260.6 us of the ragged batch, not 256.6)
  const int blocks = (pp.rows + rows8::kPrepWarps - 1) / rows8::kPrepWarps, held = 4 * ctas;
  const int st = rows8::launch_after(&rows8::rows8_prep_kernel, blocks < held ? blocks : held, rows8::kPrepThreads, 0,
                                     stream, pp, p.heads);
  if (st != MLA_OK) return st;
  return rows8::launch_after(kernel, ctas, rows8::kThreads, smem, stream, tm_lat, tm_rope, p, p8);
}

}  // namespace mla
