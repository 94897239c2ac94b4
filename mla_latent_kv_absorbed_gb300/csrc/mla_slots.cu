// What happens to a batch's rows between two steps, over a page-size-1 cache
// ("Attention backends", paragraph "Paged, ragged batches": the rows of request
// b are kv_indices[kv_indptr[b] .. kv_indptr[b+1])): requests forked, freed and
// cut to their accepted drafts, rows copied, and a pool made contiguous.  All of
// it is lists of 4-byte slot numbers and whole rows; nothing comes back to the
// host, so that a captured step can hold it.
//
// A set of slots is a bitmap.  Set bits come back as an ascending list by a
// count and a scan of the words, in one cluster of CTAs that hand their counts
// around through distributed shared memory: the order does not hang on which
// thread came first.
#include "mla_device.cuh"
#include "mla_launch.h"
#include "mla_serving.h"

namespace mla {
namespace {

constexpr int kListThreads = 256;
// 256 requests' lists (freed slots of 2^20) with 4, 8 and 16 CTAs that scan: 25.4, 19.3 and 17.0 us; a pool of 65536
// slots compacted: 56.8, 55.5 and 54.7.  (Sixteen are more than fit everywhere: a cluster may be smaller.)
constexpr int kScanThreads = 1024, kScanCtas = 16;
constexpr long long kBulkRows = 8192;              // (row, layer) pairs from which on rows go by bulk copies
constexpr int kMoveThreads = 288;                  // 4 rows of 72 pieces of 16 bytes, or 8 of 36

template <typename Kernel, typename... Args>
int launch_after(Kernel* kernel, dim3 grid, int threads, int cluster, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return MLA_ERR_CUDA;
  return cudaPeekAtLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

__device__ __forceinline__ void set_bit(uint32_t* bits, int slot) { atomicOr(bits + (slot >> 5), 1u << (slot & 31)); }

// ---------------------------------------------------------------- requests --
// The rows of an old request that its successors keep: the first `base`, then
// the drafts of its path.
struct Kept {
  int start, rows, base, count;
};
__device__ __forceinline__ int sat_add(int a, int b) {      // of numbers that are not negative
  const unsigned s = static_cast<unsigned>(a) + static_cast<unsigned>(b);
  return s > 0x7FFFFFFFu ? 0x7FFFFFFF : static_cast<int>(s);
}
__device__ __forceinline__ Kept kept_of(const RepackParams& p, int src, bool report) {
  if (src < 0 || src >= p.batch) {
    if (report && src != -1) record_status(p.status, MLA_ERR_PLAN_MISMATCH);
    return {0, 0, 0, 0};
  }
  const long long lo = __ldg(p.indptr + src), hi = __ldg(p.indptr + src + 1);
  const int a = p.path ? __ldg(p.accepted + src) : 0;      // (at once with the others)
  const long long s = min(max(lo, 0ll), p.entries), e = min(max(hi, s), p.entries);
  const int n = static_cast<int>(e - s);
  bool bad = lo != s || hi != e;
  Kept k{static_cast<int>(s), n, n, n};
  if (p.path) {
    if (n >= p.width) {
      const int take = min(max(a, 0), p.width);
      if (report && a != take) record_status(p.status, MLA_ERR_TREE);
      k.base = n - p.width;
      k.count = k.base + take;
    } else {
      bad = true;                                  // fewer rows than drafts: kept as they are
    }
  }
  if (report && bad) record_status(p.status, MLA_ERR_PLAN_MISMATCH);
  return k;
}

// The kernels below go by entries, not by requests (a long request would keep
// one block busy alone): a block takes kChunk of them, a thread kDeep in a row,
// and finds out itself whose they are, from the requests' ends in shared memory,
// 256 requests at a time.  Bound: the launches and four or five dependent loads
// each (request, list, entry, set of slots).
constexpr int kDeep = 8, kChunk = kListThreads * kDeep, kWindow = kListThreads;

// The first of n ascending ends that is past `at` (n: none).
__device__ __forceinline__ int first_past(const int* ends, int n, long long at) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > at) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Marks the slots that requests give up: all of them where no new request
// continues it, else those of the drafts off its path.  Another request may hold
// them too (a shared prefix): the lists' kernel takes those back.
__global__ void __launch_bounds__(kListThreads) repack_mark_kernel(const RepackParams p) {
  __shared__ uint32_t goes_on[(kMaxRequests + 31) / 32];
  __shared__ Kept rows_of[kWindow];
  __shared__ unsigned long long on_path[kWindow];    // a request's accepted drafts
  __shared__ int ends[kWindow];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  const long long lo = static_cast<long long>(blockIdx.x) * kChunk, hi = min(lo + kChunk, p.entries);
  const long long mine = lo + kDeep * tid;
  int slot[kDeep];
#pragma unroll
  for (int d = 0; d < kDeep; ++d) slot[d] = mine + d < hi ? __ldg(p.indices + mine + d) : 0;
  int source = tid < p.new_batch ? __ldg(p.sources + tid) : -1;
  // the window of the block's first entry: lists ascend, so the last that starts at or before it
  int r0 = 0;
  if (p.batch > kWindow) {
    int top = p.batch - 1;
    while (r0 < top) {
      const int mid = (r0 + top + 1) >> 1;
      if (__ldg(p.indptr + mid) <= lo) r0 = mid;
      else top = mid - 1;
    }
  }
  for (bool begun = false; r0 < p.batch; r0 += kWindow, begun = true) {
    const int n = min(kWindow, p.batch - r0);
    Kept k{0, 0, 0, 0};
    if (tid < n) k = kept_of(p, r0 + tid, false);
    if (!begun) {                                    // (while those loads are on their way)
      for (int i = tid; i < (p.batch + 31) / 32; i += kListThreads) goes_on[i] = 0;
      __syncthreads();
      for (int i = tid; i < p.new_batch; i += kListThreads) {
        if (i != tid) source = __ldg(p.sources + i);
        if (source >= 0 && source < p.batch) atomicOr(goes_on + (source >> 5), 1u << (source & 31));
      }
    }
    unsigned long long path = 0;
    if (k.base < k.rows && k.start + k.rows > lo && k.start + k.base < hi) {
      const int32_t* steps = p.path + static_cast<long long>(r0 + tid) * p.width;
#pragma unroll 8
      for (int i = 0; i < k.count - k.base; ++i) path |= 1ull << min(max(__ldg(steps + i), 0), p.width - 1);
    }
    __syncthreads();                                 // (the window before has been used; goes_on is made)
    on_path[tid] = path;
    rows_of[tid] = k;
    ends[tid] = k.start + k.rows;
    __syncthreads();
    if (rows_of[0].start >= hi) break;
    int a = first_past(ends, n, mine);
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const long long at = mine + d;
      if (at >= hi) break;
      while (a < n && ends[a] <= at) ++a;
      if (a >= n || at < rows_of[a].start) continue; // another window's, or nobody's
      const Kept& m = rows_of[a];
      const int o = r0 + a, step = static_cast<int>(at) - m.start - m.base;
      if ((goes_on[o >> 5] >> (o & 31) & 1) && (step < 0 || (on_path[a] >> step & 1))) continue;
      if (slot[d] >= 0 && slot[d] < p.num_slots) set_bit(p.bits, slot[d]);
      else record_status(p.status, MLA_ERR_INDEX_OOB);
    }
  }
}

// The new lists.  The lengths of the new requests are added up, a window at a
// time, until the block's entries are passed.
__global__ void __launch_bounds__(kListThreads) repack_lists_kernel(const RepackParams p) {
  __shared__ int ends[kWindow];                      // in the new lists, from the window's first on
  __shared__ Kept rows_of[kWindow];
  __shared__ int src_of[kWindow], warp_sums[kWindow / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // behind the marking kernel the inputs are there already: it started after whatever made them
  bool waited = !p.marked;
  if (waited) griddep_wait();
  griddep_launch_dependents();
  const long long lo = static_cast<long long>(blockIdx.x) * kChunk, hi = min(lo + kChunk, p.capacity);
  const long long mine = lo + kDeep * tid;
  long long before = 0;                              // entries of the windows before
  for (int r0 = 0; r0 < max(p.new_batch, 1); r0 += kWindow) {
    const int r = r0 + tid;
    const int src = r < p.new_batch ? __ldg(p.sources + r) : -1;
    const Kept k = kept_of(p, src, blockIdx.x == 0 && r < p.new_batch);
    // (256 forks of 2^31 entries pass 32 bits: past the capacity, sums are only held above it)
    int upto = k.count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto = sat_add(upto, y);
    }
    if (r0 > 0) __syncthreads();                     // the window before has been used
    if (lane == 31) warp_sums[warp] = upto;
    __syncthreads();
    for (int i = 0; i < warp; ++i) upto = sat_add(upto, warp_sums[i]);
    ends[tid] = upto;
    rows_of[tid] = k;
    src_of[tid] = src;
    __syncthreads();
    if (!waited) {
      griddep_wait();
      waited = true;
    }
    const long long total = ends[kWindow - 1];
    if (blockIdx.x == 0) {
      if (r < p.new_batch) p.new_indptr[r + 1] = static_cast<int>(min(before + upto, p.capacity));
      if (r == 0) p.new_indptr[0] = 0;
      if (tid == 0 && before + total > p.capacity) record_status(p.status, MLA_ERR_WORKSPACE);
    } else if (before >= hi) {
      break;
    }
    if (before + total > lo && before < hi) {
      int slot[kDeep];
      int a = first_past(ends, kWindow, mine - before);
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        const long long in = mine + d - before;
        slot[d] = -1;
        if (mine + d >= hi || in < 0 || in >= total) continue;
        while (ends[a] <= in) ++a;
        const Kept& m = rows_of[a];
        int at = static_cast<int>(in) - (a ? ends[a - 1] : 0);
        if (at >= m.base) {
          const int step = __ldg(p.path + static_cast<long long>(src_of[a]) * p.width + at - m.base);
          const int ok = min(max(step, 0), p.width - 1);
          if (step != ok) record_status(p.status, MLA_ERR_TREE);
          at = m.base + ok;
        }
        slot[d] = __ldg(p.indices + m.start + at);
      }
      bool there[kDeep];
#pragma unroll
      for (int d = 0; d < kDeep; ++d) there[d] = mine + d < hi && mine + d >= before && mine + d - before < total;
      if (there[0] && there[kDeep - 1] && (reinterpret_cast<uintptr_t>(p.new_indices) & 15) == 0) {
        int4* out = reinterpret_cast<int4*>(p.new_indices + mine);
        out[0] = make_int4(slot[0], slot[1], slot[2], slot[3]);
        out[1] = make_int4(slot[4], slot[5], slot[6], slot[7]);
      } else {
#pragma unroll
        for (int d = 0; d < kDeep; ++d)
          if (there[d]) p.new_indices[mine + d] = slot[d];
      }
      if (p.freed) {
        // (few are marked: a read that another block's clearing has overtaken clears once more)
        uint32_t word[kDeep];
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
          const bool in = slot[d] >= 0 && slot[d] < p.num_slots;
          if (there[d] && !in) record_status(p.status, MLA_ERR_INDEX_OOB);
          word[d] = there[d] && in ? p.bits[slot[d] >> 5] : 0;
        }
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
          const uint32_t bit = 1u << (slot[d] & 31);
          if (word[d] & bit) atomicAnd(p.bits + (slot[d] >> 5), ~bit);
        }
      }
    }
    before += total;
  }
}

// -------------------------------------------------------------------- scan --
// Exclusive sum over the cluster's threads (CTA by CTA, thread by thread); all:
// the sum of all.
__device__ __forceinline__ int cluster_scan(int x, int* warp_sums, int* cta_sums, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_ctarank(), ctas = cluster_size();
  int upto = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) warp_sums[warp] = upto;
  cluster_sync_all();                              // the other CTAs run, and this one's sums are there
  if (warp == 0) {
    const int mine = warp_sums[lane];
    int run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    warp_sums[lane] = run - mine;
    const int total = __shfl_sync(0xffffffffu, run, 31);
    if (lane < static_cast<int>(ctas))
      asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(mapa_shared(smem_u32(cta_sums + rank), lane)), "r"(total)
                   : "memory");
    __syncwarp();
  }
  cluster_sync_all();
  int before = warp_sums[warp] + upto - x;
  all = 0;
#pragma unroll
  for (int i = 0; i < kScanCtas; ++i) {
    const int sum = i < static_cast<int>(ctas) ? cta_sums[i] : 0;
    if (i < static_cast<int>(rank)) before += sum;
    all += sum;
  }
  return before;
}

// The words that a thread of the cluster has: its warp's equal share of all, in the lanes' order.
__device__ __forceinline__ void my_words(long long num_slots, long long& w0, long long& w1) {
  const long long words = (num_slots + 31) / 32, warps = cluster_size() * (kScanThreads / 32);
  const long long share = (words + warps - 1) / warps, per = (share + 31) / 32;
  const long long first = (static_cast<long long>(cluster_ctarank()) * (kScanThreads / 32) + (threadIdx.x >> 5)) * share;
  const long long end = min(first + share, words);
  w0 = min(first + (threadIdx.x & 31) * per, end);
  w1 = min(w0 + per, end);
}

// Set bits of words [w0, w1): eight loads at a time.
__device__ __forceinline__ int count_bits(const uint32_t* bits, long long w0, long long w1) {
  int n = 0;
  for (long long w = w0; w < w1; w += 8) {
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = w + i < w1 ? bits[w + i] : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) n += __popc(m[i]);
  }
  return n;
}

// Marked slots to an ascending list; the bitmap is zero again.
__global__ void __launch_bounds__(kScanThreads) freed_kernel(const RepackParams p) {
  __shared__ int warp_sums[32], cta_sums[kScanCtas];
  griddep_wait();
  griddep_launch_dependents();
  long long w0, w1;
  my_words(p.num_slots, w0, w1);
  const int mine = count_bits(p.bits, w0, w1);
  int all;
  long long at = cluster_scan(mine, warp_sums, cta_sums, all);
  for (long long w = w0; w < w1 && mine; ++w) {
    uint32_t m = p.bits[w];
    if (!m) continue;
    p.bits[w] = 0;
    for (; m; m &= m - 1, ++at)
      if (at < p.freed_capacity) p.freed[at] = static_cast<int>(32 * w) + __ffs(m) - 1;
  }
  if (threadIdx.x == 0 && cluster_ctarank() == 0) {
    p.freed_count[0] = all;
    if (all > p.freed_capacity) record_status(p.status, MLA_ERR_WORKSPACE);
  }
}

// -------------------------------------------------------------- compaction --
__device__ __forceinline__ long long entries_of(const CompactParams& c) {
  return min(max(static_cast<long long>(__ldg(c.indptr + c.batch)), 0ll), c.entries);
}

__global__ void __launch_bounds__(kListThreads) compact_mark_kernel(const CompactParams c) {
  griddep_wait();
  griddep_launch_dependents();
  const long long n = entries_of(c);
  for (long long j = static_cast<long long>(blockIdx.x) * kListThreads + threadIdx.x; j < c.entries;
       j += static_cast<long long>(gridDim.x) * kListThreads) {
    const int slot = __ldg(c.indices + j);         // (together with their number)
    if (j >= n) break;
    if (slot >= 0 && slot < c.num_slots) set_bit(c.bits, slot);
    else record_status(c.status, MLA_ERR_INDEX_OOB);
  }
}

// With n live slots: the free slots below n in ascending order, the live ones
// from n on in descending order (the k-th of them from the top of the list is
// the k-th from the end: its place needs no second sum), and, for the lists, the
// live slots before every word.
__global__ void __launch_bounds__(kScanThreads) compact_scan_kernel(const CompactParams c) {
  __shared__ int warp_sums[32], cta_sums[kScanCtas];
  griddep_wait();
  griddep_launch_dependents();
  long long w0, w1;
  my_words(c.num_slots, w0, w1);
  const int mine = count_bits(c.bits, w0, w1);
  int n;
  int run = cluster_scan(mine, warp_sums, cta_sums, n);
  const long long last_word = n >> 5;
  // a word's slots by the warp's lanes, a slot a lane
  const int lane = threadIdx.x & 31;
  const long long per = __shfl_sync(0xffffffffu, w1 - w0, 0);      // words of a lane (the last ones' may be fewer)
  for (long long i = 0; i < per; ++i) {
    const bool mine = w0 + i < w1;
    const uint32_t m = mine ? c.bits[w0 + i] : 0;
    if (mine) {
      if (m) c.bits[w0 + i] = 0;
      c.live[w0 + i] = make_uint2(m, static_cast<uint32_t>(run));
      if (w0 + i == last_word) c.counts[1] = n - run - __popc(m & ((1u << (n & 31)) - 1));
    }
    // (nothing comes of full words below n and of empty ones past it: a pool that is mostly in order)
    const long long s0 = 32 * (w0 + i);
    const bool some = mine && (s0 + 32 <= n ? m != 0xFFFFFFFFu : s0 < n || m != 0);
    for (uint32_t todo = __ballot_sync(0xffffffffu, some); todo; todo &= todo - 1) {
      const int from = __ffs(todo) - 1;
      const uint32_t word = __shfl_sync(0xffffffffu, m, from);
      const int before = __shfl_sync(0xffffffffu, run, from) + __popc(word & ((1u << lane) - 1));   // live slots
      const long long slot = 32 * (__shfl_sync(0xffffffffu, w0, from) + i) + lane;
      const bool live = word >> lane & 1;
      if (slot < n && !live) c.holes[slot - before] = static_cast<int>(slot);
      if (slot >= n && live) c.away[n - 1 - before] = static_cast<int>(slot);
    }
    run += __popc(m);
  }
  if (threadIdx.x == 0 && cluster_ctarank() == 0) {
    c.counts[0] = n;
    c.live_count[0] = n;
    if (last_word >= (c.num_slots + 31) / 32) c.counts[1] = 0;     // every slot is live
  }
}

// The lists, slot by slot: a live slot past the n lowest is the k-th of those.
template <int kThreads = kMoveThreads>
__device__ __forceinline__ void rewrite_lists(const CompactParams& c) {
  const long long total = entries_of(c);
  const int n = __ldcg(c.counts), below = n - __ldcg(c.counts + 1);
  for (long long j = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; j < total;
       j += static_cast<long long>(gridDim.x) * kThreads) {
    int slot = __ldg(c.indices + j);
    if (slot >= n && slot < c.num_slots) {
      const uint2 m = c.live[slot >> 5];
      const int rank = static_cast<int>(m.y) + __popc(m.x & ((1u << (slot & 31)) - 1));
      slot = c.holes[rank - below];
    }
    c.new_indices[j] = slot;
  }
}

// -------------------------------------------------------------------- rows --
// (Row, layer) pair u: row u / layers of the lists, layer u % layers.
struct Pair {
  long long from, to;                              // rows of the whole caches, or from < 0
};
template <bool kLists>
__device__ __forceinline__ Pair pair_of(const MoveParams& p, long long u, int count, bool report) {
  const int k = static_cast<int>(u / p.layers), l = static_cast<int>(u - static_cast<long long>(k) * p.layers);
  const int a = kLists ? __ldcg(p.from + (count - 1 - k)) : __ldg(p.from + k);
  const int z = kLists ? __ldcg(p.to + k) : __ldg(p.to + k);
  if (a < 0 || a >= p.src_slots || z < 0 || z >= p.dst_slots) {
    if (report) record_status(p.status, MLA_ERR_INDEX_OOB);
    return {-1, -1};
  }
  return {l * p.src_rows + a, l * p.dst_rows + z};
}

// Few rows: a thread has one 16-byte piece of a row, of kUnroll pairs at once.
// kLists: behind the compaction's scan, with the lists to rewrite as well.
template <int kRowBytes, bool kLists>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveParams p, const CompactParams c) {
  griddep_wait();
  griddep_launch_dependents();
  if constexpr (kLists) rewrite_lists(c);
  constexpr int kPieces = kRowBytes / 16, kRows = kMoveThreads / kPieces, kUnroll = 4;
  const int row = threadIdx.x / kPieces, piece = threadIdx.x % kPieces;
  const int count = kLists ? __ldcg(p.count_dev) : p.count;
  const long long units = static_cast<long long>(count) * p.layers, step = static_cast<long long>(gridDim.x) * kRows;
  for (long long u0 = static_cast<long long>(blockIdx.x) * kRows + row; u0 < units; u0 += kUnroll * step) {
    uint4 v[kUnroll];
    float s[kUnroll];
    long long to[kUnroll];
#pragma unroll
    for (int d = 0; d < kUnroll; ++d) {
      const long long u = u0 + d * step;
      to[d] = -1;
      if (u >= units) continue;
      const Pair m = pair_of<kLists>(p, u, count, piece == 0);
      if (m.from < 0) continue;
      to[d] = m.to;
      v[d] = *reinterpret_cast<const uint4*>(p.src + m.from * kRowBytes + 16 * piece);
      if (p.src_scales && piece == 0) s[d] = p.src_scales[m.from];
    }
#pragma unroll
    for (int d = 0; d < kUnroll; ++d) {
      if (to[d] < 0) continue;
      *reinterpret_cast<uint4*>(p.dst + to[d] * kRowBytes + 16 * piece) = v[d];
      if (p.src_scales && piece == 0) p.dst_scales[to[d]] = s[d];
    }
  }
}

// Many rows: whole rows by bulk copies through shared memory.  A warp has two
// stages of 32 rows: each lane loads its row of one while the rows of the other
// are on their way out.  Bound: HBM; 111k random rows of 1152 bytes take 39.8 us
// (6.4 TB/s read and written, 0.96 of a plain copy's rate).  us by pieces and by
// bulk copies, of 1152 and of 576 bytes: 4096 rows 3.5 and 4.2, 2.1 and 3.3; 8192
// rows 6.4 and 5.8, 3.6 and 3.7; 16384 rows 10.6 and 9.6, 6.6 and 5.8; 65536 rows
// 32.7 and 26.9, 18.3 and 15.2.
constexpr int kBulkThreads = 96;
template <int kRowBytes>
__host__ __device__ constexpr int bulk_smem() { return kBulkThreads / 32 * (2 * 32 * kRowBytes + 16) + 32; }
template <int kRowBytes, bool kLists>
__global__ void __launch_bounds__(kBulkThreads) move_bulk_kernel(const MoveParams p, const CompactParams c) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kWarps = kBulkThreads / 32, kStage = 32 * kRowBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem), rows = base + warp * 2 * kStage;
  const uint32_t bars = base + kWarps * 2 * kStage + 16 * warp;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kWarps * (2 * kStage + 16));
  const WaitCtx wc{abort_flag, p.status};
  if (lane == 0) {
    mbar_init(bars, 1);
    mbar_init(bars + 8, 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) *abort_flag = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  if constexpr (kLists) rewrite_lists<kBulkThreads>(c);
  const int count = kLists ? __ldcg(p.count_dev) : p.count;
  const long long units = static_cast<long long>(count) * p.layers;
  const long long step = 32ll * gridDim.x * kWarps, first = 32ll * (static_cast<long long>(blockIdx.x) * kWarps + warp);
  auto load = [&](long long u0, uint32_t stage) -> long long {
    const Pair m = u0 + lane < units ? pair_of<kLists>(p, u0 + lane, count, true) : Pair{-1, -1};
    const int n = __popc(__ballot_sync(0xffffffffu, m.from >= 0));
    if (lane == 0) mbar_arrive_expect_tx(bars + 8 * stage, n * kRowBytes);
    __syncwarp();
    if (m.from >= 0) {
      bulk_load(rows + stage * kStage + lane * kRowBytes, p.src + m.from * kRowBytes, kRowBytes, bars + 8 * stage);
      if (p.src_scales) p.dst_scales[m.to] = p.src_scales[m.from];
    }
    return m.to;
  };
  long long to = first < units ? load(first, 0) : -1;
  uint32_t i = 0;
  for (long long u0 = first; u0 < units; u0 += step, ++i) {
    const uint32_t stage = i & 1;
    long long next = -1;
    if (u0 + step < units) {
      bulk_wait_read();                            // this lane's rows of the other stage have left it
      __syncwarp();
      next = load(u0 + step, stage ^ 1);
    }
    if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * stage, (i >> 1) & 1, wc))) {
      // no copy outlives the block
      drain_wait(bars + 8 * stage, (i >> 1) & 1);
      if (u0 + step < units) drain_wait(bars + 8 * (stage ^ 1), ((i + 1) >> 1) & 1);
      break;
    }
    if (to >= 0) bulk_store(p.dst + to * kRowBytes, rows + stage * kStage + lane * kRowBytes, kRowBytes);
    bulk_commit();
    to = next;
  }
  bulk_wait_all();
}

template <int kRowBytes, bool kLists>
int launch_rows(const MoveParams& m, const CompactParams& c, long long most, long long entries, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms < 1) return MLA_ERR_CUDA;
  const long long units = most * m.layers;
  if (units >= kBulkRows) {
    const int smem = bulk_smem<kRowBytes>(), held = 227 * 1024 / (smem + 1024) * sms;
    const auto kernel = &move_bulk_kernel<kRowBytes, kLists>;
    if (!set_smem_limit(reinterpret_cast<const void*>(kernel), smem)) return MLA_ERR_CUDA;
    const long long need = (units + kBulkThreads - 1) / kBulkThreads;
    return launch_after(kernel, dim3(static_cast<unsigned>(need < held ? need : held)), kBulkThreads, 1, smem, stream, m, c);
  }
  const int rows = kMoveThreads * 16 / kRowBytes;
  const long long need = (units + rows - 1) / rows, lists = (entries + kMoveThreads - 1) / kMoveThreads;
  const long long want = need > lists ? need : lists, held = 7ll * sms;
  const unsigned grid = static_cast<unsigned>(want < 1 ? 1 : want < held ? want : held);
  return launch_after(move_kernel<kRowBytes, kLists>, dim3(grid), kMoveThreads, 1, 0, stream, m, c);
}

template <bool kLists>
int launch_rows(const MoveParams& m, const CompactParams& c, long long most, long long entries, cudaStream_t stream) {
  return m.row_bytes == kRow ? launch_rows<kRow, kLists>(m, c, most, entries, stream)
                             : launch_rows<2 * kRow, kLists>(m, c, most, entries, stream);
}

}  // namespace

int launch_repack(const RepackParams& params, cudaStream_t stream) {
  RepackParams p = params;
  p.marked = p.freed && p.batch > 0 && p.entries > 0;
  // (asked for before anything is launched: without the last kernel the marks would stay)
  const int ctas = p.freed ? widest_cluster(reinterpret_cast<const void*>(freed_kernel), kScanThreads, kScanCtas) : 0;
  if (p.freed && ctas < 1) return MLA_ERR_CUDA;
  if (p.marked) {
    const unsigned blocks = static_cast<unsigned>((p.entries + kChunk - 1) / kChunk);
    const int st = launch_after(repack_mark_kernel, dim3(blocks), kListThreads, 1, 0, stream, p);
    if (st != MLA_OK) return st;
  }
  const unsigned blocks = static_cast<unsigned>(p.capacity > 0 ? (p.capacity + kChunk - 1) / kChunk : 1);
  const int st = launch_after(repack_lists_kernel, dim3(blocks), kListThreads, 1, 0, stream, p);
  if (st != MLA_OK || !p.freed) return st;
  return launch_after(freed_kernel, dim3(ctas), kScanThreads, ctas, 0, stream, p);
}

int launch_move(const MoveParams& m, long long most, cudaStream_t stream) {
  return launch_rows<false>(m, CompactParams{}, most, 0, stream);
}

int launch_compact(const CompactParams& c, const MoveParams& m, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms < 1) return MLA_ERR_CUDA;
  const long long blocks = (c.entries + 4 * kListThreads - 1) / (4 * kListThreads), held = 8ll * sms;
  const unsigned grid = static_cast<unsigned>(blocks < 1 ? 1 : blocks < held ? blocks : held);
  const int ctas = widest_cluster(reinterpret_cast<const void*>(compact_scan_kernel), kScanThreads, kScanCtas);
  if (ctas < 1) return MLA_ERR_CUDA;
  int st = launch_after(compact_mark_kernel, dim3(grid), kListThreads, 1, 0, stream, c);
  if (st != MLA_OK) return st;
  st = launch_after(compact_scan_kernel, dim3(ctas), kScanThreads, ctas, 0, stream, c);
  if (st != MLA_OK) return st;
  const long long half = c.num_slots / 2;
  return launch_rows<true>(m, c, half < c.entries ? half : c.entries, c.entries, stream);
}

}  // namespace mla
