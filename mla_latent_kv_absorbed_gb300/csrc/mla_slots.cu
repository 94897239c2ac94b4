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
constexpr int kScanThreads = 1024, kScanCtas = 8;
constexpr int kMoveThreads = 288;                  // 4 rows of 72 pieces of 16 bytes, or 8 of 36

template <typename Kernel, typename... Args>
int launch_after(Kernel* kernel, dim3 grid, int threads, int cluster, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
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
  int start, base, count;
};
__device__ __forceinline__ Kept kept_of(const RepackParams& p, int src, bool report) {
  if (src < 0 || src >= p.batch) {
    if (report && src != -1) record_status(p.status, MLA_ERR_PLAN_MISMATCH);
    return {0, 0, 0};
  }
  const long long lo = __ldg(p.indptr + src), hi = __ldg(p.indptr + src + 1);
  const long long s = min(max(lo, 0ll), p.entries), e = min(max(hi, s), p.entries);
  const int n = static_cast<int>(e - s);
  bool bad = lo != s || hi != e;
  Kept k{static_cast<int>(s), n, n};
  if (p.path) {
    if (n >= p.width) {
      const int a = __ldg(p.accepted + src);
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

// Marks the slots that a request gives up: all of them where no new request
// continues it, else those of the drafts off its path.  Another request may hold
// them too (a shared prefix): the lists' kernel takes those back.
__global__ void __launch_bounds__(kListThreads) repack_mark_kernel(const RepackParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int o = blockIdx.x, tid = threadIdx.x;
  const Kept k = kept_of(p, o, false);
  bool here = false;
  for (int i = tid; i < p.new_batch; i += kListThreads) here |= __ldg(p.sources + i) == o;
  const bool goes_on = __syncthreads_or(here) != 0;
  auto give_up = [&](int j) {
    const int slot = __ldg(p.indices + j);
    if (slot >= 0 && slot < p.num_slots) set_bit(p.bits, slot);
    else record_status(p.status, MLA_ERR_INDEX_OOB);
  };
  if (!goes_on) {
    const long long lo = __ldg(p.indptr + o), hi = __ldg(p.indptr + o + 1);
    const int s = static_cast<int>(min(max(lo, 0ll), p.entries));
    const int e = static_cast<int>(min(max(hi, static_cast<long long>(s)), p.entries));
    for (long long j = s + blockIdx.y * kListThreads + tid; j < e; j += static_cast<long long>(gridDim.y) * kListThreads)
      give_up(static_cast<int>(j));
  } else if (p.path && blockIdx.y == 0 && tid < p.width) {
    const int n = __ldg(p.indptr + o + 1) - __ldg(p.indptr + o);
    if (n < p.width || k.base != n - p.width) return;
    bool kept = false;
    for (int i = 0; i < k.count - k.base; ++i)
      kept |= min(max(__ldg(p.path + static_cast<long long>(o) * p.width + i), 0), p.width - 1) == tid;
    if (!kept) give_up(k.start + k.base + tid);
  }
}

// The new lists: block (r, y) writes its share of request r, whose place it
// adds up itself from the lengths before it.
__global__ void __launch_bounds__(kListThreads) repack_lists_kernel(const RepackParams p) {
  __shared__ long long sums[kListThreads / 32];
  const int r = blockIdx.x, tid = threadIdx.x;
  // behind the marking kernel the inputs are there already: it started after whatever made them
  if (!p.freed) griddep_wait();
  long long before = 0;
  for (int i = tid; i < r; i += kListThreads) before += kept_of(p, __ldg(p.sources + i), false).count;
#pragma unroll
  for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if ((tid & 31) == 0) sums[tid >> 5] = before;
  __syncthreads();
  before = 0;
#pragma unroll
  for (int i = 0; i < kListThreads / 32; ++i) before += sums[i];
  const int src = r < p.new_batch ? __ldg(p.sources + r) : -1;
  const bool first = blockIdx.y == 0 && tid == 0;
  const Kept k = kept_of(p, src, first);
  if (p.freed) griddep_wait();
  griddep_launch_dependents();
  if (first) {
    p.new_indptr[r] = static_cast<int>(min(before, p.capacity));
    if (r == p.new_batch - 1) p.new_indptr[r + 1] = static_cast<int>(min(before + k.count, p.capacity));
    if (before + k.count > p.capacity) record_status(p.status, MLA_ERR_WORKSPACE);
  }
  const int32_t* path = p.path ? p.path + static_cast<long long>(src) * p.width : nullptr;
  const long long stride = static_cast<long long>(gridDim.y) * kListThreads;
  constexpr int kDeep = 4;
  for (long long j0 = blockIdx.y * kListThreads + tid; j0 < k.count; j0 += kDeep * stride) {
    int slot[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const long long j = j0 + d * stride;
      if (j >= k.count) continue;
      int at = static_cast<int>(j);
      if (at >= k.base) {
        const int step = __ldg(path + at - k.base), ok = min(max(step, 0), p.width - 1);
        if (step != ok) record_status(p.status, MLA_ERR_TREE);
        at = k.base + ok;
      }
      slot[d] = __ldg(p.indices + k.start + at);
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const long long j = j0 + d * stride;
      if (j >= k.count) continue;
      if (before + j < p.capacity) p.new_indices[before + j] = slot[d];
      if (!p.freed) continue;
      if (slot[d] < 0 || slot[d] >= p.num_slots) {
        record_status(p.status, MLA_ERR_INDEX_OOB);
        continue;
      }
      // (few are marked: a read that another block's clearing has overtaken clears once more)
      const uint32_t bit = 1u << (slot[d] & 31);
      if (p.bits[slot[d] >> 5] & bit) atomicAnd(p.bits + (slot[d] >> 5), ~bit);
    }
  }
}

// -------------------------------------------------------------------- scan --
// Exclusive sum over the cluster's threads (CTA by CTA, thread by thread); all:
// the sum of all.
__device__ __forceinline__ int cluster_scan(int x, int* warp_sums, int* cta_sums, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_ctarank();
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
    if (lane < kScanCtas)
      asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(mapa_shared(smem_u32(cta_sums + rank), lane)), "r"(total)
                   : "memory");
    __syncwarp();
  }
  cluster_sync_all();
  int before = warp_sums[warp] + upto - x;
  all = 0;
#pragma unroll
  for (int i = 0; i < kScanCtas; ++i) {
    if (i < static_cast<int>(rank)) before += cta_sums[i];
    all += cta_sums[i];
  }
  return before;
}

// The words that a thread of the cluster has: a stretch of its own.
__device__ __forceinline__ void my_words(long long num_slots, long long& w0, long long& w1) {
  const long long words = (num_slots + 31) / 32, threads = kScanCtas * kScanThreads;
  const long long per = (words + threads - 1) / threads;
  w0 = min((static_cast<long long>(cluster_ctarank()) * kScanThreads + threadIdx.x) * per, words);
  w1 = min(w0 + per, words);
}

// Marked slots to an ascending list; the bitmap is zero again.
__global__ void __launch_bounds__(kScanThreads) freed_kernel(const RepackParams p) {
  __shared__ int warp_sums[32], cta_sums[kScanCtas];
  griddep_wait();
  griddep_launch_dependents();
  long long w0, w1;
  my_words(p.num_slots, w0, w1);
  int mine = 0;
  for (long long w = w0; w < w1; ++w) mine += __popc(p.bits[w]);
  int all;
  long long at = cluster_scan(mine, warp_sums, cta_sums, all);
  for (long long w = w0; w < w1 && mine; ++w) {
    uint32_t m = p.bits[w];
    if (!m) continue;
    p.bits[w] = 0;
    for (; m; m &= m - 1, ++at)
      if (at < p.freed_capacity) p.freed[at] = static_cast<int>(32 * w) + __ffs(m) - 1;
  }
  if (w0 == 0 && threadIdx.x == 0 && cluster_ctarank() == 0) {
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
  for (long long j = static_cast<long long>(blockIdx.x) * kListThreads + threadIdx.x; j < n;
       j += static_cast<long long>(gridDim.x) * kListThreads) {
    const int slot = __ldg(c.indices + j);
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
  int mine = 0;
  for (long long w = w0; w < w1; ++w) mine += __popc(c.bits[w]);
  int n;
  int run = cluster_scan(mine, warp_sums, cta_sums, n);
  const long long last_word = n >> 5;
  for (long long w = w0; w < w1; ++w) {
    const uint32_t m = c.bits[w];
    if (m) c.bits[w] = 0;
    c.live[w] = make_uint2(m, static_cast<uint32_t>(run));
    // the slots of this word below n
    const uint32_t low = w < last_word ? 0xffffffffu : w > last_word ? 0u : (1u << (n & 31)) - 1;
    for (uint32_t f = ~m & low; f; f &= f - 1) {
      const int bit = __ffs(f) - 1;
      const int slot = static_cast<int>(32 * w) + bit;
      c.holes[slot - run - __popc(m & ((1u << bit) - 1))] = slot;
    }
    for (uint32_t a = m & ~low; a; a &= a - 1) {
      const int bit = __ffs(a) - 1;
      c.away[n - 1 - run - __popc(m & ((1u << bit) - 1))] = static_cast<int>(32 * w) + bit;
    }
    if (w == last_word) c.counts[1] = n - run - __popc(m & low);
    run += __popc(m);
  }
  if (threadIdx.x == 0 && cluster_ctarank() == 0) {
    c.counts[0] = n;
    c.live_count[0] = n;
    if (last_word >= (c.num_slots + 31) / 32) c.counts[1] = 0;     // every slot is live
  }
}

// The lists, slot by slot: a live slot past the n lowest is the k-th of those.
__device__ __forceinline__ void rewrite_lists(const CompactParams& c) {
  const long long total = entries_of(c);
  const int n = __ldcg(c.counts), below = n - __ldcg(c.counts + 1);
  for (long long j = static_cast<long long>(blockIdx.x) * kMoveThreads + threadIdx.x; j < total;
       j += static_cast<long long>(gridDim.x) * kMoveThreads) {
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
// A thread has one 16-byte piece of a row, of kDeep (row, layer) pairs at once.
// kLists: behind the compaction's scan, with the lists to rewrite as well.
template <int kRowBytes, bool kLists>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveParams p, const CompactParams c) {
  griddep_wait();
  griddep_launch_dependents();
  if constexpr (kLists) rewrite_lists(c);
  constexpr int kPieces = kRowBytes / 16, kRows = kMoveThreads / kPieces, kDeep = 4;
  const int row = threadIdx.x / kPieces, piece = threadIdx.x % kPieces;
  const int count = kLists ? __ldcg(p.count_dev) : p.count;
  const long long units = static_cast<long long>(count) * p.layers, step = static_cast<long long>(gridDim.x) * kRows;
  for (long long u0 = static_cast<long long>(blockIdx.x) * kRows + row; u0 < units; u0 += kDeep * step) {
    uint4 v[kDeep];
    float s[kDeep];
    long long to[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const long long u = u0 + d * step;
      to[d] = -1;
      if (u >= units) continue;
      const int k = static_cast<int>(u / p.layers), l = static_cast<int>(u - static_cast<long long>(k) * p.layers);
      const int a = kLists ? __ldcg(p.from + (count - 1 - k)) : __ldg(p.from + k);
      const int z = kLists ? __ldcg(p.to + k) : __ldg(p.to + k);
      if (a < 0 || a >= p.src_slots || z < 0 || z >= p.dst_slots) {
        if (piece == 0) record_status(p.status, MLA_ERR_INDEX_OOB);
        continue;
      }
      const long long from = l * p.src_rows + a;
      to[d] = l * p.dst_rows + z;
      v[d] = *reinterpret_cast<const uint4*>(p.src + from * kRowBytes + 16 * piece);
      if (p.src_scales && piece == 0) s[d] = p.src_scales[from];
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (to[d] < 0) continue;
      *reinterpret_cast<uint4*>(p.dst + to[d] * kRowBytes + 16 * piece) = v[d];
      if (p.src_scales && piece == 0) p.dst_scales[to[d]] = s[d];
    }
  }
}

template <bool kLists>
int launch_rows(const MoveParams& m, const CompactParams& c, long long most, long long entries, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms < 1) return MLA_ERR_CUDA;
  const int rows = kMoveThreads * 16 / m.row_bytes;
  const long long need = (most * m.layers + rows - 1) / rows, lists = (entries + kMoveThreads - 1) / kMoveThreads;
  const long long want = need > lists ? need : lists, held = 7ll * sms;
  const unsigned grid = static_cast<unsigned>(want < 1 ? 1 : want < held ? want : held);
  return m.row_bytes == kRow ? launch_after(move_kernel<kRow, kLists>, dim3(grid), kMoveThreads, 1, stream, m, c)
                             : launch_after(move_kernel<2 * kRow, kLists>, dim3(grid), kMoveThreads, 1, stream, m, c);
}

// Blocks that share a request's list: enough for eight an SM, as far as lists reach.
unsigned stripes(long long entries, int requests, int sms) {
  const long long mean = entries / (requests > 0 ? requests : 1) / (4 * kListThreads) + 1;
  const long long want = 8ll * sms / (requests > 0 ? requests : 1) + 1;
  const long long n = want < 2 * mean ? want : 2 * mean;
  return static_cast<unsigned>(n < 64 ? n : 64);
}

}  // namespace

int launch_repack(const RepackParams& p, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms < 1) return MLA_ERR_CUDA;
  if (p.freed && p.batch > 0) {
    const dim3 grid(p.batch, stripes(p.entries, p.batch, sms));
    const int st = launch_after(repack_mark_kernel, grid, kListThreads, 1, stream, p);
    if (st != MLA_OK) return st;
  }
  const dim3 grid(p.new_batch > 0 ? p.new_batch : 1, stripes(p.entries, p.new_batch, sms));
  int st = launch_after(repack_lists_kernel, grid, kListThreads, 1, stream, p);
  if (st != MLA_OK || !p.freed) return st;
  return launch_after(freed_kernel, dim3(kScanCtas), kScanThreads, kScanCtas, stream, p);
}

int launch_move(const MoveParams& m, long long most, cudaStream_t stream) {
  return launch_rows<false>(m, CompactParams{}, most, 0, stream);
}

int launch_compact(const CompactParams& c, const MoveParams& m, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms < 1) return MLA_ERR_CUDA;
  const long long blocks = (c.entries + 4 * kListThreads - 1) / (4 * kListThreads), held = 8ll * sms;
  const unsigned grid = static_cast<unsigned>(blocks < 1 ? 1 : blocks < held ? blocks : held);
  int st = launch_after(compact_mark_kernel, dim3(grid), kListThreads, 1, stream, c);
  if (st != MLA_OK) return st;
  st = launch_after(compact_scan_kernel, dim3(kScanCtas), kScanThreads, kScanCtas, stream, c);
  if (st != MLA_OK) return st;
  const long long half = c.num_slots / 2;
  return launch_rows<true>(m, c, half < c.entries ? half : c.entries, c.entries, stream);
}

}  // namespace mla
