// The paged cache's upkeep: pages handed out, shared, copied and given back, and the accepted
// tokens of a draft tree moved to their places (the entry points' rules are in
// include/mtp_cache.h).
//
// resize and fork run a planning kernel and a copying kernel.  The plan is one thread-block
// cluster, because every page handed out depends on all the counts below it: its CTAs first
// give pages back (resize), meet, mark their part of the pool's free pages in shared memory, tell
// one another how many they found, meet again, and then know each free page's rank; the page of
// rank k goes to the k-th place wanted, found by a search over the rows' running sums of wants.
// The pages to copy are left in the workspace, one (from, to) pair a row, for the copying kernel,
// which is launched beside the plan and starts when the plan has ended.
//
// What bounds a plan is its chain of dependent memory accesses (lengths, table entry, count,
// rank, place: about 0.5 us each) and the meetings, not the bytes: so what a row asks for is
// worked out once by every CTA and stays in shared memory, and loads that do not depend on a
// meeting are issued before it.  Three calls (rows freed and trimmed, forked, grown) take 16.5 to
// 17.2 us in a CUDA graph for 4 rows and a pool of 512 pages, 29 us for 256 rows, 128 forks and 16384
// pages; with the items read again at each step, four meetings and the copying kernel launched
// after the plan it was 33 and 48 us.  One CTA instead of the cluster's 8 is no faster for the
// small table (16.5 us) and takes 72 us for the large one; 1024 threads a CTA 18.0 and 29.9 us.
#include "common.cuh"
#include "host_checks.cuh"

#include "../../include/mtp_cache.h"
#include "../../include/mtp_tree.h"

#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

namespace cg = cooperative_groups;

namespace mtpattn {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanCtas = 8;
constexpr int kCopyThreads = 256;

struct PlanParams {
  int32_t* bt;
  int32_t max_pages;
  int32_t* seq_lens;
  int32_t rows;
  int32_t* ref;
  int32_t num_pages;
  const int32_t* new_lens;   // resize
  const int32_t* src;        // fork
  const int32_t* dst;
  int32_t items;             // rows (resize) or pairs (fork)
  int2* copies;              // workspace: [items] pages (from, to), from < 0: none
  int32_t* status;
};

// (of a length that has been compared with its table's: the sum passes 32 bits for others)
__device__ __forceinline__ int pages_of(int len) { return (len + kPage - 1) / kPage; }

// A plan's shared memory. An item is a row (resize) or a pair of rows (fork).
struct PlanSmem {
  uint32_t* free;            // [mask_words] a bit for each page of this CTA's part of the pool
  int* sum;                  // [items] what the items want, then the running sums
  int* tail;                 // [items] the page to be copied, or -1
  int* slot;                 // [items] table position of the first page handed out; -1: not live
  int* claim;                // [rows], fork: the first pair that names a dst
  uint8_t* bad;              // [items], fork: the source row has a bad entry
};
__host__ __device__ constexpr int mask_words(int num_pages) {
  const int per = (num_pages + kPlanCtas - 1) / kPlanCtas;
  return ((per + kPlanWarps - 1) / kPlanWarps + 31) / 32 * kPlanWarps;
}
constexpr size_t plan_smem(bool fork, int num_pages, int items, int rows) {
  return 4 * (static_cast<size_t>(mask_words(num_pages)) + 3 * static_cast<size_t>(items)) +
         (fork ? 4 * static_cast<size_t>(rows) + (items + 3) / 4 * 4 : 0);
}

// Sums of wants stop at this: more than any pool has, and two of them fit in 32 bits.
constexpr uint32_t kManyPages = 1u << 30;
static_assert(MTP_CACHE_MAX_PAGES < (1 << 30));
__device__ __forceinline__ uint32_t add_wants(uint32_t a, uint32_t b) { return min(a + b, kManyPages); }
__device__ __forceinline__ uint32_t warp_sums(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = add_wants(v, x);
  }
  return v;
}

// Inclusive running sums of want[0 .. n) in place, by the whole CTA; returns their total.
__device__ uint32_t scan_wants(int* want, int n, uint32_t* s_warp) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  uint32_t carry = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const uint32_t v = warp_sums(i0 + t < n ? min(static_cast<uint32_t>(want[i0 + t]), kManyPages) : 0, lane);
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    const uint32_t w = warp_sums(lane < kPlanWarps ? s_warp[lane] : 0u, lane);
    const uint32_t below = __shfl_sync(0xffffffffu, w, max(warp, 1) - 1);
    const uint32_t before = warp ? add_wants(carry, below) : carry;
    if (i0 + t < n) want[i0 + t] = static_cast<int>(add_wants(v, before));
    carry = add_wants(carry, __shfl_sync(0xffffffffu, w, 31));
    __syncthreads();
  }
  return carry;
}

// The free pages of this CTA's part of the pool, marked in shared memory; returns how many this
// warp found.  A warp has a contiguous piece of `words` words.
__device__ __forceinline__ int mark_free(const PlanParams& p, uint32_t* mine, int words, int lo, int end, int lane) {
  int count = 0;
#pragma unroll 4
  for (int w = 0; w < words; ++w) {
    const int page = lo + 32 * w + lane;
    const uint32_t m = __ballot_sync(0xffffffffu, page < end && __ldcg(p.ref + page) == 0);
    if (lane == 0) mine[w] = m;
    count += __popc(m);
  }
  return count;
}

template <bool Fork>
__global__ void __launch_bounds__(kPlanThreads, 1)
cache_plan_kernel(const PlanParams p) {
  extern __shared__ uint32_t s_plan[];
  __shared__ uint32_t s_warp[kPlanWarps];
  __shared__ int s_base[kPlanWarps];
  __shared__ int s_free[kPlanCtas];
  cg::cluster_group cluster = cg::this_cluster();
  constexpr int parts = kPlanCtas;
  const int part = cluster.block_rank();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int gwarp = part * kPlanWarps + warp, gwarps = parts * kPlanWarps;
  const int gt = part * kPlanThreads + t, gthreads = parts * kPlanThreads;
  const int words = mask_words(p.num_pages) / kPlanWarps;    // a warp's
  PlanSmem s;
  s.free = s_plan;
  s.sum = reinterpret_cast<int*>(s.free + words * kPlanWarps);
  s.tail = s.sum + p.items;
  s.slot = s.tail + p.items;
  s.claim = s.slot + p.items;
  s.bad = reinterpret_cast<uint8_t*>(s.claim + p.rows);
  const int64_t top = static_cast<int64_t>(p.max_pages) * kPage;
  const int per = (p.num_pages + parts - 1) / parts;
  const int end = min(static_cast<int64_t>(p.num_pages), static_cast<int64_t>(part + 1) * per);
  const int lo = static_cast<int>(min(static_cast<int64_t>(end),
                                      static_cast<int64_t>(part) * per + static_cast<int64_t>(warp) * words * 32));
  uint32_t* mine = s.free + warp * words;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // The cluster meets twice.  Before the first meeting: resize gives the surplus pages back, a warp
  // a row; fork tells all its CTAs which pairs have a source row with a bad entry.
  int found;
  if (Fork) {
    cluster.barrier_arrive();                      // all have started: their memory can be written
    for (int i = t; i < p.rows; i += kPlanThreads) s.claim[i] = INT32_MAX;
    __syncthreads();
    for (int i = t; i < p.items; i += kPlanThreads) {
      const int d = p.dst[i];
      if (d >= 0 && d < p.rows) atomicMin(&s.claim[d], i);
    }
    found = mark_free(p, mine, words, lo, end, lane);
    cluster.barrier_wait();
    for (int i = gwarp; i < p.items; i += gwarps) {
      const int src = p.src[i];
      bool bad = false;
      if (src >= 0 && src < p.rows) {
        const int len = p.seq_lens[src];
        const int n = len > 0 && len <= top ? pages_of(len) : 0;
        const int32_t* row = p.bt + static_cast<int64_t>(src) * p.max_pages;
#pragma unroll 4
        for (int j = lane; j < n; j += 32) bad |= static_cast<uint32_t>(row[j]) >= static_cast<uint32_t>(p.num_pages);
        bad = __any_sync(0xffffffffu, bad);
      }
      if (lane < parts) *cluster.map_shared_rank(&s.bad[i], lane) = bad;
    }
  } else {
    for (int i = gwarp; i < p.rows; i += gwarps) {
      const int old = p.seq_lens[i], len = p.new_lens[i];
      if (old < 0 || old > top || len < 0 || len > top) {
        if (lane == 0) set_status(p.status, MTP_CACHE_ERR_LEN);
        continue;
      }
      int32_t* row = p.bt + static_cast<int64_t>(i) * p.max_pages;
      for (int j = pages_of(len) + lane; j < pages_of(old); j += 32) {
        const int page = row[j];
        row[j] = -1;
        if (page < 0 || page >= p.num_pages) {
          set_status(p.status, MTPATTN_ERR_PAGE);
        } else if (atomicSub(&p.ref[page], 1) <= 0) {
          atomicAdd(&p.ref[page], 1);
          set_status(p.status, MTP_CACHE_ERR_REF);
        }
      }
    }
    __threadfence();
    cluster.barrier_arrive();
    // What the rows ask for: the pages beyond those they keep, and one for the last kept page where
    // it is partly filled and shared (looked at after the meeting).
    for (int i = t; i < p.items; i += kPlanThreads) {
      const int old = p.seq_lens[i], len = p.new_lens[i];
      const bool live = old >= 0 && old <= top && len >= 0 && len <= top;
      const int kept = min(old, len), have = live ? pages_of(kept) : -1;
      s.sum[i] = live ? pages_of(len) - have : 0;
      s.slot[i] = have;
      s.tail[i] = live && kept % kPage != 0 ? p.bt[static_cast<int64_t>(i) * p.max_pages + have - 1] : -1;
    }
    cluster.barrier_wait();
    for (int i = t; i < p.items; i += kPlanThreads) {
      const int page = s.tail[i];
      if (page >= 0 && page < p.num_pages && __ldcg(p.ref + page) > 1) {
        ++s.sum[i];
        --s.slot[i];
      } else {
        s.tail[i] = -1;
      }
    }
    found = mark_free(p, mine, words, lo, end, lane);
  }
  if (lane == 0) s_base[warp] = found;
  __syncthreads();
  if (warp == 0) {
    int all = lane < kPlanWarps ? s_base[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (lane < parts) *cluster.map_shared_rank(&s_free[part], lane) = all;
  }
  cluster.sync();                                  // resize: all lengths and counts have been read

  constexpr int kOwn = MTP_CACHE_MAX_ROWS / (kPlanThreads * kPlanCtas);      // items a thread, at most
  static_assert(kOwn * kPlanThreads * kPlanCtas == MTP_CACHE_MAX_ROWS);
  int err = 0, my_row[kOwn], my_len[kOwn];
#pragma unroll
  for (int o = 0; o < kOwn; ++o) my_row[o] = -1;
  if (Fork) {
    for (int i = t; i < p.items; i += kPlanThreads) {
      const int src = p.src[i], row = p.dst[i];
      const bool rows = src >= 0 && src < p.rows && row >= 0 && row < p.rows && src != row &&
                        s.claim[row] == i && p.seq_lens[row] == 0;
      const int len = rows ? p.seq_lens[src] : 0;
      const bool fits_table = len >= 0 && len <= top;
      if (!rows) err |= MTP_CACHE_ERR_ROW;
      else if (!fits_table) err |= MTP_CACHE_ERR_LEN;
      else if (s.bad[i]) err |= MTPATTN_ERR_PAGE;
      const bool live = rows && fits_table && !s.bad[i];
      const bool part_full = live && len % kPage != 0;
      s.slot[i] = live ? len / kPage : -1;
      s.tail[i] = part_full ? p.bt[static_cast<int64_t>(src) * p.max_pages + len / kPage] : -1;
      s.sum[i] = part_full;
#pragma unroll
      for (int o = 0; o < kOwn; ++o)
        if (i == gt + o * gthreads && live) {
          my_row[o] = row;
          my_len[o] = len;
        }
    }
    __syncthreads();
    cluster.barrier_arrive();                      // this CTA has read the lengths
  }
  const uint32_t total = scan_wants(s.sum, p.items, s_warp);
  int rank = 0, all_free = 0;                      // free pages before this warp's, of the pool
  for (int i = 0; i < parts; ++i) {
    if (i < part) rank += s_free[i];
    all_free += s_free[i];
  }
  rank += __reduce_add_sync(0xffffffffu, lane < warp ? s_base[lane] : 0);
  const bool fits = total <= static_cast<uint32_t>(all_free);
  if (part == 0) {
    if (!fits) err |= MTP_CACHE_ERR_FULL;
    err = __reduce_or_sync(0xffffffffu, err);
    if (err && lane == 0) set_status(p.status, err);
  }

  if (fits)
    for (int w = 0; w < words && static_cast<uint32_t>(rank) < total; ++w) {
      const uint32_t m = mine[w];
      const int k = rank + __popc(m & ((1u << lane) - 1u)), page = lo + 32 * w + lane;
      if ((m >> lane & 1u) && static_cast<uint32_t>(k) < total) {
        int a = 0, z = p.items - 1;                // the first item whose running sum passes k
        while (a < z) {
          const int mid = (a + z) / 2;
          if (s.sum[mid] > k) z = mid; else a = mid + 1;
        }
        const int nth = k - (a ? s.sum[a - 1] : 0), tail = s.tail[a];
        p.ref[page] = 1;
        p.bt[static_cast<int64_t>(Fork ? p.dst[a] : a) * p.max_pages + s.slot[a] + nth] = page;
        if (tail >= 0 && nth == 0) {
          p.copies[a] = make_int2(tail, page);
          if (!Fork) atomicSub(&p.ref[tail], 1);
        }
      }
      rank += __popc(m);
    }
  for (int i = gt; i < p.items; i += gthreads)
    if (!fits || s.tail[i] < 0) p.copies[i] = make_int2(-1, -1);

  // Shared pages are counted; lengths change last.
  if (Fork) {
    if (fits)
      for (int i = gwarp; i < p.items; i += gwarps) {
        if (s.slot[i] < 0) continue;
        const int32_t* from = p.bt + static_cast<int64_t>(p.src[i]) * p.max_pages;
        int32_t* to = p.bt + static_cast<int64_t>(p.dst[i]) * p.max_pages;
#pragma unroll 4
        for (int j = lane; j < s.slot[i]; j += 32) {
          const int page = from[j];
          to[j] = page;
          atomicAdd(&p.ref[page], 1);
        }
      }
    // A source row may be the dst of another pair: its length has been read by every CTA before
    // one is written.
    cluster.barrier_wait();
#pragma unroll
    for (int o = 0; o < kOwn; ++o)
      if (fits && my_row[o] >= 0) p.seq_lens[my_row[o]] = my_len[o];
  } else {
    for (int i = gt; i < p.rows; i += gthreads)
      if (s.slot[i] >= 0) {
        const int len = p.new_lens[i];
        p.seq_lens[i] = fits ? len : min(p.seq_lens[i], len);
      }
  }
}

// Pages from -> to, all layers, K and V: blockIdx.x the pair, blockIdx.y the layer and cache.
struct CopyParams {
  uint8_t* k;
  uint8_t* v;
  int32_t layers;
  int64_t layer_stride;      // bytes
  int64_t num_pages;
  int64_t page_bytes;
  const int2* copies;        // planned pairs, or null:
  const int32_t* src;
  const int32_t* dst;
  int32_t items;
  int32_t* status;
};

__global__ void __launch_bounds__(kCopyThreads)
cache_copy_kernel(const CopyParams p) {
  const int i = blockIdx.x;
  int from, to;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the plan, where there is one, has ended
  if (p.copies) {
    const int2 c = p.copies[i];
    if (c.x < 0) return;
    from = c.x;
    to = c.y;
  } else {
    from = p.src[i];
    to = p.dst[i];
    if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) {
      if (blockIdx.y == 0 && threadIdx.x == 0) set_status(p.status, MTPATTN_ERR_PAGE);
      return;
    }
    if (from == to) return;
  }
  for (int l = blockIdx.y; l < 2 * p.layers; l += gridDim.y) {
    uint8_t* layer = ((l & 1) ? p.v : p.k) + static_cast<int64_t>(l >> 1) * p.layer_stride;
    const uint4* a = reinterpret_cast<const uint4*>(layer + from * p.page_bytes);
    uint4* z = reinterpret_cast<uint4*>(layer + to * p.page_bytes);
    const int n = static_cast<int>(p.page_bytes / 16);
    for (int j = threadIdx.x; j < n; j += kCopyThreads) z[j] = a[j];
  }
}

// The accepted path to the front of the tree's places.  A thread owns 16 bytes of a head's row
// in one layer of one cache, and moves them for the whole path: node accept_index[j] >= j goes to
// place j, so with j ascending no place is written before it is read, in blocks of kAhead too
// (a block's places are below all later nodes' numbers).  16 lanes make a row of 256 bytes.  Bound
// by its launch and one trip to memory: 2.5 us for one path of one layer, 3.1 us for 64 of 16 layers.
constexpr int kAhead = 8;

struct CompactParams {
  uint8_t* k;
  uint8_t* v;
  int32_t layers;
  int64_t layer_stride;
  int32_t num_pages;
  int32_t hkv;
  const int32_t* bt;
  int32_t max_pages;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  int32_t total_q;
  const int32_t* index;
  const int32_t* count;
  int32_t max_path;
  int32_t* new_lens;
  int32_t* status;
};

__global__ void __launch_bounds__(kCopyThreads)
cache_compact_kernel(const CompactParams p) {
  __shared__ int64_t s_from[MTP_TREE_MAX_NODES], s_to[MTP_TREE_MAX_NODES];
  const int b = blockIdx.y, t = threadIdx.x;
  const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], n = q1 - q0, L = p.seq_lens[b];
  const int m = p.count[b];
  int err = 0;
  if (q0 < 0 || q1 <= q0 || q1 > p.total_q || n > MTP_TREE_MAX_NODES) err = MTPATTN_ERR_QLEN;
  else if (n > L) err = MTPATTN_ERR_QLEN_GT_SEQ;
  else if (L > p.max_pages * kPage) err = MTPATTN_ERR_SEQ_TOO_LONG;   // (within 32 bits: checked by the host)
  else if (m < 0 || m >= n || m >= p.max_path) err = MTP_CACHE_ERR_LEN;
  const int start = L - n;
  int mine = 0;
  if (!err && t <= m) {
    const int32_t* path = p.index + static_cast<int64_t>(b) * p.max_path;
    const int node = path[t], before = t ? path[t - 1] : -1;
    if (node <= before || node >= n || (t == 0 && node != 0)) mine |= MTP_CACHE_ERR_LEN;
    else {
      const int32_t* row = p.bt + static_cast<int64_t>(b) * p.max_pages;
      const int a = start + node, z = start + t;
      const int pa = row[a / kPage], pz = row[z / kPage];
      if (pa < 0 || pa >= p.num_pages || pz < 0 || pz >= p.num_pages) mine |= MTPATTN_ERR_PAGE;
      s_from[t] = (static_cast<int64_t>(pa) * kPage + a % kPage) * p.hkv * kHeadDim;
      s_to[t] = (static_cast<int64_t>(pz) * kPage + z % kPage) * p.hkv * kHeadDim;
    }
  }
  err |= __syncthreads_or(mine & MTP_CACHE_ERR_LEN) ? MTP_CACHE_ERR_LEN : 0;
  err |= __syncthreads_or(mine & MTPATTN_ERR_PAGE) ? MTPATTN_ERR_PAGE : 0;
  if (blockIdx.x == 0 && t == 0) {
    p.new_lens[b] = err ? L : start + m + 1;
    if (err) set_status(p.status, err);
  }
  if (err) return;
  const int units = p.layers * 2 * p.hkv;          // rows of 256 bytes a token
  const int unit = blockIdx.x * (kCopyThreads / 16) + (t >> 4);
  if (unit >= units) return;
  const int layer = unit / (2 * p.hkv), rest = unit % (2 * p.hkv);
  uint8_t* base = ((rest & 1) ? p.v : p.k) + static_cast<int64_t>(layer) * p.layer_stride +
                  (rest >> 1) * kHeadDim + (t & 15) * 16;
  for (int j0 = 1; j0 <= m; j0 += kAhead) {
    uint4 x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (j0 + u <= m) x[u] = *reinterpret_cast<const uint4*>(base + s_from[j0 + u]);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (j0 + u <= m && s_from[j0 + u] != s_to[j0 + u])
        *reinterpret_cast<uint4*>(base + s_to[j0 + u]) = x[u];
  }
}

// ---- host side -----------------------------------------------------------------------------------

int check_caches(const void* k, const void* v, int32_t layers, int64_t layer_stride,
                 int64_t num_pages, int32_t hkv) {
  if (!k || !v || layers <= 0 || num_pages <= 0 || hkv <= 0) return MTPATTN_E_ARG;
  if (num_pages > MTP_CACHE_MAX_PAGES || hkv > 65535) return MTPATTN_E_UNSUPPORTED;
  if (!ptr_aligned(k, 16) || !ptr_aligned(v, 16)) return MTPATTN_E_ARG;
  const int64_t bytes = num_pages * kPage * hkv * kHeadDim;
  if (layers > 1 && (layer_stride < bytes || layer_stride % 16)) return MTPATTN_E_ARG;
  return MTPATTN_OK;
}

// A kernel has 48 KB of shared memory, its static part counted, unless it asks for more.  The plans ask
// once per device for the most that any takes (200 KB): a call that asked for its own size could take back
// what another host thread has just asked for, and is about to launch with.
constexpr int kMaxDevices = 64;
constexpr size_t kMostPlanSmem = plan_smem(true, MTP_CACHE_MAX_PAGES, MTP_CACHE_MAX_ROWS, MTP_CACHE_MAX_ROWS);
static_assert(kMostPlanSmem + 1024 <= 227 * 1024, "a plan's shared memory");
template <bool Fork>
cudaError_t allow_plan_smem(int device) {
  static std::atomic<bool> allowed[kMaxDevices];     // setting it twice is harmless
  if (allowed[device].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(cache_plan_kernel<Fork>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kMostPlanSmem));
  if (e != cudaSuccess) cudaGetLastError();
  else allowed[device].store(true, std::memory_order_release);
  return e;
}

template <bool Fork>
cudaError_t launch_plan(const PlanParams& p, int device, cudaStream_t stream) {
  if (const cudaError_t e = allow_plan_smem<Fork>(device); e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = plan_smem(Fork, p.num_pages, p.items, p.rows);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPlanCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, cache_plan_kernel<Fork>, p);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

cudaError_t launch_copy(const CopyParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.items, std::min(2 * p.layers, 65535));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.copies ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, cache_copy_kernel, p);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

int plan_and_copy(bool fork, PlanParams& p, CopyParams& c, void* workspace, size_t bytes,
                  int device, cudaStream_t stream) {
  const size_t need = mtp_cache_workspace_size(p.rows, p.max_pages);
  if (!workspace || !ptr_aligned(workspace, 256) || bytes < need) return MTPATTN_E_WORKSPACE;
  if (device < 0 || device >= kMaxDevices) return MTPATTN_E_DEVICE;
  const void* const ptrs[] = {c.k, c.v, p.bt, p.seq_lens, p.ref, workspace};
  if (!all_on_device(ptrs, device) || (p.status && !ptr_on_device(p.status, device)) ||
      (fork ? !ptr_on_device(p.src, device) || !ptr_on_device(p.dst, device)
            : !ptr_on_device(p.new_lens, device)))
    return MTPATTN_E_DEVICE;
  p.copies = static_cast<int2*>(workspace);
  c.copies = p.copies;
  c.items = p.items;
  if ((fork ? launch_plan<true>(p, device, stream) : launch_plan<false>(p, device, stream)) != cudaSuccess)
    return MTPATTN_E_LAUNCH;
  return launch_copy(c, stream) == cudaSuccess ? MTPATTN_OK : MTPATTN_E_LAUNCH;
}

int check_table(const int32_t* bt, int32_t max_pages, const int32_t* seq_lens, int32_t rows) {
  if (rows < 0 || max_pages < 0) return MTPATTN_E_ARG;
  if (rows > 0 && (!bt || !seq_lens || max_pages == 0)) return MTPATTN_E_ARG;
  if (!ptr_aligned(bt, 4) || !ptr_aligned(seq_lens, 4)) return MTPATTN_E_ARG;
  if (rows > MTP_CACHE_MAX_ROWS || max_pages > INT32_MAX / kPage) return MTPATTN_E_UNSUPPORTED;
  return MTPATTN_OK;
}

}  // namespace
}  // namespace mtpattn

using namespace mtpattn;

extern "C" size_t mtp_cache_workspace_size(int32_t num_rows, int32_t max_pages_per_seq) {
  if (num_rows < 0 || num_rows > MTP_CACHE_MAX_ROWS || max_pages_per_seq < 0) return 0;
  const size_t bytes = static_cast<size_t>(num_rows) * sizeof(int2);
  return (bytes + 255) / 256 * 256 + 256;
}

extern "C" int mtp_cache_resize(void* k_cache, void* v_cache, int32_t num_layers,
                                int64_t layer_stride, int64_t num_pages, int32_t num_kv_heads,
                                int32_t* block_tables, int32_t max_pages_per_seq,
                                int32_t* seq_lens, int32_t num_rows, int32_t* ref_counts,
                                const int32_t* new_lens, void* workspace, size_t workspace_bytes,
                                int32_t* status, void* stream) {
  int rc = check_caches(k_cache, v_cache, num_layers, layer_stride, num_pages, num_kv_heads);
  if (rc == MTPATTN_OK) rc = check_table(block_tables, max_pages_per_seq, seq_lens, num_rows);
  if (rc != MTPATTN_OK) return rc;
  if (num_rows == 0) return MTPATTN_OK;
  if (!ref_counts || !new_lens || words_overlap(new_lens, num_rows, seq_lens, num_rows) ||
      !ptr_aligned(ref_counts, 4) || !ptr_aligned(new_lens, 4) || !ptr_aligned(status, 4))
    return MTPATTN_E_ARG;
  PlanParams p{};
  p.bt = block_tables;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.rows = p.items = num_rows;
  p.ref = ref_counts;
  p.num_pages = static_cast<int32_t>(num_pages);
  p.new_lens = new_lens;
  p.status = status;
  CopyParams c{};
  c.k = static_cast<uint8_t*>(k_cache);
  c.v = static_cast<uint8_t*>(v_cache);
  c.layers = num_layers;
  c.layer_stride = layer_stride;
  c.num_pages = num_pages;
  c.page_bytes = static_cast<int64_t>(kPage) * num_kv_heads * kHeadDim;
  return plan_and_copy(false, p, c, workspace, workspace_bytes, current_device(),
                       static_cast<cudaStream_t>(stream));
}

extern "C" int mtp_cache_fork(void* k_cache, void* v_cache, int32_t num_layers,
                              int64_t layer_stride, int64_t num_pages, int32_t num_kv_heads,
                              int32_t* block_tables, int32_t max_pages_per_seq, int32_t* seq_lens,
                              int32_t num_rows, int32_t* ref_counts, const int32_t* src,
                              const int32_t* dst, int32_t num_pairs, void* workspace,
                              size_t workspace_bytes, int32_t* status, void* stream) {
  int rc = check_caches(k_cache, v_cache, num_layers, layer_stride, num_pages, num_kv_heads);
  if (rc == MTPATTN_OK) rc = check_table(block_tables, max_pages_per_seq, seq_lens, num_rows);
  if (rc != MTPATTN_OK) return rc;
  if (num_pairs < 0 || num_pairs > num_rows) return MTPATTN_E_ARG;
  if (num_pairs == 0) return MTPATTN_OK;
  if (!ref_counts || !src || !dst || !ptr_aligned(ref_counts, 4) || !ptr_aligned(src, 4) ||
      !ptr_aligned(dst, 4) || !ptr_aligned(status, 4))
    return MTPATTN_E_ARG;
  PlanParams p{};
  p.bt = block_tables;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.rows = num_rows;
  p.items = num_pairs;
  p.ref = ref_counts;
  p.num_pages = static_cast<int32_t>(num_pages);
  p.src = src;
  p.dst = dst;
  p.status = status;
  CopyParams c{};
  c.k = static_cast<uint8_t*>(k_cache);
  c.v = static_cast<uint8_t*>(v_cache);
  c.layers = num_layers;
  c.layer_stride = layer_stride;
  c.num_pages = num_pages;
  c.page_bytes = static_cast<int64_t>(kPage) * num_kv_heads * kHeadDim;
  return plan_and_copy(true, p, c, workspace, workspace_bytes, current_device(),
                       static_cast<cudaStream_t>(stream));
}

extern "C" int mtp_cache_copy_pages(void* k_cache, void* v_cache, int32_t num_layers,
                                    int64_t layer_stride, int64_t num_pages, int32_t num_kv_heads,
                                    const int32_t* src_pages, const int32_t* dst_pages,
                                    int32_t num_pairs, int32_t* status, void* stream) {
  const int rc = check_caches(k_cache, v_cache, num_layers, layer_stride, num_pages, num_kv_heads);
  if (rc != MTPATTN_OK) return rc;
  if (num_pairs < 0) return MTPATTN_E_ARG;
  if (num_pairs == 0) return MTPATTN_OK;
  if (!src_pages || !dst_pages || !ptr_aligned(src_pages, 4) || !ptr_aligned(dst_pages, 4) ||
      !ptr_aligned(status, 4))
    return MTPATTN_E_ARG;
  const int device = current_device();
  if (device < 0) return MTPATTN_E_DEVICE;
  const void* const ptrs[] = {k_cache, v_cache, src_pages, dst_pages};
  if (!all_on_device(ptrs, device) || (status && !ptr_on_device(status, device)))
    return MTPATTN_E_DEVICE;
  CopyParams c{};
  c.k = static_cast<uint8_t*>(k_cache);
  c.v = static_cast<uint8_t*>(v_cache);
  c.layers = num_layers;
  c.layer_stride = layer_stride;
  c.num_pages = num_pages;
  c.page_bytes = static_cast<int64_t>(kPage) * num_kv_heads * kHeadDim;
  c.src = src_pages;
  c.dst = dst_pages;
  c.items = num_pairs;
  c.status = status;
  return launch_copy(c, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MTPATTN_OK
                                                                          : MTPATTN_E_LAUNCH;
}

extern "C" int mtp_cache_compact(void* k_cache, void* v_cache, int32_t num_layers,
                                 int64_t layer_stride, int64_t num_pages, int32_t num_kv_heads,
                                 const int32_t* block_tables, int32_t max_pages_per_seq,
                                 const int32_t* seq_lens, const int32_t* cu_seqlens_q,
                                 int32_t num_seqs, int32_t total_q, const int32_t* accept_index,
                                 const int32_t* accept_len, int32_t max_path,
                                 int32_t* new_seq_lens, int32_t* status, void* stream) {
  int rc = check_caches(k_cache, v_cache, num_layers, layer_stride, num_pages, num_kv_heads);
  if (rc != MTPATTN_OK) return rc;
  if (num_seqs < 0 || total_q < 0 || max_pages_per_seq < 0 || max_path < 1) return MTPATTN_E_ARG;
  if (num_seqs == 0) return total_q == 0 ? MTPATTN_OK : MTPATTN_E_ARG;
  if (total_q < num_seqs || !block_tables || !seq_lens || !cu_seqlens_q || !accept_index ||
      !accept_len || !new_seq_lens || max_pages_per_seq == 0)
    return MTPATTN_E_ARG;
  if (!ptr_aligned(block_tables, 4) || !ptr_aligned(seq_lens, 4) || !ptr_aligned(cu_seqlens_q, 4) ||
      !ptr_aligned(accept_index, 4) || !ptr_aligned(accept_len, 4) ||
      !ptr_aligned(new_seq_lens, 4) || !ptr_aligned(status, 4))
    return MTPATTN_E_ARG;
  if (max_path > MTP_TREE_MAX_NODES || num_seqs > 65535 || max_pages_per_seq > INT32_MAX / kPage ||
      total_q > static_cast<int64_t>(num_seqs) * MTP_TREE_MAX_NODES ||
      static_cast<int64_t>(num_layers) * 2 * num_kv_heads > (1 << 28))
    return MTPATTN_E_UNSUPPORTED;
  // every CTA of a sequence reads its inputs, and one of them writes the new length
  const int64_t table_words = static_cast<int64_t>(num_seqs) * max_pages_per_seq;
  const int64_t path_words = static_cast<int64_t>(num_seqs) * max_path;
  if (words_overlap(new_seq_lens, num_seqs, seq_lens, num_seqs) ||
      words_overlap(new_seq_lens, num_seqs, accept_len, num_seqs) ||
      words_overlap(new_seq_lens, num_seqs, cu_seqlens_q, static_cast<int64_t>(num_seqs) + 1) ||
      words_overlap(new_seq_lens, num_seqs, accept_index, path_words) ||
      words_overlap(new_seq_lens, num_seqs, block_tables, table_words))
    return MTPATTN_E_ARG;
  const int device = current_device();
  if (device < 0) return MTPATTN_E_DEVICE;
  const void* const ptrs[] = {k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q,
                              accept_index, accept_len, new_seq_lens};
  if (!all_on_device(ptrs, device) || (status && !ptr_on_device(status, device)))
    return MTPATTN_E_DEVICE;
  CompactParams p{};
  p.k = static_cast<uint8_t*>(k_cache);
  p.v = static_cast<uint8_t*>(v_cache);
  p.layers = num_layers;
  p.layer_stride = layer_stride;
  p.num_pages = static_cast<int32_t>(num_pages);
  p.hkv = num_kv_heads;
  p.bt = block_tables;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.cu_q = cu_seqlens_q;
  p.total_q = total_q;
  p.index = accept_index;
  p.count = accept_len;
  p.max_path = max_path;
  p.new_lens = new_seq_lens;
  p.status = status;
  const int units = num_layers * 2 * num_kv_heads;
  const dim3 grid((units + kCopyThreads / 16 - 1) / (kCopyThreads / 16), num_seqs);
  cache_compact_kernel<<<grid, kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MTPATTN_OK : MTPATTN_E_LAUNCH;
}
