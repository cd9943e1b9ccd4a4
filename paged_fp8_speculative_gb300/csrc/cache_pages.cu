// The paged cache's upkeep: pages handed out, shared, copied and given back, and the accepted
// tokens of a draft tree moved to their places (the entry points' rules are in
// include/mtp_cache.h).
//
// resize and fork run a planning kernel and a copying kernel.  The plan is one thread-block
// cluster, because every page handed out depends on all the counts below it: its CTAs first
// give pages back (resize), meet, count their part of the pool's free pages, exchange the
// counts through distributed shared memory, and then know each free page's rank; page of rank k
// goes to the k-th place wanted, found by a search over the rows' running sums of wants.  The
// pages to copy are left in the workspace, one (from, to) pair a row, for the copying kernel.
#include "common.cuh"
#include "host_checks.cuh"

#include "../../include/mtp_cache.h"
#include "../../include/mtp_tree.h"

#include <cooperative_groups.h>

#include <algorithm>

namespace cg = cooperative_groups;

namespace mtpattn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMaxPlanCtas = 8;
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
  int32_t* claim;            // workspace: [rows] (fork) the first pair that names a dst
  int32_t* status;
};

__device__ __forceinline__ int pages_of(int len) { return (len + kPage - 1) / kPage; }

// Inclusive running sums of want[0 .. n) in place, by the whole CTA; returns their total. Sums
// past 2^31 - 1 stay there: such a total is more than any pool has, and no sum is used then.
__device__ int64_t scan_wants(int* want, int n, int64_t* s_warp) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  int64_t carry = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    int64_t v = i0 + t < n ? want[i0 + t] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    int64_t below = carry, all = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
      if (w < warp) below += s_warp[w];
      all += s_warp[w];
    }
    if (i0 + t < n) want[i0 + t] = static_cast<int>(min(v + below, static_cast<int64_t>(INT32_MAX)));
    carry += all;
    __syncthreads();
  }
  return carry;
}

// What item i asks for.  resize: the row's pages beyond those it keeps, and a page for its last
// one if that is shared; fork: a page for the last, partly filled one.
struct Item {
  int row, from;             // the row that gets pages; fork: the row they are copied from
  int kept, len;             // tokens kept, tokens afterwards
  int tail;                  // the page to be copied, or -1
  int slot;                  // the table position of the first page handed out
  int want;
  bool live;
};

template <bool Fork>
__device__ __forceinline__ Item item_of(const PlanParams& p, int i) {
  Item x;
  x.live = true;
  x.tail = -1;
  x.want = 0;
  if (Fork) {
    x.from = p.src[i];
    x.row = p.dst[i];
    x.live = x.from >= 0 && x.from < p.rows && x.row >= 0 && x.row < p.rows && x.from != x.row &&
             p.seq_lens[x.row] == 0 && p.claim[x.row] == i;
    x.kept = x.len = x.live ? p.seq_lens[x.from] : 0;
    x.slot = x.kept / kPage;
    if (x.live && (x.len < 0 || x.len > static_cast<int64_t>(p.max_pages) * kPage)) {
      x.live = false;
      x.len = x.kept = x.slot = 0;
    }
    if (x.live && x.kept % kPage != 0) {
      x.tail = p.bt[static_cast<int64_t>(x.from) * p.max_pages + x.slot];
      x.want = 1;
    }
  } else {
    x.row = x.from = i;
    const int old = p.seq_lens[i];
    x.len = p.new_lens[i];
    const int64_t top = static_cast<int64_t>(p.max_pages) * kPage;
    x.live = old >= 0 && old <= top && x.len >= 0 && x.len <= top;
    if (!x.live) x.len = old;
    x.kept = min(old, x.len);
    x.slot = pages_of(x.kept);
    if (x.live) {
      x.want = pages_of(x.len) - x.slot;
      if (x.kept % kPage != 0) {
        const int page = p.bt[static_cast<int64_t>(i) * p.max_pages + x.slot - 1];
        if (page >= 0 && page < p.num_pages && p.ref[page] > 1) {
          x.tail = page;
          --x.slot;
          ++x.want;
        }
      }
    }
  }
  return x;
}

template <bool Fork>
__global__ void __launch_bounds__(kPlanThreads)
cache_plan_kernel(const PlanParams p) {
  extern __shared__ int s_want[];                  // running sums of the items' wants
  __shared__ int64_t s_warp[kPlanWarps];
  __shared__ int s_base[kPlanWarps];
  __shared__ int s_free[kMaxPlanCtas];
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), part = cluster.block_rank();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int gwarp = part * kPlanWarps + warp, gwarps = parts * kPlanWarps;
  const int gt = part * kPlanThreads + t, gthreads = parts * kPlanThreads;

  if (Fork) {
    // the first pair of a dst stands
    for (int i = gt; i < p.rows; i += gthreads) p.claim[i] = 0x7fffffff;
    __threadfence();
    cluster.sync();
    for (int i = gt; i < p.items; i += gthreads) {
      const int d = p.dst[i];
      if (d >= 0 && d < p.rows) atomicMin(&p.claim[d], i);
    }
    __threadfence();
    cluster.sync();
    // a source row with a bad entry: nobody's (a claim below 0 is no pair's)
    for (int i = gwarp; i < p.items; i += gwarps) {
      const int s = p.src[i], d = p.dst[i];
      bool bad = false;
      if (s >= 0 && s < p.rows && d >= 0 && d < p.rows) {
        const int len = p.seq_lens[s];
        const int n = len > 0 && len <= static_cast<int64_t>(p.max_pages) * kPage ? pages_of(len) : 0;
        for (int j = lane; j < n; j += 32) {
          const int page = p.bt[static_cast<int64_t>(s) * p.max_pages + j];
          bad |= page < 0 || page >= p.num_pages;
        }
        bad = __any_sync(0xffffffffu, bad);
        if (bad && lane == 0 && s != d && p.seq_lens[d] == 0 &&
            atomicCAS(&p.claim[d], i, -1) == i)
          set_status(p.status, MTPATTN_ERR_PAGE);
      }
    }
    __threadfence();
    cluster.sync();
  } else {
    // give the surplus pages back, a warp a row
    for (int i = gwarp; i < p.rows; i += gwarps) {
      const int old = p.seq_lens[i], len = p.new_lens[i];
      const int64_t top = static_cast<int64_t>(p.max_pages) * kPage;
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
    cluster.sync();
  }

  // the items' wants, every CTA for itself
  for (int i = t; i < p.items; i += kPlanThreads) s_want[i] = item_of<Fork>(p, i).want;
  __syncthreads();
  const int64_t total = scan_wants(s_want, p.items, s_warp);

  // this CTA's part of the pool, a contiguous piece a warp
  const int per = (p.num_pages + parts - 1) / parts;
  const int w_per = ((per + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
  const int64_t base = static_cast<int64_t>(part) * per;
  const int end = static_cast<int>(min(static_cast<int64_t>(p.num_pages), base + per));
  const int64_t w_lo64 = base + static_cast<int64_t>(warp) * w_per;
  const int w_lo = static_cast<int>(min(static_cast<int64_t>(end), w_lo64));
  const int w_hi = static_cast<int>(min(static_cast<int64_t>(end), w_lo64 + w_per));
  int count = 0;
  #pragma unroll 8
  for (int i = w_lo + lane; i < w_hi; i += 32) count += p.ref[i] == 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) count += __shfl_xor_sync(0xffffffffu, count, o);
  if (lane == 0) s_base[warp] = count;
  __syncthreads();
  if (t < parts) {
    int all = 0;
    for (int w = 0; w < kPlanWarps; ++w) all += s_base[w];
    *cluster.map_shared_rank(&s_free[part], t) = all;
  }
  cluster.sync();                                  // also: every item has been read
  int rank = 0, all_free = 0;                      // free pages before this warp's, of the pool
  for (int i = 0; i < parts; ++i) {
    if (i < part) rank += s_free[i];
    all_free += s_free[i];
  }
  for (int w = 0; w < warp; ++w) rank += s_base[w];
  const bool fits = total <= all_free;
  if (!fits && part == 0 && t == 0) set_status(p.status, MTP_CACHE_ERR_FULL);

  // What an item gets is written by the warps that hold the pages.  Nothing that item_of reads
  // changes meanwhile: copied pages take their places, and lengths change, afterwards.
  for (int i = gt; i < p.items; i += gthreads) p.copies[i] = make_int2(-1, -1);
  __threadfence();
  cluster.sync();
  if (fits && rank < total) {
    for (int i0 = w_lo; i0 < w_hi && rank < total; i0 += 32) {
      const int page = i0 + lane;
      const bool is_free = page < w_hi && p.ref[page] == 0;
      const uint32_t m = __ballot_sync(0xffffffffu, is_free);
      const int k = rank + __popc(m & ((1u << lane) - 1u));
      if (is_free && k < total) {
        int lo = 0, hi = p.items - 1;              // the first item whose running sum passes k
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (s_want[mid] > k) hi = mid; else lo = mid + 1;
        }
        const Item x = item_of<Fork>(p, lo);
        const int nth = k - (lo ? s_want[lo - 1] : 0);
        p.ref[page] = 1;
        if (x.tail >= 0 && nth == 0) p.copies[lo] = make_int2(x.tail, page);
        else p.bt[static_cast<int64_t>(x.row) * p.max_pages + x.slot + nth] = page;
      }
      rank += __popc(m);
    }
  }
  __threadfence();
  cluster.sync();
  // The copied pages take their places; shared pages are counted; lengths change last.
  if (Fork) {
    if (fits)
      for (int i = gwarp; i < p.items; i += gwarps) {
        const Item x = item_of<Fork>(p, i);
        if (!x.live) {
          const int s = p.src[i], d = p.dst[i];
          const bool known = s >= 0 && s < p.rows && d >= 0 && d < p.rows;
          const bool page_err = known && p.claim[d] == -1;
          const bool len_err = known && (p.seq_lens[s] < 0 || p.seq_lens[s] > static_cast<int64_t>(p.max_pages) * kPage);
          if (lane == 0 && !page_err) set_status(p.status, len_err ? MTP_CACHE_ERR_LEN : MTP_CACHE_ERR_ROW);
          continue;
        }
        const int32_t* from = p.bt + static_cast<int64_t>(x.from) * p.max_pages;
        int32_t* to = p.bt + static_cast<int64_t>(x.row) * p.max_pages;
        for (int j = lane; j < x.kept / kPage; j += 32) {
          const int page = from[j];
          to[j] = page;
          atomicAdd(&p.ref[page], 1);
        }
        if (x.tail >= 0 && lane == 0) to[x.slot] = p.copies[i].y;
      }
    // A thread has one pair at most; all lengths are read before the first is written (a
    // source row may be the dst of another pair).
    int row = -1, len = 0;
    if (fits && gt < p.items) {
      const Item x = item_of<Fork>(p, gt);
      if (x.live) {
        row = x.row;
        len = x.len;
      }
    }
    cluster.sync();
    if (row >= 0) p.seq_lens[row] = len;
  } else {
    for (int i = gt; i < p.rows; i += gthreads) {
      const int2 c = p.copies[i];
      const int old = p.seq_lens[i], len = p.new_lens[i];
      const int64_t top = static_cast<int64_t>(p.max_pages) * kPage;
      if (old < 0 || old > top || len < 0 || len > top) continue;
      if (c.x >= 0) {
        atomicSub(&p.ref[c.x], 1);
        p.bt[static_cast<int64_t>(i) * p.max_pages + (min(old, len) - 1) / kPage] = c.y;
      }
      p.seq_lens[i] = fits ? len : min(old, len);
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
// (a block's places are below all later nodes' numbers).  16 lanes make a row of 256 bytes.
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
  else if (pages_of(L) > p.max_pages) err = MTPATTN_ERR_SEQ_TOO_LONG;
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
  if (num_pages > INT32_MAX || hkv > 65535) return MTPATTN_E_UNSUPPORTED;
  if (!ptr_aligned(k, 16) || !ptr_aligned(v, 16)) return MTPATTN_E_ARG;
  const int64_t bytes = num_pages * kPage * hkv * kHeadDim;
  if (layers > 1 && (layer_stride < bytes || layer_stride % 16)) return MTPATTN_E_ARG;
  return MTPATTN_OK;
}

template <bool Fork>
cudaError_t launch_plan(const PlanParams& p, cudaStream_t stream) {
  // one CTA while its 32 warps hold the whole pool in a few loads each, else the largest
  // portable cluster
  const int parts = p.num_pages <= 4096 && p.rows <= 64 ? 1 : kMaxPlanCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.items) * sizeof(int);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, cache_plan_kernel<Fork>, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return e;
  }
  return cudaGetLastError();
}

cudaError_t launch_copy(const CopyParams& p, cudaStream_t stream) {
  const dim3 grid(p.items, std::min(2 * p.layers, 65535));
  cache_copy_kernel<<<grid, kCopyThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

int plan_and_copy(bool fork, PlanParams& p, CopyParams& c, void* workspace, size_t bytes,
                  int device, cudaStream_t stream) {
  const size_t need = mtp_cache_workspace_size(p.rows, p.max_pages);
  if (!workspace || !ptr_aligned(workspace, 256) || bytes < need) return MTPATTN_E_WORKSPACE;
  if (device < 0) return MTPATTN_E_DEVICE;
  const void* const ptrs[] = {c.k, c.v, p.bt, p.seq_lens, p.ref, workspace};
  if (!all_on_device(ptrs, device) || (p.status && !ptr_on_device(p.status, device)) ||
      (fork ? !ptr_on_device(p.src, device) || !ptr_on_device(p.dst, device)
            : !ptr_on_device(p.new_lens, device)))
    return MTPATTN_E_DEVICE;
  p.copies = static_cast<int2*>(workspace);
  p.claim = reinterpret_cast<int32_t*>(p.copies + p.rows);
  c.copies = p.copies;
  c.items = p.items;
  if ((fork ? launch_plan<true>(p, stream) : launch_plan<false>(p, stream)) != cudaSuccess)
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
  const size_t bytes = static_cast<size_t>(num_rows) * (sizeof(int2) + sizeof(int32_t));
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
  if (!ref_counts || !new_lens || new_lens == seq_lens || !ptr_aligned(ref_counts, 4) ||
      !ptr_aligned(new_lens, 4) || !ptr_aligned(status, 4))
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
      !accept_len || !new_seq_lens || new_seq_lens == seq_lens || max_pages_per_seq == 0)
    return MTPATTN_E_ARG;
  if (!ptr_aligned(block_tables, 4) || !ptr_aligned(seq_lens, 4) || !ptr_aligned(cu_seqlens_q, 4) ||
      !ptr_aligned(accept_index, 4) || !ptr_aligned(accept_len, 4) ||
      !ptr_aligned(new_seq_lens, 4) || !ptr_aligned(status, 4))
    return MTPATTN_E_ARG;
  if (max_path > MTP_TREE_MAX_NODES || num_seqs > 65535 || max_pages_per_seq > INT32_MAX / kPage ||
      total_q > static_cast<int64_t>(num_seqs) * MTP_TREE_MAX_NODES ||
      static_cast<int64_t>(num_layers) * 2 * num_kv_heads > (1 << 28))
    return MTPATTN_E_UNSUPPORTED;
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
