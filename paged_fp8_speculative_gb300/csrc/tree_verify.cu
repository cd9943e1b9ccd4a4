// Verification of drafted tokens: the walk down the draft tree, greedy or by rejection
// sampling (the entry points' formulas are in include/mtp_tree.h).
//
// A thread-block cluster takes one sequence: the walk is sequential (a node's row is chosen by
// the step before), so what can be spread is the row, and only the rows on the path are read.
// Every CTA of the cluster holds the tree in shared memory and takes the same decisions; a
// row's scan is split over the CTAs, whose results meet through distributed shared memory.
//
// Rows are read in 16-byte blocks at the addresses' own alignment, whatever the row's: block k holds
// the elements k * kVec - skew .. + kVec - 1, skew being how far the row's start lies into one.  The
// blocks at the row's ends, which may not be whole, are read an element at a time.
#include "common.cuh"
#include "host_checks.cuh"

#include "../../include/mtp_tree.h"

#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include <algorithm>

namespace cg = cooperative_groups;

namespace mtpattn {
namespace {

constexpr int kVerifyThreads = 256, kVerifyCtas = 4;   // (an SM)
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kSampleThreads = 256, kSampleCtas = 2;   // (an SM)
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kNodes = MTP_TREE_MAX_NODES;
constexpr int kChunk = 512;                        // places whose sum is kept (sampling)

struct VerifyParams {
  const void* p;             // logits, or the target's probabilities
  const void* q;             // the drafter's probabilities, or null
  int64_t p_stride, q_stride;
  int32_t vocab;
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* cu_q;
  const float* u;
  int32_t total_q, max_path;
  int32_t* accept_index;
  int32_t* accept_len;
  int32_t* out_tokens;
  int32_t* status;
};

// The tree of one sequence and the path found so far; the same in every CTA of the cluster.
struct Walk {
  int32_t tok[kNodes], par[kNodes];
  uint64_t kids[kNodes];     // children of each node, one bit each
  int32_t path[kNodes];
  int n, q0;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// Loads and checks the sequence's tree; false (the same in every thread of the cluster) if it
// is not one, with the error outputs written.
__device__ bool load_tree(const VerifyParams& p, int b, bool first_cta, Walk& w) {
  const int t = threadIdx.x;
  const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1];
  int err = (q0 < 0 || q1 <= q0 || q1 > p.total_q || q1 - q0 > kNodes) ? MTPATTN_ERR_QLEN : 0;
  const int n = err ? 0 : q1 - q0;
  if (t < kNodes) w.kids[t] = 0;
  if (t == 0) {
    w.n = n;
    w.q0 = q0;
    w.path[0] = 0;
  }
  int bad_parent = 0;
  if (t < n) {
    w.tok[t] = p.tokens[q0 + t];
    w.par[t] = t == 0 ? -1 : p.parents[q0 + t];
    bad_parent = t > 0 && (w.par[t] < 0 || w.par[t] >= t);
  }
  if (__syncthreads_or(bad_parent)) err |= MTP_TREE_ERR_PARENT;
  if (err) {
    if (first_cta) {
      if (t == 0) {
        set_status(p.status, err);
        p.accept_len[b] = -1;
      }
      if (t < p.max_path) {
        p.accept_index[static_cast<int64_t>(b) * p.max_path + t] = -1;
        p.out_tokens[static_cast<int64_t>(b) * p.max_path + t] = -1;
      }
    }
    return false;
  }
  if (t > 0 && t < n)
    atomicOr(reinterpret_cast<unsigned long long*>(&w.kids[w.par[t]]), 1ull << t);
  __syncthreads();
  return true;
}

// The outputs of a finished walk of `count` accepted nodes.
__device__ void emit(const VerifyParams& p, int b, const Walk& w, int count, int next) {
  const int t = threadIdx.x;
  if (t == 0) {
    p.accept_len[b] = count;
    if (next < 0) set_status(p.status, MTP_TREE_ERR_ROW);
  }
  if (t < p.max_path) {
    const int64_t at = static_cast<int64_t>(b) * p.max_path + t;
    p.accept_index[at] = t <= count ? w.path[t] : -1;
    p.out_tokens[at] = t < count ? w.tok[w.path[t + 1]] : (t == count ? next : -1);
  }
}

// ---- rows ----------------------------------------------------------------------------------------

// A row of `vocab` elements in blocks of kVec (16 bytes).
template <class T>
struct RowOf {
  static constexpr int kVec = 16 / sizeof(T);
  const T* at;               // the row's first element, less skew: 16-byte aligned
  int skew, end;             // elements of the row: skew .. end - 1
  __device__ __forceinline__ RowOf(const T* row, int vocab) {
    skew = static_cast<int>(reinterpret_cast<uintptr_t>(row) / sizeof(T) % kVec);
    at = row - skew;
    end = skew + vocab;
  }
  // Whole blocks: first .. last - 1.
  __device__ __forceinline__ int first() const { return skew ? 1 : 0; }
  __device__ __forceinline__ int last() const { return end / kVec; }
  __device__ __forceinline__ uint4 block(int k) const { return __ldg(reinterpret_cast<const uint4*>(at) + k); }
};

// Element i of a block.
template <class T>
__device__ __forceinline__ float element(const uint4& v, int i);
template <>
__device__ __forceinline__ float element<float>(const uint4& v, int i) {
  return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
}
template <>
__device__ __forceinline__ float element<__nv_bfloat16>(const uint4& v, int i) {
  const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
  return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
}
template <>
__device__ __forceinline__ float element<__half>(const uint4& v, int i) {
  const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
  return __half2float(__ushort_as_half(static_cast<unsigned short>(i & 1 ? w >> 16 : w)));
}

// The largest element of a block, NaN passed over (NaN if there is nothing else).
__device__ __forceinline__ float top_of(const uint4& v, float) {
  return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
}
template <class T2>
__device__ __forceinline__ T2 pair_of(uint32_t w) {
  T2 p;
  memcpy(&p, &w, 4);
  return p;
}
__device__ __forceinline__ float top_of(const uint4& v, __nv_bfloat16) {
  const __nv_bfloat162 m = __hmax2(__hmax2(pair_of<__nv_bfloat162>(v.x), pair_of<__nv_bfloat162>(v.y)),
                                   __hmax2(pair_of<__nv_bfloat162>(v.z), pair_of<__nv_bfloat162>(v.w)));
  return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float top_of(const uint4& v, __half) {
  const __half2 m = __hmax2(__hmax2(pair_of<__half2>(v.x), pair_of<__half2>(v.y)),
                            __hmax2(pair_of<__half2>(v.z), pair_of<__half2>(v.w)));
  return fmaxf(__low2float(m), __high2float(m));
}

// ---- greedy --------------------------------------------------------------------------------------

// The order of float values as an order of unsigned numbers above 0, both zeros alike.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A thread looks at its whole blocks' largest elements, and keeps the block that first has the
// largest of them; where in it, is looked up once at the end.  kUnroll blocks are in flight: what
// bounds a step is that latency, then two meetings of the cluster: 1.5 us a row of 32000 tokens, 3 us
// where 64 sequences read rows of 256 KB from HBM (5.6 TB/s meanwhile).  The elements before the first
// and behind the last whole block, at most 2 kVec - 2, are a thread's each.
template <class T>
__global__ void __launch_bounds__(kVerifyThreads, kVerifyCtas)
verify_greedy_kernel(const VerifyParams p) {
  constexpr int kUnroll = 8, kVec = RowOf<T>::kVec;
  __shared__ Walk w;
  __shared__ uint64_t s_warp[kVerifyWarps];
  __shared__ uint64_t s_best[2][kMaxCluster];      // by step parity: the CTAs' best keys
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), part = cluster.block_rank();
  const int b = blockIdx.x / parts, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const bool ok = load_tree(p, b, part == 0, w);
  // every CTA of the cluster has to be running before its shared memory is written
  cluster.sync();
  if (!ok) return;
  int cur = 0, count = 0, next = -1;
  for (int step = 0;; ++step) {
    const RowOf<T> row(static_cast<const T*>(p.p) + static_cast<int64_t>(w.q0 + cur) * p.p_stride, p.vocab);
    const int first = row.first(), last = max(first, row.last()), per = (last - first + parts - 1) / parts;
    const int lo = min(last, first + part * per), hi = min(last, lo + per);
    auto key_of = [&](float x, int place) -> uint64_t {   // largest value, then lowest token
      return static_cast<uint64_t>(order_of(x)) << 32 | static_cast<uint32_t>(~(place - row.skew));
    };
    uint64_t key = 0;                              // 0: nothing but NaN
    if (part == 0) {
      const int place = t < kVec ? row.skew + t : last * kVec + t - kVec;   // before, and behind
      if (t < 2 * kVec && place < row.end && place >= row.skew && (t >= kVec || place < first * kVec)) {
        const float x = to_f32(row.at[place]);
        if (x == x) key = key_of(x, place);
      }
    }
    float best = -INFINITY;
    int at = lo + t;                               // (what -inf leaves: this thread's first block)
#pragma unroll 1
    for (int k0 = lo + t; k0 < hi; k0 += kUnroll * kVerifyThreads) {
      uint4 v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (k0 + u * kVerifyThreads < hi) v[u] = row.block(k0 + u * kVerifyThreads);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (k0 + u * kVerifyThreads < hi) {
          const float m = top_of(v[u], T(0.f));
          if (m > best) {                           // a thread's blocks ascend: ties keep the first
            best = m;
            at = k0 + u * kVerifyThreads;
          }
        }
    }
#pragma unroll 1
    for (int k = at, found = 0; k < hi && !found; k += kVerifyThreads) {   // (one block, unless best is -inf)
      const uint4 v = row.block(k);
#pragma unroll
      for (int i = kVec - 1; i >= 0; --i)
        if (element<T>(v, i) == best) found = i + 1;
      if (found) {
        const uint64_t x = key_of(best, k * kVec + found - 1);
        key = x > key ? x : key;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
      key = other > key ? other : key;
    }
    if (lane == 0) s_warp[warp] = key;
    __syncthreads();
    if (t < parts) {
      uint64_t k = 0;
      for (int i = 0; i < kVerifyWarps; ++i) k = s_warp[i] > k ? s_warp[i] : k;
      *cluster.map_shared_rank(&s_best[step & 1][part], t) = k;
    }
    cluster.sync();
    uint64_t k = 0;
    for (int i = 0; i < parts; ++i) k = s_best[step & 1][i] > k ? s_best[step & 1][i] : k;
    next = k ? static_cast<int>(~static_cast<uint32_t>(k)) : -1;
    if (next < 0 || count == p.max_path - 1) break;
    int child = -1;
    for (uint64_t m = w.kids[cur]; m && child < 0; m &= m - 1) {
      const int i = __ffsll(static_cast<long long>(m)) - 1;
      if (w.tok[i] == next) child = i;
    }
    if (child < 0) break;
    cur = child;
    ++count;
    if (t == 0) w.path[count] = cur;               // read behind later barriers only
  }
  __syncthreads();
  if (part == 0) emit(p, b, w, count, next);
}

// ---- sampling ------------------------------------------------------------------------------------
//
// w = max(p - S q, 0) is taken to a whole number of units of 2^-45, element by element, so sums are
// exact in 64 bits and the order of summation is free.  The number is made of two digits without a
// conversion instruction (these run at a quarter rate, and one to 64 bits at half of that): with
// w = d + e, d in f32 and e its error, the low 23 bits of 1 + d are d to units of 2^-23, and what
// that leaves, with e, is at most 2^-24 + 2^-25 and becomes the second digit as the low bits of
// r 2^45 + 3 * 2^22.  A lane's digits are summed in 32 bits over a chunk, offsets and all.  Steps
// that are the same for all elements are made for two at a time (f32x2): a sum costs 9 (S = 1) or 15
// instructions an element, and is bound by them once the rows are in L2.

struct Row {
  const void* p;
  const void* q;             // null: w = p
  uint64_t S;                // in units of 2^-45, as its parts are
  float s_hi, s_lo;          // S as the sum of two floats
  __device__ __forceinline__ void set(uint64_t s) {                      // (its 24 top bits, the rest)
    S = s;
    const int below = max(0, 40 - __clzll(static_cast<long long>(s)));
    const uint64_t top = s >> below;
    constexpr float kUnitS = 2.8421709430404007e-14f;                    // 2^-45
    s_hi = static_cast<float>(static_cast<uint32_t>(top)) * kUnitS * __uint_as_float((127u + below) << 23);
    s_lo = __ull2float_rn(s - (top << below)) * kUnitS;
  }
  // 0: w = p; 1: S = 1, what the first refusal leaves; 2: any S
  __device__ __forceinline__ int mode() const { return !q ? 0 : S == (1ull << 45) ? 1 : 2; }
};

constexpr uint32_t kDigitA = 0x3F800000u, kDigitB = 0x4B400000u;          // what w = 0 gives

// A node's number times the drafter's probability of its token, exactly: m 2^-e. The walk's comparisons
// are made in integers, by every thread: FP64 instructions take two lanes a clock, so that the 20 or so
// of a refusal, in 16 warps, were most of its 4.6 us (one sequence, 32000 tokens; 2.4 us without).
struct Product {
  uint64_t m;                // 48 bits
  int e;
};
__device__ __forceinline__ int scale_of(float x, uint32_t& m) {          // x >= 0 is m 2^-scale
  const uint32_t b = __float_as_uint(x), ex = b >> 23;
  m = (b & 0x7fffffu) | (ex ? 0x800000u : 0u);
  return 150 - static_cast<int>(max(ex, 1u));
}
__device__ __forceinline__ Product product_of(float u, float q) {
  uint32_t a, b;
  const int e = scale_of(u, a) + scale_of(q, b);
  return {static_cast<uint64_t>(a) * b, e};
}
// x < p, and x z < w for z, w in units of 2^-45
__device__ __forceinline__ bool below(const Product& x, float p) {
  uint32_t m;
  const int d = x.e - scale_of(p, m);
  if (d >= 0) return (d < 64 ? x.m >> d : 0) < m;
  return x.m == 0 ? m > 0 : x.m < (1u << 24) && d > -24 && x.m << -d < m;
}
__device__ __forceinline__ bool below(const Product& x, int64_t z, int64_t w) {
  const uint64_t lo = x.m * static_cast<uint64_t>(z), hi = __umul64hi(x.m, static_cast<uint64_t>(z));
  const uint64_t v = x.e >= 128 ? 0 : x.e >= 64 ? hi >> (x.e - 64) : lo >> x.e | hi << (64 - x.e);   // x.e >= 47
  return v < static_cast<uint64_t>(w);              // (neither is negative)
}

struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("{\n .reg .b64 ra, rb, rc;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mov.b64 rc, {%6, %7};\n"
      " fma.rn.f32x2 ra, ra, rb, rc;\n mov.b64 {%0, %1}, ra;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ F2 both(float x) { return {x, x}; }
__device__ __forceinline__ F2 add2(F2 a, F2 b) { return fma2(a, both(1.f), b); }
__device__ __forceinline__ F2 sub2(F2 a, F2 b) { return fma2(b, both(-1.f), a); }

// The digits of two elements added to (a, b).
template <int kMode>
__device__ __forceinline__ void add_left(const Row& r, F2 p, F2 q, uint32_t& a, uint32_t& b) {
  p = {__saturatef(p.x), __saturatef(p.y)};          // into [0, 1]; NaN as 0
  F2 d = p, e = both(0.f);
  if (kMode == 1) {
    q = {fminf(fmaxf(q.x, 0.f), p.x), fminf(fmaxf(q.y, 0.f), p.y)};      // p - min(q, p): never below 0
    d = sub2(p, q);
    e = sub2(sub2(p, d), q);                         // exact
  }
  if (kMode == 2) {
    q = {__saturatef(q.x), __saturatef(q.y)};
    const F2 s = both(r.s_hi), h = fma2(s, q, both(0.f));                // S q = h + l
    const F2 l = fma2(both(r.s_lo), q, fma2(s, q, {-h.x, -h.y}));
    d = sub2(p, h);
    e = sub2(sub2(sub2(p, d), h), l);                // exact but for l where d > 0
    const F2 w = add2(d, e);
    const bool some_x = w.x > 0.f && d.x >= 0.f, some_y = w.y > 0.f && d.y >= 0.f;
    d = {some_x ? d.x : 0.f, some_y ? d.y : 0.f};
    e = {some_x ? e.x : 0.f, some_y ? e.y : 0.f};
  }
  const F2 one = add2(d, both(1.f));
  F2 rest = sub2(d, sub2(one, both(1.f)));
  if (kMode != 0) rest = add2(rest, e);
  const F2 low = fma2(rest, both(35184372088832.f), both(12582912.f));   // 2^45, 3 * 2^22
  a += __float_as_uint(one.x);
  a += __float_as_uint(one.y);
  b += __float_as_uint(low.x);
  b += __float_as_uint(low.y);
}
__device__ __forceinline__ int64_t fixed_of(uint32_t a, uint32_t b, int n) {   // sums over n elements
  return (static_cast<int64_t>(a - static_cast<uint32_t>(n) * kDigitA) << 22) +
         static_cast<int32_t>(b - static_cast<uint32_t>(n) * kDigitB);
}
// One element (a second one of 0 beside it).
__device__ __noinline__ int64_t fixed_left(const Row& r, float p, float q) {
  uint32_t a = 0, b = 0;
  const int mode = r.mode();
  if (mode == 0) add_left<0>(r, {p, 0.f}, {0.f, 0.f}, a, b);
  else if (mode == 1) add_left<1>(r, {p, 0.f}, {q, 0.f}, a, b);
  else add_left<2>(r, {p, 0.f}, {q, 0.f}, a, b);
  return fixed_of(a, b, 2);
}

// Sums over the warp's lanes, by redux: of 64 bits; of the digits of up to 16 elements a lane.
__device__ __forceinline__ int64_t warp_sum(int64_t v) {
  const uint32_t a = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v) & 0xffffffu);
  const uint32_t b = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 24) & 0xffffffu);
  const uint32_t c = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 48));
  return static_cast<int64_t>((static_cast<uint64_t>(c) << 48) + (static_cast<uint64_t>(b) << 24) + a);
}
__device__ __forceinline__ int64_t warp_fixed(uint32_t a, uint32_t b, int n) {
  a -= static_cast<uint32_t>(n) * kDigitA;          // up to 2^27, |b| up to 3 2^24
  const uint32_t lo = __reduce_add_sync(0xffffffffu, a & 0xffffu), hi = __reduce_add_sync(0xffffffffu, a >> 16);
  const int32_t low = __reduce_add_sync(0xffffffffu, static_cast<int32_t>(b - static_cast<uint32_t>(n) * kDigitB));
  return (static_cast<int64_t>(hi) << 38) + (static_cast<int64_t>(lo) << 22) + low;
}
static_assert(kChunk / 32 <= 16);

// Sums of the CTA's chunks [c_lo, c_hi) of kChunk places into s_sum (index c - c_lo), a warp a chunk,
// its lanes taking blocks in turn; returns the sum of the warp's chunks.  Chunks are of the target's row in its own alignment; a chunk
// with a block that is not whole, or beside a drafter's row of another alignment, is read an
// element at a time.
template <class T, int kMode>
__device__ __noinline__ int64_t chunk_sums(const Row& r, int vocab, int c_lo, int c_hi, int64_t* s_sum) {
  constexpr int kVec = RowOf<T>::kVec, kBlocks = kChunk / kVec / 32;   // blocks a lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* P = static_cast<const T*>(r.p);
  const T* Q = static_cast<const T*>(r.q);
  const RowOf<T> rp(P, vocab);
  const RowOf<T> rq(kMode ? Q : P, vocab);
  const bool alike = rp.skew == rq.skew;
  int64_t all = 0;
#pragma unroll 1
  for (int c = c_lo + warp; c < c_hi; c += kSampleWarps) {
    uint32_t a = 0, b = 0;
    const int k0 = c * (kChunk / kVec);
    if (alike && k0 >= rp.first() && k0 + kChunk / kVec <= rp.last()) {
      uint4 pv[kBlocks], qv[kBlocks];
#pragma unroll
      for (int u = 0; u < kBlocks; ++u) pv[u] = rp.block(k0 + 32 * u + lane);
      if (kMode)
#pragma unroll
        for (int u = 0; u < kBlocks; ++u) qv[u] = rq.block(k0 + 32 * u + lane);
#pragma unroll
      for (int u = 0; u < kBlocks; ++u)
#pragma unroll
        for (int i = 0; i < kVec; i += 2)
          add_left<kMode>(r, {element<T>(pv[u], i), element<T>(pv[u], i + 1)},
                          kMode ? F2{element<T>(qv[u], i), element<T>(qv[u], i + 1)} : both(0.f), a, b);
    } else {
      const int i0 = c * kChunk - rp.skew + lane;
#pragma unroll 1
      for (int h = 0; h < kChunk / 32; h += 8) {
        float pv[8], qv[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int i = i0 + 32 * (h + u);
          const bool in = i >= 0 && i < vocab;
          pv[u] = in ? to_f32(P[i]) : 0.f;
          qv[u] = kMode && in ? to_f32(Q[i]) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 8; u += 2) add_left<kMode>(r, {pv[u], pv[u + 1]}, {qv[u], qv[u + 1]}, a, b);
      }
    }
    const int64_t sum = warp_fixed(a, b, kChunk / 32);
    if (lane == 0) s_sum[c - c_lo] = sum;
    all += sum;
  }
  return all;
}

// A refusal or draw over a row of one sequence takes 1.6 us, 1.2 us of them whatever the row's length
// (dependent steps: the meeting, the decision), up to 32000 tokens, 3.6 us at 131072; 64 sequences
// together are bound by the L2 cache (9 us a refusal, 7 TB/s), and a batch of trees by its longest
// path of refusals (64 trees of 26 nodes over 131072 tokens: 64 us).  256 threads twice an SM leave
// 128 registers a thread and half as many warps to repeat the decision; 512 threads twice: 68.6 us,
// 256 four times: 62.3 us but 7.2 instead of 6.5 us for a chain over 32000 tokens.  The next chunk
// loaded while one is summed made it slower (75 to 98 us): the loads of a chunk at once are enough,
// and the registers are not.
template <class T>
__global__ void __launch_bounds__(kSampleThreads, kSampleCtas)
verify_sample_kernel(const VerifyParams p) {
  extern __shared__ int64_t s_sum[];               // the CTA's chunk sums
  __shared__ Walk w;
  __shared__ float s_p[kNodes], s_q[kNodes], s_u[kNodes];   // p, q of each node's token, its number
  __shared__ Product s_x[kNodes];                  // u q of each node's token
  __shared__ int64_t s_part[2][kMaxCluster][kSampleWarps];   // by sum parity: the warps' sums
  constexpr int kSteps = kChunk / 32;              // 32 values a step, a warp a step
  static_assert(kSteps % kSampleWarps == 0);
  __shared__ int64_t s_step[kSteps];
  __shared__ int s_next;
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), part = cluster.block_rank();
  const int b = blockIdx.x / parts, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const bool ok = load_tree(p, b, part == 0, w);
  const T* P = static_cast<const T*>(p.p);
  const T* Q = static_cast<const T*>(p.q);
  if (ok) {
    if (t < w.n) {
      const int tok = w.tok[t];
      float pv = 0.f, qv = 1.f;
      if (t > 0 && tok >= 0 && tok < p.vocab) {
        const int64_t row = w.q0 + w.par[t];
        pv = __saturatef(to_f32(P[row * p.p_stride + tok]));
        if (Q) qv = __saturatef(to_f32(Q[row * p.q_stride + tok]));
      }
      s_p[t] = pv;
      s_q[t] = qv;
      // into [0, 1 - 2^-24]; NaN as 0
      const float u = fminf(fmaxf(p.u[w.q0 + t], 0.f), 0.999999940395355224609375f);
      s_u[t] = u;
      s_x[t] = product_of(u, qv);
    }
    if (t == 0) s_next = -1;
  }
  cluster.sync();                                  // also: every CTA is running
  if (!ok) return;
  int c_lo = 0, c_hi = 0;                          // the CTA's chunks of the row
  int sums = 0;                                    // sums taken so far
  // Sum of the row over the cluster; `before`: the sum of the CTAs ahead of this one.  Refused
  // tokens (without a drafter) are taken out of their chunks.
  uint64_t gone = 0;                               // refused children of the node, one bit each
  auto total_of = [&](const Row& r, int64_t& before) -> int64_t {
    const RowOf<T> rp(static_cast<const T*>(r.p), p.vocab);
    const int chunks = (rp.end + kChunk - 1) / kChunk, per = (chunks + parts - 1) >> (31 - __clz(parts));
    c_lo = min(chunks, part * per);
    c_hi = min(chunks, c_lo + per);
    const int mode = r.mode();
    int64_t mine = mode == 0   ? chunk_sums<T, 0>(r, p.vocab, c_lo, c_hi, s_sum)
                   : mode == 1 ? chunk_sums<T, 1>(r, p.vocab, c_lo, c_hi, s_sum)
                               : chunk_sums<T, 2>(r, p.vocab, c_lo, c_hi, s_sum);
    if (gone) {
      __syncthreads();
      if (warp == 0) {
        int64_t out = 0;
        for (uint64_t m = gone; m; m &= m - 1) {
          const int i = __ffsll(static_cast<long long>(m)) - 1;
          const int c = (w.tok[i] + rp.skew) / kChunk;
          if (c >= c_lo && c < c_hi) {
            const int64_t x = fixed_left(r, s_p[i], 0.f);
            if (lane == 0) s_sum[c - c_lo] -= x;
            out += x;
          }
        }
        mine -= out;
      }
    }
    if (lane < parts) cluster.map_shared_rank(&s_part[sums & 1][part][warp], lane)[0] = mine;
    cluster.sync();
    const int64_t* from = &s_part[sums & 1][0][0];
    int64_t x = 0, ahead = 0;
#pragma unroll
    for (int i = 0; i < kMaxCluster * kSampleWarps; i += 32)
      if (i + lane < parts * kSampleWarps) {
        const int64_t v = from[i + lane];
        x += v;
        if (i + lane < part * kSampleWarps) ahead += v;
      }
    before = warp_sum(ahead);
    ++sums;
    return warp_sum(x);
  };

  // The node the walk stands at, and what its refused children have left of its row.
  int cur = 0, count = 0;
  Row r;
  int64_t left;                                    // Z, what w sums to, in units of 2^-45
  float left_hi, left_lo;                          // (without a drafter: the sum of two floats)
  uint64_t kids;                                   // children not looked at yet
  auto arrive = [&](int node) {
    cur = node;
    r.p = P + static_cast<int64_t>(w.q0 + node) * p.p_stride;
    r.q = nullptr;
    r.set(0);
    gone = 0;
    left = 1ll << 45;
    left_hi = 1.f;
    left_lo = 0.f;
    kids = count == p.max_path - 1 ? 0ull : w.kids[node];
  };
  arrive(0);
  int64_t before, all;
  for (bool ended = false;;) {                     // (one place that takes sums: its code is large)
    bool sum = false;
    while (!sum && !ended) {
      if (!kids) {
        ended = true;
        break;
      }
      const int i = __ffsll(static_cast<long long>(kids)) - 1;
      kids &= kids - 1;
      const bool known = w.tok[i] >= 0 && w.tok[i] < p.vocab;
      bool accepted, again = !known;
      float wl = 0.f;
      if (Q) {                                     // u q Z < w
        accepted = known && (r.q ? below(s_x[i], left, fixed_left(r, s_p[i], s_q[i])) : below(s_x[i], s_p[i]));
      } else {                                     // u Z < w
        for (uint64_t m = gone; m; m &= m - 1)     // a token that has left the row already
          again |= w.tok[__ffsll(static_cast<long long>(m)) - 1] == w.tok[i];
        wl = again ? 0.f : s_p[i];
        const float u = s_u[i], h = __fmul_rn(u, left_hi), l = fmaf(u, left_lo, fmaf(u, left_hi, -h));
        accepted = known && __fadd_rn(h, -wl) + l < 0.f;   // (so Z stays above 0: refused, w <= u Z < Z)
      }
      if (accepted) {
        ++count;
        if (t == 0) w.path[count] = i;
        arrive(i);
      } else if (Q) {
        r.q = Q + static_cast<int64_t>(w.q0 + cur) * p.q_stride;
        const uint64_t add = static_cast<uint64_t>(left);
        r.set(r.S + add < r.S ? ~0ull : r.S + add);
        sum = kids != 0;
      } else {                                     // Z - w in two floats
        const float d = __fadd_rn(left_hi, -wl), v = __fadd_rn(d, -left_hi);
        const float e = __fadd_rn(__fadd_rn(left_hi, -__fadd_rn(d, -v)), -__fadd_rn(wl, v)) + left_lo;
        left_hi = __fadd_rn(d, e);
        left_lo = __fadd_rn(e, -__fadd_rn(left_hi, -d));
        if (!again) gone |= 1ull << i;
      }
    }
    all = total_of(r, before);
    if (!ended) left = all;
    else if (all == 0 && (r.q || gone)) {                // nothing left of the row: p itself
      r.q = nullptr;
      r.set(0);
      gone = 0;
    } else break;
  }
  // The final draw from w: the chunk where the running sum passes u sum, the element.
  if (all > 0) {
    // the running sum passes u * all where it passes floor(u * all)
    const uint64_t u64 = __float2ull_rz(s_u[0] * 18446744073709551616.f);     // u 2^64, exact
    const int64_t goal = static_cast<int64_t>(__umul64hi(u64, static_cast<uint64_t>(all)));
    // which of 32 values in a row passes the goal; at: the sum before lane 0, then before that value
    auto first_past = [&](int64_t v, int64_t& at) -> int {
      int64_t to = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, to, o);
        if (lane >= o) to += x;
      }
      const int k = __ffs(__ballot_sync(0xffffffffu, at + to > goal)) - 1;
      at += __shfl_sync(0xffffffffu, to - v, max(k, 0));
      if (k < 0) at += __shfl_sync(0xffffffffu, to, 31);
      return k;
    };
    int64_t run = before;                          // before the 32 chunks looked at
    int chunk = -1;
    if (before <= goal)
      for (int c0 = 0; c0 < c_hi - c_lo && chunk < 0; c0 += 32) {
        const int f = first_past(c0 + lane < c_hi - c_lo ? s_sum[c0 + lane] : 0, run);
        if (f >= 0) chunk = c0 + f;
      }
    if (chunk >= 0) {                              // the same in all warps: in this CTA, or not
      const T* rp = static_cast<const T*>(r.p);
      const T* rq = static_cast<const T*>(r.q);
      const RowOf<T> row(rp, p.vocab);
      const int i0 = (c_lo + chunk) * kChunk - row.skew + lane;
      int64_t v[kSteps / kSampleWarps];
#pragma unroll
      for (int h = 0; h < kSteps / kSampleWarps; ++h) {
        const int step = h * kSampleWarps + warp, i = i0 + 32 * step;
        const bool in = i >= 0 && i < p.vocab;
        v[h] = fixed_left(r, in ? to_f32(rp[i]) : 0.f, in && rq ? to_f32(rq[i]) : 0.f);
        for (uint64_t m = gone; m; m &= m - 1)
          if (w.tok[__ffsll(static_cast<long long>(m)) - 1] == i) v[h] = 0;
        const int64_t sum = warp_sum(v[h]);
        if (lane == 0) s_step[step] = sum;
      }
      __syncthreads();
      const int step = first_past(lane < kSteps ? s_step[lane] : 0, run);
#pragma unroll
      for (int h = 0; h < kSteps / kSampleWarps; ++h)
        if (step == h * kSampleWarps + warp) {
          const int nth = first_past(v[h], run);
          if (lane == 0 && nth >= 0) *cluster.map_shared_rank(&s_next, 0) = i0 + 32 * step + nth;
        }
    }
  }
  cluster.sync();                                  // s_next is in, and no CTA leaves before
  if (part == 0) emit(p, b, w, count, s_next);
}

// ---- host side -----------------------------------------------------------------------------------

// CTAs a sequence: as many as there is room for at per_sm CTAs an SM, each with 2048 elements of
// the row at least.  64 sequences over 131072 tokens (sampled, greedy; with 512 threads): 2 CTAs 104 and
// 18 us, 4 84 and 16, 8, more than the GPU holds at once, 98 and 27.  One sequence over 16384, 32000
// and 65536 tokens, four refusals or five greedy rows: with 8192 elements at least 14.6, 19.0, 14.6
// and 10.9, 13.2, 10.9 us; with 2048 11.7, 12.5, 14.6 and 10.1, 10.3, 10.9; with 512 the same, and at
// 4096 tokens 10.9 instead of 10.7.
int cluster_size(int num_seqs, int vocab, int per_sm) {
  const int sms = device_sm_count(-1);
  int c = 1;
  while (c < kMaxCluster && static_cast<int64_t>(num_seqs) * 2 * c <= per_sm * sms && vocab / (2 * c) >= 2048)
    c *= 2;
  return c;
}

template <class K>
cudaError_t launch(K kernel, const VerifyParams& p, int num_seqs, int threads, int cluster, size_t smem,
                   cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_seqs) * cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return e;
  }
  return cudaGetLastError();
}

// The checks both entry points share; MTPATTN_OK with *run = false for an empty batch.
int check(const void* rows, int64_t stride, int32_t dtype, int32_t vocab, const int32_t* tokens,
          const int32_t* parents, const int32_t* cu_q, int32_t num_seqs, int32_t total_q,
          int32_t max_path, const int32_t* accept_index, const int32_t* accept_len,
          const int32_t* out_tokens, const int32_t* status, bool* run) {
  *run = false;
  if (num_seqs < 0 || total_q < 0 || vocab <= 0 || max_path < 1) return MTPATTN_E_ARG;
  if (num_seqs == 0) return total_q == 0 ? MTPATTN_OK : MTPATTN_E_ARG;
  if (total_q < num_seqs || !rows || !tokens || !parents || !cu_q || !accept_index ||
      !accept_len || !out_tokens || stride < vocab)
    return MTPATTN_E_ARG;
  if (dtype != MTP_F32 && dtype != MTP_BF16 && dtype != MTP_F16) return MTPATTN_E_UNSUPPORTED;
  if (!ptr_aligned(rows, dtype == MTP_F32 ? 4 : 2) || !ptr_aligned(tokens, 4) ||
      !ptr_aligned(parents, 4) || !ptr_aligned(cu_q, 4) || !ptr_aligned(accept_index, 4) ||
      !ptr_aligned(accept_len, 4) || !ptr_aligned(out_tokens, 4) || !ptr_aligned(status, 4))
    return MTPATTN_E_ARG;
  if (total_q > static_cast<int64_t>(num_seqs) * kNodes || max_path > kNodes ||
      vocab > MTP_TREE_MAX_VOCAB || num_seqs > (1 << 24))
    return MTPATTN_E_UNSUPPORTED;
  const int device = current_device();
  if (device < 0) return MTPATTN_E_DEVICE;
  const void* const ptrs[] = {rows, tokens, parents, cu_q, accept_index, accept_len, out_tokens};
  if (!all_on_device(ptrs, device) || (status && !ptr_on_device(status, device)))
    return MTPATTN_E_DEVICE;
  *run = true;
  return MTPATTN_OK;
}

}  // namespace
}  // namespace mtpattn

using namespace mtpattn;

extern "C" int mtp_tree_verify_greedy(const void* logits, int32_t dtype, int64_t row_stride,
                                      int32_t vocab, const int32_t* draft_tokens,
                                      const int32_t* parents, const int32_t* cu_seqlens_q,
                                      int32_t num_seqs, int32_t total_q, int32_t max_path,
                                      int32_t* accept_index, int32_t* accept_len,
                                      int32_t* out_tokens, int32_t* status, void* stream) {
  bool run;
  const int rc = check(logits, row_stride, dtype, vocab, draft_tokens, parents, cu_seqlens_q,
                       num_seqs, total_q, max_path, accept_index, accept_len, out_tokens, status,
                       &run);
  if (rc != MTPATTN_OK || !run) return rc;
  VerifyParams p{};
  p.p = logits;
  p.p_stride = row_stride;
  p.vocab = vocab;
  p.tokens = draft_tokens;
  p.parents = parents;
  p.cu_q = cu_seqlens_q;
  p.total_q = total_q;
  p.max_path = max_path;
  p.accept_index = accept_index;
  p.accept_len = accept_len;
  p.out_tokens = out_tokens;
  p.status = status;
  const int c = cluster_size(num_seqs, vocab, kVerifyCtas);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == MTP_F32 ? launch(verify_greedy_kernel<float>, p, num_seqs, kVerifyThreads, c, 0, st)
      : dtype == MTP_BF16 ? launch(verify_greedy_kernel<__nv_bfloat16>, p, num_seqs, kVerifyThreads, c, 0, st)
                          : launch(verify_greedy_kernel<__half>, p, num_seqs, kVerifyThreads, c, 0, st);
  return e == cudaSuccess ? MTPATTN_OK : MTPATTN_E_LAUNCH;
}

extern "C" int mtp_tree_verify_sample(const void* target_probs, int64_t target_stride,
                                      const void* draft_probs, int64_t draft_stride, int32_t dtype,
                                      int32_t vocab, const int32_t* draft_tokens,
                                      const int32_t* parents, const int32_t* cu_seqlens_q,
                                      const float* uniforms, int32_t num_seqs, int32_t total_q,
                                      int32_t max_path, int32_t* accept_index, int32_t* accept_len,
                                      int32_t* out_tokens, int32_t* status, void* stream) {
  bool run;
  const int rc = check(target_probs, target_stride, dtype, vocab, draft_tokens, parents,
                       cu_seqlens_q, num_seqs, total_q, max_path, accept_index, accept_len,
                       out_tokens, status, &run);
  if (rc != MTPATTN_OK && rc != MTPATTN_E_DEVICE) return rc;
  if (rc == MTPATTN_OK && !run) return rc;
  if (!uniforms || !ptr_aligned(uniforms, 4) ||
      (draft_probs && (draft_stride < vocab || !ptr_aligned(draft_probs, dtype == MTP_F32 ? 4 : 2))))
    return MTPATTN_E_ARG;
  if (rc != MTPATTN_OK) return rc;
  const int device = current_device();
  if (device < 0 || !ptr_on_device(uniforms, device) ||
      (draft_probs && !ptr_on_device(draft_probs, device)))
    return MTPATTN_E_DEVICE;
  VerifyParams p{};
  p.p = target_probs;
  p.q = draft_probs;
  p.p_stride = target_stride;
  p.q_stride = draft_stride;
  p.vocab = vocab;
  p.tokens = draft_tokens;
  p.parents = parents;
  p.cu_q = cu_seqlens_q;
  p.u = uniforms;
  p.total_q = total_q;
  p.max_path = max_path;
  p.accept_index = accept_index;
  p.accept_len = accept_len;
  p.out_tokens = out_tokens;
  p.status = status;
  const int c = cluster_size(num_seqs, vocab, kSampleCtas);
  const int chunks = (vocab + 8 + kChunk - 1) / kChunk;   // (a row may start up to 7 places into a block)
  const size_t smem = static_cast<size_t>((chunks + c - 1) / c) * sizeof(int64_t);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == MTP_F32 ? launch(verify_sample_kernel<float>, p, num_seqs, kSampleThreads, c, smem, st)
      : dtype == MTP_BF16 ? launch(verify_sample_kernel<__nv_bfloat16>, p, num_seqs, kSampleThreads, c, smem, st)
                          : launch(verify_sample_kernel<__half>, p, num_seqs, kSampleThreads, c, smem, st);
  return e == cudaSuccess ? MTPATTN_OK : MTPATTN_E_LAUNCH;
}
