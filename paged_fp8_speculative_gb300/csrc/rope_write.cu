// Rotary positions, rounding to e4m3 and the way of new tokens into the paged caches: the three entry
// points of mtp_rope.h are one kernel over streams of rows (q, k, v; or a latent vector and its rotated part).
//
// Bound by the bytes: each input is read once, 16 bytes at a time, and each output written once.  A thread's
// item is 16 elements of a row: a run, or in the half layout two runs of 8 whose elements are each other's
// partners, so that q can be rotated in place.  All streams' items of a CTA's tokens are one list.  What the
// heads of a token share is worked out once per CTA, while the first items are on their way: the token's place
// in the cache (a warp a token, 32 boundaries of cu_seqlens_q at a time) and its sines and cosines.
//
// Angles are 64-bit fixed-point turns: position * freq modulo 2^64 drops whole turns exactly, and the
// upper 32 bits go to sincospif, rounded to float32 (2^-26 turns): as good at far positions as at near ones, no FP64.
#include "common.cuh"
#include "host_checks.cuh"

#include "../../include/mtp_latent.h"
#include "../../include/mtp_rope.h"
#include "../../include/mtp_tree.h"

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

namespace mtpattn {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxTokens = 8;              // tokens of a CTA: a warp looks each up
constexpr int kMaxPairs = 128;             // rotated pairs of a head
constexpr int kResident = 4;               // CTAs an SM holds
constexpr int kCtaItems = 16 * kRopeThreads;

enum Target { kRowsBf16, kRowsCodes, kPageCodes };

struct Stream {
  const void* src;
  int64_t s_tok, s_head;                   // elements
  void* dst;
  int64_t d_tok, d_head;                   // elements (bytes of codes); d_tok of a page: bytes a token
  const float* descale;
  int32_t end;                             // items a token of this stream and the ones before it
  int32_t row_items;                       // items a row: 16 elements each
  uint32_t row_inverse;                    // ceil(2^32 / row_items)
  int32_t rot0, rot;                       // first rotated element, how many
  int32_t target;
};
constexpr int kStreams = 4;

struct RopeParams {
  Stream s[kStreams];                      // those that are not there: no items
  int32_t total, tokens;                   // tokens a CTA
  const int32_t* positions;
  const int64_t* freqs;
  int32_t pairs;
  float mscale;
  // where tokens go (null: nothing goes to pages)
  const int32_t* bt;
  int32_t max_pages;
  int64_t num_pages;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  int32_t num_seqs;
  int32_t* status;
};

// 8 elements as they lie in memory.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) * 8 / 16];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) * 8 / 16); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
};
__device__ __forceinline__ void widen8(const Raw8<float>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(r.w[i].x);
    x[4 * i + 1] = __uint_as_float(r.w[i].y);
    x[4 * i + 2] = __uint_as_float(r.w[i].z);
    x[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}
__device__ __forceinline__ void widen8(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen8(const Raw8<__half>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store8_bf16(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// (a, b) * f in one instruction
__device__ __forceinline__ void scale_pair(float& a, float& b, float f) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(a), "+f"(b)
      : "f"(f));
}
__device__ __forceinline__ uint2 codes8(float (&x)[8], float scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    scale_pair(x[2 * i], x[2 * i + 1], scale);
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// The sequence of row t: the last b with cu[b] <= t (32 boundaries at a time), or -1 where row t is
// before cu[0] or not before cu[num_seqs].  All lanes get it.
__device__ int find_sequence(const int32_t* cu, int num_seqs, int t, int lane) {
  if (cu[0] > t || cu[num_seqs] <= t) return -1;
  int lo = 0, n = num_seqs;                // one of lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;       // lane 0's is known to be no later than t
    const bool before = lane * step < n && (lane == 0 || cu[at] <= t);
    const uint32_t all = __ballot_sync(0xffffffffu, before);
    const int last = 31 - __clz(all);      // (bit 0 is set)
    n = min(step, n - last * step);
    lo += last * step;
  }
  return lo;
}

// What is in s_place beside rows of the cache.
constexpr int64_t kNoPlace = -1, kNotOwned = -2;

__device__ __forceinline__ bool ascends(const RopeParams& p, int q0, int q1) { return q0 >= 0 && q0 <= q1 && q1 <= p.total; }

// The row of the cache that token t of sequence b goes to.
__device__ int64_t place_of(const RopeParams& p, int b, int t, int& err) {
  const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], len = p.seq_lens[b];
  if (!ascends(p, q0, q1) || q0 > t || q1 <= t) return kNotOwned;   // (boundaries out of order)
  if (q1 - q0 > len) {
    err = MTPATTN_ERR_QLEN_GT_SEQ;
  } else if (len > p.max_pages * kPage) {
    err = MTPATTN_ERR_SEQ_TOO_LONG;
  } else {
    const int at = len - (q1 - t);
    const int page = p.bt[static_cast<int64_t>(b) * p.max_pages + at / kPage];
    if (page >= 0 && page < p.num_pages) return static_cast<int64_t>(page) * kPage + at % kPage;
    err = MTPATTN_ERR_PAGE;
  }
  return kNoPlace;
}

// One item: where it comes from and goes to.
template <typename T, bool kInterleaved>
struct Item {
  Raw8<T> x, y;              // its 8 first elements, and the others
  int e, e2;                 // where they stand in the row
  int tok, k;                // token of the CTA, stream
  int64_t dst;               // of its row, but for the token's part
  bool rotated;

  // item i of the CTA's list
  __device__ __forceinline__ void fetch(const RopeParams& p, int i, int t0, int a_token) {
    tok = static_cast<int>(static_cast<float>(i) * (1.f / static_cast<float>(a_token)));   // off by one at most
    if (tok * a_token > i) --tok;
    else if ((tok + 1) * a_token <= i) ++tok;
    int j = i - tok * a_token;
    k = (j >= p.s[0].end) + (j >= p.s[1].end) + (j >= p.s[2].end);
    const Stream& s = p.s[k];
    if (k) j -= p.s[k - 1].end;
    const int head = static_cast<int>(__umulhi(j, s.row_inverse));   // (exact: j < 2^22, row_items <= 32)
    const int item = j - head * s.row_items;
    // half layout: the pairs of runs first, then what is not rotated
    e = 16 * item;
    e2 = e + 8;
    if (kInterleaved) {
      rotated = e >= s.rot0 && e < s.rot0 + s.rot;
    } else {
      rotated = 16 * item < s.rot;
      if (rotated) {
        e = s.rot0 + 8 * item;
        e2 = e + s.rot / 2;
      } else if (e - s.rot < s.rot0) {
        e -= s.rot;
        e2 -= s.rot;
      }
    }
    dst = head * s.d_head;
    const T* src = static_cast<const T*>(s.src) + (t0 + tok) * s.s_tok + head * s.s_head;
    x.load(src + e);
    y.load(src + e2);
  }
  // turn: of the item's token; at: the token's row of the output or the cache
  __device__ __forceinline__ void store(const RopeParams& p, const float2* turn, int64_t at) const {
    const Stream& s = p.s[k];
    float a[8], b[8];
    widen8(x, a);
    widen8(y, b);
    if (rotated) {
      const float4* c = reinterpret_cast<const float4*>(turn + (kInterleaved ? (e - s.rot0) / 2 : e - s.rot0));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = c[i];                       // cosine and sine of two pairs
        if (kInterleaved) {
          float(&v)[8] = i < 2 ? a : b;
          const int h = 4 * (i & 1);
          const float v0 = v[h], v1 = v[h + 1], v2 = v[h + 2], v3 = v[h + 3];
          v[h] = v0 * f.x - v1 * f.y;
          v[h + 1] = v1 * f.x + v0 * f.y;
          v[h + 2] = v2 * f.z - v3 * f.w;
          v[h + 3] = v3 * f.z + v2 * f.w;
        } else {
          const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
          a[2 * i] = a0 * f.x - b0 * f.y;
          b[2 * i] = b0 * f.x + a0 * f.y;
          a[2 * i + 1] = a1 * f.z - b1 * f.w;
          b[2 * i + 1] = b1 * f.z + a1 * f.w;
        }
      }
    }
    if (s.target == kRowsBf16) {
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(s.dst) + at * s.d_tok + dst;
      store8_bf16(out + e, a);
      store8_bf16(out + e2, b);
    } else {
      const float scale = 1.f / *s.descale;
      uint8_t* out = static_cast<uint8_t*>(s.dst) + at * s.d_tok + dst;
      const uint2 u = codes8(a, scale), v = codes8(b, scale);
      if (kInterleaved || !rotated) {
        *reinterpret_cast<uint4*>(out + e) = make_uint4(u.x, u.y, v.x, v.y);
      } else {
        *reinterpret_cast<uint2*>(out + e) = u;
        *reinterpret_cast<uint2*>(out + e2) = v;
      }
    }
  }
};

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kernel(const __grid_constant__ RopeParams p) {
  __shared__ alignas(16) float2 s_turn[kMaxTokens][kMaxPairs];    // mscale * (cos, sin)
  __shared__ int64_t s_place[kMaxTokens];             // row of the cache, kNoPlace or kNotOwned
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t0 = blockIdx.x * p.tokens;
  const int n = min(p.tokens, p.total - t0);
  const int a_token = p.s[kStreams - 1].end, items = n * a_token;
  const int stride = gridDim.y * kRopeThreads;
  int i = blockIdx.y * kRopeThreads + tid;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");   // what came before on the stream is done
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  Item<T, kInterleaved> it;
  if (i < items) it.fetch(p, i, t0, a_token);
  for (int j = tid; j < n * p.pairs; j += kRopeThreads) {
    const int tok = j / p.pairs, pair = j - tok * p.pairs;
    const int64_t m = p.positions[t0 + tok];
    const uint64_t turn = static_cast<uint64_t>(m) * static_cast<uint64_t>(p.freqs[pair]);
    // half turns in [-1, 1): the upper 32 bits, rounded
    const int32_t top = static_cast<int32_t>(static_cast<uint32_t>(turn >> 32));
    float sn, cs;
    sincospif(static_cast<float>(top) * 0x1p-31f, &sn, &cs);
    s_turn[tok][pair] = make_float2(cs * p.mscale, sn * p.mscale);
  }
  if (p.cu_q) {
    // Where the CTA's tokens go: a warp a token.  And boundaries out of order, which every CTA looks for: they are few,
    // and the first ones on their way with the search's (one user's call 2.95 us with and without; 1024 sequences of one
    // token 7.2 to 7.4, 5000 15.9 to 17.6).
    int err = 0, q0 = 0, q1 = 0;
    if (tid < p.num_seqs) {
      q0 = p.cu_q[tid];
      q1 = p.cu_q[tid + 1];
    }
    if (warp < n) {
      const int t = t0 + warp, b = find_sequence(p.cu_q, p.num_seqs, t, lane);
      const int64_t place = b < 0 ? kNotOwned : place_of(p, b, t, err);
      if (lane == 0) s_place[warp] = place;
    }
    bool disorder = !ascends(p, q0, q1);
    for (int b = tid + kRopeThreads; b < p.num_seqs; b += kRopeThreads) disorder |= !ascends(p, p.cu_q[b], p.cu_q[b + 1]);
    if (__syncthreads_or(disorder)) {
      // Then a search proves nothing: a token is the one sequence's that claims it, and unknown if that is not one alone.
      if (tid == 0) set_status(p.status, MTPATTN_ERR_QLEN);
      err = 0;
      if (warp < n) {
        const int t = t0 + warp;
        int claims = 0, owner = 0;
        for (int b = lane; b < p.num_seqs; b += 32) {
          const int from = p.cu_q[b], to = p.cu_q[b + 1];
          if (ascends(p, from, to) && from <= t && t < to) {
            ++claims;
            owner = b;
          }
        }
        claims = __reduce_add_sync(0xffffffffu, claims);
        owner = __reduce_max_sync(0xffffffffu, owner);
        const int64_t place = claims == 1 ? place_of(p, owner, t, err) : kNotOwned;
        if (lane == 0) s_place[warp] = place;
      }
      __syncthreads();
    }
    if (err && lane == 0) set_status(p.status, err);
  } else {
    __syncthreads();
  }
  while (i < items) {
    const Item<T, kInterleaved> now = it;
    i += stride;
    if (i < items) it.fetch(p, i, t0, a_token);      // the next one is on its way
    int64_t at = t0 + now.tok;
    if (p.cu_q) {
      const int64_t place = s_place[now.tok];
      if (place == kNotOwned) continue;
      if (p.s[now.k].target == kPageCodes) at = place;
    }
    if (at >= 0) now.store(p, s_turn[now.tok], at);
  }
}

// ---- host side -----------------------------------------------------------------------------------

bool rows_ok(const void* p, int64_t s_tok, int64_t s_head) {
  return p && ptr_aligned(p, 16) && s_tok > 0 && s_head > 0 && (s_tok | s_head) % 8 == 0;
}

// The next stream of a call.
void add(RopeParams& p, const void* src, int64_t s_tok, int64_t s_head, void* dst, int64_t d_tok, int64_t d_head,
         const float* descale, int32_t heads, int32_t dim, int32_t rot0, int32_t rot, Target target) {
  int k = 0;
  while (p.s[k].row_items) ++k;
  Stream& s = p.s[k];
  s.src = src;
  s.s_tok = s_tok;
  s.s_head = s_head;
  s.dst = dst;
  s.d_tok = d_tok;
  s.d_head = d_head;
  s.descale = descale;
  s.row_items = dim / 16;
  s.row_inverse = static_cast<uint32_t>(((1ull << 32) + s.row_items - 1) / s.row_items);
  s.rot0 = rot0;
  s.rot = rot;
  s.target = target;
  const int32_t end = (k ? p.s[k - 1].end : 0) + heads * s.row_items;
  for (; k < kStreams; ++k) p.s[k].end = end;
}

template <typename T>
cudaError_t launch_typed(RopeParams& p, dim3 grid, bool interleaved, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = interleaved ? cudaLaunchKernelEx(&cfg, rope_write_kernel<T, true>, p)
                                    : cudaLaunchKernelEx(&cfg, rope_write_kernel<T, false>, p);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

int launch_rope(RopeParams& p, int32_t dtype, bool interleaved, int device, void* stream) {
  const int sms = device_sm_count(device);
  if (sms <= 0) return MTPATTN_E_DEVICE;
  const int64_t a_token = p.s[kStreams - 1].end;
  // Several CTAs a token where there are few; several tokens a CTA where there are more than the GPU holds
  // CTAs at once, so that a CTA's start counts less, but not so many that its end does.
  const int64_t room = kResident * static_cast<int64_t>(sms);
  p.tokens = static_cast<int32_t>(std::max<int64_t>(
      1, std::min<int64_t>({kMaxTokens, kCtaItems / a_token, (p.total + room - 1) / room})));
  const int64_t slices = std::max<int64_t>(1, std::min((a_token + kRopeThreads - 1) / kRopeThreads, room / p.total));
  const dim3 grid((p.total + p.tokens - 1) / p.tokens, static_cast<unsigned>(slices));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MTP_F32    ? launch_typed<float>(p, grid, interleaved, st)
                        : dtype == MTP_BF16 ? launch_typed<__nv_bfloat16>(p, grid, interleaved, st)
                                            : launch_typed<__half>(p, grid, interleaved, st);
  return e == cudaSuccess ? MTPATTN_OK : MTPATTN_E_LAUNCH;
}

bool dtype_ok(int32_t dtype) { return dtype == MTP_F32 || dtype == MTP_BF16 || dtype == MTP_F16; }

// What both appending calls ask of their tables.
int check_tables(int64_t num_pages, const int32_t* bt, int32_t max_pages, const int32_t* lens,
                 const int32_t* cu, const int32_t* status) {
  if (!bt || !lens || !cu || num_pages <= 0 || max_pages <= 0) return MTPATTN_E_ARG;
  if (!ptr_aligned(bt, 4) || !ptr_aligned(lens, 4) || !ptr_aligned(cu, 4) || !ptr_aligned(status, 4))
    return MTPATTN_E_ARG;
  return MTPATTN_OK;
}

constexpr int kMaxHeads = 65535;

}  // namespace
}  // namespace mtpattn

using namespace mtpattn;

extern "C" int mtp_rope_freqs(const double* inv_freq, int32_t n, int64_t* freqs) {
  if (n < 0 || (n > 0 && (!inv_freq || !freqs))) return MTPATTN_E_ARG;
  for (int32_t i = 0; i < n; ++i)
    if (!(inv_freq[i] >= 0) || inv_freq[i] > 1048576.0) return MTPATTN_E_ARG;
  // 1 / (2 pi) as the sum of two doubles; the fraction of a turn in two pieces, the upper one a whole number of
  // 2^-32, and one rounding of the lower (in units of 2^-64: below 2^33, so summed to 2^-20 of one).  Every fma is
  // written out, so that no compiler's choice of them can change a bit.
  const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  for (int32_t i = 0; i < n; ++i) {
    const double a = inv_freq[i] * hi;
    const double b = fma(inv_freq[i], lo, fma(inv_freq[i], hi, -a));
    const double turns = a - floor(a);                             // exact
    const double whole = floor(ldexp(turns, 32)), part = turns - ldexp(whole, -32);   // exact
    const uint64_t f = (static_cast<uint64_t>(whole) << 32) +      // (below 2^32)
                       static_cast<uint64_t>(llrint(ldexp(part, 64) + ldexp(b, 64)));
    freqs[i] = static_cast<int64_t>(f);
  }
  return MTPATTN_OK;
}

extern "C" int mtp_rope_append(const void* q, int64_t q_stride_tok, int64_t q_stride_head, const void* k,
                               int64_t k_stride_tok, int64_t k_stride_head, const void* v,
                               int64_t v_stride_tok, int64_t v_stride_head, int32_t dtype,
                               const int32_t* positions, const int64_t* freqs, int32_t rot_dim,
                               int32_t interleaved, float mscale, void* k_cache, void* v_cache,
                               int64_t num_pages, const int32_t* block_tables, int32_t max_pages_per_seq,
                               const int32_t* seq_lens, const int32_t* cu_seqlens_q, int32_t num_seqs,
                               int32_t total_q, int32_t num_q_heads, int32_t num_kv_heads,
                               const float* k_descale, const float* v_descale, void* q_out,
                               int64_t q_out_stride_tok, int64_t q_out_stride_head, int32_t* status,
                               void* stream_) {
  // 1. plain argument checks
  if (num_seqs < 0 || total_q < 0 || num_pages < 0 || max_pages_per_seq < 0 || num_q_heads < 0 ||
      num_kv_heads <= 0 || rot_dim < 0 || !dtype_ok(dtype) || !isfinite(mscale))
    return MTPATTN_E_ARG;
  if (total_q == 0) return MTPATTN_OK;
  if (num_seqs == 0) return MTPATTN_E_ARG;
  if ((q != nullptr) != (num_q_heads > 0) || (rot_dim > 0 && !freqs)) return MTPATTN_E_ARG;
  if (!k_cache || !v_cache || k_cache == v_cache || !positions || !k_descale || !v_descale) return MTPATTN_E_ARG;
  int rc = check_tables(num_pages, block_tables, max_pages_per_seq, seq_lens, cu_seqlens_q, status);
  if (rc != MTPATTN_OK) return rc;
  if (!rows_ok(k, k_stride_tok, k_stride_head) || !rows_ok(v, v_stride_tok, v_stride_head)) return MTPATTN_E_ARG;
  if (q && (!rows_ok(q, q_stride_tok, q_stride_head) || !rows_ok(q_out, q_out_stride_tok, q_out_stride_head)))
    return MTPATTN_E_ARG;
  if (q && q_out == q &&
      (dtype != MTP_BF16 || q_out_stride_tok != q_stride_tok || q_out_stride_head != q_stride_head))
    return MTPATTN_E_ARG;
  if (!ptr_aligned(k_cache, 16) || !ptr_aligned(v_cache, 16) || !ptr_aligned(positions, 4) ||
      !ptr_aligned(freqs, 8) || !ptr_aligned(k_descale, 4) || !ptr_aligned(v_descale, 4))
    return MTPATTN_E_ARG;
  // 2. the supported envelope
  if (rot_dim % 16 || rot_dim > kHeadDim) return MTPATTN_E_UNSUPPORTED;
  if (num_pages > INT32_MAX || max_pages_per_seq > INT32_MAX / kPage || num_q_heads > kMaxHeads ||
      num_kv_heads > kMaxHeads)
    return MTPATTN_E_UNSUPPORTED;
  // 3. every pointer must be memory the kernels can reach on the current device
  const int device = current_device();
  if (device < 0) return MTPATTN_E_DEVICE;
  const void* const ptrs[] = {k, v, positions, k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q,
                              k_descale, v_descale};
  if (!all_on_device(ptrs, device) || (status && !ptr_on_device(status, device)) ||
      (rot_dim && !ptr_on_device(freqs, device)) ||
      (q && (!ptr_on_device(q, device) || !ptr_on_device(q_out, device))))
    return MTPATTN_E_DEVICE;
  const bool il = interleaved != 0;
  const int64_t row = static_cast<int64_t>(num_kv_heads) * kHeadDim;
  RopeParams p{};
  if (q)
    add(p, q, q_stride_tok, q_stride_head, q_out, q_out_stride_tok, q_out_stride_head, nullptr, num_q_heads, kHeadDim, 0,
        rot_dim, kRowsBf16);
  add(p, k, k_stride_tok, k_stride_head, k_cache, row, kHeadDim, k_descale, num_kv_heads, kHeadDim, 0, rot_dim, kPageCodes);
  add(p, v, v_stride_tok, v_stride_head, v_cache, row, kHeadDim, v_descale, num_kv_heads, kHeadDim, 0, 0, kPageCodes);
  p.total = total_q;
  p.positions = positions;
  p.freqs = freqs;
  p.pairs = rot_dim / 2;
  p.mscale = mscale;
  p.bt = block_tables;
  p.max_pages = max_pages_per_seq;
  p.num_pages = num_pages;
  p.seq_lens = seq_lens;
  p.cu_q = cu_seqlens_q;
  p.num_seqs = num_seqs;
  p.status = status;
  return launch_rope(p, dtype, il, device, stream_);
}

extern "C" int mtp_rope_latent_append(const void* q_rope, int64_t q_stride_tok, int64_t q_stride_head,
                                      const void* latent, int64_t latent_stride, const void* k_rope,
                                      int64_t k_rope_stride, int32_t dtype, const int32_t* positions,
                                      const int64_t* freqs, int32_t interleaved, float mscale, void* cache,
                                      int64_t num_pages, const int32_t* block_tables,
                                      int32_t max_pages_per_seq, const int32_t* seq_lens,
                                      const int32_t* cu_seqlens_q, int32_t num_seqs, int32_t total_q,
                                      int32_t num_heads, const float* descale, void* q_out,
                                      int64_t q_out_stride_tok, int64_t q_out_stride_head, int32_t* status,
                                      void* stream_) {
  if (num_seqs < 0 || total_q < 0 || num_pages < 0 || max_pages_per_seq < 0 || num_heads < 0 ||
      !dtype_ok(dtype) || !isfinite(mscale))
    return MTPATTN_E_ARG;
  if (total_q == 0) return MTPATTN_OK;
  if (num_seqs == 0) return MTPATTN_E_ARG;
  if ((q_rope != nullptr) != (num_heads > 0)) return MTPATTN_E_ARG;
  if (!cache || !positions || !freqs || !descale) return MTPATTN_E_ARG;
  int rc = check_tables(num_pages, block_tables, max_pages_per_seq, seq_lens, cu_seqlens_q, status);
  if (rc != MTPATTN_OK) return rc;
  if (!rows_ok(latent, latent_stride, 8) || !rows_ok(k_rope, k_rope_stride, 8)) return MTPATTN_E_ARG;
  if (q_rope && (!rows_ok(q_rope, q_stride_tok, q_stride_head) || !rows_ok(q_out, q_out_stride_tok, q_out_stride_head)))
    return MTPATTN_E_ARG;
  if (q_rope && q_out == q_rope &&
      (dtype != MTP_BF16 || q_out_stride_tok != q_stride_tok || q_out_stride_head != q_stride_head))
    return MTPATTN_E_ARG;
  if (!ptr_aligned(cache, 16) || !ptr_aligned(positions, 4) || !ptr_aligned(freqs, 8) || !ptr_aligned(descale, 4))
    return MTPATTN_E_ARG;
  if (num_pages > INT32_MAX || max_pages_per_seq > INT32_MAX / kPage || num_heads > kMaxHeads)
    return MTPATTN_E_UNSUPPORTED;
  const int device = current_device();
  if (device < 0) return MTPATTN_E_DEVICE;
  const void* const ptrs[] = {latent, k_rope, positions, freqs, cache, block_tables, seq_lens, cu_seqlens_q, descale};
  if (!all_on_device(ptrs, device) || (status && !ptr_on_device(status, device)) ||
      (q_rope && (!ptr_on_device(q_rope, device) || !ptr_on_device(q_out, device))))
    return MTPATTN_E_DEVICE;
  const bool il = interleaved != 0;
  RopeParams p{};
  if (q_rope)
    add(p, q_rope, q_stride_tok, q_stride_head, q_out, q_out_stride_tok, q_out_stride_head, nullptr, num_heads,
        MTP_LATENT_ROPE_DIM, 0, MTP_LATENT_ROPE_DIM, kRowsBf16);
  add(p, latent, latent_stride, 0, cache, MTP_LATENT_ROW, 0, descale, 1, MTP_LATENT_DIM, 0, 0, kPageCodes);
  add(p, k_rope, k_rope_stride, 0, static_cast<uint8_t*>(cache) + MTP_LATENT_DIM, MTP_LATENT_ROW, 0, descale, 1,
      MTP_LATENT_ROPE_DIM, 0, MTP_LATENT_ROPE_DIM, kPageCodes);
  p.total = total_q;
  p.positions = positions;
  p.freqs = freqs;
  p.pairs = MTP_LATENT_ROPE_DIM / 2;
  p.mscale = mscale;
  p.bt = block_tables;
  p.max_pages = max_pages_per_seq;
  p.num_pages = num_pages;
  p.seq_lens = seq_lens;
  p.cu_q = cu_seqlens_q;
  p.num_seqs = num_seqs;
  p.status = status;
  return launch_rope(p, dtype, il, device, stream_);
}

extern "C" int mtp_rope_prefill(const void* q, int64_t q_stride_tok, int64_t q_stride_head, const void* k,
                                int64_t k_stride_tok, int64_t k_stride_head, const void* k_rope,
                                int64_t k_rope_stride, const void* v, int64_t v_stride_tok,
                                int64_t v_stride_head, int32_t dtype, const int32_t* positions,
                                const int64_t* freqs, int32_t interleaved, float mscale, int32_t total,
                                int32_t num_q_heads, int32_t num_kv_heads, const float* q_descale,
                                const float* k_descale, const float* v_descale, void* q8, void* k8, void* v8,
                                void* stream_) {
  constexpr int kNope = 128, kRot = MTP_LATENT_ROPE_DIM, kQk = kNope + kRot, kV = 128;
  if (total < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || !dtype_ok(dtype) || !isfinite(mscale))
    return MTPATTN_E_ARG;
  if (total == 0) return MTPATTN_OK;
  if (!positions || !freqs || !q_descale || !k_descale || !v_descale || !q8 || !k8 || !v8) return MTPATTN_E_ARG;
  if (!rows_ok(q, q_stride_tok, q_stride_head) || !rows_ok(k, k_stride_tok, k_stride_head) ||
      !rows_ok(v, v_stride_tok, v_stride_head) || !rows_ok(k_rope, k_rope_stride, 8))
    return MTPATTN_E_ARG;
  if (!ptr_aligned(q8, 16) || !ptr_aligned(k8, 16) || !ptr_aligned(v8, 16) || !ptr_aligned(positions, 4) ||
      !ptr_aligned(freqs, 8) || !ptr_aligned(q_descale, 4) || !ptr_aligned(k_descale, 4) || !ptr_aligned(v_descale, 4))
    return MTPATTN_E_ARG;
  if (num_q_heads % num_kv_heads || num_q_heads > kMaxHeads) return MTPATTN_E_UNSUPPORTED;
  const int device = current_device();
  if (device < 0) return MTPATTN_E_DEVICE;
  const void* const ptrs[] = {q, k, k_rope, v, positions, freqs, q_descale, k_descale, v_descale, q8, k8, v8};
  if (!all_on_device(ptrs, device)) return MTPATTN_E_DEVICE;
  const bool il = interleaved != 0;
  RopeParams p{};
  const int64_t k_row = static_cast<int64_t>(num_kv_heads) * kQk;
  add(p, q, q_stride_tok, q_stride_head, q8, static_cast<int64_t>(num_q_heads) * kQk, kQk, q_descale, num_q_heads, kQk, kNope,
      kRot, kRowsCodes);
  add(p, k, k_stride_tok, k_stride_head, k8, k_row, kQk, k_descale, num_kv_heads, kNope, 0, 0, kRowsCodes);
  add(p, k_rope, k_rope_stride, 0, static_cast<uint8_t*>(k8) + kNope, k_row, kQk, k_descale, num_kv_heads, kRot, 0, kRot,
      kRowsCodes);
  add(p, v, v_stride_tok, v_stride_head, v8, static_cast<int64_t>(num_kv_heads) * kV, kV, v_descale, num_kv_heads, kV, 0, 0,
      kRowsCodes);
  p.total = total;
  p.positions = positions;
  p.freqs = freqs;
  p.pairs = kRot / 2;
  p.mscale = mscale;
  return launch_rope(p, dtype, il, device, stream_);
}
