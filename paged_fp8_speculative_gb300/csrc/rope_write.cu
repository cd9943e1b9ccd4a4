// Rotary positions, rounding to e4m3 and the way of new tokens into the paged caches: the three entry
// points of mtp_rope.h are one kernel over streams of rows (q, k, v; or a latent vector and its rotated part).
//
// Bound by the bytes: each input is read once, in blocks of 8 elements, and each output written once (16
// bytes of bf16, 8 codes).  A thread's item is a block of 8 elements, or in the half layout the two blocks
// whose elements are each other's partners, so that q can be rotated in place.  What the heads of a token
// share is worked out once per CTA: the token's place in the cache (a warp a token, 32 boundaries of
// cu_seqlens_q at a time) and its sines and cosines.
//
// Angles are 64-bit fixed-point turns: position * freq modulo 2^64 drops whole turns exactly, and the
// upper 32 bits, at most 2^-33 turns off, go to sincospif: no loss at far positions, no FP64.
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

enum Target { kRowsBf16, kRowsCodes, kPageCodes };

struct Stream {
  const void* src;
  int64_t s_tok, s_head;                   // elements
  void* dst;
  int64_t d_tok, d_head;                   // elements (bytes of codes); d_tok of a page: bytes a token
  const float* descale;
  int32_t heads, blocks;                   // blocks of 8 elements a row
  int32_t items;                           // a row's: its blocks, less one for each pair of blocks
  int32_t rot0;                            // first rotated element; the rotated ones are rot_dim or none
  int32_t rot;
  int32_t target;
};

struct RopeParams {
  Stream s[4];
  int32_t streams;
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

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8<__half>(const __half* p, float (&x)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
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
__device__ __forceinline__ void store8_codes(uint8_t* p, const float (&x)[8], float scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * scale, x[2 * i + 1] * scale), __NV_SATFINITE,
                                    __NV_E4M3);
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
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

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads)
rope_write_kernel(const RopeParams p) {
  __shared__ float2 s_turn[kMaxTokens][kMaxPairs];    // mscale * (cos, sin)
  __shared__ int64_t s_place[kMaxTokens];             // row of the cache, -1: none
  __shared__ bool s_known[kMaxTokens];                // the token belongs to a sequence
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t0 = blockIdx.x * p.tokens;
  const int n = min(p.tokens, p.total - t0);
  if (warp < n) {
    const int t = t0 + warp;
    if (p.pairs) {
      const int64_t m = p.positions[t];
      for (int i = lane; i < p.pairs; i += 32) {
        const uint64_t turn = static_cast<uint64_t>(m) * static_cast<uint64_t>(p.freqs[i]);
        // half turns in [-1, 1): the upper 32 bits, rounded
        const int32_t top = static_cast<int32_t>(static_cast<uint32_t>(turn >> 32));
        float sn, cs;
        sincospif(static_cast<float>(top) * 0x1p-31f, &sn, &cs);
        s_turn[warp][i] = make_float2(cs * p.mscale, sn * p.mscale);
      }
    }
    if (p.cu_q) {
      const int b = find_sequence(p.cu_q, p.num_seqs, t, lane);
      if (lane == 0) {
        int64_t place = -1;
        bool known = false;
        int err = 0;
        if (b >= 0) {
          const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], len = p.seq_lens[b];
          if (q0 < 0 || q0 > t || q1 <= t || q1 > p.total) {
            err = MTPATTN_ERR_QLEN;
          } else {
            known = true;
            if (q1 - q0 > len) err = MTPATTN_ERR_QLEN_GT_SEQ;
            else if (len > p.max_pages * kPage) err = MTPATTN_ERR_SEQ_TOO_LONG;
            else {
              const int at = len - (q1 - t);
              const int page = p.bt[static_cast<int64_t>(b) * p.max_pages + at / kPage];
              if (page < 0 || page >= p.num_pages) err = MTPATTN_ERR_PAGE;
              else place = static_cast<int64_t>(page) * kPage + at % kPage;
            }
          }
        }
        if (err) set_status(p.status, err);
        s_place[warp] = place;
        s_known[warp] = known;
      }
    } else if (lane == 0) {
      s_known[warp] = true;
    }
  }
  __syncthreads();

  const int first = blockIdx.y * kRopeThreads + tid, stride = gridDim.y * kRopeThreads;
  for (int k = 0; k < p.streams; ++k) {
    const Stream& s = p.s[k];
    const int row_items = s.heads * s.items;
    float scale = 1.f;
    if (s.target != kRowsBf16) scale = 1.f / *s.descale;
    for (int j = first; j < n * row_items; j += stride) {
      const int tok = j / row_items, rest = j - tok * row_items;
      const int head = rest / s.items, item = rest - head * s.items;
      if (!s_known[tok] || (s.target == kPageCodes && s_place[tok] < 0)) continue;
      const T* src = static_cast<const T*>(s.src) + (t0 + tok) * s.s_tok + head * s.s_head;
      const int64_t out = (s.target == kPageCodes ? s_place[tok] : t0 + tok) * s.d_tok + head * s.d_head;
      // half layout: the pairs of blocks first, then the blocks outside the rotated part
      int e = item * 8, partner = -1;
      if (!kInterleaved && s.rot) {
        if (item < s.rot / 16) {
          e += s.rot0;
          partner = e + s.rot / 2;
        } else {
          e -= s.rot / 2;
          if (e >= s.rot0) e += s.rot;
        }
      }
      float x[8], y[8];
      load8(src + e, x);
      if (!kInterleaved && partner >= 0) {
        load8(src + partner, y);
        const float2* turn = &s_turn[tok][e - s.rot0];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 c = turn[i];
          const float a = x[i], b = y[i];
          x[i] = a * c.x - b * c.y;
          y[i] = b * c.x + a * c.y;
        }
        if (s.target == kRowsBf16) store8_bf16(static_cast<__nv_bfloat16*>(s.dst) + out + partner, y);
        else store8_codes(static_cast<uint8_t*>(s.dst) + out + partner, y, scale);
      }
      if (kInterleaved && e >= s.rot0 && e < s.rot0 + s.rot) {
        const float2* turn = &s_turn[tok][(e - s.rot0) / 2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 c = turn[i];
          const float a = x[2 * i], b = x[2 * i + 1];
          x[2 * i] = a * c.x - b * c.y;
          x[2 * i + 1] = b * c.x + a * c.y;
        }
      }
      if (s.target == kRowsBf16) store8_bf16(static_cast<__nv_bfloat16*>(s.dst) + out + e, x);
      else store8_codes(static_cast<uint8_t*>(s.dst) + out + e, x, scale);
    }
  }
}

// ---- host side -----------------------------------------------------------------------------------

bool rows_ok(const void* p, int64_t s_tok, int64_t s_head) {
  return p && ptr_aligned(p, 16) && s_tok > 0 && s_head > 0 && (s_tok | s_head) % 8 == 0;
}

Stream stream(const void* src, int64_t s_tok, int64_t s_head, void* dst, int64_t d_tok, int64_t d_head,
              const float* descale, int32_t heads, int32_t dim, int32_t rot0, int32_t rot, bool interleaved,
              Target target) {
  Stream s{};
  s.src = src;
  s.s_tok = s_tok;
  s.s_head = s_head;
  s.dst = dst;
  s.d_tok = d_tok;
  s.d_head = d_head;
  s.descale = descale;
  s.heads = heads;
  s.blocks = dim / 8;
  s.items = dim / 8 - (interleaved ? 0 : rot / 16);
  s.rot0 = rot0;
  s.rot = rot;
  s.target = target;
  return s;
}

template <typename T>
cudaError_t launch_typed(const RopeParams& p, dim3 grid, bool interleaved, cudaStream_t st) {
  if (interleaved) rope_write_kernel<T, true><<<grid, kRopeThreads, 0, st>>>(p);
  else rope_write_kernel<T, false><<<grid, kRopeThreads, 0, st>>>(p);
  return cudaGetLastError();
}

int launch_rope(RopeParams& p, int32_t dtype, bool interleaved, int device, void* stream) {
  int64_t items = 0;
  for (int k = 0; k < p.streams; ++k) items += static_cast<int64_t>(p.s[k].heads) * p.s[k].items;
  const int sms = device_sm_count(device);
  if (sms <= 0) return MTPATTN_E_DEVICE;
  p.tokens = 1;
  const int64_t slices = std::max<int64_t>(1, std::min<int64_t>((items + kRopeThreads - 1) / kRopeThreads,
                                                                 8 * sms / std::max(1, p.total)));
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
  // 1 / (2 pi) as the sum of two doubles; the fraction of a turn in two pieces, each a whole number of
  // 2^-64 after its rounding (explicit fma: the same on every host)
  const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  for (int32_t i = 0; i < n; ++i) {
    const double a = inv_freq[i] * hi;
    const double b = fma(inv_freq[i], hi, -a) + inv_freq[i] * lo;
    const double turns = a - floor(a);                             // exact
    const double whole = floor(ldexp(turns, 32)), part = turns - ldexp(whole, -32);   // exact
    uint64_t f = static_cast<uint64_t>(whole) << 32;               // (below 2^32)
    f += static_cast<uint64_t>(llrint(ldexp(part, 64)));           // below 2^32, exact but for the last bit
    f += static_cast<uint64_t>(llrint(ldexp(b, 64)));              // a few units, either sign
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
    p.s[p.streams++] = stream(q, q_stride_tok, q_stride_head, q_out, q_out_stride_tok, q_out_stride_head, nullptr,
                              num_q_heads, kHeadDim, 0, rot_dim, il, kRowsBf16);
  p.s[p.streams++] = stream(k, k_stride_tok, k_stride_head, k_cache, row, kHeadDim, k_descale, num_kv_heads,
                            kHeadDim, 0, rot_dim, il, kPageCodes);
  p.s[p.streams++] = stream(v, v_stride_tok, v_stride_head, v_cache, row, kHeadDim, v_descale, num_kv_heads,
                            kHeadDim, 0, 0, il, kPageCodes);
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
    p.s[p.streams++] = stream(q_rope, q_stride_tok, q_stride_head, q_out, q_out_stride_tok, q_out_stride_head,
                              nullptr, num_heads, MTP_LATENT_ROPE_DIM, 0, MTP_LATENT_ROPE_DIM, il, kRowsBf16);
  p.s[p.streams++] = stream(latent, latent_stride, 0, cache, MTP_LATENT_ROW, 0, descale, 1, MTP_LATENT_DIM, 0, 0,
                            il, kPageCodes);
  p.s[p.streams++] = stream(k_rope, k_rope_stride, 0, static_cast<uint8_t*>(cache) + MTP_LATENT_DIM, MTP_LATENT_ROW,
                            0, descale, 1, MTP_LATENT_ROPE_DIM, 0, MTP_LATENT_ROPE_DIM, il, kPageCodes);
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
  p.streams = 4;
  p.s[0] = stream(q, q_stride_tok, q_stride_head, q8, static_cast<int64_t>(num_q_heads) * kQk, kQk, q_descale,
                  num_q_heads, kQk, kNope, kRot, il, kRowsCodes);
  p.s[1] = stream(k, k_stride_tok, k_stride_head, k8, static_cast<int64_t>(num_kv_heads) * kQk, kQk, k_descale,
                  num_kv_heads, kNope, 0, 0, il, kRowsCodes);
  p.s[2] = stream(k_rope, k_rope_stride, 0, static_cast<uint8_t*>(k8) + kNope,
                  static_cast<int64_t>(num_kv_heads) * kQk, kQk, k_descale, num_kv_heads, kRot, 0, kRot, il, kRowsCodes);
  p.s[3] = stream(v, v_stride_tok, v_stride_head, v8, static_cast<int64_t>(num_kv_heads) * kV, kV, v_descale,
                  num_kv_heads, kV, 0, 0, il, kRowsCodes);
  p.total = total;
  p.positions = positions;
  p.freqs = freqs;
  p.pairs = kRot / 2;
  p.mscale = mscale;
  return launch_rope(p, dtype, il, device, stream_);
}
