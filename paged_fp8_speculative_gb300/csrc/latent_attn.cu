// Latent attention over the paged cache (mtp_latent.h): the plain kernel.  A CTA has up to 8 heads of one
// new token, and goes over the sequence's keys 32 at a time with a running maximum and sum, everything in
// float32.
#include "common.cuh"
#include "host_checks.cuh"

#include "../../include/mtp_latent.h"

#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>
#include <atomic>

namespace mtpattn {
namespace {

constexpr int kRow = MTP_LATENT_ROW, kDim = MTP_LATENT_DIM;
constexpr int kPlainThreads = 128, kPlainRows = 8, kPlainKeys = 32;
constexpr int kPlainSmem = (kPlainRows + kPlainKeys) * kRow * 4 + kPlainRows * kPlainKeys * 4;

struct LatentParams {
  const __nv_bfloat16* q;
  int64_t q_stride_tok, q_stride_head;
  const uint8_t* cache;
  int64_t num_pages;
  const int32_t* block_tables;
  int32_t max_pages;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  const uint64_t* mask;
  int32_t num_seqs, total_q, heads;
  const float* descale;
  float scale_log2;
  __nv_bfloat16* out;
  int64_t out_stride_tok, out_stride_head;
  int32_t* status;
};

__global__ void __launch_bounds__(kPlainThreads) latent_plain_kernel(const LatentParams p) {
  extern __shared__ float smem[];
  float* s_q = smem;                                    // [8][576]
  float* s_k = s_q + kPlainRows * kRow;                 // [32][576]
  float* s_p = s_k + kPlainKeys * kRow;                 // [8][32]
  __shared__ float s_m[kPlainRows], s_l[kPlainRows], s_f[kPlainRows];
  const int b = blockIdx.x, i = blockIdx.y, h0 = blockIdx.z * kPlainRows, tid = threadIdx.x;
  const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], n = q1 - q0, L = p.seq_lens[b];
  if (q0 < 0 || q1 < q0 || q1 > p.total_q) {
    if (tid == 0 && i == 0) set_status(p.status, MTPATTN_ERR_QLEN);
    return;
  }
  int err = 0;
  if (n < 1 || n > MTP_LATENT_MAX_NODES) err = MTPATTN_ERR_QLEN;
  else if (n > L) err = MTPATTN_ERR_QLEN_GT_SEQ;
  else if (L > p.max_pages * kPage) err = MTPATTN_ERR_SEQ_TOO_LONG;
  const int rows = min(kPlainRows, p.heads - h0);
  const int32_t* bt = p.block_tables + static_cast<int64_t>(b) * p.max_pages;
  if (!err) {
    int bad = 0;
    for (int j = tid; j < (L + kPage - 1) / kPage; j += kPlainThreads) bad |= bt[j] < 0 || bt[j] >= p.num_pages;
    if (__syncthreads_or(bad)) err = MTPATTN_ERR_PAGE;
  }
  if (err) {
    if (tid == 0) set_status(p.status, err);
    for (int t = i; t < n; t += gridDim.y)
      for (int r = 0; r < rows; ++r)
        for (int d = tid; d < kDim; d += kPlainThreads)
          p.out[(q0 + t) * p.out_stride_tok + (h0 + r) * p.out_stride_head + d] = __float2bfloat16(0.f);
    return;
  }
  if (i >= n) return;
  for (int x = tid; x < rows * kRow; x += kPlainThreads)
    s_q[x] = __bfloat162float(p.q[(q0 + i) * p.q_stride_tok + (h0 + x / kRow) * p.q_stride_head + x % kRow]);
  __syncthreads();
  if (tid < kPlainRows) {
    s_m[tid] = -INFINITY;
    s_l[tid] = 0.f;
    if (tid < rows)
      for (int x = 0; x < kRow; ++x)
        if (!isfinite(s_q[tid * kRow + x])) s_l[tid] = NAN;
  }
  const float scale = p.scale_log2 * *p.descale;
  const uint64_t word = p.mask ? p.mask[q0 + i] : (2ull << i) - 1;
  float o[kPlainRows][4] = {};
  for (int j0 = 0; j0 < L; j0 += kPlainKeys) {
    __syncthreads();
    const int keys = min(kPlainKeys, L - j0);
    for (int x = tid; x < kPlainKeys * kRow; x += kPlainThreads) {
      const int j = j0 + x / kRow;
      float v = 0.f;
      if (j < L && (j < L - n || (word >> (j - L + n) & 1))) {
        __nv_fp8_e4m3 c;
        c.__x = p.cache[(static_cast<int64_t>(bt[j / kPage]) * kPage + j % kPage) * kRow + x % kRow];
        v = static_cast<float>(c);
      }
      s_k[x] = v;
    }
    __syncthreads();
    for (int x = tid; x < rows * kPlainKeys; x += kPlainThreads) {
      const int r = x / kPlainKeys, k = x % kPlainKeys, j = j0 + k;
      float s = -INFINITY;
      if (k < keys && (j < L - n || (word >> (j - L + n) & 1))) {
        s = 0.f;
        for (int d = 0; d < kRow; ++d) s += s_q[r * kRow + d] * s_k[k * kRow + d];
        s *= scale;
      }
      s_p[x] = s;
    }
    __syncthreads();
    if (tid < rows) {
      float top = s_m[tid], sum = 0.f;
      for (int k = 0; k < kPlainKeys; ++k) top = fmaxf(top, s_p[tid * kPlainKeys + k]);
      const float ref = top == -INFINITY ? 0.f : top;
      for (int k = 0; k < kPlainKeys; ++k) {
        const float e = exp2f(s_p[tid * kPlainKeys + k] - ref);
        s_p[tid * kPlainKeys + k] = e;
        sum += e;
      }
      s_f[tid] = exp2f(s_m[tid] - ref);
      s_l[tid] = s_l[tid] * s_f[tid] + sum;
      s_m[tid] = top;
    }
    __syncthreads();
    for (int r = 0; r < rows; ++r) {
      const float f = s_f[r];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float acc = o[r][c] * f;
        for (int k = 0; k < kPlainKeys; ++k) acc += s_p[r * kPlainKeys + k] * s_k[k * kRow + c * 128 + tid];
        o[r][c] = acc;
      }
    }
  }
  __syncthreads();
  for (int r = 0; r < rows; ++r) {
    const float l = s_l[r], w = l == 0.f ? 0.f : *p.descale / l;
    for (int c = 0; c < 4; ++c)
      p.out[(q0 + i) * p.out_stride_tok + (h0 + r) * p.out_stride_head + c * 128 + tid] =
          __float2bfloat16(l == 0.f ? 0.f : o[r][c] * w);
  }
}

}  // namespace
}  // namespace mtpattn

using namespace mtpattn;

extern "C" size_t mtp_latent_attn_workspace_size(int32_t num_seqs, int32_t total_q, int32_t num_heads,
                                                 int32_t max_pages_per_seq) {
  if (num_seqs < 0 || total_q < 0 || num_heads <= 0 || num_heads > MTP_LATENT_MAX_HEADS || max_pages_per_seq < 0)
    return 0;
  return device_sm_count(-1) > 0 ? 256 : 0;
}

extern "C" int mtp_latent_attn_fwd(const void* q, int64_t q_stride_tok, int64_t q_stride_head,
                                   const void* cache, int64_t num_pages, const int32_t* block_tables,
                                   int32_t max_pages_per_seq, const int32_t* seq_lens,
                                   const int32_t* cu_seqlens_q, const uint64_t* tree_mask, int32_t num_seqs,
                                   int32_t total_q, int32_t num_heads, const float* descale,
                                   float softmax_scale, void* workspace, size_t workspace_bytes, void* out,
                                   int64_t out_stride_tok, int64_t out_stride_head, int32_t* status,
                                   void* stream) {
  // 1. plain argument checks
  if (num_seqs < 0 || total_q < 0 || num_pages < 0 || max_pages_per_seq < 0 || num_heads <= 0)
    return MTPATTN_E_ARG;
  if (num_seqs == 0) return total_q == 0 ? MTPATTN_OK : MTPATTN_E_ARG;
  if (total_q < num_seqs) return MTPATTN_E_ARG;          // every sequence has a new token
  if (!q || !cache || !block_tables || !seq_lens || !cu_seqlens_q || !descale || !out || num_pages == 0 ||
      max_pages_per_seq == 0)
    return MTPATTN_E_ARG;
  if (!isfinite(softmax_scale)) return MTPATTN_E_ARG;
  if (q_stride_tok <= 0 || q_stride_head <= 0 || out_stride_tok <= 0 || out_stride_head <= 0 ||
      (q_stride_tok | q_stride_head | out_stride_tok | out_stride_head) % 8 != 0)
    return MTPATTN_E_ARG;
  if (!ptr_aligned(q, 16) || !ptr_aligned(out, 16) || !ptr_aligned(cache, 16) || !ptr_aligned(block_tables, 4) ||
      !ptr_aligned(seq_lens, 4) || !ptr_aligned(cu_seqlens_q, 4) || !ptr_aligned(tree_mask, 8) ||
      !ptr_aligned(descale, 4) || !ptr_aligned(status, 4))
    return MTPATTN_E_ARG;
  // 2. the supported envelope
  if (num_heads > MTP_LATENT_MAX_HEADS || total_q > static_cast<int64_t>(num_seqs) * MTP_LATENT_MAX_NODES ||
      num_pages > INT32_MAX || max_pages_per_seq > INT32_MAX / kPage - 8)
    return MTPATTN_E_UNSUPPORTED;
  // 3. the workspace
  const int device = current_device();
  if (device < 0 || device >= 64) return MTPATTN_E_DEVICE;
  const size_t need = mtp_latent_attn_workspace_size(num_seqs, total_q, num_heads, max_pages_per_seq);
  if (!workspace || !ptr_aligned(workspace, 256) || workspace_bytes < need) return MTPATTN_E_WORKSPACE;
  // 4. every pointer must be memory the kernels can read on the current device
  const void* const ptrs[] = {q, cache, block_tables, seq_lens, cu_seqlens_q, descale, workspace, out};
  if (!all_on_device(ptrs, device) || (tree_mask && !ptr_on_device(tree_mask, device)) ||
      (status && !ptr_on_device(status, device)))
    return MTPATTN_E_DEVICE;
  LatentParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride_tok = q_stride_tok;
  p.q_stride_head = q_stride_head;
  p.cache = static_cast<const uint8_t*>(cache);
  p.num_pages = num_pages;
  p.block_tables = block_tables;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.cu_q = cu_seqlens_q;
  p.mask = tree_mask;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.heads = num_heads;
  p.descale = descale;
  p.scale_log2 = softmax_scale * kLog2e;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.out_stride_tok = out_stride_tok;
  p.out_stride_head = out_stride_head;
  p.status = status;
  static std::atomic<bool> attr_set[64];               // per device; setting it twice is harmless
  if (!attr_set[device].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(latent_plain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlainSmem) !=
        cudaSuccess) {
      cudaGetLastError();
      return MTPATTN_E_LAUNCH;
    }
    attr_set[device].store(true, std::memory_order_release);
  }
  const dim3 grid(num_seqs, std::min(MTP_LATENT_MAX_NODES, total_q), (num_heads + kPlainRows - 1) / kPlainRows);
  latent_plain_kernel<<<grid, kPlainThreads, kPlainSmem, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MTPATTN_OK : MTPATTN_E_LAUNCH;
}
