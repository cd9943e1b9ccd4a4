// Attention of draft trees over the paged cache: the plain kernel.
//
// One CTA per (node, query head); its eight warps walk the keys of the sequence, a lane holding
// 8 of the 256 dims, each warp with its own running maximum and sum (one pass over the keys);
// the warps' partial results are merged by their maxima at the end.
#include "common.cuh"
#include "host_checks.cuh"

#include "../../include/mtp_tree.h"

#include <cuda_fp8.h>
#include <math.h>

namespace mtpattn {
namespace {

struct TreeAttnParams {
  const __nv_bfloat16* q;
  int64_t q_stride_tok, q_stride_head;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  int64_t num_pages;
  const int32_t* block_tables;
  int32_t max_pages;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  const uint64_t* mask;
  int32_t num_seqs, total_q, hq, hkv, ratio;
  const float* k_descale;
  const float* v_descale;
  float scale_log2;
  __nv_bfloat16* out;
  int64_t out_stride_tok, out_stride_head;
  int32_t* status;
};

constexpr int kWarps = 8;

__device__ __forceinline__ float e4m3_f32(uint8_t c) {
  __nv_fp8_e4m3 x;
  x.__x = c;
  return static_cast<float>(x);
}

__global__ void __launch_bounds__(kWarps * 32)
tree_attn_plain_kernel(const TreeAttnParams p) {
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][kHeadDim];
  __shared__ int s_bad;
  const int b = blockIdx.x / MTP_TREE_MAX_NODES, i = blockIdx.x % MTP_TREE_MAX_NODES;
  const int head = blockIdx.y, h = head / p.ratio;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1];
  if (q0 < 0 || q1 <= q0 || q1 > p.total_q) {
    if (i == 0 && head == 0 && threadIdx.x == 0) set_status(p.status, MTPATTN_ERR_QLEN);
    return;
  }
  const int n = q1 - q0, L = p.seq_lens[b];
  int err = 0;
  if (n > MTP_TREE_MAX_NODES) err = MTPATTN_ERR_QLEN;
  else if (n > L) err = MTPATTN_ERR_QLEN_GT_SEQ;
  else if ((L + kPage - 1) / kPage > p.max_pages) err = MTPATTN_ERR_SEQ_TOO_LONG;
  if (threadIdx.x == 0) s_bad = err;
  __syncthreads();
  const int32_t* bt = p.block_tables + static_cast<int64_t>(b) * p.max_pages;
  const int pages = err ? 0 : (L + kPage - 1) / kPage;
  for (int j = threadIdx.x; j < pages; j += kWarps * 32)
    if (bt[j] < 0 || bt[j] >= p.num_pages) atomicOr(&s_bad, MTPATTN_ERR_PAGE);
  __syncthreads();
  if (s_bad && i == 0 && head == 0 && threadIdx.x == 0) set_status(p.status, s_bad);
  // rows past the sequence's 64th node (too many nodes: an error) are zeroed by the slot mod 64
  for (int t = i; t < n; t += MTP_TREE_MAX_NODES) {
    __nv_bfloat16* orow = p.out + (int64_t)(q0 + t) * p.out_stride_tok + head * p.out_stride_head;
    if (s_bad) {
      if (threadIdx.x < kHeadDim) orow[threadIdx.x] = __float2bfloat16(0.f);
      continue;
    }
    const __nv_bfloat16* qrow = p.q + (int64_t)(q0 + t) * p.q_stride_tok + head * p.q_stride_head;
    float qv[8], o[8];
    const float sc = p.scale_log2 * __ldg(p.k_descale);
    for (int d = 0; d < 8; ++d) {
      qv[d] = __bfloat162float(qrow[8 * lane + d]);
      o[d] = 0.f;
    }
    const uint64_t see = p.mask[q0 + t];
    float m = -INFINITY, l = 0.f;
    for (int j = warp; j < L; j += kWarps) {
      const int node = j - (L - n);
      if (node >= 0 && !((see >> node) & 1)) continue;
      const int64_t off = ((static_cast<int64_t>(bt[j / kPage]) * kPage + j % kPage) * p.hkv + h) * kHeadDim + 8 * lane;
      const uint2 kw = *reinterpret_cast<const uint2*>(p.k_cache + off);
      const uint2 vw = *reinterpret_cast<const uint2*>(p.v_cache + off);
      float s = 0.f;
      for (int d = 0; d < 8; ++d) s += qv[d] * e4m3_f32((d < 4 ? kw.x : kw.y) >> (8 * (d & 3)) & 0xff);
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= sc;
      const float mn = s != s ? s : fmaxf(m, s);
      const float a = m == mn ? 1.f : exp2f(m - mn), e = s == mn ? 1.f : exp2f(s - mn);
      l = l * a + e;
      for (int d = 0; d < 8; ++d) o[d] = o[d] * a + e * e4m3_f32((d < 4 ? vw.x : vw.y) >> (8 * (d & 3)) & 0xff);
      m = mn;
    }
    if (lane == 0) {
      s_m[warp] = m;
      s_l[warp] = l;
    }
    for (int d = 0; d < 8; ++d) s_o[warp][8 * lane + d] = o[d];
    __syncthreads();
    if (threadIdx.x < kHeadDim) {
      float M = -INFINITY, lt = 0.f, ot = 0.f;
      for (int w = 0; w < kWarps; ++w) M = s_m[w] != s_m[w] ? s_m[w] : fmaxf(M, s_m[w]);
      for (int w = 0; w < kWarps; ++w)
        if (s_l[w] != 0.f) {
          const float e = exp2f(s_m[w] - M);
          lt += s_l[w] * e;
          ot += s_o[w][threadIdx.x] * e;
        }
      orow[threadIdx.x] = __float2bfloat16(lt == 0.f ? 0.f : ot / lt * __ldg(p.v_descale));
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(MTP_TREE_MAX_NODES)
tree_mask_kernel(const int32_t* parents, const int32_t* cu_q, int32_t total_q, uint64_t* mask,
                 int32_t* status) {
  __shared__ int32_t par[MTP_TREE_MAX_NODES];
  const int b = blockIdx.x, i = threadIdx.x;
  const int q0 = cu_q[b], q1 = cu_q[b + 1], n = q1 - q0;
  if (q0 < 0 || q1 <= q0 || q1 > total_q || n > MTP_TREE_MAX_NODES) {
    if (i == 0) set_status(status, MTPATTN_ERR_QLEN);
    return;
  }
  if (i < n) par[i] = i == 0 ? -1 : parents[q0 + i];
  __syncthreads();
  if (i >= n) return;
  // up the path; a node's parent has a smaller number, so at most n steps
  uint64_t word = 0;
  int at = i;
  while (true) {
    word |= 1ull << at;
    if (at == 0) break;
    const int up = par[at];
    if (up < 0 || up >= at) {
      set_status(status, MTP_TREE_ERR_PARENT);
      break;
    }
    at = up;
  }
  mask[q0 + i] = word;
}

}  // namespace
}  // namespace mtpattn

using namespace mtpattn;

extern "C" int mtp_tree_mask(const int32_t* parents, const int32_t* cu_seqlens_q, int32_t num_seqs,
                             int32_t total_q, uint64_t* mask, int32_t* status, void* stream) {
  if (num_seqs < 0 || total_q < 0) return MTPATTN_E_ARG;
  if (num_seqs == 0) return total_q == 0 ? MTPATTN_OK : MTPATTN_E_ARG;
  if (total_q < num_seqs || !parents || !cu_seqlens_q || !mask) return MTPATTN_E_ARG;
  if (!ptr_aligned(parents, 4) || !ptr_aligned(cu_seqlens_q, 4) || !ptr_aligned(mask, 8) ||
      !ptr_aligned(status, 4))
    return MTPATTN_E_ARG;
  if (total_q > static_cast<int64_t>(num_seqs) * MTP_TREE_MAX_NODES) return MTPATTN_E_UNSUPPORTED;
  const int device = current_device();
  if (device < 0) return MTPATTN_E_DEVICE;
  const void* const ptrs[] = {parents, cu_seqlens_q, mask};
  if (!all_on_device(ptrs, device) || (status && !ptr_on_device(status, device)))
    return MTPATTN_E_DEVICE;
  tree_mask_kernel<<<num_seqs, MTP_TREE_MAX_NODES, 0, static_cast<cudaStream_t>(stream)>>>(
      parents, cu_seqlens_q, total_q, mask, status);
  return cudaGetLastError() == cudaSuccess ? MTPATTN_OK : MTPATTN_E_LAUNCH;
}

extern "C" size_t mtp_tree_attn_workspace_size(int32_t num_seqs, int32_t total_q,
                                               int32_t num_q_heads, int32_t num_kv_heads,
                                               int32_t max_pages_per_seq) {
  if (num_seqs < 0 || total_q < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      max_pages_per_seq < 0 || num_q_heads % num_kv_heads)
    return 0;
  return 256;
}

extern "C" int mtp_tree_attn_fwd(const void* q, int64_t q_stride_tok, int64_t q_stride_head,
                                 const void* k_cache, const void* v_cache, int64_t num_pages,
                                 const int32_t* block_tables, int32_t max_pages_per_seq,
                                 const int32_t* seq_lens, const int32_t* cu_seqlens_q,
                                 const uint64_t* tree_mask, int32_t num_seqs, int32_t total_q,
                                 int32_t num_q_heads, int32_t num_kv_heads,
                                 const float* k_descale, const float* v_descale,
                                 float softmax_scale, void* workspace, size_t workspace_bytes,
                                 void* out, int64_t out_stride_tok, int64_t out_stride_head,
                                 int32_t* status, void* stream) {
  // 1. plain argument checks
  if (num_seqs < 0 || total_q < 0 || num_pages < 0 || max_pages_per_seq < 0 || num_q_heads <= 0 ||
      num_kv_heads <= 0)
    return MTPATTN_E_ARG;
  if (num_seqs == 0) return total_q == 0 ? MTPATTN_OK : MTPATTN_E_ARG;
  if (total_q < num_seqs) return MTPATTN_E_ARG;          // every sequence has its root
  if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !cu_seqlens_q || !tree_mask ||
      !k_descale || !v_descale || !out || num_pages == 0 || max_pages_per_seq == 0)
    return MTPATTN_E_ARG;
  if (!isfinite(softmax_scale)) return MTPATTN_E_ARG;
  if (q_stride_tok <= 0 || q_stride_head <= 0 || out_stride_tok <= 0 || out_stride_head <= 0 ||
      (q_stride_tok | q_stride_head | out_stride_tok | out_stride_head) % 8 != 0)
    return MTPATTN_E_ARG;
  if (!ptr_aligned(q, 16) || !ptr_aligned(out, 16) || !ptr_aligned(k_cache, 16) ||
      !ptr_aligned(v_cache, 16) || !ptr_aligned(block_tables, 4) || !ptr_aligned(seq_lens, 4) ||
      !ptr_aligned(cu_seqlens_q, 4) || !ptr_aligned(tree_mask, 8) || !ptr_aligned(k_descale, 4) ||
      !ptr_aligned(v_descale, 4) || !ptr_aligned(status, 4))
    return MTPATTN_E_ARG;
  // 2. the supported envelope
  if (num_q_heads % num_kv_heads) return MTPATTN_E_UNSUPPORTED;
  const int ratio = num_q_heads / num_kv_heads;
  if (ratio > MTP_TREE_MAX_RATIO) return MTPATTN_E_UNSUPPORTED;
  if (total_q > static_cast<int64_t>(num_seqs) * MTP_TREE_MAX_NODES) return MTPATTN_E_UNSUPPORTED;
  if (num_pages > INT32_MAX || max_pages_per_seq > INT32_MAX / kPage || num_q_heads > 65535)
    return MTPATTN_E_UNSUPPORTED;
  // 3. the workspace
  const int device = current_device();
  if (device < 0) return MTPATTN_E_DEVICE;
  const size_t need = mtp_tree_attn_workspace_size(num_seqs, total_q, num_q_heads, num_kv_heads,
                                                   max_pages_per_seq);
  if (!workspace || !ptr_aligned(workspace, 256) || workspace_bytes < need)
    return MTPATTN_E_WORKSPACE;
  // 4. every pointer must be memory the kernels can read on the current device
  const void* const ptrs[] = {q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q, tree_mask,
                              k_descale, v_descale, workspace, out};
  if (!all_on_device(ptrs, device) || (status && !ptr_on_device(status, device)))
    return MTPATTN_E_DEVICE;

  TreeAttnParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride_tok = q_stride_tok;
  p.q_stride_head = q_stride_head;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.num_pages = num_pages;
  p.block_tables = block_tables;
  p.max_pages = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.cu_q = cu_seqlens_q;
  p.mask = tree_mask;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.hq = num_q_heads;
  p.hkv = num_kv_heads;
  p.ratio = ratio;
  p.k_descale = k_descale;
  p.v_descale = v_descale;
  p.scale_log2 = softmax_scale * kLog2e;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.out_stride_tok = out_stride_tok;
  p.out_stride_head = out_stride_head;
  p.status = status;
  const dim3 grid(static_cast<unsigned>(num_seqs) * MTP_TREE_MAX_NODES, num_q_heads);
  tree_attn_plain_kernel<<<grid, kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MTPATTN_OK : MTPATTN_E_LAUNCH;
}
