// The Python binding of the draft-tree, cache, rotary and latent entry points (include/mtp_tree.h,
// include/mtp_cache.h, include/mtp_rope.h, include/mtp_latent.h): argument checks, the outputs that were
// not given, and the call.  These calls take 3 to 20 us on the GPU; the same steps in Python took 10 to 17 us of host time a call on a
// Grace core (an attribute of a tensor 0.1 us, torch.empty 1.6 us, a call through ctypes 1.5 us).
// Nothing is computed here.
//
// Functions take positional arguments only (the wrappers in api.py give them names, defaults and
// documentation); None stands for what is not given.  A refused argument is a ValueError, a status
// of the library the class that set_error was given, an error of torch's what torch makes of it.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "../../include/mtp_cache.h"
#include "../../include/mtp_latent.h"
#include "../../include/mtp_rope.h"
#include "../../include/mtp_tree.h"

namespace {

PyObject* g_error = nullptr;               // MtpAttnError

struct Refused {
  std::string what;
};

#define REFUSE_IF(cond, message) \
  do {                           \
    if (cond) throw Refused{message}; \
  } while (0)

const at::Tensor& tensor(PyObject* o, const char* name) {
  REFUSE_IF(!THPVariable_Check(o), std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
bool given(PyObject* o) { return o != Py_None; }

int32_t integer(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{std::string(name) + " must be an integer"};
  }
  REFUSE_IF(v < INT32_MIN || v > INT32_MAX, std::string(name) + " must be a 32-bit integer");
  return static_cast<int32_t>(v);
}

void vector(const at::Tensor& t, const char* name, int64_t n) {
  REFUSE_IF(t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous(),
            std::string(name) + " must be a contiguous int32 vector of " + std::to_string(n));
}
int32_t sequences(const at::Tensor& cu) {
  REFUSE_IF(cu.scalar_type() != at::kInt || cu.dim() != 1 || cu.size(0) < 1 || !cu.is_contiguous(),
            "cu_seqlens_q must be a contiguous int32 vector of num_seqs + 1");
  REFUSE_IF(cu.size(0) - 1 > INT32_MAX, "cu_seqlens_q is too long");
  return static_cast<int32_t>(cu.size(0) - 1);
}
void words(const at::Tensor& t, const char* name, int64_t n) {
  REFUSE_IF((t.scalar_type() != at::kLong && t.scalar_type() != at::kUInt64) || t.dim() != 1 ||
                t.size(0) != n || !t.is_contiguous(),
            std::string(name) + " must be a contiguous int64 vector, one word per node");
}
int32_t count32(int64_t n, const char* name) {
  REFUSE_IF(n > INT32_MAX, std::string(name) + " is too large");
  return static_cast<int32_t>(n);
}
const int32_t* ints(const at::Tensor& t) { return static_cast<const int32_t*>(t.const_data_ptr()); }
int32_t* ints_out(const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }
// A workspace is taken as the bytes from its first one on.
const at::Tensor& workspace_of(PyObject* o) {
  const at::Tensor& t = tensor(o, "workspace");
  REFUSE_IF(!t.is_contiguous(), "workspace must be contiguous");
  return t;
}
int32_t* status_of(PyObject* o) {
  if (!given(o)) return nullptr;
  const at::Tensor& t = tensor(o, "status");
  REFUSE_IF(t.scalar_type() != at::kInt || t.numel() < 1, "status must be an int32 tensor of one word");
  return static_cast<int32_t*>(t.data_ptr());
}

// The stream of a call on tensors of t's device: a handle, or the current one.  The library launches
// on the current device: tensors of another one are refused here, where the message can say so
// (CPU tensors by the library).
void* stream_of(PyObject* o, const at::Tensor& t) {
  if (t.is_cuda()) {
    const int now = c10::cuda::current_device();
    REFUSE_IF(t.get_device() != now, "tensors are on cuda:" + std::to_string(t.get_device()) +
                                         ", the current device is cuda:" + std::to_string(now));
  }
  if (given(o)) {
    void* h = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused{"stream must be a torch.cuda.Stream or a handle"};
    }
    return h;
  }
  return t.is_cuda() ? static_cast<void*>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream()) : nullptr;
}

PyObject* finish(int rc, PyObject* result) {       // steals result
  if (rc == MTPATTN_OK) return result;
  Py_XDECREF(result);
  PyObject* e = g_error ? PyObject_CallFunction(g_error, "i", rc) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_Format(PyExc_RuntimeError, "mtpattn status %d", rc);
  }
  return nullptr;
}

// A Python function from one that throws.
template <PyObject* (*kBody)(PyObject* const*)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t) {
  try {
    return kBody(args);
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
  } catch (const std::exception&) {              // torch's own: torch.OutOfMemoryError among them
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}
template <PyObject* (*kBody)(PyObject* const*), int kArgs>
PyObject* entry(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%d arguments are wanted, not %zd", kArgs, n);
    return nullptr;
  }
  return guarded<kBody>(self, args, n);
}

// ---- draft trees ---------------------------------------------------------------------------------

// parents, cu_seqlens_q, out, status, stream
PyObject* tree_mask(PyObject* const* a) {
  const at::Tensor &parents = tensor(a[0], "parents"), &cu = tensor(a[1], "cu_seqlens_q");
  const int64_t total = parents.numel();
  vector(parents, "parents", total);
  const int32_t seqs = sequences(cu);
  void* stream = stream_of(a[4], parents);
  at::Tensor out = given(a[2]) ? tensor(a[2], "out") : at::empty({total}, parents.options().dtype(at::kLong));
  words(out, "out", total);
  const int rc = mtp_tree_mask(ints(parents), ints(cu), seqs, count32(total, "parents"),
                               static_cast<uint64_t*>(out.data_ptr()), status_of(a[3]), stream);
  return finish(rc, rc ? nullptr : THPVariable_Wrap(std::move(out)));
}

bool is_codes(at::ScalarType t) { return t == at::kByte || t == at::kFloat8_e4m3fn; }

// q, k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q, tree_mask, k_descale, v_descale,
// softmax_scale, out, workspace, status, stream
PyObject* tree_attn(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_cache"), &v = tensor(a[2], "v_cache");
  const at::Tensor &table = tensor(a[3], "block_tables"), &lens = tensor(a[4], "seq_lens");
  const at::Tensor &cu = tensor(a[5], "cu_seqlens_q"), &mask = tensor(a[6], "tree_mask");
  const at::Tensor &kd = tensor(a[7], "k_descale"), &vd = tensor(a[8], "v_descale");
  void* stream = stream_of(a[13], q);
  REFUSE_IF(q.scalar_type() != at::kBFloat16 || q.dim() != 3 || q.size(2) != MTPATTN_HEAD_DIM || q.stride(2) != 1,
            "q must be bf16 [total_q, H_q, 256] with unit stride on head_dim");
  REFUSE_IF(!is_codes(k.scalar_type()) || v.scalar_type() != k.scalar_type(),
            "k_cache / v_cache must be uint8 or float8_e4m3fn codes");
  REFUSE_IF(k.dim() != 4 || k.size(1) != MTPATTN_PAGE_SIZE || k.size(3) != MTPATTN_HEAD_DIM,
            "k_cache must be [num_pages, 16, H_kv, 256]");
  REFUSE_IF(v.sizes() != k.sizes() || !k.is_contiguous() || !v.is_contiguous(),
            "k_cache and v_cache must be contiguous and of the same shape");
  const int32_t total = count32(q.size(0), "q"), hq = count32(q.size(1), "q"), hkv = count32(k.size(2), "k_cache");
  const int32_t seqs = sequences(cu);
  vector(lens, "seq_lens", seqs);
  REFUSE_IF(table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != seqs || !table.is_contiguous(),
            "block_tables must be a contiguous int32 [B, max_pages] tensor");
  const int32_t width = count32(table.size(1), "block_tables");
  words(mask, "tree_mask", total);
  REFUSE_IF(kd.scalar_type() != at::kFloat || kd.numel() != 1, "k_descale must be a 1-element float32 tensor");
  REFUSE_IF(vd.scalar_type() != at::kFloat || vd.numel() != 1, "v_descale must be a 1-element float32 tensor");
  const double scale = PyFloat_AsDouble(a[9]);
  if (scale == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{"softmax_scale must be a number"};
  }
  at::Tensor out = given(a[10]) ? tensor(a[10], "out") : at::empty(q.sizes(), q.options());
  REFUSE_IF(out.scalar_type() != at::kBFloat16 || out.sizes() != q.sizes() || out.stride(2) != 1,
            "out must be bf16 [total_q, H_q, 256] with unit stride on head_dim");
  at::Tensor made;
  const at::Tensor& ws = given(a[11]) ? workspace_of(a[11]) : made;
  if (!ws.defined()) {
    const size_t need = mtp_tree_attn_workspace_size(seqs, total, hq, hkv, width);
    made = at::empty({static_cast<int64_t>(need < 256 ? 256 : need)}, q.options().dtype(at::kByte));
  }
  const int rc = mtp_tree_attn_fwd(
      q.const_data_ptr(), q.stride(0), q.stride(1), k.const_data_ptr(), v.const_data_ptr(), k.size(0), ints(table), width,
      ints(lens), ints(cu), static_cast<const uint64_t*>(mask.const_data_ptr()), seqs, total, hq, hkv,
      static_cast<const float*>(kd.const_data_ptr()), static_cast<const float*>(vd.const_data_ptr()),
      static_cast<float>(scale), ws.data_ptr(), ws.nbytes(), out.data_ptr(), out.stride(0), out.stride(1),
      status_of(a[12]), stream);
  return finish(rc, rc ? nullptr : THPVariable_Wrap(std::move(out)));
}

// What the two verifications share: checks, and the outputs.
struct Verify {
  int32_t dtype, total, vocab, seqs, width;
  int64_t stride;
  at::Tensor index, count, said;
};

int32_t dtype_of(const at::Tensor& t) {
  const at::ScalarType s = t.scalar_type();
  return s == at::kFloat ? MTP_F32 : s == at::kBFloat16 ? MTP_BF16 : s == at::kHalf ? MTP_F16 : -1;
}
int64_t row_stride(const at::Tensor& t) {  // a single row's stride means nothing to torch
  return t.size(0) > 1 ? t.stride(0) : std::max(t.stride(0), t.size(1));
}

// An int32 tensor on like's device, every element of which the call writes: at::empty without the way
// through the dispatcher.  stream_of has made sure that a CUDA device is the current one.
at::Tensor ints_like(const at::Tensor& like, at::IntArrayRef sizes) {
  if (!like.is_cuda()) return at::empty(sizes, like.options().dtype(at::kInt));
  return at::detail::empty_generic(sizes, c10::cuda::CUDACachingAllocator::get(),
                                   c10::DispatchKeySet(c10::DispatchKey::CUDA), at::kInt, std::nullopt);
}

// tokens, parents, cu, max_path, accept_index, accept_len, out_tokens at a
Verify verify_args(const at::Tensor& rows, const char* name, PyObject* const* a) {
  Verify r;
  r.dtype = dtype_of(rows);
  REFUSE_IF(r.dtype < 0 || rows.dim() != 2 || (rows.size(1) > 1 && rows.stride(1) != 1),
            std::string(name) + " must be float32, bfloat16 or float16 [total_q, vocab] with unit stride along the vocabulary");
  r.total = count32(rows.size(0), name);
  r.vocab = count32(rows.size(1), name);
  r.stride = row_stride(rows);
  vector(tensor(a[0], "draft_tokens"), "draft_tokens", r.total);
  vector(tensor(a[1], "parents"), "parents", r.total);
  r.seqs = sequences(tensor(a[2], "cu_seqlens_q"));
  r.width = integer(a[3], "max_path");
  REFUSE_IF(r.width < 1 || r.width > MTP_TREE_MAX_NODES, "max_path must be 1 to 64");
  // (a storage each: one that is kept, or grows in place, does not touch the others)
  r.index = given(a[4]) ? tensor(a[4], "accept_index") : ints_like(rows, {r.seqs, r.width});
  r.count = given(a[5]) ? tensor(a[5], "accept_len") : ints_like(rows, {r.seqs});
  r.said = given(a[6]) ? tensor(a[6], "out_tokens") : ints_like(rows, {r.seqs, r.width});
  for (const auto& [t, what] : {std::pair<const at::Tensor&, const char*>(r.index, "accept_index"),
                                std::pair<const at::Tensor&, const char*>(r.said, "out_tokens")})
    REFUSE_IF(t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != r.seqs || t.size(1) != r.width || !t.is_contiguous(),
              std::string(what) + " must be a contiguous int32 [num_seqs, max_path] tensor");
  vector(r.count, "accept_len", r.seqs);
  return r;
}
PyObject* verify_result(int rc, Verify& r) {
  if (rc) return finish(rc, nullptr);
  PyObject* t = PyTuple_New(3);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(std::move(r.index)));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(std::move(r.count)));
  PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(std::move(r.said)));
  return t;
}

// logits, draft_tokens, parents, cu_seqlens_q, max_path, accept_index, accept_len, out_tokens,
// status, stream
PyObject* verify_greedy(PyObject* const* a) {
  const at::Tensor& logits = tensor(a[0], "logits");
  void* stream = stream_of(a[9], logits);
  Verify r = verify_args(logits, "logits", a + 1);
  const int rc = mtp_tree_verify_greedy(logits.const_data_ptr(), r.dtype, r.stride, r.vocab, ints(tensor(a[1], "")),
                                        ints(tensor(a[2], "")), ints(tensor(a[3], "")), r.seqs, r.total, r.width,
                                        ints_out(r.index), ints_out(r.count), ints_out(r.said), status_of(a[8]), stream);
  return verify_result(rc, r);
}

// target_probs, draft_probs, draft_tokens, parents, cu_seqlens_q, uniforms, max_path, accept_index,
// accept_len, out_tokens, status, stream
PyObject* verify_sample(PyObject* const* a) {
  const at::Tensor &p = tensor(a[0], "target_probs"), &u = tensor(a[5], "uniforms");
  void* stream = stream_of(a[11], p);
  PyObject* const common[] = {a[2], a[3], a[4], a[6], a[7], a[8], a[9]};
  Verify r = verify_args(p, "target_probs", common);
  const void* q = nullptr;
  int64_t q_stride = 0;
  if (given(a[1])) {
    const at::Tensor& t = tensor(a[1], "draft_probs");
    REFUSE_IF(t.scalar_type() != p.scalar_type() || t.sizes() != p.sizes() || (r.vocab > 1 && t.stride(1) != 1),
              "draft_probs must have target_probs' type and shape and unit stride along the vocabulary");
    q = t.const_data_ptr();
    q_stride = row_stride(t);
  }
  REFUSE_IF(u.scalar_type() != at::kFloat || u.dim() != 1 || u.size(0) != r.total || !u.is_contiguous(),
            "uniforms must be a contiguous float32 vector, one number per node");
  const int rc = mtp_tree_verify_sample(p.const_data_ptr(), r.stride, q, q_stride, r.dtype, r.vocab, ints(tensor(a[2], "")),
                                        ints(tensor(a[3], "")), ints(tensor(a[4], "")),
                                        static_cast<const float*>(u.const_data_ptr()), r.seqs, r.total, r.width,
                                        ints_out(r.index), ints_out(r.count), ints_out(r.said), status_of(a[10]), stream);
  return verify_result(rc, r);
}

// ---- the cache -----------------------------------------------------------------------------------

// One layer's caches [num_pages, 16, H_kv, 256], or a stack's behind num_layers; or, without v_cache,
// latent vectors [num_pages, 16, 576].
struct Cache {
  void *k, *v;
  int32_t layers, hkv;
  int64_t layer_stride, pages;
};
Cache cache_args(const at::Tensor& k, PyObject* v_) {
  const bool latent = !given(v_);
  const at::Tensor& v = latent ? k : tensor(v_, "v_cache");
  REFUSE_IF(!is_codes(k.scalar_type()) || v.scalar_type() != k.scalar_type(),
            "k_cache / v_cache must be uint8 or float8_e4m3fn codes");
  const int64_t n = k.dim(), one = latent ? 3 : 4;            // axes of a layer
  const int64_t row = latent ? MTP_LATENT_ROW : MTPATTN_HEAD_DIM;
  REFUSE_IF((n != one && n != one + 1) || k.size(n - one + 1) != MTPATTN_PAGE_SIZE || k.size(n - 1) != row,
            latent ? "k_cache without v_cache must be [num_pages, 16, 576], or that behind num_layers"
                   : "k_cache must be [num_pages, 16, H_kv, 256], or that behind num_layers");
  REFUSE_IF(v.sizes() != k.sizes() || v.strides() != k.strides(), "k_cache and v_cache must be of the same shape and strides");
  Cache c;
  c.layers = n == one + 1 ? count32(k.size(0), "k_cache") : 1;
  c.pages = k.size(n - one);
  c.hkv = latent ? 0 : count32(k.size(n - 2), "k_cache");
  REFUSE_IF(c.layers > 0 && !k.is_contiguous() && !(n == one + 1 && k.select(0, 0).is_contiguous()),
            "a layer's cache must be contiguous");
  c.layer_stride = c.layers > 1 ? k.stride(0) : c.pages * MTPATTN_PAGE_SIZE * (latent ? row : c.hkv * row);
  c.k = k.data_ptr();
  c.v = latent ? nullptr : v.data_ptr();
  return c;
}
struct Table {
  int32_t rows, width;
};
Table table_args(const at::Tensor& t, const at::Tensor& lens, const at::Tensor& refs, int64_t pages) {
  REFUSE_IF(t.scalar_type() != at::kInt || t.dim() != 2 || !t.is_contiguous(),
            "block_tables must be a contiguous int32 [num_rows, max_pages] tensor");
  vector(lens, "seq_lens", t.size(0));
  vector(refs, "ref_counts", pages);
  return {count32(t.size(0), "block_tables"), count32(t.size(1), "block_tables")};
}
at::Tensor cache_workspace(PyObject* o, const at::Tensor& like, const Table& t) {
  if (given(o)) return workspace_of(o);
  const size_t need = mtp_cache_workspace_size(t.rows, t.width);
  return at::empty({static_cast<int64_t>(need < 256 ? 256 : need)}, like.options().dtype(at::kByte));
}

// k_cache, v_cache, block_tables, seq_lens, ref_counts, new_lens, workspace, status, stream
PyObject* cache_resize(PyObject* const* a) {
  const at::Tensor &k = tensor(a[0], "k_cache"), &table = tensor(a[2], "block_tables");
  const at::Tensor &lens = tensor(a[3], "seq_lens"), &refs = tensor(a[4], "ref_counts"), &to = tensor(a[5], "new_lens");
  void* stream = stream_of(a[8], table);
  const Cache c = cache_args(k, a[1]);
  const Table t = table_args(table, lens, refs, c.pages);
  vector(to, "new_lens", t.rows);
  const at::Tensor ws = cache_workspace(a[6], table, t);
  const int rc = mtp_cache_resize(c.k, c.v, c.layers, c.layer_stride, c.pages, c.hkv, ints_out(table), t.width,
                                  ints_out(lens), t.rows, ints_out(refs), ints(to), ws.data_ptr(), ws.nbytes(),
                                  status_of(a[7]), stream);
  return finish(rc, rc ? nullptr : Py_NewRef(Py_None));
}

// k_cache, v_cache, block_tables, seq_lens, ref_counts, src, dst, workspace, status, stream
PyObject* cache_fork(PyObject* const* a) {
  const at::Tensor &k = tensor(a[0], "k_cache"), &table = tensor(a[2], "block_tables");
  const at::Tensor &lens = tensor(a[3], "seq_lens"), &refs = tensor(a[4], "ref_counts");
  const at::Tensor &src = tensor(a[5], "src"), &dst = tensor(a[6], "dst");
  void* stream = stream_of(a[9], table);
  const Cache c = cache_args(k, a[1]);
  const Table t = table_args(table, lens, refs, c.pages);
  vector(src, "src", src.numel());
  vector(dst, "dst", src.numel());
  const at::Tensor ws = cache_workspace(a[7], table, t);
  const int rc = mtp_cache_fork(c.k, c.v, c.layers, c.layer_stride, c.pages, c.hkv, ints_out(table), t.width,
                                ints_out(lens), t.rows, ints_out(refs), ints(src), ints(dst),
                                count32(src.numel(), "src"), ws.data_ptr(), ws.nbytes(), status_of(a[8]), stream);
  return finish(rc, rc ? nullptr : Py_NewRef(Py_None));
}

// k_cache, v_cache, src_pages, dst_pages, status, stream
PyObject* cache_copy_pages(PyObject* const* a) {
  const at::Tensor& k = tensor(a[0], "k_cache");
  const at::Tensor &src = tensor(a[2], "src_pages"), &dst = tensor(a[3], "dst_pages");
  void* stream = stream_of(a[5], k);
  const Cache c = cache_args(k, a[1]);
  vector(src, "src_pages", src.numel());
  vector(dst, "dst_pages", src.numel());
  const int rc = mtp_cache_copy_pages(c.k, c.v, c.layers, c.layer_stride, c.pages, c.hkv, ints(src), ints(dst),
                                      count32(src.numel(), "src_pages"), status_of(a[4]), stream);
  return finish(rc, rc ? nullptr : Py_NewRef(Py_None));
}

// k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q, accept_index, accept_len, new_seq_lens,
// status, stream
PyObject* cache_compact(PyObject* const* a) {
  const at::Tensor &k = tensor(a[0], "k_cache"), &table = tensor(a[2], "block_tables");
  const at::Tensor &lens = tensor(a[3], "seq_lens"), &cu = tensor(a[4], "cu_seqlens_q");
  const at::Tensor &index = tensor(a[5], "accept_index"), &count = tensor(a[6], "accept_len");
  void* stream = stream_of(a[9], k);
  const Cache c = cache_args(k, a[1]);
  const int32_t seqs = sequences(cu);
  REFUSE_IF(table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != seqs || !table.is_contiguous(),
            "block_tables must be a contiguous int32 [B, max_pages] tensor, cu_seqlens_q [B + 1]");
  vector(lens, "seq_lens", seqs);
  vector(count, "accept_len", seqs);
  REFUSE_IF(index.scalar_type() != at::kInt || index.dim() != 2 || index.size(0) != seqs || !index.is_contiguous(),
            "accept_index must be a contiguous int32 [B, max_path] tensor");
  at::Tensor out = given(a[7]) ? tensor(a[7], "new_seq_lens") : at::empty_like(lens);
  vector(out, "new_seq_lens", seqs);
  const int64_t most = static_cast<int64_t>(seqs) * MTP_TREE_MAX_NODES;
  const int rc = mtp_cache_compact(c.k, c.v, c.layers, c.layer_stride, c.pages, c.hkv, ints(table),
                                   count32(table.size(1), "block_tables"), ints(lens), ints(cu), seqs,
                                   count32(most, "cu_seqlens_q"), ints(index), ints(count),
                                   count32(index.size(1), "accept_index"), ints_out(out), status_of(a[8]), stream);
  return finish(rc, rc ? nullptr : THPVariable_Wrap(std::move(out)));
}

// ---- rotary positions and new tokens (include/mtp_rope.h) ----------------------------------------

float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{std::string(name) + " must be a number"};
  }
  return static_cast<float>(v);
}
int32_t truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    throw Refused{std::string(name) + " must be a truth value"};
  }
  return v;
}
const float* one_float(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  REFUSE_IF(t.scalar_type() != at::kFloat || t.numel() != 1, std::string(name) + " must be a 1-element float32 tensor");
  return static_cast<const float*>(t.const_data_ptr());
}

// [tokens, heads, dim], or without heads [tokens, dim] where dim alone is a row.  An axis of one element
// has a stride that means nothing to torch: it gets one that the library takes.
struct Rows {
  const void* p;
  int64_t tokens, tok, head;
  int32_t heads;
};
Rows rows_of(const at::Tensor& t, const char* name, at::ScalarType type, int64_t tokens, int64_t dim, bool headed) {
  const int64_t n = headed ? 3 : 2;
  REFUSE_IF(t.scalar_type() != type || t.dim() != n || t.size(n - 1) != dim || (tokens >= 0 && t.size(0) != tokens) ||
                t.stride(n - 1) != 1,
            std::string(name) + " must be " + c10::toString(type) + (headed ? " [tokens, heads, " : " [tokens, ") +
                std::to_string(dim) + "] with unit stride along the last axis, one row per token");
  Rows r;
  r.p = t.const_data_ptr();
  r.tokens = t.size(0);
  r.heads = headed ? count32(t.size(1), name) : 1;
  r.head = headed && r.heads > 1 ? t.stride(1) : dim;
  r.tok = r.tokens > 1 ? t.stride(0) : r.head * r.heads;
  return r;
}
const int64_t* freqs_of(const at::Tensor& t, int64_t n) {
  REFUSE_IF(t.scalar_type() != at::kLong || t.dim() != 1 || (n >= 0 && t.size(0) != n) || !t.is_contiguous(),
            "freqs must be a contiguous int64 vector, one per rotated pair (mtp_rope_freqs makes it)");
  return static_cast<const int64_t*>(t.const_data_ptr());
}
int32_t rope_dtype(const at::Tensor& t, const char* name) {
  const int32_t d = dtype_of(t);
  REFUSE_IF(d < 0, std::string(name) + " must be float32, bfloat16 or float16");
  return d;
}
// Block tables, lengths and boundaries of the sequences that new tokens belong to.
struct Places {
  const int32_t *bt, *lens, *cu;
  int32_t seqs, width;
};
Places places_of(PyObject* table_, PyObject* lens_, PyObject* cu_) {
  const at::Tensor &table = tensor(table_, "block_tables"), &lens = tensor(lens_, "seq_lens");
  const at::Tensor& cu = tensor(cu_, "cu_seqlens_q");
  Places p;
  p.seqs = sequences(cu);
  vector(lens, "seq_lens", p.seqs);
  REFUSE_IF(table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != p.seqs || !table.is_contiguous(),
            "block_tables must be a contiguous int32 [B, max_pages] tensor");
  p.width = count32(table.size(1), "block_tables");
  p.bt = ints(table);
  p.lens = ints(lens);
  p.cu = ints(cu);
  return p;
}
const at::Tensor& latent_cache(PyObject* o) {
  const at::Tensor& t = tensor(o, "cache");
  REFUSE_IF(!is_codes(t.scalar_type()) || t.dim() != 3 || t.size(1) != MTPATTN_PAGE_SIZE || t.size(2) != MTP_LATENT_ROW ||
                !t.is_contiguous(),
            "cache must be contiguous uint8 or float8_e4m3fn codes [num_pages, 16, 576]");
  return t;
}
at::Tensor rotated_out(PyObject* o, const at::Tensor& q, int64_t dim) {
  if (given(o)) return tensor(o, "q_out");
  return at::empty({q.size(0), q.size(1), dim}, q.options().dtype(at::kBFloat16));
}

// q, k, v, positions, freqs, k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q, k_descale, v_descale,
// mscale, interleaved, q_out, status, stream
PyObject* rope_append(PyObject* const* a) {
  const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &positions = tensor(a[3], "positions");
  const at::Tensor &kc = tensor(a[5], "k_cache"), &vc = tensor(a[6], "v_cache");
  void* stream = stream_of(a[16], k);
  const int32_t dtype = rope_dtype(k, "k");
  const Rows kr = rows_of(k, "k", k.scalar_type(), -1, MTPATTN_HEAD_DIM, true);
  const Rows vr = rows_of(v, "v", k.scalar_type(), kr.tokens, MTPATTN_HEAD_DIM, true);
  REFUSE_IF(vr.heads != kr.heads, "k and v must have the same heads");
  const int32_t total = count32(kr.tokens, "k");
  vector(positions, "positions", total);
  const int64_t* freqs = nullptr;
  int32_t rot = 0;
  if (given(a[4])) {
    freqs = freqs_of(tensor(a[4], "freqs"), -1);
    REFUSE_IF(tensor(a[4], "freqs").size(0) > MTPATTN_HEAD_DIM / 2, "freqs has more than 128 pairs");
    rot = static_cast<int32_t>(2 * tensor(a[4], "freqs").size(0));
  }
  REFUSE_IF(!is_codes(kc.scalar_type()) || vc.scalar_type() != kc.scalar_type() || kc.dim() != 4 ||
                kc.size(1) != MTPATTN_PAGE_SIZE || kc.size(2) != kr.heads || kc.size(3) != MTPATTN_HEAD_DIM ||
                vc.sizes() != kc.sizes() || !kc.is_contiguous() || !vc.is_contiguous(),
            "k_cache and v_cache must be contiguous uint8 or float8_e4m3fn codes [num_pages, 16, H_kv, 256], H_kv as in k");
  const Places at_ = places_of(a[7], a[8], a[9]);
  const float *kd = one_float(a[10], "k_descale"), *vd = one_float(a[11], "v_descale");
  Rows qr{}, outr{};
  at::Tensor out;
  if (given(a[0])) {
    const at::Tensor& q = tensor(a[0], "q");
    qr = rows_of(q, "q", k.scalar_type(), total, MTPATTN_HEAD_DIM, true);
    out = rotated_out(a[14], q, MTPATTN_HEAD_DIM);
    outr = rows_of(out, "q_out", at::kBFloat16, total, MTPATTN_HEAD_DIM, true);
    REFUSE_IF(outr.heads != qr.heads, "q_out must have q's heads");
  } else {
    REFUSE_IF(given(a[14]), "q_out without q");
  }
  const int rc = mtp_rope_append(qr.heads ? qr.p : nullptr, qr.tok, qr.head, kr.p, kr.tok, kr.head, vr.p, vr.tok, vr.head, dtype,
                                 ints(positions), freqs, rot, truth(a[13], "interleaved"), number(a[12], "mscale"),
                                 kc.data_ptr(), vc.data_ptr(), kc.size(0), at_.bt, at_.width, at_.lens, at_.cu, at_.seqs,
                                 total, qr.heads, kr.heads, kd, vd, qr.heads ? out.data_ptr() : nullptr, outr.tok, outr.head,
                                 status_of(a[15]), stream);
  return finish(rc, rc ? nullptr : out.defined() ? THPVariable_Wrap(std::move(out)) : Py_NewRef(Py_None));
}

// q_rope, latent, k_rope, positions, freqs, cache, block_tables, seq_lens, cu_seqlens_q, descale, mscale,
// interleaved, q_out, status, stream
PyObject* rope_latent_append(PyObject* const* a) {
  const at::Tensor &c = tensor(a[1], "latent"), &kr = tensor(a[2], "k_rope"), &positions = tensor(a[3], "positions");
  void* stream = stream_of(a[14], c);
  const int32_t dtype = rope_dtype(c, "latent");
  const Rows cr = rows_of(c, "latent", c.scalar_type(), -1, MTP_LATENT_DIM, false);
  const Rows rr = rows_of(kr, "k_rope", c.scalar_type(), cr.tokens, MTP_LATENT_ROPE_DIM, false);
  const int32_t total = count32(cr.tokens, "latent");
  vector(positions, "positions", total);
  const int64_t* freqs = freqs_of(tensor(a[4], "freqs"), MTP_LATENT_ROPE_DIM / 2);
  const at::Tensor& cache = latent_cache(a[5]);
  const Places at_ = places_of(a[6], a[7], a[8]);
  Rows qr{}, outr{};
  at::Tensor out;
  if (given(a[0])) {
    const at::Tensor& q = tensor(a[0], "q_rope");
    qr = rows_of(q, "q_rope", c.scalar_type(), total, MTP_LATENT_ROPE_DIM, true);
    out = rotated_out(a[12], q, MTP_LATENT_ROPE_DIM);
    outr = rows_of(out, "q_out", at::kBFloat16, total, MTP_LATENT_ROPE_DIM, true);
    REFUSE_IF(outr.heads != qr.heads, "q_out must have q_rope's heads");
  } else {
    REFUSE_IF(given(a[12]), "q_out without q_rope");
  }
  const int rc = mtp_rope_latent_append(qr.heads ? qr.p : nullptr, qr.tok, qr.head, cr.p, cr.tok, rr.p, rr.tok, dtype,
                                        ints(positions), freqs, truth(a[11], "interleaved"), number(a[10], "mscale"),
                                        cache.data_ptr(), cache.size(0), at_.bt, at_.width, at_.lens, at_.cu, at_.seqs,
                                        total, qr.heads, one_float(a[9], "descale"), qr.heads ? out.data_ptr() : nullptr,
                                        outr.tok, outr.head, status_of(a[13]), stream);
  return finish(rc, rc ? nullptr : out.defined() ? THPVariable_Wrap(std::move(out)) : Py_NewRef(Py_None));
}

at::Tensor codes_out(PyObject* o, const char* name, const at::Tensor& like, int64_t heads, int64_t dim) {
  at::Tensor t = given(o) ? tensor(o, name) : at::empty({like.size(0), heads, dim}, like.options().dtype(at::kFloat8_e4m3fn));
  REFUSE_IF(!is_codes(t.scalar_type()) || t.dim() != 3 || t.size(0) != like.size(0) || t.size(1) != heads ||
                t.size(2) != dim || !t.is_contiguous(),
            std::string(name) + " must be contiguous uint8 or float8_e4m3fn [tokens, heads, " + std::to_string(dim) + "]");
  return t;
}

// q, k, k_rope, v, positions, freqs, q_descale, k_descale, v_descale, mscale, interleaved, q_out, k_out,
// v_out, stream
PyObject* rope_prefill(PyObject* const* a) {
  constexpr int64_t kNope = 128, kQk = kNope + MTP_LATENT_ROPE_DIM, kV = 128;
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &kr = tensor(a[2], "k_rope"), &v = tensor(a[3], "v");
  const at::Tensor& positions = tensor(a[4], "positions");
  void* stream = stream_of(a[14], q);
  const int32_t dtype = rope_dtype(q, "q");
  const Rows qr = rows_of(q, "q", q.scalar_type(), -1, kQk, true);
  const Rows nr = rows_of(k, "k", q.scalar_type(), qr.tokens, kNope, true);
  const Rows rr = rows_of(kr, "k_rope", q.scalar_type(), qr.tokens, MTP_LATENT_ROPE_DIM, false);
  const Rows vr = rows_of(v, "v", q.scalar_type(), qr.tokens, kV, true);
  REFUSE_IF(vr.heads != nr.heads, "k and v must have the same heads");
  const int32_t total = count32(qr.tokens, "q");
  vector(positions, "positions", total);
  const int64_t* freqs = freqs_of(tensor(a[5], "freqs"), MTP_LATENT_ROPE_DIM / 2);
  const float *qd = one_float(a[6], "q_descale"), *kd = one_float(a[7], "k_descale"), *vd = one_float(a[8], "v_descale");
  const float mscale = number(a[9], "mscale");
  const int32_t interleaved = truth(a[10], "interleaved");
  at::Tensor q8 = codes_out(a[11], "q_out", q, qr.heads, kQk), k8 = codes_out(a[12], "k_out", q, nr.heads, kQk);
  at::Tensor v8 = codes_out(a[13], "v_out", q, nr.heads, kV);
  const int rc = mtp_rope_prefill(qr.p, qr.tok, qr.head, nr.p, nr.tok, nr.head, rr.p, rr.tok, vr.p, vr.tok, vr.head, dtype,
                                  ints(positions), freqs, interleaved, mscale, total, qr.heads, nr.heads, qd, kd, vd,
                                  q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), stream);
  if (rc) return finish(rc, nullptr);
  PyObject* t = PyTuple_New(3);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(std::move(q8)));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(std::move(k8)));
  PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(std::move(v8)));
  return t;
}

// ---- latent attention (include/mtp_latent.h) -----------------------------------------------------

// q, cache, block_tables, seq_lens, cu_seqlens_q, descale, softmax_scale, tree_mask, out, workspace, status,
// stream
PyObject* latent_attn(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  void* stream = stream_of(a[11], q);
  const Rows qr = rows_of(q, "q", at::kBFloat16, -1, MTP_LATENT_ROW, true);
  const int32_t total = count32(qr.tokens, "q");
  const at::Tensor& cache = latent_cache(a[1]);
  const Places at_ = places_of(a[2], a[3], a[4]);
  const float* descale = one_float(a[5], "descale");
  const uint64_t* mask = nullptr;
  if (given(a[7])) {
    words(tensor(a[7], "tree_mask"), "tree_mask", total);
    mask = static_cast<const uint64_t*>(tensor(a[7], "").const_data_ptr());
  }
  at::Tensor out = given(a[8]) ? tensor(a[8], "out") : at::empty({qr.tokens, qr.heads, MTP_LATENT_DIM}, q.options());
  const Rows outr = rows_of(out, "out", at::kBFloat16, qr.tokens, MTP_LATENT_DIM, true);
  REFUSE_IF(outr.heads != qr.heads, "out must have q's heads");
  at::Tensor made;
  const at::Tensor& ws = given(a[9]) ? workspace_of(a[9]) : made;
  if (!ws.defined()) {
    const size_t need = mtp_latent_attn_workspace_size(at_.seqs, total, qr.heads, at_.width);
    made = at::empty({static_cast<int64_t>(need < 256 ? 256 : need)}, q.options().dtype(at::kByte));
  }
  const int rc = mtp_latent_attn_fwd(qr.p, qr.tok, qr.head, cache.const_data_ptr(), cache.size(0), at_.bt, at_.width, at_.lens,
                                     at_.cu, mask, at_.seqs, total, qr.heads, descale, number(a[6], "softmax_scale"),
                                     ws.data_ptr(), ws.nbytes(), out.data_ptr(), outr.tok, outr.head, status_of(a[10]), stream);
  return finish(rc, rc ? nullptr : THPVariable_Wrap(std::move(out)));
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XDECREF(g_error);
  g_error = Py_NewRef(cls);
  return Py_NewRef(Py_None);
}

#define ENTRY(name, args) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, args>)), METH_FASTCALL, nullptr}

PyMethodDef kMethods[] = {
    ENTRY(tree_mask, 5),        ENTRY(tree_attn, 14),        ENTRY(verify_greedy, 10), ENTRY(verify_sample, 12),
    ENTRY(cache_resize, 9),     ENTRY(cache_fork, 10),       ENTRY(cache_copy_pages, 6), ENTRY(cache_compact, 10),
    ENTRY(rope_append, 17),     ENTRY(rope_latent_append, 15), ENTRY(rope_prefill, 15), ENTRY(latent_attn, 12),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
