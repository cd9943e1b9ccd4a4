// The Python binding of the draft-tree and cache entry points (include/mtp_tree.h,
// include/mtp_cache.h): argument checks, the outputs that were not given, and the call.  These calls
// take 3 to 20 us on the GPU; the same steps in Python took 10 to 17 us of host time a call on a
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
  const at::Tensor& ws = given(a[11]) ? tensor(a[11], "workspace") : made;
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

// One layer's caches [num_pages, 16, H_kv, 256], or a stack's behind num_layers.
struct Cache {
  void *k, *v;
  int32_t layers, hkv;
  int64_t layer_stride, pages;
};
Cache cache_args(const at::Tensor& k, const at::Tensor& v) {
  REFUSE_IF(!is_codes(k.scalar_type()) || v.scalar_type() != k.scalar_type(),
            "k_cache / v_cache must be uint8 or float8_e4m3fn codes");
  const int64_t n = k.dim();
  REFUSE_IF((n != 4 && n != 5) || k.size(n - 3) != MTPATTN_PAGE_SIZE || k.size(n - 1) != MTPATTN_HEAD_DIM,
            "k_cache must be [num_pages, 16, H_kv, 256], or that behind num_layers");
  REFUSE_IF(v.sizes() != k.sizes() || v.strides() != k.strides(), "k_cache and v_cache must be of the same shape and strides");
  Cache c;
  c.layers = n == 5 ? count32(k.size(0), "k_cache") : 1;
  c.pages = k.size(n - 4);
  c.hkv = count32(k.size(n - 2), "k_cache");
  REFUSE_IF(c.layers > 0 && !k.is_contiguous() && !(n == 5 && k.select(0, 0).is_contiguous()),
            "a layer's cache must be contiguous");
  c.layer_stride = c.layers > 1 ? k.stride(0) : c.pages * c.hkv * (MTPATTN_PAGE_SIZE * MTPATTN_HEAD_DIM);
  c.k = k.data_ptr();
  c.v = v.data_ptr();
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
  if (given(o)) return tensor(o, "workspace");
  const size_t need = mtp_cache_workspace_size(t.rows, t.width);
  return at::empty({static_cast<int64_t>(need < 256 ? 256 : need)}, like.options().dtype(at::kByte));
}

// k_cache, v_cache, block_tables, seq_lens, ref_counts, new_lens, workspace, status, stream
PyObject* cache_resize(PyObject* const* a) {
  const at::Tensor &k = tensor(a[0], "k_cache"), &v = tensor(a[1], "v_cache"), &table = tensor(a[2], "block_tables");
  const at::Tensor &lens = tensor(a[3], "seq_lens"), &refs = tensor(a[4], "ref_counts"), &to = tensor(a[5], "new_lens");
  void* stream = stream_of(a[8], table);
  const Cache c = cache_args(k, v);
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
  const at::Tensor &k = tensor(a[0], "k_cache"), &v = tensor(a[1], "v_cache"), &table = tensor(a[2], "block_tables");
  const at::Tensor &lens = tensor(a[3], "seq_lens"), &refs = tensor(a[4], "ref_counts");
  const at::Tensor &src = tensor(a[5], "src"), &dst = tensor(a[6], "dst");
  void* stream = stream_of(a[9], table);
  const Cache c = cache_args(k, v);
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
  const at::Tensor &k = tensor(a[0], "k_cache"), &v = tensor(a[1], "v_cache");
  const at::Tensor &src = tensor(a[2], "src_pages"), &dst = tensor(a[3], "dst_pages");
  void* stream = stream_of(a[5], k);
  const Cache c = cache_args(k, v);
  vector(src, "src_pages", src.numel());
  vector(dst, "dst_pages", src.numel());
  const int rc = mtp_cache_copy_pages(c.k, c.v, c.layers, c.layer_stride, c.pages, c.hkv, ints(src), ints(dst),
                                      count32(src.numel(), "src_pages"), status_of(a[4]), stream);
  return finish(rc, rc ? nullptr : Py_NewRef(Py_None));
}

// k_cache, v_cache, block_tables, seq_lens, cu_seqlens_q, accept_index, accept_len, new_seq_lens,
// status, stream
PyObject* cache_compact(PyObject* const* a) {
  const at::Tensor &k = tensor(a[0], "k_cache"), &v = tensor(a[1], "v_cache"), &table = tensor(a[2], "block_tables");
  const at::Tensor &lens = tensor(a[3], "seq_lens"), &cu = tensor(a[4], "cu_seqlens_q");
  const at::Tensor &index = tensor(a[5], "accept_index"), &count = tensor(a[6], "accept_len");
  void* stream = stream_of(a[9], k);
  const Cache c = cache_args(k, v);
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
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
