// Native marshalling of the mixture-of-experts and the attention calls: reads the tensors'
// addresses, strides and types, checks their shapes and calls the C ABI
// (include/lora.h) on the given or the current stream. The same through ctypes
// takes about 4.7 us a call on the host, more than most of these kernels run
// for a decode step; this takes 2.3 us. Each function returns the lora_status;
// arguments that are no tensors, of the wrong shape or type, or not on the
// current device raise.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <type_traits>

#include "lora.h"

namespace {

// A check that failed, with the Python exception type to raise.
struct Refused {
  PyObject *type;
  std::string what;
};

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + ": expected a tensor"};
  return THPVariable_Unpack(o);
}

std::string describe(const at::Tensor &t) {
  std::string s = "shape (";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  s += "), strides (";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.stride(i));
  return s + ")";
}

// The tensors of a call, checked together once their shapes and types are known to be right: a kernel of the current
// device uses them.
class Call {
 public:
  void uses(const at::Tensor &t, const char *name) {
    if (n_ < kMost && t.numel() > 0) used_[n_++] = {&t, name};
  }
  // The stream to launch on: a raw one, or for None the current device's current one.
  lora_stream_t stream(PyObject *o);

 private:
  static constexpr int kMost = 12;
  struct { const at::Tensor *t; const char *name; } used_[kMost];
  int n_ = 0;
};

// A matrix of at least `rows` contiguous rows, `width` wide (any width when negative).
struct Mat {
  void *p;
  int64_t ld;  // row stride in elements
  int32_t dtype;
  Mat(Call &call, PyObject *o, int64_t rows, int64_t width, const char *name, bool bytes = false) {
    const at::Tensor &t = tensor(o, name);
    call.uses(t, name);
    if (t.dim() != 2 || (width >= 0 && t.size(1) != width) || t.size(0) < rows || (t.stride(1) != 1 && t.size(1) > 1))
      throw Refused{PyExc_ValueError, std::string(name) + ": expected [" + std::to_string(rows) + ", " +
                                          (width >= 0 ? std::to_string(width) : std::string("any")) +
                                          "] with contiguous rows, got " + describe(t)};
    const at::ScalarType st = t.scalar_type();
    dtype = st == at::kBFloat16 ? LORA_BF16 : LORA_F32;
    if (bytes ? st != at::kByte : st != at::kBFloat16 && st != at::kFloat)
      throw Refused{PyExc_TypeError, std::string(name) + ": expected " + (bytes ? "uint8" : "bf16 or fp32") + ", got " +
                                         c10::toString(st)};
    if (t.size(0) > 1 && t.stride(0) < t.size(1))
      throw Refused{PyExc_ValueError, std::string(name) + ": expected rows that do not overlap, got " + describe(t)};
    // A single row's stride means nothing (torch may report any value): its length, rounded to the ABI's 16 bytes.
    const int64_t es = (int64_t)t.element_size();
    ld = t.size(0) > 1 ? t.stride(0) : (t.size(1) * es + 15) / 16 * 16 / es;
    p = t.data_ptr();
  }
};

// Scale bytes of at least `rows` rows of `cols` elements: a byte a block in every row. A kernel that `loads` them
// takes 16 at a time, so the bytes up to the next multiple of 16 belong to the tensor's memory, after the last row too.
struct Scales : Mat {
  Scales(Call &call, PyObject *o, int64_t rows, int64_t cols, const char *name, bool loads = false)
      : Mat(call, o, rows, -1, name, true) {
    const at::Tensor &t = tensor(o, name);
    const int64_t blocks = cols / LORA_MX_BLOCK, row = loads ? (blocks + 15) / 16 * 16 : blocks;
    if (t.size(1) < blocks)
      throw Refused{PyExc_ValueError, std::string(name) + ": expected at least " + std::to_string(blocks) +
                                          " columns, a byte for " + std::to_string(LORA_MX_BLOCK) + " elements, got " + describe(t)};
    if (loads && rows > 0 &&
        t.storage_offset() + (rows - 1) * ld + row > (int64_t)t.storage().nbytes())
      throw Refused{PyExc_ValueError, std::string(name) + ": expected rows of " + std::to_string(row) +
                                          " bytes of memory (mx4_buffers allocates them), got " + describe(t)};
  }
};

// n contiguous int32 or fp32 elements; None gives a null pointer.
template <typename T> T *vec(Call &call, PyObject *o, int64_t n, const char *name) {
  if (o == Py_None) return nullptr;
  const at::Tensor &t = tensor(o, name);
  call.uses(t, name);
  constexpr at::ScalarType want = std::is_floating_point_v<T> ? at::kFloat : at::kInt;
  if (t.numel() != n || !t.is_contiguous() || t.scalar_type() != want)
    throw Refused{PyExc_ValueError, std::string(name) + ": expected " + std::to_string(n) + " contiguous " +
                                        c10::toString(want) + " elements, got " + describe(t) + " " +
                                        c10::toString(t.scalar_type())};
  return static_cast<T *>(t.data_ptr());
}

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return v;
}
int32_t int32(PyObject *o, const char *name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) throw Refused{PyExc_ValueError, std::string(name) + " outside 32 bits"};
  return (int32_t)v;
}
double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return v;
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{nullptr, ""};
  return v != 0;
}
lora_stream_t Call::stream(PyObject *o) {
  for (int i = 0; i < n_; ++i)
    if (!used_[i].t->is_cuda())
      throw Refused{PyExc_ValueError, std::string(used_[i].name) + ": expected a CUDA tensor, got one on " + used_[i].t->device().str()};
  lora_stream_t s;
  int current;
  if (o == Py_None) {
    const c10::cuda::CUDAStream c = c10::cuda::getCurrentCUDAStream();
    s = (lora_stream_t)c.stream();
    current = (int)c.device_index();
  } else {
    s = (lora_stream_t)(intptr_t)integer(o);
    current = (int)c10::cuda::current_device();
  }
  for (int i = 0; i < n_; ++i)
    if ((int)used_[i].t->get_device() != current)
      throw Refused{PyExc_ValueError, std::string(used_[i].name) + ": on " + used_[i].t->device().str() +
                                          ", but the current device is cuda:" + std::to_string(current)};
  return s;
}
int64_t rows_of(PyObject *o, const char *name, int dim = 0) {
  const at::Tensor &t = tensor(o, name);
  if (t.dim() != 2) throw Refused{PyExc_ValueError, std::string(name) + ": expected a matrix, got " + describe(t)};
  return t.size(dim);
}
int32_t narrow(int64_t v, const char *name) {
  if (v > INT32_MAX) throw Refused{PyExc_ValueError, std::string(name) + " past 32 bits"};
  return (int32_t)v;
}

// Runs a call without the interpreter lock.
template <typename F> int unlocked(F f) {
  int st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS return st;
}

// (logits, topk, score, renormalize, scale, expert_map, local_experts or None, topk_ids, topk_w, pair_slot, stream)
int moe_route(PyObject *const *a) {
  Call call;
  const int64_t T = rows_of(a[0], "logits"), E = rows_of(a[0], "logits", 1);
  const Mat l(call, a[0], T, E, "logits");
  const int32_t topk = int32(a[1], "topk"), score = int32(a[2], "score");
  const bool renorm = truth(a[3]);
  const float scale = (float)number(a[4]);
  const int32_t *map = vec<int32_t>(call, a[5], E, "expert_map");
  const int32_t local = a[6] == Py_None ? narrow(E, "experts") : int32(a[6], "local_experts");
  const int64_t n = T * topk;
  int32_t *ids = vec<int32_t>(call, a[7], n, "topk_ids");
  float *w = vec<float>(call, a[8], n, "topk_w");
  int32_t *slot = vec<int32_t>(call, a[9], n, "pair_slot");
  lora_stream_t s = call.stream(a[10]);
  const int32_t t32 = narrow(T, "tokens"), e32 = narrow(E, "experts");
  return unlocked([&] {
    return lora_moe_route(l.p, l.ld, l.dtype, t32, e32, topk, score, renorm, scale, map, local, ids, w,
                          slot, s);
  });
}

// (address of the lora_expert_desc, of the lora_meta, x, y, x_scale or None, stream, the weights, one of the metadata's
// tensors or None)
int moe_product(PyObject *const *a) {
  Call call;
  const lora_expert_desc *d = (const lora_expert_desc *)(intptr_t)integer(a[0]);
  const lora_meta *m = (const lora_meta *)(intptr_t)integer(a[1]);
  const int64_t P = m->num_tokens, div = d->x_row_div > 1 ? d->x_row_div : 1, rows = (P + div - 1) / div;
  const bool mx = d->dtype == LORA_MXFP4;
  if (mx && a[4] == Py_None)
    throw Refused{PyExc_TypeError, "moe_product: 4-bit weights take x as mx4_quantize gives it, with x_scale"};
  const Mat x(call, a[2], rows, mx ? d->d_in / 2 : d->d_in, "x", mx);
  if (!mx && x.dtype != d->dtype) throw Refused{PyExc_TypeError, "moe_product: x is not of the experts' weights' type"};
  const uint8_t *sp = nullptr;
  int64_t lds = 0;
  if (mx) {
    const Scales sc(call, a[4], rows, d->d_in, "x_scale", true);
    sp = static_cast<const uint8_t *>(sc.p);
    lds = sc.ld;
  }
  const Mat y(call, a[3], P, d->d_out, "y");
  call.uses(tensor(a[6], "the experts' weights"), "the experts' weights");
  if (a[7] != Py_None) call.uses(tensor(a[7], "the metadata"), "the metadata");
  lora_stream_t s = call.stream(a[5]);
  return unlocked([&] { return lora_moe_product(d, m, x.p, mx ? 2 * x.ld : x.ld, sp, lds, y.p, y.ld, y.dtype, s); });
}

// (x, codes, scales, stream), (y, codes, scales, stream): rows of x or y to the 4-bit format, or from it
template <bool kTo> int mx4(PyObject *const *a) {
  Call call;
  const int64_t rows = rows_of(a[0], kTo ? "x" : "y"), cols = rows_of(a[0], kTo ? "x" : "y", 1);
  const Mat m(call, a[0], rows, cols, kTo ? "x" : "y"), c(call, a[1], rows, cols / 2, "codes", true);
  const Scales sc(call, a[2], rows, cols, "scales");
  lora_stream_t s = call.stream(a[3]);
  const int32_t n = narrow(cols, "columns");
  uint8_t *cp = static_cast<uint8_t *>(c.p), *sp = static_cast<uint8_t *>(sc.p);
  return unlocked([&] {
    return kTo ? lora_mx_quantize(m.p, m.ld, m.dtype, rows, n, cp, c.ld, sp, sc.ld, s)
               : lora_mx_dequantize(cp, c.ld, sp, sc.ld, rows, n, m.p, m.ld, m.dtype, s);
  });
}

// (y13, h, pair_slot or None, stream)
int moe_act(PyObject *const *a) {
  Call call;
  const int64_t P = rows_of(a[1], "h"), inter = rows_of(a[1], "h", 1);
  const Mat y(call, a[0], P, 2 * inter, "y13"), h(call, a[1], P, inter, "h");
  const int32_t *slot = vec<int32_t>(call, a[2], P, "pair_slot");
  lora_stream_t s = call.stream(a[3]);
  const int32_t p32 = narrow(P, "pairs"), i32 = narrow(inter, "columns");
  return unlocked([&] { return lora_moe_act(y.p, y.ld, y.dtype, slot, p32, i32, h.p, h.ld, h.dtype, s); });
}

// (y13, codes, scales, pair_slot or None, stream)
int moe_act_mx4(PyObject *const *a) {
  Call call;
  const int64_t P = rows_of(a[0], "y13"), inter = rows_of(a[0], "y13", 1) / 2;
  const Mat y(call, a[0], P, 2 * inter, "y13"), c(call, a[1], P, inter / 2, "codes", true);
  const Scales sc(call, a[2], P, inter, "scales");
  const int32_t *slot = vec<int32_t>(call, a[3], P, "pair_slot");
  lora_stream_t s = call.stream(a[4]);
  const int32_t p32 = narrow(P, "pairs"), i32 = narrow(inter, "columns");
  return unlocked([&] {
    return lora_moe_act_mx(y.p, y.ld, y.dtype, slot, p32, i32, static_cast<uint8_t *>(c.p), c.ld,
                           static_cast<uint8_t *>(sc.p), sc.ld, s);
  });
}

// (y, topk_w, out, pair_slot or None, accumulate, stream)
int moe_combine(PyObject *const *a) {
  Call call;
  const int64_t T = rows_of(a[1], "topk_w"), topk = rows_of(a[1], "topk_w", 1), n = rows_of(a[2], "out", 1);
  const Mat y(call, a[0], T * topk, n, "y"), out(call, a[2], T, n, "out");
  const float *w = vec<float>(call, a[1], T * topk, "topk_w");
  const int32_t *slot = vec<int32_t>(call, a[3], T * topk, "pair_slot");
  const bool accumulate = truth(a[4]);
  lora_stream_t s = call.stream(a[5]);
  const int32_t t32 = narrow(T, "tokens"), k32 = narrow(topk, "choices"), n32 = narrow(n, "columns");
  return unlocked([&] {
    return lora_moe_combine(y.p, y.ld, y.dtype, w, slot, t32, k32, n32, out.p, out.ld, out.dtype, accumulate, s);
  });
}

// ---- attention

lora_seqs *seqs_at(PyObject *o) { return (lora_seqs *)(intptr_t)integer(o); }

// Rows of the batch in the sequences' type, `heads` heads wide.
Mat rows_for(Call &call, const lora_seqs *s, PyObject *o, int64_t heads, const char *name) {
  const Mat m(call, o, s->num_tokens, heads * s->head_dim, name);
  if (m.dtype != s->dtype) throw Refused{PyExc_TypeError, std::string(name) + ": not of the attention's type"};
  return m;
}
// A page table of at least `rows` rows, and its row stride.
int64_t table_of(Call &call, PyObject *o, int64_t rows, int64_t pages) {
  const at::Tensor &t = tensor(o, "block_table");
  call.uses(t, "block_table");
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) < rows || t.size(1) < pages || (t.size(1) > 1 && t.stride(1) != 1) ||
      (t.size(0) > 1 && t.stride(0) < t.size(1)))
    throw Refused{PyExc_ValueError, "block_table: expected int32 [" + std::to_string(rows) + ", " + std::to_string(pages) +
                                        "] with contiguous rows, got " + describe(t) + " " + c10::toString(t.scalar_type())};
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}
// Scratch: its address and bytes.
struct Scratch {
  void *p;
  size_t bytes;
  Scratch(Call &call, PyObject *o) {
    const at::Tensor &t = tensor(o, "ws");
    call.uses(t, "ws");
    if (!t.is_contiguous()) throw Refused{PyExc_ValueError, "ws: expected contiguous memory, got " + describe(t)};
    p = t.data_ptr();
    bytes = (size_t)t.numel() * t.element_size();
  }
};
void check_cache(Call &call, const lora_seqs *s, PyObject *k, PyObject *v) {
  for (PyObject *o : {k, v}) {
    const at::Tensor &t = tensor(o, "cache");
    call.uses(t, "cache");
    if (t.dim() != 4 || t.size(1) != s->page_size || t.size(2) != s->num_kv_heads || t.size(3) != s->head_dim)
      throw Refused{PyExc_ValueError, "cache: expected [pages, " + std::to_string(s->page_size) + ", " +
                                          std::to_string(s->num_kv_heads) + ", " + std::to_string(s->head_dim) + "], got " + describe(t)};
    if (t.scalar_type() != (s->dtype == LORA_BF16 ? at::kBFloat16 : at::kFloat))
      throw Refused{PyExc_TypeError, std::string("cache: not of the attention's type, got ") + c10::toString(t.scalar_type())};
  }
}

// (address of the lora_seqs, rows, q_start, kv_len or None, block_table or None, most rows, most sequences, plan): fills the struct
int prepare_seqs(PyObject *const *a) {
  Call call;
  lora_seqs *s = seqs_at(a[0]);
  const int32_t T = int32(a[1], "num_tokens"), most_t = int32(a[5], "max_tokens"), most_s = int32(a[6], "max_seqs");
  const at::Tensor &qs = tensor(a[2], "q_start");
  const int64_t S = qs.numel() - 1;
  if (S < 0 || S > most_s)
    throw Refused{PyExc_ValueError, "q_start: expected one more element than up to " + std::to_string(most_s) + " sequences, got " + describe(qs)};
  if (T < 0 || T > most_t)
    throw Refused{PyExc_ValueError, "num_tokens " + std::to_string(T) + " outside [0, " + std::to_string(most_t) + "]"};
  const int32_t *start = vec<int32_t>(call, a[2], S + 1, "q_start"), *len = vec<int32_t>(call, a[3], S, "kv_len");
  const int32_t *table = nullptr;
  int64_t ld = 0;
  if (a[4] != Py_None) {
    if (s->page_size == 0) throw Refused{PyExc_ValueError, "block_table: these sequences have no pages"};
    ld = table_of(call, a[4], S, s->max_pages);
    table = static_cast<const int32_t *>(tensor(a[4], "block_table").data_ptr());
  }
  call.uses(tensor(a[7], "the plan"), "the plan");
  call.stream(Py_None);  // every tensor is on the current device
  s->q_start = start;
  s->kv_len = len;
  s->num_seqs = (int32_t)S;
  s->num_tokens = T;
  s->block_table = table;
  s->ld_table = ld;
  return LORA_OK;
}

// (address of the lora_seqs, of the lora_kv_cache, k, v, the cache's k and v, block_table or None, plan, stream)
int kv_write(PyObject *const *a) {
  Call call;
  const lora_seqs *s = seqs_at(a[0]);
  const lora_kv_cache *c = (const lora_kv_cache *)(intptr_t)integer(a[1]);
  if (a[6] == Py_None) throw Refused{PyExc_ValueError, "kv_write: prepare() was given no block_table"};
  const Mat k = rows_for(call, s, a[2], s->num_kv_heads, "k"), v = rows_for(call, s, a[3], s->num_kv_heads, "v");
  check_cache(call, s, a[4], a[5]);
  call.uses(tensor(a[6], "block_table"), "block_table");
  call.uses(tensor(a[7], "the plan"), "the plan");
  lora_stream_t st = call.stream(a[8]);
  return unlocked([&] { return lora_kv_write(s, c, k.p, k.ld, v.p, v.ld, st); });
}

// (address of the lora_seqs, q, k, v, out, lse or None, ws, plan, stream)
int attn_prompt(PyObject *const *a) {
  Call call;
  const lora_seqs *s = seqs_at(a[0]);
  if (s->kv_len != nullptr) throw Refused{PyExc_ValueError, "attn_prompt: prepare() was given kv_len"};
  const Mat q = rows_for(call, s, a[1], s->num_heads, "q"), k = rows_for(call, s, a[2], s->num_kv_heads, "k"),
            v = rows_for(call, s, a[3], s->num_kv_heads, "v"), out = rows_for(call, s, a[4], s->num_heads, "out");
  float *lse = vec<float>(call, a[5], (int64_t)s->num_tokens * s->num_heads, "lse");
  const Scratch ws(call, a[6]);
  call.uses(tensor(a[7], "the plan"), "the plan");
  lora_stream_t st = call.stream(a[8]);
  return unlocked([&] {
    return lora_attn_prompt(s, q.p, q.ld, k.p, k.ld, v.p, v.ld, out.p, out.ld, lse, ws.p, ws.bytes, st);
  });
}

// (address of the lora_seqs, of the lora_kv_cache, q, out, lse or None, ws, the cache's k and v, block_table or None, plan, stream)
int attn_paged(PyObject *const *a) {
  Call call;
  const lora_seqs *s = seqs_at(a[0]);
  const lora_kv_cache *c = (const lora_kv_cache *)(intptr_t)integer(a[1]);
  if (a[8] == Py_None) throw Refused{PyExc_ValueError, "attn_paged: prepare() was given no block_table"};
  const Mat q = rows_for(call, s, a[2], s->num_heads, "q"), out = rows_for(call, s, a[3], s->num_heads, "out");
  float *lse = vec<float>(call, a[4], (int64_t)s->num_tokens * s->num_heads, "lse");
  const Scratch ws(call, a[5]);
  check_cache(call, s, a[6], a[7]);
  call.uses(tensor(a[8], "block_table"), "block_table");
  call.uses(tensor(a[9], "the plan"), "the plan");
  lora_stream_t st = call.stream(a[10]);
  return unlocked([&] { return lora_attn_paged(s, c, q.p, q.ld, out.p, out.ld, lse, ws.p, ws.bytes, st); });
}

// The Python entry of F, which takes N arguments: no C++ exception leaves it.
template <int (*F)(PyObject *const *), int N> PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
  try {
    return PyLong_FromLong(F(args));
  } catch (const Refused &r) {
    if (r.type != nullptr) PyErr_SetString(r.type, r.what.c_str());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
template <int (*F)(PyObject *const *), int N> PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<moe_route, 11>("moe_route"),
                         method<moe_product, 8>("moe_product"),
                         method<mx4<true>, 4>("mx4_quantize"),
                         method<mx4<false>, 4>("mx4_dequantize"),
                         method<moe_act, 4>("moe_act"),
                         method<moe_act_mx4, 5>("moe_act_mx4"),
                         method<moe_combine, 6>("moe_combine"),
                         method<prepare_seqs, 8>("prepare_seqs"),
                         method<kv_write, 9>("kv_write"),
                         method<attn_prompt, 9>("attn_prompt"),
                         method<attn_paged, 11>("attn_paged"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe_binding(void) { return PyModule_Create(&module); }
