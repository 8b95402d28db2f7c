// The paged calls of the Python binding: argument checks, output and workspace
// tensors, and the library call, in one step from Python.
//
// A step of a serving loop makes these calls once a layer, and at its sizes a
// kernel runs for a few microseconds: taken apart in Python (attribute reads,
// two allocations, a foreign call of eighteen arguments) the same work on the
// host takes about 20 us a call, here about 5.  Nothing is computed here and
// nothing kept between calls; a failed check raises what the Python checks of
// the other calls raise, and a status other than KVQ_OK goes back as an int.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/kvq.h"

namespace {

using at::Tensor;

// The Python error that is set, as the exception HANDLE_TH_ERRORS restores.
[[noreturn]] void raise_pending() {
  python_error e;
  e.persist();
  throw e;
}
[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  raise_pending();
}
[[noreturn]] void refuse_type(const std::string& what) {
  PyErr_SetString(PyExc_TypeError, what.c_str());
  raise_pending();
}

std::string device_name(const c10::Device& d) { return d.str(); }

Tensor unpack(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse_type(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
Tensor unpack_optional(PyObject* o, const char* name) { return o == Py_None ? Tensor() : unpack(o, name); }

kvq_dtype dtype_code(const Tensor& t) {
  if (t.scalar_type() == at::kFloat) return KVQ_F32;
  if (t.scalar_type() == at::kBFloat16) return KVQ_BF16;
  refuse_type(std::string("unsupported dtype ") + c10::toString(t.scalar_type()) + ": float32 or bfloat16");
}

void check_index(const Tensor& t, const char* name, int64_t n, const c10::Device& dev) {
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.numel() != n)
    refuse(std::string(name) + " must be int32 [" + std::to_string(n) + "]");
  if (t.device() != dev || !t.is_contiguous()) refuse(std::string(name) + " must be contiguous on " + device_name(dev));
}

// The row stride of t [T, heads, D], whose rows may lie any distance apart.
int64_t check_rows(const Tensor& t, const char* name, int64_t T, int64_t heads, int64_t D, const c10::Device& dev) {
  if (t.device() != dev) refuse(std::string(name) + " must be on " + device_name(dev));
  if (t.dim() != 3 || t.size(0) != T || t.size(1) != heads || t.size(2) != D)
    refuse(std::string(name) + " must be [" + std::to_string(T) + ", " + std::to_string(heads) + ", " +
           std::to_string(D) + "]");
  if ((D > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != D))
    refuse(std::string(name) + ": the heads of a row must lie one after the other");
  if (T > 1 && t.stride(0) < heads * D) refuse(std::string(name) + ": rows must not overlap");
  return T > 1 ? t.stride(0) : heads * D;
}

void check_dense(const Tensor& t, const char* name, const c10::Device& dev) {
  if (t.device() != dev) refuse(std::string(name) + " must be on " + device_name(dev));
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
}

// The rotation of a call; table stays null without one.
kvq_rope rope_arg(const Tensor& rope, bool interleaved, int64_t D, const c10::Device& dev) {
  kvq_rope r{};
  if (!rope.defined()) return r;
  check_dense(rope, "rope", dev);
  if (rope.scalar_type() != at::kFloat || rope.dim() != 2) refuse("rope must be float32 [n_pos, rot_dim]");
  const int64_t n_pos = rope.size(0), rot = rope.size(1);
  if (rot < 2 || rot % 2 || rot > D || n_pos < 1) refuse("rot_dim must be even, at least 2 and at most D");
  r.table = rope.const_data_ptr<float>();
  r.n_pos = static_cast<int32_t>(n_pos);
  r.rot_dim = static_cast<int32_t>(rot);
  r.interleaved = interleaved;
  return r;
}

Tensor new_dense(c10::IntArrayRef sizes, at::ScalarType type, const c10::Device& dev) {
  return Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
}

int32_t to_i32(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) raise_pending();
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " must fit 32 bits");
  return static_cast<int32_t>(v);
}
double to_double(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) raise_pending();
  return v;
}
bool to_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) raise_pending();
  return v != 0;
}
int32_t rows32(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse(std::string(name) + " has too many rows");
  return static_cast<int32_t>(n);
}

// The cache of a call: address of its kvq_paged_cache and its device's index.
struct CacheArg {
  const kvq_paged_cache* c;
  c10::Device dev;
  CacheArg(PyObject* address, PyObject* index)
      : c(static_cast<const kvq_paged_cache*>(PyLong_AsVoidPtr(address))),
        dev(c10::kCUDA, static_cast<c10::DeviceIndex>(to_i32(index, "device"))) {
    if (!c) raise_pending();
  }
};

struct BatchArg {
  Tensor table, lengths, cu;
  int32_t S, max_pages;
  BatchArg(PyObject* t, PyObject* l, PyObject* c, const char* lengths_name, const c10::Device& dev)
      : table(unpack(t, "block_table")), lengths(unpack(l, lengths_name)), cu(unpack(c, "cu")) {
    if (table.scalar_type() != at::kInt || table.dim() != 2) refuse("block_table must be int32 [S, max_pages]");
    if (table.device() != dev || !table.is_contiguous())
      refuse("block_table must be contiguous on " + device_name(dev));
    S = rows32(table.size(0), "block_table");
    max_pages = rows32(table.size(1), "block_table");
    check_index(lengths, lengths_name, S, dev);
    check_index(cu, "cu", static_cast<int64_t>(S) + 1, dev);
  }
};

void* stream_of(const c10::Device& dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
const int32_t* i32(const Tensor& t) { return t.defined() ? t.const_data_ptr<int32_t>() : nullptr; }

void arity(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) refuse_type("expected " + std::to_string(want) + " arguments");
}

// (Q, K, positions, rope, q_weight, k_weight, eps, interleaved, q_out, k_out) -> (q_out, k_out) or a status
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 10);
  const Tensor Q = unpack(a[0], "Q"), K = unpack_optional(a[1], "K"), pos = unpack_optional(a[2], "positions"),
               rope = unpack_optional(a[3], "rope"), qw = unpack_optional(a[4], "q_weight"),
               kw = unpack_optional(a[5], "k_weight");
  Tensor qo = unpack_optional(a[8], "q_out"), ko = unpack_optional(a[9], "k_out");
  if (!Q.is_cuda()) refuse("Q must be on a CUDA device");
  if (Q.dim() != 3) refuse("Q must be [T, H_q, D]");
  const c10::Device dev = Q.device();
  const int64_t T = Q.size(0), H_q = Q.size(1), D = Q.size(2);
  const kvq_dtype code = dtype_code(Q);
  const int64_t qs = check_rows(Q, "Q", T, H_q, D, dev);
  int64_t H_kv = 0, ks = 0;
  if (K.defined()) {
    if (K.dim() != 3 || K.scalar_type() != Q.scalar_type()) refuse("K must be [T, H_kv, D] of Q's dtype");
    H_kv = K.size(1);
    ks = check_rows(K, "K", T, H_kv, D, dev);
  }
  for (const auto& [w, name] : {std::pair<const Tensor&, const char*>{qw, "q_weight"}, {kw, "k_weight"}})
    if (w.defined() && (w.device() != dev || w.scalar_type() != Q.scalar_type() || w.dim() != 1 || w.numel() != D ||
                        !w.is_contiguous()))
      refuse(std::string(name) + " must be contiguous [D] of Q's dtype on " + device_name(dev));
  const kvq_rope r = rope_arg(rope, to_bool(a[7]), D, dev);
  if (r.table) {
    if (!pos.defined()) refuse("a rotation needs positions");
    check_index(pos, "positions", T, dev);
  }
  const c10::cuda::CUDAGuard guard(dev);
  if (!qo.defined()) qo = new_dense({T, H_q, D}, Q.scalar_type(), dev);
  if (K.defined() && !ko.defined()) ko = new_dense({T, H_kv, D}, Q.scalar_type(), dev);
  if (!K.defined() && ko.defined()) refuse("k_out without K");
  for (const auto& [o, x, name] : {std::tuple<const Tensor&, const Tensor&, const char*>{qo, Q, "q_out"}, {ko, K, "k_out"}})
    if (x.defined() && (o.sizes() != x.sizes() || o.scalar_type() != x.scalar_type() || o.device() != dev ||
                        !o.is_contiguous()))
      refuse(std::string(name) + " must be contiguous and match its input");
  if (T > 0) {
    const kvq_status st = kvq_qk_norm_rope(ptr(Q), qs, ptr(K), ks, code, rows32(T, "Q"), rows32(H_q, "Q"),
                                           rows32(H_kv, "K"), rows32(D, "Q"), ptr(qw), ptr(kw),
                                           static_cast<float>(to_double(a[6])), r.table ? i32(pos) : nullptr, &r,
                                           ptr(qo), ptr(ko), stream_of(dev));
    if (st != KVQ_OK) return PyLong_FromLong(st);
  }
  PyObject* out = PyTuple_New(2);
  if (!out) raise_pending();
  PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(qo));
  if (K.defined()) {
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(ko));
  } else {
    Py_INCREF(Py_None);
    PyTuple_SET_ITEM(out, 1, Py_None);
  }
  return out;
  END_HANDLE_TH_ERRORS
}

// (cache, device, K, V, block_table, lengths, cu, max_new, rope, interleaved, slots) -> a status
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 11);
  const CacheArg cache(a[0], a[1]);
  const Tensor K = unpack(a[2], "K"), V = unpack(a[3], "V"), rope = unpack_optional(a[8], "rope"),
               slots = unpack_optional(a[10], "slots");
  const BatchArg batch(a[4], a[5], a[6], "lengths", cache.dev);
  if (K.dim() != 3 || K.scalar_type() != V.scalar_type()) refuse("K and V must be [T, H_kv, D] of one dtype");
  const int64_t T = K.size(0), H = cache.c->pages.H_kv, D = cache.c->pages.D;
  const int64_t ks = check_rows(K, "K", T, H, D, cache.dev), vs = check_rows(V, "V", T, H, D, cache.dev);
  if (slots.defined()) check_index(slots, "slots", batch.S, cache.dev);
  else if (batch.S > cache.c->tail_slots) refuse("more sequences than the cache has tail slots");
  const kvq_rope r = rope_arg(rope, to_bool(a[9]), D, cache.dev);
  const kvq_dtype code = dtype_code(K);
  const int32_t max_new = to_i32(a[7], "max_new");
  if (T == 0 || batch.S == 0) return PyLong_FromLong(KVQ_OK);
  const c10::cuda::CUDAGuard guard(cache.dev);
  return PyLong_FromLong(kvq_paged_append(cache.c, ptr(K), ks, ptr(V), vs, code, i32(batch.table), batch.max_pages,
                                          i32(batch.lengths), i32(batch.cu), i32(slots), batch.S, rows32(T, "K"),
                                          max_new, &r, stream_of(cache.dev)));
  END_HANDLE_TH_ERRORS
}

// (cache, device, block_table, starts, cu, rows, max_rows, bf16) -> (K, V) or a status
PyObject* paged_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 8);
  const CacheArg cache(a[0], a[1]);
  const BatchArg batch(a[2], a[3], a[4], "starts", cache.dev);
  const int32_t rows = to_i32(a[5], "rows"), max_rows = to_i32(a[6], "max_rows");
  if (rows < 0) refuse("rows must not be negative");
  const bool bf16 = to_bool(a[7]);
  const c10::cuda::CUDAGuard guard(cache.dev);
  const at::ScalarType type = bf16 ? at::kBFloat16 : at::kFloat;
  const Tensor K = new_dense({rows, cache.c->pages.H_kv, cache.c->pages.D}, type, cache.dev);
  const Tensor V = new_dense({rows, cache.c->pages.H_kv, cache.c->pages.D}, type, cache.dev);
  if (rows > 0 && batch.S > 0) {
    const kvq_status st =
        kvq_paged_gather(cache.c, i32(batch.table), batch.max_pages, i32(batch.lengths), i32(batch.cu), batch.S, rows,
                         max_rows, ptr(K), ptr(V), bf16 ? KVQ_BF16 : KVQ_F32, stream_of(cache.dev));
    if (st != KVQ_OK) return PyLong_FromLong(st);
  }
  PyObject* out = PyTuple_New(2);
  if (!out) raise_pending();
  PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(K));
  PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(V));
  return out;
  END_HANDLE_TH_ERRORS
}

// (cache, device, Q, block_table, lengths, cu, max_q, scale, causal, out, workspace, splits) -> out or a status
PyObject* paged_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 12);
  const CacheArg cache(a[0], a[1]);
  const Tensor Q = unpack(a[2], "Q");
  const BatchArg batch(a[3], a[4], a[5], "lengths", cache.dev);
  check_dense(Q, "Q", cache.dev);
  if (Q.dim() != 3 || Q.size(2) != cache.c->pages.D) refuse("Q must be [T, H_q, D]");
  const int32_t T = rows32(Q.size(0), "Q"), H_q = rows32(Q.size(1), "Q");
  const kvq_dtype code = dtype_code(Q);
  const int32_t max_q = to_i32(a[6], "max_q"), splits = to_i32(a[11], "splits");
  const c10::cuda::CUDAGuard guard(cache.dev);
  Tensor out = unpack_optional(a[9], "out"), ws = unpack_optional(a[10], "workspace");
  if (!out.defined()) {
    out = new_dense(Q.sizes(), Q.scalar_type(), cache.dev);
  } else {
    check_dense(out, "out", cache.dev);
    if (out.sizes() != Q.sizes() || out.scalar_type() != Q.scalar_type()) refuse("out must match Q");
  }
  if (T > 0 && batch.S > 0) {
    if (!ws.defined()) {
      const size_t need = kvq_paged_workspace_size(cache.c, code, batch.S, T, max_q, H_q, splits);
      ws = new_dense({static_cast<int64_t>(need > 16 ? need : 16)}, at::kByte, cache.dev);
    } else {
      check_dense(ws, "workspace", cache.dev);
    }
    const kvq_status st = kvq_paged_attend(ptr(Q), code, cache.c, i32(batch.table), batch.max_pages,
                                           i32(batch.lengths), i32(batch.cu), batch.S, T, max_q, H_q,
                                           static_cast<float>(to_double(a[7])), to_bool(a[8]), ptr(out), ptr(ws),
                                           static_cast<size_t>(ws.numel()) * ws.element_size(), splits,
                                           stream_of(cache.dev));
    if (st != KVQ_OK) return PyLong_FromLong(st);
  }
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(qk_norm_rope)), METH_FASTCALL, nullptr},
    {"paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_append)), METH_FASTCALL, nullptr},
    {"paged_gather", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_gather)), METH_FASTCALL, nullptr},
    {"paged_attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_attend)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__calls() { return PyModule_Create(&kModule); }
