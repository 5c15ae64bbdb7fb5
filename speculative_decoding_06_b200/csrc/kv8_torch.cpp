// Python binding of the spec_kv8_* calls over torch tensors: argument checks and
// marshalling only.  A step's calls last a few microseconds on the GPU; checking a
// dozen tensors through the ctypes binding took 15-19 us per call on the host, here
// 4-6 with the launch.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <optional>
#include <string>

#include "../../include/spec.h"

namespace {

constexpr int64_t kHd = 128;

// what the wrapper raises: a ValueError for tensors that do not fit, or the library's error code
struct BadValue : std::exception {
  std::string msg;
  explicit BadValue(std::string m) : msg(std::move(m)) {}
};

[[noreturn]] void bad(const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  throw BadValue(buf);
}

struct Cache {
  spec_kv8* h;
  c10::DeviceIndex device;
  int64_t hkv;
};

const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (o == Py_None && optional) return nullptr;
  if (!THPVariable_Check(o)) bad("%s must be a torch tensor", name);
  return &THPVariable_Unpack(o);
}

void on_device(const at::Tensor& t, const Cache& c, const char* name) {
  if (!t.is_cuda() || t.get_device() != c.device) bad("%s must be on cuda:%d", name, (int)c.device);
}

// a contiguous int32 tensor of this shape (d1 < 0: one dimension)
int32_t* ints(const at::Tensor* t, const Cache& c, const char* name, int64_t d0, int64_t d1 = -1) {
  if (!t) return nullptr;
  on_device(*t, c, name);
  if (t->scalar_type() != at::kInt || !t->is_contiguous()) bad("%s must be a contiguous int32 tensor", name);
  if (t->dim() != (d1 < 0 ? 1 : 2) || t->size(0) != d0 || (d1 >= 0 && t->size(1) != d1))
    bad("%s must have shape [%lld%s%s]", name, (long long)d0, d1 < 0 ? "" : "][",
        d1 < 0 ? "" : std::to_string(d1).c_str());
  return t->data_ptr<int32_t>();
}

// [rows][heads][128] with contiguous values of a head (the stride of a dimension of one counts for nothing)
void rows_of(const at::Tensor& t, const Cache& c, const char* name, int64_t heads, int64_t* row_stride,
             int64_t* head_stride) {
  on_device(t, c, name);
  if (t.dim() != 3 || t.size(1) != heads || t.size(2) != kHd || (t.numel() && t.stride(2) != 1))
    bad("%s must be [rows][%lld][128] with contiguous values", name, (long long)heads);
  *head_stride = heads == 1 ? kHd : t.stride(1);
  *row_stride = t.size(0) <= 1 ? heads * kHd : t.stride(0);
}

int dtype_of(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kFloat: return SPEC_DTYPE_F32;
    case at::kBFloat16: return SPEC_DTYPE_BF16;
    case at::kHalf: return SPEC_DTYPE_F16;
    default: bad("%s must be fp32, bf16 or fp16", name);
  }
}

int to_int(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::exception();
  if (v < INT32_MIN || v > INT32_MAX) bad("%s does not fit 32 bits", name);
  return (int)v;
}

int count(int64_t n, const char* name) {
  if (n > INT32_MAX) bad("%s does not fit 32 bits", name);
  return (int)n;
}

Cache cache_of(PyObject* const* args) {
  Cache c;
  c.h = static_cast<spec_kv8*>(PyLong_AsVoidPtr(args[0]));
  c.device = (c10::DeviceIndex)to_int(args[1], "device");
  c.hkv = to_int(args[2], "n_kv_heads");
  if (!c.h) bad("the cache is closed");
  return c;
}

// Runs `body`, which returns a new reference, on the cache's device; C++ exceptions become Python's.
template <typename F>
PyObject* guarded(F&& body) {
  try {
    return body();
  } catch (const BadValue& e) {
    PyErr_SetString(PyExc_ValueError, e.msg.c_str());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

// plan(h, device, hkv, n_pages, lengths, add, tables, ring, state, max_rows, seq_ids, offsets, slots, lengths_out,
//      state_out, status) -> return code
PyObject* py_plan(PyObject*, PyObject* const* p, Py_ssize_t n) {
  if (!arity(n, 16)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Cache c = cache_of(p);
    const at::Tensor *tables = tensor(p[6], "tables"), *add = tensor(p[5], "add");
    if (tables->dim() != 2) bad("tables must be [n_seqs][max_blocks]");
    if (add->dim() != 1) bad("add must be [batch]");
    const int64_t n_seqs = tables->size(0), blocks = tables->size(1), batch = add->size(0);
    spec_kv8_plan_args a{};
    a.max_rows = to_int(p[9], "max_rows");
    a.lengths = ints(tensor(p[4], "lengths"), c, "lengths", n_seqs);
    a.add = ints(add, c, "add", batch);
    a.tables = ints(tables, c, "tables", n_seqs, blocks);
    a.ring = ints(tensor(p[7], "ring"), c, "ring", to_int(p[3], "n_pages"));
    a.state = ints(tensor(p[8], "state"), c, "state", 2);
    a.seq_ids = ints(tensor(p[10], "seq_ids", true), c, "seq_ids", batch);
    a.offsets = ints(tensor(p[11], "offsets"), c, "offsets", batch + 1);
    a.slots = ints(tensor(p[12], "slots"), c, "slots", a.max_rows < 0 ? 0 : a.max_rows);
    a.lengths_out = ints(tensor(p[13], "lengths"), c, "lengths", n_seqs);
    a.state_out = ints(tensor(p[14], "state"), c, "state", 2);
    a.status = ints(tensor(p[15], "status"), c, "status", 1);
    a.batch = count(batch, "batch");
    a.n_seqs = count(n_seqs, "n_seqs");
    a.max_blocks = count(blocks, "max_blocks");
    c10::cuda::CUDAGuard guard(c.device);
    return PyLong_FromLong(spec_kv8_plan(c.h, &a, c10::cuda::getCurrentCUDAStream(c.device).stream()));
  });
}

// append(h, device, hkv, layer, k, v, slots, src_rows) -> return code
PyObject* py_append(PyObject*, PyObject* const* p, Py_ssize_t n) {
  if (!arity(n, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Cache c = cache_of(p);
    const at::Tensor &k = *tensor(p[4], "k"), &v = *tensor(p[5], "v");
    const at::Tensor* slots = tensor(p[6], "slots");
    if (k.scalar_type() != v.scalar_type()) bad("k and v must have one dtype");
    spec_kv8_append_args a{};
    a.dtype = dtype_of(k, "k");
    rows_of(k, c, "k", c.hkv, &a.k_row_stride, &a.k_head_stride);
    rows_of(v, c, "v", c.hkv, &a.v_row_stride, &a.v_head_stride);
    if (k.size(0) != v.size(0)) bad("k and v have %lld and %lld rows", (long long)k.size(0), (long long)v.size(0));
    const int64_t rows = slots->dim() == 1 ? slots->size(0) : -1;
    a.k = k.data_ptr();
    a.v = v.data_ptr();
    a.slots = ints(slots, c, "slots", rows);
    a.src_rows = ints(tensor(p[7], "src_rows", true), c, "src_rows", rows);
    a.rows = count(rows, "rows");
    a.n_src = count(k.size(0), "rows");
    c10::cuda::CUDAGuard guard(c.device);
    return PyLong_FromLong(
        spec_kv8_append(c.h, to_int(p[3], "layer"), &a, c10::cuda::getCurrentCUDAStream(c.device).stream()));
  });
}

// attention(h, device, hkv, layer, q, tables, lengths, offsets, max_prefix, max_nodes, k_new, v_new, parents, seq_ids,
//           scale, out, lse, workspace) -> (return code, out, lse)
PyObject* py_attention(PyObject*, PyObject* const* p, Py_ssize_t n) {
  if (!arity(n, 18)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Cache c = cache_of(p);
    const at::Tensor &q = *tensor(p[4], "q"), &tables = *tensor(p[5], "tables"), &offsets = *tensor(p[7], "offsets");
    const at::Tensor *k = tensor(p[10], "k_new", true), *v = tensor(p[11], "v_new", true);
    const at::Tensor *out = tensor(p[15], "out", true), *lse = tensor(p[16], "lse", true);
    const at::Tensor* ws = tensor(p[17], "workspace", true);
    if (q.dim() != 3) bad("q must be [rows][n_q_heads][128]");
    if (tables.dim() != 2) bad("tables must be [n_seqs][max_blocks]");
    if (offsets.dim() != 1 || offsets.size(0) < 1) bad("offsets must be [batch + 1]");
    const int64_t rows = q.size(0), hq = q.size(1), batch = offsets.size(0) - 1;
    spec_kv8_attention_args a{};
    a.dtype = dtype_of(q, "q");
    if (a.dtype == SPEC_DTYPE_F32) bad("q must be bf16 or fp16");
    rows_of(q, c, "q", hq, &a.q_row_stride, &a.q_head_stride);
    a.q = q.data_ptr();
    if (!k != !v) bad("k_new and v_new go together");
    if (k) {
      if (k->scalar_type() != q.scalar_type() || v->scalar_type() != q.scalar_type())
        bad("k_new and v_new must have q's dtype");
      rows_of(*k, c, "k_new", c.hkv, &a.k_row_stride, &a.k_head_stride);
      rows_of(*v, c, "v_new", c.hkv, &a.v_row_stride, &a.v_head_stride);
      if (k->size(0) != rows || v->size(0) != rows) bad("k_new and v_new must have q's %lld rows", (long long)rows);
      a.k_new = k->data_ptr();
      a.v_new = v->data_ptr();
    }
    a.n_seqs = count(tables.size(0), "n_seqs");
    a.max_blocks = count(tables.size(1), "max_blocks");
    a.batch = count(batch, "batch");
    a.rows = count(rows, "rows");
    a.n_q_heads = count(hq, "n_q_heads");
    a.max_prefix = to_int(p[8], "max_prefix");
    a.max_nodes = to_int(p[9], "max_nodes");
    a.scale = (float)PyFloat_AsDouble(p[14]);
    if (PyErr_Occurred()) return nullptr;
    a.tables = ints(&tables, c, "tables", a.n_seqs, a.max_blocks);
    a.lengths = ints(tensor(p[6], "lengths"), c, "lengths", a.n_seqs);
    a.offsets = ints(&offsets, c, "offsets", batch + 1);
    a.parents = ints(tensor(p[12], "parents", true), c, "parents", rows);
    a.seq_ids = ints(tensor(p[13], "seq_ids", true), c, "seq_ids", batch);
    c10::cuda::CUDAGuard guard(c.device);
    at::Tensor new_out, new_lse, new_ws;
    if (!out) {
      new_out = at::empty({rows, hq, kHd}, q.options());
      out = &new_out;
      a.fill |= SPEC_KV8_FILL_OUT;  // (nothing of new memory stays as it was)
    } else if (out->scalar_type() != q.scalar_type() || out->dim() != 3 || out->size(0) != rows ||
               (rows && hq > 1 && out->stride(1) != kHd)) {
      bad("out must have q's dtype and shape, its heads contiguous");
    }
    int64_t head_stride;
    rows_of(*out, c, "out", hq, &a.out_row_stride, &head_stride);
    a.out = out->data_ptr();
    if (!lse) {
      new_lse = at::empty({rows, hq}, q.options().dtype(at::kFloat));
      lse = &new_lse;
      a.fill |= SPEC_KV8_FILL_LSE;
    } else if (lse->scalar_type() != at::kFloat || lse->dim() != 2 || lse->size(0) != rows || lse->size(1) != hq ||
               !lse->is_contiguous()) {
      bad("lse must be contiguous fp32 [rows][n_q_heads]");
    }
    on_device(*lse, c, "lse");
    a.lse = lse->data_ptr<float>();
    if (!ws) {
      const size_t bytes = spec_kv8_attention_workspace(c.h, a.batch, a.n_q_heads, a.max_nodes, a.max_prefix);
      new_ws = at::empty({(int64_t)bytes}, q.options().dtype(at::kByte));
      if (bytes) new_ws.narrow(0, 0, std::min<int64_t>(bytes, SPEC_KV8_WORKSPACE_ZERO)).zero_();
      ws = &new_ws;
    }
    on_device(*ws, c, "workspace");
    if (!ws->is_contiguous()) bad("workspace must be contiguous");
    a.workspace = ws->data_ptr();
    a.workspace_bytes = ws->nbytes();
    const int rc = spec_kv8_attention(c.h, to_int(p[3], "layer"), &a, c10::cuda::getCurrentCUDAStream(c.device).stream());
    PyObject* r = PyTuple_New(3);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, PyLong_FromLong(rc));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(*out));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(*lse));
    return r;
  });
}

PyMethodDef kMethods[] = {
    {"plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_plan)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_append)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_kv8", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv8() { return PyModule_Create(&kModule); }
