// The Python side of the cache calls: argument checks, output allocation and the call of the C
// entry point, for torch tensors.
//
// A call marshals some twenty values for kernels that may take a few microseconds.  In Python
// (attribute reads, ctypes conversions) that cost 25 us a call on a GB300 host; here, with the
// tensors' fields at hand, it is a small part of the launch itself.  cache.py documents the calls and
// passes their arguments on in order.

#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <array>
#include <cmath>
#include <optional>
#include <string>

#include "specdec.h"

namespace {

// An error that becomes a Python exception of the given type.
struct Refused {
  PyObject* type;
  std::string what;
};
[[noreturn]] void value_error(const std::string& what) { throw Refused{PyExc_ValueError, what}; }

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}
std::string text(at::ScalarType t) { return std::string(c10::toString(t)); }

bool half(at::ScalarType t) { return t == at::kBFloat16 || t == at::kHalf; }
specdec_dtype code(at::ScalarType t) { return t == at::kBFloat16 ? SPECDEC_BF16 : SPECDEC_F16; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + " must be a torch.Tensor"};
  return THPVariable_Unpack(o);
}

// The first three strides of a [.., .., .., D] tensor in units of `unit`, 0 for dimensions of one
// entry (whose stride means nothing); false where the last dimension is not contiguous.
bool strides(const at::Tensor& t, int64_t unit, int64_t (&out)[3]) {
  if (t.stride(3) != 1) return false;
  for (int i = 0; i < 3; ++i) out[i] = t.size(i) == 1 ? 0 : t.stride(i) * unit;
  return true;
}

struct View {
  const void* p = nullptr;
  int64_t st[3] = {0, 0, 0};
};
View view(const at::Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape, c10::Device device) {
  if (t.scalar_type() != dtype) value_error(std::string(name) + " must be " + text(dtype) + ", got " + text(t.scalar_type()));
  if (t.sizes() != shape) value_error(std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
  if (t.device() != device) value_error(std::string(name) + " is on " + t.device().str() + ", expected " + device.str());
  View v;
  if (!strides(t, 1, v.st)) value_error(std::string(name) + "'s last dimension must be contiguous");
  v.p = t.data_ptr();
  return v;
}

// A contiguous tensor's address (None: null).
template <typename P>
const P* small(PyObject* o, const char* name, at::ScalarType dtype, at::IntArrayRef shape, c10::Device device) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != dtype || t.sizes() != shape || t.device() != device || !t.is_contiguous())
    value_error(std::string(name) + " must be a contiguous " + text(dtype) + " tensor of shape " + text(shape) + " on " +
                device.str() + ", got " + text(t.scalar_type()) + " " + text(t.sizes()) + " on " + t.device().str());
  return static_cast<const P*>(t.data_ptr());
}

double number(PyObject* o) {
  const double d = PyFloat_AsDouble(o);
  if (d == -1.0 && PyErr_Occurred()) throw python_error();
  return d;
}
// An int argument; values that do not fit an int are refused, not cut.
int integer(PyObject* o, const char* name) {
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (v == -1 && !over && PyErr_Occurred()) throw python_error();
  if (over || v > INT32_MAX || v < INT32_MIN) value_error(std::string(name) + " does not fit an int");
  return static_cast<int>(v);
}
bool truth(PyObject* o) {
  const int yes = PyObject_IsTrue(o);
  if (yes < 0) throw python_error();
  return yes != 0;
}
int dimension(int64_t v, const char* name) {
  if (v > INT32_MAX) value_error(std::string(name) + " does not fit an int");
  return static_cast<int>(v);
}

c10::Device cuda_device(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) value_error(std::string("the cache calls take CUDA tensors, ") + name + " is on " + t.device().str());
  return t.device();
}

specdec_kv_pages pages(PyObject* ko, PyObject* vo, PyObject* table, int64_t B, c10::Device device, int64_t head_dim,
                       PyObject* ks, PyObject* vs, PyObject* k_scale, PyObject* v_scale) {
  const at::Tensor &k = tensor(ko, "k_pages"), &v = tensor(vo, "v_pages");
  const at::ScalarType dt = k.scalar_type();
  const bool four = dt == at::kByte;
  if ((!four && !half(dt)) || k.dim() != 4)
    value_error("pages must be [num_pages, page_size, kv_heads, head_dim] of bfloat16 or float16, or uint8 codes [..., head_dim / 2]");
  if (v.scalar_type() != dt || v.sizes() != k.sizes() || k.device() != device || v.device() != device)
    value_error("k_pages and v_pages must have the same type and shape, on the call's device");
  const int64_t unit = four ? 1 : 2;
  int64_t st[3], other[3];
  if (!strides(k, unit, st) || !strides(v, unit, other) || st[0] != other[0] || st[1] != other[1] || st[2] != other[2])
    value_error("k_pages and v_pages must have the same strides and a contiguous last dimension");
  specdec_kv_pages pg{};
  pg.num_pages = dimension(k.size(0), "num_pages");
  pg.page_size = dimension(k.size(1), "page_size");
  pg.kv_heads = dimension(k.size(2), "kv_heads");
  pg.head_dim = dimension(k.size(3) * (four ? 2 : 1), "head_dim");
  if (head_dim >= 0 && pg.head_dim != head_dim)
    value_error("the pages hold heads of " + std::to_string(pg.head_dim) + ", the call has " + std::to_string(head_dim));
  pg.k = k.data_ptr();
  pg.v = v.data_ptr();
  pg.page_stride = st[0];
  pg.slot_stride = st[1];
  pg.head_stride = st[2];
  if (!THPVariable_Check(table) || THPVariable_Unpack(table).dim() != 2) value_error("block_table must be [B, max_pages] int32");
  const int64_t per = THPVariable_Unpack(table).size(1);
  pg.block_table = small<int32_t>(table, "block_table", at::kInt, {B, per}, device);
  pg.max_pages = dimension(per, "max_pages");
  pg.k_scale = pg.v_scale = 1.f;
  if (!four) {
    if (ks != Py_None || vs != Py_None) value_error("16-bit pages have no scales");
    pg.format = code(dt);
    return pg;
  }
  const int64_t want[4] = {k.size(0), k.size(1), k.size(2), pg.head_dim / 16};
  int64_t sst[2][3];
  void* sp[2];
  for (int i = 0; i < 2; ++i) {
    PyObject* o = i ? vs : ks;
    const std::string name = i ? "v_scales" : "k_scales";
    if (!THPVariable_Check(o)) value_error("pages held in 4 bits need " + name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if ((t.scalar_type() != at::kByte && t.scalar_type() != at::kFloat8_e4m3fn) || t.sizes() != at::IntArrayRef(want, 4) || t.device() != device)
      value_error(name + " must be E4M3 bytes of shape " + text(at::IntArrayRef(want, 4)) + " on " + device.str());
    if (!strides(t, 1, sst[i])) value_error(name + "'s last dimension must be contiguous");
    sp[i] = t.data_ptr();
  }
  if (sst[0][0] != sst[1][0] || sst[0][1] != sst[1][1] || sst[0][2] != sst[1][2])
    value_error("k_scales and v_scales must have the same strides");
  pg.k_scales = sp[0];
  pg.v_scales = sp[1];
  pg.scale_page_stride = sst[0][0];
  pg.scale_slot_stride = sst[0][1];
  pg.scale_head_stride = sst[0][2];
  pg.format = SPECDEC_KV4;
  pg.k_scale = static_cast<float>(number(k_scale));
  pg.v_scale = static_cast<float>(number(v_scale));
  return pg;
}

// The result dict's entries (a new reference each, handed over to the dict).
void put(PyObject* dict, const char* key, at::Tensor t) {
  PyObject* o = THPVariable_Wrap(std::move(t));
  if (o == nullptr) throw python_error();
  const int rc = PyDict_SetItemString(dict, key, o);
  Py_DECREF(o);
  if (rc != 0) throw python_error();
}
struct Dict {
  PyObject* p = PyDict_New();
  ~Dict() { Py_XDECREF(p); }
  PyObject* release() {
    PyObject* r = p;
    p = nullptr;
    return r;
  }
};

// A nonzero return code raises the package's SpecdecError.
void checked(int rc, const char* what) {
  if (rc == SPECDEC_OK) return;
  PyObject* m = PyImport_ImportModule("speculative_decoding_token_temperature_gb300.cache");
  if (m == nullptr) throw python_error();
  PyObject* r = PyObject_CallMethod(m, "_failed", "iss", rc, what, specdec_last_error());
  Py_DECREF(m);
  Py_XDECREF(r);
  throw python_error();
}

// A workspace per device and stream, for the streams that were last used: a program may make any
// number of them, and a workspace takes up to 42 MB.  (From the allocator for each call it cost 2 us a call,
// 7.5 against 9.7.)  What is let go returns to the allocator's memory of its stream, whose order covers
// the kernels that still use it.  During a capture a graph gets its own: a kept one may be replaced by a
// larger one later.  (The table is never destroyed: its tensors must not outlive CUDA.)
constexpr size_t kKeptWorkspaces = 8;
struct Kept {
  cudaStream_t stream = nullptr;
  c10::DeviceIndex device = -1;
  at::Tensor ws;
};
at::Tensor workspace(int64_t bytes, c10::Device device, cudaStream_t stream) {
  const auto options = at::TensorOptions().dtype(at::kByte).device(device);
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  C10_CUDA_CHECK(cudaStreamIsCapturing(stream, &status));
  if (status != cudaStreamCaptureStatusNone) return at::empty({bytes}, options);
  static auto* const kept = new std::array<Kept, kKeptWorkspaces>();  // the last used first
  size_t at = 0;
  while (at + 1 < kKeptWorkspaces && ((*kept)[at].stream != stream || (*kept)[at].device != device.index())) ++at;
  std::rotate(kept->begin(), kept->begin() + at, kept->begin() + at + 1);
  Kept& k = kept->front();
  if (k.stream != stream || k.device != device.index()) k = Kept{stream, device.index(), at::Tensor()};
  if (!k.ws.defined() || k.ws.numel() < bytes) {
    k.ws = at::Tensor();
    k.ws = at::empty({bytes}, options);
  }
  return k.ws;
}

at::TensorOptions on(c10::Device device, at::ScalarType t) { return at::TensorOptions().dtype(t).device(device); }

template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F&& f) {
  HANDLE_TH_ERRORS
  if (given != wanted) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// q, k, turns, context_len, query_len, depth, q_weight, k_weight, eps, interleaved, v, k_pages, v_pages, block_table
PyObject* rotate_qk(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 14, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &turns = tensor(a[2], "turns");
    const at::ScalarType dt = q.scalar_type();
    if (q.dim() != 4 || !half(dt)) value_error("q must be [B, n, q_heads, D] bfloat16 or float16");
    if (k.dim() != 4) value_error("k must be [B, n, kv_heads, D]");
    const c10::Device dev = cuda_device(q, "q");
    const int64_t B = q.size(0), n = q.size(1), hq = q.size(2), D = q.size(3), hkv = k.size(2);
    const View qv = view(q, "q", dt, q.sizes(), dev), kv = view(k, "k", dt, {B, n, hkv, D}, dev);
    if (turns.dim() != 1) value_error("turns must be [rot / 2] int64");
    const int64_t half_rot = turns.size(0);
    const auto* tp = small<uint64_t>(a[2], "turns", at::kLong, {half_rot}, dev);
    const auto* lens = small<int32_t>(a[3], "context_len", at::kInt, {B}, dev);
    const auto* ql = small<int32_t>(a[4], "query_len", at::kInt, {B}, dev);
    const auto* depth = small<int32_t>(a[5], "depth", at::kInt, {n}, dev);
    const auto* wq = small<void>(a[6], "q_weight", dt, {D}, dev);
    const auto* wk = small<void>(a[7], "k_weight", dt, {D}, dev);
    const float eps = static_cast<float>(number(a[8]));
    const int interleaved = truth(a[9]) ? 1 : 0;
    const bool paged = a[11] != Py_None || a[12] != Py_None || a[13] != Py_None;
    View vv;
    specdec_kv_pages pg{};
    if (paged) {
      vv = view(tensor(a[10], "v"), "v", dt, {B, n, hkv, D}, dev);
      pg = pages(a[11], a[12], a[13], B, dev, D, Py_None, Py_None, nullptr, nullptr);
    }
    const c10::cuda::OptionalCUDAGuard guard(dev);
    at::Tensor out_q = at::empty({B, n, hq, D}, on(dev, dt)), status = at::empty({B}, on(dev, at::kInt)), out_k;
    if (!paged) out_k = at::empty({B, n, hkv, D}, on(dev, dt));
    checked(specdec_rotate_qk(qv.p, qv.st, kv.p, kv.st, vv.p, vv.st, code(dt), wq, wk, eps, tp, dimension(2 * half_rot, "rot"),
                              interleaved, lens, ql, depth, dimension(B, "B"), dimension(n, "n"), dimension(hq, "q_heads"),
                              dimension(hkv, "kv_heads"), dimension(D, "D"), out_q.data_ptr(), paged ? nullptr : out_k.data_ptr(),
                              paged ? &pg : nullptr, static_cast<int32_t*>(status.data_ptr()),
                              c10::cuda::getCurrentCUDAStream(dev.index()).stream()),
            "specdec_rotate_qk");
    Dict out;
    put(out.p, "q", std::move(out_q));
    put(out.p, "status", std::move(status));
    if (!paged) put(out.p, "k", std::move(out_k));
    return out.release();
  });
}

// k, v, k_pages, v_pages, block_table, context_len, query_len, k_scales, v_scales, k_scale, v_scale
PyObject* append_kv4(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 11, [&]() -> PyObject* {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const at::ScalarType dt = k.scalar_type();
    if (k.dim() != 4 || !half(dt)) value_error("k must be [B, n, kv_heads, D] bfloat16 or float16");
    const c10::Device dev = cuda_device(k, "k");
    const int64_t B = k.size(0), n = k.size(1), hkv = k.size(2), D = k.size(3);
    const View kv = view(k, "k", dt, k.sizes(), dev), vv = view(v, "v", dt, k.sizes(), dev);
    const specdec_kv_pages pg = pages(a[2], a[3], a[4], B, dev, D, a[7], a[8], a[9], a[10]);
    if (pg.kv_heads != hkv) value_error("the pages hold " + std::to_string(pg.kv_heads) + " heads, k has " + std::to_string(hkv));
    const auto* lens = small<int32_t>(a[5], "context_len", at::kInt, {B}, dev);
    const auto* ql = small<int32_t>(a[6], "query_len", at::kInt, {B}, dev);
    const c10::cuda::OptionalCUDAGuard guard(dev);
    at::Tensor status = at::empty({B}, on(dev, at::kInt));
    checked(specdec_append_kv4(kv.p, kv.st, vv.p, vv.st, code(dt), lens, ql, dimension(B, "B"), dimension(n, "n"), &pg,
                               static_cast<int32_t*>(status.data_ptr()), c10::cuda::getCurrentCUDAStream(dev.index()).stream()),
            "specdec_append_kv4");
    Dict out;
    put(out.p, "status", std::move(status));
    return out.release();
  });
}

// k_pages, v_pages, block_table, context_len, n, query_len, k_scales, v_scales, k_scale, v_scale, bfloat16?
PyObject* read_kv4(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 11, [&]() -> PyObject* {
    const at::Tensor &k = tensor(a[0], "k_pages"), &len = tensor(a[3], "context_len");
    const c10::Device dev = cuda_device(k, "k_pages");
    if (len.dim() != 1) value_error("context_len must be [B] int32");
    const int64_t B = len.size(0);
    const int n = integer(a[4], "n");
    const at::ScalarType dt = truth(a[10]) ? at::kBFloat16 : at::kHalf;
    const specdec_kv_pages pg = pages(a[0], a[1], a[2], B, dev, -1, a[6], a[7], a[8], a[9]);
    const auto* lens = small<int32_t>(a[3], "context_len", at::kInt, {B}, dev);
    const auto* ql = small<int32_t>(a[5], "query_len", at::kInt, {B}, dev);
    const c10::cuda::OptionalCUDAGuard guard(dev);
    const int64_t shape[4] = {B, n > 0 ? n : 0, pg.kv_heads, pg.head_dim};
    at::Tensor out_k = at::empty(at::IntArrayRef(shape, 4), on(dev, dt)), out_v = at::empty(at::IntArrayRef(shape, 4), on(dev, dt));
    at::Tensor status = at::empty({B}, on(dev, at::kInt));
    checked(specdec_read_kv4(lens, ql, dimension(B, "B"), n, &pg, code(dt), out_k.data_ptr(), out_v.data_ptr(),
                             static_cast<int32_t*>(status.data_ptr()), c10::cuda::getCurrentCUDAStream(dev.index()).stream()),
            "specdec_read_kv4");
    Dict out;
    put(out.p, "k", std::move(out_k));
    put(out.p, "v", std::move(out_v));
    put(out.p, "status", std::move(status));
    return out.release();
  });
}

// q, k_pages, v_pages, block_table, context_len, query_len, tree_mask, depth, window, sinks, scale, k_scales, v_scales,
// k_scale, v_scale, with_lse
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 16, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    const at::ScalarType dt = q.scalar_type();
    if (q.dim() != 4 || !half(dt)) value_error("q must be [B, n, q_heads, D] bfloat16 or float16");
    const c10::Device dev = cuda_device(q, "q");
    const int64_t B = q.size(0), n = q.size(1), hq = q.size(2), D = q.size(3);
    const View qv = view(q, "q", dt, q.sizes(), dev);
    const specdec_kv_pages pg = pages(a[1], a[2], a[3], B, dev, D, a[11], a[12], a[13], a[14]);
    if (pg.format != SPECDEC_KV4 && pg.format != code(dt))
      value_error("q is " + text(dt) + ", the pages are " + text(THPVariable_Unpack(a[1]).scalar_type()));
    const auto* lens = small<int32_t>(a[4], "context_len", at::kInt, {B}, dev);
    const auto* ql = small<int32_t>(a[5], "query_len", at::kInt, {B}, dev);
    const auto* mask = small<uint8_t>(a[6], "tree_mask", at::kByte, {n, n}, dev);
    const auto* depth = small<int32_t>(a[7], "depth", at::kInt, {n}, dev);
    const int window = integer(a[8], "window"), sinks = integer(a[9], "sinks");
    const float scale = a[10] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D))) : static_cast<float>(number(a[10]));
    const bool with_lse = truth(a[15]);
    const int Bi = dimension(B, "B"), ni = dimension(n, "n"), hi = dimension(hq, "q_heads"), Di = dimension(D, "D");
    const c10::cuda::OptionalCUDAGuard guard(dev);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    at::Tensor o = at::empty({B, n, hq, D}, on(dev, dt)), status = at::empty({B}, on(dev, at::kInt)), lse;
    if (with_lse) lse = at::empty({B, n, hq}, on(dev, at::kFloat));
    const size_t need = specdec_attend_workspace_bytes(Bi, ni, hi, pg.kv_heads, Di);
    at::Tensor ws = workspace(need > 0 ? static_cast<int64_t>(need) : 256, dev, stream);
    checked(specdec_attend(qv.p, qv.st, code(dt), &pg, lens, ql, mask, depth, Bi, ni, hi, window, sinks, scale, o.data_ptr(),
                           with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr, static_cast<int32_t*>(status.data_ptr()),
                           ws.data_ptr(), static_cast<size_t>(ws.numel()), stream),
            "specdec_attend");
    Dict out;
    put(out.p, "out", std::move(o));
    put(out.p, "status", std::move(status));
    if (with_lse) put(out.p, "lse", std::move(lse));
    return out.release();
  });
}

#define CALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(rotate_qk), CALL(append_kv4), CALL(read_kv4), CALL(attend), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cache_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_calls() { return PyModule_Create(&module); }
