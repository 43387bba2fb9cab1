// py_binding.cpp -- marshalling of torch tensors into the generation path's entry points.
//
// A step of generation is three launches of a few microseconds each per layer; taking the tensors
// apart in Python and passing twenty arguments through ctypes took 15 to 20 us a call on the host of a
// GB300, several times the kernels.  These functions do the same checks, allocate the outputs and
// call the C entry point of libattn_gb300.so; nothing is computed here.  Each runs on the current
// stream of its tensors' device.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <optional>
#include <string>

#include "attn_gb300.h"

namespace {

PyObject* g_error = nullptr;  // the binding's exception class, called with (entry point, status)

// Raised through torch's translation as ValueError.
void require(bool ok, const char* message) { TORCH_CHECK_VALUE(ok, message); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}
at::Tensor maybe(PyObject* o, const char* name) { return o == Py_None ? at::Tensor() : tensor(o, name); }

int integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, name, " does not fit 32 bits");
  return static_cast<int>(v);
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(v);
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

// The address of a contiguous tensor of this type and shape on this device (null: no tensor).
void* address(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, at::Device dev,
              const char* name) {
  if (!t.defined()) return nullptr;
  TORCH_CHECK_VALUE(t.scalar_type() == type && t.sizes() == shape && t.device() == dev &&
                        t.is_contiguous(),
                    name, " must be a contiguous ", type, " tensor of shape ", shape, " on ", dev);
  return t.data_ptr();
}

// The workspace given for a call on `dev` (undefined: none).  Its size is the entry point's to check.
at::Tensor workspace(PyObject* o, at::Device dev) {
  const at::Tensor ws = maybe(o, "workspace");
  require(!ws.defined() || (ws.device() == dev && ws.is_contiguous()),
          "the workspace must be contiguous and on the inputs' device");
  return ws;
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

// A contiguous tensor over part of `whole`'s memory, `at` bytes in (a multiple of the type's size): one
// allocation for a call's small outputs, each 0.8 us of host time by itself.
at::Tensor carve(const at::Tensor& whole, int64_t at, at::IntArrayRef shape, at::ScalarType type) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(whole.storage()), whole.key_set(), c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_storage_offset(at / static_cast<int64_t>(c10::elementSize(type)));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

PyObject* wrap(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
PyObject* pack(std::initializer_list<at::Tensor> ts) {
  PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!out) throw python_error();
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(out, i++, wrap(t));
  return out;
}

void check(const char* entry, int rc) {
  if (rc == 0) return;
  if (PyObject* e = PyObject_CallFunction(g_error, "si", entry, rc)) {
    PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e)), e);
    Py_DECREF(e);
  }
  throw python_error();
}

struct Launch {
  c10::cuda::CUDAGuard guard;
  void* stream;
  explicit Launch(at::Device dev)
      : guard(dev), stream(c10::cuda::getCurrentCUDAStream(dev.index()).stream()) {}
};

attn_kv_cache cache_struct(PyObject* const* a, int64_t H_kv, int64_t d, at::Device dev) {
  const at::Tensor &k = tensor(a[0], "cache.k"), &v = tensor(a[1], "cache.v");
  require(k.dim() == 4 && k.sizes() == v.sizes() && k.scalar_type() == v.scalar_type() &&
              k.device() == dev && v.device() == dev,
          "cache k and v must be [num_pages, H_kv, page_size, d] tensors of one type on the inputs' "
          "device");
  const int64_t n = k.size(0), page = k.size(2);
  require(k.size(1) == H_kv && k.size(3) == d,
          "the cache's heads or head dim differ from the inputs'");
  // strides of dimensions of one element are free
  const int64_t want[4] = {0, page * d, d, 1};
  bool inner = true;
  for (int i = 1; i < 4; ++i)
    for (const at::Tensor* t : {&k, &v}) inner &= k.size(i) <= 1 || t->stride(i) == want[i];
  require(inner && (n <= 1 || k.stride(0) == v.stride(0)),
          "cache pages must be contiguous, with one page stride for k and v");
  attn_kv_cache c{};
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.page_stride = n > 1 ? k.stride(0) : H_kv * page * d;
  require(n <= INT32_MAX && page <= INT32_MAX, "the cache has too many pages");
  c.num_pages = static_cast<int32_t>(n);
  c.page_size = static_cast<int32_t>(page);
  if (k.scalar_type() == at::kBFloat16) {
    c.dtype = ATTN_CACHE_BF16;
    return c;
  }
  require(k.scalar_type() == at::kFloat8_e4m3fn || k.scalar_type() == at::kByte,
          "a cache is bf16, float8_e4m3fn or uint8 codes");
  c.dtype = ATTN_CACHE_E4M3;
  const at::Tensor ks = maybe(a[2], "cache.k_scale"), vs = maybe(a[3], "cache.v_scale");
  require(ks.defined() && vs.defined(), "an E4M3 cache needs k_scale and v_scale");
  const int64_t shape[3] = {n, H_kv, page};
  c.k_scale = static_cast<float*>(address(ks, at::kFloat, shape, dev, "k_scale"));
  c.v_scale = static_cast<float*>(address(vs, at::kFloat, shape, dev, "v_scale"));
  return c;
}

void argc(Py_ssize_t got, Py_ssize_t want) {
  TORCH_CHECK_TYPE(got == want, "expected ", want, " arguments, got ", got);
}

// (k, v, k_scale, v_scale, H_kv, d) -> (page_stride, num_pages, page_size, dtype)
PyObject* py_cache_layout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  argc(n, 6);
  const attn_kv_cache c = cache_struct(a, integer(a[4], "H_kv"), integer(a[5], "d"),
                                       tensor(a[0], "cache.k").device());
  return Py_BuildValue("(Liii)", static_cast<long long>(c.page_stride), c.num_pages, c.page_size,
                       c.dtype);
  END_HANDLE_TH_ERRORS
}

// (seq_lens, cu_new, T, block_table, free_pages, free_head, page_size)
PyObject* py_slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  argc(n, 7);
  const at::Tensor &lens = tensor(a[0], "seq_lens"), &cu = tensor(a[1], "cu_new");
  const at::Tensor &table = tensor(a[3], "block_table"), &free = tensor(a[4], "free_pages");
  const at::Tensor& head = tensor(a[5], "free_head");
  const int T = integer(a[2], "T"), page = integer(a[6], "page_size");
  const at::Device dev = lens.device();
  require(dev.is_cuda() && lens.dim() == 1 && table.dim() == 2 && free.dim() == 1,
          "seq_lens [B], block_table [B, max_pages] and free_pages [n] must be CUDA tensors");
  const int64_t B = lens.size(0), cols = table.size(1), spare = free.size(0);
  require(B <= INT32_MAX && cols <= INT32_MAX && spare <= INT32_MAX, "sizes must fit 32 bits");
  require(T >= 0, "T must not be negative");
  const auto* lp = static_cast<const int32_t*>(address(lens, at::kInt, {B}, dev, "seq_lens"));
  const auto* cp = static_cast<const int32_t*>(address(cu, at::kInt, {B + 1}, dev, "cu_new"));
  auto* tp = static_cast<int32_t*>(address(table, at::kInt, {B, cols}, dev, "block_table"));
  const auto* fp = static_cast<const int32_t*>(address(free, at::kInt, {spare}, dev, "free_pages"));
  const auto* hp = static_cast<const int32_t*>(address(head, at::kInt, {1}, dev, "free_head"));
  Launch on(dev);
  // Slots and positions are done with after the step, lengths and head are kept: together in one
  // allocation only where that holds a token's 12 bytes a request, not a prompt's.
  const int64_t t = T, kept = 4 * B + 4, at = t <= B ? 12 * t : 0;
  const at::Tensor step = make({12 * t + (t <= B ? kept : 0)}, at::kByte, dev);
  const at::Tensor state = t <= B ? step : make({kept}, at::kByte, dev);
  at::Tensor slots = carve(step, 0, {t}, at::kLong), pos = carve(step, 8 * t, {t}, at::kInt);
  at::Tensor lens_out = carve(state, at, {B}, at::kInt);
  at::Tensor head_out = carve(state, at + 4 * B, {1}, at::kInt);
  if (B == 0) head_out.copy_(head);
  check("attn_kv_slots",
        attn_kv_slots(lp, cp, tp, fp, hp, static_cast<int64_t*>(slots.data_ptr()),
                      static_cast<int32_t*>(pos.data_ptr()),
                      static_cast<int32_t*>(lens_out.data_ptr()),
                      static_cast<int32_t*>(head_out.data_ptr()), static_cast<int>(B), T,
                      static_cast<int>(cols), static_cast<int>(spare), page, on.stream));
  return pack({slots, pos, table, lens_out, head_out});
  END_HANDLE_TH_ERRORS
}

// What the step before attention and its backward take alike.
struct Rope {
  at::Device dev;
  int64_t B, N, d, ld;
  int H, H_kv, rot;
  bool packed;
  const void *wq, *wk;
  const double* inv_freq;
  const int32_t* positions;
  at::SmallVector<int64_t, 4> shape(int heads) const {
    at::SmallVector<int64_t, 4> s;
    if (!packed) s.push_back(B);
    s.push_back(heads);
    s.push_back(N);
    s.push_back(d);
    return s;
  }
};

Rope rope_inputs(const at::Tensor& qkv, int H, int H_kv, PyObject* positions, PyObject* inv_freq,
                 PyObject* wq, PyObject* wk) {
  require(qkv.scalar_type() == at::kBFloat16 && qkv.is_cuda() && (qkv.dim() == 2 || qkv.dim() == 3),
          "qkv must be a bf16 CUDA tensor [B, N, (H + 2 H_kv) d] or [T, (H + 2 H_kv) d]");
  const int64_t heads = static_cast<int64_t>(H) + 2 * static_cast<int64_t>(H_kv);
  const int64_t width = qkv.size(-1);
  require(H > 0 && H_kv > 0 && H % H_kv == 0 && width % heads == 0,
          "qkv's rows must hold H + 2 H_kv heads, H a multiple of H_kv");
  Rope r{qkv.device(), 1, qkv.size(-2), width / heads, width, H, H_kv, 0, qkv.dim() == 2,
         nullptr, nullptr, nullptr, nullptr};
  if (!r.packed) r.B = qkv.size(0);
  require(r.B <= INT32_MAX && r.N <= INT32_MAX && r.d <= INT32_MAX, "sizes must fit 32 bits");
  bool even = width <= 1 || qkv.stride(-1) == 1;
  if (r.N > 1) {
    r.ld = qkv.stride(-2);
    even &= r.B <= 1 || qkv.stride(0) == r.N * r.ld;
  } else if (r.B > 1) {
    r.ld = qkv.stride(0);
  }
  require(r.B * r.N == 0 || even, "qkv's rows must be contiguous and evenly spaced");
  const at::Tensor f = maybe(inv_freq, "inv_freq"), pos = maybe(positions, "positions");
  if (f.defined()) {
    require(f.dim() == 1 && f.size(0) <= 1024, "inv_freq must be one-dimensional");
    require(pos.defined(), "a rotation needs positions");
    r.rot = static_cast<int>(2 * f.size(0));
    r.inv_freq = static_cast<const double*>(address(f, at::kDouble, f.sizes(), r.dev, "inv_freq"));
    r.positions = static_cast<const int32_t*>(
        address(pos, at::kInt, qkv.sizes().slice(0, qkv.dim() - 1), r.dev, "positions"));
  }
  r.wq = address(maybe(wq, "wq"), at::kBFloat16, {r.d}, r.dev, "wq");
  r.wk = address(maybe(wk, "wk"), at::kBFloat16, {r.d}, r.dev, "wk");
  return r;
}

// (qkv, H, H_kv, positions, inv_freq, interleaved, wq, wk, eps, rope_scale, cache k, v, k_scale,
//  v_scale (or None), slots, with_kv)
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  argc(n, 16);
  const at::Tensor& qkv = tensor(a[0], "qkv");
  const Rope r = rope_inputs(qkv, integer(a[1], "H"), integer(a[2], "H_kv"), a[3], a[4], a[6], a[7]);
  const bool has_cache = a[10] != Py_None, with_kv = truth(a[15]);
  attn_kv_cache c{};
  const int64_t* sp = nullptr;
  if (has_cache) {
    require(a[14] != Py_None, "a cache needs slots");
    c = cache_struct(a + 10, r.H_kv, r.d, r.dev);
    const at::Tensor& slots = tensor(a[14], "slots");
    const int64_t flat[1] = {r.B * r.N};
    sp = static_cast<const int64_t*>(
        address(slots, at::kLong, slots.dim() == 1 ? at::IntArrayRef(flat)
                                                   : qkv.sizes().slice(0, qkv.dim() - 1),
                r.dev, "slots"));
  }
  Launch on(r.dev);
  at::Tensor q = make(r.shape(r.H), at::kBFloat16, r.dev), k, v;
  if (with_kv) {
    k = make(r.shape(r.H_kv), at::kBFloat16, r.dev);
    v = make(r.shape(r.H_kv), at::kBFloat16, r.dev);
  }
  check("attn_qkv_rope",
        attn_qkv_rope(qkv.data_ptr(), r.ld, r.wq, r.wk, real(a[8]), r.inv_freq, r.rot, truth(a[5]),
                      real(a[9]), r.positions, q.data_ptr(), with_kv ? k.data_ptr() : nullptr,
                      with_kv ? v.data_ptr() : nullptr, has_cache ? &c : nullptr, sp,
                      static_cast<int>(r.B), static_cast<int>(r.N), r.H, r.H_kv,
                      static_cast<int>(r.d), on.stream));
  return pack({q, k, v});
  END_HANDLE_TH_ERRORS
}

// (dq, dk, dv, qkv, positions, inv_freq, interleaved, wq, wk, eps, rope_scale, workspace)
PyObject* py_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  argc(n, 12);
  const at::Tensor &dq = tensor(a[0], "dq"), &dk = tensor(a[1], "dk"), &dv = tensor(a[2], "dv");
  const at::Tensor& qkv = tensor(a[3], "qkv");
  at::Tensor ws = workspace(a[11], qkv.device());
  require(dq.dim() >= 3 && dk.dim() >= 3, "dq and dk must be [B, heads, N, d] or [heads, T, d]");
  require(dq.size(-3) <= INT32_MAX && dk.size(-3) <= INT32_MAX, "sizes must fit 32 bits");
  const Rope r = rope_inputs(qkv, static_cast<int>(dq.size(-3)), static_cast<int>(dk.size(-3)), a[4],
                             a[5], a[7], a[8]);
  const void* qp = address(dq, at::kBFloat16, r.shape(r.H), r.dev, "dq");
  const void* kp = address(dk, at::kBFloat16, r.shape(r.H_kv), r.dev, "dk");
  const void* vp = address(dv, at::kBFloat16, r.shape(r.H_kv), r.dev, "dv");
  const int B = static_cast<int>(r.B), N = static_cast<int>(r.N), d = static_cast<int>(r.d);
  Launch on(r.dev);
  at::Tensor dqkv = make(qkv.sizes(), at::kBFloat16, r.dev);
  at::Tensor dw[2];
  if (r.wq || r.wk) {
    const size_t need = attn_qkv_rope_bwd_workspace_bytes(B, N, r.H, r.H_kv, d);
    if (!ws.defined() && need) ws = make({static_cast<int64_t>(need)}, at::kByte, r.dev);
    const at::Tensor both = r.B * r.N ? make({2 * r.d}, at::kFloat, r.dev)
                                      : at::zeros({2 * r.d}, at::TensorOptions().dtype(at::kFloat).device(r.dev));
    for (int i = 0; i < 2; ++i)
      if (i ? r.wk : r.wq) dw[i] = carve(both, 4 * i * r.d, {r.d}, at::kFloat);
  }
  auto ptr = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  check("attn_qkv_rope_bwd",
        attn_qkv_rope_bwd(qp, kp, vp, qkv.data_ptr(), r.ld, r.wq, r.wk, real(a[9]), r.inv_freq, r.rot,
                          truth(a[6]), real(a[10]), r.positions, dqkv.data_ptr(),
                          qkv.size(-1), static_cast<float*>(ptr(dw[0])),
                          static_cast<float*>(ptr(dw[1])), B, N, r.H, r.H_kv, d, ptr(ws),
                          ws.defined() ? ws.nbytes() : 0, on.stream));
  return pack({dqkv, dw[0], dw[1]});
  END_HANDLE_TH_ERRORS
}

// (q, cache k, v, k_scale, v_scale, block_table, seq_lens, scale or None, workspace, out, lse)
PyObject* py_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  argc(n, 11);
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "cache.k");
  const at::Tensor &table = tensor(a[5], "block_table"), &lens = tensor(a[6], "seq_lens");
  at::Tensor ws = workspace(a[8], q.device());
  require(q.scalar_type() == at::kBFloat16 && q.is_cuda() && q.is_contiguous() &&
              (q.dim() == 3 || (q.dim() == 4 && q.size(2) == 1)),
          "q must be a contiguous bf16 CUDA tensor [B, H, 1, d] or [B, H, d]");
  const at::Device dev = q.device();
  const int64_t B = q.size(0), H = q.size(1), d = q.size(-1);
  require(k.dim() == 4 && k.size(1) > 0 && H % k.size(1) == 0,
          "the number of K/V heads must divide the number of query heads");
  const int64_t H_kv = k.size(1);
  const attn_kv_cache c = cache_struct(a + 1, H_kv, d, dev);
  require(table.dim() == 2, "block_table must be [B, max_pages]");
  const int64_t cols = table.size(1);
  require(B <= INT32_MAX && H <= INT32_MAX && d <= INT32_MAX && cols <= INT32_MAX,
          "sizes must fit 32 bits");
  const auto* tp = static_cast<const int32_t*>(address(table, at::kInt, {B, cols}, dev, "block_table"));
  const auto* lp = static_cast<const int32_t*>(address(lens, at::kInt, {B}, dev, "seq_lens"));
  const at::IntArrayRef rows = q.sizes().slice(0, q.dim() - 1);
  at::Tensor out = maybe(a[9], "out"), lse = maybe(a[10], "lse");
  address(out, at::kBFloat16, q.sizes(), dev, "out");
  address(lse, at::kFloat, rows, dev, "lse");
  const float scale = a[7] == Py_None ? 1.f / std::sqrt(static_cast<float>(d)) : real(a[7]);
  const int Bi = static_cast<int>(B), Hi = static_cast<int>(H), Ki = static_cast<int>(H_kv);
  Launch on(dev);
  if (!ws.defined())
    ws = make({static_cast<int64_t>(attn_fwd_paged_workspace_bytes(Bi, Hi, Ki, static_cast<int>(d)))},
              at::kByte, dev);
  if (!out.defined()) out = make(q.sizes(), at::kBFloat16, dev);
  if (!lse.defined()) lse = make(rows, at::kFloat, dev);
  check("attn_fwd_paged",
        attn_fwd_paged(q.data_ptr(), &c, tp, lp, out.data_ptr(), static_cast<float*>(lse.data_ptr()),
                       Bi, Hi, Ki, static_cast<int>(d), static_cast<int>(cols), scale, ws.data_ptr(),
                       ws.nbytes(), on.stream));
  return pack({out, lse});
  END_HANDLE_TH_ERRORS
}

PyObject* py_set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

#define FAST(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST("cache_layout", py_cache_layout), FAST("kv_slots", py_slots),
                           FAST("qkv_rope", py_rope), FAST("qkv_rope_bwd", py_rope_bwd),
                           FAST("attn_fwd_paged", py_paged),
                           {"set_error", py_set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_attn_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_binding() { return PyModule_Create(&g_module); }
