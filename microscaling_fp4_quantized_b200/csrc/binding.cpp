// Python binding of the paged cache operators: argument checks, output allocation and the call of the C
// entry point, all natively. A step of a running batch takes 3 to 7 us on the GPU; checking its dozen
// arguments and filling the C structures through ctypes took 20 to 30 us of host time, this takes 5 (half of it
// the launch, 0.6 for each tensor that is allocated). The C functions are handed over by address
// (`bind`), so that the library in use is the one the package has loaded.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <optional>
#include <string>

#include "sage_fp4.h"

namespace {

using at::Tensor;

struct Entry {
  decltype(&sage_fp4_norm_rope) norm_rope;
  decltype(&sage_fp4_cache_append) append;
  decltype(&sage_fp4_cache_gather) gather;
  decltype(&sage_fp4_decode_workspace_bytes) workspace;
  decltype(&sage_fp4_attn_decode) decode;
  PyObject* check;  // Python: check(status, what), raises
} g = {};

struct Cache {
  sage_fp4_cache_t c;
  at::Device device = at::Device(at::kCPU);
  at::ScalarType dtype = at::kBFloat16;
};

const char* const kCapsule = "microscaling_fp4_quantized_b200.cache";

struct Refused : std::exception {  // a ValueError or TypeError with a message
  std::string text;
  PyObject* type;
  explicit Refused(std::string t, PyObject* ty = PyExc_ValueError) : text(std::move(t)), type(ty) {}
};
struct Raised : std::exception {};  // a Python error is already set

// (a macro: the message is put together only when it is needed)
#define REFUSE_IF(bad, text)        \
  do {                              \
    if (bad) throw Refused((text)); \
  } while (0)

const char* name_of(at::ScalarType t) {
  return t == at::kBFloat16 ? "torch.bfloat16" : "torch.float16";
}

std::string where(at::Device d) { return d.str(); }

const Tensor* tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor", PyExc_TypeError);
  return &THPVariable_Unpack(o);
}
const Tensor* tensor_or_none(PyObject* o, const char* name) { return o == Py_None ? nullptr : tensor(o, name); }

// A dimension of size 1 has no stride that could matter.
int64_t stride(const Tensor& t, int64_t d) { return t.size(d) != 1 ? t.stride(d) : 0; }

bool shape_is(const Tensor& t, at::IntArrayRef s) { return t.sizes() == s; }

std::string text_of(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

void check_rows(const char* name, const Tensor& t, int64_t dim, at::ScalarType dtype, at::Device dev) {
  REFUSE_IF(!t.is_cuda() || t.device() != dev, std::string(name) + " must be a CUDA tensor on " + where(dev));
  REFUSE_IF(t.dim() != dim, std::string(name) + " must have " + std::to_string(dim) + " dimensions");
  REFUSE_IF(t.scalar_type() != dtype, std::string(name) + " must be " + name_of(dtype));
  REFUSE_IF(t.size(dim - 1) != 1 && t.stride(dim - 1) != 1,
            std::string(name) + ": the channel (last) dimension must be contiguous");
}

void check_table(const char* name, const Tensor& t, at::IntArrayRef shape, at::Device dev) {
  REFUSE_IF(!t.is_cuda() || t.device() != dev || t.scalar_type() != at::kInt,
            std::string(name) + " must be an int32 CUDA tensor on " + where(dev));
  REFUSE_IF(!shape_is(t, shape) || !t.is_contiguous(),
            std::string(name) + " must be contiguous with shape " + text_of(shape));
}

sage_dtype_t code_of(at::ScalarType t) {
  if (t == at::kBFloat16) return SAGE_BF16;
  if (t == at::kHalf) return SAGE_F16;
  throw Refused("unsupported dtype; use bfloat16 or float16", PyExc_TypeError);
}

// Norm weights and rotation table; false: there are neither.
bool make_rope(sage_fp4_rope_t* r, int64_t D, at::ScalarType dtype, at::Device dev, const Tensor* qw, const Tensor* kw,
               double eps, const Tensor* rope, bool interleaved) {
  if (qw == nullptr && kw == nullptr && rope == nullptr) return false;
  std::memset(r, 0, sizeof(*r));
  const Tensor* w[2] = {qw, kw};
  const char* const names[2] = {"q_weight", "k_weight"};
  for (int i = 0; i < 2; ++i) {
    if (w[i] == nullptr) continue;
    REFUSE_IF(!w[i]->is_cuda() || w[i]->device() != dev || !shape_is(*w[i], {D}) || !w[i]->is_contiguous(),
              std::string(names[i]) + " must be a contiguous [" + std::to_string(D) + "] CUDA tensor on " + where(dev));
    const at::ScalarType t = w[i]->scalar_type();
    REFUSE_IF((t != dtype && t != at::kFloat) || (i == 1 && qw != nullptr && qw->scalar_type() != t),
              std::string("norm weights must both be ") + name_of(dtype) + " or both float32");
    r->weight_f32 = t == at::kFloat;
    (i == 0 ? r->q_weight : r->k_weight) = w[i]->data_ptr();
  }
  r->eps = static_cast<float>(eps);
  if (rope != nullptr) {
    REFUSE_IF(!rope->is_cuda() || rope->device() != dev || rope->scalar_type() != at::kFloat || rope->dim() != 2 ||
                  !rope->is_contiguous(),
              "rope must be a contiguous float32 CUDA tensor [positions, rotary_dim] on " + where(dev));
    REFUSE_IF(rope->size(0) > INT32_MAX || rope->size(1) > INT32_MAX, "rope is too large");
    // A table of no positions has no address; any aligned one says that there is a table.
    r->rope = rope->numel() > 0 ? static_cast<const float*>(rope->data_ptr()) : reinterpret_cast<const float*>(16);
    r->rope_len = static_cast<int>(rope->size(0));
    r->rotary_dim = static_cast<int>(rope->size(1));
  }
  r->interleaved = interleaved;
  return true;
}

int to_int(int64_t v, const char* what) {
  REFUSE_IF(v > INT32_MAX, std::string(what) + " is too large");
  return static_cast<int>(v);
}

// dims: of (sequence, head, token); -1: no such dimension.
sage_fp4_rows_t make_rows(const Tensor& x, const Tensor& y, const int (&dims)[3]) {
  sage_fp4_rows_t r;
  r.x = x.data_ptr();
  r.y = y.data_ptr();
  r.heads = to_int(x.size(dims[1]), "the number of heads");
  for (int i = 0; i < 3; ++i) {
    r.x_stride[i] = dims[i] >= 0 ? stride(x, dims[i]) : 0;
    r.y_stride[i] = dims[i] >= 0 ? stride(y, dims[i]) : 0;
  }
  return r;
}

const Cache& cache_of(PyObject* o) {
  void* p = PyCapsule_GetPointer(o, kCapsule);
  if (p == nullptr) throw Raised();
  return *static_cast<Cache*>(p);
}

sage_fp4_batch_t make_batch(const Cache& c, const Tensor& table, const Tensor& lens, const Tensor* cu) {
  REFUSE_IF(!table.is_cuda() || table.device() != c.device || table.scalar_type() != at::kInt,
            "page_table must be an int32 CUDA tensor on " + where(c.device));
  REFUSE_IF(table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1),
            "page_table must be [sequences, pages] with contiguous rows");
  const int64_t B = table.size(0);
  check_table("seq_lens", lens, {B}, c.device);
  if (cu != nullptr) check_table("cu_seqlens", *cu, {B + 1}, c.device);
  sage_fp4_batch_t b;
  b.B = to_int(B, "the number of sequences");
  b.page_table = static_cast<const int32_t*>(table.data_ptr());
  b.table_stride = stride(table, 0);
  b.table_width = to_int(table.size(1), "the page table");
  b.seq_lens = static_cast<const int32_t*>(lens.data_ptr());
  b.cu_seqlens = cu != nullptr ? static_cast<const int32_t*>(cu->data_ptr()) : nullptr;
  return b;
}

// total < 0: any number of rows.
void check_dense(const char* name, const Tensor& t, const Cache& c, int64_t total) {
  check_rows(name, t, 3, c.dtype, c.device);
  REFUSE_IF(t.size(1) != c.c.Hkv || t.size(2) != c.c.D || (total >= 0 && t.size(0) != total),
            std::string(name) + " must be [" + (total >= 0 ? std::to_string(total) : std::string("tokens")) + ", " +
                std::to_string(c.c.Hkv) + ", " + std::to_string(c.c.D) + "]");
}

// Other Python threads run meanwhile: an allocation may wait for the device and a launch for room in its
// queue, which may itself be waiting for a host function in Python.
class Unlocked {
  PyThreadState* s = PyEval_SaveThread();

 public:
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(s); }
};

Tensor empty_rows(at::IntArrayRef shape, at::ScalarType dtype, at::Device dev) {
  const Unlocked u;
  return Tensor(at::detail::empty_cuda(shape, dtype, dev, std::nullopt));
}

void* stream_of(at::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

template <typename F>
void run(const char* what, F call) {
  int status;
  {
    const Unlocked u;
    status = call();
  }
  if (status == SAGE_OK) return;
  PyObject* r = PyObject_CallFunction(g.check, "is", status, what);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, what);
  throw Raised();
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

// Runs f, turning its exceptions into Python's.
template <typename F>
PyObject* guarded(PyObject* const*, Py_ssize_t n, Py_ssize_t want, F f) {
  HANDLE_TH_ERRORS
  try {
    if (n != want) throw Refused("wrong number of arguments", PyExc_TypeError);
    REFUSE_IF(g.decode == nullptr, "the library is not bound");
    return f();
  } catch (const Refused& e) {
    PyErr_SetString(e.type, e.text.c_str());
    return nullptr;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* wrap_pair(const Tensor& a, const std::optional<Tensor>& b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = b.has_value() ? THPVariable_Wrap(*b) : Py_NewRef(Py_None);
  PyObject* t = x != nullptr && y != nullptr ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return t;
}

// (q, k, q_weight, k_weight, eps, rope, positions, interleaved, tensor_layout, q_out, k_out)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 11, [&]() -> PyObject* {
    const Tensor& q = *tensor(a[0], "q");
    const Tensor* k = tensor_or_none(a[1], "k");
    const Tensor *qw = tensor_or_none(a[2], "q_weight"), *kw = tensor_or_none(a[3], "k_weight");
    const double eps = number(a[4]);
    const Tensor *rope = tensor_or_none(a[5], "rope"), *pos = tensor_or_none(a[6], "positions");
    const bool inter = truth(a[7]);
    const char* layout = PyUnicode_AsUTF8(a[8]);
    if (layout == nullptr) throw Raised();
    const Tensor *qo = tensor_or_none(a[9], "q_out"), *ko = tensor_or_none(a[10], "k_out");
    int dims[3] = {-1, 1, 0};
    const bool hnd = std::strcmp(layout, "HND") == 0;
    if (q.dim() == 4 && (hnd || std::strcmp(layout, "NHD") == 0)) {
      dims[0] = 0;
      dims[1] = hnd ? 1 : 2;
      dims[2] = hnd ? 2 : 1;
    } else {
      REFUSE_IF(q.dim() != 3, "q must be [B, H, N, D] ('HND'), [B, N, H, D] ('NHD') or [tokens, H, D]");
      REFUSE_IF(rope != nullptr && pos == nullptr, "packed rows need positions");
    }
    const int64_t rank = q.dim(), D = q.size(rank - 1);
    const at::Device dev = q.device();
    const at::ScalarType dtype = q.scalar_type();
    const sage_dtype_t code = code_of(dtype);
    check_rows("q", q, rank, dtype, dev);
    const int64_t B = dims[0] >= 0 ? q.size(0) : 1, N = q.size(dims[2]);
    if (k != nullptr) {
      check_rows("k", *k, rank, dtype, dev);
      REFUSE_IF(k->size(rank - 1) != D || k->size(dims[2]) != N || (dims[0] >= 0 && k->size(0) != B),
                "q and k disagree on batch, tokens or head dimension");
    } else {
      REFUSE_IF(ko != nullptr || kw != nullptr, "k_out and k_weight need k");
    }
    if (pos != nullptr) {
      if (dims[0] >= 0) check_table("positions", *pos, {B, N}, dev);
      else check_table("positions", *pos, {N}, dev);
    }
    sage_fp4_rope_t r;
    const bool some = make_rope(&r, D, dtype, dev, qw, kw, eps, rope, inter);
    auto output = [&](const char* name, const Tensor& x, const Tensor* y) {
      if (y == nullptr) return empty_rows(x.sizes(), dtype, dev);
      check_rows(name, *y, rank, dtype, dev);
      REFUSE_IF(y->sizes() != x.sizes(), std::string(name) + " must have the shape of its input");
      return *y;
    };
    const c10::cuda::CUDAGuard guard(dev);
    const Tensor q_out = output("q_out", q, qo);
    std::optional<Tensor> k_out;
    if (k != nullptr) k_out = output("k_out", *k, ko);
    const sage_fp4_rows_t qr = make_rows(q, q_out, dims);
    sage_fp4_rows_t kr;
    if (k != nullptr) kr = make_rows(*k, *k_out, dims);
    const int b = to_int(B, "the batch"), t = to_int(N, "the number of tokens"), d = to_int(D, "the head dimension");
    run("sage_fp4_norm_rope", [&] {
      return g.norm_rope(&qr, k != nullptr ? &kr : nullptr, b, t, d, code, some ? &r : nullptr,
                         pos != nullptr ? static_cast<const int32_t*>(pos->data_ptr()) : nullptr, stream_of(dev));
    });
    return wrap_pair(q_out, k_out);
  });
}

// (cache, k, v, page_table, seq_lens, cu_seqlens, q, q_weight, k_weight, eps, rope, interleaved, q_out)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 13, [&]() -> PyObject* {
    const Cache& c = cache_of(a[0]);
    const Tensor &k = *tensor(a[1], "k"), &v = *tensor(a[2], "v");
    const Tensor &table = *tensor(a[3], "page_table"), &lens = *tensor(a[4], "seq_lens");
    const Tensor* cu = tensor_or_none(a[5], "cu_seqlens");
    const Tensor* q = tensor_or_none(a[6], "q");
    const Tensor *qw = tensor_or_none(a[7], "q_weight"), *kw = tensor_or_none(a[8], "k_weight");
    const double eps = number(a[9]);
    const Tensor* rope = tensor_or_none(a[10], "rope");
    const bool inter = truth(a[11]);
    const Tensor* qo = tensor_or_none(a[12], "q_out");
    const sage_fp4_batch_t b = make_batch(c, table, lens, cu);
    check_dense("k", k, c, -1);
    const int64_t total = k.size(0);
    check_dense("v", v, c, total);
    REFUSE_IF(cu == nullptr && total != b.B, "without cu_seqlens, k and v hold one token per sequence");
    sage_fp4_rope_t r;
    const bool some = make_rope(&r, c.c.D, c.dtype, c.device, qw, kw, eps, rope, inter);
    const c10::cuda::CUDAGuard guard(c.device);
    std::optional<Tensor> q_out;
    sage_fp4_rows_t rows;
    if (q != nullptr) {
      check_rows("q", *q, 3, c.dtype, c.device);
      REFUSE_IF(q->size(0) != total || q->size(2) != c.c.D,
                "q must be [" + std::to_string(total) + ", heads, " + std::to_string(c.c.D) + "]");
      if (qo == nullptr) {
        q_out = empty_rows(q->sizes(), c.dtype, c.device);
      } else {
        check_rows("q_out", *qo, 3, c.dtype, c.device);
        REFUSE_IF(qo->sizes() != q->sizes(), "q_out must have the shape of q");
        q_out = *qo;
      }
      rows = make_rows(*q, *q_out, {-1, 1, 0});
    } else {
      REFUSE_IF(qo != nullptr || qw != nullptr, "q_out and q_weight need q");
    }
    const int64_t ks[2] = {stride(k, 1), stride(k, 0)}, vs[2] = {stride(v, 1), stride(v, 0)};
    const int t = to_int(total, "the number of tokens");
    run("sage_fp4_cache_append", [&] {
      return g.append(&c.c, &b, k.data_ptr(), ks, v.data_ptr(), vs, t, some ? &r : nullptr,
                      q != nullptr ? &rows : nullptr, stream_of(c.device));
    });
    return q_out.has_value() ? THPVariable_Wrap(*q_out) : Py_NewRef(Py_None);
  });
}

// (cache, page_table, seq_lens, cu_seqlens, total, k_out, v_out)
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 7, [&]() -> PyObject* {
    const Cache& c = cache_of(a[0]);
    const Tensor &table = *tensor(a[1], "page_table"), &lens = *tensor(a[2], "seq_lens");
    const Tensor* cu = tensor_or_none(a[3], "cu_seqlens");
    const Tensor *ko = tensor_or_none(a[5], "k_out"), *vo = tensor_or_none(a[6], "v_out");
    const sage_fp4_batch_t b = make_batch(c, table, lens, cu);
    REFUSE_IF((ko == nullptr) != (vo == nullptr), "pass both of k_out and v_out, or neither");
    int64_t total;
    if (a[4] != Py_None) {
      total = PyLong_AsLongLong(a[4]);
      if (total == -1 && PyErr_Occurred()) throw Raised();
    } else {
      REFUSE_IF(ko == nullptr && cu != nullptr, "cu_seqlens needs total, the number of rows");
      total = ko != nullptr && ko->dim() > 0 ? ko->size(0) : b.B;
    }
    REFUSE_IF(total < 0 || (cu == nullptr && total != b.B), "without cu_seqlens there is one row per sequence");
    const c10::cuda::CUDAGuard guard(c.device);
    Tensor k, v;
    if (ko == nullptr) {
      k = empty_rows({total, c.c.Hkv, c.c.D}, c.dtype, c.device);
      v = empty_rows({total, c.c.Hkv, c.c.D}, c.dtype, c.device);
    } else {
      check_dense("k_out", *ko, c, total);
      check_dense("v_out", *vo, c, total);
      k = *ko;
      v = *vo;
    }
    const int64_t ks[2] = {stride(k, 1), stride(k, 0)}, vs[2] = {stride(v, 1), stride(v, 0)};
    const int t = to_int(total, "total");
    run("sage_fp4_cache_gather", [&] {
      return g.gather(&c.c, &b, k.data_ptr(), ks, v.data_ptr(), vs, t, stream_of(c.device));
    });
    return wrap_pair(k, v);
  });
}

// (cache, page_table, seq_lens, heads)
PyObject* workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 4, [&]() -> PyObject* {
    const Cache& c = cache_of(a[0]);
    const sage_fp4_batch_t b = make_batch(c, *tensor(a[1], "page_table"), *tensor(a[2], "seq_lens"), nullptr);
    const long heads = PyLong_AsLong(a[3]);
    if (heads == -1 && PyErr_Occurred()) throw Raised();
    return PyLong_FromSize_t(g.workspace(&c.c, &b, to_int(heads, "the number of heads")));
  });
}

// (cache, q, page_table, seq_lens, sm_scale, out, workspace)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 7, [&]() -> PyObject* {
    const Cache& c = cache_of(a[0]);
    const Tensor &q = *tensor(a[1], "q"), &table = *tensor(a[2], "page_table"), &lens = *tensor(a[3], "seq_lens");
    const double scale = a[4] == Py_None ? 0.0 : number(a[4]);
    const Tensor *out_ = tensor_or_none(a[5], "out"), *ws = tensor_or_none(a[6], "workspace");
    const sage_fp4_batch_t b = make_batch(c, table, lens, nullptr);
    const int64_t H = q.dim() == 3 ? q.size(1) : 0;
    for (const Tensor* t : {&q, out_}) {
      if (t == nullptr) continue;
      const char* name = t == &q ? "q" : "out";
      check_rows(name, *t, 3, c.dtype, c.device);
      REFUSE_IF(!shape_is(*t, {b.B, H, c.c.D}),
                std::string(name) + " must be [" + std::to_string(b.B) + ", heads, " + std::to_string(c.c.D) + "]");
    }
    REFUSE_IF(H % c.c.Hkv != 0, "the number of query heads must be a multiple of the cache's heads");
    const int heads = to_int(H, "the number of heads");
    const c10::cuda::CUDAGuard guard(c.device);
    const Tensor out = out_ != nullptr ? *out_ : empty_rows(q.sizes(), c.dtype, c.device);
    Tensor own;
    if (ws == nullptr) {
      const size_t need = g.workspace(&c.c, &b, heads);
      own = empty_rows({static_cast<int64_t>(need > 0 ? need : 256)}, at::kByte, c.device);
      ws = &own;
    } else {
      REFUSE_IF(!ws->is_cuda() || ws->device() != c.device || ws->scalar_type() != at::kByte || !ws->is_contiguous(),
                "workspace must be a contiguous uint8 CUDA tensor on " + where(c.device));
    }
    const int64_t qs[2] = {stride(q, 0), stride(q, 1)}, os[2] = {stride(out, 0), stride(out, 1)};
    run("sage_fp4_attn_decode", [&] {
      return g.decode(&c.c, &b, q.data_ptr(), qs, out.data_ptr(), os, heads, static_cast<float>(scale),
                      ws->data_ptr(), static_cast<size_t>(ws->numel()), stream_of(c.device));
    });
    return THPVariable_Wrap(out);
  });
}

void free_cache(PyObject* o) { delete static_cast<Cache*>(PyCapsule_GetPointer(o, kCapsule)); }

// (address of a sage_fp4_cache_t, device index) -> handle; the structure is copied.
PyObject* make_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2) return PyErr_Format(PyExc_TypeError, "wrong number of arguments");
  const void* p = PyLong_AsVoidPtr(a[0]);
  const long index = PyLong_AsLong(a[1]);
  if (PyErr_Occurred()) return nullptr;
  const auto* given = static_cast<const sage_fp4_cache_t*>(p);
  if (given->Hkv < 1 || given->page_size < 1) {  // the calls divide by both
    PyErr_SetString(PyExc_ValueError, "a cache needs at least one head and one slot per page");
    return nullptr;
  }
  auto* c = new Cache;
  c->c = *given;
  c->device = at::Device(at::kCUDA, static_cast<at::DeviceIndex>(index));
  c->dtype = c->c.dtype == SAGE_F16 ? at::kHalf : at::kBFloat16;
  PyObject* o = PyCapsule_New(c, kCapsule, free_cache);
  if (o == nullptr) delete c;
  return o;
}

// (addresses of the five entry points, check)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return PyErr_Format(PyExc_TypeError, "wrong number of arguments");
  void* p[5];
  for (int i = 0; i < 5; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  g.norm_rope = reinterpret_cast<decltype(g.norm_rope)>(p[0]);
  g.append = reinterpret_cast<decltype(g.append)>(p[1]);
  g.gather = reinterpret_cast<decltype(g.gather)>(p[2]);
  g.workspace = reinterpret_cast<decltype(g.workspace)>(p[3]);
  g.decode = reinterpret_cast<decltype(g.decode)>(p[4]);
  Py_XSETREF(g.check, Py_NewRef(a[5]));
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"bind", FAST(bind)},       {"make_cache", FAST(make_cache)}, {"norm_rope", FAST(norm_rope)},
                         {"append", FAST(append)},   {"gather", FAST(gather)},         {"workspace", FAST(workspace)},
                         {"decode", FAST(decode)},   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
