// binding.cpp -- the Python calls around the cache (norms and rotary positions, the
// store with them, rows read back, differential heads), as one CPython function
// each: the checks of the tensors, the outputs, the C structures and the call into
// libkvq.
//
// These calls run once per layer in a decode step whose kernels take 2 to 5 us.
// Marshalled through ctypes a store of one token and its read-back took 27 to 34 us of
// the host's time, most of it attribute reads of five tensors and three
// torch.empty calls; here the same steps are a few loads each.
//
// Nothing in here computes: a refused argument raises ValueError or TypeError
// before the library is called, and a status of the library's goes to the binding's
// own error class.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <sstream>
#include <string>

#include "../../include/kvq.h"

namespace {

// The library's entry points (resolved by the ctypes loader, so that there is one
// libkvq in the process) and the function that raises for a status.
decltype(&kvq_norm_rope) p_norm_rope;
decltype(&kvq_norm_rope_store) p_norm_rope_store;
decltype(&kvq_load) p_load;
decltype(&kvq_load_seqs) p_load_seqs;
decltype(&kvq_merge_diff) p_merge_diff;
decltype(&kvq_diff_heads) p_diff_heads;
decltype(&kvq_prefill_diff_workspace_size) p_prefill_diff_workspace_size;
decltype(&kvq_prefill_diff) p_prefill_diff;
PyObject* raise_status;

struct Refused {  // a Python error is set
};

template <typename... A>
[[noreturn]] void refuse(PyObject* type, const A&... parts) {
  std::ostringstream s;
  s << "kvq: ";
  (s << ... << parts);
  PyErr_SetString(type, s.str().c_str());
  throw Refused();
}

std::string shape_of(at::IntArrayRef s) {
  std::ostringstream o;
  o << "[";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << "]";
  return o.str();
}

bool given(PyObject* o) { return o != Py_None; }

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, what, " must be a tensor, not ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// The call's device: the current one, on which its first tensor has to be.
int device_of(const at::Tensor& t) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, "expected a CUDA tensor, got one on ", t.device());
  const int dev = c10::cuda::current_device();
  if (t.get_device() != dev)
    refuse(PyExc_ValueError, "a tensor is on ", t.device(), ", the current device is cuda:", dev);
  return dev;
}

void on_device(const at::Tensor& t, const char* what, int dev) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, "expected a CUDA tensor, got one on ", t.device());
  if (t.get_device() != dev)
    refuse(PyExc_ValueError, what, " is on ", t.device(), ", the current device is cuda:", dev);
}

void of_type(const at::Tensor& t, const char* what, at::ScalarType type) {
  if (t.scalar_type() != type) refuse(PyExc_TypeError, what, " must be ", type, ", got ", t.scalar_type());
}

int32_t code_of(at::ScalarType t, const char* what) {
  if (t == at::kFloat) return KVQ_DT_F32;
  if (t == at::kBFloat16) return KVQ_DT_BF16;
  refuse(PyExc_TypeError, what, " must be fp32 or bf16, got ", t);
}

at::ScalarType scalar_type(PyObject* o, at::ScalarType none) {
  if (!given(o)) return none;
  if (!THPDtype_Check(o)) refuse(PyExc_TypeError, "dtype must be a torch.dtype, not ", Py_TYPE(o)->tp_name);
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// Contiguous int32 metadata of a given shape.
const int32_t* ints(const at::Tensor& t, const char* what, int dev, at::IntArrayRef shape) {
  on_device(t, what, dev);
  of_type(t, what, at::kInt);
  if (t.sizes() != shape || !t.is_contiguous())
    refuse(PyExc_ValueError, what, " must be contiguous ", shape_of(shape), ", got ", shape_of(t.sizes()));
  return static_cast<const int32_t*>(t.data_ptr());
}

int32_t* status_of(PyObject* o, int dev) {
  if (!given(o)) return nullptr;
  const at::Tensor& t = tensor(o, "status");
  on_device(t, "status", dev);
  of_type(t, "status", at::kInt);
  if (t.numel() < 1) refuse(PyExc_ValueError, "status is empty");
  return static_cast<int32_t*>(t.data_ptr());
}

// kvq_rows of a tensor [tokens, heads, width] whose last dimension is contiguous.
kvq_rows rows(const at::Tensor& t, const char* what, int dev, int64_t tokens, int64_t heads, int64_t width) {
  if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != width)
    refuse(PyExc_ValueError, what, " must be [", tokens, ", ", heads, ", ", width, "], got ", shape_of(t.sizes()));
  if (t.stride(2) != 1) refuse(PyExc_ValueError, "the last dimension of ", what, " must be contiguous");
  on_device(t, what, dev);
  if (heads > INT32_MAX) refuse(PyExc_ValueError, what, " has ", heads, " heads");
  return kvq_rows{t.data_ptr(), code_of(t.scalar_type(), what), static_cast<int32_t>(heads), t.stride(0), t.stride(1)};
}

void three(const at::Tensor& t, const char* what) {
  if (t.dim() != 3) refuse(PyExc_ValueError, what, " must be [tokens, heads, width], got ", shape_of(t.sizes()));
}

// An output [n, heads, width]: the one given, or a new one.
at::Tensor fresh(int64_t n, int64_t heads, int64_t width, at::ScalarType type, int dev) {
  code_of(type, "an output");
  return at::detail::empty_cuda({n, heads, width}, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)),
                                std::nullopt);
}

long long integer(PyObject* o, const char* what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, what, " must be an integer");
  }
  return v;
}

int32_t integer32(PyObject* o, const char* what) {
  const long long v = integer(o, what);
  if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, what, " is out of range: ", v);
  return static_cast<int32_t>(v);
}

// A handle of the Python side: (address of its C structure, its axes, its device).
struct Handle {
  const void* at;
  long long n, dev;
};
Handle handle(PyObject* o, const char* what) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3) refuse(PyExc_TypeError, "bad ", what);
  return Handle{PyLong_AsVoidPtr(PyTuple_GET_ITEM(o, 0)), integer(PyTuple_GET_ITEM(o, 1), what),
                integer(PyTuple_GET_ITEM(o, 2), what)};
}

float real(PyObject* o, const char* what) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, what, " must be a number");
  }
  return static_cast<float>(v);
}

// A norm of the Python side, (weight, eps, offset): the weight's address is read in every
// call, since its storage may have been replaced since the last one.
struct Normed {
  kvq_norm norm{};
  bool is_given = false;
  const kvq_norm* get() const { return is_given ? &norm : nullptr; }
};
Normed norm_of(PyObject* o, const char* what, int dev, int64_t width) {
  Normed r;
  if (!given(o)) return r;
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3) refuse(PyExc_TypeError, "bad ", what);
  const at::Tensor& w = tensor(PyTuple_GET_ITEM(o, 0), "a norm's weight");
  if (w.numel() != width) refuse(PyExc_ValueError, what, " is for rows of ", w.numel(), ", not ", width);
  on_device(w, what, dev);
  if (!w.is_contiguous()) refuse(PyExc_ValueError, "the weight of ", what, " must be contiguous");
  r.norm = kvq_norm{w.data_ptr(), code_of(w.scalar_type(), what), real(PyTuple_GET_ITEM(o, 1), "eps"),
                    real(PyTuple_GET_ITEM(o, 2), "offset")};
  r.is_given = true;
  return r;
}

// The rope and its positions, int32 [n] (one axis) or [axes, n].
struct Turned {
  const kvq_rope* rope = nullptr;
  const int32_t* pos = nullptr;
  int64_t stride = 0;
};
Turned rope_of(PyObject* o, PyObject* positions, int dev, int64_t n) {
  Turned r;
  if (!given(o)) return r;
  const Handle h = handle(o, "rope");
  if (h.dev != dev) refuse(PyExc_ValueError, "the rope's table is on cuda:", h.dev, ", the current device is cuda:", dev);
  if (!given(positions)) refuse(PyExc_ValueError, "rotary positions need positions");
  const at::Tensor& p = tensor(positions, "positions");
  on_device(p, "positions", dev);
  of_type(p, "positions", at::kInt);
  const bool flat = p.dim() == 1 && h.n == 1 && p.size(0) == n;
  if (!flat && !(p.dim() == 2 && p.size(0) == h.n && p.size(1) == n))
    refuse(PyExc_ValueError, "positions must be [", h.n, ", ", n, "], got ", shape_of(p.sizes()));
  if (n > 1 && p.stride(-1) != 1) refuse(PyExc_ValueError, "positions of an axis must be contiguous");
  r.rope = static_cast<const kvq_rope*>(h.at);
  r.pos = static_cast<const int32_t*>(p.data_ptr());
  r.stride = h.n > 1 ? p.stride(0) : n;
  return r;
}

// A cache of the Python side, (address of its C structure, its planes' device).
const kvq_cache* cache_of(PyObject* o, int dev) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) refuse(PyExc_TypeError, "bad cache");
  const void* p = PyLong_AsVoidPtr(PyTuple_GET_ITEM(o, 0));
  if (!p) refuse(PyExc_TypeError, "bad cache");
  const long long d = integer(PyTuple_GET_ITEM(o, 1), "a cache's device");
  if (d != dev) refuse(PyExc_ValueError, "the cache is on cuda:", d, ", the current device is cuda:", dev);
  return static_cast<const kvq_cache*>(p);
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

// The library's answer: a status that is not KVQ_OK becomes the binding's error.
void checked(int32_t status, const char* where) {
  if (status == KVQ_OK) return;
  PyObject* r = PyObject_CallFunction(raise_status, "is", static_cast<int>(status), where);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, where);
  throw Refused();
}

PyObject* back(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// ---------------------------------------------------------------- the calls

// norm_rope(x, positions, rope, norm, out, dtype, status)
PyObject* norm_rope(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  three(x, "x");
  const int dev = device_of(x);
  const int64_t n = x.size(0), heads = x.size(1), width = x.size(2);
  const kvq_rows rx = rows(x, "x", dev, n, heads, width);
  at::Tensor y;
  if (given(a[4])) y = tensor(a[4], "out");
  else y = fresh(n, heads, width, scalar_type(a[5], x.scalar_type()), dev);
  const kvq_rows ry = rows(y, "out", dev, n, heads, width);
  const Turned r = rope_of(a[2], a[1], dev, n);
  checked(p_norm_rope(&rx, &ry, n, static_cast<int32_t>(width), norm_of(a[3], "norm", dev, width).get(), r.rope, r.pos,
                      r.stride, status_of(a[6], dev), stream_of(dev)),
          "kvq_norm_rope");
  return given(a[4]) ? back(a[4]) : THPVariable_Wrap(y);
}

// norm_rope_store(cache, q, k, v, slots, positions, rope, q_norm, k_norm, q_out, rotate, status)
PyObject* norm_rope_store(PyObject* const* a) {
  const at::Tensor& k = tensor(a[2], "k");
  three(k, "k");
  const int dev = device_of(k);
  const kvq_cache* c = cache_of(a[0], dev);
  const bool fp8 = c->format == KVQ_FMT_FP8_ROW;  // one tensor of latent and rope parts, no v
  const int64_t n = k.size(0), Hk = c->num_kv_heads, D = c->head_dim + (fp8 ? c->rope_dim : 0);
  const kvq_rows rk = rows(k, "k", dev, n, Hk, D);
  if (fp8 && given(a[3])) refuse(PyExc_ValueError, "fp8 latent rows take no v");
  kvq_rows rv;
  if (!fp8) rv = rows(tensor(a[3], "v"), "v", dev, n, Hk, D);
  kvq_rows rq, ro;
  at::Tensor out;
  const bool with_q = given(a[1]);
  if (with_q) {
    const at::Tensor& q = tensor(a[1], "q");
    three(q, "q");
    const int64_t Hq = q.size(1);
    rq = rows(q, "q", dev, n, Hq, D);
    out = given(a[9]) ? tensor(a[9], "q_out") : fresh(n, Hq, D, at::kFloat, dev);
    ro = rows(out, "q_out", dev, n, Hq, D);
  } else if (given(a[9])) {
    refuse(PyExc_ValueError, "q_out without q");
  }
  const Turned r = rope_of(a[6], a[5], dev, n);
  checked(p_norm_rope_store(c, with_q ? &rq : nullptr, &rk, fp8 ? nullptr : &rv, n,
                            norm_of(a[7], "q_norm", dev, c->head_dim).get(),
                            norm_of(a[8], "k_norm", dev, c->head_dim).get(), r.rope, r.pos, r.stride,
                            ints(tensor(a[4], "slot_mapping"), "slot_mapping", dev, {n}), with_q ? &ro : nullptr,
                            integer32(a[10], "rotate"), status_of(a[11], dev), stream_of(dev)),
          "kvq_norm_rope_store");
  return !with_q ? back(Py_None) : given(a[9]) ? back(a[9]) : THPVariable_Wrap(out);
}

// The outputs of a load: new ones where neither is given.
struct Loaded {
  at::Tensor k, v;
  kvq_rows rk, rv;
  bool with_k, with_v, made;
  Loaded(const kvq_cache* c, int64_t n, PyObject* ko, PyObject* vo, PyObject* dtype, int dev) {
    const bool fp8 = c->format == KVQ_FMT_FP8_ROW;
    const int64_t Hk = c->num_kv_heads, width = c->head_dim + (fp8 ? c->rope_dim : 0);
    if (n < 0) refuse(PyExc_ValueError, n, " tokens");
    made = !given(ko) && !given(vo);
    with_k = made || given(ko);
    with_v = made ? !fp8 : given(vo);
    const at::ScalarType type = made ? scalar_type(dtype, at::kBFloat16) : at::kBFloat16;
    if (with_k) {
      k = made ? fresh(n, Hk, width, type, dev) : tensor(ko, "k");
      rk = rows(k, "k", dev, n, Hk, width);
    }
    if (with_v) {
      v = made ? fresh(n, Hk, width, type, dev) : tensor(vo, "v");
      rv = rows(v, "v", dev, n, Hk, width);
    }
  }
  PyObject* result(PyObject* ko, PyObject* vo) const {
    PyObject* t = PyTuple_New(2);
    if (!t) throw Refused();
    PyTuple_SET_ITEM(t, 0, made ? THPVariable_Wrap(k) : back(ko));
    PyTuple_SET_ITEM(t, 1, made && with_v ? THPVariable_Wrap(v) : back(made ? Py_None : vo));
    return t;
  }
};

int32_t rotates(const kvq_cache* c, PyObject* o) {
  if (!given(o)) return c->format == KVQ_FMT_Q4_HAD32 || c->format == KVQ_FMT_TQ4 ? 1 : 0;
  return integer32(o, "rotate_back");
}

// load(cache, slots, k, v, dtype, rotate_back, status)
PyObject* load(PyObject* const* a) {
  const at::Tensor& slots = tensor(a[1], "slots");
  const int dev = device_of(slots);
  const kvq_cache* c = cache_of(a[0], dev);
  if (slots.dim() != 1) refuse(PyExc_ValueError, "slots must be [tokens], got ", shape_of(slots.sizes()));
  const int64_t n = slots.size(0);
  const int32_t* at = ints(slots, "slots", dev, {n});
  const Loaded o(c, n, a[2], a[3], a[4], dev);
  checked(p_load(c, at, n, rotates(c, a[5]), o.with_k ? &o.rk : nullptr, o.with_v ? &o.rv : nullptr,
                 status_of(a[6], dev), stream_of(dev)),
          "kvq_load");
  return o.result(a[2], a[3]);
}

// load_seqs(cache, block_tables, cu_lens, n_tok, starts, k, v, dtype, rotate_back, status)
PyObject* load_seqs(PyObject* const* a) {
  const at::Tensor &bt = tensor(a[1], "block_tables"), &cu = tensor(a[2], "cu_lens");
  const int dev = device_of(cu);
  const kvq_cache* c = cache_of(a[0], dev);
  if (cu.dim() != 1 || cu.size(0) < 1)
    refuse(PyExc_ValueError, "cu_lens must be [sequences + 1], got ", shape_of(cu.sizes()));
  if (bt.dim() != 2) refuse(PyExc_ValueError, "block_tables must be [sequences, pages], got ", shape_of(bt.sizes()));
  const int64_t B = cu.size(0) - 1, pages = bt.size(1), n = integer(a[3], "n_tok");
  if (B > INT32_MAX || pages > INT32_MAX) refuse(PyExc_ValueError, "block_tables is too large");
  const int32_t* tables = ints(bt, "block_tables", dev, {B, pages});
  const int32_t* starts = given(a[4]) ? ints(tensor(a[4], "starts"), "starts", dev, {B}) : nullptr;
  const int32_t* lens = ints(cu, "cu_lens", dev, {B + 1});
  const Loaded o(c, n, a[5], a[6], a[7], dev);
  checked(p_load_seqs(c, tables, static_cast<int32_t>(pages), static_cast<int32_t>(B), starts, lens, n,
                      rotates(c, a[8]), o.with_k ? &o.rk : nullptr, o.with_v ? &o.rv : nullptr, status_of(a[9], dev),
                      stream_of(dev)),
          "kvq_load_seqs");
  return o.result(a[5], a[6]);
}

// lambda: fp32 [heads] (one set) or [rows, heads]; its address and row stride.
const float* lambda_of(PyObject* o, int dev, int64_t n, int64_t heads, int64_t& stride) {
  const at::Tensor& t = tensor(o, "lam");
  on_device(t, "lam", dev);
  of_type(t, "lam", at::kFloat);
  const bool one = t.dim() == 1 && t.size(0) == heads;
  if ((!one && !(t.dim() == 2 && t.size(0) == n && t.size(1) == heads)) || (heads > 1 && t.stride(-1) != 1))
    refuse(PyExc_ValueError, "lam must be [", heads, "] or [", n, ", ", heads, "] with contiguous rows, got ",
           shape_of(t.sizes()));
  stride = one ? 0 : t.stride(0);
  return static_cast<const float*>(t.data_ptr());
}

at::Tensor diff_out(PyObject* o, PyObject* dtype, int dev, int64_t n, int64_t heads, int64_t width) {
  if (!given(o)) return fresh(n, heads, width, scalar_type(dtype, at::kFloat), dev);
  const at::Tensor& t = tensor(o, "out");
  on_device(t, "out", dev);
  if (t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) != width || !t.is_contiguous())
    refuse(PyExc_ValueError, "out must be contiguous [", n, ", ", heads, ", ", width, "], got ", shape_of(t.sizes()));
  return t;
}

// merge_diff(cache, workspace, num_seqs, num_q_heads, seq_lens, max_seq_len, lam, norm, out_scale, out, dtype, n_sel,
//            rotate_back)
PyObject* merge_diff(PyObject* const* a) {
  const at::Tensor &ws = tensor(a[1], "workspace"), &lens = tensor(a[4], "seq_lens");
  const int dev = device_of(lens);
  const kvq_cache* c = cache_of(a[0], dev);
  on_device(ws, "workspace", dev);
  if (!ws.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
  const int32_t B = integer32(a[2], "num_seqs"), Hq = integer32(a[3], "num_q_heads");
  if (B < 0 || Hq < 0) refuse(PyExc_ValueError, "num_seqs ", B, ", num_q_heads ", Hq);
  const at::Tensor out = diff_out(a[9], a[10], dev, B, Hq / 2, c->head_dim);
  int64_t stride;
  const float* lam = lambda_of(a[6], dev, B, Hq / 2, stride);
  checked(p_merge_diff(c, ws.data_ptr(), static_cast<size_t>(ws.numel()) * ws.element_size(), B, Hq,
                       ints(lens, "seq_lens", dev, {B}), integer32(a[5], "max_seq_len"), integer32(a[11], "n_sel"),
                       rotates(c, a[12]), lam, stride, norm_of(a[7], "norm", dev, c->head_dim).get(),
                       real(a[8], "out_scale"), out.data_ptr(), code_of(out.scalar_type(), "out"), stream_of(dev)),
          "kvq_merge_diff");
  return given(a[9]) ? back(a[9]) : THPVariable_Wrap(out);
}

// diff_heads(x, lam, norm, out_scale, out, dtype)
PyObject* diff_heads(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  three(x, "x");
  const int dev = device_of(x);
  of_type(x, "x", at::kFloat);
  if (!x.is_contiguous()) refuse(PyExc_ValueError, "x must be contiguous");
  const int64_t n = x.size(0), Hq = x.size(1), width = x.size(2);
  if (Hq > INT32_MAX || width > INT32_MAX) refuse(PyExc_ValueError, "x is too large");
  const at::Tensor out = diff_out(a[4], a[5], dev, n, Hq / 2, width);
  int64_t stride;
  const float* lam = lambda_of(a[1], dev, n, Hq / 2, stride);
  checked(p_diff_heads(static_cast<const float*>(x.data_ptr()), n, static_cast<int32_t>(Hq),
                       static_cast<int32_t>(width), lam, stride, norm_of(a[2], "norm", dev, width).get(),
                       real(a[3], "out_scale"), out.data_ptr(), code_of(out.scalar_type(), "out"), stream_of(dev)),
          "kvq_diff_heads");
  return given(a[4]) ? back(a[4]) : THPVariable_Wrap(out);
}

// prefill_diff(cache, q, q_start, block_table, sm_scale, lam, norm, out_scale, out, dtype, workspace, status)
PyObject* prefill_diff(PyObject* const* a) {
  const at::Tensor &q = tensor(a[1], "q"), &bt = tensor(a[3], "block_table");
  three(q, "q");
  const int dev = device_of(q);
  const kvq_cache* c = cache_of(a[0], dev);
  const int32_t qt = code_of(q.scalar_type(), "q");
  if (!q.is_contiguous()) refuse(PyExc_ValueError, "q must be contiguous");
  const int64_t n = q.size(0), Hq = q.size(1);
  if (q.size(2) != c->head_dim || n > INT32_MAX || Hq > INT32_MAX)
    refuse(PyExc_ValueError, "q must be [rows, heads, ", c->head_dim, "], got ", shape_of(q.sizes()));
  on_device(bt, "block_table", dev);
  of_type(bt, "block_table", at::kInt);
  if (!bt.is_contiguous() || bt.numel() > INT32_MAX) refuse(PyExc_ValueError, "block_table must be contiguous");
  const int32_t q_start = integer32(a[2], "q_start");
  const at::Tensor out = diff_out(a[8], a[9], dev, n, Hq / 2, c->head_dim);
  int64_t stride;
  const float* lam = lambda_of(a[5], dev, n, Hq / 2, stride);
  at::Tensor ws;
  if (given(a[10])) {
    ws = tensor(a[10], "workspace");
    on_device(ws, "workspace", dev);
    if (!ws.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
  } else {
    const size_t bytes = p_prefill_diff_workspace_size(c, static_cast<int32_t>(n), static_cast<int32_t>(Hq), q_start);
    ws = at::detail::empty_cuda({static_cast<int64_t>(bytes)}, at::kByte,
                                at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
  }
  checked(p_prefill_diff(c, q.data_ptr(), qt, static_cast<int32_t>(n), static_cast<int32_t>(Hq), q_start,
                         static_cast<const int32_t*>(bt.data_ptr()), static_cast<int32_t>(bt.numel()),
                         real(a[4], "sm_scale"), lam, stride, norm_of(a[6], "norm", dev, c->head_dim).get(),
                         real(a[7], "out_scale"), ws.data_ptr(), static_cast<size_t>(ws.numel()) * ws.element_size(),
                         out.data_ptr(), code_of(out.scalar_type(), "out"), status_of(a[11], dev), stream_of(dev)),
          "kvq_prefill_diff");
  return given(a[8]) ? back(a[8]) : THPVariable_Wrap(out);
}

// init(addresses of the entry points, raise_status)
PyObject* init(PyObject* const* a) {
  void** slots[] = {reinterpret_cast<void**>(&p_norm_rope), reinterpret_cast<void**>(&p_norm_rope_store),
                    reinterpret_cast<void**>(&p_load),      reinterpret_cast<void**>(&p_load_seqs),
                    reinterpret_cast<void**>(&p_merge_diff), reinterpret_cast<void**>(&p_diff_heads),
                    reinterpret_cast<void**>(&p_prefill_diff_workspace_size),
                    reinterpret_cast<void**>(&p_prefill_diff)};
  constexpr int kEntries = sizeof(slots) / sizeof(slots[0]);
  if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != kEntries) refuse(PyExc_TypeError, "bad entry points");
  for (int i = 0; i < kEntries; ++i) *slots[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[0], i));
  Py_INCREF(a[1]);
  Py_XDECREF(raise_status);
  raise_status = a[1];
  return back(Py_None);
}

// A function of N positional arguments; every C++ exception becomes a Python one, torch's
// their own (a failed allocation: torch.OutOfMemoryError).
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "kvq: %d arguments, got %d", N, static_cast<int>(n));
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused&) {
  } catch (const std::exception&) {
    torch::translate_exception_to_python(std::current_exception());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "kvq: unknown error");
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&call<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<init, 2>("init"),
                         method<norm_rope, 7>("norm_rope"),
                         method<norm_rope_store, 12>("norm_rope_store"),
                         method<load, 7>("load"),
                         method<load_seqs, 10>("load_seqs"),
                         method<merge_diff, 13>("merge_diff"),
                         method<diff_heads, 6>("diff_heads"),
                         method<prefill_diff, 12>("prefill_diff"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvq_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvq_calls() { return PyModule_Create(&module); }
