// bind.cpp -- the serving calls' argument marshalling, as a Python extension: tensor
// checks, output allocation and the call of the C ABI (include/rfb_attn.h), whose
// functions it gets as addresses from the library that the ctypes binding loaded.
//
// A decode step makes these calls thousands of times a second, and its kernels
// take a few microseconds: marshalling in the interpreter cost more than the
// kernels (rotary_fwd 12.8 us a call, attn_fwd_cache 16 us, of which the C entries
// with their launches take 2.2 and 4.5 us).  Nothing is computed here.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <sstream>
#include <string>

#include "rfb_attn.h"

namespace {

struct Api {
  decltype(&rfb_rotary) rotary = nullptr;
  decltype(&rfb_cache_append) append = nullptr;
  decltype(&rfb_attn_fwd_cache_workspace_size) workspace = nullptr;
  decltype(&rfb_attn_fwd_cache_counts) attn = nullptr;
  decltype(&rfb_cache_evict) evict = nullptr;
  decltype(&rfb_strerror) strerror = nullptr;
  decltype(&rfb_last_cuda_error) cuda_error = nullptr;
} api;

// An exception with the Python type it becomes.
struct Refusal {
  PyObject* type;
  std::string text;
};
template <typename... A>
[[noreturn]] void refuse(PyObject* type, const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw Refusal{type, s.str()};
}

std::string shape_text(at::IntArrayRef s) {
  std::string o = "(";
  for (size_t i = 0; i < s.size(); ++i) o += (i ? ", " : "") + std::to_string(s[i]);
  return o + (s.size() == 1 ? ",)" : ")");
}

std::string device_text(at::Device d) {
  return d.is_cuda() ? "cuda:" + std::to_string(d.index()) : "another device";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

void require(const char* name, const at::Tensor& t, at::ScalarType dtype, at::IntArrayRef shape,
             at::Device device, bool contiguous = true) {
  if (t.scalar_type() == dtype && t.device() == device && t.sizes() == shape &&
      (!contiguous || t.is_contiguous()))
    return;
  if (t.scalar_type() != dtype) {
    const char* want = dtype == at::kBFloat16 ? "bfloat16" : dtype == at::kFloat  ? "float32"
                       : dtype == at::kDouble ? "float64"  : dtype == at::kInt    ? "int32"
                       : dtype == at::kHalf   ? "float16"  : "of another type";
    refuse(PyExc_TypeError, name, " must be torch.", want, ", got ", c10::toString(t.scalar_type()));
  }
  if (t.device() != device) refuse(PyExc_ValueError, name, " must live on ", device_text(device));
  if (t.sizes() != shape)
    refuse(PyExc_ValueError, name, " has shape ", shape_text(t.sizes()), ", expected ", shape_text(shape));
  refuse(PyExc_ValueError, name, " must be contiguous");
}

// Whether the memory of two tensors meets: the stretches from their first to their last element.
bool meet(const at::Tensor& x, const at::Tensor& y) {
  if (x.numel() == 0 || y.numel() == 0) return false;
  const auto end = [](const at::Tensor& t) {
    int64_t last = 0;
    for (int64_t i = 0; i < t.dim(); ++i) last += (t.size(i) - 1) * t.stride(i);
    return static_cast<const char*>(t.const_data_ptr()) + (last + 1) * t.element_size();
  };
  return static_cast<const char*>(x.const_data_ptr()) < end(y) &&
         static_cast<const char*>(y.const_data_ptr()) < end(x);
}
void apart(const char* name, const at::Tensor& x, const char* other, const at::Tensor& y) {
  if (meet(x, y)) refuse(PyExc_ValueError, name, " must not share memory with ", other);
}
// The memory of a contiguous tensor.
struct Span {
  const char* name = "";
  const char *lo = nullptr, *hi = nullptr;
  Span() = default;
  Span(const char* n, const at::Tensor& t)
      : name(n), lo(t.defined() ? static_cast<const char*>(t.const_data_ptr()) : nullptr),
        hi(t.defined() ? lo + t.numel() * t.element_size() : nullptr) {}
  bool meets(const Span& o) const { return lo < hi && o.lo < o.hi && lo < o.hi && o.lo < hi; }
  void apart(const Span& o) const {
    if (meets(o)) refuse(PyExc_ValueError, name, " must not share memory with ", o.name);
  }
  // In place or apart.
  void same_or_apart(const Span& o) const {
    if (lo != o.lo) apart(o);
  }
};

void check(int rc, const char* what) {
  if (rc == RFB_OK) return;
  std::string s = std::string(what) + " failed: " + api.strerror(rc) + " (status " + std::to_string(rc);
  if (rc == RFB_ERR_CUDA) {
    int site = 0;
    const int code = api.cuda_error(&site);
    s += "; CUDA error " + std::to_string(code) + " at site " + std::to_string(site);
  }
  throw Refusal{PyExc_RuntimeError, s + ")"};
}

// Calls into the library without the interpreter lock (a launch waits where the
// stream's queue is full).
template <typename F, typename... A>
int call(F f, A... a) {
  PyThreadState* s = PyEval_SaveThread();
  const int rc = f(a...);
  PyEval_RestoreThread(s);
  return rc;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int small(int64_t v, const char* name) {
  if (v < 0 || v > 0x7fffffffLL) refuse(PyExc_ValueError, name, " = ", v, " is out of range");
  return static_cast<int>(v);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

// A contiguous tensor from torch's caching allocator: at::empty's own back end, without the
// dispatcher's 0.3 us a tensor (rotary_fwd 5.9 -> 5.6 us a call, attn_fwd_cache 8.4 -> 7.9).
at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, at::Device device) {
  return at::detail::empty_cuda(sizes, type, device, std::nullopt);
}

// The current stream of a device, which is made current for the call.
struct Launch {
  c10::cuda::CUDAGuard guard;
  void* stream;
  explicit Launch(at::Device d)
      : guard(d), stream(c10::cuda::getCurrentCUDAStream(d.index()).stream()) {}
};

PyObject* pair(const at::Tensor& a, PyObject* b) {
  PyObject* x = THPVariable_Wrap(a);
  if (!x || !b) {
    Py_XDECREF(x);
    Py_XDECREF(b);
    return nullptr;
  }
  PyObject* r = PyTuple_Pack(2, x, b);
  Py_DECREF(x);
  Py_DECREF(b);
  return r;
}

// ------------------------------------------------------------------- calls
// rotary(q, k, positions, freqs, layout, amplitude, inverse, q_out, k_out)
PyObject* rotary(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  if (!q.is_cuda()) refuse(PyExc_ValueError, "q must live on a CUDA device");
  const at::Device dev = q.device();
  const at::ScalarType dt = q.scalar_type();
  const int dtype = dt == at::kBFloat16 ? 0 : dt == at::kHalf ? 1 : dt == at::kFloat ? 2 : -1;
  if (dtype < 0)
    refuse(PyExc_TypeError, "q must be bfloat16, float16 or float32, got ", c10::toString(dt));
  if (q.dim() != 4) refuse(PyExc_ValueError, "q must be [B, H, N, d]");
  const int64_t B = q.size(0), H = q.size(1), N = q.size(2), d = q.size(3);
  const bool has_k = a[1] != Py_None;
  long long strides[6] = {q.stride(0), q.stride(1), q.stride(2), 0, 0, 0};
  int64_t Hk = 0;
  at::Tensor k;
  if (d > 1 && q.stride(3) != 1) refuse(PyExc_ValueError, "q must have contiguous channels");
  if (has_k) {
    k = tensor(a[1], "k");
    if (k.dim() != 4) refuse(PyExc_ValueError, "k must be [B, H, N, d]");
    Hk = k.size(1);
    require("k", k, dt, {B, Hk, N, d}, dev, false);
    if (d > 1 && k.stride(3) != 1) refuse(PyExc_ValueError, "k must have contiguous channels");
    strides[3] = k.stride(0), strides[4] = k.stride(1), strides[5] = k.stride(2);
  }
  const at::Tensor& freqs = tensor(a[3], "freqs");
  if (freqs.dim() != 1) refuse(PyExc_ValueError, "freqs must be [rot / 2]");
  const int64_t pairs = freqs.size(0);
  require("freqs", freqs, at::kDouble, {pairs}, dev);
  if (2 * pairs > d)
    refuse(PyExc_ValueError, "freqs has ", pairs, " pairs, more than half of d = ", d);
  const at::Tensor& pos = tensor(a[2], "positions");
  if (pos.dim() != 1 && pos.dim() != 2)
    refuse(PyExc_ValueError, "positions must be [N] or [B, N]");
  if (pos.dim() == 2)
    require("positions", pos, at::kInt, {B, N}, dev);
  else
    require("positions", pos, at::kInt, {N}, dev);
  Launch on(dev);
  at::Tensor qo, ko;
  if (a[7] == Py_None) {
    qo = make(q.sizes(), dt, dev);
  } else {
    qo = tensor(a[7], "q_out");
    require("q_out", qo, dt, q.sizes(), dev);
    apart("q_out", qo, "q", q);
    if (has_k) apart("q_out", qo, "k", k);
    apart("q_out", qo, "positions", pos);
    apart("q_out", qo, "freqs", freqs);
  }
  if (has_k) {
    if (a[8] == Py_None) {
      ko = make(k.sizes(), dt, dev);
    } else {
      ko = tensor(a[8], "k_out");
      require("k_out", ko, dt, k.sizes(), dev);
      apart("k_out", ko, "q", q);
      apart("k_out", ko, "k", k);
      apart("k_out", ko, "q_out", qo);
      apart("k_out", ko, "positions", pos);
      apart("k_out", ko, "freqs", freqs);
    }
  }
  check(call(api.rotary, q.const_data_ptr(), has_k ? k.const_data_ptr() : nullptr, qo.data_ptr(),
             has_k ? ko.data_ptr() : nullptr, static_cast<const int*>(pos.const_data_ptr()),
             static_cast<const double*>(freqs.const_data_ptr()), small(B, "B"), small(H, "H"),
             small(Hk, "Hk"), small(N, "N"), small(d, "d"), small(2 * pairs, "rot"), strides,
             strides + 3, static_cast<long long>(pos.dim() == 2 ? N : 0),
             static_cast<int>(integer(a[4])), dtype, static_cast<float>(number(a[5])),
             static_cast<int>(integer(a[6])), on.stream),
        "rfb_rotary");
  if (!has_k) Py_INCREF(Py_None);
  return pair(qo, has_k ? THPVariable_Wrap(ko) : Py_None);
}

constexpr const char* kPart[6] = {"the cache's k",       "the cache's v",       "the cache's w",
                                  "the cache's k_scale", "the cache's v_scale", "the cache's w_scale"};
// A cache's tensors, kept alive, with their sizes.
struct Cache {
  at::Tensor t[6];  // k, v, w, their scales; w and its scale may be undefined
  int64_t B, Hk, cap, d, r;
  at::Device on{at::kCPU};
  Span span[6];        // where they lay when the cache was made
  bool meets = false;  // one in another's memory
  // For the calls that write the tensors: none may lie in another's memory or in the mass's.
  void own_memory(const Span& mass) const {
    for (int i = 0; meets && i < 6; ++i)
      for (int k = 0; k < i; ++k) span[i].apart(span[k]);
    for (const Span& x : span) mass.apart(x);
  }
  // What a tensor was at the start it may no longer be (resize_, set_, .data, a freed storage).
  bool as_made(int i) const {
    const at::Tensor& x = t[i];
    if (!x.defined()) return true;
    const int64_t c = i < 2 ? d : r;
    return x.const_data_ptr() == span[i].lo && x.is_contiguous() &&
           (i < 3 ? x.sizes() == at::IntArrayRef({B, Hk, cap, c})
                  : x.sizes() == at::IntArrayRef({B, Hk, cap / 32}));
  }
  void* ptr(int i) const { return t[i].defined() ? t[i].data_ptr() : nullptr; }
  float* scale(int i) const { return static_cast<float*>(ptr(3 + i)); }
  at::Device device() const { return on; }
};
constexpr const char* kCacheName = "rank_biased_window_b200.Cache8";

Cache& cache_of(PyObject* o) {
  void* p = PyCapsule_GetPointer(o, kCacheName);
  if (!p) throw python_error();
  Cache& c = *static_cast<Cache*>(p);
  for (int i = 0; i < 6; ++i)
    if (!c.as_made(i))
      refuse(PyExc_ValueError, kPart[i],
             " is not what it was when the cache was made (size, layout or memory)");
  return c;
}

// cache(k, v, w, k_scale, v_scale, w_scale): checked by the caller.
PyObject* cache(PyObject* const* a) {
  auto* c = new Cache;
  for (int i = 0; i < 6; ++i)
    if (a[i] != Py_None) c->t[i] = THPVariable_Unpack(a[i]);
  c->B = c->t[0].size(0), c->Hk = c->t[0].size(1), c->cap = c->t[0].size(2), c->d = c->t[0].size(3);
  c->r = c->t[2].defined() ? c->t[2].size(3) : 0;
  c->on = c->t[0].device();
  for (int i = 0; i < 6; ++i) {
    c->span[i] = Span(kPart[i], c->t[i]);
    for (int k = 0; k < i; ++k) c->meets |= c->span[i].meets(c->span[k]);
  }
  return PyCapsule_New(c, kCacheName, [](PyObject* o) {
    delete static_cast<Cache*>(PyCapsule_GetPointer(o, kCacheName));
  });
}

const at::Tensor& mass_of(PyObject* o, const Cache& c) {
  const at::Tensor& t = tensor(o, "mass");
  require("mass", t, at::kFloat, {c.B, c.Hk, c.cap}, c.device());
  return t;
}
float* floats(const at::Tensor& t) { return static_cast<float*>(t.data_ptr()); }

// append(cache, mass, k, v, w, start, counts)
PyObject* append(PyObject* const* a) {
  const Cache& c = cache_of(a[0]);
  const at::Device dev = c.device();
  at::Tensor x[3];
  const char* names[3] = {"k", "v", "w"};
  if (c.r == 0 && a[4] != Py_None)
    refuse(PyExc_ValueError, "w given, but the cache holds no factors (r = 0)");
  const int tensors = c.r ? 3 : 2;
  long long strides[9] = {};
  int64_t n = 0;
  for (int i = 0; i < tensors; ++i) {
    x[i] = tensor(a[2 + i], names[i]);
    if (x[i].dim() != 4) refuse(PyExc_ValueError, names[i], " must be [B, Hk, n, channels]");
    if (i == 0) n = x[0].size(2);
    require(names[i], x[i], at::kBFloat16, {c.B, c.Hk, n, i < 2 ? c.d : c.r}, dev, false);
    for (int k = 0; k < 3; ++k) strides[3 * i + k] = x[i].stride(k);
    if (n > 0 && (x[i].stride(3) != 1 || ((x[i].stride(0) | x[i].stride(1) | x[i].stride(2)) & 7)))
      refuse(PyExc_ValueError, names[i],
             " must have contiguous channels and strides of multiples of 8");
  }
  const at::Tensor& start = tensor(a[5], "start");
  require("start", start, at::kInt, {c.B}, dev);
  const int* counts = nullptr;
  if (a[6] != Py_None) {
    const at::Tensor& t = tensor(a[6], "counts");
    require("counts", t, at::kInt, {c.B}, dev);
    counts = static_cast<const int*>(t.const_data_ptr());
  }
  const at::Tensor kept = a[1] == Py_None ? at::Tensor() : mass_of(a[1], c);
  c.own_memory(Span("the cache's mass", kept));
  float* mass = kept.defined() ? floats(kept) : nullptr;
  Launch on(dev);
  check(call(api.append, x[0].const_data_ptr(), x[1].const_data_ptr(),
             c.r ? x[2].const_data_ptr() : nullptr, strides, c.ptr(0), c.ptr(1), c.ptr(2), c.scale(0),
             c.scale(1), c.scale(2), mass, static_cast<const int*>(start.const_data_ptr()), counts,
             small(c.B, "B"), small(c.Hk, "Hk"), small(n, "n"), small(c.cap, "capacity"),
             static_cast<int>(c.d), static_cast<int>(c.r), on.stream),
        "rfb_cache_append");
  Py_RETURN_NONE;
}

// attn(cache, q, u, lengths, scale, causal, mass, mass_out, decay, out, lse, workspace, counts=None)
PyObject* attn(PyObject* const* a) {
  const Cache& c = cache_of(a[0]);
  const at::Device dev = c.device();
  const at::Tensor& q = tensor(a[1], "q");
  if (q.dim() != 4) refuse(PyExc_ValueError, "q must be [B, H, Nq, d]");
  const int64_t H = q.size(1), Nq = q.size(2);
  require("q", q, at::kBFloat16, {c.B, H, Nq, c.d}, dev);
  const void* u = nullptr;
  if (c.r) {
    const at::Tensor& t = tensor(a[2], "u");
    require("u", t, at::kBFloat16, {c.B, H, Nq, c.r}, dev);
    u = t.const_data_ptr();
  } else if (a[2] != Py_None) {
    refuse(PyExc_ValueError, "u given, but the cache holds no factors (r = 0)");
  }
  if (H && (c.Hk == 0 || H % c.Hk))
    refuse(PyExc_ValueError, H, " query heads are not a multiple of the cache's ", c.Hk);
  const at::Tensor& lengths = tensor(a[3], "lengths");
  require("lengths", lengths, at::kInt, {c.B}, dev);
  const int* counts = nullptr;
  if (a[12] != Py_None) {
    const at::Tensor& t = tensor(a[12], "counts");
    require("counts", t, at::kInt, {c.B}, dev);
    counts = static_cast<const int*>(t.const_data_ptr());
  }
  const float* mass = nullptr;
  float* mass_out = nullptr;
  if (a[6] != Py_None) {
    if (a[7] == Py_None)
      refuse(PyExc_ValueError, "mass needs mass_out (which may be the same tensor)");
    mass = floats(mass_of(a[6], c));
  }
  if (a[7] != Py_None) {
    const at::Tensor& t = tensor(a[7], "mass_out");
    require("mass_out", t, at::kFloat, {c.B, c.Hk, c.cap}, dev);
    mass_out = floats(t);
  }
  const double scale = a[4] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.d)) : number(a[4]);
  const float decay = static_cast<float>(number(a[8]));
  const int causal = PyObject_IsTrue(a[5]);
  if (causal < 0) throw python_error();
  const int B = small(c.B, "B"), h = small(H, "H"), hk = small(c.Hk, "Hk"), nq = small(Nq, "Nq"),
            cap = small(c.cap, "capacity"), d = static_cast<int>(c.d);
  at::Tensor out, lse, ws;
  if (a[9] != Py_None) {
    out = tensor(a[9], "out");
    require("out", out, at::kBFloat16, q.sizes(), dev);
  }
  if (a[10] != Py_None) {
    lse = tensor(a[10], "lse");
    require("lse", lse, at::kFloat, {c.B, H, Nq}, dev);
  }
  if (a[11] != Py_None) {
    ws = tensor(a[11], "workspace");
    if (ws.device() != dev || !ws.is_contiguous())
      refuse(PyExc_ValueError, "workspace must be a contiguous tensor on ", device_text(dev));
  }
  // what is written, of the caller's: apart from what is read and from one another
  if (out.defined() || lse.defined() || ws.defined() || mass_out) {
    const auto given = [&](int i) { return a[i] == Py_None ? at::Tensor() : THPVariable_Unpack(a[i]); };
    const Span written[4] = {{"out", out}, {"lse", lse}, {"workspace", ws}, {"mass_out", given(7)}};
    const Span read[4] = {{"q", q}, {"u", given(2)}, {"lengths", lengths}, {"counts", given(12)}};
    const Span mass_in("mass", given(6));
    for (int i = 0; i < 4; ++i) {
      const Span& x = written[i];
      if (x.lo == x.hi) continue;
      for (int k = 0; k < i; ++k) x.apart(written[k]);
      for (const Span& y : read) x.apart(y);
      for (const Span& y : c.span) x.apart(y);
      if (i < 3) x.apart(mass_in);
      else x.same_or_apart(mass_in);
    }
  }
  Launch on(dev);
  if (!out.defined()) out = make(q.sizes(), at::kBFloat16, dev);
  if (!lse.defined()) lse = make({c.B, H, Nq}, at::kFloat, dev);
  const size_t need = api.workspace(B, h, hk, nq, cap, d, mass_out != nullptr);
  if (!ws.defined()) ws = make({static_cast<int64_t>(need) + 16}, at::kByte, dev);
  const int rc = call(api.attn, q.const_data_ptr(), u, c.ptr(0), c.ptr(1), c.ptr(2), c.scale(0),
                      c.scale(1), c.scale(2), static_cast<const int*>(lengths.const_data_ptr()),
                      counts, mass, mass_out, decay, out.data_ptr(), static_cast<float*>(lse.data_ptr()),
                      ws.data_ptr(), ws.nbytes(), B, h, hk, nq, cap, d, static_cast<int>(c.r),
                      static_cast<float>(scale), causal, on.stream);
  if (rc == RFB_ERR_WORKSPACE)
    refuse(PyExc_RuntimeError, "rfb_attn_fwd_cache: workspace of ", need, " bytes needed");
  check(rc, "rfb_attn_fwd_cache");
  return pair(out, THPVariable_Wrap(lse));
}

// evict(cache, mass, to, to_mass, lengths, keep, recent): caches checked by the caller.
PyObject* evict(PyObject* const* a) {
  const Cache &c = cache_of(a[0]), &to = cache_of(a[2]);
  const at::Device dev = c.device();
  const at::Tensor &mass = mass_of(a[1], c), &to_mass = mass_of(a[3], to);
  const at::Tensor& lengths = tensor(a[4], "lengths");
  require("lengths", lengths, at::kInt, {c.B}, dev);
  // each tensor in the place of its own kind or in no other's
  to.own_memory(Span("the cache's mass", to_mass));
  if (&c != &to) {
    const Span from("", mass), into("", to_mass);
    for (int i = 0; i < 7; ++i)
      for (int k = 0; k < 7; ++k) {
        const Span &x = i < 6 ? to.span[i] : into, &y = k < 6 ? c.span[k] : from;
        if (x.meets(y) && !(i == k && x.lo == y.lo))
          refuse(PyExc_ValueError, "out must not share memory with the cache");
      }
  }
  const int keep = small(integer(a[5]), "keep"), recent = small(integer(a[6]), "recent");
  Launch on(dev);
  at::Tensor n = make({c.B}, at::kInt, dev);
  at::Tensor kept = make({c.B, c.Hk, keep}, at::kInt, dev);
  check(call(api.evict, c.ptr(0), c.ptr(1), c.ptr(2), c.scale(0), c.scale(1), c.scale(2),
             floats(mass), to.ptr(0), to.ptr(1), to.ptr(2),
             to.scale(0), to.scale(1), to.scale(2), floats(to_mass), static_cast<const int*>(lengths.const_data_ptr()), static_cast<int*>(n.data_ptr()),
             static_cast<int*>(kept.data_ptr()), small(c.B, "B"), small(c.Hk, "Hk"),
             small(c.cap, "capacity"), small(to.cap, "capacity"), static_cast<int>(c.d),
             static_cast<int>(c.r), keep, recent, on.stream),
        "rfb_cache_evict");
  return pair(n, THPVariable_Wrap(kept));
}

// init(addresses of the library's functions in the order of Api)
PyObject* init(PyObject* const* a) {
  const auto at_ = [&](int i) { return reinterpret_cast<void*>(integer(a[i])); };
  api.rotary = reinterpret_cast<decltype(api.rotary)>(at_(0));
  api.append = reinterpret_cast<decltype(api.append)>(at_(1));
  api.workspace = reinterpret_cast<decltype(api.workspace)>(at_(2));
  api.attn = reinterpret_cast<decltype(api.attn)>(at_(3));
  api.evict = reinterpret_cast<decltype(api.evict)>(at_(4));
  api.strerror = reinterpret_cast<decltype(api.strerror)>(at_(5));
  api.cuda_error = reinterpret_cast<decltype(api.cuda_error)>(at_(6));
  Py_RETURN_NONE;
}

// No C++ exception leaves an entry.  The last MORE arguments may be left out (None).
template <PyObject* (*F)(PyObject* const*), int N, int MORE>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n < N || n > N + MORE) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  PyObject* all[N + MORE];
  if (n < N + MORE) {
    for (int i = 0; i < N + MORE; ++i) all[i] = i < n ? args[i] : Py_None;
    args = all;
  }
  try {
    return F(args);
  } catch (const Refusal& e) {
    PyErr_SetString(e.type, e.text.c_str());
  } catch (python_error& e) {
    e.restore();
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define RFB_ENTRY(NAME, N, MORE)                                                                  \
  {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<NAME, N, MORE>)), METH_FASTCALL, \
   ""}
PyMethodDef methods[] = {RFB_ENTRY(rotary, 9, 0), RFB_ENTRY(cache, 6, 0), RFB_ENTRY(append, 7, 0),
                         RFB_ENTRY(attn, 12, 1),  RFB_ENTRY(evict, 7, 0), RFB_ENTRY(init, 7, 0),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving_bind", "", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving_bind() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", RFB_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
