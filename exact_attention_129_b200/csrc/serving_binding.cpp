// serving_binding.cpp -- the Python binding of attn_rotary, attn_paged_append
// and attn_paged_fwd (serving.py documents the functions): tensor checks,
// output allocation, device and stream, and the autograd node of the rotation.
//
// It is compiled, where the binding of the training kernels is ctypes, because
// a decoding step calls these a few times per layer on kernels of 3 to 10 us:
// checking and marshalling in Python took 12 to 19 us a call (and 120 us for a
// forward and backward through a Python autograd function), more than the GPU's
// work.  It still goes through the C ABI only: init() gets the addresses of the
// functions of the loaded libattn.so.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <sstream>
#include <stdexcept>
#include <string>
#include <utility>
#include <vector>

#include "attn.h"

namespace {

using at::Tensor;

struct Abi {
  decltype(&attn_rotary) rotary = nullptr;
  decltype(&attn_paged_append) append = nullptr;
  decltype(&attn_paged_fwd) fwd = nullptr;
  decltype(&attn_paged_workspace_size) workspace = nullptr;
  bool need_cuda = true;
};
Abi abi;
PyObject* attn_error = nullptr;

// thrown by the checks -> ValueError; by a refused call -> AttnError(name, code).
// (std::exceptions, because a backward runs in a thread of the autograd engine, which
// carries those to the caller and ends the process for any other.)
struct BadValue : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct Refused : std::runtime_error {
  Refused(const char* n, int c)
      : std::runtime_error(std::string(n) + ": status " + std::to_string(c)), name(n), code(c) {}
  const char* name;
  int code;
};

template <class... A>
[[noreturn]] void bad(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw BadValue(s.str());
}

struct Rows {  // a [tokens, heads, head_dim] tensor as the C ABI takes it
  void* p = nullptr;
  int64_t st = 0, sh = 0;
};

int32_t int32_of(const char* name, int64_t v) {
  if (v < INT32_MIN || v > INT32_MAX) bad(name, " is out of range: ", v);
  return static_cast<int32_t>(v);
}

void check_device(const char* name, const Tensor& t, c10::Device dev) {
  if (t.device() != dev) bad(name, " is on ", t.device(), ", expected ", dev);
}

Rows rows_of(const char* name, const Tensor& t, c10::Device dev) {
  if (t.dim() != 3) bad(name, " must be [tokens, heads, head_dim], got shape ", t.sizes());
  if (t.scalar_type() != at::kBFloat16) bad(name, " must be torch.bfloat16, got ", t.dtype());
  check_device(name, t, dev);
  const auto s = t.strides();
  if (s[2] != 1 || s[0] % 8 || s[1] % 8 || reinterpret_cast<uintptr_t>(t.data_ptr()) % 16)
    bad(name, " must have a contiguous head_dim, strides that are multiples of 8 and a 16-byte "
        "aligned start, got strides ", s);
  return {t.data_ptr(), s[0], s[1]};
}

// strides under which no two elements share memory: each one past what those below it span
bool disjoint(const Tensor& t) {
  std::vector<std::pair<int64_t, int64_t>> dims;
  for (int64_t i = 0; i < t.dim(); ++i)
    if (t.size(i) > 1) dims.emplace_back(t.stride(i), t.size(i));
  std::sort(dims.begin(), dims.end());
  int64_t span = 1;
  for (const auto& [stride, n] : dims) {
    if (stride < span) return false;
    span += stride * (n - 1);
  }
  return true;
}

// an output for the rows `src`: other memory, or the very same
Rows out_rows(const char* name, const Tensor& t, const Tensor& src, c10::Device dev) {
  const Rows r = rows_of(name, t, dev);
  if (t.sizes() != src.sizes())
    bad(name, " must have shape ", src.sizes(), ", got ", t.sizes());
  // no two threads may write one element
  if (!disjoint(t)) bad(name, " overlaps itself, strides ", t.strides());
  return r;
}

Rows fresh_rows(const Tensor& src, Tensor* out) {
  *out = at::empty(src.sizes(), src.options());
  return {out->data_ptr(), src.size(1) * src.size(2), src.size(2)};
}

const int32_t* ints(const char* name, const Tensor& t, c10::Device dev, int64_t n) {
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    bad(name, " must be a contiguous int32 tensor of shape [", n, "], got ", t.dtype(), " ",
        t.sizes());
  check_device(name, t, dev);
  return t.data_ptr<int32_t>();
}

int64_t batch_of(const char* name, const Tensor& t) {
  if (t.dim() != 1 || t.size(0) < 2) bad(name, " must be a 1-D int32 tensor of batch + 1 offsets");
  return t.size(0) - 1;
}

const double* freqs(const Tensor& t, c10::Device dev, int64_t d, int32_t* n) {
  if (t.scalar_type() != at::kDouble || t.dim() != 1 || !t.is_contiguous())
    bad("inv_freq must be a contiguous 1-D float64 tensor");
  check_device("inv_freq", t, dev);
  if (t.size(0) % 8 || 2 * t.size(0) > d)
    bad("2 * len(inv_freq) must be a multiple of 16 up to head_dim ", d, ", got ", 2 * t.size(0));
  *n = static_cast<int32_t>(t.size(0));
  return t.data_ptr<double>();
}

void need_cuda(const Tensor& t) {
  if (abi.need_cuda && !t.is_cuda()) bad("exact_attention_129_b200 runs on CUDA tensors only");
}

attn_stream_t stream_of(c10::Device dev) {
  if (!dev.is_cuda()) return nullptr;
  return reinterpret_cast<attn_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

// ---------------------------------------------------------------------------
// rotary
// ---------------------------------------------------------------------------
struct RotaryArgs {
  Tensor inv_freq, cu, offsets, positions;
  bool interleaved = false, inverse = false;
  double mscale = 1.0;
};

void rotary_run(const Tensor& q, const Tensor& k, const RotaryArgs& a, Tensor& q_out,
                Tensor& k_out) {
  const auto dev = q.device();
  const Rows qr = rows_of("q", q, dev);
  const int64_t t = q.size(0), d = q.size(2);
  Rows kr;
  if (k.defined()) {
    kr = rows_of("k", k, dev);
    if (k.size(0) != t || k.size(2) != d)
      bad("k ", k.sizes(), " does not match q ", q.sizes());
  } else if (k_out.defined()) {
    bad("k_out without k");
  }
  int32_t nf = 0;
  const double* f = freqs(a.inv_freq, dev, d, &nf);
  if (a.positions.defined() && a.cu.defined()) bad("positions and cu_seqlens exclude each other");
  if (a.offsets.defined() && !a.cu.defined()) bad("offsets need cu_seqlens");
  const int32_t *pos = nullptr, *cu = nullptr, *off = nullptr;
  int64_t batch = 0;
  if (a.positions.defined()) pos = ints("positions", a.positions, dev, t);
  if (a.cu.defined()) {
    batch = batch_of("cu_seqlens", a.cu);
    cu = ints("cu_seqlens", a.cu, dev, batch + 1);
    if (a.offsets.defined()) off = ints("offsets", a.offsets, dev, batch);
    if (k.defined() && q_out.defined() != k_out.defined())
      bad("with cu_seqlens, pass both outputs or neither");
  }
  const bool zero = !q_out.defined();
  Rows qo, ko;
  if (q_out.defined()) qo = out_rows("q_out", q_out, q, dev);
  if (k_out.defined()) ko = out_rows("k_out", k_out, k, dev);
  need_cuda(q);
  const c10::cuda::OptionalCUDAGuard guard(dev.is_cuda() ? std::optional<c10::Device>(dev)
                                                         : std::nullopt);
  if (!q_out.defined()) qo = fresh_rows(q, &q_out);
  if (k.defined() && !k_out.defined()) ko = fresh_rows(k, &k_out);
  if (t == 0) return;
  const int rc = abi.rotary(qr.p, qr.st, qr.sh, kr.p, kr.st, kr.sh, qo.p, qo.st, qo.sh, ko.p,
                            ko.st, ko.sh, f, nf, a.interleaved, static_cast<float>(a.mscale),
                            a.inverse, pos, cu, off, int32_of("batch", batch), zero,
                            int32_of("tokens", t), int32_of("nheads_q", q.size(1)),
                            k.defined() ? int32_of("nheads_kv", k.size(1)) : 0,
                            int32_of("head_dim", d), stream_of(dev));
  if (rc != ATTN_OK) throw Refused("attn_rotary", rc);
}

// a gradient as the kernel can read it
Tensor readable(const Tensor& t) {
  const auto s = t.strides();
  if (t.dim() == 3 && s[2] == 1 && s[0] % 8 == 0 && s[1] % 8 == 0 &&
      reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0)
    return t;
  return t.clone(at::MemoryFormat::Contiguous);
}

// The rotation is linear and its transpose is the rotation the other way, so the
// backward is the same node with `inverse` flipped (and differentiable itself).
struct RotaryNode : public torch::autograd::Function<RotaryNode> {
  static torch::autograd::variable_list forward(torch::autograd::AutogradContext* ctx,
                                                const Tensor& q, const std::optional<Tensor>& k,
                                                const Tensor& inv_freq,
                                                const std::optional<Tensor>& cu,
                                                const std::optional<Tensor>& offsets,
                                                const std::optional<Tensor>& positions,
                                                bool interleaved, bool inverse, double mscale) {
    RotaryArgs a{inv_freq, cu.value_or(Tensor()), offsets.value_or(Tensor()),
                 positions.value_or(Tensor()), interleaved, inverse, mscale};
    ctx->save_for_backward({a.inv_freq, a.cu, a.offsets, a.positions});
    ctx->saved_data["interleaved"] = interleaved;
    ctx->saved_data["inverse"] = inverse;
    ctx->saved_data["mscale"] = mscale;
    ctx->saved_data["k"] = k.has_value();
    Tensor qo, ko;
    rotary_run(q, k.value_or(Tensor()), a, qo, ko);
    if (k.has_value()) return {qo, ko};
    return {qo};
  }

  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    const auto saved = ctx->get_saved_variables();
    const bool has_k = ctx->saved_data["k"].toBool();
    auto opt = [](const Tensor& t) {
      return t.defined() ? std::optional<Tensor>(t) : std::nullopt;
    };
    const bool interleaved = ctx->saved_data["interleaved"].toBool();
    const bool inverse = !ctx->saved_data["inverse"].toBool();
    const double mscale = ctx->saved_data["mscale"].toDouble();
    auto turn = [&](const Tensor& q,
                    const std::optional<Tensor>& k) -> torch::autograd::variable_list {
      if (at::GradMode::is_enabled())  // a gradient of the gradient is wanted
        return apply(q, k, saved[0], opt(saved[1]), opt(saved[2]), opt(saved[3]), interleaved,
                     inverse, mscale);
      Tensor qo, ko;
      rotary_run(q, k.value_or(Tensor()),
                 {saved[0], saved[1], saved[2], saved[3], interleaved, inverse, mscale}, qo, ko);
      return {qo, ko};
    };
    Tensor dq, dk;
    const bool want_q = ctx->needs_input_grad(0) && grads[0].defined();
    const bool want_k = has_k && ctx->needs_input_grad(1) && grads[1].defined();
    if (want_q && want_k) {
      auto both = turn(readable(grads[0]), readable(grads[1]));
      dq = both[0], dk = both[1];
    } else if (want_q) {
      dq = turn(readable(grads[0]), std::nullopt)[0];
    } else if (want_k) {
      dk = turn(readable(grads[1]), std::nullopt)[0];
    }
    return {dq, dk, Tensor(), Tensor(), Tensor(), Tensor(), Tensor(), Tensor(), Tensor()};
  }
};

// ---------------------------------------------------------------------------
// the paged cache
// ---------------------------------------------------------------------------
struct CacheArgs {
  Tensor k, v, k_scale, v_scale, table;
};

attn_paged_cache_t cache_of(const CacheArgs& a, c10::Device dev) {
  attn_paged_cache_t c{};
  const auto type = a.k.scalar_type();
  if (type != at::kBFloat16 && type != at::kFloat8_e4m3fn)
    bad("k_cache must be bfloat16 or float8_e4m3fn, got ", a.k.dtype());
  const bool e4m3 = type == at::kFloat8_e4m3fn;
  if (a.k.dim() != 4 || a.v.sizes() != a.k.sizes() || a.v.scalar_type() != type)
    bad("k_cache and v_cache must be [num_pages, page_size, nheads_kv, head_dim] of one type, got ",
        a.k.sizes(), " and ", a.v.sizes());
  const auto shape = a.k.sizes();
  if (shape[1] != 16 && shape[1] != 32 && shape[1] != 64 && shape[1] != 128)
    bad("page_size must be 16, 32, 64 or 128, got ", shape[1]);
  const int64_t step = e4m3 ? 16 : 8;
  auto pool = [&](const char* name, const Tensor& t, void** p, int64_t* page, int64_t* token,
                  int64_t* head) {
    check_device(name, t, dev);
    const auto s = t.strides();
    if (s[3] != 1 || s[0] % step || s[1] % step || s[2] % step ||
        reinterpret_cast<uintptr_t>(t.data_ptr()) % 16)
      bad(name, " must have a contiguous head_dim, strides that are multiples of 16 bytes and a "
          "16-byte aligned start, got strides ", s);
    *p = t.data_ptr();
    *page = s[0], *token = s[1], *head = s[2];
  };
  pool("k_cache", a.k, &c.k, &c.k_s_page, &c.k_s_token, &c.k_s_head);
  pool("v_cache", a.v, &c.v, &c.v_s_page, &c.v_s_token, &c.v_s_head);
  auto scale = [&](const char* name, const Tensor& t) -> float* {
    if (!t.defined() || t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != shape[0] ||
        t.size(1) != shape[2] || !t.is_contiguous() || t.device() != dev)
      bad(name, " must be a contiguous float32 tensor of shape [", shape[0], ", ", shape[2],
          "] on ", dev, " for an e4m3 cache");
    return t.data_ptr<float>();
  };
  if (e4m3) {
    c.k_scale = scale("k_scale", a.k_scale);
    c.v_scale = scale("v_scale", a.v_scale);
  } else if (a.k_scale.defined() || a.v_scale.defined()) {
    bad("scales belong to an e4m3 cache");
  }
  if (a.table.scalar_type() != at::kInt || a.table.dim() != 2 ||
      (a.table.size(1) > 1 && a.table.stride(1) != 1))
    bad("block_table must be int32 [batch, pages_per_seq] with contiguous rows");
  check_device("block_table", a.table, dev);
  c.block_table = a.table.data_ptr<int32_t>();
  c.table_stride = a.table.stride(0);
  c.type = e4m3 ? ATTN_CACHE_E4M3 : ATTN_CACHE_BF16;
  c.num_pages = int32_of("num_pages", shape[0]);
  c.page_size = static_cast<int32_t>(shape[1]);
  c.pages_per_seq = int32_of("pages_per_seq", a.table.size(1));
  c.nheads_kv = int32_of("nheads_kv", shape[2]);
  c.head_dim = int32_of("head_dim", shape[3]);
  return c;
}

int64_t sequences(const char* name, const Tensor& cu, const Tensor& seqlens, const Tensor& table,
                  c10::Device dev, const int32_t** cup, const int32_t** lens) {
  const int64_t batch = batch_of(name, cu);
  *cup = ints(name, cu, dev, batch + 1);
  *lens = ints("seqlens_k", seqlens, dev, batch);
  if (table.size(0) != batch)
    bad("block_table has ", table.size(0), " rows for ", batch, " sequences");
  return batch;
}

struct AppendArgs {
  Tensor k, v, cu, seqlens, q, q_out, inv_freq;
  CacheArgs cache;
  int64_t max_seqlen;
  bool interleaved;
  double mscale;
};

Tensor append_run(AppendArgs& a) {
  const auto dev = a.k.device();
  const Rows k = rows_of("k", a.k, dev), v = rows_of("v", a.v, dev);
  if (a.v.sizes() != a.k.sizes()) bad("v must have shape ", a.k.sizes(), ", got ", a.v.sizes());
  const attn_paged_cache_t c = cache_of(a.cache, dev);
  if (!disjoint(a.cache.k) || !disjoint(a.cache.v))
    bad("k_cache and v_cache are written: they must not overlap themselves");
  const int64_t t = a.k.size(0), d = c.head_dim;
  if (a.k.size(1) != c.nheads_kv || a.k.size(2) != d)
    bad("k ", a.k.sizes(), " does not match the cache's ", c.nheads_kv, " heads of ", d);
  const int32_t *cu, *lens;
  const int64_t batch = sequences("cu_seqlens", a.cu, a.seqlens, a.cache.table, dev, &cu, &lens);
  Rows q, qo;
  if (a.q.defined()) {
    q = rows_of("q", a.q, dev);
    if (a.q.size(0) != t || a.q.size(2) != d)
      bad("q ", a.q.sizes(), " does not match k ", a.k.sizes());
    if (a.q_out.defined()) qo = out_rows("q_out", a.q_out, a.q, dev);
  } else if (a.q_out.defined()) {
    bad("q_out without q");
  }
  int32_t nf = 0;
  const double* f = a.inv_freq.defined() ? freqs(a.inv_freq, dev, d, &nf) : nullptr;
  need_cuda(a.k);
  const c10::cuda::OptionalCUDAGuard guard(dev.is_cuda() ? std::optional<c10::Device>(dev)
                                                         : std::nullopt);
  if (a.q.defined() && !a.q_out.defined()) qo = fresh_rows(a.q, &a.q_out);
  if (t == 0) return a.q_out;
  const int rc = abi.append(&c, k.p, k.st, k.sh, v.p, v.st, v.sh, q.p, q.st, q.sh, qo.p, qo.st,
                            qo.sh, cu, lens, int32_of("batch", batch), int32_of("tokens", t),
                            int32_of("max_seqlen", a.max_seqlen),
                            a.q.defined() ? int32_of("nheads_q", a.q.size(1)) : 0, f, nf,
                            a.interleaved, static_cast<float>(a.mscale), stream_of(dev));
  if (rc != ATTN_OK) throw Refused("attn_paged_append", rc);
  return a.q_out;
}

struct FwdArgs {
  Tensor q, cu, seqlens, out, lse, workspace;
  CacheArgs cache;
  int64_t max_q, max_k, left, right, splits;
  double scale, softcap;
  bool causal, return_lse, default_scale;
};

void like(const char* name, const Tensor& t, at::IntArrayRef shape, at::ScalarType type,
          c10::Device dev) {
  if (!t.defined()) return;
  if (t.sizes() != shape) bad(name, " must have shape ", shape, ", got ", t.sizes());
  if (t.scalar_type() != type) bad(name, " must be ", type, ", got ", t.dtype());
  if (!t.is_contiguous()) bad(name, " must be contiguous");
  check_device(name, t, dev);
}

void fwd_run(FwdArgs& a) {
  const auto dev = a.q.device();
  if (a.q.dim() != 3) bad("q must be [tokens, heads, head_dim], got shape ", a.q.sizes());
  like("q", a.q, a.q.sizes(), at::kBFloat16, dev);
  const attn_paged_cache_t c = cache_of(a.cache, dev);
  const int64_t t = a.q.size(0), hq = a.q.size(1), d = a.q.size(2);
  if (c.head_dim != d) bad("q and the cache differ in head_dim: ", d, " and ", c.head_dim);
  if (hq < 1 || c.nheads_kv < 1 || hq % c.nheads_kv)
    bad("nheads_q ", hq, " is not a multiple of nheads_kv ", c.nheads_kv);
  const int32_t *cu, *lens;
  const int64_t batch = sequences("cu_seqlens_q", a.cu, a.seqlens, a.cache.table, dev, &cu, &lens);
  like("out", a.out, a.q.sizes(), at::kBFloat16, dev);
  like("lse", a.lse, {hq, t}, at::kFloat, dev);
  if (a.workspace.defined() && (!a.workspace.is_contiguous() || a.workspace.device() != dev))
    bad("workspace must be a contiguous tensor on q's device");
  need_cuda(a.q);
  const c10::cuda::OptionalCUDAGuard guard(dev.is_cuda() ? std::optional<c10::Device>(dev)
                                                         : std::nullopt);
  if (!a.out.defined()) a.out = at::empty(a.q.sizes(), a.q.options());
  if (!a.return_lse)
    a.lse = Tensor();
  else if (!a.lse.defined())
    a.lse = at::empty({hq, t}, a.q.options().dtype(at::kFloat));
  if (t == 0) return;
  const int32_t b = int32_of("batch", batch), tq = int32_of("tokens", t),
                mq = int32_of("max_seqlen_q", a.max_q), mk = int32_of("max_seqlen_k", a.max_k),
                h = int32_of("nheads_q", hq), wl = int32_of("window", a.left),
                wr = int32_of("window", a.right), splits = int32_of("num_splits", a.splits);
  if (!a.workspace.defined()) {
    const size_t need = abi.workspace(&c, b, tq, mq, mk, h, a.causal, wl, wr, splits);
    if (need) a.workspace = at::empty({static_cast<int64_t>(need)}, a.q.options().dtype(at::kByte));
  }
  const double scale = a.default_scale ? 1.0 / std::sqrt(static_cast<double>(d)) : a.scale;
  const int rc = abi.fwd(&c, a.q.data_ptr(), cu, lens, b, tq, mq, mk, h,
                         static_cast<float>(scale), a.causal, wl, wr,
                         static_cast<float>(a.softcap), splits, a.return_lse, a.out.data_ptr(),
                         a.lse.defined() ? a.lse.data_ptr<float>() : nullptr,
                         a.workspace.defined() ? a.workspace.data_ptr() : nullptr,
                         a.workspace.defined() ? a.workspace.nbytes() : 0, stream_of(dev));
  if (rc != ATTN_OK) throw Refused("attn_paged_fwd", rc);
}

// ---------------------------------------------------------------------------
// Python
// ---------------------------------------------------------------------------
struct PyFail {};  // a Python error is set

Tensor tensor_of(const char* name, PyObject* o, bool optional = false) {
  if (optional && o == Py_None) return Tensor();
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor%s, got %s", name,
                 optional ? " or None" : "", Py_TYPE(o)->tp_name);
    throw PyFail{};
  }
  return THPVariable_Unpack(o);
}
int64_t long_of(PyObject* o) {
  // as int(): floats and numpy integers too
  PyObject* i = PyNumber_Long(o);
  const long long v = i ? PyLong_AsLongLong(i) : -1;
  Py_XDECREF(i);
  if (v == -1 && PyErr_Occurred()) throw PyFail{};
  return v;
}
double double_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyFail{};
  return v;
}
bool bool_of(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyFail{};
  return v != 0;
}
PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* wrap_pair(const Tensor& a, const Tensor& b) {
  PyObject *x = wrap(a), *y = wrap(b);
  PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

struct NoGil {
  PyThreadState* s = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(s); }
};

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  try {
    if (n != want) {
      PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
      return nullptr;
    }
    if (!abi.fwd) {
      PyErr_SetString(PyExc_ImportError, "libattn.so has not been loaded");
      return nullptr;
    }
    return f();
  } catch (const PyFail&) {
  } catch (const BadValue& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Refused& e) {
    PyObject* x = PyObject_CallFunction(attn_error, "si", e.name, e.code);
    if (x) {
      PyErr_SetObject(attn_error, x);
      Py_DECREF(x);
    }
  } catch (...) {  // torch's own errors, out of memory among them
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

RotaryArgs rotary_args(PyObject* const* a, bool inverse) {
  RotaryArgs r;
  r.inv_freq = tensor_of("inv_freq", a[2]);
  r.cu = tensor_of("cu_seqlens", a[3], true);
  r.offsets = tensor_of("offsets", a[4], true);
  r.positions = tensor_of("positions", a[5], true);
  r.interleaved = bool_of(a[6]);
  r.mscale = double_of(a[7]);
  r.inverse = inverse;
  return r;
}

// q, k, inv_freq, cu_seqlens, offsets, positions, interleaved, mscale, inverse, q_out, k_out
PyObject* py_rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const Tensor q = tensor_of("q", a[0]), k = tensor_of("k", a[1], true);
    const RotaryArgs r = rotary_args(a, bool_of(a[8]));
    Tensor qo = tensor_of("q_out", a[9], true), ko = tensor_of("k_out", a[10], true);
    {
      NoGil nogil;
      rotary_run(q, k, r, qo, ko);
    }
    return wrap_pair(qo, ko);
  });
}

// q, k, inv_freq, cu_seqlens, offsets, positions, interleaved, mscale
PyObject* py_rotary_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const Tensor q = tensor_of("q", a[0]), k = tensor_of("k", a[1], true);
    const RotaryArgs r = rotary_args(a, false);
    if (r.inv_freq.requires_grad()) bad("inv_freq has no gradient here: pass it detached");
    auto opt = [](const Tensor& t) {
      return t.defined() ? std::optional<Tensor>(t) : std::nullopt;
    };
    torch::autograd::variable_list out;
    {
      NoGil nogil;
      out = RotaryNode::apply(q, opt(k), r.inv_freq, opt(r.cu), opt(r.offsets), opt(r.positions),
                              r.interleaved, false, r.mscale);
    }
    return wrap_pair(out[0], out.size() > 1 ? out[1] : Tensor());
  });
}

CacheArgs cache_args(PyObject* k, PyObject* v, PyObject* table, PyObject* ks, PyObject* vs) {
  return {tensor_of("k_cache", k), tensor_of("v_cache", v), tensor_of("k_scale", ks, true),
          tensor_of("v_scale", vs, true), tensor_of("block_table", table)};
}

// k, v, k_cache, v_cache, block_table, cu_seqlens, seqlens_k, max_seqlen, k_scale, v_scale, q,
// q_out, inv_freq, interleaved, mscale
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    AppendArgs r{tensor_of("k", a[0]),          tensor_of("v", a[1]),
                 tensor_of("cu_seqlens", a[5]), tensor_of("seqlens_k", a[6]),
                 tensor_of("q", a[10], true),   tensor_of("q_out", a[11], true),
                 tensor_of("inv_freq", a[12], true),
                 cache_args(a[2], a[3], a[4], a[8], a[9]),
                 long_of(a[7]),                 bool_of(a[13]),
                 double_of(a[14])};
    Tensor out;
    {
      NoGil nogil;
      out = append_run(r);
    }
    return wrap(out);
  });
}

// q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k, max_seqlen_q, max_seqlen_k, k_scale,
// v_scale, scale, causal, window, softcap, return_lse, out, lse, num_splits, workspace
PyObject* py_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 19, [&] {
    FwdArgs r;
    r.q = tensor_of("q", a[0]);
    r.cache = cache_args(a[1], a[2], a[3], a[8], a[9]);
    r.cu = tensor_of("cu_seqlens_q", a[4]);
    r.seqlens = tensor_of("seqlens_k", a[5]);
    r.max_q = long_of(a[6]);
    r.max_k = long_of(a[7]);
    r.default_scale = a[10] == Py_None;
    r.scale = r.default_scale ? 0.0 : double_of(a[10]);
    r.causal = bool_of(a[11]);
    r.left = r.right = -1;
    if (a[12] != Py_None) {
      PyObject* w = PySequence_Fast(a[12], "window must be None or (left, right)");
      if (!w) throw PyFail{};
      PyObject* l = PySequence_Fast_GET_SIZE(w) == 2 ? PySequence_Fast_GET_ITEM(w, 0) : nullptr;
      PyObject* g = l ? PySequence_Fast_GET_ITEM(w, 1) : nullptr;
      try {
        if (!l) bad("window must be None or (left, right)");
        if (l != Py_None) r.left = std::max<int64_t>(-1, std::min<int64_t>(long_of(l), 1 << 30));
        if (g != Py_None) r.right = std::max<int64_t>(-1, std::min<int64_t>(long_of(g), 1 << 30));
      } catch (...) {
        Py_DECREF(w);
        throw;
      }
      Py_DECREF(w);
    }
    r.softcap = a[13] == Py_None ? 0.0 : double_of(a[13]);
    r.return_lse = bool_of(a[14]);
    r.out = tensor_of("out", a[15], true);
    r.lse = tensor_of("lse", a[16], true);
    r.splits = long_of(a[17]);
    r.workspace = tensor_of("workspace", a[18], true);
    {
      NoGil nogil;
      fwd_run(r);
    }
    return wrap_pair(r.out, r.lse);
  });
}

// k_cache, v_cache, block_table, k_scale, v_scale, batch, total_q, max_seqlen_q, max_seqlen_k,
// nheads_q, causal, window_left, window_right, num_splits
PyObject* py_workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    const CacheArgs c = cache_args(a[0], a[1], a[2], a[3], a[4]);
    const attn_paged_cache_t abi_cache = cache_of(c, c.k.device());
    const int32_t v[] = {int32_of("batch", long_of(a[5])), int32_of("total_q", long_of(a[6])),
                         int32_of("max_seqlen_q", long_of(a[7])),
                         int32_of("max_seqlen_k", long_of(a[8])),
                         int32_of("nheads_q", long_of(a[9])), bool_of(a[10]),
                         int32_of("window", long_of(a[11])), int32_of("window", long_of(a[12])),
                         int32_of("num_splits", long_of(a[13]))};
    const auto dev = c.k.device();
    const c10::cuda::OptionalCUDAGuard guard(dev.is_cuda() ? std::optional<c10::Device>(dev)
                                                           : std::nullopt);
    return PyLong_FromSize_t(
        abi.workspace(&abi_cache, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8]));
  });
}

// init(AttnError, addresses of attn_rotary, attn_paged_append, attn_paged_fwd,
// attn_paged_workspace_size, need_cuda): the tests of the marshalling give addresses of their own
// and CPU tensors
PyObject* py_init(PyObject*, PyObject* args) {
  PyObject* error;
  unsigned long long r, p, f, w;
  int cuda;
  if (!PyArg_ParseTuple(args, "OKKKKp", &error, &r, &p, &f, &w, &cuda)) return nullptr;
  Py_INCREF(error);
  Py_XDECREF(attn_error);
  attn_error = error;
  abi = {reinterpret_cast<decltype(&attn_rotary)>(r),
         reinterpret_cast<decltype(&attn_paged_append)>(p),
         reinterpret_cast<decltype(&attn_paged_fwd)>(f),
         reinterpret_cast<decltype(&attn_paged_workspace_size)>(w), cuda != 0};
  Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"init", py_init, METH_VARARGS, nullptr},
    {"rotary", fast(py_rotary), METH_FASTCALL, nullptr},
    {"rotary_grad", fast(py_rotary_grad), METH_FASTCALL, nullptr},
    {"append", fast(py_append), METH_FASTCALL, nullptr},
    {"fwd", fast(py_fwd), METH_FASTCALL, nullptr},
    {"workspace_size", fast(py_workspace), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&module); }
