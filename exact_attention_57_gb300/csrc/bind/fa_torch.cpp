// fa_torch.cpp — the torch side of the serving operators' Python wrappers
// (fa.py), compiled: a server calls them several times in every layer of every
// step, where a kernel takes about as long as a launch, and the same checks in
// Python took 8 to 20 us a call.  Each function checks its tensors, allocates
// what was not given, makes one call of the C ABI (include/fa.h) on the given or
// current stream, and returns the outputs, or the status as an int when that
// call refused.  The C entry points come from bind(), as addresses of the loaded
// library, so that this module and ctypes share one libfa.so.
#include <Python.h>

#include <ATen/ExpandUtils.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>

#include "fa.h"

namespace {

using at::Tensor;

decltype(&fa_kv_plan) p_kv_plan = nullptr;
decltype(&fa_rope) p_rope = nullptr;
decltype(&fa_kv4_append) p_append = nullptr;
decltype(&fa_kv4_gather) p_gather = nullptr;
decltype(&fa_fwd_kv4) p_attention = nullptr;
decltype(&fa_fwd_kv4_workspace) p_workspace = nullptr;

struct Bad {  // becomes a ValueError
  const char *what;
};

bool none(PyObject *o) { return o == Py_None; }

const Tensor &tensor(PyObject *o, const char *what) {
  if (!THPVariable_Check(o)) throw Bad{what};
  return THPVariable_Unpack(o);
}

long long integer(PyObject *o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return x;
}

int int32(PyObject *o) {
  const long long x = integer(o);
  if (x < -2147483648LL || x > 2147483647LL) throw Bad{"an integer argument does not fit 32 bits"};
  return static_cast<int>(x);
}

bool truth(PyObject *o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw python_error();
  return x != 0;
}

// Device and stream of a call; what it allocates belongs to the stream.
struct Call {
  int dev;
  std::optional<c10::cuda::CUDAGuard> device;
  std::optional<c10::cuda::CUDAStreamGuard> own;
  cudaStream_t stream;

  Call(const Tensor &first, PyObject *s) : dev(first.get_device()) {
    if (!first.is_cuda()) throw Bad{"CUDA tensors expected"};
    if (none(s)) {
      device.emplace(static_cast<c10::DeviceIndex>(dev));
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    } else {
      stream = reinterpret_cast<cudaStream_t>(static_cast<uintptr_t>(integer(s)));
      own.emplace(c10::cuda::getStreamFromExternal(stream, static_cast<c10::DeviceIndex>(dev)));
    }
  }
  // Memory from torch's allocator, without the dispatcher (half the time of
  // at::empty for tensors that are plain outputs).
  Tensor make(at::IntArrayRef sizes, at::ScalarType type) const {
    return Tensor(at::detail::empty_cuda(
        sizes, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt));
  }
  // One like x: its strides, or dense ones in their order.
  Tensor like(const Tensor &x) const {
    if (x.is_contiguous()) return make(x.sizes(), x.scalar_type());
    const at::Device d(at::kCUDA, static_cast<c10::DeviceIndex>(dev));
    if (x.is_non_overlapping_and_dense())
      return Tensor(at::detail::empty_strided_cuda(x.sizes(), x.strides(), x.scalar_type(), d));
    return Tensor(at::detail::empty_strided_cuda(
        x.sizes(), at::infer_dense_strides(x.sizes(), x.strides()), x.scalar_type(), d));
  }
  void here(const Tensor &t) const {
    if (!t.is_cuda() || t.get_device() != dev)
      throw Bad{"tensors on one CUDA device expected"};
  }
};

void flat(const Tensor &t, at::ScalarType type, const char *what) {
  if (t.scalar_type() != type || !t.is_contiguous()) throw Bad{what};
}

int dtype_code(const Tensor &t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return FA_DTYPE_BF16;
    case at::kHalf: return FA_DTYPE_F16;
    case at::kFloat: return FA_DTYPE_F32;
    default: throw Bad{"bf16, fp16 or fp32 tensors expected"};
  }
}

template <typename T = void>
T *ptr(const Tensor &t) {
  return static_cast<T *>(t.data_ptr());
}

// The interpreter lock, let go for one call of the library (the first call of a
// process loads its kernels).  The arguments are computed before it.
struct Unlocked {
  PyThreadState *state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

template <typename F, typename... A>
int run(F *f, A... args) {
  Unlocked u;
  return f(args...);
}

PyObject *status(int st) { return PyLong_FromLong(st); }

// The four arrays of a 4-bit cache.
struct Cache {
  const Tensor *kc, *ks, *vc, *vs;
  int blocks, Hk, bs, d;

  Cache(PyObject *const *a, const Call &call)
      : kc(&tensor(a[0], kWhat)), ks(&tensor(a[1], kWhat)), vc(&tensor(a[2], kWhat)),
        vs(&tensor(a[3], kWhat)) {
    for (const Tensor *t : {kc, ks, vc, vs}) {
      flat(*t, at::kByte, kWhat);
      if (t->dim() != 4) throw Bad{kWhat};
      call.here(*t);
    }
    const auto n = kc->sizes();
    for (const Tensor *t : {ks, vc, vs}) {
      const auto m = t->sizes();
      if (m[0] != n[0] || m[1] != n[1] || m[2] != n[2] || m[3] != (t == vc ? n[3] : n[3] / 8))
        throw Bad{kWhat};
    }
    if (n[0] > 2147483647 || n[1] > 65535 || n[2] > 65535 || n[3] > 65535) throw Bad{kWhat};
    blocks = static_cast<int>(n[0]);
    Hk = static_cast<int>(n[1]);
    bs = static_cast<int>(n[2]);
    d = static_cast<int>(2 * n[3]);
  }
  static constexpr const char *kWhat =
      "cache: contiguous uint8 codes [blocks, Hk, block_size, d/2] and scales "
      "[blocks, Hk, block_size, d/16] expected";
};

int count(int64_t n) {
  if (n > 2147483647) throw Bad{"more than 2^31 - 1 elements in a length"};
  return static_cast<int>(n);
}

// ------------------------------------------------------------------ plan
PyObject *kv_plan(PyObject *const *a) {
  const Tensor &cached = tensor(a[0], "cached_lens: a tensor expected");
  const Tensor &fresh = tensor(a[1], "new_lens: a tensor expected");
  const Tensor &free_blocks = tensor(a[2], "free_blocks: a tensor expected");
  const Tensor &table = tensor(a[3], "block_table: a tensor expected");
  const int bs = int32(a[4]), cap = int32(a[5]);
  const Call call(cached, a[8]);
  constexpr const char *kInts = "contiguous int32 tensors expected";
  for (const Tensor *t : {&cached, &fresh, &free_blocks, &table}) {
    flat(*t, at::kInt, kInts);
    call.here(*t);
  }
  const int B = count(cached.numel());
  if (table.dim() != 2 || table.size(0) != B || fresh.numel() != B)
    throw Bad{"cached_lens [B], new_lens [B], block_table [B, max_blocks] expected"};
  const int *head = nullptr;
  if (!none(a[6])) {
    const Tensor &h = tensor(a[6], "free_head: a tensor expected");
    call.here(h);
    if (h.scalar_type() != at::kInt || h.numel() < 1)
      throw Bad{"free_head: an int32 tensor of one element expected"};
    head = ptr<int>(h);
  }
  Tensor out[5];
  PyObject *given = none(a[7]) ? nullptr : a[7];
  const int64_t sizes[5] = {cap, cap, B + 1LL, B, 2};
  if (given) {
    if (!PyTuple_Check(given) || PyTuple_GET_SIZE(given) != 5)
      throw Bad{"out: a tuple of five tensors expected"};
    for (int i = 0; i < 5; ++i) {
      out[i] = tensor(PyTuple_GET_ITEM(given, i), "out: a tuple of five tensors expected");
      flat(out[i], i == 0 ? at::kLong : at::kInt,
           "out: contiguous int64 slots and int32 tensors expected");
      call.here(out[i]);
      if (out[i].numel() != sizes[i])
        throw Bad{"out: slots, positions [capacity], cu_seqlens [B+1], seq_lens [B], counts [2] "
                  "expected"};
    }
  } else {
    for (int i = 0; i < 5; ++i)
      out[i] = call.make({sizes[i] > 0 ? sizes[i] : 0}, i == 0 ? at::kLong : at::kInt);
  }
  const int st = run(p_kv_plan, ptr<int>(cached), ptr<int>(fresh), ptr<int>(free_blocks), head,
                     ptr<int>(table), ptr<long long>(out[0]), ptr<int>(out[1]), ptr<int>(out[2]),
                     ptr<int>(out[3]), ptr<int>(out[4]), B, count(table.size(1)), bs,
                     count(free_blocks.numel()), cap, call.stream);
  if (st != FA_OK) return status(st);
  if (given) {
    Py_INCREF(given);
    return given;
  }
  PyObject *r = PyTuple_New(5);
  if (!r) return nullptr;
  for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(out[i]));
  return r;
}

// ------------------------------------------------------------------ rotary
void strides(const Tensor &x, const Tensor &y, long long (&s)[6]) {
  const auto a = x.strides(), b = y.strides();
  const size_t n = a.size();
  if (a[n - 1] != 1 || b[n - 1] != 1) throw Bad{"rows of contiguous elements expected"};
  if (n == 4) {  // [B, H, N, d]
    s[0] = a[0], s[1] = a[1], s[2] = a[2], s[3] = b[0], s[4] = b[1], s[5] = b[2];
  } else {       // [T, H, d]
    s[0] = 0, s[1] = a[1], s[2] = a[0], s[3] = 0, s[4] = b[1], s[5] = b[0];
  }
}

PyObject *rotary(PyObject *const *a) {
  const Tensor &q = tensor(a[0], "q: a tensor expected");
  const Tensor &pos = tensor(a[2], "positions: a tensor expected");
  const Tensor &table = tensor(a[3], "table: a tensor expected");
  const bool interleaved = truth(a[4]), inverse = truth(a[8]);
  const Call call(q, a[7]);
  call.here(pos);
  call.here(table);
  const int64_t nd = q.dim();
  if (nd != 3 && nd != 4) throw Bad{"q [B,H,N,d] or [T,H,d] expected"};
  const auto n = q.sizes(), at_ = pos.sizes();
  const int64_t B = nd == 4 ? n[0] : 1, H = n[1], N = nd == 4 ? n[2] : n[0], d = n[nd - 1];
  flat(pos, at::kInt, "positions: contiguous int32 [axes, B, N] (or [axes, T]) expected");
  if (nd == 4 ? at_.size() != 3 || at_[1] != B || at_[2] != N : at_.size() != 2 || at_[1] != N)
    throw Bad{"positions: contiguous int32 [axes, B, N] (or [axes, T]) expected"};
  flat(table, at::kLong, "table: the tensor of rotary_table() expected");
  const int code = dtype_code(q);
  auto output = [&](const Tensor &x, PyObject *o) -> Tensor {
    if (none(o)) return call.like(x);
    const Tensor &y = tensor(o, "q_out, k_out: tensors expected");
    call.here(y);
    if (y.sizes() != x.sizes() || y.scalar_type() != x.scalar_type())
      throw Bad{"q_out, k_out: the shapes and dtype of q and k expected"};
    return y;
  };
  long long qs[6], ks[6] = {};
  Tensor k, ko;
  const Tensor qo = output(q, a[5]);
  strides(q, qo, qs);
  const bool has_k = !none(a[1]);
  if (has_k) {
    k = tensor(a[1], "k: a tensor expected");
    call.here(k);
    const auto m = k.sizes();
    if (k.dim() != nd || m[0] != n[0] || m[nd - 1] != d || (nd == 4 && m[2] != N) ||
        k.scalar_type() != q.scalar_type())
      throw Bad{"k: q's shape but for the heads, and its dtype expected"};
    ko = output(k, a[6]);
    strides(k, ko, ks);
  }
  const int st = run(p_rope, ptr(q), ptr(qo), qs, count(H), has_k ? ptr(k) : nullptr, has_k ?
                     ptr(ko) : nullptr, has_k ? ks : nullptr, has_k ? count(k.size(1)) : 0,
                     ptr<int>(pos), count(at_[0]), ptr<unsigned long long>(table), count(B),
                     count(N), count(d), count(2 * table.numel()), interleaved, inverse, code,
                     call.stream);
  if (st != FA_OK) return status(st);
  PyObject *r = PyTuple_New(2);
  if (!r) return nullptr;
  auto give = [](const Tensor &t, PyObject *o) {  // a tensor that was given comes back itself
    if (none(o)) return THPVariable_Wrap(t);
    Py_INCREF(o);
    return o;
  };
  PyTuple_SET_ITEM(r, 0, give(qo, a[5]));
  if (has_k) {
    PyTuple_SET_ITEM(r, 1, give(ko, a[6]));
  } else {
    Py_INCREF(Py_None);
    PyTuple_SET_ITEM(r, 1, Py_None);
  }
  return r;
}

// ------------------------------------------------------------------ cache
PyObject *append(PyObject *const *a) {
  const Tensor &k = tensor(a[0], "k: a tensor expected");
  const Tensor &v = tensor(a[1], "v: a tensor expected");
  const Tensor &slots = tensor(a[2], "slots: a tensor expected");
  const Call call(k, a[9]);
  call.here(v);
  call.here(slots);
  const Cache c(a + 3, call);
  const int ke = int32(a[7]), ve = int32(a[8]);
  flat(slots, at::kLong, "slots: a contiguous int64 tensor expected");
  const int T = count(slots.numel());
  for (const Tensor *x : {&k, &v}) {
    if (x->dim() != 3 || x->size(0) != T || x->size(1) != c.Hk || x->size(2) != c.d ||
        x->scalar_type() != k.scalar_type() || x->stride(2) != 1 ||
        (c.Hk > 1 && x->stride(1) != c.d))
      throw Bad{"k, v [T, Hk, d] of one dtype with contiguous rows expected"};
  }
  const long long row = static_cast<long long>(c.Hk) * c.d;  // of one token, the stride says nothing
  const long long ks = T > 1 ? k.stride(0) : row, vs = T > 1 ? v.stride(0) : row;
  const int code = dtype_code(k);
  const int st = run(p_append, ptr(k), ptr(v), ks, vs, ptr<long long>(slots), T, ptr(*c.kc),
                     ptr(*c.ks), ptr(*c.vc), ptr(*c.vs), c.blocks, c.Hk, c.bs, c.d, ke, ve, code,
                     call.stream);
  if (st != FA_OK) return status(st);
  Py_RETURN_NONE;
}

PyObject *gather(PyObject *const *a) {
  const Tensor &slots = tensor(a[0], "slots: a tensor expected");
  const Call call(slots, a[9]);
  const Cache c(a + 1, call);
  const int ke = int32(a[6]), ve = int32(a[7]);
  flat(slots, at::kLong, "slots: a contiguous int64 tensor expected");
  const int R = count(slots.numel());
  Tensor out[2];
  PyObject *given = none(a[8]) ? nullptr : a[8];
  if (given) {
    if (!PyTuple_Check(given) || PyTuple_GET_SIZE(given) != 2)
      throw Bad{"out: a tuple of two tensors expected"};
    for (int i = 0; i < 2; ++i) {
      out[i] = tensor(PyTuple_GET_ITEM(given, i), "out: a tuple of two tensors expected");
      call.here(out[i]);
      if (out[i].dim() != 3 || out[i].size(0) != R || out[i].size(1) != c.Hk ||
          out[i].size(2) != c.d || !out[i].is_contiguous() ||
          out[i].scalar_type() != out[0].scalar_type())
        throw Bad{"out: two contiguous [R, Hk, d] tensors of the dtype expected"};
    }
  }
  if (!none(a[5])) {
    if (!THPDtype_Check(a[5])) throw Bad{"dtype: a torch dtype expected"};
    const at::ScalarType type = reinterpret_cast<THPDtype *>(a[5])->scalar_type;
    if (given && out[0].scalar_type() != type)
      throw Bad{"out: two contiguous [R, Hk, d] tensors of the dtype expected"};
    if (!given)
      for (Tensor &t : out) t = call.make({R, c.Hk, c.d}, type);
  } else if (!given) {
    for (Tensor &t : out) t = call.make({R, c.Hk, c.d}, at::kBFloat16);
  }
  const int code = dtype_code(out[0]);
  const int st = run(p_gather, ptr<long long>(slots), R, ptr(*c.kc), ptr(*c.ks), ptr(*c.vc),
                     ptr(*c.vs), ptr(out[0]), ptr(out[1]), c.blocks, c.Hk, c.bs, c.d, ke, ve, code,
                     call.stream);
  if (st != FA_OK) return status(st);
  if (given) {
    Py_INCREF(given);
    return given;
  }
  PyObject *r = PyTuple_New(2);
  if (!r) return nullptr;
  for (int i = 0; i < 2; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(out[i]));
  return r;
}

// ------------------------------------------------------------------ attention
PyObject *attention(PyObject *const *a) {
  const Tensor &q = tensor(a[0], "q: a tensor expected");
  const Tensor &table = tensor(a[5], "block_table: a tensor expected");
  const Tensor &lens = tensor(a[6], "seq_lens_k: a tensor expected");
  const Call call(q, a[16]);
  call.here(table);
  call.here(lens);
  const Cache c(a + 1, call);
  const int max_k = int32(a[7]), max_q = int32(a[9]);
  const bool causal = truth(a[11]);
  const int ke = int32(a[12]), ve = int32(a[13]);
  if (q.dim() != 3 || q.size(2) != c.d || !q.is_contiguous())
    throw Bad{"q: a contiguous [total_q, Hq, d] tensor expected"};
  constexpr const char *kInts =
      "seq_lens_k [B], block_table [B, max_blocks], cu_seqlens_q [B+1]: contiguous int32 tensors "
      "expected";
  flat(table, at::kInt, kInts);
  flat(lens, at::kInt, kInts);
  const int B = count(lens.numel()), total = count(q.size(0)), Hq = count(q.size(1));
  if (table.dim() != 2 || table.size(0) != B) throw Bad{kInts};
  const int *cu = nullptr;
  if (!none(a[8])) {
    const Tensor &t = tensor(a[8], kInts);
    flat(t, at::kInt, kInts);
    call.here(t);
    if (t.numel() != B + 1LL) throw Bad{kInts};
    cu = ptr<int>(t);
  }
  double scale = 1.0 / std::sqrt(static_cast<double>(c.d));
  if (!none(a[10])) {
    scale = PyFloat_AsDouble(a[10]);
    if (scale == -1.0 && PyErr_Occurred()) throw python_error();
  }
  const int code = dtype_code(q);
  Tensor out, lse, ws;
  PyObject *const *g = a + 14;  // (out, lse), workspace
  PyObject *po = PyTuple_GET_ITEM(g[0], 0), *pl = PyTuple_GET_ITEM(g[0], 1);
  if (none(po)) {
    out = call.like(q);
  } else {
    out = tensor(po, "out: a contiguous tensor like q expected");
    call.here(out);
    if (out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type() || !out.is_contiguous())
      throw Bad{"out: a contiguous tensor like q expected"};
  }
  if (none(pl)) {
    lse = call.make({Hq, total}, at::kFloat);
  } else {
    lse = tensor(pl, "lse: a contiguous float32 [Hq, total_q] tensor expected");
    call.here(lse);
    if (lse.dim() != 2 || lse.size(0) != Hq || lse.size(1) != total ||
        lse.scalar_type() != at::kFloat || !lse.is_contiguous())
      throw Bad{"lse: a contiguous float32 [Hq, total_q] tensor expected"};
  }
  unsigned long long ws_bytes = 0;
  if (none(g[1])) {
    ws_bytes = p_workspace(B, Hq, c.Hk, max_q, c.d);
    if (ws_bytes > 0)
      ws = call.make({static_cast<int64_t>(ws_bytes)}, at::kByte);
  } else {
    ws = tensor(g[1], "workspace: a tensor expected");
    call.here(ws);
    if (!ws.is_contiguous()) throw Bad{"workspace: a contiguous tensor expected"};
    ws_bytes = ws.nbytes();
  }
  const int st = run(p_attention, ptr(q), ptr(out), ptr<float>(lse), ptr(*c.kc), ptr(*c.ks),
                     ptr(*c.vc), ptr(*c.vs), ptr<int>(table), ptr<int>(lens), cu, B, Hq, c.Hk,
                     total, max_q, max_k, c.blocks, c.bs, count(table.size(1)), c.d,
                     static_cast<float>(scale), causal, ke, ve, code, ws.defined() ? ptr(ws) :
                     nullptr, ws_bytes, call.stream);
  if (st != FA_OK) return status(st);
  PyObject *r = PyTuple_New(2);
  if (!r) return nullptr;
  auto give = [](const Tensor &t, PyObject *o) {
    if (none(o)) return THPVariable_Wrap(t);
    Py_INCREF(o);
    return o;
  };
  PyTuple_SET_ITEM(r, 0, give(out, po));
  PyTuple_SET_ITEM(r, 1, give(lse, pl));
  return r;
}

// One entry: the number of arguments, and exceptions on their way to Python.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", N, n);
    return nullptr;
  }
  if (!p_workspace) {
    PyErr_SetString(PyExc_RuntimeError, "bind() comes first");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Bad &b) {
    PyErr_SetString(PyExc_ValueError, b.what);
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// bind(addresses of the six C entry points)
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "six addresses expected");
    return nullptr;
  }
  void *p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is null");
      return nullptr;
    }
  }
  p_kv_plan = reinterpret_cast<decltype(p_kv_plan)>(p[0]);
  p_rope = reinterpret_cast<decltype(p_rope)>(p[1]);
  p_append = reinterpret_cast<decltype(p_append)>(p[2]);
  p_gather = reinterpret_cast<decltype(p_gather)>(p[3]);
  p_attention = reinterpret_cast<decltype(p_attention)>(p[4]);
  p_workspace = reinterpret_cast<decltype(p_workspace)>(p[5]);
  Py_RETURN_NONE;
}

#define ENTRY(name, f, n) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f, n>)), METH_FASTCALL, \
   nullptr}
PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL,
     nullptr},
    ENTRY("kv_plan", kv_plan, 9), ENTRY("rotary", rotary, 9), ENTRY("kv4_append", append, 10),
    ENTRY("kv4_gather", gather, 10), ENTRY("attention_kv4", attention, 17),
    {nullptr, nullptr, 0, nullptr}};
#undef ENTRY

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch(void) { return PyModule_Create(&g_module); }
