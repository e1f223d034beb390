// Argument marshalling of the operators between the linears, from Python: each function checks the
// tensors of one call (device, type, shape, layout), passes their addresses and pitches to the C
// entry point and returns its status. No arithmetic, no copies.
//
// Compiled because the checks are what small calls cost: through ctypes, with each check an
// interpreted call, one took 0.4 us and the 22 tensors of an append 8 us, beside 3 us for the
// launch itself. `dev` is the device the call runs on, `stream` a raw hipStream_t.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "fp8rl_block.h"

namespace {

// A Python exception has been set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Raised{};
}

bool none(PyObject* o) { return o == nullptr || o == Py_None; }

std::string shape_of(c10::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name, int dev) {
  if (!THPVariable_Check(o))
    raise(PyExc_ValueError, std::string(name) + " must be a device (cuda) tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a device (cuda) tensor");
  if (t.get_device() != dev)
    raise(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
                                ", the call runs on cuda:" + std::to_string(dev));
  return t;
}

void need_type(const at::Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", got " +
                               c10::toString(t.scalar_type()));
}

void need_shape(const at::Tensor& t, const char* name, c10::IntArrayRef shape) {
  if (t.sizes() != shape)
    raise(PyExc_ValueError, std::string(name) + " has shape " + shape_of(t.sizes()) +
                                ", expected " + shape_of(shape));
}

void need_2d(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) raise(PyExc_ValueError, std::string(name) + " must be 2-D");
}

// A matrix of rows: its address and row pitch (that of one row does not matter).
struct Rows {
  void* p = nullptr;
  int64_t ld = 0;
};

Rows matrix(const at::Tensor& t, const char* name, at::ScalarType type, int64_t rows,
            int64_t cols) {
  need_type(t, name, type);
  need_shape(t, name, {rows, cols});
  if (cols > 1 && t.stride(1) != 1)
    raise(PyExc_ValueError, std::string(name) + " must have unit stride along its last dimension");
  return {t.data_ptr(), rows > 1 ? t.stride(0) : cols};
}

Rows matrix(PyObject* o, const char* name, int dev, at::ScalarType type, int64_t rows,
            int64_t cols) {
  return none(o) ? Rows{} : matrix(tensor(o, name, dev), name, type, rows, cols);
}

// The address of a contiguous tensor of n values.
template <typename T = void>
T* flat(PyObject* o, const char* name, int dev, at::ScalarType type, int64_t n) {
  if (none(o)) return nullptr;
  const at::Tensor& t = tensor(o, name, dev);
  need_type(t, name, type);
  if (t.numel() != n)
    raise(PyExc_ValueError, std::string(name) + " has " + std::to_string(t.numel()) +
                                " values, expected " + std::to_string(n));
  if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
  return static_cast<T*>(t.data_ptr());
}

// The address of a contiguous matrix.
template <typename T>
T* dense(PyObject* o, const char* name, int dev, at::ScalarType type, int64_t rows, int64_t cols) {
  if (none(o)) return nullptr;
  need_shape(tensor(o, name, dev), name, {rows, cols});
  return flat<T>(o, name, dev, type, rows * cols);
}

int out_type(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return FP8RL_OUT_BF16;
  if (t.scalar_type() == at::kFloat) return FP8RL_OUT_F32;
  raise(PyExc_TypeError, std::string(name) + " must be BFloat16 or Float, got " +
                             c10::toString(t.scalar_type()));
}

// A call's workspace: the caller's, or memory beside t that lives until the call returns (the
// caching allocator hands it out again only behind what the stream has been given).
struct Workspace {
  at::Tensor own;
  void* p = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* o, size_t need, const at::Tensor& t, int dev) {
    if (!none(o)) {
      const at::Tensor& w = tensor(o, "workspace", dev);
      if (!w.is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
      p = w.data_ptr(), bytes = w.nbytes();
    } else if (need > 0) {
      own = at::empty({(int64_t)need}, t.options().dtype(at::kByte));
      p = own.data_ptr(), bytes = need;
    }
  }
};

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return (float)v;
}

void* stream_of(PyObject* o) {
  void* s = PyLong_AsVoidPtr(o);
  if (!s && PyErr_Occurred()) throw Raised{};
  return s;
}

constexpr at::ScalarType kBf16 = at::kBFloat16;

// x, weight, residual, eps, h, y, xq, sa, scale_fmt, dev, stream
int add_rmsnorm_quant(PyObject* const* a) {
  const int dev = (int)integer(a[9]);
  const at::Tensor& x = tensor(a[0], "x", dev);
  need_2d(x, "x");
  const int64_t M = x.size(0), K = x.size(1);
  const Rows rx = matrix(x, "x", kBf16, M, K);
  auto* w = flat<uint16_t>(a[1], "weight", dev, kBf16, K);
  const Rows rr = matrix(a[2], "residual", dev, kBf16, M, K);
  const float eps = number(a[3]);
  const Rows rh = matrix(a[4], "h", dev, kBf16, M, K);
  const Rows ry = matrix(a[5], "y", dev, kBf16, M, K);
  const Rows rq = matrix(a[6], "xq", dev, at::kByte, M, K);
  auto* sa = dense<float>(a[7], "sa", dev, at::kFloat, M, K / 128);
  const int fmt = (int)integer(a[8]);
  void* stream = stream_of(a[10]);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = fp8rl_add_rmsnorm_quant((uint16_t*)rx.p, rx.ld, (uint16_t*)rr.p, rr.ld, w, eps, M, K,
                                   (uint16_t*)rh.p, rh.ld, (uint16_t*)ry.p, ry.ld, (uint8_t*)rq.p,
                                   rq.ld, sa, fmt, stream);
  Py_END_ALLOW_THREADS
  return status;
}

// dy, h, weight, dh, eps, dx, dw, workspace, dev, stream
int add_rmsnorm_bwd(PyObject* const* a) {
  const int dev = (int)integer(a[8]);
  const at::Tensor& dy = tensor(a[0], "dy", dev);
  need_2d(dy, "dy");
  const int64_t M = dy.size(0), K = dy.size(1);
  const Rows rg = matrix(dy, "dy", kBf16, M, K);
  const Rows rh = matrix(a[1], "h", dev, kBf16, M, K);
  auto* w = flat<uint16_t>(a[2], "weight", dev, kBf16, K);
  const Rows rd = matrix(a[3], "dh", dev, kBf16, M, K);
  const float eps = number(a[4]);
  const Rows rx = matrix(a[5], "dx", dev, kBf16, M, K);
  auto* dw = flat<float>(a[6], "dw", dev, at::kFloat, K);
  const Workspace ws(a[7], dw ? fp8rl_add_rmsnorm_bwd_workspace_bytes(M, K) : 0, dy, dev);
  void* stream = stream_of(a[9]);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = fp8rl_add_rmsnorm_bwd((uint16_t*)rg.p, rg.ld, (uint16_t*)rh.p, rh.ld, w,
                                 (uint16_t*)rd.p, rd.ld, eps, M, K, (uint16_t*)rx.p, rx.ld, dw,
                                 ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return status;
}

// topk_ids, E, expert_offsets, row_ids, pos, workspace, dev, stream
int moe_sort(PyObject* const* a) {
  const int dev = (int)integer(a[6]);
  const at::Tensor& ids = tensor(a[0], "topk_ids", dev);
  need_2d(ids, "topk_ids");
  if (ids.scalar_type() != at::kInt && ids.scalar_type() != at::kLong)
    raise(PyExc_TypeError, std::string("topk_ids must be Int or Long, got ") +
                               c10::toString(ids.scalar_type()));
  if (!ids.is_contiguous()) raise(PyExc_ValueError, "topk_ids must be contiguous");
  const int64_t T = ids.size(0), k = ids.size(1), E = integer(a[1]);
  if (E < 0 || E >= int64_t{1} << 31)
    raise(PyExc_ValueError, "E is " + std::to_string(E) + ", out of range");
  // (what does not fit the C types is out of its range as well)
  const int32_t k32 = k > 65 ? 65 : (int32_t)k, e32 = E > 1025 ? 1025 : (int32_t)E;
  auto* off = flat<int32_t>(a[2], "expert_offsets", dev, at::kInt, E + 1);
  auto* rows = flat<int32_t>(a[3], "row_ids", dev, at::kInt, T * k);
  auto* pos = dense<int32_t>(a[4], "pos", dev, at::kInt, T, k);
  const Workspace ws(a[5], fp8rl_moe_sort_workspace_bytes(T, k32, e32), ids, dev);
  void* stream = stream_of(a[7]);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = fp8rl_moe_sort(ids.data_ptr(),
                          ids.scalar_type() == at::kLong ? FP8RL_IDS_I64 : FP8RL_IDS_I32, T, k32,
                          e32, off, rows, pos, ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return status;
}

// pos [T][top_k] of a call: its address and top_k (65, which is refused, for anything wider).
struct Pos {
  const int32_t* p;
  int64_t T, k;
  int32_t k32;
  Pos(PyObject* o, int dev) {
    const at::Tensor& t = tensor(o, "pos", dev);
    need_2d(t, "pos");
    T = t.size(0), k = t.size(1), k32 = k > 65 ? 65 : (int32_t)k;
    p = dense<int32_t>(o, "pos", dev, at::kInt, T, k);
  }
};

// x, pos, out, dev, stream
int moe_dispatch(PyObject* const* a) {
  const int dev = (int)integer(a[3]);
  const at::Tensor &x = tensor(a[0], "x", dev), &out = tensor(a[2], "out", dev);
  need_2d(x, "x");
  need_2d(out, "out");
  const Pos pos(a[1], dev);
  const int64_t N = x.size(1), R = out.size(0);
  const Rows rx = matrix(x, "x", kBf16, pos.T, N), ro = matrix(out, "out", kBf16, R, N);
  void* stream = stream_of(a[4]);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = fp8rl_moe_dispatch((uint16_t*)rx.p, rx.ld, pos.p, pos.T, pos.k32, N, (uint16_t*)ro.p, R,
                              ro.ld, stream);
  Py_END_ALLOW_THREADS
  return status;
}

// y, pos, weights, out, dev, stream
int moe_combine(PyObject* const* a) {
  const int dev = (int)integer(a[4]);
  const at::Tensor &y = tensor(a[0], "y", dev), &out = tensor(a[3], "out", dev);
  need_2d(y, "y");
  const Pos pos(a[1], dev);
  const int64_t R = y.size(0), N = y.size(1);
  const int yt = out_type(y, "y"), ot = out_type(out, "out");
  const Rows ry = matrix(y, "y", y.scalar_type(), R, N);
  auto* w = dense<float>(a[2], "weights", dev, at::kFloat, pos.T, pos.k);
  const Rows ro = matrix(out, "out", out.scalar_type(), pos.T, N);
  void* stream = stream_of(a[5]);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = fp8rl_moe_combine(ry.p, yt, R, ry.ld, pos.p, w, pos.T, pos.k32, N, ro.p, ot, ro.ld,
                             stream);
  Py_END_ALLOW_THREADS
  return status;
}

// dout, y, pos, weights, dy, dweights, dev, stream
int moe_combine_bwd(PyObject* const* a) {
  const int dev = (int)integer(a[6]);
  const at::Tensor &dout = tensor(a[0], "dout", dev), &dy = tensor(a[4], "dy", dev);
  need_2d(dout, "dout");
  need_2d(dy, "dy");
  const Pos pos(a[2], dev);
  const int64_t N = dout.size(1), R = dy.size(0);
  const Rows rg = matrix(dout, "dout", kBf16, pos.T, N);
  const int yt = out_type(dy, "dy");
  const Rows ry = matrix(a[1], "y", dev, dy.scalar_type(), R, N);
  auto* w = dense<float>(a[3], "weights", dev, at::kFloat, pos.T, pos.k);
  const Rows rd = matrix(dy, "dy", dy.scalar_type(), R, N);
  auto* dw = dense<float>(a[5], "dweights", dev, at::kFloat, pos.T, pos.k);
  void* stream = stream_of(a[7]);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = fp8rl_moe_combine_bwd((uint16_t*)rg.p, rg.ld, ry.p, ry.ld, yt, R, pos.p, w, pos.T,
                                 pos.k32, N, rd.p, rd.ld, dw, stream);
  Py_END_ALLOW_THREADS
  return status;
}

// q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_out, interleaved, q_weight,
// k_weight, eps, q_scale, k_scale, v_scale, dev, stream
int rope_kv_append(PyObject* const* a) {
  const int dev = (int)integer(a[16]);
  const at::Tensor &k = tensor(a[1], "k", dev), &kc = tensor(a[6], "k_cache", dev),
                   &vc = tensor(a[7], "v_cache", dev);
  need_2d(k, "k");
  if (kc.dim() != 4)
    raise(PyExc_ValueError, "k_cache must be 4-D: [page][place][head][column]");
  fp8rl_rope_kv_args r{};
  const int64_t pages = kc.size(0), page = kc.size(1), heads = kc.size(2), D = kc.size(3);
  constexpr int64_t kInt = (int64_t{1} << 31) - 1;
  if (page > kInt || heads > kInt || D > kInt)
    raise(PyExc_ValueError, "k_cache has a dimension past 2^31");
  const int64_t T = k.size(0);
  r.T = T;
  r.kv_heads = (int32_t)heads, r.head_dim = (int32_t)D;
  const Rows rk = matrix(k, "k", kBf16, T, heads * D);
  const Rows rv = matrix(tensor(a[2], "v", dev), "v", kBf16, T, heads * D);
  r.k = (uint16_t*)rk.p, r.ld_k = rk.ld, r.v = (uint16_t*)rv.p, r.ld_v = rv.ld;

  const at::ScalarType kind = none(a[14]) ? kBf16 : at::kByte;
  need_type(kc, "k_cache", kind);
  need_type(vc, "v_cache", kind);
  need_shape(vc, "v_cache", kc.sizes());
  if (kc.numel() > 0) {
    if (kc.strides() != vc.strides())
      raise(PyExc_ValueError, "k_cache and v_cache must have the same strides");
    if (D > 1 && kc.stride(3) != 1)
      raise(PyExc_ValueError, "k_cache must have unit stride along its last dimension");
  }
  r.k_cache = kc.data_ptr(), r.v_cache = vc.data_ptr();
  r.num_pages = pages, r.page_size = (int32_t)page;
  // a dimension of one entry has no stride to speak of
  r.page_stride = pages > 1 ? kc.stride(0) : 0;
  r.slot_stride = page > 1 ? kc.stride(1) : D;
  r.head_stride = heads > 1 ? kc.stride(2) : D;

  if (!none(a[0])) {
    const at::Tensor &q = tensor(a[0], "q", dev), &qo = tensor(a[8], "q_out", dev);
    need_2d(q, "q");
    const int64_t cols = q.size(1);
    if (D == 0 || cols % D || cols / D > kInt)
      raise(PyExc_ValueError, "q has " + std::to_string(cols) +
                                  " columns, no multiple of the head width " + std::to_string(D));
    r.q_heads = (int32_t)(cols / D);
    const Rows rq = matrix(q, "q", kBf16, T, cols);
    const Rows ro = matrix(qo, "q_out", none(a[13]) ? kBf16 : at::kByte, T, cols);
    r.q = (uint16_t*)rq.p, r.ld_q = rq.ld, r.q_out = ro.p, r.ld_qo = ro.ld;
  }
  if (!none(a[4])) {
    const at::Tensor& table = tensor(a[4], "cos_sin", dev);
    need_2d(table, "cos_sin");
    if (table.size(1) > kInt) raise(PyExc_ValueError, "cos_sin is too wide");
    r.max_pos = table.size(0), r.rot_dim = (int32_t)table.size(1);
    r.cos_sin = flat<float>(a[4], "cos_sin", dev, at::kFloat, table.numel());
    r.positions = flat<int64_t>(a[3], "positions", dev, at::kLong, T);
  }
  r.slot_mapping = flat<int64_t>(a[5], "slot_mapping", dev, at::kLong, T);
  const int on = PyObject_IsTrue(a[9]);
  if (on < 0) throw Raised{};
  r.interleaved = on;
  r.q_weight = flat<uint16_t>(a[10], "q_weight", dev, kBf16, D);
  r.k_weight = flat<uint16_t>(a[11], "k_weight", dev, kBf16, D);
  r.eps = number(a[12]);
  r.q_scale = flat<float>(a[13], "q_scale", dev, at::kFloat, 1);
  r.k_scale = flat<float>(a[14], "k_scale", dev, at::kFloat, 1);
  r.v_scale = flat<float>(a[15], "v_scale", dev, at::kFloat, 1);
  void* stream = stream_of(a[17]);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = fp8rl_rope_kv_append(&r, stream);
  Py_END_ALLOW_THREADS
  return status;
}

// A function of N arguments as a Python callable: its status, or NULL with the exception set.
template <int (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(F(args));
  } catch (const Raised&) {
    return nullptr;
  } catch (...) {  // torch's own, as its functions raise them (a workspace that does not fit, say)
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

#define FP8RL_CALL(name, n) \
  {#name, (PyCFunction)(void (*)(void))call<name, n>, METH_FASTCALL, nullptr}

PyMethodDef kMethods[] = {FP8RL_CALL(add_rmsnorm_quant, 11),
                          FP8RL_CALL(add_rmsnorm_bwd, 10),
                          FP8RL_CALL(moe_sort, 8),
                          FP8RL_CALL(moe_dispatch, 5),
                          FP8RL_CALL(moe_combine, 6),
                          FP8RL_CALL(moe_combine_bwd, 8),
                          FP8RL_CALL(rope_kv_append, 18),
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods,
                       nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&kModule); }
