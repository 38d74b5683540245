// marshal.cpp -- argument checks of the Python binding for the query/key norm,
// the 8-bit cache, the block-sparse decode and the paged cache, natively: a call checks every
// tensor (type, device, dtype, shape, density) and hands pointers and sizes to
// the C entry point whose address it is given, on the tensors' own device.
// (With the checks in Python a call took 10 to 20 us of the host's time, with
// these about 3, the launch included.)
//
// Every function takes (address, stream handle, arguments...) positionally and
// returns the C status; a tensor that does not fit raises TypeError or
// ValueError before anything is called.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <c10/core/DeviceGuard.h>

#include <cstdint>
#include <initializer_list>
#include <string>

namespace {

struct Raised {};  // a Python exception is set

// The C call, on the tensors' device, while other Python threads may run.  (Its
// arguments are made before: what they raise needs the interpreter's lock.)
template <typename F, typename... A>
int call(c10::Device device, F fn, A... args) {
  const c10::DeviceGuard guard(device);
  PyThreadState* state = PyEval_SaveThread();
  const int code = fn(args...);
  PyEval_RestoreThread(state);
  return code;
}

[[noreturn]] void fail(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Raised{};
}

using Shape = std::initializer_list<int64_t>;

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o))
    fail(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

void typed(const at::Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type)
    fail(PyExc_TypeError, std::string(name) + " must be " + at::toString(type) + ", got " +
                              at::toString(t.scalar_type()));
  if (!t.is_cuda()) fail(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
}

// The tensor that names a call's device and some of its sizes.
const at::Tensor& lead(PyObject* o, const char* name, at::ScalarType type, int dims_a,
                       int dims_b = -1) {
  const at::Tensor& t = tensor(o, name);
  typed(t, name, type);
  if (t.dim() != dims_a && t.dim() != dims_b)
    fail(PyExc_ValueError, std::string(name) + " has " + std::to_string(t.dim()) +
                               " dims, shape " + text(t.sizes()));
  return t;
}

struct Call {
  const char* where;
  c10::Device device;

  void placed(const at::Tensor& t, const char* name, at::IntArrayRef shape) const {
    if (t.sizes() != shape)
      fail(PyExc_ValueError, std::string(where) + ": " + name + " must have shape " +
                                 text(shape) + ", got " + text(t.sizes()));
    if (t.device() != device)
      fail(PyExc_ValueError, std::string(where) + ": " + name + " is on " + t.device().str() +
                                 ", not on " + device.str());
  }
  // A dense tensor of this type and shape; its pointer.
  void* dense(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    const at::Tensor& t = tensor(o, name);
    typed(t, name, type);
    placed(t, name, shape);
    if (!t.is_contiguous())
      fail(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t.data_ptr();
  }
  void* dense(PyObject* o, const char* name, at::ScalarType type, Shape shape) const {
    return dense(o, name, type, at::IntArrayRef(shape.begin(), shape.size()));
  }
  void* optional(PyObject* o, const char* name, at::ScalarType type, Shape shape) const {
    return o == Py_None ? nullptr : dense(o, name, type, shape);
  }
  // [tokens.., heads, D] rows: a token's heads dense, tokens evenly spaced (a
  // view of a fused projection buffer will do); *stride from token to token.
  void* rows(PyObject* o, const char* name, at::IntArrayRef shape, int64_t* stride) const {
    const at::Tensor& t = tensor(o, name);
    typed(t, name, at::kBFloat16);
    placed(t, name, shape);
    const int n = (int)shape.size();
    const int64_t H = shape[n - 2], D = shape[n - 1];
    *stride = H * D;
    if (t.is_contiguous()) return t.data_ptr();
    const auto st = t.strides();
    bool ok = (D == 1 || st[n - 1] == 1) && (H == 1 || st[n - 2] == D);
    if (n == 3) {
      if (shape[0] > 1) *stride = st[0];
    } else {
      const int64_t B = shape[0], S = shape[1];
      if (S > 1) *stride = st[1];
      else if (B > 1) *stride = st[0];
      ok = ok && (B == 1 || S == 1 || st[0] == S * st[1]);
    }
    if (!ok)
      fail(PyExc_ValueError, std::string(where) + ": the heads of a token of " + name +
                                 " must be dense and its tokens evenly spaced, got strides " +
                                 text(st));
    return t.data_ptr();
  }
  void* workspace(PyObject* o, size_t* bytes) const {
    const at::Tensor& t = tensor(o, "workspace");
    if (!t.is_contiguous() || t.device() != device)
      fail(PyExc_ValueError, std::string(where) + ": workspace must be a contiguous tensor on " +
                                 device.str());
    *bytes = t.nbytes();
    return t.data_ptr();
  }
};

int64_t whole(PyObject* o, int64_t lo = INT32_MIN, int64_t hi = INT32_MAX) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v < lo || v > hi) fail(PyExc_ValueError, "an integer argument is out of range");
  return v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return (float)v;
}
void* handle(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised{};
  return p;
}
int narrow(int64_t v) {
  if (v > INT32_MAX) fail(PyExc_ValueError, "a tensor's size is out of range");
  return (int)v;
}
int64_t blocks_of(int64_t L, int64_t block) {
  return block > 0 ? (L + block - 1) / block : 0;
}

constexpr auto kBF16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kI32 = at::kInt;
constexpr auto kE4M3 = at::kFloat8_e4m3fn;

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// fn, stream, q, k, q_weight, k_weight, eps, positions, cos, sin, q_out, k_out
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int {
    const at::Tensor& q = lead(a[2], "q", kBF16, 3);
    const at::Tensor& k = lead(a[3], "k", kBF16, 3);
    const Call c{"attn_qk_norm_rope", q.device()};
    const int64_t N = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = k.size(1);
    int64_t qs, ks, L = INT32_MAX;  // without tables any position will do
    void* qp = c.rows(a[2], "q", {N, Hq, D}, &qs);
    void* kp = c.rows(a[3], "k", {N, Hkv, D}, &ks);
    if ((a[8] == Py_None) != (a[9] == Py_None))
      fail(PyExc_ValueError, "attn_qk_norm_rope: give both cos_table and sin_table, or neither");
    if (a[8] != Py_None) L = lead(a[8], "cos_table", kF32, 2).size(0);
    auto fn = reinterpret_cast<int (*)(const void*, const void*, int64_t, int64_t, const void*,
                                       const void*, float, const void*, const void*, const void*,
                                       int, int, int, int, int, void*, void*, void*)>(handle(a[0]));
    void* wq = c.optional(a[4], "q_weight", kBF16, {D});
    void* wk = c.optional(a[5], "k_weight", kBF16, {D});
    void* pos = c.dense(a[7], "positions", kI32, {N});
    void* cos = c.optional(a[8], "cos_table", kF32, {L, D});
    void* sin = c.optional(a[9], "sin_table", kF32, {L, D});
    void* qo = c.dense(a[10], "q_out", kBF16, {N, Hq, D});
    void* ko = c.dense(a[11], "k_out", kBF16, {N, Hkv, D});
    const float eps = real(a[6]);
    void* stream = handle(a[1]);
    return call(c.device, fn, qp, kp, qs, ks, wq, wk, eps, pos, cos, sin, narrow(N), narrow(Hq),
                narrow(Hkv), narrow(D), narrow(L), qo, ko, stream);
  });
}

// fn, stream, q, k_new, v_new, q_weight, k_weight, eps, positions, k_cache, v_cache, cos, sin, q_out
PyObject* qk_norm_rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> int {
    const at::Tensor& q = lead(a[2], "q", kBF16, 3, 4);
    const at::Tensor& k = lead(a[3], "k_new", kBF16, (int)q.dim());
    const at::Tensor& cache = lead(a[9], "k_cache", kBF16, 4);
    const Call c{"attn_qk_norm_rope_append", q.device()};
    const int dims = (int)q.dim();
    const int64_t B = q.size(0), S = dims == 4 ? q.size(1) : 1, Hq = q.size(dims - 2);
    const int64_t D = q.size(dims - 1), Hkv = k.size(dims - 2), L = cache.size(2);
    const int64_t four_k[4] = {B, S, Hkv, D}, three_k[3] = {B, Hkv, D};
    const at::IntArrayRef new_rows =
        dims == 4 ? at::IntArrayRef(four_k, 4) : at::IntArrayRef(three_k, 3);
    int64_t qs, ks, vs;
    void* qp = c.rows(a[2], "q", q.sizes(), &qs);
    void* kp = c.rows(a[3], "k_new", new_rows, &ks);
    void* vp = c.rows(a[4], "v_new", new_rows, &vs);
    if ((a[11] == Py_None) != (a[12] == Py_None))
      fail(PyExc_ValueError,
           "attn_qk_norm_rope_append: give both cos_table and sin_table, or neither");
    auto fn = reinterpret_cast<int (*)(const void*, const void*, const void*, int64_t, int64_t,
                                       int64_t, const void*, const void*, float, const void*,
                                       const void*, const void*, void*, void*, int, int, int, int,
                                       int, int, void*, void*)>(handle(a[0]));
    void* wq = c.optional(a[5], "q_weight", kBF16, {D});
    void* wk = c.optional(a[6], "k_weight", kBF16, {D});
    void* pos = c.dense(a[8], "positions", kI32, {B});
    void* kc = c.dense(a[9], "k_cache", kBF16, {B, Hkv, L, D});
    void* vc = c.dense(a[10], "v_cache", kBF16, {B, Hkv, L, D});
    void* cos = c.optional(a[11], "cos_table", kF32, {L, D});
    void* sin = c.optional(a[12], "sin_table", kF32, {L, D});
    void* qo = c.dense(a[13], "q_out", kBF16, q.sizes());
    const float eps = real(a[7]);
    void* stream = handle(a[1]);
    return call(c.device, fn, qp, kp, vp, qs, ks, vs, wq, wk, eps, pos, cos, sin, kc, vc, narrow(B),
                narrow(S), narrow(Hq), narrow(Hkv), narrow(D), narrow(L), qo, stream);
  });
}

// fn, stream, k_new, v_new, positions, k_cache, v_cache, k_scale, v_scale, block, k_bounds
PyObject* kv8_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> int {
    const at::Tensor& cache = lead(a[5], "k_cache", kE4M3, 4);
    const at::Tensor& k = lead(a[2], "k_new", kBF16, 3, 4);
    const Call c{"attn_kv8_append", cache.device()};
    const int64_t B = cache.size(0), Hkv = cache.size(1), L = cache.size(2), D = cache.size(3);
    const int64_t S = k.dim() == 4 ? k.size(1) : 1, block = whole(a[9]), nb = blocks_of(L, block);
    const int64_t four[4] = {B, S, Hkv, D}, three[3] = {B, Hkv, D};
    const at::IntArrayRef rows =
        k.dim() == 4 ? at::IntArrayRef(four, 4) : at::IntArrayRef(three, 3);
    auto fn = reinterpret_cast<int (*)(const void*, const void*, int64_t, int64_t, const void*,
                                       void*, void*, void*, void*, void*, int, int, int, int, int,
                                       int, void*)>(handle(a[0]));
    int64_t kst, vst;
    void* kn = c.rows(a[2], "k_new", rows, &kst);
    void* vn = c.rows(a[3], "v_new", rows, &vst);
    void* pos = c.dense(a[4], "positions", kI32, {B});
    void* kc = c.dense(a[5], "k_cache", kE4M3, {B, Hkv, L, D});
    void* vc = c.dense(a[6], "v_cache", kE4M3, {B, Hkv, L, D});
    void* ks = c.dense(a[7], "k_scale", kF32, {B, Hkv, nb});
    void* vs = c.dense(a[8], "v_scale", kF32, {B, Hkv, nb});
    void* bounds = c.optional(a[10], "k_bounds", kBF16, {B, Hkv, nb, 2, D});
    void* stream = handle(a[1]);
    return call(c.device, fn, kn, vn, kst, vst, pos, kc, vc, ks, vs, bounds, narrow(B), narrow(S),
                narrow(Hkv), narrow(L), narrow(D), (int)block, stream);
  });
}

// What the three decode calls share: q, positions, k_cache, v_cache, k_scale,
// v_scale, block at a[2..8], out and workspace at the given places.
struct Decode {
  int64_t B, Hq, Hkv, L, D, nb;
  int block;
  void *q, *pos, *kc, *vc, *ks, *vs, *out, *ws;
  size_t ws_bytes;
  Call c;
  Decode(const char* where, PyObject* const* a, int out_at, int ws_at)
      : c{where, lead(a[2], "q", kBF16, 3).device()} {
    const at::Tensor& t = THPVariable_Unpack(a[2]);
    const at::Tensor& cache = lead(a[4], "k_cache", kE4M3, 4);
    B = t.size(0);
    Hq = t.size(1);
    D = t.size(2);
    Hkv = cache.size(1);
    L = cache.size(2);
    block = (int)whole(a[8]);
    nb = blocks_of(L, block);
    q = c.dense(a[2], "q", kBF16, {B, Hq, D});
    pos = c.dense(a[3], "positions", kI32, {B});
    kc = c.dense(a[4], "k_cache", kE4M3, {B, Hkv, L, D});
    vc = c.dense(a[5], "v_cache", kE4M3, {B, Hkv, L, D});
    ks = c.dense(a[6], "k_scale", kF32, {B, Hkv, nb});
    vs = c.dense(a[7], "v_scale", kF32, {B, Hkv, nb});
    out = c.dense(a[out_at], "out", kBF16, {B, Hq, D});
    ws = c.workspace(a[ws_at], &ws_bytes);
  }
};

// fn, stream, q, positions, k_cache, v_cache, k_scale, v_scale, block, scale, out, workspace
PyObject* decode_kv8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int {
    const Decode d("attn_decode_step_kv8", a, 10, 11);
    auto fn = reinterpret_cast<int (*)(const void*, const void*, const void*, const void*,
                                       const void*, const void*, int, int, int, int, int, int,
                                       float, void*, void*, size_t, void*)>(handle(a[0]));
    const float scale = real(a[9]);
    void* stream = handle(a[1]);
    return call(d.c.device, fn, d.q, d.pos, d.kc, d.vc, d.ks, d.vs, narrow(d.B), narrow(d.Hq),
                narrow(d.Hkv), narrow(d.L), narrow(d.D), d.block, scale, d.out, d.ws, d.ws_bytes,
                stream);
  });
}

// fn, stream, q, positions, k_cache, v_cache, k_scale, v_scale, block, block_index, scale, out,
// workspace
PyObject* decode_kv8_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> int {
    const Decode d("attn_decode_step_kv8_blocks", a, 11, 12);
    const int64_t count = lead(a[9], "block_index", kI32, 3).size(2);
    void* index = d.c.dense(a[9], "block_index", kI32, {d.B, d.Hkv, count});
    auto fn = reinterpret_cast<int (*)(const void*, const void*, const void*, const void*,
                                       const void*, const void*, const void*, int, int, int, int,
                                       int, int, int, float, void*, void*, size_t, void*)>(
        handle(a[0]));
    const float scale = real(a[10]);
    void* stream = handle(a[1]);
    return call(d.c.device, fn, d.q, d.pos, d.kc, d.vc, d.ks, d.vs, index, narrow(count),
                narrow(d.B), narrow(d.Hq), narrow(d.Hkv), narrow(d.L), narrow(d.D), d.block, scale,
                d.out, d.ws, d.ws_bytes, stream);
  });
}

// fn, stream, q, positions, k_cache, v_cache, k_scale, v_scale, block, k_bounds, count, first,
// recent, scale, out, workspace
PyObject* decode_kv8_sparse(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> int {
    const Decode d("attn_decode_step_kv8_sparse", a, 14, 15);
    void* bounds = d.c.dense(a[9], "k_bounds", kBF16, {d.B, d.Hkv, d.nb, 2, d.D});
    auto fn = reinterpret_cast<int (*)(const void*, const void*, const void*, const void*,
                                       const void*, const void*, const void*, int, int, int, int,
                                       int, int, int, int, int, float, void*, void*, size_t,
                                       void*)>(handle(a[0]));
    const int count = (int)whole(a[10]), first = (int)whole(a[11]), recent = (int)whole(a[12]);
    const float scale = real(a[13]);
    void* stream = handle(a[1]);
    return call(d.c.device, fn, d.q, d.pos, d.kc, d.vc, d.ks, d.vs, bounds, count, first, recent,
                narrow(d.B), narrow(d.Hq), narrow(d.Hkv), narrow(d.L), narrow(d.D), d.block, scale,
                d.out, d.ws, d.ws_bytes, stream);
  });
}

// fn, stream, q, positions, k_bounds, L, block, out
PyObject* block_scores(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> int {
    const at::Tensor& q = lead(a[2], "q", kBF16, 3);
    const at::Tensor& bounds = lead(a[4], "k_bounds", kBF16, 5);
    const Call c{"attn_block_scores", q.device()};
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = bounds.size(1);
    const int64_t L = whole(a[5]), block = whole(a[6]), nb = blocks_of(L, block);
    auto fn = reinterpret_cast<int (*)(const void*, const void*, const void*, int, int, int, int,
                                       int, int, void*, void*)>(handle(a[0]));
    void* qp = c.dense(a[2], "q", kBF16, {B, Hq, D});
    void* pos = c.dense(a[3], "positions", kI32, {B});
    void* bp = c.dense(a[4], "k_bounds", kBF16, {B, Hkv, nb, 2, D});
    void* out = c.dense(a[7], "out", kF32, {B, Hkv, nb});
    void* stream = handle(a[1]);
    return call(c.device, fn, qp, pos, bp, narrow(B), narrow(Hq), narrow(Hkv), (int)L, narrow(D),
                (int)block, out, stream);
  });
}

// fn, stream, scores, positions, L, block, count, first, recent, out
PyObject* block_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> int {
    const at::Tensor& s = lead(a[2], "scores", kF32, 3);
    const Call c{"attn_block_select", s.device()};
    const int64_t B = s.size(0), Hkv = s.size(1), L = whole(a[4]), block = whole(a[5]);
    const int64_t nb = blocks_of(L, block), count = whole(a[6]);
    const int first = (int)whole(a[7]), recent = (int)whole(a[8]);
    auto fn = reinterpret_cast<int (*)(const void*, const void*, int, int, int, int, int, int, int,
                                       void*, void*)>(handle(a[0]));
    void* sp = c.dense(a[2], "scores", kF32, {B, Hkv, nb});
    void* pos = c.dense(a[3], "positions", kI32, {B});
    void* out = c.dense(a[9], "out", kI32, {B, Hkv, count});
    void* stream = handle(a[1]);
    return call(c.device, fn, sp, pos, narrow(B), narrow(Hkv), (int)L, (int)block, (int)count,
                first, recent, out, stream);
  });
}

// A pool: k_pages and v_pages [P, Hkv, page, D] with the same strides, D dense.
struct Pool {
  int64_t P, Hkv, page, D, page_stride, head_stride, row_stride;
  void *k, *v;
  Pool(const Call& c, PyObject* ko, PyObject* vo) {
    const at::Tensor& t = lead(ko, "k_pages", kBF16, 4);
    const at::Tensor& u = lead(vo, "v_pages", kBF16, 4);
    P = t.size(0);
    Hkv = t.size(1);
    page = t.size(2);
    D = t.size(3);
    c.placed(t, "k_pages", t.sizes());
    c.placed(u, "v_pages", t.sizes());
    const auto st = t.strides(), su = u.strides();
    bool ok = D <= 1 || (st[3] == 1 && su[3] == 1);
    for (int i = 0; i < 3; ++i) ok = ok && (t.size(i) <= 1 || st[i] == su[i]);
    if (!ok)
      fail(PyExc_ValueError, std::string(c.where) +
                                 ": the rows of k_pages and v_pages must be dense and their "
                                 "strides alike, got " + text(st) + " and " + text(su));
    page_stride = P > 1 ? st[0] : Hkv * page * D;
    head_stride = Hkv > 1 ? st[1] : page * D;
    row_stride = page > 1 ? st[2] : D;
    k = t.data_ptr();
    v = u.data_ptr();
  }
};

// fn, stream, k_new, v_new, positions, lengths, page_table, k_pages, v_pages
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> int {
    const at::Tensor& k = lead(a[2], "k_new", kBF16, 3, 4);
    const Call c{"attn_paged_append", k.device()};
    const Pool pool(c, a[7], a[8]);
    const int64_t B = k.size(0), S = k.dim() == 4 ? k.size(1) : 1;
    const int64_t M = lead(a[6], "page_table", kI32, 2).size(1);
    const int64_t four[4] = {B, S, pool.Hkv, pool.D}, three[3] = {B, pool.Hkv, pool.D};
    const at::IntArrayRef rows =
        k.dim() == 4 ? at::IntArrayRef(four, 4) : at::IntArrayRef(three, 3);
    auto fn = reinterpret_cast<int (*)(const void*, const void*, int64_t, int64_t, const void*,
                                       const void*, const void*, void*, void*, int64_t, int64_t,
                                       int64_t, int, int, int, int, int, int, int, void*)>(
        handle(a[0]));
    int64_t kst, vst;
    void* kn = c.rows(a[2], "k_new", rows, &kst);
    void* vn = c.rows(a[3], "v_new", rows, &vst);
    void* pos = c.dense(a[4], "positions", kI32, {B});
    void* len = c.optional(a[5], "lengths", kI32, {B});
    void* table = c.dense(a[6], "page_table", kI32, {B, M});
    void* stream = handle(a[1]);
    return call(c.device, fn, kn, vn, kst, vst, pos, len, table, pool.k, pool.v, pool.page_stride,
                pool.head_stride, pool.row_stride, narrow(B), narrow(S), narrow(pool.Hkv),
                narrow(pool.D), narrow(pool.P), narrow(pool.page), narrow(M), stream);
  });
}

// fn, stream, q, positions, lengths, page_table, k_pages, v_pages, scale, out, workspace
PyObject* decode_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> int {
    const at::Tensor& q = lead(a[2], "q", kBF16, 3, 4);
    const Call c{"attn_decode_step_paged", q.device()};
    const Pool pool(c, a[6], a[7]);
    const int dims = (int)q.dim();
    const int64_t B = q.size(0), S = dims == 4 ? q.size(1) : 1, Hq = q.size(dims - 2);
    const int64_t M = lead(a[5], "page_table", kI32, 2).size(1);
    const int64_t four[4] = {B, S, Hq, pool.D}, three[3] = {B, Hq, pool.D};
    const at::IntArrayRef rows = dims == 4 ? at::IntArrayRef(four, 4) : at::IntArrayRef(three, 3);
    auto fn = reinterpret_cast<int (*)(const void*, const void*, const void*, const void*,
                                       const void*, const void*, int64_t, int64_t, int64_t, int,
                                       int, int, int, int, int, int, int, float, void*, void*,
                                       size_t, void*)>(handle(a[0]));
    void* qp = c.dense(a[2], "q", kBF16, rows);
    void* pos = c.dense(a[3], "positions", kI32, {B});
    void* len = c.optional(a[4], "lengths", kI32, {B});
    void* table = c.dense(a[5], "page_table", kI32, {B, M});
    void* out = c.dense(a[9], "out", kBF16, rows);
    size_t ws_bytes;
    void* ws = c.workspace(a[10], &ws_bytes);
    const float scale = real(a[8]);
    void* stream = handle(a[1]);
    return call(c.device, fn, qp, pos, len, table, pool.k, pool.v, pool.page_stride,
                pool.head_stride, pool.row_stride, narrow(B), narrow(S), narrow(Hq),
                narrow(pool.Hkv), narrow(pool.D), narrow(pool.P), narrow(pool.page), narrow(M),
                scale, out, ws, ws_bytes, stream);
  });
}

// fn, stream, page_table, page_refs, positions, lengths, k_pages, v_pages, tokens, taken, workspace
PyObject* pages_reserve(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> int {
    const at::Tensor& t = lead(a[2], "page_table", kI32, 2);
    const Call c{"attn_pages_reserve", t.device()};
    const Pool pool(c, a[6], a[7]);
    const int64_t B = t.size(0), M = t.size(1), S = whole(a[8]);
    auto fn = reinterpret_cast<int (*)(void*, void*, const void*, const void*, void*, void*,
                                       int64_t, int64_t, int64_t, int, int, int, int, int, int,
                                       int, void*, void*, size_t, void*)>(handle(a[0]));
    void* table = c.dense(a[2], "page_table", kI32, {B, M});
    void* refs = c.dense(a[3], "page_refs", kI32, {pool.P});
    void* pos = c.dense(a[4], "positions", kI32, {B});
    void* len = c.optional(a[5], "lengths", kI32, {B});
    void* taken = c.dense(a[9], "taken", kI32, {B});
    size_t ws_bytes;
    void* ws = c.workspace(a[10], &ws_bytes);
    void* stream = handle(a[1]);
    return call(c.device, fn, table, refs, pos, len, pool.k, pool.v, pool.page_stride,
                pool.head_stride, pool.row_stride, narrow(B), (int)S, narrow(pool.Hkv),
                narrow(pool.D), narrow(pool.P), narrow(pool.page), narrow(M), taken, ws, ws_bytes,
                stream);
  });
}

// fn, stream, page_table, page_refs, page, parents, lengths, workspace
PyObject* pages_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> int {
    const at::Tensor& t = lead(a[2], "page_table", kI32, 2);
    const Call c{"attn_pages_fork", t.device()};
    const int64_t B = t.size(0), M = t.size(1);
    const int64_t P = lead(a[3], "page_refs", kI32, 1).size(0);
    auto fn = reinterpret_cast<int (*)(void*, void*, const void*, const void*, int, int, int, int,
                                       void*, size_t, void*)>(handle(a[0]));
    void* table = c.dense(a[2], "page_table", kI32, {B, M});
    void* refs = c.dense(a[3], "page_refs", kI32, {P});
    const int page = (int)whole(a[4]);
    void* parents = c.optional(a[5], "parents", kI32, {B});
    void* len = c.optional(a[6], "lengths", kI32, {B});
    size_t ws_bytes;
    void* ws = c.workspace(a[7], &ws_bytes);
    void* stream = handle(a[1]);
    return call(c.device, fn, table, refs, parents, len, narrow(B), narrow(M), narrow(P), page, ws,
                ws_bytes, stream);
  });
}

// fn, stream, page_table, page_refs, k_pages, v_pages, page_map, workspace
PyObject* pages_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> int {
    const at::Tensor& t = lead(a[2], "page_table", kI32, 2);
    const Call c{"attn_pages_compact", t.device()};
    const Pool pool(c, a[4], a[5]);
    const int64_t B = t.size(0), M = t.size(1);
    auto fn = reinterpret_cast<int (*)(void*, void*, void*, void*, int64_t, int64_t, int64_t, int,
                                       int, int, int, int, int, void*, void*, size_t, void*)>(
        handle(a[0]));
    void* table = c.dense(a[2], "page_table", kI32, {B, M});
    void* refs = c.dense(a[3], "page_refs", kI32, {pool.P});
    void* map = c.dense(a[6], "page_map", kI32, {pool.P});
    size_t ws_bytes;
    void* ws = c.workspace(a[7], &ws_bytes);
    void* stream = handle(a[1]);
    return call(c.device, fn, table, refs, pool.k, pool.v, pool.page_stride, pool.head_stride,
                pool.row_stride, narrow(B), narrow(M), narrow(pool.Hkv), narrow(pool.D),
                narrow(pool.P), narrow(pool.page), map, ws, ws_bytes, stream);
  });
}

#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, ""}
PyMethodDef kMethods[] = {ENTRY(qk_norm_rope),      ENTRY(qk_norm_rope_append),
                          ENTRY(kv8_append),        ENTRY(decode_kv8),
                          ENTRY(decode_kv8_blocks), ENTRY(decode_kv8_sparse),
                          ENTRY(block_scores),      ENTRY(block_select),
                          ENTRY(paged_append),      ENTRY(decode_paged),
                          ENTRY(pages_reserve),     ENTRY(pages_fork),
                          ENTRY(pages_compact),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_gqa_marshal",
                       "Argument checks of the 8-bit and the paged cache's binding.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gqa_marshal(void) { return PyModule_Create(&kModule); }
