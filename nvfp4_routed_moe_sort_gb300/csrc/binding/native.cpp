// Python module _native: the calls of the operators around the routed experts on torch tensors.
//
// These operators run for microseconds at decode sizes. Checked in Python and marshalled by
// ctypes, a call took 7 to 11 us of host time on a GB300 host, more than the kernel; here it
// takes about 3, of which the launch is 1.5. Each function checks what the C entry point cannot see
// (types, shapes, strides, and that every tensor lies on the current device), then makes the one C call on
// torch's current stream. A wrong tensor raises ValueError, a refusal by the library its MoEError.
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "moe_nvfp4.h"

namespace {

struct Raised {};  // a Python exception is set

PyObject* moe_error = nullptr;

[[noreturn]] void refuse(const char* what, const char* need) {
  PyErr_Format(PyExc_ValueError, "%s must be %s", what, need);
  throw Raised();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(what, "a torch tensor");
  return THPVariable_Unpack(o);
}
const at::Tensor* maybe(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }
void* pointer(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

bool is(const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape) {
  return t.scalar_type() == type && t.is_cuda() && t.sizes() == at::IntArrayRef(shape.begin(), shape.size());
}
void dense(const at::Tensor* t, at::ScalarType type, std::initializer_list<int64_t> shape, const char* what, const char* need) {
  if (t && !(is(*t, type, shape) && t->is_contiguous())) refuse(what, need);
}
// rows whose values lie side by side
void rows(const at::Tensor* t, at::ScalarType type, int64_t n, int64_t width, const char* what, const char* need) {
  if (t && !(is(*t, type, {n, width}) && (t->stride(1) == 1 || width == 1))) refuse(what, need);
}
// values between rows: a single row's stride says nothing
int64_t ld(const at::Tensor& t, int64_t width) { return t.size(0) > 1 ? t.stride(0) : width; }

int32_t int32_size(int64_t n, const char* what) {
  if (n > INT32_MAX) refuse(what, "of fewer than 2^31 values along each dimension");
  return static_cast<int32_t>(n);
}
long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return static_cast<float>(v);
}

// a launch runs on the current device: pointers into another one's memory are none there
void check_device(const char* what, long device, long current) {
  if (device == current) return;
  PyErr_Format(PyExc_ValueError, "%s is on cuda:%ld, the call would run on cuda:%ld", what, device, current);
  throw Raised();
}
struct Named {
  const at::Tensor* t;  // may be null
  const char* what;
};
void on_device(std::initializer_list<Named> tensors, long current) {
  for (const Named& n : tensors)
    if (n.t) check_device(n.what, n.t->device().index(), current);
}
// checks them, and gives torch's current stream on that device; the first one is never null
moe_stream_t stream_of(std::initializer_list<Named> tensors) {
  const c10::DeviceIndex device = tensors.begin()->t->device().index();
  on_device(tensors, device);
  check_device(tensors.begin()->what, device, c10::cuda::current_device());
  return c10::cuda::getCurrentCUDAStream(device).stream();
}

PyObject* done(moe_status_t st, const char* call) {
  if (st == MOE_OK) Py_RETURN_NONE;
  PyErr_Format(moe_error ? moe_error : PyExc_RuntimeError, "%s: %s", call, moe_status_string(st));
  throw Raised();
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd given", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kE4m3 = at::kFloat8_e4m3fn;

// (error class): what a refusal by the library raises
PyObject* set_error(PyObject* const* a) {
  Py_INCREF(a[0]);
  Py_XSETREF(moe_error, a[0]);
  Py_RETURN_NONE;
}

// () -> what no other stream of this process is ever called, unlike its handle
PyObject* stream_id(PyObject* const*) {
  unsigned long long id = 0;
  if (cudaStreamGetId(c10::cuda::getCurrentCUDAStream().stream(), &id) != cudaSuccess) {
    PyErr_SetString(PyExc_RuntimeError, "cudaStreamGetId failed");
    throw Raised();
  }
  return PyLong_FromUnsignedLongLong(id);
}

// (what, device, current device): refuses a tensor `what` of another device
PyObject* refuse_device(PyObject* const* a) {
  const char* what = PyUnicode_AsUTF8(a[0]);
  if (!what) throw Raised();
  check_device(what, integer(a[1]), integer(a[2]));
  Py_RETURN_NONE;
}

// (x, weight, residual, eps, fp8_scale, y, residual_out, y8, y8_scale)
PyObject* add_rms_norm(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  if (x.dim() != 2) refuse("x", "[M, H]");
  const int64_t M = x.size(0), H = x.size(1);
  rows(&x, kBf16, M, H, "x", "bf16 rows on the GPU, their values side by side");
  const at::Tensor& w = tensor(a[1], "weight");
  dense(&w, kBf16, {H}, "weight", "contiguous bf16 [H] on the GPU");
  const at::Tensor* r = maybe(a[2], "residual");
  rows(r, kBf16, M, H, "residual", "bf16 rows on the GPU of x's shape, their values side by side");
  const long fp8 = integer(a[4]);
  const int64_t groups = fp8 == MOE_FP8_PER_GROUP ? (H + MOE_FP8_GROUP - 1) / MOE_FP8_GROUP : 1;
  const at::Tensor *y = maybe(a[5], "y"), *ro = maybe(a[6], "residual_out"), *y8 = maybe(a[7], "y8"), *sc = maybe(a[8], "scales");
  dense(y, kBf16, {M, H}, "the output", "contiguous bf16 [M, H] on the GPU");
  dense(ro, kBf16, {M, H}, "the residual's output", "contiguous bf16 [M, H] on the GPU");
  dense(y8, kE4m3, {M, H}, "the FP8 output", "contiguous float8_e4m3fn [M, H] on the GPU");
  dense(sc, at::kFloat, {M, groups}, "the scales", "contiguous float32 [M, 1] or [M, ceil(H / 128)] on the GPU");
  if ((y8 != nullptr) != (fp8 != MOE_FP8_NONE) || (sc != nullptr) != (fp8 != MOE_FP8_NONE))
    refuse("the FP8 output and its scales", "given with fp8, and only then");
  const moe_stream_t stream =
      stream_of({{&x, "x"}, {&w, "weight"}, {r, "residual"}, {y, "the output"}, {ro, "the residual's output"},
                 {y8, "the FP8 output"}, {sc, "the scales"}});
  return done(moe_add_rmsnorm(static_cast<const uint16_t*>(x.data_ptr()), ld(x, H), static_cast<const uint16_t*>(pointer(r)),
                              r ? ld(*r, H) : H, static_cast<const uint16_t*>(w.data_ptr()), int32_size(M, "x"),
                              int32_size(H, "x"), real(a[3]), static_cast<int32_t>(fp8), static_cast<uint16_t*>(pointer(y)),
                              static_cast<uint16_t*>(pointer(ro)), static_cast<uint8_t*>(pointer(y8)),
                              static_cast<float*>(pointer(sc)), stream),
              "moe_add_rmsnorm");
}

// (x, x_scale, w, w_sf, alpha, activation, out)
PyObject* fp4_linear(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[2], "w"), &sf = tensor(a[3], "w_sf"), &alpha = tensor(a[4], "alpha");
  const at::Tensor* xs = maybe(a[1], "x_scale");
  if (x.dim() != 2 || w.dim() != 2) refuse("x and w", "[M, K] and [N, K/2]");
  const int64_t M = x.size(0), K = x.size(1), N = w.size(0);
  dense(&w, at::kByte, {N, K / 2}, "w", "contiguous uint8 [N, K/2] on the GPU");
  dense(&sf, at::kByte, {N, K / 16}, "w_sf", "contiguous uint8 [N, K/16] on the GPU");
  if (alpha.scalar_type() != at::kFloat || alpha.numel() != 1 || !alpha.is_cuda()) refuse("alpha", "one float32 value on the GPU");
  int32_t mode = MOE_FP8_NONE;
  if (!xs) {
    rows(&x, kBf16, M, K, "x without x_scale", "bf16 rows on the GPU, their values side by side");
  } else {
    rows(&x, kE4m3, M, K, "x with x_scale", "float8_e4m3fn rows on the GPU, their values side by side");
    const bool one = xs->dim() == 2 && xs->size(1) == 1;
    mode = one ? MOE_FP8_PER_TOKEN : MOE_FP8_PER_GROUP;
    dense(xs, at::kFloat, {M, one ? 1 : (K + MOE_FP8_GROUP - 1) / MOE_FP8_GROUP}, "x_scale",
          "contiguous float32 [M, 1] or [M, ceil(K / 128)] on the GPU");
  }
  const long act = integer(a[5]);
  const bool gated = act == MOE_ACT_SWIGLU || act == MOE_ACT_GEGLU;
  if (gated && N % 2) refuse("w", "of an even number of rows for a gated activation");
  const at::Tensor& out = tensor(a[6], "out");
  dense(&out, kBf16, {M, gated ? N / 2 : N}, "out", "contiguous bf16 [M, N] (gated: [M, N/2]) on the GPU");
  const moe_stream_t stream =
      stream_of({{&x, "x"}, {xs, "x_scale"}, {&w, "w"}, {&sf, "w_sf"}, {&alpha, "alpha"}, {&out, "out"}});
  // one of several matrices' scalars lies where it lies; the C entry wants 16-byte alignment, and gets a copy
  const at::Tensor scalar = reinterpret_cast<uintptr_t>(alpha.data_ptr()) % 16 ? alpha.clone() : alpha;
  return done(moe_linear_fp4(x.data_ptr(), ld(x, K), static_cast<const float*>(pointer(xs)), mode, int32_size(M, "x"),
                             int32_size(K, "x"), static_cast<const uint8_t*>(w.data_ptr()),
                             static_cast<const uint8_t*>(sf.data_ptr()), static_cast<const float*>(scalar.data_ptr()),
                             int32_size(N, "w"), static_cast<int32_t>(act), static_cast<uint16_t*>(out.data_ptr()), stream),
              "moe_linear_fp4");
}

// A cache as kv_cache() checked it; the NVFP4KVCache object that holds it also holds the tensors.
struct Cache {
  moe_kv_cache_t c;
  int32_t* status;
  long device;
};
const char* const kCapsule = "moe_kv_cache";

void drop_cache(PyObject* o) { delete static_cast<Cache*>(PyCapsule_GetPointer(o, kCapsule)); }
const Cache& cache_of(PyObject* o) {
  const auto* c = static_cast<const Cache*>(PyCapsule_GetPointer(o, kCapsule));
  if (!c) throw Raised();
  return *c;
}

// (k, k_sf, v, v_sf, k_scale, v_scale, dev_status)
PyObject* kv_cache(PyObject* const* a) {
  const at::Tensor &k = tensor(a[0], "k"), &ks = tensor(a[1], "k_sf"), &v = tensor(a[2], "v"), &vs = tensor(a[3], "v_sf");
  const at::Tensor* status = maybe(a[6], "dev_status");
  if (k.dim() != 4) refuse("k", "[num_pages, num_kv_heads, page_size, head_dim/2]");
  const int64_t P = k.size(0), H = k.size(1), S = k.size(2), half = k.size(3), sf = half / 8;
  const int64_t d[3] = {S * half, half, 1}, f[3] = {S * sf, sf, 1};
  const bool ok = is(k, at::kByte, {P, H, S, half}) && is(v, at::kByte, {P, H, S, half}) && is(ks, at::kByte, {P, H, S, sf}) &&
                  is(vs, at::kByte, {P, H, S, sf}) && k.strides() == v.strides() && ks.strides() == vs.strides() &&
                  k.strides().slice(1) == at::IntArrayRef(d, 3) && ks.strides().slice(1) == at::IntArrayRef(f, 3);
  if (!ok)
    refuse("k, v and k_sf, v_sf", "uint8 [num_pages, num_kv_heads, page_size, head_dim/2] and [..., head_dim/16] on the GPU, each "
                                  "page contiguous, with the same strides for keys and values");
  if (status && (status->scalar_type() != at::kInt || !status->is_cuda() || status->numel() < 1))
    refuse("dev_status", "int32 on the GPU");
  const long device = k.device().index();
  on_device({{&ks, "k_sf"}, {&v, "v"}, {&vs, "v_sf"}, {status, "dev_status"}}, device);
  const auto p = [](const at::Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); };
  auto* c = new Cache{{p(k), p(ks), p(v), p(vs), int32_size(P, "k"), int32_size(S, "k"), int32_size(H, "k"),
                       int32_size(2 * half, "k"), k.stride(0), ks.stride(0), real(a[4]), real(a[5])},
                      static_cast<int32_t*>(pointer(status)), device};
  PyObject* o = PyCapsule_New(c, kCapsule, drop_cache);
  if (!o) {
    delete c;
    throw Raised();
  }
  return o;
}

// (cache, k_new, v_new, slots, k_seen, v_seen)
PyObject* kv_append(PyObject* const* a) {
  const Cache& c = cache_of(a[0]);
  const at::Tensor &k = tensor(a[1], "k_new"), &v = tensor(a[2], "v_new"), &slots = tensor(a[3], "slots");
  const int64_t H = c.c.num_kv_heads, D = c.c.head_dim, N = k.dim() == 3 ? k.size(0) : -1;
  for (const at::Tensor* t : {&k, &v})
    if (!is(*t, kBf16, {N, H, D}) || t->stride(2) != 1 || (H > 1 && t->stride(1) != D))
      refuse(t == &k ? "k_new" : "v_new", "bf16 [N, num_kv_heads, head_dim] on the GPU, each token's values contiguous");
  dense(&slots, at::kLong, {N}, "slots", "contiguous int64 [N] on the GPU");
  const at::Tensor *ks = maybe(a[4], "seen[0]"), *vs = maybe(a[5], "seen[1]");
  dense(ks, kBf16, {N, H, D}, "seen[0]", "contiguous bf16 of k_new's shape on the GPU");
  dense(vs, kBf16, {N, H, D}, "seen[1]", "contiguous bf16 of k_new's shape on the GPU");
  const moe_stream_t stream =
      stream_of({{&k, "k_new"}, {&v, "v_new"}, {&slots, "slots"}, {ks, "seen[0]"}, {vs, "seen[1]"}});
  check_device("the cache", c.device, k.device().index());
  return done(moe_kv_append(&c.c, static_cast<const uint16_t*>(k.data_ptr()), ld(k, H * D),
                            static_cast<const uint16_t*>(v.data_ptr()), ld(v, H * D),
                            static_cast<const int64_t*>(slots.data_ptr()), int32_size(N, "k_new"),
                            static_cast<uint16_t*>(pointer(ks)), static_cast<uint16_t*>(pointer(vs)), c.status, stream),
              "moe_kv_append");
}

struct Queries {
  int32_t batch, q_len, heads, pages;
  int64_t ld_q, ld_table;
};
Queries queries(const Cache& c, const at::Tensor& q, const at::Tensor& table) {
  const int64_t D = c.c.head_dim;
  if (q.dim() != 4 || q.scalar_type() != kBf16 || !q.is_cuda() || q.size(3) != D)
    refuse("q", "bf16 [batch, q_len, num_q_heads, head_dim] on the GPU");
  const int64_t B = q.size(0), T = q.size(1), H = q.size(2);
  const int64_t step = T > 1 ? q.stride(1) : B > 1 ? q.stride(0) : H * D;
  if (q.stride(3) != 1 || (H > 1 && q.stride(2) != D) || (B > 1 && q.stride(0) != T * step))
    refuse("q", "of contiguous rows [num_q_heads, head_dim] that are evenly spaced");
  if (table.dim() != 2 || !is(table, at::kInt, {B, table.size(1)}) || (table.stride(1) != 1 && table.size(1) > 1))
    refuse("page_table", "int32 [batch, max_pages] on the GPU, a sequence's pages side by side");
  return {int32_size(B, "q"), int32_size(T, "q"), int32_size(H, "q"), int32_size(table.size(1), "page_table"), step,
          ld(table, table.size(1))};
}

// (cache, q, page_table) -> bytes
PyObject* kv_workspace(PyObject* const* a) {
  const Cache& c = cache_of(a[0]);
  const Queries n = queries(c, tensor(a[1], "q"), tensor(a[2], "page_table"));
  return PyLong_FromSize_t(moe_kv_attend_workspace_bytes(&c.c, n.batch, n.q_len, n.heads, n.pages));
}

// (cache, q, page_table, seq_lens, softmax_scale, out, lse, workspace)
PyObject* kv_attend(PyObject* const* a) {
  const Cache& c = cache_of(a[0]);
  const at::Tensor &q = tensor(a[1], "q"), &table = tensor(a[2], "page_table"), &lens = tensor(a[3], "seq_lens");
  const Queries n = queries(c, q, table);
  dense(&lens, at::kInt, {n.batch}, "seq_lens", "contiguous int32 [batch] on the GPU");
  const at::Tensor &out = tensor(a[5], "out"), *lse = maybe(a[6], "lse"), *ws = maybe(a[7], "workspace");
  dense(&out, kBf16, {n.batch, n.q_len, n.heads, c.c.head_dim}, "out", "contiguous bf16 of q's shape on the GPU");
  dense(lse, at::kFloat, {n.batch, n.q_len, n.heads}, "lse", "contiguous float32 [batch, q_len, num_q_heads] on the GPU");
  if (ws && !(ws->is_cuda() && ws->is_contiguous())) refuse("workspace", "contiguous on the GPU");
  const moe_stream_t stream =
      stream_of({{&q, "q"}, {&table, "page_table"}, {&lens, "seq_lens"}, {&out, "out"}, {lse, "lse"}, {ws, "workspace"}});
  check_device("the cache", c.device, q.device().index());
  return done(moe_kv_attend(&c.c, static_cast<const uint16_t*>(q.data_ptr()), n.ld_q, n.batch, n.q_len, n.heads,
                            static_cast<const int32_t*>(table.data_ptr()), n.ld_table, n.pages,
                            static_cast<const int32_t*>(lens.data_ptr()), real(a[4]), static_cast<uint16_t*>(out.data_ptr()),
                            static_cast<float*>(pointer(lse)), pointer(ws), ws ? ws->nbytes() : 0, c.status, stream),
              "moe_kv_attend");
}

int32_t* status_word(const at::Tensor* t) {
  if (t && (t->scalar_type() != at::kInt || !t->is_cuda() || t->numel() < 1)) refuse("dev_status", "int32 on the GPU");
  return static_cast<int32_t*>(pointer(t));
}

// (x, block_rows, y, scale)
PyObject* quantize_fp8(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  if (x.dim() != 2) refuse("x", "[M, K]");
  const int64_t M = x.size(0), K = x.size(1);
  rows(&x, kBf16, M, K, "x", "bf16 rows on the GPU, their values side by side");
  const long block = integer(a[1]);
  if (block != 1 && block != MOE_FP8_GROUP) refuse("rows", "1 or 128");
  const at::Tensor &y = tensor(a[2], "y"), &sc = tensor(a[3], "the scales");
  dense(&y, kE4m3, {M, K}, "y", "contiguous float8_e4m3fn [M, K] on the GPU");
  dense(&sc, at::kFloat, {(M + block - 1) / block, (K + MOE_FP8_GROUP - 1) / MOE_FP8_GROUP}, "the scales",
        "contiguous float32 [ceil(M / rows), ceil(K / 128)] on the GPU");
  const moe_stream_t stream = stream_of({{&x, "x"}, {&y, "y"}, {&sc, "the scales"}});
  return done(moe_quantize_fp8(static_cast<const uint16_t*>(x.data_ptr()), ld(x, K), int32_size(M, "x"), int32_size(K, "x"),
                               static_cast<int32_t>(block), static_cast<uint8_t*>(y.data_ptr()),
                               static_cast<float*>(sc.data_ptr()), stream),
              "moe_quantize_fp8");
}

// (x, x_scale, w, w_scale, activation, out, dev_status)
PyObject* fp8_linear(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "x"), &xs = tensor(a[1], "x_scale"), &w = tensor(a[2], "w"), &ws = tensor(a[3], "w_scale");
  if (x.dim() != 2 || w.dim() != 2) refuse("x and w", "[M, K] and [N, K]");
  const int64_t M = x.size(0), K = x.size(1), N = w.size(0), groups = (K + MOE_FP8_GROUP - 1) / MOE_FP8_GROUP;
  rows(&x, kE4m3, M, K, "x", "float8_e4m3fn rows on the GPU, their values side by side");
  const bool one = xs.dim() == 2 && xs.size(1) == 1;
  dense(&xs, at::kFloat, {M, one ? 1 : groups}, "x_scale", "contiguous float32 [M, 1] or [M, ceil(K / 128)] on the GPU");
  dense(&w, kE4m3, {N, K}, "w", "contiguous float8_e4m3fn [N, K] on the GPU");
  dense(&ws, at::kFloat, {(N + MOE_FP8_GROUP - 1) / MOE_FP8_GROUP, groups}, "w_scale",
        "contiguous float32 [ceil(N / 128), ceil(K / 128)] on the GPU");
  const long act = integer(a[4]);
  const bool gated = act == MOE_ACT_SWIGLU || act == MOE_ACT_GEGLU;
  const at::Tensor& out = tensor(a[5], "out");
  dense(&out, kBf16, {M, gated ? N / 2 : N}, "out", "contiguous bf16 [M, N] (gated: [M, N/2]) on the GPU");
  const at::Tensor* status = maybe(a[6], "dev_status");
  int32_t* const word = status_word(status);
  const moe_stream_t stream = stream_of(
      {{&x, "x"}, {&xs, "x_scale"}, {&w, "w"}, {&ws, "w_scale"}, {&out, "out"}, {status, "dev_status"}});
  return done(moe_linear_fp8(static_cast<const uint8_t*>(x.data_ptr()), ld(x, K), static_cast<const float*>(xs.data_ptr()),
                             one ? MOE_FP8_PER_TOKEN : MOE_FP8_PER_GROUP, int32_size(M, "x"), int32_size(K, "x"),
                             static_cast<const uint8_t*>(w.data_ptr()), static_cast<const float*>(ws.data_ptr()),
                             int32_size(N, "w"), static_cast<int32_t>(act), static_cast<uint16_t*>(out.data_ptr()), word, stream),
              "moe_linear_fp8");
}

// tokens [N, heads, dim] whose values lie side by side, with a stride between tokens
void tokens(const at::Tensor* t, int64_t n, int64_t heads, int64_t dim, const char* what) {
  if (t && !(is(*t, kBf16, {n, heads, dim}) && (t->stride(2) == 1 || dim == 1) && (heads == 1 || t->stride(1) == dim)))
    refuse(what, "bf16 [N, num_heads, head_dim] on the GPU (an output like its input), each token's values contiguous");
}

// (q, k, positions, inv_freq, axes, adjacent, q_out, k_out, dev_status)
PyObject* rotary(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  const at::Tensor* k = maybe(a[1], "k");
  if (q.dim() != 3 || (k && k->dim() != 3)) refuse("q and k", "[N, num_heads, head_dim]");
  const int64_t N = q.size(0), H = q.size(1), D = q.size(2), Hk = k ? k->size(1) : 0;
  tokens(&q, N, H, D, "q");
  tokens(k, N, Hk, D, "k");
  const at::Tensor &pos = tensor(a[2], "positions"), &freq = tensor(a[3], "inv_freq");
  const int64_t A = pos.dim() == 2 ? pos.size(0) : 1;
  if (pos.dim() < 1 || pos.dim() > 2 || (pos.scalar_type() != at::kInt && pos.scalar_type() != at::kLong) || !pos.is_cuda() ||
      pos.size(-1) != N || (pos.stride(-1) != 1 && N > 1))
    refuse("positions", "int32 or int64 [N] or [num_axes, N] on the GPU, an axis' positions side by side");
  const int64_t half = freq.dim() == 1 ? freq.size(0) : 0;
  dense(&freq, at::kDouble, {half}, "inv_freq", "contiguous float64 [rotary_dim / 2] on the GPU");
  const at::Tensor* axes = maybe(a[4], "axes");
  dense(axes, at::kByte, {half}, "axes", "contiguous uint8 of inv_freq's size on the GPU");
  if (!axes && A > 1) refuse("axes", "given where positions has several axes");
  const int adjacent = PyObject_IsTrue(a[5]);
  if (adjacent < 0) throw Raised();
  const at::Tensor &qo = tensor(a[6], "q_out"), *ko = maybe(a[7], "k_out"), *status = maybe(a[8], "dev_status");
  if ((k != nullptr) != (ko != nullptr)) refuse("k_out", "given with k, and only then");
  tokens(&qo, N, H, D, "q_out");
  tokens(ko, N, Hk, D, "k_out");
  int32_t* const word = status_word(status);
  const moe_stream_t stream =
      stream_of({{&q, "q"}, {k, "k"}, {&pos, "positions"}, {&freq, "inv_freq"}, {axes, "axes"}, {&qo, "q_out"}, {ko, "k_out"},
                 {status, "dev_status"}});
  return done(moe_rotary(static_cast<const uint16_t*>(q.data_ptr()), ld(q, H * D), int32_size(H, "q"),
                         static_cast<const uint16_t*>(pointer(k)), k ? ld(*k, Hk * D) : 0, int32_size(Hk, "k"), int32_size(D, "q"),
                         int32_size(2 * half, "inv_freq"), adjacent, pos.data_ptr(), pos.scalar_type() == at::kInt ? 4 : 8,
                         A > 1 ? pos.stride(0) : N, int32_size(A, "positions"), static_cast<const double*>(freq.data_ptr()),
                         static_cast<const uint8_t*>(pointer(axes)), int32_size(N, "q"), static_cast<uint16_t*>(qo.data_ptr()),
                         ld(qo, H * D), static_cast<uint16_t*>(pointer(ko)), ko ? ld(*ko, Hk * D) : 0, word, stream),
              "moe_rotary");
}

// (logits, uniform, temperature, top_k, top_p, min_p, tokens)
PyObject* sample_tokens(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "logits");
  const bool f32 = x.scalar_type() == at::kFloat;
  if (x.dim() != 2) refuse("logits", "[B, V]");
  const int64_t B = x.size(0), V = x.size(1);
  rows(&x, f32 ? at::kFloat : kBf16, B, V, "logits", "bf16 or float32 rows on the GPU, their values side by side");
  const at::Tensor& u = tensor(a[1], "uniform");
  dense(&u, at::kFloat, {B}, "uniform", "contiguous float32 [B] on the GPU");
  const at::Tensor *t = maybe(a[2], "temperature"), *k = maybe(a[3], "top_k"), *p = maybe(a[4], "top_p"), *m = maybe(a[5], "min_p");
  dense(t, at::kFloat, {B}, "temperature", "contiguous float32 [B] on the GPU");
  dense(k, at::kInt, {B}, "top_k", "contiguous int32 [B] on the GPU");
  dense(p, at::kFloat, {B}, "top_p", "contiguous float32 [B] on the GPU");
  dense(m, at::kFloat, {B}, "min_p", "contiguous float32 [B] on the GPU");
  const at::Tensor& out = tensor(a[6], "out");
  dense(&out, at::kInt, {B}, "out", "contiguous int32 [B] on the GPU");
  const moe_stream_t stream = stream_of({{&x, "logits"}, {&u, "uniform"}, {t, "temperature"}, {k, "top_k"}, {p, "top_p"},
                                         {m, "min_p"}, {&out, "out"}});
  return done(moe_sample(x.data_ptr(), f32 ? MOE_LOGITS_F32 : MOE_LOGITS_BF16, ld(x, V), int32_size(B, "logits"),
                         int32_size(V, "logits"), static_cast<const float*>(u.data_ptr()), static_cast<const float*>(pointer(t)),
                         static_cast<const int32_t*>(pointer(k)), static_cast<const float*>(pointer(p)),
                         static_cast<const float*>(pointer(m)), static_cast<int32_t*>(out.data_ptr()), stream),
              "moe_sample");
}

#define ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(set_error, 1), ENTRY(stream_id, 0), ENTRY(refuse_device, 3), ENTRY(add_rms_norm, 9), ENTRY(fp4_linear, 7), ENTRY(kv_cache, 7),
                         ENTRY(kv_append, 6), ENTRY(kv_workspace, 3), ENTRY(kv_attend, 8),
                         ENTRY(quantize_fp8, 4), ENTRY(fp8_linear, 7), ENTRY(rotary, 9), ENTRY(sample_tokens, 7), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", "calls of libmoe_nvfp4 on torch tensors", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
