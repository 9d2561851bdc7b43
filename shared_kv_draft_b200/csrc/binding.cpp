// Argument checks and marshalling of the tree and rotary calls for Python: a native module beside the
// ctypes binding, because these calls run once a layer and their checks are many (an attention call has ten
// tensors). It computes nothing. Python signatures and documentation are in orthrus.py, whose
// functions pass their arguments on by position; here each tensor's device, type, shape and strides are
// checked (ValueError), and the C entry point is called on the tensors' device and the given or
// current stream (OrthrusError for its error codes).
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "orthrus.h"

namespace {

struct Refused {  // becomes a ValueError
  std::string what;
};
struct Raised {};  // a Python exception is set

const char* g_call = "";  // the running call's name (the GIL is held throughout)

[[noreturn]] void refuse(const std::string& what) { throw Refused{std::string(g_call) + ": " + what}; }

void want(bool ok, const char* what) {
  if (!ok) refuse(what);
}

int32_t i32(int64_t n) {
  if (n > INT32_MAX) refuse("a size is past 31 bits");
  return (int32_t)n;
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

std::string text(at::IntArrayRef shape) {
  std::string s = "[";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + "]";
}

void dense(const at::Tensor& t, const char* name, int64_t dev, at::ScalarType type, at::IntArrayRef shape) {
  if (t.scalar_type() == type && t.get_device() == dev && t.sizes() == shape && t.is_contiguous()) return;
  refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor on device " + std::to_string(dev) +
         " of shape " + text(shape));
}

void* dense(PyObject* o, const char* name, int64_t dev, at::ScalarType type, at::IntArrayRef shape) {
  const at::Tensor& t = tensor(o, name);
  dense(t, name, dev, type, shape);
  return t.data_ptr();
}

int32_t* ints(PyObject* o, const char* name, int64_t dev, at::IntArrayRef shape) {
  return (int32_t*)dense(o, name, dev, at::kInt, shape);
}

int32_t* optional_ints(PyObject* o, const char* name, int64_t dev, at::IntArrayRef shape) {
  return o == Py_None ? nullptr : ints(o, name, dev, shape);
}

int32_t* status_word(PyObject* o, int64_t dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "status");
  if (t.scalar_type() != at::kInt || t.get_device() != dev || t.numel() != 1) refuse("status must be one int32 on the device");
  return (int32_t*)t.data_ptr();
}

// The type codes of orthrus.h; -1 for others.
int type_code(at::ScalarType t) {
  return t == at::kFloat ? ORTHRUS_FP32 : t == at::kBFloat16 ? ORTHRUS_BF16 : t == at::kHalf ? ORTHRUS_FP16 : -1;
}

// The tensors' device as the current one, and the call's stream on it.
struct Place {
  std::optional<c10::cuda::CUDAGuard> guard;
  orthrus_stream stream;
  Place(int64_t dev, PyObject* s) {
    if (c10::cuda::current_device() != dev) guard.emplace((c10::DeviceIndex)dev);
    if (s == Py_None) {
      stream = (orthrus_stream)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
      return;
    }
    PyObject* h = PyObject_GetAttrString(s, "cuda_stream");
    if (!h) throw Raised{};
    stream = (orthrus_stream)PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Raised{};
  }
};

void check(const char* entry, orthrus_status code) {
  if (code == ORTHRUS_OK) return;
  PyObject* m = PyImport_ImportModule("shared_kv_draft_b200.orthrus");
  PyObject* cls = m ? PyObject_GetAttrString(m, "OrthrusError") : nullptr;
  PyObject* e = cls ? PyObject_CallFunction(cls, "si", entry, (int)code) : nullptr;
  if (e) PyErr_SetObject(cls, e);
  Py_XDECREF(e);
  Py_XDECREF(cls);
  Py_XDECREF(m);
  throw Raised{};
}

// A function of n positional arguments as a Python method.
template <void (*F)(PyObject* const*), int N>
PyObject* method(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    F(args);
    Py_RETURN_NONE;
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised{};
  return x;
}

// parents, depth, mask, n_nodes, status, stream
void tree_layout(PyObject* const* a) {
  g_call = "tree_layout";
  const at::Tensor& parents = tensor(a[0], "parents");
  const int64_t dev = parents.get_device();
  want(dev >= 0 && parents.dim() == 2, "parents must be [batch][nodes] on a GPU");
  const int64_t B = parents.size(0), N = parents.size(1);
  dense(parents, "parents", dev, at::kInt, {B, N});
  int32_t* depth = ints(a[1], "depth", dev, {B, N});
  uint64_t* mask = (uint64_t*)dense(a[2], "mask", dev, at::kLong, {B, N, (N + 63) / 64});
  int32_t *n_nodes = optional_ints(a[3], "n_nodes", dev, {B}), *status = status_word(a[4], dev);
  Place p(dev, a[5]);
  check("orthrus_tree_layout", orthrus_tree_layout((const int32_t*)parents.data_ptr(), n_nodes, i32(B), i32(N), depth, mask,
                                                   status, p.stream));
}

// q, k_cache, v_cache, k_blk, v_blk, len, mask, out, workspace, n_nodes, scale, status, stream
void tree_attention(PyObject* const* a) {
  g_call = "tree_attention";
  const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &kb = tensor(a[3], "k_blk"), &mask = tensor(a[6], "mask"),
                   &out = tensor(a[7], "out"), &ws = tensor(a[8], "workspace");
  const int64_t dev = q.get_device();
  const at::ScalarType t = q.scalar_type(), to = out.scalar_type();
  want(dev >= 0 && q.dim() == 4 && (t == at::kHalf || t == at::kBFloat16),
       "q must be fp16 or bf16 [batch][kv heads][nodes*group][d] on a GPU");
  const int64_t B = q.size(0), H = q.size(1), R = q.size(2), d = q.size(3);
  want(mask.dim() == 3 && mask.size(1) > 0, "mask must be [batch][nodes][words]");
  const int64_t N = mask.size(1), G = R / N;
  want(G * N == R, "mask does not fit q");
  want(kc.dim() == 4 && kb.dim() == 4 && kb.size(2) >= N, "a cache or block has another shape");
  const int64_t cap = kc.size(2), rows = kb.size(2);
  dense(q, "q", dev, t, {B, H, R, d});
  dense(kc, "k_cache", dev, t, {B, H, cap, d});
  const void* vc = dense(a[2], "v_cache", dev, t, {B, H, cap, d});
  dense(kb, "k_blk", dev, t, {B, H, rows, d});
  const void* vb = dense(a[4], "v_blk", dev, t, {B, H, rows, d});
  dense(mask, "mask", dev, at::kLong, {B, N, (N + 63) / 64});
  const int32_t *len = ints(a[5], "len", dev, {B}), *n_nodes = optional_ints(a[9], "n_nodes", dev, {B});
  const bool planes = out.dim() == 3;
  want(to == at::kBFloat16 || (to == at::kHalf && !planes), "out must be fp16 or bf16, planes bf16");
  if (planes) dense(out, "out", dev, to, {2, B * N, H * G * d});
  else dense(out, "out", dev, to, {B * N, H * G * d});
  want(ws.get_device() == dev && ws.is_contiguous(), "workspace must be contiguous on q's device");
  int32_t* status = status_word(a[11], dev);
  const float scale = (float)number(a[10]);
  Place p(dev, a[12]);
  check("orthrus_tree_attention",
        orthrus_tree_attention(q.data_ptr(), kc.data_ptr(), vc, kb.data_ptr(), vb, len, n_nodes, (const uint64_t*)mask.data_ptr(),
                               i32(B), i32(H), i32(G), i32(N), i32(d), i32(cap), i32(rows), type_code(t), planes ? ORTHRUS_BF16_PLANES : type_code(to), scale,
                               out.data_ptr(), ws.data_ptr(), ws.nbytes(), status, p.stream));
}

// parents, tokens, argmax, k_blk, v_blk, k_cache, v_cache, len, new_len, pending, accept_len, path, committed,
// n_nodes, status, stream
void tree_commit(PyObject* const* a) {
  g_call = "tree_commit";
  const at::Tensor &parents = tensor(a[0], "parents"), &kb = tensor(a[3], "k_blk"), &kc = tensor(a[5], "k_cache");
  const int64_t dev = parents.get_device();
  want(dev >= 0 && parents.dim() == 2, "parents must be [batch][nodes] on a GPU");
  const int64_t B = parents.size(0), N = parents.size(1);
  const at::ScalarType t = kc.scalar_type();
  want(kc.dim() == 5 && kb.dim() == 5 && kc.element_size() == 2 && kb.size(3) >= N,
       "caches and blocks must be five-dimensional with 16-bit elements, a block with a row for every node");
  const int64_t L = kc.size(0), H = kc.size(2), cap = kc.size(3), d = kc.size(4), rows = kb.size(3);
  dense(parents, "parents", dev, at::kInt, {B, N});
  const int32_t *tokens = ints(a[1], "tokens", dev, {B, N}), *argmax = ints(a[2], "argmax", dev, {B, N});
  dense(kb, "k_blk", dev, t, {L, B, H, rows, d});
  const void* vb = dense(a[4], "v_blk", dev, t, {L, B, H, rows, d});
  dense(kc, "k_cache", dev, t, {L, B, H, cap, d});
  void* vc = dense(a[6], "v_cache", dev, t, {L, B, H, cap, d});
  const int32_t* len = ints(a[7], "len", dev, {B});
  int32_t *new_len = ints(a[8], "new_len", dev, {B}), *pending = ints(a[9], "pending", dev, {B}),
          *accept_len = ints(a[10], "accept_len", dev, {B}), *path = ints(a[11], "path", dev, {B, N}),
          *committed = ints(a[12], "committed", dev, {B, N});
  const int32_t* n_nodes = optional_ints(a[13], "n_nodes", dev, {B});
  int32_t* status = status_word(a[14], dev);
  Place p(dev, a[15]);
  check("orthrus_tree_commit",
        orthrus_tree_commit((const int32_t*)parents.data_ptr(), tokens, argmax, n_nodes, kb.data_ptr(), vb, i32(rows),
                            kc.data_ptr(), vc, i32(L), i32(B), i32(H), i32(cap), i32(d), i32(N), len, new_len, pending, accept_len, path, committed, status, p.stream));
}

// rope, parts, len, offsets, inverse, status, stream
void rotary(PyObject* const* a) {
  g_call = "rotary";
  Py_buffer view;
  if (PyObject_GetBuffer(a[0], &view, PyBUF_SIMPLE)) throw Raised{};
  struct Release {
    Py_buffer* v;
    ~Release() { PyBuffer_Release(v); }
  } release{&view};
  want(view.len == (Py_ssize_t)sizeof(orthrus_rope), "rope must be a Rope");
  const orthrus_rope* rope = (const orthrus_rope*)view.buf;
  struct Parts {
    PyObject* o;
    ~Parts() { Py_XDECREF(o); }
  } parts{PySequence_Fast(a[1], "parts must be a sequence")};
  if (!parts.o) throw Raised{};
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(parts.o);
  want(n >= 1 && n <= ORTHRUS_ROTARY_MAX_PARTS, "1 to 3 parts");
  orthrus_rotary_part p[ORTHRUS_ROTARY_MAX_PARTS];
  int64_t dev = -1, B = 0, T = 0;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* it = PySequence_Fast_GET_ITEM(parts.o, i);
    const bool tuple = PyTuple_Check(it);
    want((tuple || PyList_Check(it)) && Py_SIZE(it) >= 2 && Py_SIZE(it) <= 3, "a part is (src, dst) or (src, dst, flags)");
    auto item = [&](int k) { return tuple ? PyTuple_GET_ITEM(it, k) : PyList_GET_ITEM(it, k); };
    const at::Tensor &src = tensor(item(0), "src"), &dst = tensor(item(1), "dst");
    long flags = 0;
    if (Py_SIZE(it) == 3) {
      flags = PyLong_AsLong(item(2));
      if (flags == -1 && PyErr_Occurred()) throw Raised{};
      want(flags >= 0 && flags < (1 << 16), "flags out of range");
    }
    if (i == 0) {
      dev = src.get_device();
      want(dev >= 0 && src.dim() == 4, "src must be [batch][tokens][heads][d] on a GPU");
      B = src.size(0);
      T = src.size(1);
    }
    const int st = type_code(src.scalar_type()), dt = type_code(dst.scalar_type());
    want(st >= 0 && dt >= 0 && src.get_device() == dev && dst.get_device() == dev,
         "tensors must be fp32, bf16 or fp16 on one GPU");
    want(src.dim() == 4 && src.size(0) == B && src.size(1) == T && src.size(3) == rope->head_dim && src.stride(3) == 1,
         "src must be [batch][tokens][heads][d] with a dense last dimension");
    const int64_t nd = dst.dim();
    const bool grouped = nd == 5;
    want((nd == 4 || grouped) && dst.size(0) == B && dst.size(nd - 1) == rope->head_dim && dst.stride(nd - 1) == 1 &&
             (grouped ? dst.size(2) * dst.size(3) : dst.size(2)) == src.size(2) &&
             ((flags & ORTHRUS_ROTARY_APPEND) || dst.size(1) == T) && dst.size(1) <= INT32_MAX && src.size(2) <= INT32_MAX,
         "dst must be [batch][rows][heads][d] or [batch][rows][kv heads][group][d] with a dense last dimension");
    orthrus_rotary_part& x = p[i];
    x.src = src.data_ptr();
    x.dst = dst.data_ptr();
    x.src_type = st;
    x.dst_type = dt;
    x.heads = (int32_t)src.size(2);
    x.group = grouped ? (int32_t)dst.size(3) : 1;
    x.flags = (int32_t)flags;
    x.rows = (int32_t)dst.size(1);
    x.src_batch = src.stride(0);
    x.src_token = src.stride(1);
    x.src_head = src.stride(2);
    x.dst_batch = dst.stride(0);
    x.dst_token = dst.stride(1);
    x.dst_kv = dst.stride(2);
    x.dst_head = grouped ? dst.stride(3) : 0;
  }
  want(B <= INT32_MAX && T <= INT32_MAX, "too many tokens");
  const int32_t *len = optional_ints(a[2], "len", dev, {B}), *offsets = optional_ints(a[3], "offsets", dev, {B, T});
  const int inverse = PyObject_IsTrue(a[4]);
  if (inverse < 0) throw Raised{};
  int32_t* status = status_word(a[5], dev);
  Place place(dev, a[6]);
  check("orthrus_rotary", orthrus_rotary(rope, p, (int32_t)n, (int32_t)B, (int32_t)T, len, offsets, inverse, status, place.stream));
}

#define FAST(f, n) \
  { #f, (PyCFunction)(void (*)(void))method<f, n>, METH_FASTCALL, nullptr }
PyMethodDef g_methods[] = {FAST(tree_layout, 6), FAST(tree_attention, 13), FAST(tree_commit, 16), FAST(rotary, 7),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", "Checks and marshalling of the tree and rotary calls.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&g_module);
  if (m && PyModule_AddStringConstant(m, "built_for", ORTHRUS_BUILT_FOR)) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
