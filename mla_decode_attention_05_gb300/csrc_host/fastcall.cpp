// The binding's short way: the checks and calls of the operators whose calls are
// short on the GPU, without the interpreter.  (From Python a call's checks,
// argument conversions and allocations take 10 to 20 us, several times what a
// decode step's insert or projection takes on the GPU.)
//
// Every function answers with its result where all arguments are plain tensors
// that the call can take as they are, with the library's (negative) error code
// where the library refuses it, and with None in every other case: the Python
// function then goes its own way, which also has the error messages.  So
// nothing here decides what is allowed; it only recognises common calls.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mla_decode.h"

namespace {

decltype(&mla_kv_insert_rope) insert_rope_fn;
decltype(&mla_kv_expand) expand_fn;
decltype(&mla_prefill) prefill_fn;
decltype(&mla_prefill_workspace_bytes) prefill_ws_fn;
decltype(&mla_value_project) value_fn;

// A plain tensor, or null.
const at::Tensor *tensor(PyObject *o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

// An optional one: false if it is neither None nor a plain tensor.
bool optional(PyObject *o, const at::Tensor *&t) {
  t = o == Py_None ? nullptr : tensor(o);
  return o == Py_None || t != nullptr;
}

bool on(const at::Tensor *t, int dev) { return t && t->is_cuda() && t->get_device() == dev; }

bool whole(const at::Tensor *t, int dev, at::ScalarType type, int64_t dims) {
  return on(t, dev) && t->scalar_type() == type && t->dim() == dims && t->is_contiguous();
}

// A bf16 tensor of two or three axes whose last has w contiguous values and whose
// other strides are multiples of 8; a, b: those strides (an axis of one entry
// has none that matters: w).
bool rows(const at::Tensor *t, int dev, int64_t dims, int64_t w, int64_t &a, int64_t &b) {
  if (!on(t, dev) || t->scalar_type() != at::kBFloat16 || t->dim() != dims) return false;
  if (t->size(dims - 1) != w || t->stride(dims - 1) != 1) return false;
  a = t->size(0) > 1 ? t->stride(0) : w;
  b = dims == 3 && t->size(1) > 1 ? t->stride(1) : w;
  return a % 8 == 0 && b % 8 == 0;
}

bool sized(const at::Tensor &t, std::initializer_list<int64_t> want) { return t.sizes() == at::IntArrayRef(want); }

// Format of a cache by its type and row width, or -1.
int format_of(const at::Tensor &c) {
  if (c.dim() != 3) return -1;
  if (c.scalar_type() == at::kBFloat16) return c.size(2) == 576 ? MLA_KV_BF16 : -1;
  if (c.scalar_type() != at::kByte) return -1;
  return c.size(2) == 640 ? MLA_KV_FP8_E4M3 : c.size(2) == 576 ? MLA_KV_FP8_E4M3_TENSOR : -1;
}

constexpr int64_t kMostInt = 0x7FFFFFFF;

mla_stream_t stream_of(int dev) {
  return reinterpret_cast<mla_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
}

// Lets the interpreter's other threads run while this one allocates and
// launches, as the Python way does: both can block (an allocation waits for
// PyTorch's allocator, a launch for room in the stream's queue), and what they
// wait for may need the interpreter.
struct Unlocked {
  PyThreadState *state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

PyObject *none() { Py_RETURN_NONE; }
PyObject *code(int rc) { return PyLong_FromLong(rc); }

// value_project(attn, w_uv, out | None) -> out
PyObject *value_project(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 3 || !value_fn) return none();
  const at::Tensor *attn = tensor(args[0]), *w = tensor(args[1]), *given;
  if (!attn || !w || !attn->is_cuda() || !optional(args[2], given)) return none();
  const int dev = attn->get_device();
  int64_t at_tok, at_head, w_head, w_row;
  if (dev != c10::cuda::current_device() || !rows(attn, dev, 3, 512, at_tok, at_head) ||
      !rows(w, dev, 3, 512, w_head, w_row))
    return none();
  const int64_t N = attn->size(0), H = attn->size(1);
  if (w->size(0) != H || w->size(1) != 128 || N > kMostInt) return none();
  if (given && (!whole(given, dev, at::kBFloat16, 3) || !sized(*given, {N, H, 128}))) return none();
  at::Tensor out;
  int rc;
  {
    Unlocked others;
    out = given ? *given : at::empty({N, H, 128}, attn->options());
    rc = value_fn(attn->data_ptr(), at_tok, at_head, w->data_ptr(), w_row, w_head, (int)N, (int)H, out.data_ptr(),
                  stream_of(dev));
  }
  return rc < 0 ? code(rc) : THPVariable_Wrap(out);
}

// prefill(q, k_nope, k_pe, v, cu_q, cu_k, scale, causal, workspace | None, out | None, lse | None) -> (out, lse)
PyObject *prefill(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 11 || !prefill_fn || !PyFloat_CheckExact(args[6]) || !PyBool_Check(args[7])) return none();
  const at::Tensor *q = tensor(args[0]), *kn = tensor(args[1]), *kp = tensor(args[2]), *v = tensor(args[3]);
  const at::Tensor *cq = tensor(args[4]), *ck = tensor(args[5]), *space, *out_given, *lse_given;
  if (!q || !q->is_cuda() || !optional(args[8], space) || !optional(args[9], out_given) ||
      !optional(args[10], lse_given))
    return none();
  const int dev = q->get_device();
  int64_t qt, qh, kt, kh, pt, pb, vt, vh;
  if (dev != c10::cuda::current_device() || !rows(q, dev, 3, 192, qt, qh) || !rows(kn, dev, 3, 128, kt, kh) ||
      !rows(kp, dev, 2, 64, pt, pb) || !rows(v, dev, 3, 128, vt, vh) || !whole(cq, dev, at::kInt, 1) ||
      !whole(ck, dev, at::kInt, 1))
    return none();
  const int64_t Nq = q->size(0), H = q->size(1), Nk = kn->size(0), B = cq->size(0) - 1;
  if (kn->size(1) != H || v->size(0) != Nk || v->size(1) != H || kp->size(0) != Nk || B < 0 || ck->size(0) != B + 1 ||
      Nq > kMostInt || Nk > kMostInt || H > kMostInt || B > kMostInt)
    return none();
  if (out_given && (!whole(out_given, dev, at::kBFloat16, 3) || !sized(*out_given, {Nq, H, 128}))) return none();
  if (lse_given && (!whole(lse_given, dev, at::kFloat, 2) || !sized(*lse_given, {H, Nq}))) return none();
  if (space && !(on(space, dev) && space->is_contiguous())) return none();
  const float scale = (float)PyFloat_AS_DOUBLE(args[6]);
  const int causal = args[7] == Py_True ? 1 : 0;
  at::Tensor out, lse, room;
  int rc;
  {
    Unlocked others;
    out = out_given ? *out_given : at::empty({Nq, H, 128}, q->options());
    lse = lse_given ? *lse_given : at::empty({H, Nq}, q->options().dtype(at::kFloat));
    size_t bytes = prefill_ws_fn((int)B, (int)H, (int)Nq, (int)Nk);
    if (space) {
      room = *space;
      bytes = space->nbytes();
    } else if (bytes) {
      room = at::empty({(int64_t)bytes}, q->options().dtype(at::kByte));
    }
    rc = prefill_fn(q->data_ptr(), qt, qh, kn->data_ptr(), kt, kh, kp->data_ptr(), pt, v->data_ptr(), vt, vh,
                    cq->data_ptr<int32_t>(), ck->data_ptr<int32_t>(), (int)B, (int)H, (int)Nq, (int)Nk, scale, causal,
                    room.defined() ? room.data_ptr() : nullptr, bytes, out.data_ptr(), lse.data_ptr<float>(),
                    stream_of(dev));
  }
  if (rc < 0) return code(rc);
  PyObject *a = THPVariable_Wrap(out), *b = THPVariable_Wrap(lse);
  PyObject *r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}

// kv_expand(cache, block_table, cu, w_uk, w_uv, total, scales | None, kv | None, k_pe | None) -> (kv, k_pe)
PyObject *kv_expand(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 9 || !expand_fn || !PyLong_CheckExact(args[5])) return none();
  const at::Tensor *c = tensor(args[0]), *bt = tensor(args[1]), *cu = tensor(args[2]);
  const at::Tensor *uk = tensor(args[3]), *uv = tensor(args[4]), *sc, *kv_given, *pe_given;
  if (!c || !c->is_cuda() || !optional(args[6], sc) || !optional(args[7], kv_given) || !optional(args[8], pe_given))
    return none();
  const int dev = c->get_device(), fmt = format_of(*c);
  int overflow = 0;
  const long total = PyLong_AsLongAndOverflow(args[5], &overflow);
  int64_t uk_head, uk_row, uv_head, uv_row;
  if (dev != c10::cuda::current_device() || fmt < 0 || !c->is_contiguous() || overflow || total < 0 ||
      total > kMostInt || !whole(bt, dev, at::kInt, 2) || !whole(cu, dev, at::kInt, 1) ||
      !rows(uk, dev, 3, 512, uk_head, uk_row) || !rows(uv, dev, 3, 512, uv_head, uv_row))
    return none();
  const int64_t H = uk->size(0), B = bt->size(0);
  if (uk->size(1) != 128 || uv->size(0) != H || uv->size(1) != 128 || cu->size(0) != B + 1 || H > kMostInt ||
      B > kMostInt || bt->size(1) > kMostInt || c->size(0) > kMostInt || c->size(1) > kMostInt)
    return none();
  if (fmt == MLA_KV_FP8_E4M3 && (!whole(sc, dev, at::kFloat, 3) || !sized(*sc, {c->size(0), c->size(1), 4})))
    return none();
  if (fmt == MLA_KV_FP8_E4M3_TENSOR &&
      !(on(sc, dev) && sc->scalar_type() == at::kFloat && sc->is_contiguous() && sc->numel() == 1))
    return none();
  if (kv_given && (!whole(kv_given, dev, at::kBFloat16, 3) || !sized(*kv_given, {total, H, 256}))) return none();
  if (pe_given && (!whole(pe_given, dev, at::kBFloat16, 2) || !sized(*pe_given, {total, 64}))) return none();
  at::Tensor kv, pe;
  int rc;
  {
    Unlocked others;
    kv = kv_given ? *kv_given : at::empty({total, H, 256}, uk->options());
    pe = pe_given ? *pe_given : at::empty({total, 64}, uk->options());
    rc = expand_fn(c->data_ptr(), fmt, (int)c->size(0), (int)c->size(1), bt->data_ptr<int32_t>(), (int)bt->size(1),
                   cu->data_ptr<int32_t>(), (int)B, (int)total, fmt != MLA_KV_BF16 ? sc->data_ptr<float>() : nullptr,
                   uk->data_ptr(), uk_row, uk_head, uv->data_ptr(), uv_row, uv_head, (int)H, kv.data_ptr(),
                   pe.data_ptr(), stream_of(dev));
  }
  if (rc < 0) return code(rc);
  PyObject *a = THPVariable_Wrap(kv), *b = THPVariable_Wrap(pe);
  PyObject *r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}

// kv_insert_rope(kv_c, k_pe, w_kva, slots, cache, eps, positions, cos_sin, interleaved, q_pe | None, q_out | None,
//                scales | None, k_scale_inv | None, fp8_per_tensor) -> True
PyObject *kv_insert_rope(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 14 || !insert_rope_fn || !PyFloat_CheckExact(args[5]) || !PyBool_Check(args[8]) || !PyBool_Check(args[13]))
    return none();
  const at::Tensor *kc = tensor(args[0]), *kp = tensor(args[1]), *w = tensor(args[2]), *slots = tensor(args[3]);
  const at::Tensor *c = tensor(args[4]), *pos = tensor(args[6]), *cs = tensor(args[7]), *q, *qo, *sc, *ksi;
  if (!kc || !kc->is_cuda() || !c || !optional(args[9], q) || !optional(args[10], qo) || !optional(args[11], sc) ||
      !optional(args[12], ksi))
    return none();
  const int dev = kc->get_device();
  if (dev != c10::cuda::current_device() || !on(kp, dev) || !on(c, dev) || !c->is_contiguous() || c->dim() != 3)
    return none();
  if (kc->scalar_type() != at::kBFloat16 || kc->dim() != 2 || kc->size(1) < 512 || kc->stride(1) != 1 ||
      kp->scalar_type() != at::kBFloat16 || kp->dim() != 2 || kp->size(1) < 64 || kp->stride(1) != 1)
    return none();
  const int64_t N = kc->size(0);
  const int64_t ld_kv = N > 1 ? kc->stride(0) : kc->size(1), ld_pe = N > 1 ? kp->stride(0) : kp->size(1);
  if (N == 0 || N > kMostInt || kp->size(0) != N || ld_kv > kMostInt || ld_pe > kMostInt ||
      !whole(w, dev, at::kBFloat16, 1) || w->size(0) != 512 || !whole(slots, dev, at::kLong, 1) ||
      slots->size(0) != N || !whole(pos, dev, at::kLong, 1) || pos->size(0) != N || !whole(cs, dev, at::kFloat, 2) ||
      cs->size(1) != 64 || cs->size(0) > kMostInt)
    return none();
  int fmt = -1;
  if (c->scalar_type() == at::kBFloat16 && c->size(2) == 576) fmt = MLA_KV_BF16;
  if (c->scalar_type() == at::kByte)
    fmt = args[13] == Py_True ? (c->size(2) == 576 ? MLA_KV_FP8_E4M3_TENSOR : -1) : (c->size(2) == 640 ? MLA_KV_FP8_E4M3 : -1);
  if (fmt < 0 || c->size(0) > kMostInt || c->size(1) > kMostInt) return none();
  if (fmt == MLA_KV_FP8_E4M3 && (!whole(sc, dev, at::kFloat, 3) || !sized(*sc, {c->size(0), c->size(1), 4})))
    return none();
  if (fmt == MLA_KV_FP8_E4M3_TENSOR &&
      !(on(ksi, dev) && ksi->scalar_type() == at::kFloat && ksi->is_contiguous() && ksi->numel() >= 1))
    return none();
  int64_t qt = 0, qh = 0, ot = 0, oh = 0, H = 0;
  if (q) {
    if (!qo) qo = q;
    if (!rows(q, dev, 3, 64, qt, qh) || !rows(qo, dev, 3, 64, ot, oh)) return none();
    H = q->size(1);
    if (q->size(0) != N || qo->size(0) != N || qo->size(1) != H || H > kMostInt) return none();
    // tokens before heads or whole, without overlap (the stride of an axis of
    // one entry does not matter); the same place only with the same strides
    const bool apart = (H < 2 || oh >= 64) && (N < 2 || ot >= (H < 2 ? 0 : oh * (H - 1)) + 64);
    if (!qo->is_contiguous() && !apart) return none();
    if (q->data_ptr() == qo->data_ptr() && (qt != ot || qh != oh)) return none();
  } else if (qo) {
    return none();
  }
  const float eps = (float)PyFloat_AS_DOUBLE(args[5]);
  const int interleaved = args[8] == Py_True ? 1 : 0;
  int rc;
  {
    Unlocked others;
    rc = insert_rope_fn(kc->data_ptr(), (int)ld_kv, kp->data_ptr(), (int)ld_pe, w->data_ptr(), eps,
                        slots->data_ptr<int64_t>(), pos->data_ptr<int64_t>(), cs->data_ptr<float>(), (int)cs->size(0),
                        interleaved, (int)N, c->data_ptr(), fmt, (int)c->size(0), (int)c->size(1),
                        fmt == MLA_KV_FP8_E4M3 ? sc->data_ptr<float>() : nullptr,
                        fmt == MLA_KV_FP8_E4M3_TENSOR ? ksi->data_ptr<float>() : nullptr,
                        q ? q->data_ptr() : nullptr, qt, qh, q ? qo->data_ptr() : nullptr, ot, oh, (int)H,
                        stream_of(dev));
  }
  if (rc < 0) return code(rc);
  Py_RETURN_TRUE;
}

// C++ exceptions (an allocation that failed, say) become Python's.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  try {
    return F(self, args, n);
  } catch (const c10::OutOfMemoryError &) {
    PyErr_Clear();
    return none();  // the Python way raises it as torch does
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// bind(addresses of the library's functions, in this order)
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void *at[5];
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
    return nullptr;
  }
  for (int i = 0; i < 5; i++) {
    at[i] = PyLong_AsVoidPtr(args[i]);
    if (!at[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  insert_rope_fn = reinterpret_cast<decltype(insert_rope_fn)>(at[0]);
  expand_fn = reinterpret_cast<decltype(expand_fn)>(at[1]);
  prefill_fn = reinterpret_cast<decltype(prefill_fn)>(at[2]);
  prefill_ws_fn = reinterpret_cast<decltype(prefill_ws_fn)>(at[3]);
  value_fn = reinterpret_cast<decltype(value_fn)>(at[4]);
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<f>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    FAST(value_project), FAST(prefill), FAST(kv_expand), FAST(kv_insert_rope),
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fastcall() { return PyModule_Create(&module); }
