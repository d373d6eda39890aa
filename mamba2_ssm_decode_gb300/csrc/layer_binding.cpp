// layer_binding.cpp -- the Python side of the calls around the state update:
// checks that torch tensors describe the layout the C ABI expects, and calls
// it.  Native because the calls are short: one user's next token takes the GPU
// 3 us, looking at its tensors from Python took 6 to 10 us more, from here it
// takes less than one.  No compute, no copies.
//
// Positional functions only; layer_api.py has the signatures and defaults.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <string>
#include <vector>

#include "../../include/ssu.h"

namespace {

using at::Tensor;

struct Refused {
  PyObject* type;
  std::string what;
};

template <class... T>
[[noreturn]] void refuse(PyObject* type, const T&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  throw Refused{type, s.str()};
}
template <class... T>
void value_if(bool bad, const T&... parts) {
  if (bad) refuse(PyExc_ValueError, parts...);
}
template <class... T>
void unsupported_if(bool bad, const T&... parts) {
  if (bad) refuse(PyExc_NotImplementedError, parts...);
}

const Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, " must be a torch.Tensor or None");
  return &THPVariable_Unpack(o);
}

const Tensor& needed(PyObject* o, const char* name) {
  const Tensor* t = tensor(o, name);
  if (!t) refuse(PyExc_TypeError, name, " must be a torch.Tensor");
  return *t;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{nullptr, ""};
  return v;
}

int one_device(std::initializer_list<const Tensor*> ts) {
  int d = -1;
  for (const Tensor* t : ts) {
    if (!t) continue;
    value_if(!t->is_cuda(), "libssu_gb300 works on CUDA tensors only (there is no CPU path)");
    if (d < 0) d = t->get_device();
    value_if(t->get_device() != d, "all tensors must be on one device, got cuda:", d, " and cuda:",
             (int)t->get_device());
  }
  return d;
}

bool float_code(const Tensor& t, ssu_dtype* d) {
  switch (t.scalar_type()) {
    case at::kFloat: *d = SSU_F32; return true;
    case at::kBFloat16: *d = SSU_BF16; return true;
    case at::kHalf: *d = SSU_F16; return true;
    default: return false;
  }
}

ssu_dtype float_of(const Tensor& t, const char* name) {
  ssu_dtype d = SSU_F32;
  unsupported_if(!float_code(t, &d), name, " dtype ", t.scalar_type(), " is not supported");
  return d;
}

ssu_dtype index_of(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kInt) return SSU_I32;
  if (t.scalar_type() == at::kLong) return SSU_I64;
  refuse(PyExc_ValueError, name, " must be int32 or int64, got ", t.scalar_type());
}

const void* data(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

// A contiguous [n] tensor.
const void* vector(const Tensor* t, const char* name, int64_t n) {
  if (!t) return nullptr;
  value_if(t->dim() != 1 || t->size(0) != n, name, " must be [", n, "], got ", t->sizes());
  value_if(!t->is_contiguous(), name, " must be contiguous");
  return t->data_ptr();
}

// Row stride of a [rows, dim] operand with unit dim stride.
int64_t rows2(const Tensor& t, const char* name, int64_t rows, int64_t dim) {
  value_if(t.dim() != 2 || t.size(0) != rows || t.size(1) != dim, name, " must be [", rows, ", ",
           dim, "], got ", t.sizes());
  value_if(dim > 1 && t.stride(1) != 1, name, " must be contiguous along channels (stride 1), got ",
           t.strides());
  return t.stride(0);
}

// Slot vector of a one-token call as a table of one step.
ssu_slot_table slots_of(const Tensor* t, const char* name, int64_t n) {
  if (!t) return ssu_slot_table{};
  return ssu_slot_table{vector(t, name, n), n, 1, 1, 1};
}

// Slot table of a packed call: [S, T], or flat with entry (s, t) = s + t.
ssu_slot_table table(const Tensor* t, const char* name, int64_t nseqs) {
  if (!t) return ssu_slot_table{};
  if (t->dim() == 1) {
    const int64_t n = t->size(0), step = t->stride(0);
    return ssu_slot_table{t->data_ptr(), n ? (n - 1) * step + 1 : 0, step, step, n};
  }
  value_if(t->dim() != 2, name, " must be the flat [rows] or the 2-D [sequences, steps] slot table; "
           "got ", t->sizes());
  const int64_t S = t->size(0), T = t->size(1), ss = t->stride(0), ts = t->stride(1);
  value_if(S < nseqs, name, " must have a row for each of the ", nseqs, " sequences, got ",
           t->sizes());
  return ssu_slot_table{t->data_ptr(), S && T ? (S - 1) * ss + (T - 1) * ts + 1 : 0, ss, ts, T};
}

// The sequences of a call.
struct Seqs {
  enum Form { kOneToken, kPacked, kPrompt };
  Form form;
  const Tensor *cu, *na, *src, *dst, *init;
  int64_t nseqs, steps;
  ssu_dtype meta = SSU_I32, index = SSU_I32;

  // args: cu_seqlens, num_accepted, src, dst, has_initial_state
  Seqs(PyObject* form_, PyObject* const* a, PyObject* nseqs_, PyObject* steps_)
      : form((Form)integer(form_)), cu(tensor(a[0], "cu_seqlens")),
        na(tensor(a[1], "num_accepted_tokens")), src(tensor(a[2], "state_batch_indices")),
        dst(tensor(a[3], "dst_state_batch_indices")), init(tensor(a[4], "has_initial_state")),
        nseqs(integer(nseqs_)), steps(integer(steps_)) {}

  void check(int64_t rows) {
    if (form == kOneToken) nseqs = rows;
    if (form == kPrompt) {
      value_if(!cu || cu->dim() != 1 || cu->size(0) < 1, "cu_seqlens must hold the start of every "
               "sequence and the end of the last");
      nseqs = cu->size(0) - 1;
    }
    if (nseqs < 0) {
      value_if(!cu && !na && !src && !dst, "a packed multi-token call must carry per-sequence "
               "metadata: state_batch_indices, dst_state_batch_indices, num_accepted_tokens or "
               "cu_seqlens");
      nseqs = cu ? cu->numel() - 1 : na ? na->numel() : src ? src->size(0) : dst->size(0);
    }
    vector(cu, "cu_seqlens", nseqs + 1);
    vector(na, "num_accepted_tokens", nseqs);
    if (cu) meta = index_of(*cu, "cu_seqlens");
    if (na) {
      const ssu_dtype d = index_of(*na, "num_accepted_tokens");
      value_if(cu && d != meta, "cu_seqlens and num_accepted_tokens must share a dtype");
      meta = d;
    }
    if (src) index = index_of(*src, "state_batch_indices");
    if (dst) {
      const ssu_dtype d = index_of(*dst, "dst_state_batch_indices");
      value_if(src && d != index,
               "state_batch_indices and dst_state_batch_indices must share a dtype");
      index = d;
    }
    if (init) {
      vector(init, "has_initial_state", nseqs);
      value_if(init->scalar_type() != at::kBool && init->scalar_type() != at::kByte,
               "has_initial_state must be bool or uint8, got ", init->scalar_type());
    }
  }

  // f: the decode form, g: the prompt form of a call
  template <class P, class F, class G>
  ssu_status call(const P& p, int64_t rows, F f, G g, CUstream_st* stream) const {
    if (form == kPrompt)
      return g(&p, nseqs, rows, data(cu), meta, vector(src, "state_batch_indices", nseqs),
               vector(dst, "dst_state_batch_indices", nseqs), index,
               static_cast<const uint8_t*>(data(init)), stream);
    const bool one = form == kOneToken;
    const ssu_slot_table s = one ? slots_of(src, "state_batch_indices", nseqs)
                                 : table(src, "state_batch_indices", nseqs);
    const ssu_slot_table d = one ? slots_of(dst, "dst_state_batch_indices", nseqs)
                                 : table(dst, "dst_state_batch_indices", nseqs);
    return f(&p, nseqs, rows, data(cu), one ? 1 : steps, data(na), meta, &s, &d, index, stream);
  }
};

CUstream_st* stream_of(PyObject* o, int device) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
  return reinterpret_cast<CUstream_st*>((intptr_t)integer(o));
}

void done(ssu_status st) {
  if (st == SSU_OK) return;
  const char* what = ssu_last_error();
  if (!*what) what = ssu_status_string(st);
  if (st == SSU_ERR_INVALID_ARGUMENT) refuse(PyExc_ValueError, what);
  if (st == SSU_ERR_UNSUPPORTED) refuse(PyExc_NotImplementedError, what);
  refuse(PyExc_RuntimeError, "libssu_gb300: ", what);
}

// conv(form, conv_state, x, weight, bias, activation, cu, na, src, dst, init, pad, out, nseqs,
//      steps, disable, stream)
void conv(PyObject* const* a) {
  const Tensor* state = tensor(a[1], "conv_state");
  const Tensor &x = needed(a[2], "x"), &w = needed(a[3], "weight"), &out = needed(a[12], "out");
  const Tensor* bias = tensor(a[4], "bias");
  Seqs q(a[0], a + 6, a[13], a[14]);
  const int dev = one_device({&x, state, &w, bias, q.cu, q.na, q.src, q.dst, q.init, &out});
  value_if(x.dim() != 2, "x must be [rows, channels], got ", x.sizes());
  const int64_t rows = x.size(0), C = x.size(1);
  ssu_conv_params p{};
  p.io_dtype = float_of(x, "x");
  value_if(w.dim() != 2 || w.size(0) != C, "weight must be [", C, ", width], got ", w.sizes());
  value_if(!w.is_contiguous(), "weight must be contiguous");
  value_if(w.scalar_type() != x.scalar_type() && w.scalar_type() != at::kFloat, "weight must be ",
           x.scalar_type(), " or fp32, got ", w.scalar_type());
  const int64_t W = w.size(1);
  p.weight = w.data_ptr();
  p.weight_dtype = float_of(w, "weight");
  p.bias = vector(bias, "bias", C);
  value_if(bias && bias->scalar_type() != w.scalar_type(), "bias must have weight's dtype (",
           w.scalar_type(), "), got ", bias ? bias->scalar_type() : at::kFloat);
  if (state) {
    value_if(state->dim() != 3 || state->size(1) != W - 1 || state->size(2) != C,
             "conv_state must be [slots, ", W - 1, ", ", C, "], got ", state->sizes());
    value_if(state->scalar_type() != x.scalar_type(), "conv_state must be ", x.scalar_type(),
             ", got ", state->scalar_type());
    value_if(!state->is_contiguous(), "conv_state must be contiguous");
    p.conv_state = state->data_ptr();
    p.slots = state->size(0);
  }
  p.channels = C;
  p.width = W;
  p.x = x.data_ptr();
  p.x_row_stride = rows2(x, "x", rows, C);
  value_if(out.scalar_type() != x.scalar_type(), "out must be ", x.scalar_type(), ", got ",
           out.scalar_type());
  p.out = out.data_ptr();
  p.out_row_stride = rows2(out, "out", rows, C);
  p.activation = (int)integer(a[5]);
  p.pad_slot_id = integer(a[11]);
  p.disable_state_update = truth(a[15]);
  q.check(rows);
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  done(q.call(p, rows, ssu_conv_update, ssu_conv_fwd_varlen, stream_of(a[16], dev)));
}

// scan(form, state, x, dt, A, B, C, D, z, dt_bias, softplus, cu, na, src, dst, init, pad, out,
//      nseqs, steps, disable, stream)
void scan(PyObject* const* a) {
  const Tensor* state = tensor(a[1], "state");
  const Tensor &x = needed(a[2], "x"), &dt = needed(a[3], "dt"), &A = needed(a[4], "A");
  const Tensor &B = needed(a[5], "B"), &C = needed(a[6], "C"), &out = needed(a[17], "out");
  const Tensor *D = tensor(a[7], "D"), *z = tensor(a[8], "z"), *bias = tensor(a[9], "dt_bias");
  Seqs q(a[0], a + 11, a[18], a[19]);
  const int dev = one_device({&x, state, &dt, &A, &B, &C, D, z, bias, q.cu, q.na, q.src, q.dst,
                              q.init, &out});
  value_if(x.dim() != 2, "x must be [rows, channels], got ", x.sizes());
  const int64_t rows = x.size(0), dim = x.size(1);
  const auto io = x.scalar_type();
  ssu_scan_params p{};
  p.io_dtype = float_of(x, "x");
  value_if(A.dim() != 2 || A.size(0) != dim, "A must be [", dim, ", dstate], got ", A.sizes());
  unsupported_if(A.scalar_type() != at::kFloat, "A must be fp32, got ", A.scalar_type());
  const int64_t N = A.size(1);
  value_if(N > 1 && A.stride(1) != 1, "A must be contiguous along dstate");
  const int64_t nd = B.dim();
  value_if(B.sizes() != C.sizes() || (nd != 2 && nd != 3) || B.size(0) != rows ||
               B.size(nd - 1) != N,
           "B/C must be [", rows, ", groups, ", N, "] or [", rows, ", ", N, "]; got B=", B.sizes(),
           ", C=", C.sizes());
  value_if(B.scalar_type() != io || C.scalar_type() != io, "B and C must share the x dtype");
  value_if(N > 1 && (B.stride(nd - 1) != 1 || C.stride(nd - 1) != 1),
           "B and C must be contiguous along dstate");
  value_if(dt.scalar_type() != io && dt.scalar_type() != at::kFloat, "dt must be ", io,
           " or fp32, got ", dt.scalar_type());
  value_if(z && z->scalar_type() != io, "z must match x in shape and dtype");
  value_if(out.scalar_type() != io && out.scalar_type() != at::kFloat, "out must be ", io,
           " (or fp32), got ", out.scalar_type());
  p.D = static_cast<const float*>(vector(D, "D", dim));
  unsupported_if(D && D->scalar_type() != at::kFloat, "D must be fp32");
  p.dt_bias = static_cast<const float*>(vector(bias, "dt_bias", dim));
  unsupported_if(bias && bias->scalar_type() != at::kFloat, "dt_bias must be fp32");
  if (state) {
    value_if(state->dim() != 3 || state->size(1) != dim || state->size(2) != N,
             "state must be [slots, ", dim, ", ", N, "], got ", state->sizes());
    value_if(!state->is_contiguous(), "state must be contiguous");
    p.state = state->data_ptr();
    p.state_dtype = float_of(*state, "state");
    p.slots = state->size(0);
  }
  p.channels = dim;
  p.dstate = N;
  p.ngroups = nd == 3 ? B.size(1) : 1;
  p.x = x.data_ptr();
  p.x_row_stride = rows2(x, "x", rows, dim);
  if (z) {
    p.z = z->data_ptr();
    p.z_row_stride = rows2(*z, "z", rows, dim);
  }
  p.out = out.data_ptr();
  p.out_dtype = float_of(out, "out");
  p.out_row_stride = rows2(out, "out", rows, dim);
  p.dt = dt.data_ptr();
  p.dt_dtype = float_of(dt, "dt");
  p.dt_row_stride = rows2(dt, "dt", rows, dim);
  p.B = B.data_ptr();
  p.B_row_stride = B.stride(0);
  p.B_group_stride = nd == 3 ? B.stride(1) : N;
  p.C = C.data_ptr();
  p.C_row_stride = C.stride(0);
  p.C_group_stride = nd == 3 ? C.stride(1) : N;
  p.A = static_cast<const float*>(A.data_ptr());
  p.A_row_stride = A.stride(0);
  p.dt_softplus = truth(a[10]);
  p.pad_slot_id = integer(a[16]);
  p.disable_state_update = truth(a[20]);
  q.check(rows);
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  done(q.call(p, rows, ssu_scan_update, ssu_scan_fwd_varlen, stream_of(a[21], dev)));
}

// Pools [slots, ...] that share the slot ids, and the device that they and `others` are on.
struct Pools {
  std::vector<ssu_pool> pool;
  int64_t slots = 0;
  int device;

  Pools(PyObject* list, std::initializer_list<const Tensor*> others) {
    device = one_device(others);
    PyObject* seq = PySequence_Fast(list, "pools must be a sequence of tensors");
    if (!seq) throw Refused{nullptr, ""};
    struct Release {
      PyObject* o;
      ~Release() { Py_DECREF(o); }
    } release{seq};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    value_if(n == 0, "at least one pool is required");
    pool.reserve(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
      const Tensor& t = needed(PySequence_Fast_GET_ITEM(seq, i), "a pool");
      value_if(one_device({&t}) != device, "all tensors must be on one device");
      if (i == 0) slots = t.dim() ? t.size(0) : 0;
      value_if(t.dim() < 1 || t.size(0) != slots, "pool ", i, " must hold ", slots,
               " slots like the first, got ", t.sizes());
      const int64_t es = t.element_size(), per = slots ? t.numel() / slots : 0;
      int64_t stride = per;
      if (!t.is_contiguous()) {
        int64_t inner = 1;  // of a slot, from its last dimension
        for (int64_t k = t.dim() - 1; k > 0; --k) {
          value_if(t.size(k) > 1 && t.stride(k) != inner, "pool ", i, ": a slot must be contiguous");
          inner *= t.size(k);
        }
        stride = t.stride(0);
      }
      pool.push_back(ssu_pool{t.data_ptr(), per * es, stride * es});
    }
  }
};

const void* ids_of(const Tensor& t, const char* name, ssu_dtype* d) {
  *d = index_of(t, name);
  return vector(&t, name, t.numel());
}

// slots_copy(pools, src, dst, pad, stream)
void slots_copy(PyObject* const* a) {
  const Tensor &src = needed(a[1], "src"), &dst = needed(a[2], "dst");
  const Pools p(a[0], {&src, &dst});
  ssu_dtype d, dd;
  const void *s = ids_of(src, "src", &d), *t = ids_of(dst, "dst", &dd);
  value_if(d != dd || src.numel() != dst.numel(), "src and dst must share their length and dtype");
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)p.device));
  done(ssu_slots_copy(p.pool.data(), (int)p.pool.size(), p.slots, s, t, d, src.numel(),
                      integer(a[3]), stream_of(a[4], p.device)));
}

// slots_clear(pools, ids, pad, stream)
void slots_clear(PyObject* const* a) {
  const Tensor& ids = needed(a[1], "slots");
  const Pools p(a[0], {&ids});
  ssu_dtype d;
  const void* s = ids_of(ids, "slots", &d);
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)p.device));
  done(ssu_slots_clear(p.pool.data(), (int)p.pool.size(), p.slots, s, d, ids.numel(),
                       integer(a[2]), stream_of(a[3], p.device)));
}

// slots_compact(pools, table, out, num_live, workspace, pad, stream)
void slots_compact(PyObject* const* a) {
  const Tensor &t = needed(a[1], "table"), &out = needed(a[2], "out");
  const Tensor& live = needed(a[3], "num_live");
  const Tensor* ws = tensor(a[4], "workspace");
  const Pools p(a[0], {&t, &out, &live, ws});
  const ssu_dtype d = index_of(t, "table");
  value_if(!t.is_contiguous(), "table must be contiguous");
  value_if(out.sizes() != t.sizes() || out.scalar_type() != t.scalar_type() ||
               !out.is_contiguous(),
           "out must match table's shape and dtype");
  value_if(live.scalar_type() != at::kInt || live.numel() != 1, "num_live must be one int32");
  value_if(ws && !ws->is_contiguous(), "workspace must be contiguous");
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)p.device));
  done(ssu_slots_compact(p.pool.data(), (int)p.pool.size(), p.slots, t.data_ptr(), out.data_ptr(),
                         d, t.numel(), integer(a[5]), static_cast<int32_t*>(live.data_ptr()),
                         ws ? ws->data_ptr() : nullptr, ws ? (int64_t)ws->nbytes() : 0,
                         stream_of(a[6], p.device)));
}

template <void (*F)(PyObject* const*), int ARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != ARGS) {
    PyErr_Format(PyExc_TypeError, "%d arguments are needed, got %zd", ARGS, n);
    return nullptr;
  }
  try {
    F(args);
    Py_RETURN_NONE;
  } catch (const Refused& r) {
    if (r.type) PyErr_SetString(r.type, r.what.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <void (*F)(PyObject* const*), int ARGS>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, ARGS>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<conv, 17>("conv"),
                         method<scan, 22>("scan"),
                         method<slots_copy, 5>("slots_copy"),
                         method<slots_clear, 4>("slots_clear"),
                         method<slots_compact, 7>("slots_compact"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_binding(void) { return PyModule_Create(&module); }
