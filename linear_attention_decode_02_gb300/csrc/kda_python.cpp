// CPython side of the binding for the calls of a decode step that follow one
// another too quickly for ctypes: it turns torch tensors into kda_tensor
// descriptors, allocates what the caller gives no tensor for, and calls the
// library on the current stream of the tensors' device.
//
// A call of a small step keeps the GPU busy for 2 to 9 us; its host time, on
// the Grace host, was 13 to 23 us through ctypes, of which describing a tensor
// took 1.1 us (7 to 11 of them) and allocating one through Python 2 us.
//
// The library is reached through the addresses that bind() is given.  A call
// returns its result, or the library's status as an int where that is not 0.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/cuda/CUDAContextLight.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/record_function.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstring>

#include "../../include/kda.h"

namespace {

struct Library {
  decltype(&kda_rope_append) rope_append;
  decltype(&kda_paged_attention_decode) attention;
  decltype(&kda_paged_attention_workspace) attention_workspace;
  decltype(&kda_beam_select) beam;
  decltype(&kda_beam_select_workspace) beam_workspace;
  decltype(&kda_pool_move) move;
  decltype(&kda_page_assign) page_assign;
  decltype(&kda_rope_axes_append) rope_axes;
  decltype(&kda_prefix_attention_decode) prefix;
  decltype(&kda_prefix_attention_workspace) prefix_workspace;
} lib;

// A Python exception is set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(type, fmt, ap);
  va_end(ap);
  throw Raised();
}

// Runs a call's body; C++ exceptions become Python's.
template <typename Body>
PyObject* guarded(const Body& body) {
  try {
    return body();
  } catch (const Raised&) {
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

void need_arity(const char* name, Py_ssize_t got, Py_ssize_t want) {
  if (got != want) raise(PyExc_TypeError, "%s takes %zd arguments, not %zd", name, want, got);
}

const at::Tensor& tensor_of(PyObject* o) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "expected a tensor, got %s", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

int64_t int64_of(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
int32_t int32_of(PyObject* o) {
  const int64_t v = int64_of(o);
  if (v > INT32_MAX || v < INT32_MIN) raise(PyExc_OverflowError, "argument does not fit 32 bits");
  return static_cast<int32_t>(v);
}
float float_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return static_cast<float>(v);
}
bool truth_of(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

int32_t dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return KDA_F32;
    case at::kBFloat16: return KDA_BF16;
    case at::kInt: return KDA_I32;
    default: raise(PyExc_TypeError, "unsupported dtype %s", c10::toString(t.scalar_type()));
  }
}

void describe(const at::Tensor& t, kda_tensor* d) {
  if (t.layout() != at::kStrided) raise(PyExc_TypeError, "expected a strided tensor");
  if (t.dim() < 1 || t.dim() > 4) raise(PyExc_ValueError, "rank %d not in 1..4", static_cast<int>(t.dim()));
  std::memset(d, 0, sizeof(*d));
  d->dtype = dtype_of(t);
  d->ndim = static_cast<int32_t>(t.dim());
  for (int i = 0; i < d->ndim; ++i) {
    d->shape[i] = t.size(i);
    d->stride[i] = t.stride(i);
  }
  d->data = t.numel() > 0 ? t.data_ptr() : nullptr;
}

// Whether at::empty would go straight to its CUDA function: no mode or transform has
// put a dispatch key of its own in the way, no profiler listens, and nothing is to be
// filled for determinism.
bool plain_allocation() {
  const c10::impl::LocalDispatchKeySet keys = c10::impl::tls_local_dispatch_key_set();
  return keys.included_ == c10::default_included_set && keys.excluded_ == c10::default_excluded_set &&
         !at::hasCallbacks() && !at::globalContext().deterministicAlgorithms();
}

// The device and stream of a call: those of its first tensor, and the device
// made the current one.  A tensor of the host or of another device is
// refused: its address would mean something else, or nothing, to the kernels.
struct Call {
  c10::cuda::OptionalCUDAGuard guard;
  c10::Device device;
  void* stream;
  explicit Call(const at::Tensor& first) : device(first.device()) {
    check(first);
    guard.set_index(device.index());
    stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
  }
  void check(const at::Tensor& t) const {
    if (!t.is_cuda()) raise(PyExc_ValueError, "expected CUDA tensors, got one of the host");
    if (t.device() != device)
      raise(PyExc_ValueError, "expected every tensor on cuda:%d, got one on cuda:%d", static_cast<int>(device.index()),
            static_cast<int>(t.device().index()));
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    // at::empty without its dispatch, 0.5 us a tensor (page assignment of 8 sequences 8.5 -> 6.7 us a call), where that is the same
    if (plain_allocation()) return at::detail::empty_cuda(shape, type, device, std::nullopt);
    return at::empty(shape, at::TensorOptions().dtype(type).device(device));
  }
  int sms() const { return at::cuda::getDeviceProperties(device.index())->multiProcessorCount; }
};

// Descriptors of a call's tensors; None is a null one.
template <int N>
struct Described {
  kda_tensor d[N];
  const kda_tensor* p[N];
  int n = 0;
  void add(const Call& call, PyObject* o) {
    if (o == Py_None) {
      p[n++] = nullptr;
    } else {
      add(call, tensor_of(o));
    }
  }
  void add(const Call& call, const at::Tensor& t) {
    call.check(t);
    describe(t, &d[n]);
    p[n] = &d[n];
    ++n;
  }
};

template <typename F>
kda_status without_gil(const F& f) {
  PyThreadState* state = PyEval_SaveThread();
  const kda_status s = f();
  PyEval_RestoreThread(state);
  return s;
}

// Workspaces of the calls that are given none.  One is kept for each host
// thread (in its thread state's dictionary), device and stream: calls of one
// thread on one stream follow one another, and no other call sees it.  A call
// that is being captured gets its own from the graph's pool, so graphs share
// theirs neither with each other nor with eager calls.  One of more than 16 MB
// (the paged attention's never is, beams' only over tens of thousands of rows, that of
// attention under shared prefixes mostly; such calls take far longer than allocating it)
// goes back to the allocator with the call.
constexpr Py_ssize_t kKept = 16;
constexpr int64_t kKeptFloats = 4 << 20;
PyObject* s_workspaces;

at::Tensor workspace(const Call& call, PyObject* given, int64_t floats) {
  if (given != Py_None) return tensor_of(given);
  if (floats > kKeptFloats || c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
    return call.empty({floats}, at::kFloat);
  PyObject* state = PyThreadState_GetDict();  // borrowed
  if (state == nullptr) return call.empty({floats}, at::kFloat);
  PyObject* kept = PyDict_GetItemWithError(state, s_workspaces);  // borrowed
  if (kept == nullptr) {
    if (PyErr_Occurred()) throw Raised();
    kept = PyDict_New();
    if (kept == nullptr) throw Raised();
    const int bad = PyDict_SetItem(state, s_workspaces, kept);
    Py_DECREF(kept);
    if (bad != 0) throw Raised();
  }
  // Stream handles are addresses, or one of CUDA's few small ones: 64 devices fit below them.
  PyObject* key = PyLong_FromUnsignedLongLong(reinterpret_cast<uintptr_t>(call.stream) * 64 + call.device.index());
  if (key == nullptr) throw Raised();
  PyObject* held = PyDict_GetItemWithError(kept, key);  // borrowed
  if (held != nullptr) {
    const at::Tensor& t = THPVariable_Unpack(held);
    if (t.numel() >= floats) {
      Py_DECREF(key);
      return t;
    }
  } else if (PyErr_Occurred()) {
    Py_DECREF(key);
    throw Raised();
  }
  // Past the dispatcher: what a mode gives instead, a tensor without memory say, is not for other calls.
  at::Tensor t = at::detail::empty_cuda({floats}, at::kFloat, call.device, std::nullopt);
  if (held == nullptr && PyDict_Size(kept) >= kKept) PyDict_Clear(kept);
  PyObject* wrapped = THPVariable_Wrap(t);
  const int bad = wrapped == nullptr ? -1 : PyDict_SetItem(kept, key, wrapped);
  Py_XDECREF(wrapped);
  Py_DECREF(key);
  if (bad != 0) throw Raised();
  return t;
}

// The given tensor as a new reference, or the one allocated in its place.
PyObject* result(PyObject* given, const at::Tensor& made) {
  if (given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  return THPVariable_Wrap(made);
}

// rope_append(q, k, v, phase_steps, cu_seqlens, seq_lens, page_table, k_pages, v_pages, q_out, interleaved, amplitude)
PyObject* rope_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_arity("rope_append", n, 12);
    const at::Tensor& q = tensor_of(args[0]);
    const Call call(q);
    Described<10> t;
    for (int i = 0; i < 9; ++i) t.add(call, args[i]);
    at::Tensor made;
    if (args[9] == Py_None) {
      made = call.empty(q.sizes(), tensor_of(args[7]).scalar_type());
      t.add(call, made);
    } else {
      t.add(call, args[9]);
    }
    const int32_t interleaved = truth_of(args[10]) ? 1 : 0;
    const float amplitude = float_of(args[11]);
    const kda_status s = without_gil([&] {
      return lib.rope_append(t.p[0], t.p[1], t.p[2], t.p[3], t.p[4], t.p[5], t.p[6], t.p[7], t.p[8], t.p[9], interleaved,
                             amplitude, call.stream);
    });
    return s != KDA_OK ? PyLong_FromLong(s) : result(args[9], made);
  });
}

// rope_axes_append(q, k, v, phase_steps, pair_axes, positions, slots, k_pages, v_pages, q_out, interleaved, amplitude)
PyObject* rope_axes_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_arity("rope_axes_append", n, 12);
    const at::Tensor& q = tensor_of(args[0]);
    const Call call(q);
    Described<10> t;
    for (int i = 0; i < 9; ++i) t.add(call, args[i]);
    at::Tensor made;
    if (args[9] == Py_None) {
      made = call.empty(q.sizes(), tensor_of(args[7]).scalar_type());
      t.add(call, made);
    } else {
      t.add(call, args[9]);
    }
    const int32_t interleaved = truth_of(args[10]) ? 1 : 0;
    const float amplitude = float_of(args[11]);
    const kda_status s = without_gil([&] {
      return lib.rope_axes(t.p[0], t.p[1], t.p[2], t.p[3], t.p[4], t.p[5], t.p[6], t.p[7], t.p[8], t.p[9], interleaved,
                           amplitude, call.stream);
    });
    return s != KDA_OK ? PyLong_FromLong(s) : result(args[9], made);
  });
}

// page_assign(seq_lens, new_lens, shared_lens, page_table, free_pages, free_state, page_size, rows, lens_out, state_out,
// cu_seqlens, slots): the last four as a tuple
PyObject* page_assign(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_arity("page_assign", n, 12);
    const at::Tensor& lens = tensor_of(args[0]);
    const Call call(lens);
    Described<10> t;
    for (int i = 0; i < 6; ++i) t.add(call, args[i]);
    const int32_t page_size = int32_of(args[6]), rows = int32_of(args[7]);
    if (rows < 0) raise(PyExc_ValueError, "rows must not be negative");
    const int64_t N = lens.size(0);  // rank 1 at least: the descriptor's check
    const int64_t size[4] = {N, 2, N + 1, rows};
    at::Tensor made[4];
    for (int i = 0; i < 4; ++i) {
      if (args[8 + i] == Py_None) {
        made[i] = call.empty({size[i]}, at::kInt);
        t.add(call, made[i]);
      } else {
        const at::Tensor& given = tensor_of(args[8 + i]);
        if (i == 3 && (given.dim() != 1 || given.size(0) != rows))
          raise(PyExc_ValueError, "slots must be of [rows], rows is %d", static_cast<int>(rows));
        t.add(call, given);
      }
    }
    const kda_status s = without_gil([&] {
      return lib.page_assign(t.p[0], t.p[1], t.p[2], t.p[3], t.p[4], t.p[5], page_size, t.p[6], t.p[7], t.p[8], t.p[9],
                             call.stream);
    });
    if (s != KDA_OK) return PyLong_FromLong(s);
    PyObject* four = PyTuple_New(4);
    for (int i = 0; i < 4 && four != nullptr; ++i) {
      PyObject* o = result(args[8 + i], made[i]);
      if (o == nullptr) {
        Py_DECREF(four);
        return nullptr;
      }
      PyTuple_SET_ITEM(four, i, o);
    }
    return four;
  });
}

// The attention calls; `starts` and `prefixes` null without shared prefixes.
PyObject* attend(PyObject* const* five, PyObject* starts, PyObject* prefixes, PyObject* given_work, PyObject* given_out,
                 PyObject* given_lse, bool both, int32_t window, PyObject* given_scale) {
  const at::Tensor &q = tensor_of(five[0]), &k = tensor_of(five[1]);
  const Call call(q);
  const bool shared = starts != nullptr;
  Described<10> t;
  for (int i = 0; i < 5; ++i) t.add(call, five[i]);
  if (shared) {
    t.add(call, starts);
    t.add(call, prefixes);
  }
  if (q.dim() != 3 || k.dim() != 4) raise(PyExc_ValueError, "q must be [N, Hq, D] and the pages of rank 4");
  int64_t floats = 0;
  if (given_work == Py_None) {
    const auto small = [](int64_t x) { return static_cast<int32_t>(std::min<int64_t>(x, INT32_MAX)); };
    const int32_t hq = small(q.size(1)), hkv = small(k.size(2)), d = small(q.size(2)), dtype = dtype_of(q);
    const kda_status s = shared ? lib.prefix_workspace(q.size(0), hq, hkv, d, dtype, call.sms(), &floats)
                                : lib.attention_workspace(hq, hkv, d, dtype, call.sms(), &floats);
    if (s != KDA_OK) return PyLong_FromLong(s);
  }
  const at::Tensor work = workspace(call, given_work, floats);
  t.add(call, work);
  at::Tensor out, lse;
  if (given_out == Py_None) {
    out = call.empty(q.sizes(), at::kBFloat16);
    t.add(call, out);
  } else {
    t.add(call, given_out);
  }
  if (given_lse == Py_None && both) {
    lse = call.empty({q.size(0), q.size(1)}, at::kFloat);
    t.add(call, lse);
  } else {
    t.add(call, given_lse);
  }
  const float scale = given_scale == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(q.size(2))))
                                             : float_of(given_scale);
  const kda_status s = without_gil([&] {
    return shared ? lib.prefix(t.p[0], t.p[1], t.p[2], t.p[3], t.p[4], t.p[5], t.p[6], t.p[7], window, scale, t.p[8],
                               t.p[9], call.stream)
                  : lib.attention(t.p[0], t.p[1], t.p[2], t.p[3], t.p[4], t.p[5], window, scale, t.p[6], t.p[7],
                                  call.stream);
  });
  if (s != KDA_OK) return PyLong_FromLong(s);
  PyObject* o = result(given_out, out);
  if (!both || o == nullptr) return o;
  PyObject* e = result(given_lse, lse);
  PyObject* pair = e != nullptr ? PyTuple_Pack(2, o, e) : nullptr;
  Py_DECREF(o);
  Py_XDECREF(e);
  return pair;
}

// attention(q, k_pages, v_pages, page_table, seq_lens, workspace, out, lse, return_lse, window, scale or None)
PyObject* attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_arity("attention", n, 11);
    return attend(args, nullptr, nullptr, args[5], args[6], args[7], truth_of(args[8]), int32_of(args[9]), args[10]);
  });
}

// prefix_attention(q, k_pages, v_pages, page_table, seq_lens, group_starts, prefix_lens, workspace, out, lse, return_lse,
// window, scale or None)
PyObject* prefix_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_arity("prefix_attention", n, 13);
    return attend(args, args[5], args[6], args[7], args[8], args[9], truth_of(args[10]), int32_of(args[11]), args[12]);
  });
}

// beam(logits, scores, finished, workspace, out or None, num_out, eos_token); out a tuple of three tensors
PyObject* beam(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_arity("beam", n, 7);
    const at::Tensor& x = tensor_of(args[0]);
    const Call call(x);
    Described<7> t;
    for (int i = 0; i < 3; ++i) t.add(call, args[i]);
    if (x.dim() != 3) raise(PyExc_ValueError, "logits must be [N, B, V]");
    const int32_t num_out = int32_of(args[5]), eos = int32_of(args[6]);
    PyObject* given[3] = {Py_None, Py_None, Py_None};
    if (args[4] != Py_None) {
      if (!PyTuple_Check(args[4]) || PyTuple_GET_SIZE(args[4]) != 3)
        raise(PyExc_TypeError, "out must be a tuple of three tensors");
      for (int i = 0; i < 3; ++i) given[i] = PyTuple_GET_ITEM(args[4], i);
      // The library goes by the tensors; a workspace for num_out might be too small for them, or they for num_out.
      for (PyObject* o : given) {
        const at::Tensor& t = tensor_of(o);
        if (t.dim() != 2 || t.size(1) != num_out)
          raise(PyExc_ValueError, "out must be of [N, num_out] tensors, num_out is %d", static_cast<int>(num_out));
      }
    }
    int64_t floats = 0;  // refuses sizes before anything of them is allocated
    const kda_status sizes = lib.beam_workspace(x.size(0), static_cast<int32_t>(std::min<int64_t>(x.size(1), INT32_MAX)),
                                                x.size(2), num_out, dtype_of(x), call.sms(), &floats);
    if (sizes != KDA_OK) return PyLong_FromLong(sizes);
    const at::Tensor work = workspace(call, args[3], floats);
    t.add(call, work);
    at::Tensor made[3];
    for (int i = 0; i < 3; ++i) {
      if (args[4] == Py_None) {
        made[i] = call.empty({x.size(0), num_out}, i == 0 ? at::kFloat : at::kInt);
        t.add(call, made[i]);
      } else {
        t.add(call, tensor_of(given[i]));
      }
    }
    const kda_status s = without_gil([&] {
      return lib.beam(t.p[0], t.p[1], t.p[2], eos, t.p[3], t.p[4], t.p[5], t.p[6], call.stream);
    });
    if (s != KDA_OK) return PyLong_FromLong(s);
    if (args[4] != Py_None) {
      Py_INCREF(args[4]);
      return args[4];
    }
    PyObject* three = PyTuple_New(3);
    for (int i = 0; i < 3 && three != nullptr; ++i) {
      PyObject* o = THPVariable_Wrap(made[i]);
      if (o == nullptr) {
        Py_DECREF(three);
        return nullptr;
      }
      PyTuple_SET_ITEM(three, i, o);
    }
    return three;
  });
}

// move(pools, src_slots, dst_slots, parents); pools a list or tuple (more than 256 are refused by the library, from the
// count alone)
PyObject* move(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_arity("move", n, 4);
    constexpr Py_ssize_t MOST = 256;
    if (!PyList_Check(args[0]) && !PyTuple_Check(args[0]))  // a tensor would pass for the sequence of its rows
      raise(PyExc_TypeError, "pools must be a list or tuple of tensors");
    const Call call(tensor_of(args[1]));
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(args[0]);
    kda_tensor pool[MOST];
    const kda_tensor* pools[MOST];
    for (Py_ssize_t i = 0; i < count && i < MOST; ++i) {
      const at::Tensor& p = tensor_of(PySequence_Fast_GET_ITEM(args[0], i));
      call.check(p);
      describe(p, &pool[i]);
      pools[i] = &pool[i];
    }
    Described<3> t;
    for (int i = 1; i < 4; ++i) t.add(call, args[i]);
    const kda_status s = without_gil([&] {
      return lib.move(pools, count > MOST ? static_cast<int32_t>(MOST) + 1 : static_cast<int32_t>(count), t.p[0], t.p[1],
                      t.p[2], call.stream);
    });
    if (s != KDA_OK) return PyLong_FromLong(s);
    Py_RETURN_NONE;
  });
}

// describe(tensor): the bytes of its descriptor
PyObject* describe_bytes(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_arity("describe", n, 1);
    kda_tensor d;
    describe(tensor_of(args[0]), &d);
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&d), sizeof(d));
  });
}

// bind(addresses of rope_append, attention, attention_workspace, beam, beam_workspace, move, page_assign, rope_axes,
// prefix, prefix_workspace)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    constexpr Py_ssize_t COUNT = 10;
    need_arity("bind", n, COUNT);
    void* address[COUNT];
    for (Py_ssize_t i = 0; i < COUNT; ++i) {
      address[i] = PyLong_AsVoidPtr(args[i]);
      if (address[i] == nullptr) {
        if (PyErr_Occurred()) throw Raised();
        raise(PyExc_ValueError, "null address");
      }
    }
    lib.rope_append = reinterpret_cast<decltype(lib.rope_append)>(address[0]);
    lib.attention = reinterpret_cast<decltype(lib.attention)>(address[1]);
    lib.attention_workspace = reinterpret_cast<decltype(lib.attention_workspace)>(address[2]);
    lib.beam = reinterpret_cast<decltype(lib.beam)>(address[3]);
    lib.beam_workspace = reinterpret_cast<decltype(lib.beam_workspace)>(address[4]);
    lib.move = reinterpret_cast<decltype(lib.move)>(address[5]);
    lib.page_assign = reinterpret_cast<decltype(lib.page_assign)>(address[6]);
    lib.rope_axes = reinterpret_cast<decltype(lib.rope_axes)>(address[7]);
    lib.prefix = reinterpret_cast<decltype(lib.prefix)>(address[8]);
    lib.prefix_workspace = reinterpret_cast<decltype(lib.prefix_workspace)>(address[9]);
    Py_RETURN_NONE;
  });
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"rope_append", fast(rope_append), METH_FASTCALL, nullptr},
                         {"attention", fast(attention), METH_FASTCALL, nullptr},
                         {"beam", fast(beam), METH_FASTCALL, nullptr},
                         {"move", fast(move), METH_FASTCALL, nullptr},
                         {"rope_axes_append", fast(rope_axes_append), METH_FASTCALL, nullptr},
                         {"page_assign", fast(page_assign), METH_FASTCALL, nullptr},
                         {"prefix_attention", fast(prefix_attention), METH_FASTCALL, nullptr},
                         {"describe", fast(describe_bytes), METH_FASTCALL, nullptr},
                         {"bind", fast(bind), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef definition = {PyModuleDef_HEAD_INIT, "_kda_python", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_python() {
  s_workspaces = PyUnicode_InternFromString("linear_attention_decode_02_gb300 workspaces");
  if (s_workspaces == nullptr) return nullptr;
  return PyModule_Create(&definition);
}
