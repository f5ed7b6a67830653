// The short way from Python to the prompt calls of the convolution and the scan and to
// the product: their tensors are looked at in C++ (25 ns a tensor, where Python's
// attributes take 500), the struct is filled and the library called, without the
// interpreter's lock.  Each function takes a call only where everything is as the
// library wants it, and otherwise returns None and leaves it to the checks in api.py,
// which say what is wrong or do what is rarer (a workspace, another current device).
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "../../include/kda.h"

namespace {

int (*conv_prompt)(const kda_conv_prompt_args *, void *);
int64_t (*ssm_workspace)(const kda_ssm_prompt_args *);
int (*ssm_prompt)(const kda_ssm_prompt_args *, void *);
int (*linear)(const kda_linear_args *, void *);

constexpr int64_t kMost = INT32_MAX;

// What a call's tensors have to agree on; `ok` falls where one does not.
struct Look {
  int index = -1;
  bool ok = true;

  const at::Tensor *tensor(PyObject *o) {
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || (index >= 0 && t.get_device() != index)) ok = false;
    if (index < 0) index = t.get_device();
    return &t;
  }
  // BF16 rows: [rows, width], 2^31 - 1 of each at most, `stride` elements apart.
  void *rows(PyObject *o, int64_t rows, int64_t width, int64_t *stride) {
    const at::Tensor *t = tensor(o);
    if (!ok || t->scalar_type() != at::kBFloat16 || t->dim() != 2 || t->size(0) != rows ||
        t->size(1) != width || width < 1 || rows > kMost || width > kMost)
      return fail();
    *stride = rows > 1 ? t->stride(0) : (width + 7) / 8 * 8;
    if ((t->stride(1) != 1 && width > 1) || *stride % 8 != 0 || *stride < width) return fail();
    return t->data_ptr();
  }
  // A contiguous tensor of these sizes (-1: any).
  void *whole(PyObject *o, at::ScalarType type, std::initializer_list<int64_t> sizes) {
    const at::Tensor *t = tensor(o);
    if (!ok || t->scalar_type() != type || t->dim() != static_cast<int64_t>(sizes.size()) ||
        !t->is_contiguous())
      return fail();
    int64_t i = 0;
    for (const int64_t n : sizes) {
      if ((n >= 0 && t->size(i) != n) || t->size(i) > kMost) return fail();
      ++i;
    }
    return t->data_ptr();
  }
  void *maybe(PyObject *o, at::ScalarType type, std::initializer_list<int64_t> sizes) {
    return o == Py_None ? nullptr : whole(o, type, sizes);
  }
  int32_t *words(PyObject *o) {                    // the error word, of any shape
    if (o == Py_None) return nullptr;
    const at::Tensor *t = tensor(o);
    if (!ok || t->scalar_type() != at::kInt || !t->is_contiguous()) return static_cast<int32_t *>(fail());
    return static_cast<int32_t *>(t->data_ptr());
  }
  int64_t size(PyObject *o, int64_t dim, int64_t of) {
    const at::Tensor *t = tensor(o);
    if (!ok || t->dim() != of) {
      fail();
      return 0;
    }
    return t->size(dim);
  }
  void *fail() {
    ok = false;
    return nullptr;
  }
  // The stream that was asked for, or the current one of the tensors' device, which has
  // to be the current device.
  bool stream(PyObject *o, void **handle) {
    if (!ok || c10::cuda::current_device() != index) return false;
    if (o == Py_None) {
      *handle = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
      return true;
    }
    PyObject *device = PyObject_GetAttrString(o, "device_index");
    PyObject *stream = device ? PyObject_GetAttrString(o, "cuda_stream") : nullptr;
    const bool there = stream && PyLong_AsLong(device) == index;
    if (there) *handle = PyLong_AsVoidPtr(stream);
    Py_XDECREF(device);
    Py_XDECREF(stream);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return false;
    }
    return there;
  }
};

template <class Args>
PyObject *launched(int (*entry)(const Args *, void *), const Args &args, void *stream) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = entry(&args, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

// Runs `call`; None where it does not take the arguments or PyTorch throws (the way
// through api.py meets the same and says so).
template <class Call>
PyObject *taken(Py_ssize_t n, Py_ssize_t want, Call call) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    if (PyObject *done = call()) return done;
  } catch (const std::exception &) {
  }
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

// x, weight, output, bias, residual, activation, err, stream
PyObject *py_linear(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return taken(n, 8, [&]() -> PyObject * {
    Look look;
    kda_linear_args a = {};
    const int64_t rows = look.size(o[0], 0, 2), inner = look.ok ? look.size(o[0], 1, 2) : 0;
    const int64_t outer = look.ok ? look.size(o[1], 0, 2) : 0;
    if (!look.ok) return nullptr;
    a.x = look.rows(o[0], rows, inner, &a.x_stride);
    a.weight = look.rows(o[1], outer, inner, &a.w_stride);
    a.output = look.rows(o[2], rows, outer, &a.o_stride);
    a.bias = look.maybe(o[3], at::kBFloat16, {outer});
    if (o[4] != Py_None) a.residual = look.rows(o[4], rows, outer, &a.r_stride);
    a.err = look.words(o[6]);
    void *stream;
    if (!look.stream(o[7], &stream)) return nullptr;
    a.rows = static_cast<int32_t>(rows);
    a.inner = static_cast<int32_t>(inner);
    a.outer = static_cast<int32_t>(outer);
    a.activation = static_cast<int32_t>(PyLong_AsLong(o[5]));
    return launched(linear, a, stream);
  });
}

// The sequences of a prompt call: their number, starts and slots.
template <class Args>
void sequences(Look *look, Args *a, PyObject *starts, PyObject *src, PyObject *dst) {
  const int64_t n = look->size(starts, 0, 1) - 1;
  if (n < 0) look->fail();
  a->seq_starts = static_cast<const int32_t *>(look->whole(starts, at::kInt, {n + 1}));
  a->src_slots = static_cast<const int32_t *>(look->maybe(src, at::kInt, {n}));
  a->dst_slots = static_cast<const int32_t *>(look->maybe(dst, at::kInt, {n}));
  a->seqs = static_cast<int32_t>(n);
}

// x, weight, seq_starts, output, bias, window, src_slots, dst_slots, silu, err, stream
PyObject *py_conv_prompt(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return taken(n, 11, [&]() -> PyObject * {
    Look look;
    kda_conv_prompt_args a = {};
    const int64_t rows = look.size(o[0], 0, 2), channels = look.ok ? look.size(o[0], 1, 2) : 0;
    const at::Tensor *w = look.ok ? look.tensor(o[1]) : nullptr;
    if (!look.ok || (w->dim() != 2 && w->dim() != 3)) return nullptr;
    const bool blocks = w->dim() == 3;
    const int64_t parts = blocks ? w->size(0) : 1, taps = w->size(blocks), wide = w->size(blocks + 1);
    if (parts < 1 || parts > kMost || taps > kMost || wide > kMost || parts * wide != channels) return nullptr;
    a.weight = blocks ? look.whole(o[1], at::kBFloat16, {parts, taps, wide})
                      : look.whole(o[1], at::kBFloat16, {taps, wide});
    a.x = look.rows(o[0], rows, channels, &a.x_stride);
    a.output = look.rows(o[3], rows, channels, &a.o_stride);
    if (!look.ok) return nullptr;
    sequences(&look, &a, o[2], o[6], o[7]);
    a.bias = look.maybe(o[4], at::kBFloat16, {channels});
    if (o[5] == Py_None) {
      if (a.src_slots || a.dst_slots) return nullptr;
    } else {
      const at::Tensor *window = look.tensor(o[5]);
      if (!look.ok) return nullptr;
      a.window_f32 = window->scalar_type() == at::kFloat;
      a.window = look.whole(o[5], a.window_f32 ? at::kFloat : at::kBFloat16, {-1, channels, -1});
      if (!look.ok) return nullptr;
      a.num_slots = static_cast<int32_t>(window->size(0));
      a.width = static_cast<int32_t>(window->size(2));
    }
    a.err = look.words(o[9]);
    void *stream;
    if (!look.stream(o[10], &stream)) return nullptr;
    a.channels = static_cast<int32_t>(channels);
    a.parts = static_cast<int32_t>(parts);
    a.taps = static_cast<int32_t>(taps);
    a.tokens = static_cast<int32_t>(rows);
    a.silu = o[8] == Py_True;
    return launched(conv_prompt, a, stream);
  });
}

// x, dt, a, b, c, seq_starts, output, d, z, dt_bias, softplus, state, src_slots,
// dst_slots, max_seq (or None), err, path, stream
PyObject *py_ssm_prompt(PyObject *, PyObject *const *o, Py_ssize_t n) {
  return taken(n, 18, [&]() -> PyObject * {
    Look look;
    kda_ssm_prompt_args a = {};
    const int64_t rows = look.size(o[0], 0, 2), channels = look.ok ? look.size(o[0], 1, 2) : 0;
    const int64_t states = look.ok ? look.size(o[2], 1, 2) : 0, wide = look.ok ? look.size(o[3], 1, 2) : 0;
    if (!look.ok || states < 1 || wide < states || wide % states != 0) return nullptr;
    a.x = look.rows(o[0], rows, channels, &a.x_stride);
    a.dt = look.rows(o[1], rows, channels, &a.dt_stride);
    a.a = static_cast<const float *>(look.whole(o[2], at::kFloat, {channels, states}));
    a.b = look.rows(o[3], rows, wide, &a.b_stride);
    a.c = look.rows(o[4], rows, wide, &a.c_stride);
    a.output = look.rows(o[6], rows, channels, &a.o_stride);
    a.d = static_cast<const float *>(look.maybe(o[7], at::kFloat, {channels}));
    if (o[8] != Py_None) a.z = look.rows(o[8], rows, channels, &a.z_stride);
    a.dt_bias = static_cast<const float *>(look.maybe(o[9], at::kFloat, {channels}));
    if (!look.ok) return nullptr;
    sequences(&look, &a, o[5], o[12], o[13]);
    if (o[11] == Py_None) {
      if (a.src_slots || a.dst_slots) return nullptr;
    } else {
      a.state = static_cast<float *>(look.whole(o[11], at::kFloat, {-1, channels, states}));
      if (!look.ok) return nullptr;
      a.num_slots = static_cast<int32_t>(THPVariable_Unpack(o[11]).size(0));
    }
    a.err = look.words(o[15]);
    void *stream;
    if (!look.stream(o[17], &stream)) return nullptr;
    a.channels = static_cast<int32_t>(channels);
    a.states = static_cast<int32_t>(states);
    a.groups = static_cast<int32_t>(wide / states);
    a.tokens = static_cast<int32_t>(rows);
    a.max_seq = a.tokens;
    if (o[14] != Py_None) {
      if (!PyLong_CheckExact(o[14])) return nullptr;
      const int64_t most = PyLong_AsLongLong(o[14]);
      if (PyErr_Occurred()) {
        PyErr_Clear();
        return nullptr;
      }
      if (most < rows) a.max_seq = most < 0 ? -1 : static_cast<int32_t>(most);
    }
    a.softplus = o[10] == Py_True;
    const long path = PyLong_Check(o[16]) ? PyLong_AsLong(o[16]) : -1;
    if (path < 0 || path > 2) {
      PyErr_Clear();
      return nullptr;
    }
    a.path = static_cast<int32_t>(path);
    if (ssm_workspace(&a) > 0) return nullptr;
    return launched(ssm_prompt, a, stream);
  });
}

// Addresses of the library's kda_conv_prompt, kda_ssm_prompt_workspace, kda_ssm_prompt
// and kda_linear.
PyObject *py_setup(PyObject *, PyObject *const *o, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "four addresses");
    return nullptr;
  }
  void *at[4];
  for (int i = 0; i < 4; ++i) at[i] = PyLong_AsVoidPtr(o[i]);
  if (PyErr_Occurred()) return nullptr;
  conv_prompt = reinterpret_cast<decltype(conv_prompt)>(at[0]);
  ssm_workspace = reinterpret_cast<decltype(ssm_workspace)>(at[1]);
  ssm_prompt = reinterpret_cast<decltype(ssm_prompt)>(at[2]);
  linear = reinterpret_cast<decltype(linear)>(at[3]);
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"setup", reinterpret_cast<PyCFunction>(py_setup), METH_FASTCALL, nullptr},
    {"conv_prompt", reinterpret_cast<PyCFunction>(py_conv_prompt), METH_FASTCALL, nullptr},
    {"ssm_prompt", reinterpret_cast<PyCFunction>(py_ssm_prompt), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(py_linear), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "kda_bind", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kda_bind() { return PyModule_Create(&kModule); }
