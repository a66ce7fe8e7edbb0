/*
 * Argument marshalling of the block operators' Python entry points
 * (rms_norm_quant, qk_norm_rope, gemm_fused) on the CPython C API: takes
 * pointers, shapes and pitches of torch tensors through their Python
 * attributes, refuses what does not fit, and calls the C ABI.  A call of these
 * operators on one token costs the host more than the GPU: checked and
 * marshalled in Python over ctypes, an rms_norm_quant call took 9.3 us.
 * It knows nothing of torch's or CUDA's headers: bind() hands it the ABI's
 * addresses and the objects that it compares with.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

typedef int (*norm_fn)(const void*, int, int64_t, const void*, int64_t, void*, int64_t, const float*, float, int, int,
                       void*, int, int64_t, float*, float*, void*);
typedef int (*rope_fn)(const void*, int64_t, int64_t, void*, int64_t, int64_t, int, const float*, const void*, int64_t,
                       int64_t, void*, int64_t, int64_t, int, const float*, int, int, int, const int32_t*, int64_t,
                       const int*, int, const double*, float, int, void*);
typedef int (*gemm_fn)(const void*, int64_t, const float*, const void*, int64_t, const float*, int, const float*, int,
                       const float*, const void*, int64_t, int, int, int, void*, int, int64_t, void*);

static norm_fn call_norm;
static rope_fn call_rope;
static gemm_fn call_gemm;
static int gpus;                                              /* GPUs that torch sees */
static PyObject *refuse, *raw_stream, *current_device;        /* Python callables */
static PyObject *dt_bf16, *dt_fp16, *dt_fp32, *dt_fp64, *dt_int8, *dt_int32;
static PyObject *s_shape, *s_stride, *s_dtype, *s_is_cuda, *s_data_ptr, *s_numel, *s_is_contiguous, *s_get_device,
    *s_cuda_stream;

enum { MAX_AXES = 4, BLOCK = 256 };           /* CONVROT_MAX_AXES, CONVROT_BLOCK */

/* ---- integers of Python objects; -1 with an exception set on failure */
static int to_ll(PyObject* o, long long* v) {
  *v = PyLong_AsLongLong(o);
  return *v == -1 && PyErr_Occurred() ? -1 : 0;
}

static int to_int(PyObject* o, int* v) {
  long long w;
  if (to_ll(o, &w)) return -1;
  if (w != (int)w) {
    PyErr_SetString(PyExc_OverflowError, "a size exceeds 32 bits");
    return -1;
  }
  *v = (int)w;
  return 0;
}

static int method_ll(PyObject* t, PyObject* name, long long* v) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (!r) return -1;
  const int bad = to_ll(r, v);
  Py_DECREF(r);
  return bad;
}

/* The integers of t.shape or t.stride(): at most `most`; returns how many, -1 on failure. */
static int ints(PyObject* seq, long long* out, int most) {
  if (!seq) return -1;
  int n = -1;
  if (PyTuple_Check(seq) && PyTuple_GET_SIZE(seq) <= most) {
    n = (int)PyTuple_GET_SIZE(seq);
    for (int i = 0; i < n; ++i)
      if (to_ll(PyTuple_GET_ITEM(seq, i), &out[i])) {
        n = -1;
        break;
      }
  } else if (PyTuple_Check(seq)) {
    n = most + 1;                              /* too many dimensions: the caller refuses */
  } else {
    PyErr_SetString(PyExc_TypeError, "a tensor is needed");
  }
  Py_DECREF(seq);
  return n;
}

static int shape_of(PyObject* t, long long* out, int most) { return ints(PyObject_GetAttr(t, s_shape), out, most); }

static int is_cuda(PyObject* t) {
  PyObject* r = PyObject_GetAttr(t, s_is_cuda);
  if (!r) return -1;
  const int yes = r == Py_True;
  Py_DECREF(r);
  return yes;
}

/* Borrowed reference to one of the known types, or NULL (no exception) for another. */
static PyObject* dtype_of(PyObject* t) {
  PyObject* known[] = {dt_bf16, dt_fp16, dt_fp32, dt_fp64, dt_int8, dt_int32};
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return NULL;
  PyObject* found = NULL;
  for (int i = 0; i < 6; ++i)
    if (d == known[i]) found = known[i];
  Py_DECREF(d);
  return found;
}

/* Raises the ValueError that names the tensor and what is needed; always -1. */
static int refusal(const char* fn, const char* name, PyObject* t, PyObject* need) {
  if (PyErr_Occurred() || !need) {
    Py_XDECREF(need);
    return -1;
  }
  PyObject* r = PyObject_CallFunction(refuse, "ssOO", fn, name, t, need);
  Py_XDECREF(r);
  Py_DECREF(need);
  return -1;
}

typedef struct {
  void* ptr;
  int64_t ld;
} matrix_t;

/* A device matrix of `dtype`, rows x at least cols, with contiguous rows; None is a null pointer. */
static int matrix(const char* fn, const char* name, PyObject* t, long long rows, long long cols, PyObject* dtype,
                  matrix_t* out) {
  out->ptr = NULL;
  out->ld = 0;
  if (t == Py_None) return 0;
  long long shape[2], stride[2], p;
  const int d = shape_of(t, shape, 2);
  if (d < 0) return -1;
  if (d == 2 && shape[0] == rows && shape[1] >= cols && dtype && dtype_of(t) == dtype && is_cuda(t) == 1) {
    if (ints(PyObject_CallMethodNoArgs(t, s_stride), stride, 2) != 2) return -1;
    if (stride[1] == 1 || cols <= 1) {
      if (method_ll(t, s_data_ptr, &p)) return -1;
      out->ptr = (void*)(uintptr_t)p;
      /* a single row has no pitch: torch may report any stride for it */
      out->ld = rows > 1 || stride[0] > shape[1] ? stride[0] : shape[1];
      return 0;
    }
  }
  return refusal(fn, name, t, dtype ? PyUnicode_FromFormat("a %S CUDA matrix [%lld, >= %lld] with contiguous rows", dtype,
                                                           rows, cols)
                                    : PyUnicode_FromString("of a supported type"));
}

/* A contiguous device vector of n values of `dtype`; None is a null pointer. */
static int vector(const char* fn, const char* name, PyObject* t, long long n, PyObject* dtype, void** out) {
  *out = NULL;
  if (t == Py_None) return 0;
  long long count, p;
  if (dtype_of(t) == dtype && is_cuda(t) == 1) {
    if (method_ll(t, s_numel, &count)) return -1;
    if (count == n) {
      PyObject* r = PyObject_CallMethodNoArgs(t, s_is_contiguous);
      if (!r) return -1;
      const int whole = r == Py_True;
      Py_DECREF(r);
      if (whole) {
        if (method_ll(t, s_data_ptr, &p)) return -1;
        *out = (void*)(uintptr_t)p;
        return 0;
      }
    }
  }
  return refusal(fn, name, t, PyUnicode_FromFormat("a contiguous %S CUDA vector of %lld", dtype, n));
}

/* Codes of the storage types and of the codes' types (convrot_dtype, convrot_codes); -1 refused. */
static int storage_code(const char* fn, const char* name, PyObject* t, PyObject** dtype) {
  *dtype = dtype_of(t);
  if (*dtype && *dtype == dt_bf16) return 0;
  if (*dtype && *dtype == dt_fp16) return 1;
  if (*dtype && *dtype == dt_fp32) return 2;
  return refusal(fn, name, t, PyUnicode_FromString("bfloat16, float16 or float32"));
}

static int codes_code(const char* fn, const char* name, PyObject* t, PyObject** dtype) {
  *dtype = dtype_of(t);
  if (*dtype && *dtype == dt_int8) return 0;
  if (*dtype && *dtype == dt_fp16) return 1;
  return refusal(fn, name, t, PyUnicode_FromString("int8 or float16 codes"));
}

/*
 * The device that holds every tensor of a call (None aside), which has to be
 * the calling thread's current one: the C ABI launches there, and the stream
 * is one of its streams.  `names` are the tensors' names; -1 refused.  With
 * one GPU there is nothing to ask (0.8 us of a one-token call's 6).
 */
static int device_of(const char* fn, PyObject* const* t, const char* const* names, int n, int* device) {
  long long first = 0, d, current;
  *device = 0;
  if (gpus == 1) return 0;
  for (int i = 0; i < n; ++i) {
    if (t[i] == Py_None) continue;
    if (method_ll(t[i], s_get_device, &d)) return -1;
    if (i == 0) first = d;                       /* the first one is always given */
    if (d != first) return refusal(fn, names[i], t[i], PyUnicode_FromFormat("on cuda:%lld like %s", first, names[0]));
  }
  PyObject* r = PyObject_CallNoArgs(current_device);
  if (!r) return -1;
  const int bad = to_ll(r, &current);
  Py_DECREF(r);
  if (bad) return -1;
  if (first != current)
    return refusal(fn, names[0], t[0], PyUnicode_FromFormat("on the current device (cuda:%lld)", current));
  *device = (int)first;
  return 0;
}

/* The given stream (a handle or an object with cuda_stream), or the current one of the device. */
static int stream_of(int device, PyObject* stream, void** out) {
  long long v;
  PyObject* r;
  if (stream == Py_None) {
    PyObject* dev = PyLong_FromLong(device);
    if (!dev) return -1;
    r = PyObject_CallOneArg(raw_stream, dev);
    Py_DECREF(dev);
  } else if (PyLong_Check(stream)) {
    r = Py_NewRef(stream);
  } else {
    r = PyObject_GetAttr(stream, s_cuda_stream);
  }
  if (!r) return -1;
  const int bad = to_ll(r, &v);
  Py_DECREF(r);
  *out = (void*)(uintptr_t)v;
  return bad;
}

static int want(Py_ssize_t n, Py_ssize_t needed) {
  if (n == needed) return 0;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return -1;
}

static int to_float(PyObject* o, float* v) {
  const double d = PyFloat_AsDouble(o);
  *v = (float)d;
  return d == -1.0 && PyErr_Occurred() ? -1 : 0;
}

static int rows_of(PyObject* t, int* rows) {
  long long shape[3];
  const int d = shape_of(t, shape, 3);
  if (d < 0) return -1;
  if (d < 1 || d > 3 || shape[0] != (int)shape[0]) {
    PyErr_SetString(PyExc_ValueError, "a matrix with less than 2^31 rows is needed");
    return -1;
  }
  *rows = (int)shape[0];
  return 0;
}

/* Codes in a row of K elements: whole rotation blocks, all of which are written. */
static long long padded(long long K) { return (K + BLOCK - 1) / BLOCK * BLOCK; }

/* (x, K, a_q, a_scale, residual, h, weight, eps, a_norm, stream) -> status */
static PyObject* rms_norm_quant(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  const char* fn = "rms_norm_quant";
  int M, K, dtype, fmt, dev, status;
  float eps;
  PyObject *dt, *cdt;
  matrix_t x, r, h, q;
  void *w, *s, *nb, *st;
  if (want(n, 10) || to_int(a[1], &K) || rows_of(a[0], &M) || (dtype = storage_code(fn, "x", a[0], &dt)) < 0 ||
      (fmt = codes_code(fn, "a_q", a[2], &cdt)) < 0 || matrix(fn, "x", a[0], M, K, dt, &x) ||
      matrix(fn, "a_q", a[2], M, padded(K), cdt, &q) || vector(fn, "a_scale", a[3], M, dt_fp32, &s) ||
      matrix(fn, "residual", a[4], M, K, dt, &r) || matrix(fn, "h", a[5], M, K, dt, &h) ||
      vector(fn, "weight", a[6], K, dt_fp32, &w) || to_float(a[7], &eps) ||
      vector(fn, "a_norm", a[8], M, dt_fp32, &nb))
    return NULL;
  PyObject* const used[] = {a[0], a[2], a[3], a[4], a[5], a[6], a[8]};
  static const char* const names[] = {"x", "a_q", "a_scale", "residual", "h", "weight", "a_norm"};
  if (device_of(fn, used, names, 7, &dev) || stream_of(dev, a[9], &st)) return NULL;
  Py_BEGIN_ALLOW_THREADS                         /* a launch waits while the launch queue is full */
  status = call_norm(x.ptr, dtype, x.ld, r.ptr, r.ld, h.ptr, h.ld, w, eps, M, K, q.ptr, fmt, q.ld, s, nb, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

typedef struct {
  void* ptr;
  int64_t tok, head;
  int heads;
} heads_t;

/* [M, heads, D] of `dtype` on the device, a head's values contiguous; `like` gives the number of heads. */
static int heads(const char* fn, const char* name, PyObject* t, long long M, long long D, PyObject* dtype,
                 const heads_t* like, heads_t* out) {
  out->ptr = NULL;
  out->tok = out->head = out->heads = 0;
  if (t == Py_None) return 0;
  long long shape[3], stride[3], p;
  const int d = shape_of(t, shape, 3);
  if (d < 0) return -1;
  if (d == 3 && shape[0] == M && shape[2] == D && shape[1] == (int)shape[1] && (!like || shape[1] == like->heads) &&
      dtype_of(t) == dtype && is_cuda(t) == 1) {
    if (ints(PyObject_CallMethodNoArgs(t, s_stride), stride, 3) != 3) return -1;
    if (stride[2] == 1 || D <= 1) {
      if (method_ll(t, s_data_ptr, &p)) return -1;
      out->ptr = (void*)(uintptr_t)p;
      out->tok = stride[0];
      out->head = stride[1];
      out->heads = (int)shape[1];
      return 0;
    }
  }
  return refusal(fn, name, t, PyUnicode_FromFormat("a %S CUDA tensor [%lld, heads, %lld] with its input's heads, contiguous",
                                                   dtype, M, D));
}

/* (q, k, pos, inv_freq, axis_pairs, q_out, k_out, q_weight, k_weight, eps, interleaved, stream) -> status */
static PyObject* qk_norm_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  const char* fn = "qk_norm_rope";
  if (want(n, 12)) return NULL;
  int pairs[MAX_AXES], axes, dtype, dev, status;
  long long shape[3], sum = 0;
  float eps;
  PyObject* dt;
  heads_t q, k, qo, ko;
  matrix_t pos;
  void *f, *qw, *kw, *st;
  PyObject* seq = PySequence_Fast(a[4], "axis_pairs must be a sequence");
  if (!seq) return NULL;
  const Py_ssize_t given = PySequence_Fast_GET_SIZE(seq);
  int bad = given > MAX_AXES;
  if (bad) PyErr_Format(PyExc_ValueError, "%s: at most %d axes", fn, MAX_AXES);
  for (Py_ssize_t i = 0; !bad && i < given; ++i) {
    bad = to_int(PySequence_Fast_GET_ITEM(seq, i), &pairs[i]);
    sum += bad ? 0 : pairs[i];
  }
  Py_DECREF(seq);
  if (bad) return NULL;
  axes = (int)given;
  const int d = shape_of(a[0], shape, 3);
  if (d < 0) return NULL;
  if (d != 3 || shape[0] != (int)shape[0] || shape[2] != (int)shape[2]) {
    refusal(fn, "q", a[0], PyUnicode_FromString("[tokens, heads, head width]"));
    return NULL;
  }
  if ((a[1] == Py_None) != (a[6] == Py_None)) {
    PyErr_Format(PyExc_ValueError, "%s: k and k_out belong together", fn);
    return NULL;
  }
  const int interleaved = PyObject_IsTrue(a[10]);
  if (interleaved < 0 || (dtype = storage_code(fn, "q", a[0], &dt)) < 0 ||
      heads(fn, "q", a[0], shape[0], shape[2], dt, NULL, &q) || heads(fn, "k", a[1], shape[0], shape[2], dt, NULL, &k) ||
      heads(fn, "q_out", a[5], shape[0], shape[2], dt, &q, &qo) || heads(fn, "k_out", a[6], shape[0], shape[2], dt, &k, &ko) ||
      matrix(fn, "pos", a[2], shape[0], axes, dt_int32, &pos) || vector(fn, "inv_freq", a[3], sum, dt_fp64, &f) ||
      vector(fn, "q_weight", a[7], shape[2], dt_fp32, &qw) || vector(fn, "k_weight", a[8], shape[2], dt_fp32, &kw) ||
      to_float(a[9], &eps))
    return NULL;
  PyObject* const used[] = {a[0], a[1], a[2], a[3], a[5], a[6], a[7], a[8]};
  static const char* const names[] = {"q", "k", "pos", "inv_freq", "q_out", "k_out", "q_weight", "k_weight"};
  if (device_of(fn, used, names, 8, &dev) || stream_of(dev, a[11], &st)) return NULL;
  Py_BEGIN_ALLOW_THREADS                         /* a launch waits while the launch queue is full */
  status = call_rope(q.ptr, q.tok, q.head, qo.ptr, qo.tok, qo.head, q.heads, qw, k.ptr, k.tok, k.head, ko.ptr,
                     ko.tok, ko.head, k.heads, kw, dtype, (int)shape[0], (int)shape[2], pos.ptr, pos.ld, pairs,
                     axes, f, eps, interleaved, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

/* (a_q, a_scale, w_q, w_scale, out, K_p or None, bias, act, gate, residual, stream) -> status */
static PyObject* gemm_fused(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  const char* fn = "gemm_fused";
  if (want(n, 11)) return NULL;
  long long sa[2], sw[2], kp;
  int act, fmt, dtype, dev, status;
  PyObject *cdt, *odt;
  matrix_t aq, wq, out, res;
  void *as, *ws, *b, *g, *st;
  const int da = shape_of(a[0], sa, 2), dw = da < 0 ? -1 : shape_of(a[2], sw, 2);
  if (dw < 0) return NULL;
  if (da != 2 || dw != 2 || sa[0] != (int)sa[0] || sw[0] != (int)sw[0]) {
    PyErr_Format(PyExc_ValueError, "%s: a_q and w_q must be matrices", fn);
    return NULL;
  }
  kp = sa[1];
  if (a[5] != Py_None && to_ll(a[5], &kp)) return NULL;
  if (kp != (int)kp) {
    PyErr_SetString(PyExc_OverflowError, "a size exceeds 32 bits");
    return NULL;
  }
  if (to_int(a[7], &act) || (fmt = codes_code(fn, "a_q", a[0], &cdt)) < 0 || (dtype = storage_code(fn, "out", a[4], &odt)) < 0 ||
      matrix(fn, "a_q", a[0], sa[0], kp, cdt, &aq) || vector(fn, "a_scale", a[1], sa[0], dt_fp32, &as) ||
      matrix(fn, "w_q", a[2], sw[0], kp, cdt, &wq) || vector(fn, "w_scale", a[3], sw[0], dt_fp32, &ws) ||
      matrix(fn, "out", a[4], sa[0], sw[0], odt, &out) || vector(fn, "bias", a[6], sw[0], dt_fp32, &b) ||
      vector(fn, "gate", a[8], sw[0], dt_fp32, &g) || matrix(fn, "residual", a[9], sa[0], sw[0], odt, &res))
    return NULL;
  PyObject* const used[] = {a[0], a[1], a[2], a[3], a[4], a[6], a[8], a[9]};
  static const char* const names[] = {"a_q", "a_scale", "w_q", "w_scale", "out", "bias", "gate", "residual"};
  if (device_of(fn, used, names, 8, &dev) || stream_of(dev, a[10], &st)) return NULL;
  Py_BEGIN_ALLOW_THREADS                         /* a launch waits while the launch queue is full */
  status = call_gemm(aq.ptr, aq.ld, as, wq.ptr, wq.ld, ws, fmt, b, act, g, res.ptr, res.ld, (int)sa[0],
                     (int)sw[0], (int)kp, out.ptr, dtype, out.ld, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

/* (norm, rope, gemm addresses, GPUs, refuse, raw_stream, current_device, bf16, fp16, fp32, fp64, int8, int32): once, at load. */
static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  long long p[3];
  if (want(n, 13)) return NULL;
  for (int i = 0; i < 3; ++i)
    if (to_ll(a[i], &p[i])) return NULL;
  if (to_int(a[3], &gpus)) return NULL;
  call_norm = (norm_fn)(uintptr_t)p[0];
  call_rope = (rope_fn)(uintptr_t)p[1];
  call_gemm = (gemm_fn)(uintptr_t)p[2];
  PyObject** kept[] = {&refuse, &raw_stream, &current_device, &dt_bf16, &dt_fp16, &dt_fp32, &dt_fp64, &dt_int8, &dt_int32};
  for (int i = 0; i < 9; ++i) Py_XSETREF(*kept[i], Py_NewRef(a[4 + i]));
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, NULL},
                                {"rms_norm_quant", (PyCFunction)(void (*)(void))rms_norm_quant, METH_FASTCALL, NULL},
                                {"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, NULL},
                                {"gemm_fused", (PyCFunction)(void (*)(void))gemm_fused, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
  const struct {
    PyObject** name;
    const char* text;
  } names[] = {{&s_shape, "shape"},       {&s_stride, "stride"}, {&s_dtype, "dtype"},
               {&s_is_cuda, "is_cuda"},   {&s_data_ptr, "data_ptr"}, {&s_numel, "numel"},
               {&s_is_contiguous, "is_contiguous"}, {&s_get_device, "get_device"}, {&s_cuda_stream, "cuda_stream"}};
  for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
    if (!(*names[i].name = PyUnicode_InternFromString(names[i].text))) return NULL;
  return PyModule_Create(&module);
}
