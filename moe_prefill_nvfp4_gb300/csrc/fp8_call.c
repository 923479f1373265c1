/* fp8_call.c -- Python argument marshalling of the FP8 calls (module _fp8_call), the part of the binding
 * whose own time counts: one token's product takes a few microseconds on the GPU, and the same marshalling
 * in Python (tensor attributes, ctypes structures, checks) took longer than that (row quantiser 9.8 us a
 * call, dense product 12.5 us; here 8.6 both, of which 3.1 and 4.3 remain when outputs are given).  It
 * reads tensors through their Python attributes, so it depends on no PyTorch header, allocates outputs with
 * torch.empty_strided, and calls the C ABI (include/moe_prefill.h), which repeats every check that matters
 * to the device, but for the GPU that the pointers belong to, which is checked here alone.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "moe_prefill.h"

/* set by init() */
static PyObject *g_error, *g_empty, *g_f8, *g_bf16, *g_f32, *g_i32, *g_raw_stream, *g_current_device;
static PyObject* g_no_text; /* "" */
/* interned names */
static PyObject *n_dtype, *n_shape, *n_stride, *n_data_ptr, *n_device, *n_get_device, *n_cuda_stream;
static PyObject* kw_empty; /* ("dtype", "device") */

typedef struct {
  PyObject* dtype; /* borrowed: torch's type objects live as long as torch */
  void* ptr;
  int nd;
  int64_t shape[3], stride[3];
} Tensor;

static int ints(PyObject* tuple, int64_t* out) {
  const Py_ssize_t n = PyTuple_GET_SIZE(tuple);
  for (Py_ssize_t i = 0; i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (out[i] == -1 && PyErr_Occurred()) return -1;
  }
  return (int)n;
}

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

/* Reads a CUDA tensor of nd dimensions and one of two element types (d1 may be NULL).  *gpu is the GPU of the
 * call's tensors, -1 before the first: the kernel runs on one GPU and gets every pointer. */
static int read_tensor(PyObject* t, const char* name, int nd, PyObject* d0, PyObject* d1, Tensor* out, int* gpu) {
  PyObject *dtype = PyObject_GetAttr(t, n_dtype), *index = NULL, *shape = NULL, *stride = NULL, *ptr = NULL;
  int ok = 0;
  if (dtype == NULL) return 0;
  if ((index = PyObject_CallMethodNoArgs(t, n_get_device)) == NULL || (shape = PyObject_GetAttr(t, n_shape)) == NULL)
    goto done;
  const long device = PyLong_AsLong(index); /* -1: not on a GPU */
  if (device == -1 && PyErr_Occurred()) goto done;
  if ((dtype != d0 && dtype != d1) || device < 0 || !PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != nd) {
    PyErr_Format(PyExc_ValueError, "%s: need a CUDA tensor of %d dimensions and type %R%s%S, got %R %R%s", name, nd, d0,
                 d1 ? " or " : "", d1 ? d1 : g_no_text, dtype, shape, device < 0 ? " not on a GPU" : "");
    goto done;
  }
  if (*gpu < 0) *gpu = (int)device;
  if (device != *gpu) {
    PyErr_Format(PyExc_ValueError, "%s: on GPU %ld, the tensors before it are on GPU %d", name, device, *gpu);
    goto done;
  }
  if ((stride = PyObject_CallMethodNoArgs(t, n_stride)) == NULL || (ptr = PyObject_CallMethodNoArgs(t, n_data_ptr)) == NULL)
    goto done;
  out->dtype = dtype;
  out->nd = nd;
  if (ints(shape, out->shape) < 0 || ints(stride, out->stride) < 0) goto done;
  out->ptr = PyLong_AsVoidPtr(ptr);
  ok = !PyErr_Occurred();
done:
  Py_XDECREF(dtype);
  Py_XDECREF(index);
  Py_XDECREF(shape);
  Py_XDECREF(stride);
  Py_XDECREF(ptr);
  return ok;
}

static int unit_columns(const Tensor* t, const char* name) {
  if (t->stride[t->nd - 1] == 1 || t->shape[t->nd - 1] <= 1) return 1;
  PyErr_Format(PyExc_ValueError, "%s: need unit column stride, got %lld", name, (long long)t->stride[t->nd - 1]);
  return 0;
}

/* Row stride; a single row has none, whatever its tensor says: it counts as whole pieces of `piece` elements. */
static int64_t row_stride(const Tensor* t, int64_t piece) {
  return t->shape[t->nd - 2] > 1 ? t->stride[t->nd - 2] : ceil_div(t->shape[t->nd - 1], piece) * piece;
}

static int same_shape(const Tensor* t, const char* name, int64_t rows, int64_t cols) {
  if (t->shape[t->nd - 2] == rows && t->shape[t->nd - 1] == cols) return 1;
  PyErr_Format(PyExc_ValueError, "%s: need [%lld, %lld], got [%lld, %lld]", name, (long long)rows, (long long)cols,
               (long long)t->shape[t->nd - 2], (long long)t->shape[t->nd - 1]);
  return 0;
}

/* A new reference to `given` (checked: an E4M3, BF16 or FP32 matrix of that shape), or a new tensor with
 * the strides (ld, 1) or, by_column, (1, rows). */
static PyObject* output(PyObject* given, const char* name, PyObject* dtype, PyObject* device, int64_t rows, int64_t cols,
                        int64_t ld, int by_column, Tensor* out, int* gpu) {
  if (given != Py_None) {
    if (!read_tensor(given, name, 2, dtype, NULL, out, gpu) || !same_shape(out, name, rows, cols)) return NULL;
    return Py_NewRef(given);
  }
  PyObject* size = Py_BuildValue("(LL)", (long long)rows, (long long)cols);
  PyObject* stride = by_column ? Py_BuildValue("(iL)", 1, (long long)rows) : Py_BuildValue("(Li)", (long long)ld, 1);
  PyObject *t = NULL, *ptr = NULL;
  if (size != NULL && stride != NULL) {
    PyObject* const args[4] = {size, stride, dtype, device};
    t = PyObject_Vectorcall(g_empty, args, 2, kw_empty);
  }
  Py_XDECREF(size);
  Py_XDECREF(stride);
  if (t == NULL || (ptr = PyObject_CallMethodNoArgs(t, n_data_ptr)) == NULL) {
    Py_XDECREF(t);
    return NULL;
  }
  out->dtype = dtype;
  out->nd = 2;
  out->ptr = PyLong_AsVoidPtr(ptr);
  Py_DECREF(ptr);
  out->shape[0] = rows;
  out->shape[1] = cols;
  out->stride[0] = by_column ? 1 : ld;
  out->stride[1] = by_column ? rows : 1;
  return t;
}

static PyObject* codes_out(PyObject* given, const char* name, PyObject* device, int64_t rows, int64_t cols, Tensor* out,
                           int64_t* ld, int* gpu) {
  PyObject* t = output(given, name, g_f8, device, rows, cols, ceil_div(cols, 16) * 16, 0, out, gpu);
  if (t != NULL && !unit_columns(out, name)) Py_CLEAR(t);
  *ld = t ? row_stride(out, 16) : 0;
  return t;
}

static PyObject* product_out(PyObject* given, PyObject* c_dtype, PyObject* device, int64_t rows, int64_t cols, Tensor* out,
                             int64_t* ld, int* code, int* gpu) {
  if (c_dtype != g_bf16 && c_dtype != g_f32) {
    PyErr_SetString(PyExc_ValueError, "c_dtype: torch.bfloat16 or torch.float32");
    return NULL;
  }
  *code = c_dtype == g_bf16 ? MOE_DTYPE_BF16 : MOE_DTYPE_F32;
  PyObject* t = output(given, "out", c_dtype, device, rows, cols, ceil_div(cols, 8) * 8, 0, out, gpu);
  if (t != NULL && !unit_columns(out, "out")) Py_CLEAR(t);
  *ld = t ? row_stride(out, 8) : 0;
  return t;
}

/* The stream handle: `stream`'s, or the current one of the tensors' GPU, which has to be the current GPU: the
 * library launches there, and the default stream's handle is the same on all of them. */
static int stream_of(PyObject* stream, int gpu, void** out) {
  PyObject* now = PyObject_CallNoArgs(g_current_device);
  if (now == NULL) return 0;
  const long current = PyLong_AsLong(now);
  PyObject* h = NULL;
  if (current == -1 && PyErr_Occurred()) {
  } else if (current != gpu) {
    PyErr_Format(PyExc_ValueError, "tensors on GPU %d, the current one is GPU %ld", gpu, current);
  } else if (stream != Py_None) {
    h = PyObject_GetAttr(stream, n_cuda_stream);
  } else {
    h = PyObject_CallOneArg(g_raw_stream, now);
  }
  Py_DECREF(now);
  if (h == NULL) return 0;
  *out = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  return !PyErr_Occurred();
}

static PyObject* fail(int rc, const char* what) {
  PyObject* e = PyObject_CallFunction(g_error, "is", rc, what);
  if (e != NULL) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return NULL;
}

static int fits(int64_t v, const char* name) {
  if (v >= 0 && v <= INT32_MAX) return 1;
  PyErr_Format(PyExc_ValueError, "%s: %lld is not a 32-bit size", name, (long long)v);
  return 0;
}

static int want(Py_ssize_t got, Py_ssize_t n) {
  if (got == n) return 1;
  PyErr_Format(PyExc_TypeError, "need %zd arguments, got %zd", n, got);
  return 0;
}

/* (first, second) or the error rc */
static PyObject* pair_or_fail(int rc, const char* what, PyObject* a, PyObject* b) {
  PyObject* r = rc == MOE_OK ? PyTuple_Pack(2, a, b) : fail(rc, what);
  Py_DECREF(a);
  Py_DECREF(b);
  return r;
}

/* quantize(x, out, scales, stream, blocks) */
static PyObject* quantize(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor x, q, s;
  int64_t ld_q;
  void* st;
  int gpu = -1;
  if (!want(n, 5) || !read_tensor(a[0], "x", 2, g_bf16, g_f32, &x, &gpu) || !unit_columns(&x, "x") || !fits(x.shape[0], "rows") ||
      !fits(x.shape[1], "columns") || !stream_of(a[3], gpu, &st))
    return NULL;
  const int blocks = a[4] == Py_True;
  const int64_t R = x.shape[0], K = x.shape[1], G = ceil_div(K, 128), SR = blocks ? ceil_div(R, 128) : R;
  PyObject* device = PyObject_GetAttr(a[0], n_device);
  if (device == NULL) return NULL;
  PyObject *tq = codes_out(a[1], "out", device, R, K, &q, &ld_q, &gpu), *ts = NULL;
  if (tq != NULL) ts = output(a[2], "scales", g_f32, device, SR, G, G, !blocks, &s, &gpu);
  Py_DECREF(device);
  if (ts != NULL && blocks && s.shape[0] * s.shape[1] > 1 && ((s.stride[1] != 1 && G > 1) || (s.stride[0] != G && SR > 1))) {
    PyErr_SetString(PyExc_ValueError, "scales: need a contiguous tensor");
    Py_CLEAR(ts);
  }
  if (ts == NULL) {
    Py_XDECREF(tq);
    return NULL;
  }
  const int dt = x.dtype == g_bf16 ? MOE_DTYPE_BF16 : MOE_DTYPE_F32;
  const int64_t ld_x = row_stride(&x, 1);
  int rc = MOE_OK;
  if (blocks)
    rc = moe_fp8_quantize_blocks(x.ptr, dt, ld_x, (int)R, (int)K, q.ptr, ld_q, s.ptr, st);
  else if (R > 0)
    rc = moe_fp8_quantize_rows(x.ptr, dt, ld_x, (int)R, (int)K, q.ptr, ld_q, s.ptr, s.stride[0], s.stride[1], st);
  return pair_or_fail(rc, blocks ? "moe_fp8_quantize_blocks" : "moe_fp8_quantize_rows", tq, ts);
}

/* activation rows [rows, K] with their scales */
static int read_rows(PyObject* tq, PyObject* ts, const char* nq, const char* ns, moe_fp8_rows* A, int64_t* K, int* gpu) {
  Tensor q, s;
  if (!read_tensor(tq, nq, 2, g_f8, NULL, &q, gpu) || !read_tensor(ts, ns, 2, g_f32, NULL, &s, gpu)) return 0;
  *K = q.shape[1];
  if (!unit_columns(&q, nq) || !same_shape(&s, ns, q.shape[0], ceil_div(*K, 128)) || !fits(q.shape[0], "rows")) return 0;
  A->q = q.ptr;
  A->ld = row_stride(&q, 16);
  A->s = s.ptr;
  A->s_row = s.stride[0];
  A->s_grp = s.stride[1];
  A->rows = (int)q.shape[0];
  return 1;
}

/* a weight [N, K] (nd 2) or [experts, N, K] (nd 3) with its scales */
static int read_weight(PyObject* tq, PyObject* ts, const char* nq, const char* ns, int nd, int64_t first,
                       moe_fp8_weight* W, int* gpu) {
  Tensor w, ws;
  if (!read_tensor(tq, nq, nd, g_f8, NULL, &w, gpu) || !read_tensor(ts, ns, nd, g_f32, NULL, &ws, gpu)) return 0;
  const int64_t N = w.shape[nd - 2], K = w.shape[nd - 1], G = ceil_div(K, 128), NB = ceil_div(N, 128);
  if (!unit_columns(&w, nq) || !same_shape(&ws, ns, NB, G)) return 0;
  const int64_t count = nd == 3 ? w.shape[0] : 1;
  if (nd == 3 && ws.shape[0] != count) {
    PyErr_Format(PyExc_ValueError, "%s: need %lld experts, got %lld", ns, (long long)count, (long long)ws.shape[0]);
    return 0;
  }
  if ((G > 1 && ws.stride[nd - 1] != 1) || (NB > 1 && ws.stride[nd - 2] != G) || (count > 1 && ws.stride[0] != NB * G)) {
    PyErr_Format(PyExc_ValueError, "%s: need a contiguous tensor", ns);
    return 0;
  }
  if (!fits(N, "N") || !fits(K, "K") || !fits(count, "experts") || !fits(first, "first")) return 0;
  W->q = w.ptr;
  W->ld = row_stride(&w, 16);
  W->expert_stride = count > 1 ? w.stride[0] : 0;
  W->s = ws.ptr;
  W->first = (int)first;
  W->count = (int)count;
  W->N = (int)N;
  W->K = (int)K;
  return 1;
}

/* the operands of a product: rows, their scales, a weight, its scales */
static int operands(PyObject* const* a, int nd, int64_t first, moe_fp8_rows* A, moe_fp8_weight* W, int* gpu) {
  int64_t K;
  if (!read_rows(a[0], a[1], "A", "a_scales", A, &K, gpu) ||
      !read_weight(a[2], a[3], "W", "w_scales", nd, first, W, gpu))
    return 0;
  if (K == W->K) return 1;
  PyErr_Format(PyExc_ValueError, "A, W: %lld and %lld columns", (long long)K, (long long)W->K);
  return 0;
}

/* gemm(A, a_scales, W, w_scales, out, c_dtype, stream) */
static PyObject* gemm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  moe_fp8_rows A;
  moe_fp8_weight W;
  Tensor c;
  int64_t ld;
  int code, gpu = -1;
  void* st;
  if (!want(n, 7) || !operands(a, 2, 0, &A, &W, &gpu) || !stream_of(a[6], gpu, &st)) return NULL;
  PyObject* device = PyObject_GetAttr(a[0], n_device);
  if (device == NULL) return NULL;
  PyObject* out = product_out(a[4], a[5], device, A.rows, W.N, &c, &ld, &code, &gpu);
  Py_DECREF(device);
  if (out == NULL || A.rows == 0) return out;
  const int rc = moe_fp8_gemm(&A, &W, c.ptr, ld, code, st);
  if (rc == MOE_OK) return out;
  Py_DECREF(out);
  return fail(rc, "moe_fp8_gemm");
}

/* expert_offsets [E + 1] and gather_ids [>= R] (or None): contiguous int32 */
static int groups(PyObject* offsets, PyObject* gather, int64_t R, Tensor* off, const void** ids, int* gpu) {
  Tensor g;
  *ids = NULL;
  if (!read_tensor(offsets, "expert_offsets", 1, g_i32, NULL, off, gpu) || !unit_columns(off, "expert_offsets")) return 0;
  if (gather == Py_None) return 1;
  if (!read_tensor(gather, "gather_ids", 1, g_i32, NULL, &g, gpu) || !unit_columns(&g, "gather_ids")) return 0;
  if (g.shape[0] < R) {
    PyErr_Format(PyExc_ValueError, "gather_ids: need %lld entries, got %lld", (long long)R, (long long)g.shape[0]);
    return 0;
  }
  *ids = g.ptr;
  return 1;
}

/* grouped(A, a_scales, W, w_scales, expert_offsets, R, gather_ids, first, out, c_dtype, stream) */
static PyObject* grouped(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  moe_fp8_rows A;
  moe_fp8_weight W;
  Tensor off, c;
  const void* ids;
  int64_t ld;
  int code, gpu = -1;
  void* st;
  if (!want(n, 11)) return NULL;
  const int64_t R = PyLong_AsLongLong(a[5]), first = PyLong_AsLongLong(a[7]);
  if (PyErr_Occurred() || !fits(R, "R") || !operands(a, 3, first, &A, &W, &gpu) ||
      !groups(a[4], a[6], R, &off, &ids, &gpu) || !stream_of(a[10], gpu, &st))
    return NULL;
  PyObject* device = PyObject_GetAttr(a[0], n_device);
  if (device == NULL) return NULL;
  PyObject* out = product_out(a[8], a[9], device, R, W.N, &c, &ld, &code, &gpu);
  Py_DECREF(device);
  if (out == NULL || R == 0) return out;
  const int rc = moe_fp8_grouped_gemm(&A, ids, &W, off.ptr, (int)off.shape[0] - 1, (int)R, c.ptr, ld, code, st);
  if (rc == MOE_OK) return out;
  Py_DECREF(out);
  return fail(rc, "moe_fp8_grouped_gemm");
}

/* grouped_swiglu(A, a_scales, W, w_scales, expert_offsets, R, limit, gather_ids, first, out, scales, stream) */
static PyObject* grouped_swiglu(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  moe_fp8_rows A;
  moe_fp8_weight W;
  Tensor off, q, s;
  const void* ids;
  int64_t ld;
  int gpu = -1;
  void* st;
  if (!want(n, 12)) return NULL;
  const int64_t R = PyLong_AsLongLong(a[5]), first = PyLong_AsLongLong(a[8]);
  const double limit = PyFloat_AsDouble(a[6]);
  if (PyErr_Occurred() || !fits(R, "R") || !operands(a, 3, first, &A, &W, &gpu) ||
      !groups(a[4], a[7], R, &off, &ids, &gpu) || !stream_of(a[11], gpu, &st))
    return NULL;
  const int64_t I = W.N / 2;
  PyObject* device = PyObject_GetAttr(a[0], n_device);
  if (device == NULL) return NULL;
  PyObject *tq = codes_out(a[9], "out", device, R, I, &q, &ld, &gpu), *ts = NULL;
  if (tq != NULL) ts = output(a[10], "scales", g_f32, device, R, ceil_div(I, 128), 0, 1, &s, &gpu);
  Py_DECREF(device);
  if (ts == NULL) {
    Py_XDECREF(tq);
    return NULL;
  }
  int rc = MOE_OK;
  if (R > 0)
    rc = moe_fp8_grouped_gemm_swiglu(&A, ids, &W, off.ptr, (int)off.shape[0] - 1, (int)R, (float)limit, q.ptr, ld, s.ptr,
                                     s.stride[0], s.stride[1], st);
  return pair_or_fail(rc, "moe_fp8_grouped_gemm_swiglu", tq, ts);
}

/* add_rms_norm(x, weight, residual, eps, normed, residual_out, out, scales, stream) -> (q, s, h or None, y or None) */
static PyObject* add_rms_norm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor x, w, r = {0}, h = {0}, y = {0}, q, s;
  int64_t ld_q;
  void* st;
  int gpu = -1;
  if (!want(n, 9)) return NULL;
  const double eps = PyFloat_AsDouble(a[3]);
  if (PyErr_Occurred() || !read_tensor(a[0], "x", 2, g_bf16, g_f32, &x, &gpu) || !unit_columns(&x, "x") ||
      !read_tensor(a[1], "weight", 1, g_bf16, g_f32, &w, &gpu) || !unit_columns(&w, "weight") ||
      !fits(x.shape[0], "rows") || !fits(x.shape[1], "columns"))
    return NULL;
  const int64_t R = x.shape[0], K = x.shape[1];
  if (w.shape[0] != K) {
    PyErr_Format(PyExc_ValueError, "weight: need [%lld], got [%lld]", (long long)K, (long long)w.shape[0]);
    return NULL;
  }
  const int add = a[2] != Py_None;
  if (add && (!read_tensor(a[2], "residual", 2, g_bf16, g_f32, &r, &gpu) || !same_shape(&r, "residual", R, K) ||
              !unit_columns(&r, "residual")))
    return NULL;
  if (!add && a[5] != Py_None) {
    PyErr_SetString(PyExc_ValueError, "residual_out: there is no residual");
    return NULL;
  }
  if (!stream_of(a[8], gpu, &st)) return NULL;
  PyObject* device = PyObject_GetAttr(a[0], n_device);
  if (device == NULL) return NULL;
  PyObject *tq = NULL, *ts = NULL, *th = NULL, *ty = NULL, *result = NULL;
  tq = codes_out(a[6], "out", device, R, K, &q, &ld_q, &gpu);
  if (tq != NULL) ts = output(a[7], "scales", g_f32, device, R, ceil_div(K, 128), 0, 1, &s, &gpu);
  if (ts != NULL)
    th = add ? output(a[5], "residual_out", r.dtype, device, R, K, K, 0, &h, &gpu) : Py_NewRef(Py_None);
  if (th != NULL && add && !unit_columns(&h, "residual_out")) Py_CLEAR(th);
  if (th != NULL) {
    if (a[4] == Py_None || a[4] == Py_False)
      ty = Py_NewRef(Py_None);
    else
      ty = output(a[4] == Py_True ? Py_None : a[4], "normed", g_bf16, device, R, K, K, 0, &y, &gpu);
    if (ty != NULL && ty != Py_None && !unit_columns(&y, "normed")) Py_CLEAR(ty);
  }
  Py_DECREF(device);
  if (ty != NULL) {
    int rc = MOE_OK;
    if (R > 0)
      rc = moe_fp8_add_rms_norm(x.ptr, x.dtype == g_bf16 ? MOE_DTYPE_BF16 : MOE_DTYPE_F32, row_stride(&x, 1),
                                add ? r.ptr : NULL, add && r.dtype == g_f32 ? MOE_DTYPE_F32 : MOE_DTYPE_BF16,
                                add ? row_stride(&r, 1) : 0, w.ptr, w.dtype == g_bf16 ? MOE_DTYPE_BF16 : MOE_DTYPE_F32,
                                (float)eps, (int)R, (int)K, add ? h.ptr : NULL, add ? row_stride(&h, 1) : 0,
                                ty != Py_None ? y.ptr : NULL, ty != Py_None ? row_stride(&y, 1) : 0, q.ptr, ld_q, s.ptr,
                                s.stride[0], s.stride[1], st);
    result = rc == MOE_OK ? PyTuple_Pack(4, tq, ts, th, ty) : fail(rc, "moe_fp8_add_rms_norm");
  }
  Py_XDECREF(tq);
  Py_XDECREF(ts);
  Py_XDECREF(th);
  Py_XDECREF(ty);
  return result;
}

/* A contiguous tensor of `nd` dimensions or None (*ptr NULL). */
static int read_plain(PyObject* t, const char* name, int nd, PyObject* dtype, int64_t d0, int64_t d1, const void** ptr,
                      int* gpu) {
  Tensor v;
  *ptr = NULL;
  if (t == Py_None) return 1;
  if (!read_tensor(t, name, nd, dtype, NULL, &v, gpu)) return 0;
  if (v.shape[0] != d0 || (nd == 2 && v.shape[1] != d1)) {
    PyErr_Format(PyExc_ValueError, nd == 2 ? "%s: need [%lld, %lld]" : "%s: need [%lld]", name, (long long)d0, (long long)d1);
    return 0;
  }
  if (!unit_columns(&v, name)) return 0;
  if (nd == 2 && d0 > 1 && v.stride[0] != d1) {
    PyErr_Format(PyExc_ValueError, "%s: need a contiguous tensor", name);
    return 0;
  }
  *ptr = v.ptr;
  return 1;
}

/* The workspace: `given` (a tensor of bytes), or a new one. */
static PyObject* workspace(PyObject* given, PyObject* device, size_t bytes, void** ptr, size_t* have, int* gpu) {
  Tensor v;
  if (given != Py_None) {
    PyObject *count = NULL, *at = NULL, *index = PyObject_CallMethodNoArgs(given, n_get_device);
    const long where = index != NULL ? PyLong_AsLong(index) : -1;
    Py_XDECREF(index);
    if (PyErr_Occurred()) return NULL;
    if (where != *gpu) {
      PyErr_Format(PyExc_ValueError, "ws: on GPU %ld, the tensors before it are on GPU %d", where, *gpu);
      return NULL;
    }
    PyObject* whole = PyObject_CallMethod(given, "is_contiguous", NULL);
    if (whole == NULL) return NULL;
    const int ok = whole == Py_True;
    Py_DECREF(whole);
    if (!ok) {
      PyErr_SetString(PyExc_ValueError, "ws: need a contiguous tensor");
      return NULL;
    }
    count = PyObject_GetAttrString(given, "nbytes");
    if (count != NULL) at = PyObject_CallMethodNoArgs(given, n_data_ptr);
    if (at != NULL) {
      *have = PyLong_AsSize_t(count);
      *ptr = PyLong_AsVoidPtr(at);
    }
    Py_XDECREF(count);
    Py_XDECREF(at);
    return PyErr_Occurred() ? NULL : Py_NewRef(given);
  }
  *have = bytes;
  PyObject* t = output(Py_None, "ws", g_f8, device, 1, (int64_t)bytes, (int64_t)bytes, 0, &v, gpu);
  *ptr = t != NULL ? v.ptr : NULL;
  return t;
}

/* few_fp8(x, gate_up, its scales, down, its scales, top_k, w_router, logits, router_bias, limit, renormalize,
 * routed_scale, num_experts, first, shared, shared_limit, rows, ws, out, stream) */
static PyObject* few_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor x = {0}, o;
  moe_fp8_weight gu, dn, sgu, sdn;
  moe_fp8_rows rows;
  const void *router, *logits, *bias;
  void *st, *ws;
  size_t have;
  int gpu = -1;
  if (!want(n, 20)) return NULL;
  moe_prefill_config c = {0};
  const int64_t top_k = PyLong_AsLongLong(a[5]), first = PyLong_AsLongLong(a[13]);
  c.swiglu_limit = (float)PyFloat_AsDouble(a[9]);
  c.renormalize = PyObject_IsTrue(a[10]);
  c.routed_scale = (float)PyFloat_AsDouble(a[11]);
  const float shared_limit = (float)PyFloat_AsDouble(a[15]);
  if (PyErr_Occurred() || !fits(top_k, "top_k")) return NULL;
  const int by_rows = a[16] != Py_None, with_shared = a[14] != Py_None;
  if (by_rows && (!PyTuple_Check(a[16]) || PyTuple_GET_SIZE(a[16]) != 2)) {
    PyErr_SetString(PyExc_ValueError, "rows: need a tuple of codes and scales");
    return NULL;
  }
  if (with_shared && (!PyTuple_Check(a[14]) || PyTuple_GET_SIZE(a[14]) != 4)) {
    PyErr_SetString(PyExc_ValueError, "shared: need a tuple of gate_up, its scales, down, its scales");
    return NULL;
  }
  if (a[0] == Py_None && (!by_rows || a[6] != Py_None)) {
    PyErr_SetString(PyExc_ValueError, "x: needed for the router, and where there are no rows");
    return NULL;
  }
  int64_t T = 0, H = 0;
  if (a[0] != Py_None) {
    if (!read_tensor(a[0], "x", 2, g_bf16, NULL, &x, &gpu)) return NULL;
    T = x.shape[0];
    H = x.shape[1];
    if (!unit_columns(&x, "x") || (T > 1 && x.stride[0] != H)) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "x: need a contiguous tensor");
      return NULL;
    }
  }
  if (by_rows) {
    int64_t K;
    if (!read_rows(PyTuple_GET_ITEM(a[16], 0), PyTuple_GET_ITEM(a[16], 1), "rows", "rows' scales", &rows, &K, &gpu)) return NULL;
    if (a[0] == Py_None) {
      T = rows.rows;
      H = K;
    }
    if (rows.rows != T || K != H) {
      PyErr_Format(PyExc_ValueError, "rows: need [%lld, %lld], got [%d, %lld]", (long long)T, (long long)H, rows.rows, (long long)K);
      return NULL;
    }
  }
  if (!read_weight(a[1], a[2], "w_gate_up", "s_gate_up", 3, first, &gu, &gpu) ||
      !read_weight(a[3], a[4], "w_down", "s_down", 3, first, &dn, &gpu))
    return NULL;
  if (with_shared && (!read_weight(PyTuple_GET_ITEM(a[14], 0), PyTuple_GET_ITEM(a[14], 1), "shared gate_up",
                                   "its scales", 2, 0, &sgu, &gpu) ||
                      !read_weight(PyTuple_GET_ITEM(a[14], 2), PyTuple_GET_ITEM(a[14], 3), "shared down", "its scales", 2,
                                   0, &sdn, &gpu)))
    return NULL;
  const int64_t E = a[12] == Py_None ? gu.count : PyLong_AsLongLong(a[12]);
  if (PyErr_Occurred() || !fits(E, "num_experts") || !fits(T, "tokens") || !fits(H, "columns")) return NULL;
  if (!read_plain(a[6], "w_router", 2, g_bf16, E, H, &router, &gpu) ||
      !read_plain(a[7], "logits", 2, g_f32, T, E, &logits, &gpu) ||
      !read_plain(a[8], "router_bias", 1, g_f32, E, 0, &bias, &gpu) || !stream_of(a[19], gpu, &st))
    return NULL;
  c.hidden = (int)H;
  c.moe_intermediate = dn.K;
  c.num_experts = (int)E;
  c.top_k = (int)top_k;
  PyObject* device = PyObject_GetAttr(a[1], n_device);
  if (device == NULL) return NULL;
  PyObject *tws = NULL, *out = output(a[18], "out", g_bf16, device, T, H, H, 0, &o, &gpu);
  if (out != NULL && (!unit_columns(&o, "out") || row_stride(&o, 1) != H)) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "out: need a contiguous tensor");
    Py_CLEAR(out);
  }
  if (out != NULL && T > 0) {
    tws = workspace(a[17], device, moe_few_workspace_bytes(&c, 1, with_shared ? sdn.K : 0, (int)T), &ws, &have, &gpu);
    if (tws == NULL) Py_CLEAR(out);
  }
  Py_DECREF(device);
  if (out == NULL || T == 0) return out;
  const int rc = moe_fp8_few_forward(&c, x.ptr, by_rows ? &rows : NULL, (int)T, router, logits, bias, &gu, &dn,
                                     with_shared ? &sgu : NULL, with_shared ? &sdn : NULL, shared_limit, ws, have, o.ptr, st);
  Py_DECREF(tws);
  if (rc == MOE_OK) return out;
  Py_DECREF(out);
  return fail(rc, "moe_fp8_few_forward");
}

/* few_w4(cfg, x, gate_up's handle, down's handle, w_router, logits, router_bias, shared_out, ws, out, stream) */
static PyObject* few_w4(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor x, o;
  const void *router, *logits, *bias, *shared;
  void *st, *ws, *tables[2];
  size_t have;
  int gpu = -1;
  moe_prefill_config c;
  Py_buffer view;
  if (!want(n, 11) || PyObject_GetBuffer(a[0], &view, PyBUF_SIMPLE) < 0) return NULL;
  const int whole = view.len == sizeof c;
  if (whole) c = *(const moe_prefill_config*)view.buf;
  PyBuffer_Release(&view);
  if (!whole) {
    PyErr_SetString(PyExc_ValueError, "cfg: need a MoePrefillConfig");
    return NULL;
  }
  for (int i = 0; i < 2; ++i) {
    PyObject* v = PyObject_GetAttrString(a[2 + i], "value");
    if (v == NULL) return NULL;
    tables[i] = v != Py_None ? PyLong_AsVoidPtr(v) : NULL;
    Py_DECREF(v);
    if (PyErr_Occurred()) return NULL;
  }
  if (!read_tensor(a[1], "x", 2, g_bf16, NULL, &x, &gpu)) return NULL;
  const int64_t T = x.shape[0], H = x.shape[1], E = c.num_experts;
  if (!unit_columns(&x, "x") || (T > 1 && x.stride[0] != H) || H != c.hidden) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "x: need a contiguous tensor of %d columns", c.hidden);
    return NULL;
  }
  if (!fits(T, "tokens") || !read_plain(a[4], "w_router", 2, g_bf16, E, H, &router, &gpu) ||
      !read_plain(a[5], "logits", 2, g_f32, T, E, &logits, &gpu) ||
      !read_plain(a[6], "router_bias", 1, g_f32, E, 0, &bias, &gpu) ||
      !read_plain(a[7], "shared_out", 2, g_bf16, T, H, &shared, &gpu) || !stream_of(a[10], gpu, &st))
    return NULL;
  PyObject* device = PyObject_GetAttr(a[1], n_device);
  if (device == NULL) return NULL;
  PyObject *tws = NULL, *out = output(a[9], "out", g_bf16, device, T, H, H, 0, &o, &gpu);
  if (out != NULL && (!unit_columns(&o, "out") || row_stride(&o, 1) != H)) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "out: need a contiguous tensor");
    Py_CLEAR(out);
  }
  if (out != NULL && T > 0) {
    tws = workspace(a[8], device, moe_few_workspace_bytes(&c, 0, 0, (int)T), &ws, &have, &gpu);
    if (tws == NULL) Py_CLEAR(out);
  }
  Py_DECREF(device);
  if (out == NULL || T == 0) return out;
  const int rc = moe_w4a16_few_forward(&c, x.ptr, (int)T, router, logits, bias, tables[0], tables[1], shared, ws, have, o.ptr, st);
  Py_DECREF(tws);
  if (rc == MOE_OK) return out;
  Py_DECREF(out);
  return fail(rc, "moe_w4a16_few_forward");
}

/* init(MoeError, torch.empty_strided, float8_e4m3fn, bfloat16, float32, int32, device index -> stream handle,
 * current device index) */
static PyObject* init(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  PyObject** to[8] = {&g_error, &g_empty, &g_f8, &g_bf16, &g_f32, &g_i32, &g_raw_stream, &g_current_device};
  if (!want(n, 8)) return NULL;
  for (int i = 0; i < 8; ++i) Py_XSETREF(*to[i], Py_NewRef(a[i]));
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))init, METH_FASTCALL, NULL},
    {"quantize", (PyCFunction)(void (*)(void))quantize, METH_FASTCALL, NULL},
    {"gemm", (PyCFunction)(void (*)(void))gemm, METH_FASTCALL, NULL},
    {"grouped", (PyCFunction)(void (*)(void))grouped, METH_FASTCALL, NULL},
    {"grouped_swiglu", (PyCFunction)(void (*)(void))grouped_swiglu, METH_FASTCALL, NULL},
    {"add_rms_norm", (PyCFunction)(void (*)(void))add_rms_norm, METH_FASTCALL, NULL},
    {"few_fp8", (PyCFunction)(void (*)(void))few_fp8, METH_FASTCALL, NULL},
    {"few_w4", (PyCFunction)(void (*)(void))few_w4, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8_call", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fp8_call(void) {
  n_dtype = PyUnicode_InternFromString("dtype");
  g_no_text = PyUnicode_InternFromString("");
  n_shape = PyUnicode_InternFromString("shape");
  n_stride = PyUnicode_InternFromString("stride");
  n_data_ptr = PyUnicode_InternFromString("data_ptr");
  n_device = PyUnicode_InternFromString("device");
  n_get_device = PyUnicode_InternFromString("get_device");
  n_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  kw_empty = Py_BuildValue("(ss)", "dtype", "device");
  if (PyErr_Occurred()) return NULL;
  return PyModule_Create(&module);
}
