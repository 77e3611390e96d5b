/*
 * operands.c -- the CPython module _operands: reads the tensors that the
 * binding's operator calls are given (shape, type, layout, address), checks
 * that they fit each other, and makes the call of the C ABI.
 *
 * A decode step makes such a call once a layer. On eight ranks of 5 tokens the
 * norm and rotation take 7.4 microseconds of host time here (Grace cores), and
 * took 14.3 with the attributes read from Python; an in-place addition of torch
 * takes 7.3. Tensors are read through their Python attributes, so the module
 * needs no torch headers; the C ABI's functions are those of the library that the
 * binding has loaded, by address. Nothing here touches the data.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>
#include <stdbool.h>
#include <stdint.h>

#include "rar.h"

enum { F32 = RAR_F32, BF16 = RAR_BF16, I32 = 2, OTHER = 3 };
enum { MAX_DIMS = 6 };

/* Set once by setup(): attribute names, torch's dtypes, the exception, the C ABI. */
static PyObject *s_shape, *s_dtype, *s_is_cuda, *s_is_contiguous, *s_stride, *s_data_ptr, *s_cuda_stream;
static PyObject *dtype_of[3]; /* by F32, BF16, I32 */
static PyObject *error_class, *current_device, *current_stream;
static struct {
  __typeof__(&rar_page_tables) page_tables;
  __typeof__(&rar_qk_norm_rope) qk_norm_rope;
  __typeof__(&rar_qk_norm_rope_cached) qk_norm_rope_cached;
  __typeof__(&rar_qk_norm_rope_backward) qk_norm_rope_backward;
  __typeof__(&rar_decode_attention) decode_attention;
  __typeof__(&rar_token_logprobs) token_logprobs;
  __typeof__(&rar_token_logprobs_backward) token_logprobs_backward;
  __typeof__(&rar_prompt_attention_ex) prompt_attention;
  __typeof__(&rar_prompt_attention_cached_ex) prompt_attention_cached;
  __typeof__(&rar_prompt_attention_backward_ex) prompt_attention_backward;
  __typeof__(&rar_embed_tokens) embed_tokens;
  __typeof__(&rar_embed_tokens_backward) embed_tokens_backward;
} abi;

/* Raises RarError(RAR_ERR_ARG, "name: what"); false, for the callers' returns. */
static bool refuse(const char* name, const char* what) {
  PyObject* e = PyObject_CallFunction(error_class, "iN", (int)RAR_ERR_ARG, PyUnicode_FromFormat("%s: %s", name, what));
  if (e != NULL) {
    PyErr_SetObject(error_class, e);
    Py_DECREF(e);
  }
  return false;
}

typedef struct {
  int dims, dtype;
  int64_t size[MAX_DIMS], stride[MAX_DIMS]; /* strides in elements */
  bool contiguous;
  char* data;
} Tensor;

static int64_t bytes_of(int dtype) { return dtype == BF16 ? 2 : 4; }

static bool truth(PyObject* o, bool* value) { /* steals o */
  if (o == NULL) return false;
  *value = o == Py_True;
  Py_DECREF(o);
  return true;
}

static bool integers(PyObject* tuple, int* count, int64_t* values) { /* steals tuple */
  bool ok = tuple != NULL && PyTuple_Check(tuple) && PyTuple_GET_SIZE(tuple) <= MAX_DIMS;
  if (ok) {
    *count = (int)PyTuple_GET_SIZE(tuple);
    for (int i = 0; i < *count && ok; i++) {
      values[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
      ok = !(values[i] == -1 && PyErr_Occurred());
    }
  }
  Py_XDECREF(tuple);
  return ok;
}

/* A tensor in device memory of one of the operators' types. */
static bool read_tensor(PyObject* t, const char* name, Tensor* out) {
  bool cuda = false;
  if (!integers(PyObject_GetAttr(t, s_shape), &out->dims, out->size) || !truth(PyObject_GetAttr(t, s_is_cuda), &cuda) ||
      !truth(PyObject_CallMethodNoArgs(t, s_is_contiguous), &out->contiguous)) {
    if (PyErr_Occurred()) return false;
    return refuse(name, "a tensor of at most 6 dimensions");
  }
  if (!cuda) return refuse(name, "in device memory");
  PyObject* dtype = PyObject_GetAttr(t, s_dtype);
  if (dtype == NULL) return false;
  out->dtype = dtype == dtype_of[F32] ? F32 : dtype == dtype_of[BF16] ? BF16 : dtype == dtype_of[I32] ? I32 : OTHER;
  Py_DECREF(dtype);
  if (out->contiguous) {
    int64_t s = 1;
    for (int i = out->dims - 1; i >= 0; i--) {
      out->stride[i] = s;
      s *= out->size[i];
    }
  } else {
    int dims = 0;
    if (!integers(PyObject_CallMethodNoArgs(t, s_stride), &dims, out->stride)) return false;
  }
  PyObject* data = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (data == NULL) return false;
  out->data = (char*)PyLong_AsVoidPtr(data);
  Py_DECREF(data);
  return !(out->data == NULL && PyErr_Occurred());
}

/* Tensor i of a list or tuple, held and bounds-checked: reading a subclass's attributes may run Python. */
static bool read_item(PyObject* x, Py_ssize_t i, const char* name, Tensor* out) {
  PyObject* t = PySequence_GetItem(x, i);
  if (t == NULL) return false;
  const bool ok = read_tensor(t, name, out);
  Py_DECREF(t);
  return ok;
}

/* A per-rank argument: a sequence of alike tensors, or one with the rank first. */
typedef struct {
  int ranks, dims, dtype;
  int64_t size[MAX_DIMS]; /* of a rank's tensor */
  int64_t row;            /* elements from row to row; the dimensions after a row's are dense */
  int64_t head;           /* of rows of heads: from head to head */
  bool dense;             /* no gaps between the rows either */
  void* data[RAR_MAX_RANKS];
} Ranked;

static bool lay_out(const int64_t* size, const int64_t* stride, int dims, const char* name, Ranked* out) {
  int64_t width = 1;
  for (int i = dims - 1; i > 0; i--) {
    if (size[i] != 1 && stride[i] != width) return refuse(name, "dense after its first dimension");
    width *= size[i];
  }
  out->dims = dims;
  for (int i = 0; i < dims; i++) out->size[i] = size[i];
  out->row = size[0] > 1 ? stride[0] : width;
  out->dense = out->row == width;
  return true;
}

/* [tokens, heads, head_dim] of which the last dimension alone is dense. */
static bool lay_out_heads(const int64_t* size, const int64_t* stride, const char* name, Ranked* out) {
  if (size[2] != 1 && stride[2] != 1) return refuse(name, "dense in its last dimension");
  out->dims = 3;
  for (int i = 0; i < 3; i++) out->size[i] = size[i];
  out->head = size[1] > 1 ? stride[1] : size[2];
  out->row = size[0] > 1 ? stride[0] : size[1] * out->head;
  out->dense = false;
  return true;
}

static bool read_laid_out(PyObject* x, const char* name, int dims, bool heads, Ranked* out) {
  Tensor t;
  if (PyList_Check(x) || PyTuple_Check(x)) {
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(x);
    if (n < 1 || n > RAR_MAX_RANKS) return refuse(name, "1 to 32 ranks");
    Tensor first;
    for (Py_ssize_t r = 0; r < n; r++) {
      if (!read_item(x, r, name, &t)) return false;
      if (r == 0) first = t;
      bool alike = t.dims == dims && t.dtype == first.dtype;
      for (int i = 0; i < dims && alike; i++) alike = t.size[i] == first.size[i] && t.stride[i] == first.stride[i];
      if (!alike) return refuse(name, "the ranks' tensors are alike and of the operator's dimensions");
      out->data[r] = t.data;
    }
    out->ranks = (int)n;
    out->dtype = first.dtype;
    return heads ? lay_out_heads(first.size, first.stride, name, out) : lay_out(first.size, first.stride, dims, name, out);
  }
  if (!read_tensor(x, name, &t)) return false;
  if (t.dims != dims + 1 || t.size[0] < 1 || t.size[0] > RAR_MAX_RANKS)
    return refuse(name, "1 to 32 ranks of the operator's dimensions");
  out->ranks = (int)t.size[0];
  out->dtype = t.dtype;
  const int64_t step = t.stride[0] * bytes_of(t.dtype);
  for (int r = 0; r < out->ranks; r++) out->data[r] = t.data == NULL ? NULL : t.data + r * step;
  return heads ? lay_out_heads(t.size + 1, t.stride + 1, name, out) : lay_out(t.size + 1, t.stride + 1, dims, name, out);
}
static bool read_ranked(PyObject* x, const char* name, int dims, Ranked* out) { return read_laid_out(x, name, dims, false, out); }
static bool read_heads(PyObject* x, const char* name, Ranked* out) { return read_laid_out(x, name, 3, true, out); }

static bool same_size(const Ranked* a, const Ranked* b) {
  if (a->ranks != b->ranks || a->dims != b->dims) return false;
  for (int i = 0; i < a->dims; i++)
    if (a->size[i] != b->size[i]) return false;
  return true;
}

/* A contiguous tensor of `count` elements (any number if below 0) of one type. */
static bool read_flat(PyObject* x, const char* name, int dtype, int64_t count, void** data, int64_t* found) {
  Tensor t;
  if (!read_tensor(x, name, &t)) return false;
  int64_t n = 1;
  for (int i = 0; i < t.dims; i++) n *= t.size[i];
  if (t.dtype != dtype || !t.contiguous || (count >= 0 && n != count))
    return refuse(name, dtype == I32   ? "contiguous int32 of the operator's size"
                        : dtype == F32 ? "contiguous float32 of the operator's size"
                                       : "contiguous bfloat16 of the operator's size");
  *data = t.data;
  if (found != NULL) *found = n;
  return true;
}

typedef struct {
  int32_t* data;
  int64_t stride;
  int columns;
} Table;

static bool read_table(PyObject* x, int64_t rows, Table* out) {
  Tensor t;
  if (!read_tensor(x, "block_table", &t)) return false;
  if (t.dtype != I32 || t.dims != 2 || t.size[0] != rows || (t.size[1] != 1 && t.stride[1] != 1) || t.size[1] > INT32_MAX)
    return refuse("block_table", "int32 [requests, max_blocks] with dense rows");
  out->data = (int32_t*)t.data;
  out->columns = (int)t.size[1];
  out->stride = rows > 1 ? t.stride[0] : t.size[1];
  return true;
}

typedef struct {
  void* data;
  size_t bytes;
  void* stream;
} Place;

/* workspace pointer, workspace bytes, stream: None (torch's current one), a handle, or a torch stream */
static bool read_place(PyObject* const* args, Place* out) {
  out->data = PyLong_AsVoidPtr(args[0]);
  out->bytes = PyLong_AsSize_t(args[1]);
  if (PyErr_Occurred()) return false;
  PyObject* handle;
  if (args[2] == Py_None) {
    PyObject* device = PyObject_CallNoArgs(current_device);
    if (device == NULL) return false;
    handle = PyObject_CallOneArg(current_stream, device);
    Py_DECREF(device);
  } else {
    handle = PyLong_Check(args[2]) ? Py_NewRef(args[2]) : PyObject_GetAttr(args[2], s_cuda_stream);
  }
  if (handle == NULL) return false;
  out->stream = PyLong_AsVoidPtr(handle);
  Py_DECREF(handle);
  return !PyErr_Occurred();
}

static bool floating(int dtype, const char* name) {
  if (dtype == F32 || dtype == BF16) return true;
  PyErr_Format(PyExc_TypeError, "%s: unsupported dtype (float32 or bfloat16)", name);
  return false;
}
static bool fits_int(int64_t v, const char* name) { return v <= INT32_MAX || refuse(name, "fewer than 2^31"); }

#define ARGUMENTS(count)                                                            \
  if (n != (count)) return PyErr_Format(PyExc_TypeError, "%d arguments are wanted", (int)(count))
#define CALL(...)                 \
  rar_status st;                  \
  Py_BEGIN_ALLOW_THREADS          \
  st = (__VA_ARGS__);             \
  Py_END_ALLOW_THREADS            \
  return PyLong_FromLong((long)st)

/* lens, new_tokens, free_pages, free_count, block_table, page_size, num_pages, lens_out, starts, positions, slots,
   free_count_out, place */
static PyObject* page_tables(PyObject* self, PyObject* const* v, Py_ssize_t n) {
  ARGUMENTS(15);
  void *lens, *add, *free_pages, *count, *lens_out, *starts, *positions, *slots, *count_out;
  int64_t requests, num_free, tokens;
  Table table;
  Place w;
  if (!read_flat(v[0], "lens", I32, -1, &lens, &requests) || !read_flat(v[1], "new_tokens", I32, requests, &add, NULL) ||
      !read_flat(v[2], "free_pages", I32, -1, &free_pages, &num_free) ||
      !read_flat(v[3], "free_count", I32, 1, &count, NULL) || !read_table(v[4], requests, &table) ||
      !read_flat(v[7], "lens_out", I32, requests, &lens_out, NULL) ||
      !read_flat(v[8], "starts", I32, requests + 1, &starts, NULL) ||
      !read_flat(v[9], "positions", I32, -1, &positions, &tokens) ||
      !read_flat(v[10], "slots", I32, tokens, &slots, NULL) ||
      !read_flat(v[11], "free_count_out", I32, 1, &count_out, NULL) || !read_place(v + 12, &w) ||
      !fits_int(requests, "lens") || !fits_int(num_free, "free_pages") || !fits_int(tokens, "positions"))
    return NULL;
  const int64_t page_size = PyLong_AsLongLong(v[5]), num_pages = PyLong_AsLongLong(v[6]);
  if (PyErr_Occurred()) return NULL;
  if (page_size < 0 || num_pages < 0) {
    refuse("page_size, num_pages", "not negative");
    return NULL;
  }
  if (!fits_int(page_size, "page_size") || !fits_int(num_pages, "num_pages")) return NULL;
  CALL(abi.page_tables(lens, add, (int)requests, free_pages, (int)num_free, count, (int)page_size, (int)num_pages, table.data,
                       table.stride, table.columns, lens_out, starts, positions, slots, (int)tokens, count_out, w.data,
                       w.bytes, w.stream));
}

/* What the forms of the norm and rotation share. */
typedef struct {
  Ranked qkv, q;
  int64_t tokens, max_pos, rot;
  int q_heads, kv_heads, dim, interleaved;
  float eps;
  void *q_weight, *k_weight, *cos_sin, *positions;
} Rope;

/* qkv, q_weight, k_weight, cos_sin, positions, queries, eps, interleaved; kv_heads from the keys */
static bool read_rope(PyObject* const* v, int64_t kv_heads, Rope* r) {
  Tensor t;
  if (!read_ranked(v[0], "qkv", 2, &r->qkv) || !read_ranked(v[5], "queries", 3, &r->q) || !floating(r->qkv.dtype, "qkv"))
    return false;
  r->tokens = r->q.size[0];
  const int64_t q_heads = r->q.size[1], dim = r->q.size[2];
  if (r->q.ranks != r->qkv.ranks || r->q.dtype != r->qkv.dtype || r->qkv.size[0] != r->tokens ||
      r->qkv.size[1] != (q_heads + 2 * kv_heads) * dim)
    return refuse("qkv", "[tokens, (q_heads + 2 kv_heads) head_dim], queries [tokens, q_heads, head_dim], of one dtype");
  if (!read_flat(v[1], "q_weight", r->qkv.dtype, dim, &r->q_weight, NULL) ||
      !read_flat(v[2], "k_weight", r->qkv.dtype, dim, &r->k_weight, NULL) || !read_tensor(v[3], "cos_sin", &t) ||
      !read_flat(v[4], "positions", I32, r->tokens, &r->positions, NULL))
    return false;
  if (t.dtype != F32 || t.dims != 2 || !t.contiguous) return refuse("cos_sin", "contiguous float32 [max_pos, rot_dim]");
  r->cos_sin = t.data;
  r->max_pos = t.size[0];
  r->rot = t.size[1];
  r->eps = (float)PyFloat_AsDouble(v[6]);
  r->interleaved = PyObject_IsTrue(v[7]);
  if (PyErr_Occurred()) return false;
  if (!fits_int(r->max_pos, "cos_sin") || !fits_int(r->rot, "cos_sin") || !fits_int(q_heads, "queries") ||
      !fits_int(kv_heads, "keys") || !fits_int(dim, "queries"))
    return false;
  r->q_heads = (int)q_heads;
  r->kv_heads = (int)kv_heads;
  r->dim = (int)dim;
  return true;
}
static bool keys_fit(const Ranked* k, const Rope* r, const char* name) {
  return (k->ranks == r->q.ranks && k->dtype == r->q.dtype && k->size[0] == r->tokens && k->size[1] == r->kv_heads &&
          k->size[2] == r->dim) ||
         refuse(name, "[tokens, kv_heads, head_dim] of qkv's dtype");
}

/* qkv .. interleaved as read_rope, k_out, place */
static PyObject* qk_norm_rope(PyObject* self, PyObject* const* v, Py_ssize_t n) {
  ARGUMENTS(12);
  Rope r;
  Ranked k;
  Place w;
  if (!read_ranked(v[8], "k_out", 3, &k) || !read_rope(v, k.size[1], &r) || !keys_fit(&k, &r, "k_out") ||
      !read_place(v + 9, &w))
    return NULL;
  CALL(abi.qk_norm_rope((const void* const*)r.qkv.data, r.q.ranks, r.tokens, r.qkv.row, r.q_weight, r.k_weight, r.cos_sin,
                        (int)r.max_pos, (int)r.rot, r.interleaved, r.positions, r.q_heads, r.kv_heads, r.dim,
                        (rar_dtype)r.q.dtype, r.eps, r.q.data, r.q.row, k.data, k.row, w.data, w.bytes, w.stream));
}

/* Paged caches of alike shape and type, without gaps. */
static bool read_caches(PyObject* k_cache, PyObject* v_cache, Ranked* k, Ranked* v) {
  if (!read_ranked(k_cache, "k_cache", 4, k) || !read_ranked(v_cache, "v_cache", 4, v)) return false;
  if (!k->dense || !v->dense || k->dtype != v->dtype || !same_size(k, v))
    return refuse("k_cache, v_cache", "contiguous [num_pages, kv_heads, page_size, head_dim], alike");
  return fits_int(k->size[0], "k_cache") && fits_int(k->size[1], "k_cache") && fits_int(k->size[2], "k_cache");
}

/* qkv .. interleaved as read_rope, slots, k_cache, v_cache, place */
static PyObject* qk_norm_rope_cached(PyObject* self, PyObject* const* v, Py_ssize_t n) {
  ARGUMENTS(14);
  Rope r;
  Ranked k, c;
  Place w;
  void* slots;
  if (!read_caches(v[9], v[10], &k, &c) || !read_rope(v, k.size[1], &r) ||
      !read_flat(v[8], "slots", I32, r.tokens, &slots, NULL))
    return NULL;
  if (k.ranks != r.q.ranks || k.dtype != r.q.dtype || k.size[3] != r.dim) {
    refuse("k_cache, v_cache", "[num_pages, kv_heads, page_size, head_dim] of qkv's dtype for each rank");
    return NULL;
  }
  if (!read_place(v + 11, &w)) return NULL;
  CALL(abi.qk_norm_rope_cached((const void* const*)r.qkv.data, r.q.ranks, r.tokens, r.qkv.row, r.q_weight, r.k_weight,
                               r.cos_sin, (int)r.max_pos, (int)r.rot, r.interleaved, r.positions, slots, r.q_heads,
                               r.kv_heads, r.dim, (rar_dtype)r.q.dtype, r.eps, r.q.data, r.q.row, k.data, c.data,
                               (int)k.size[0], (int)k.size[2], w.data, w.bytes, w.stream));
}

/* qkv .. interleaved as read_rope with dq for queries, dk, dv, dqkv, dq_weight, dk_weight, place */
static PyObject* qk_norm_rope_backward(PyObject* self, PyObject* const* v, Py_ssize_t n) {
  ARGUMENTS(16);
  Rope r;
  Ranked k, c, d, wq, wk;
  Place w;
  if (!read_ranked(v[8], "dk", 3, &k) || !read_ranked(v[9], "dv", 3, &c) || !read_rope(v, k.size[1], &r) ||
      !keys_fit(&k, &r, "dk") || !keys_fit(&c, &r, "dv") || !read_ranked(v[10], "dqkv", 2, &d) ||
      !read_ranked(v[11], "dq_weight", 1, &wq) || !read_ranked(v[12], "dk_weight", 1, &wk))
    return NULL;
  if (!same_size(&d, &r.qkv) || d.dtype != r.qkv.dtype) {
    refuse("dqkv", "as qkv");
    return NULL;
  }
  if (wq.ranks != r.q.ranks || !same_size(&wq, &wk) || wq.dtype != F32 || wk.dtype != F32 || wq.size[0] != r.dim ||
      !wq.dense || !wk.dense) {
    refuse("dq_weight, dk_weight", "float32 [head_dim] for each rank");
    return NULL;
  }
  if (!read_place(v + 13, &w)) return NULL;
  CALL(abi.qk_norm_rope_backward((const void* const*)r.qkv.data, r.q.ranks, r.tokens, r.qkv.row, r.q_weight, r.k_weight,
                                 r.cos_sin, (int)r.max_pos, (int)r.rot, r.interleaved, r.positions, r.q_heads, r.kv_heads,
                                 r.dim, (rar_dtype)r.q.dtype, r.eps, (const void* const*)r.q.data, r.q.row,
                                 (const void* const*)k.data, k.row, (const void* const*)c.data, c.row, d.data, d.row,
                                 (float* const*)wq.data, (float* const*)wk.data, w.data, w.bytes, w.stream));
}

/* q, k_cache, v_cache, block_table, lens, out, lse or None, scale or None, place */
static PyObject* decode_attention(PyObject* self, PyObject* const* v, Py_ssize_t n) {
  ARGUMENTS(11);
  Ranked q, k, c, out, lse;
  Table table;
  Place w;
  void* lens;
  if (!read_ranked(v[0], "q", 3, &q) || !floating(q.dtype, "q") || !read_caches(v[1], v[2], &k, &c) ||
      !read_table(v[3], q.size[0], &table) || !read_flat(v[4], "lens", I32, q.size[0], &lens, NULL) ||
      !read_ranked(v[5], "out", 3, &out))
    return NULL;
  if (k.ranks != q.ranks || k.dtype != q.dtype || k.size[3] != q.size[2] || !same_size(&out, &q) || out.dtype != q.dtype ||
      q.size[0] > INT32_MAX || q.size[1] > INT32_MAX || q.size[2] > INT32_MAX) {
    refuse("q, out", "[batch, q_heads, head_dim] of the caches' dtype and head_dim for each rank");
    return NULL;
  }
  const bool with_lse = v[6] != Py_None;
  if (with_lse) {
    if (!read_ranked(v[6], "lse", 2, &lse)) return NULL;
    if (lse.ranks != q.ranks || lse.dtype != F32 || !lse.dense || lse.size[0] != q.size[0] || lse.size[1] != q.size[1]) {
      refuse("lse", "contiguous float32 [batch, q_heads] for each rank");
      return NULL;
    }
  }
  const double scale = v[7] == Py_None ? 1.0 / sqrt((double)q.size[2]) : PyFloat_AsDouble(v[7]);
  if (PyErr_Occurred() || !read_place(v + 8, &w)) return NULL;
  CALL(abi.decode_attention((const void* const*)q.data, q.row, (const void* const*)k.data, (const void* const*)c.data,
                            q.ranks, (int)q.size[0], (int)q.size[1], (int)k.size[1], (int)q.size[2], (rar_dtype)q.dtype,
                            (int)k.size[0], (int)k.size[2], table.data, table.stride, table.columns, lens, (float)scale,
                            out.data, out.row, with_lse ? (float* const*)lse.data : NULL, w.data, w.bytes, w.stream));
}

/* Vocabulary shards: as read_ranked, but the shards may differ in width. */
typedef struct {
  int ranks, dtype;
  int64_t rows, width[RAR_MAX_RANKS], row[RAR_MAX_RANKS];
  void* data[RAR_MAX_RANKS];
} Shards;

static bool read_shards(PyObject* x, const char* name, Shards* out) {
  Ranked r;
  if (!PyList_Check(x) && !PyTuple_Check(x)) {
    if (!read_ranked(x, name, 2, &r)) return false;
    out->ranks = r.ranks;
    out->dtype = r.dtype;
    out->rows = r.size[0];
    for (int i = 0; i < r.ranks; i++) {
      out->width[i] = r.size[1];
      out->row[i] = r.row;
      out->data[i] = r.data[i];
    }
    return floating(out->dtype, name);
  }
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(x);
  if (n < 1 || n > RAR_MAX_RANKS) return refuse(name, "1 to 32 ranks");
  for (Py_ssize_t i = 0; i < n; i++) {
    Tensor t;
    if (!read_item(x, i, name, &t)) return false;
    if (t.dims != 2 || !lay_out(t.size, t.stride, 2, name, &r))
      return PyErr_Occurred() ? false : refuse(name, "[rows, vocabulary of the shard]");
    if (i == 0) {
      out->rows = t.size[0];
      out->dtype = t.dtype;
    }
    if (t.size[0] != out->rows || t.dtype != out->dtype) return refuse(name, "[rows, vocabulary of the shard], of one dtype");
    out->width[i] = t.size[1];
    out->row[i] = r.row;
    out->data[i] = t.data;
  }
  out->ranks = (int)n;
  return floating(out->dtype, name);
}

/* logits, tokens, logprob, entropy, lse, top_values, top_ids (both None: no alternatives), place */
static PyObject* token_logprobs(PyObject* self, PyObject* const* v, Py_ssize_t n) {
  ARGUMENTS(10);
  Shards x;
  Place w;
  void *tokens, *logprob, *entropy, *lse, *values = NULL, *ids = NULL;
  int64_t top = 0;
  if (!read_shards(v[0], "logits", &x) || !read_flat(v[1], "tokens", I32, x.rows, &tokens, NULL) ||
      !read_flat(v[2], "logprob", F32, x.rows, &logprob, NULL) || !read_flat(v[3], "entropy", F32, x.rows, &entropy, NULL) ||
      !read_flat(v[4], "lse", F32, x.rows, &lse, NULL))
    return NULL;
  if (v[6] != Py_None) {
    Tensor t;
    if (!read_tensor(v[6], "top_ids", &t)) return NULL;
    if (t.dtype != I32 || !t.contiguous || t.dims != 2 || t.size[0] != x.rows) {
      refuse("top_ids", "contiguous int32 [rows, top]");
      return NULL;
    }
    top = t.size[1];
    ids = t.data;
    if (!fits_int(top, "top_ids") || (top > 0 && !read_flat(v[5], "top_values", F32, x.rows * top, &values, NULL))) return NULL;
  }
  if (!read_place(v + 7, &w)) return NULL;
  CALL(abi.token_logprobs((const void* const*)x.data, x.width, x.row, x.ranks, x.rows, (rar_dtype)x.dtype, tokens, logprob,
                          entropy, lse, (int)top, values, ids, w.data, w.bytes, w.stream));
}

/* logits, tokens, lse, entropy, grad_logprob, grad_entropy or None, dlogits, place */
static PyObject* token_logprobs_backward(PyObject* self, PyObject* const* v, Py_ssize_t n) {
  ARGUMENTS(10);
  Shards x, d;
  Place w;
  void *tokens, *lse, *entropy, *gl, *gh = NULL;
  if (!read_shards(v[0], "logits", &x) || !read_shards(v[6], "dlogits", &d) ||
      !read_flat(v[1], "tokens", I32, x.rows, &tokens, NULL) || !read_flat(v[2], "lse", F32, x.rows, &lse, NULL) ||
      !read_flat(v[3], "entropy", F32, x.rows, &entropy, NULL) ||
      !read_flat(v[4], "grad_logprob", F32, x.rows, &gl, NULL) ||
      (v[5] != Py_None && !read_flat(v[5], "grad_entropy", F32, x.rows, &gh, NULL)))
    return NULL;
  bool alike = d.ranks == x.ranks && d.rows == x.rows && d.dtype == x.dtype;
  for (int r = 0; r < x.ranks && alike; r++) alike = d.width[r] == x.width[r];
  if (!alike) {
    refuse("dlogits", "as logits");
    return NULL;
  }
  if (!read_place(v + 7, &w)) return NULL;
  CALL(abi.token_logprobs_backward((const void* const*)x.data, x.width, x.row, x.ranks, x.rows, (rar_dtype)x.dtype, tokens,
                                   lse, entropy, gl, gh, d.data, d.row, w.data, w.bytes, w.stream));
}

/* Queries, [tokens, heads, head_dim] a rank, and what the forms of the attention over prompts share. */
typedef struct {
  Ranked q;
  void* starts;
  int sequences;
  float scale;
} Prompt;

/* q, starts, scale or None */
static bool read_prompt(PyObject* q, PyObject* starts, PyObject* scale, Prompt* p) {
  int64_t bounds;
  if (!read_heads(q, "q", &p->q) || !floating(p->q.dtype, "q") ||
      !read_flat(starts, "starts", I32, -1, &p->starts, &bounds) || !fits_int(bounds, "starts") ||
      !fits_int(p->q.size[1], "q") || !fits_int(p->q.size[2], "q"))
    return false;
  if (bounds < 1) return refuse("starts", "one more than the sequences");
  p->sequences = (int)(bounds - 1);
  p->scale = (float)(scale == Py_None ? 1.0 / sqrt((double)p->q.size[2]) : PyFloat_AsDouble(scale));
  return !PyErr_Occurred();
}
/* A tensor as the queries are. */
static bool read_like(PyObject* x, const char* name, const Ranked* q, Ranked* out) {
  if (!read_heads(x, name, out)) return false;
  return (same_size(out, q) && out->dtype == q->dtype) || refuse(name, "as q");
}
/* Keys or values: [tokens, kv_heads, head_dim] with the queries' tokens and head_dim. */
static bool read_keys(PyObject* x, const char* name, const Ranked* q, Ranked* out) {
  if (!read_heads(x, name, out)) return false;
  return (out->ranks == q->ranks && out->dtype == q->dtype && out->size[0] == q->size[0] && out->size[2] == q->size[2] &&
          out->size[1] <= INT32_MAX) ||
         refuse(name, "[tokens, kv_heads, head_dim] of q's tokens, head_dim and dtype");
}
static bool read_lse(PyObject* x, const Ranked* q, Ranked* out) {
  if (!read_ranked(x, "lse", 2, out)) return false;
  return (out->ranks == q->ranks && out->dtype == F32 && out->dense && out->size[0] == q->size[0] &&
          out->size[1] == q->size[1]) ||
         refuse("lse", "contiguous float32 [tokens, q_heads] for each rank");
}

/* q, k, v, starts, out, lse or None, scale or None, place */
static PyObject* prompt_attention(PyObject* self, PyObject* const* v, Py_ssize_t n) {
  ARGUMENTS(10);
  Prompt p;
  Ranked k, c, out, lse;
  Place w;
  if (!read_prompt(v[0], v[3], v[6], &p) || !read_keys(v[1], "k", &p.q, &k) || !read_keys(v[2], "v", &p.q, &c) ||
      !read_like(v[4], "out", &p.q, &out) || (v[5] != Py_None && !read_lse(v[5], &p.q, &lse)))
    return NULL;
  if (!same_size(&k, &c)) {
    refuse("k, v", "alike");
    return NULL;
  }
  if (!read_place(v + 7, &w)) return NULL;
  CALL(abi.prompt_attention((const void* const*)p.q.data, p.q.row, p.q.head, (const void* const*)k.data, k.row, k.head,
                            (const void* const*)c.data, c.row, c.head, p.q.ranks, p.q.size[0], (int)p.q.size[1],
                            (int)k.size[1], (int)p.q.size[2], (rar_dtype)p.q.dtype, p.starts, p.sequences, p.scale,
                            out.data, out.row, out.head, v[5] != Py_None ? (float* const*)lse.data : NULL, w.data, w.bytes, w.stream));
}

/* q, k_cache, v_cache, block_table, starts, lens, out, lse or None, scale or None, place */
static PyObject* prompt_attention_cached(PyObject* self, PyObject* const* v, Py_ssize_t n) {
  ARGUMENTS(12);
  Prompt p;
  Ranked k, c, out, lse;
  Table table;
  Place w;
  void* lens;
  if (!read_prompt(v[0], v[4], v[8], &p) || !read_caches(v[1], v[2], &k, &c) || !read_table(v[3], p.sequences, &table) ||
      !read_flat(v[5], "lens", I32, p.sequences, &lens, NULL) || !read_like(v[6], "out", &p.q, &out) ||
      (v[7] != Py_None && !read_lse(v[7], &p.q, &lse)))
    return NULL;
  if (k.ranks != p.q.ranks || k.dtype != p.q.dtype || k.size[3] != p.q.size[2]) {
    refuse("k_cache, v_cache", "[num_pages, kv_heads, page_size, head_dim] of q's dtype and head_dim for each rank");
    return NULL;
  }
  if (!read_place(v + 9, &w)) return NULL;
  CALL(abi.prompt_attention_cached((const void* const*)p.q.data, p.q.row, p.q.head, (const void* const*)k.data,
                                   (const void* const*)c.data, p.q.ranks, p.q.size[0], (int)p.q.size[1], (int)k.size[1],
                                   (int)p.q.size[2], (rar_dtype)p.q.dtype, (int)k.size[0], (int)k.size[2], table.data,
                                   table.stride, table.columns, p.starts, lens, p.sequences, p.scale, out.data, out.row, out.head,
                                   v[7] != Py_None ? (float* const*)lse.data : NULL, w.data, w.bytes, w.stream));
}

/* q, k, v, starts, out, lse, dout, dq, dk, dv, scale or None, place */
static PyObject* prompt_attention_backward(PyObject* self, PyObject* const* v, Py_ssize_t n) {
  ARGUMENTS(14);
  Prompt p;
  Ranked k, c, out, lse, dout, dq, dk, dv;
  Place w;
  if (!read_prompt(v[0], v[3], v[10], &p) || !read_keys(v[1], "k", &p.q, &k) || !read_keys(v[2], "v", &p.q, &c) ||
      !read_like(v[4], "out", &p.q, &out) || !read_lse(v[5], &p.q, &lse) || !read_like(v[6], "dout", &p.q, &dout) ||
      !read_like(v[7], "dq", &p.q, &dq) || !read_keys(v[8], "dk", &p.q, &dk) || !read_keys(v[9], "dv", &p.q, &dv))
    return NULL;
  if (!same_size(&k, &c) || !same_size(&k, &dk) || !same_size(&k, &dv)) {
    refuse("k, v, dk, dv", "alike");
    return NULL;
  }
  if (!read_place(v + 11, &w)) return NULL;
  CALL(abi.prompt_attention_backward((const void* const*)p.q.data, p.q.row, p.q.head, (const void* const*)k.data, k.row,
                                     k.head, (const void* const*)c.data, c.row, c.head, p.q.ranks, p.q.size[0], (int)p.q.size[1],
                                     (int)k.size[1], (int)p.q.size[2], (rar_dtype)p.q.dtype, p.starts, p.sequences, p.scale,
                                     (const void* const*)out.data, out.row, out.head, (const float* const*)lse.data,
                                     (const void* const*)dout.data, dout.row, dout.head, dq.data, dq.row, dq.head, dk.data,
                                     dk.row, dk.head, dv.data, dv.row, dv.head, w.data, w.bytes, w.stream));
}

/* [tokens, width] rows that the ranks share. */
static bool read_shared_rows(PyObject* x, const char* name, int dtype, int64_t rows, int64_t width, void** data,
                             int64_t* stride) {
  Tensor t;
  if (!read_tensor(x, name, &t)) return false;
  if (t.dims != 2 || t.dtype != dtype || t.size[0] != rows || t.size[1] != width || (width > 1 && t.stride[1] != 1))
    return refuse(name, "[tokens, hidden] with dense rows");
  *data = t.data;
  *stride = rows > 1 ? t.stride[0] : width;
  return true;
}
static bool one_width(const Shards* x, const char* name, int64_t* hidden) {
  *hidden = x->width[0];
  for (int r = 1; r < x->ranks; r++)
    if (x->width[r] != *hidden) return refuse(name, "of one width");
  return fits_int(*hidden, name);
}

/* Table shards: as read_shards, but alike in width and not in rows. */
static bool read_tables(PyObject* x, const char* name, Shards* out, int64_t* vocab, int64_t* hidden) {
  if (PyList_Check(x) || PyTuple_Check(x)) {
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(x);
    if (n < 1 || n > RAR_MAX_RANKS) return refuse(name, "1 to 32 ranks");
    Ranked r;
    for (Py_ssize_t i = 0; i < n; i++) {
      Tensor t;
      if (!read_item(x, i, name, &t)) return false;
      if (t.dims != 2 || !lay_out(t.size, t.stride, 2, name, &r))
        return PyErr_Occurred() ? false : refuse(name, "[vocabulary of the shard, hidden]");
      if (i == 0) out->dtype = t.dtype;
      if (t.dtype != out->dtype) return refuse(name, "of one dtype");
      vocab[i] = t.size[0];
      out->width[i] = t.size[1];
      out->row[i] = r.row;
      out->data[i] = t.data;
    }
    out->ranks = (int)n;
  } else {
    if (!read_shards(x, name, out)) return false;
    for (int r = 0; r < out->ranks; r++) vocab[r] = out->rows;
  }
  return one_width(out, name, hidden);
}

/* tokens, tables, out, scale, place */
static PyObject* embed_tokens(PyObject* self, PyObject* const* v, Py_ssize_t n) {
  ARGUMENTS(7);
  Shards x;
  Place w;
  void *tokens, *out;
  int64_t count, hidden, stride, vocab[RAR_MAX_RANKS];
  if (!read_flat(v[0], "tokens", I32, -1, &tokens, &count) || !read_tables(v[1], "tables", &x, vocab, &hidden) ||
      !floating(x.dtype, "tables") || !read_shared_rows(v[2], "out", x.dtype, count, hidden, &out, &stride))
    return NULL;
  const float scale = (float)PyFloat_AsDouble(v[3]);
  if (PyErr_Occurred() || !read_place(v + 4, &w)) return NULL;
  CALL(abi.embed_tokens(tokens, count, (const void* const*)x.data, vocab, x.row, x.ranks, (int)hidden, (rar_dtype)x.dtype,
                        scale, out, stride, w.data, w.bytes, w.stream));
}

/* tokens, dout, dtables, scale, accumulate, place */
static PyObject* embed_tokens_backward(PyObject* self, PyObject* const* v, Py_ssize_t n) {
  ARGUMENTS(8);
  Shards x;
  Place w;
  Tensor t;
  void *tokens, *dout;
  int64_t count, hidden, stride, vocab[RAR_MAX_RANKS];
  if (!read_flat(v[0], "tokens", I32, -1, &tokens, &count) || !read_tables(v[2], "dtables", &x, vocab, &hidden) ||
      !read_tensor(v[1], "dout", &t) || !floating(t.dtype, "dout") ||
      !read_shared_rows(v[1], "dout", t.dtype, count, hidden, &dout, &stride))
    return NULL;
  if (x.dtype != F32) {
    refuse("dtables", "float32 [vocabulary of the shard, hidden] for each rank");
    return NULL;
  }
  const float scale = (float)PyFloat_AsDouble(v[3]);
  const int accumulate = PyObject_IsTrue(v[4]);
  if (PyErr_Occurred() || !read_place(v + 5, &w)) return NULL;
  CALL(abi.embed_tokens_backward(tokens, count, dout, stride, (rar_dtype)t.dtype, scale, (float* const*)x.data, vocab, x.row,
                                 x.ranks, (int)hidden, accumulate, w.data, w.bytes, w.stream));
}

/* setup(RarError, (float32, bfloat16, int32), addresses of the functions in the order of `abi`, function of the
   current device, function of a device's current stream handle) */
static PyObject* setup(PyObject* self, PyObject* args) {
  PyObject *cls, *dtypes, *addresses, *device, *stream;
  if (!PyArg_ParseTuple(args, "OO!O!OO", &cls, &PyTuple_Type, &dtypes, &PyTuple_Type, &addresses, &device, &stream))
    return NULL;
  if (PyTuple_GET_SIZE(dtypes) != 3 || PyTuple_GET_SIZE(addresses) * sizeof(void*) != sizeof abi)
    return PyErr_Format(PyExc_TypeError, "three dtypes and an address for each function are wanted");
  void** to = (void**)&abi;
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(addresses); i++) to[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addresses, i));
  if (PyErr_Occurred()) return NULL;
  for (int i = 0; i < 3; i++) Py_XSETREF(dtype_of[i], Py_NewRef(PyTuple_GET_ITEM(dtypes, i)));
  Py_XSETREF(error_class, Py_NewRef(cls));
  Py_XSETREF(current_device, Py_NewRef(device));
  Py_XSETREF(current_stream, Py_NewRef(stream));
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, NULL}, FAST(page_tables), FAST(qk_norm_rope), FAST(qk_norm_rope_cached),
    FAST(qk_norm_rope_backward), FAST(decode_attention), FAST(token_logprobs), FAST(token_logprobs_backward),
    FAST(prompt_attention), FAST(prompt_attention_cached), FAST(prompt_attention_backward), FAST(embed_tokens),
    FAST(embed_tokens_backward),
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_operands", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__operands(void) {
  s_shape = PyUnicode_InternFromString("shape");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_is_cuda = PyUnicode_InternFromString("is_cuda");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_stride = PyUnicode_InternFromString("stride");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (s_shape == NULL || s_dtype == NULL || s_is_cuda == NULL || s_is_contiguous == NULL || s_stride == NULL ||
      s_data_ptr == NULL || s_cuda_stream == NULL)
    return NULL;
  return PyModule_Create(&module);
}
