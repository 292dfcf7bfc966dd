// binding.cpp -- the usual calls of the Python binding without the interpreter's
// part: arguments checked, outputs allocated and the C ABI called in one go (a
// call of these operators takes 5 to 10 us on the GPU; checking and marshalling it
// in Python took 13).
//
// Every function here does a whole call or nothing: it returns None for anything
// that is not the plain valid case -- another device or stream, an output that is
// given, a wrong type, shape or stride, an error code -- and the Python function,
// which knows all cases and their errors, goes on from there.  The C ABI's
// functions arrive as addresses (init), so there is one copy of the library.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/TracerMode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "entro.h"

namespace {

decltype(&entro_quantize_tokens) f_quantize;
decltype(&entro_matmul_i8) f_matmul;
decltype(&entro_attention_prompt) f_prompt;
decltype(&entro_kv_append) f_append;
decltype(&entro_kv_read) f_read;
decltype(&entro_kv_attend) f_attend;

using at::ScalarType;
using at::Tensor;

// A tensor argument on device `index` (-1: sets it), without a gradient to take or a tangent to carry on; null if it is
// none of that.
const Tensor *tensor(PyObject *o, int &index) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided) return nullptr;
    const int at = t.get_device();
    if (index < 0) index = at;
    if (at != index || (t.requires_grad() && c10::GradMode::is_enabled()) || t._fw_grad(0).defined()) return nullptr;
    return &t;
}
// The same, or None (which leaves `t` null).
bool maybe_tensor(PyObject *o, int &index, const Tensor *&t) {
    t = nullptr;
    return o == Py_None || (t = tensor(o, index)) != nullptr;
}
// The status word: None, or an int32 tensor
bool status_word(PyObject *o, int &index, const Tensor *&t) {
    return maybe_tensor(o, index, t) && (!t || (t->scalar_type() == ScalarType::Int && t->numel() >= 1));
}
bool vector(const Tensor *t, ScalarType type, int64_t n) {
    return t && t->scalar_type() == type && t->dim() == 1 && t->size(0) == n && t->is_contiguous();
}
template <typename T = void>
T *data(const Tensor *t) {
    return t ? static_cast<T *>(t->data_ptr()) : nullptr;
}
int type_of(ScalarType t) {
    switch (t) {
        case ScalarType::Float: return ENTRO_F32;
        case ScalarType::BFloat16: return ENTRO_BF16;
        case ScalarType::Half: return ENTRO_F16;
        case ScalarType::Byte: return ENTRO_U8;
        case ScalarType::Char: return ENTRO_S8;
        default: return -1;
    }
}
bool half_type(ScalarType t) { return t == ScalarType::BFloat16 || t == ScalarType::Half; }

Tensor make(c10::IntArrayRef size, ScalarType type, int index) {
    return at::detail::empty_cuda(size, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(index)), std::nullopt);
}
// The current device, and no trace being taken: a call's result would be a constant of it.
bool here(int index) { return c10::cuda::current_device() == index && !at::tracer::impl::is_dispatch_enabled(); }
void *stream(int index) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream(); }

// [tokens, heads, dim] in 16-byte pieces: token and head stride (0 where there is one)
struct Rows {
    int64_t token = 0, head = 0;
    bool of(const Tensor *t, ScalarType type, int64_t heads, int64_t dim) {
        if (!t || t->scalar_type() != type || t->dim() != 3 || t->size(1) != heads || t->size(2) != dim || t->stride(2) != 1) return false;
        token = t->size(0) > 1 ? t->stride(0) : 0;
        head = heads > 1 ? t->stride(1) : 0;
        return ((token | head) & 7) == 0 && (reinterpret_cast<uintptr_t>(t->data_ptr()) & 15) == 0;
    }
};

bool number(PyObject *o, double &v) {
    if (PyFloat_CheckExact(o)) v = PyFloat_AS_DOUBLE(o);
    else if (PyLong_CheckExact(o)) {
        v = PyLong_AsDouble(o);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return false;
        }
    } else return false;
    return true;
}
// None: 1 / sqrt(dim)
bool scale_of(PyObject *o, int64_t dim, float &scale) {
    double v = 1.0 / std::sqrt(static_cast<double>(dim));
    if (o != Py_None && !number(o, v)) return false;
    scale = static_cast<float>(v);
    return scale > 0.0f && scale <= 2.0e38f;
}

// quantize_tokens(x) -> (codes, scale, sum)
PyObject *quantize_tokens(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int index = -1;
    const Tensor *x = n == 1 ? tensor(args[0], index) : nullptr;
    if (!x || !half_type(x->scalar_type()) || x->dim() != 2 || x->size(1) < 1 || x->stride(1) != 1 || !here(index)) Py_RETURN_NONE;
    const int64_t tokens = x->size(0), cols = x->size(1), pitch = (cols + 15) / 16 * 16;
    Tensor codes = make({tokens, pitch}, ScalarType::Char, index);
    Tensor scale = make({tokens}, ScalarType::Float, index), sum = make({tokens}, ScalarType::Int, index);
    if (f_quantize(x->data_ptr(), type_of(x->scalar_type()), tokens, cols, tokens > 1 ? x->stride(0) : pitch, data<int8_t>(&codes), pitch,
                   data<float>(&scale), data<int32_t>(&sum), stream(index)) != ENTRO_OK)
        Py_RETURN_NONE;
    if (pitch != cols) codes = codes.narrow(1, 0, cols);
    PyObject *r = PyTuple_New(3);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(codes)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(scale)));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(sum)));
    return r;
    END_HANDLE_TH_ERRORS
}

// matmul_i8(codes, scale, sum, w, w_scale, w_zero, out type, status) -> out
PyObject *matmul_i8(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8) Py_RETURN_NONE;
    int index = -1;
    const Tensor *q = tensor(args[0], index), *xs = q ? tensor(args[1], index) : nullptr, *xz = xs ? tensor(args[2], index) : nullptr,
                 *w = xz ? tensor(args[3], index) : nullptr, *ws = nullptr, *wz = nullptr, *status = nullptr;
    if (!w || !here(index) || !status_word(args[7], index, status)) Py_RETURN_NONE;
    if (q->scalar_type() != ScalarType::Char || q->dim() != 2 || q->stride(1) != 1) Py_RETURN_NONE;
    const ScalarType wt = w->scalar_type();
    if ((wt != ScalarType::Byte && wt != ScalarType::Char) || w->dim() != 2 || w->stride(1) != 1) Py_RETURN_NONE;
    const int64_t tokens = q->size(0), cols = q->size(1), rows = w->size(0), pitch = (cols + 15) / 16 * 16;
    if (cols < 1 || w->size(1) != cols || !vector(xs, ScalarType::Float, tokens) || !vector(xz, ScalarType::Int, tokens)) Py_RETURN_NONE;
    double all = 0.0;
    if (!number(args[4], all) && (!(ws = tensor(args[4], index)) || !vector(ws, ScalarType::Float, rows))) Py_RETURN_NONE;
    long zero = 0;
    if (PyLong_CheckExact(args[5])) {
        int over = 0;
        zero = PyLong_AsLongAndOverflow(args[5], &over);
        if (over || zero < INT32_MIN || zero > INT32_MAX) Py_RETURN_NONE;
    } else if (args[5] != Py_None && (!(wz = tensor(args[5], index)) || !vector(wz, ScalarType::Int, rows))) {
        Py_RETURN_NONE;
    }
    const long out_type = PyLong_CheckExact(args[6]) ? PyLong_AsLong(args[6]) : -1;
    if (out_type != ENTRO_F32 && out_type != ENTRO_BF16 && out_type != ENTRO_F16) Py_RETURN_NONE;
    Tensor out = make({tokens, rows}, out_type == ENTRO_F32 ? ScalarType::Float : out_type == ENTRO_BF16 ? ScalarType::BFloat16 : ScalarType::Half, index);
    if (f_matmul(data<int8_t>(q), tokens > 1 ? q->stride(0) : pitch, data<float>(xs), data<int32_t>(xz), tokens, w->data_ptr(), type_of(wt),
                 rows > 1 ? w->stride(0) : pitch, rows, cols, data<float>(ws), static_cast<float>(all), data<int32_t>(wz), static_cast<int32_t>(zero),
                 out.data_ptr(), static_cast<int32_t>(out_type), rows, data<int32_t>(status), stream(index)) != ENTRO_OK)
        Py_RETURN_NONE;
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// attention_prompt(q, k, v, cu_seqlens, cu_keys, scale, status) -> out
PyObject *attention_prompt(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7) Py_RETURN_NONE;
    int index = -1;
    const Tensor *q = tensor(args[0], index), *k = q ? tensor(args[1], index) : nullptr, *v = k ? tensor(args[2], index) : nullptr,
                 *cu = v ? tensor(args[3], index) : nullptr, *cu_keys = nullptr, *status = nullptr;
    if (!cu || !here(index) || !maybe_tensor(args[4], index, cu_keys) || !status_word(args[6], index, status)) Py_RETURN_NONE;
    const ScalarType type = q->scalar_type();
    if (!half_type(type) || q->dim() != 3 || k->dim() != 3 || cu->dim() != 1 || cu->size(0) < 1) Py_RETURN_NONE;
    const int64_t tokens = q->size(0), heads = q->size(1), dim = q->size(2), keys = k->size(0), kv = k->size(1), batch = cu->size(0) - 1;
    Rows qs, ks, vs;
    float scale;
    if (kv < 1 || heads < 1 || heads % kv || v->size(0) != keys || !qs.of(q, type, heads, dim) || !ks.of(k, type, kv, dim) || !vs.of(v, type, kv, dim) ||
        !scale_of(args[5], dim, scale) || !vector(cu, ScalarType::Int, batch + 1) || (cu_keys && !vector(cu_keys, ScalarType::Int, batch + 1)) ||
        batch > INT32_MAX || (dim != 64 && dim != 96 && dim != 128))
        Py_RETURN_NONE;
    Tensor out = make({tokens, heads, dim}, type, index);
    if (f_prompt(type_of(type), static_cast<int32_t>(dim), q->data_ptr(), qs.token, qs.head, static_cast<int32_t>(heads), tokens, k->data_ptr(),
                 ks.token, ks.head, v->data_ptr(), vs.token, vs.head, static_cast<int32_t>(kv), keys, data<int32_t>(cu), data<int32_t>(cu_keys),
                 static_cast<int32_t>(batch), scale, out.data_ptr(), heads * dim, dim, data<int32_t>(status), stream(index)) != ENTRO_OK)
        Py_RETURN_NONE;
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// What the cache's calls share: the cache (address of its entro_kv_cache, device), the page table and the tail slots.
struct CacheCall {
    const entro_kv_cache *cache = nullptr;
    int index = -1;
    const Tensor *table = nullptr, *slots = nullptr;
    int64_t batch = 0, width = 0, stride = 0;
    ScalarType type = ScalarType::Half;
    bool of(PyObject *address, PyObject *device, PyObject *page_table, PyObject *slot_of) {
        cache = static_cast<const entro_kv_cache *>(PyLong_AsVoidPtr(address));
        index = static_cast<int>(PyLong_AsLong(device));
        if (!cache || PyErr_Occurred()) {
            PyErr_Clear();
            return false;
        }
        if (index < 0 || !here(index) || !(table = tensor(page_table, index)) || !maybe_tensor(slot_of, index, slots)) return false;
        if (table->scalar_type() != ScalarType::Int || table->dim() != 2) return false;
        batch = table->size(0), width = table->size(1), stride = batch > 1 ? table->stride(0) : width;
        if ((width > 1 && table->stride(1) != 1) || stride < width || batch > INT32_MAX || width > INT32_MAX) return false;
        type = cache->type == ENTRO_BF16 ? ScalarType::BFloat16 : ScalarType::Half;
        return slots ? vector(slots, ScalarType::Int, batch) : batch <= cache->slots;
    }
};

// kv_append(cache, device, k, v, cu_seqlens, page_table, lens, slots, status) -> True
PyObject *kv_append(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    CacheCall c;
    if (n != 9 || !c.of(args[0], args[1], args[5], args[7])) Py_RETURN_NONE;
    const Tensor *k = tensor(args[2], c.index), *v = tensor(args[3], c.index), *cu = tensor(args[4], c.index), *lens = tensor(args[6], c.index), *status;
    Rows ks, vs;
    if (!status_word(args[8], c.index, status) || !ks.of(k, c.type, c.cache->kv_heads, c.cache->head_dim) ||
        !vs.of(v, c.type, c.cache->kv_heads, c.cache->head_dim) || k->size(0) != v->size(0) || !vector(cu, ScalarType::Int, c.batch + 1) ||
        !vector(lens, ScalarType::Int, c.batch))
        Py_RETURN_NONE;
    if (f_append(c.cache, k->data_ptr(), ks.token, ks.head, v->data_ptr(), vs.token, vs.head, k->size(0), data<int32_t>(cu), data<int32_t>(c.table),
                 c.stride, static_cast<int32_t>(c.width), data<int32_t>(lens), data<int32_t>(c.slots), static_cast<int32_t>(c.batch),
                 data<int32_t>(status), stream(c.index)) != ENTRO_OK)
        Py_RETURN_NONE;
    Py_RETURN_TRUE;
    END_HANDLE_TH_ERRORS
}

// kv_read(cache, device, page_table, cu_seqlens, tokens, slots, status) -> (k, v)
PyObject *kv_read(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    CacheCall c;
    if (n != 7 || !c.of(args[0], args[1], args[2], args[5]) || !PyLong_CheckExact(args[4])) Py_RETURN_NONE;
    const Tensor *cu = tensor(args[3], c.index), *status;
    int over = 0;
    const long tokens = PyLong_AsLongAndOverflow(args[4], &over);
    if (over || tokens < 0 || !status_word(args[6], c.index, status) || !vector(cu, ScalarType::Int, c.batch + 1)) Py_RETURN_NONE;
    const int64_t heads = c.cache->kv_heads, dim = c.cache->head_dim;
    Tensor k = make({tokens, heads, dim}, c.type, c.index), v = make({tokens, heads, dim}, c.type, c.index);
    if (f_read(c.cache, k.data_ptr(), heads * dim, dim, v.data_ptr(), heads * dim, dim, tokens, data<int32_t>(cu), data<int32_t>(c.table), c.stride,
               static_cast<int32_t>(c.width), data<int32_t>(c.slots), static_cast<int32_t>(c.batch), data<int32_t>(status), stream(c.index)) != ENTRO_OK)
        Py_RETURN_NONE;
    PyObject *r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(k)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(v)));
    return r;
    END_HANDLE_TH_ERRORS
}

// kv_attend(cache, device, workspace bytes, q, page_table, lens, slots, scale, status) -> out
PyObject *kv_attend(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    CacheCall c;
    if (n != 9 || !c.of(args[0], args[1], args[4], args[6]) || !PyLong_CheckExact(args[2])) Py_RETURN_NONE;
    const long bytes = PyLong_AsLong(args[2]);
    const Tensor *q = tensor(args[3], c.index), *lens = tensor(args[5], c.index), *status;
    const int64_t dim = c.cache->head_dim, heads = q && q->dim() == 3 ? q->size(1) : 0;
    Rows qs;
    float scale;
    if (bytes < 1 || !status_word(args[8], c.index, status) || heads < 1 || heads % c.cache->kv_heads || !qs.of(q, c.type, heads, dim) ||
        q->size(0) != c.batch || !vector(lens, ScalarType::Int, c.batch) || !scale_of(args[7], dim, scale))
        Py_RETURN_NONE;
    // a workspace of the call's own, from the pool of the stream it runs on: calls never share one
    Tensor work = make({bytes}, ScalarType::Byte, c.index), out = make({c.batch, heads, dim}, c.type, c.index);
    if (f_attend(c.cache, q->data_ptr(), qs.token, qs.head, static_cast<int32_t>(heads), data<int32_t>(c.table), c.stride,
                 static_cast<int32_t>(c.width), data<int32_t>(lens), data<int32_t>(c.slots), static_cast<int32_t>(c.batch), scale, out.data_ptr(),
                 heads * dim, dim, work.data_ptr(), static_cast<uint64_t>(bytes), data<int32_t>(status), stream(c.index)) != ENTRO_OK)
        Py_RETURN_NONE;
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// init(addresses of the six functions)
PyObject *init(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "six addresses");
        return nullptr;
    }
    void *p[6];
    for (int i = 0; i < 6; i++) p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
    f_quantize = reinterpret_cast<decltype(f_quantize)>(p[0]);
    f_matmul = reinterpret_cast<decltype(f_matmul)>(p[1]);
    f_prompt = reinterpret_cast<decltype(f_prompt)>(p[2]);
    f_append = reinterpret_cast<decltype(f_append)>(p[3]);
    f_read = reinterpret_cast<decltype(f_read)>(p[4]);
    f_attend = reinterpret_cast<decltype(f_attend)>(p[5]);
    Py_RETURN_NONE;
}

#define ENTRO_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRO_METHOD(init),      ENTRO_METHOD(quantize_tokens), ENTRO_METHOD(matmul_i8), ENTRO_METHOD(attention_prompt),
                         ENTRO_METHOD(kv_append), ENTRO_METHOD(kv_read),         ENTRO_METHOD(kv_attend), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
