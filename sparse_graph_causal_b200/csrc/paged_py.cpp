// paged_py.cpp -- argument marshalling of the paged cache's Python calls.
//
// A serving step makes these calls once or twice per layer on a few tokens,
// where the GPU is done in four to six microseconds, and reading the tensors'
// addresses, types, shapes and strides in Python and handing them over by ctypes
// takes as long again: 8.3 to 9.9 us a call on the host, 4.0 to 4.4 through this
// module (a bare launch takes 3 to 4).  It reads them in C++ and calls
// the library's C entry points; it computes nothing.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/sparse_attn.h"

namespace {

// A Python error is set.
struct Raised {};

[[noreturn]] void raise_value(const std::string &message) {
    PyErr_SetString(PyExc_ValueError, message.c_str());
    throw Raised();
}

std::string text(at::IntArrayRef shape) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + ")";
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) raise_value(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

bool lies_on(const at::Tensor &t, int64_t index) {
    return t.is_cuda() && t.get_device() == index;
}

// Address of a contiguous tensor of this type and shape on CUDA device `index`.
void *array(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape,
            int64_t index) {
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type || t.sizes() != shape || !lies_on(t, index) || !t.is_contiguous())
        raise_value(std::string(name) + " must be a contiguous " + toString(type) +
                    " tensor of shape " + text(shape) + " on cuda:" + std::to_string(index));
    return t.data_ptr();
}

int32_t row_type(const at::Tensor &t) {
    return t.scalar_type() == at::kBFloat16 ? SA_BF16 : t.scalar_type() == at::kFloat ? SA_FP32 : -1;
}

int64_t integer(PyObject *o) {
    const int64_t x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised();
    return x;
}

template <typename T>
T *pointer(PyObject *o) {
    if (o == Py_None) return nullptr;
    return reinterpret_cast<T *>(static_cast<uintptr_t>(integer(o)));
}

// call(stream) with the tensors' device current, on its current stream unless
// one is given.
template <typename F>
PyObject *call_on(int64_t index, PyObject *stream, F call) {
    const c10::cuda::OptionalCUDAGuard guard(
        index == c10::cuda::current_device()
            ? std::nullopt
            : std::optional<c10::Device>(c10::Device(c10::kCUDA, (c10::DeviceIndex)index)));
    void *s = stream == Py_None
                  ? (void *)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream()
                  : pointer<void>(stream);
    return PyLong_FromLong(call(s));
}

// Runs a binding; what it throws becomes a Python error.
template <typename F>
PyObject *guarded(Py_ssize_t given, Py_ssize_t wanted, F run) {
    if (given != wanted) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return run();
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// length, n_new, block_table, free_pages, free_count, page_size, batch
// (address of its sa_paged_step), index, length_out, free_count_out, stream
PyObject *plan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        sa_paged_step s = *pointer<const sa_paged_step>(a[6]);
        const int64_t index = integer(a[7]);
        const at::Tensor &table = tensor(a[2], "block_table"), &free_pages = tensor(a[3], "free_pages");
        if (table.dim() != 2 || table.size(0) != s.B)
            raise_value("block_table must be [B, max_pages], B that of the batch (" +
                        std::to_string(s.B) + ")");
        s.max_pages = table.size(1);
        s.page_size = integer(a[5]);
        s.n_stack = free_pages.numel();
        const int64_t one = 1;
        s.len = (const int64_t *)array(a[0], "length", at::kLong, s.B, index);
        s.n_new = (const int32_t *)array(a[1], "n_new", at::kInt, s.B, index);
        s.block_table = (int32_t *)array(a[2], "block_table", at::kInt, table.sizes(), index);
        s.free_pages = (int32_t *)array(a[3], "free_pages", at::kInt, s.n_stack, index);
        s.free_count = (const int64_t *)array(a[4], "free_count", at::kLong, one, index);
        s.len_out = a[8] == Py_None ? const_cast<int64_t *>(s.len)
                                    : (int64_t *)array(a[8], "length_out", at::kLong, s.B, index);
        s.free_count_out = a[9] == Py_None
                               ? const_cast<int64_t *>(s.free_count)
                               : (int64_t *)array(a[9], "free_count_out", at::kLong, one, index);
        return call_on(index, a[10], [&](void *t) { return sparse_attn_paged_plan(&s, t); });
    });
}

// New rows [N, Hkv, D] or [N, Hkv, 1, D] with any stride between tokens.
int64_t token_rows(PyObject *o, const char *name, const sa_paged_cache &c, int64_t index,
                   sa_tensor *rows) {
    const at::Tensor &t = tensor(o, name);
    const int64_t d = t.dim() - 1;  // the columns' dimension
    if (!lies_on(t, index) || (d != 2 && !(d == 3 && t.size(2) == 1)) || t.size(1) != c.Hkv ||
        t.size(d) != c.D || t.stride(d) != 1 || (c.Hkv > 1 && t.stride(1) != c.D) ||
        row_type(t) < 0)
        raise_value(std::string(name) + " must be bf16 or fp32 [N, " + std::to_string(c.Hkv) +
                    ", " + std::to_string(c.D) + "] with contiguous heads on cuda:" +
                    std::to_string(index));
    *rows = {t.data_ptr(), row_type(t), t.size(0), c.Hkv, 1, c.D};
    return t.size(0) > 1 ? t.stride(0) : c.Hkv * c.D;
}

// k_new, v_new, cache (address), index, slot, stream
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const sa_paged_cache &c = *pointer<const sa_paged_cache>(a[2]);
        const int64_t index = integer(a[3]);
        sa_tensor k, v;
        const int64_t ks = token_rows(a[0], "k_new", c, index, &k);
        const int64_t vs = token_rows(a[1], "v_new", c, index, &v);
        const int64_t *slot = (const int64_t *)array(a[4], "slot", at::kLong, k.B, index);
        if (k.B == 0 && v.B == 0) return PyLong_FromLong(SA_OK);
        return call_on(index, a[5], [&](void *t) {
            return sparse_attn_paged_append(&k, ks, &v, vs, slot, &c, t);
        });
    });
}

// q, cache (address), index, block_table, pos, graph, scale, row, out, lse,
// workspace, stream
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 12, [&] {
        const sa_paged_cache &c = *pointer<const sa_paged_cache>(a[1]);
        const int64_t index = integer(a[2]);
        const at::Tensor &q = tensor(a[0], "q"), &table = tensor(a[3], "block_table");
        if (!lies_on(q, index) || q.dim() != 4 || !q.is_contiguous() || row_type(q) < 0)
            raise_value("q must be a contiguous bf16 or fp32 [N, H, 1, D] tensor on cuda:" +
                        std::to_string(index));
        if (table.dim() != 2) raise_value("block_table must be [rows, max_pages]");
        const int64_t N = q.size(0), H = q.size(1), lse_shape[] = {N, H};
        const sa_tensor tq = {q.data_ptr(), row_type(q), N, H, q.size(2), q.size(3)};
        sa_tensor to = tq;
        to.ptr = array(a[8], "out", q.scalar_type(), q.sizes(), index);
        float *lse = (float *)array(a[9], "lse", at::kFloat, lse_shape, index);
        const int32_t *pages =
            (const int32_t *)array(a[3], "block_table", at::kInt, table.sizes(), index);
        const int64_t *pos = (const int64_t *)array(a[4], "pos", at::kLong, N, index);
        const int32_t *row =
            a[7] == Py_None ? nullptr : (const int32_t *)array(a[7], "row", at::kInt, N, index);
        void *ws = nullptr;
        size_t ws_bytes = 0;
        if (a[10] != Py_None) {
            const at::Tensor &w = tensor(a[10], "workspace");
            if (!lies_on(w, index) || !w.is_contiguous())
                raise_value("workspace must be contiguous on cuda:" + std::to_string(index));
            ws = w.data_ptr();
            ws_bytes = w.nbytes();
        }
        const double scale = PyFloat_AsDouble(a[6]);
        if (scale == -1.0 && PyErr_Occurred()) throw Raised();
        const sa_graph g = pointer<std::remove_pointer_t<sa_graph>>(a[5]);
        if (N == 0) return PyLong_FromLong(SA_OK);
        return call_on(index, a[11], [&](void *t) {
            return sparse_attn_paged_decode(&tq, &c, pages, table.size(0), table.size(1), row, pos,
                                            g, (float)scale, &to, lse, ws, ws_bytes, t);
        });
    });
}

PyMethodDef methods[] = {
    {"plan", (PyCFunction)(void (*)())plan, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)())append, METH_FASTCALL, nullptr},
    {"decode", (PyCFunction)(void (*)())decode, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods,
                      nullptr,               nullptr,  nullptr, nullptr};

}  // namespace

// The module works on the tensors of the torch that it was built with.
PyMODINIT_FUNC PyInit__paged() {
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
    const char *v = version ? PyUnicode_AsUTF8(version) : nullptr;
    const bool same = v && std::string(v) == SA_TORCH_VERSION;
    if (v && !same)
        PyErr_Format(PyExc_ImportError,
                     "built for torch %s, torch is %s", SA_TORCH_VERSION, v);
    Py_XDECREF(version);
    Py_XDECREF(torch);
    return same ? PyModule_Create(&module) : nullptr;
}
