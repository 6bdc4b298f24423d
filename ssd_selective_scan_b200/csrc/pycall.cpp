// pycall.cpp -- the Python extension behind diag.py: checks of tensors'
// types, shapes, strides and devices, and direct calls of the entry points of
// include/ssd_diag.h.
//
// A decode step's calls run for a few microseconds on the device, and each
// takes up to 14 tensors and 28 arguments: checked by interpreted code and
// converted by ctypes, they took the host longer than the device.  Here a
// tensor's check reads its fields (about 0.1 us, where it took 1), and an
// argument is converted by its C type.
//
// No state; errors are Python exceptions (torch's own C++ ones are translated).
// SSD_BUILT_FOR names the torch and Python of the headers (build.py).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <limits>
#include <tuple>
#include <type_traits>
#include <utility>

#include "ssd_diag.h"

namespace {

constexpr int kMaxDims = 8;

bool arity(const char* fn, Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) PyErr_Format(PyExc_TypeError, "%s: %zd arguments expected, %zd given", fn, want, n);
    return n == want;
}

const at::Tensor* as_tensor(PyObject* o, PyObject* name)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%U must be a tensor", name);
        return nullptr;
    }
    return &THPVariable_Unpack(o);
}

// The integers of a tuple (a shape); -1 on an error.
int as_dims(PyObject* o, int64_t* v)
{
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) > kMaxDims) {
        PyErr_SetString(PyExc_TypeError, "a shape must be a tuple");
        return -1;
    }
    const int n = (int)PyTuple_GET_SIZE(o);
    for (int i = 0; i < n; ++i) {
        v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
        if (v[i] == -1 && PyErr_Occurred()) return -1;
    }
    return n;
}

bool has_shape(const at::Tensor& t, const int64_t* v, int n)
{
    if (t.dim() != n) return false;
    for (int i = 0; i < n; ++i)
        if (t.size(i) != v[i]) return false;
    return true;
}

void bad_dense(PyObject* name, PyObject* dtype, PyObject* shape, PyObject* device)
{
    PyObject* plain = PySequence_Tuple(shape);   // a torch.Size prints as a tuple
    if (plain) PyErr_Format(PyExc_ValueError, "%U must be a contiguous %S tensor of shape %S on %S", name, dtype, plain, device);
    Py_XDECREF(plain);
}

PyObject* pointer(const at::Tensor& t) { return PyLong_FromVoidPtr(t.data_ptr()); }

// dense(t, name, dtype, shape, device): the pointer of a contiguous tensor of
// this type and shape (None passes)
PyObject* dense(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!arity("dense", n, 5)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;
    const at::Tensor* t = as_tensor(a[0], a[1]);
    int64_t dims[kMaxDims];
    const int nd = t ? as_dims(a[3], dims) : -1;
    if (nd < 0) return nullptr;
    if (!THPDtype_Check(a[2]) || !THPDevice_Check(a[4])) {
        PyErr_SetString(PyExc_TypeError, "dense: a dtype and a device expected");
        return nullptr;
    }
    if (t->scalar_type() != reinterpret_cast<THPDtype*>(a[2])->scalar_type || t->device() != reinterpret_cast<THPDevice*>(a[4])->device ||
        !has_shape(*t, dims, nd) || !t->is_contiguous()) {
        bad_dense(a[1], a[2], a[3], a[4]);
        return nullptr;
    }
    return pointer(*t);
    END_HANDLE_TH_ERRORS
}

// The spacing of the rows of a [*lead, E] tensor, its strides st[0 .. nlead]; a
// dimension of one row says nothing about it.  -1 (and an exception) where the
// rows are not dense and evenly spaced.
int64_t row_stride(const at::Tensor& t, const int64_t* st, PyObject* name, const int64_t* lead, int nlead, int64_t E)
{
    const int64_t L = lead[nlead - 1];
    const bool some = t.numel() > 0;
    if (st[nlead] != 1 && E > 1 && some) {
        PyErr_Format(PyExc_ValueError, "%U must have dense rows", name);
        return -1;
    }
    if (nlead == 1) return L > 1 ? st[0] : E;
    if (!some) return E;
    if (lead[0] > 1 && L > 1 && st[0] != L * st[1]) {
        PyErr_Format(PyExc_ValueError, "%U must have evenly spaced rows", name);
        return -1;
    }
    return L > 1 ? st[1] : lead[0] > 1 ? st[0] : E;
}

bool lead_of(PyObject* o, int64_t* lead, int& nlead)
{
    nlead = as_dims(o, lead);
    if (nlead < 0) return false;
    if (nlead != 1 && nlead != 2) PyErr_SetString(PyExc_TypeError, "one or two leading dimensions expected");
    return nlead == 1 || nlead == 2;
}

// rows(t, name, lead, E, like): (pointer, row stride) of a [*lead, E] tensor of
// like's type and device whose rows are evenly spaced and dense
PyObject* rows(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!arity("rows", n, 5)) return nullptr;
    if (a[0] == Py_None) return Py_BuildValue("(OO)", Py_None, a[3]);
    const at::Tensor* t = as_tensor(a[0], a[1]);
    const at::Tensor* like = t ? as_tensor(a[4], a[1]) : nullptr;
    int64_t dims[kMaxDims];
    int nlead;
    if (!like || !lead_of(a[2], dims, nlead)) return nullptr;
    dims[nlead] = PyLong_AsLongLong(a[3]);
    if (dims[nlead] == -1 && PyErr_Occurred()) return nullptr;
    if (!has_shape(*t, dims, nlead + 1) || t->scalar_type() != like->scalar_type() || t->device() != like->device()) {
        PyObject* last = PyTuple_Pack(1, a[3]);
        PyObject* shape = last ? PySequence_Concat(a[2], last) : nullptr;
        Py_XDECREF(last);
        PyObject* of = PyObject_GetAttrString(a[4], "dtype");
        PyObject* on = PyObject_GetAttrString(a[4], "device");
        if (shape && of && on) PyErr_Format(PyExc_ValueError, "%U must be a %S tensor of shape %S on %S", a[1], of, shape, on);
        Py_XDECREF(shape);
        Py_XDECREF(of);
        Py_XDECREF(on);
        return nullptr;
    }
    const int64_t s = row_stride(*t, t->strides().data(), a[1], dims, nlead, dims[nlead]);
    if (s < 0) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "%U must have dense rows", a[1]);
    return Py_BuildValue("(NL)", pointer(*t), (long long)s);
    END_HANDLE_TH_ERRORS
}

// bc(B, C, lead, like): [*lead, G, N] tensors as (pointer, pointer, row stride, G, N)
PyObject* bc(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!arity("bc", n, 4)) return nullptr;
    PyObject* names[2] = {PyUnicode_InternFromString("B"), PyUnicode_InternFromString("C")};
    struct Release {
        PyObject** p;
        ~Release() { Py_XDECREF(p[0]); Py_XDECREF(p[1]); }
    } release{names};
    if (!names[0] || !names[1]) return nullptr;
    const at::Tensor* t[2] = {as_tensor(a[0], names[0]), nullptr};
    if (!t[0] || !(t[1] = as_tensor(a[1], names[1]))) return nullptr;
    const at::Tensor* like = as_tensor(a[3], names[0]);
    int64_t lead[kMaxDims];
    int nlead;
    if (!like || !lead_of(a[2], lead, nlead)) return nullptr;
    if (t[0]->sizes() != t[1]->sizes() || t[0]->dim() != nlead + 2 || !std::equal(lead, lead + nlead, t[0]->sizes().begin()))
        return PyErr_Format(PyExc_ValueError, "B and C must share the shape (%S, G, N)", a[2]);
    const int64_t G = t[0]->size(nlead), N = t[0]->size(nlead + 1);
    int64_t stride = 0;
    for (int i = 0; i < 2; ++i) {
        if (t[i]->scalar_type() != like->scalar_type() || t[i]->device() != like->device())
            return PyErr_Format(PyExc_ValueError, "B and C must have u's type and device");
        if (G > 1 && t[i]->stride(nlead) != N && t[i]->numel())
            return PyErr_Format(PyExc_ValueError, "%U: dense (G, N) rows expected", names[i]);
        int64_t st[3];
        for (int k = 0; k < nlead; ++k) st[k] = t[i]->stride(k);
        st[nlead] = t[i]->stride(nlead + 1);
        const int64_t s = row_stride(*t[i], st, names[i], lead, nlead, G * N);
        if (s < 0) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "%U: dense (G, N) rows expected", names[i]);
        if (i && s != stride) return PyErr_Format(PyExc_ValueError, "B and C must share one row stride");
        stride = s;
    }
    return Py_BuildValue("(NNLLL)", pointer(*t[0]), pointer(*t[1]), (long long)stride, (long long)G, (long long)N);
    END_HANDLE_TH_ERRORS
}

// where(like): (device, raw handle of its current stream, whether it is the
// current device) of a CUDA tensor
PyObject* where(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!arity("where", n, 1)) return nullptr;
    if (!THPVariable_Check(a[0])) {
        PyErr_SetString(PyExc_TypeError, "a tensor expected");
        return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(a[0]);
    if (!t.is_cuda()) {
        PyErr_SetString(PyExc_ValueError, "CUDA tensors expected");
        return nullptr;
    }
    const c10::Device dev = t.device();
    const auto stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    return Py_BuildValue("(NKN)", THPDevice_New(dev), (unsigned long long)(uintptr_t)stream,
                         PyBool_FromLong(c10::cuda::current_device() == dev.index()));
    END_HANDLE_TH_ERRORS
}

// map_in(cu_seqlens, seq_of, slot_of, init_slot, T, device): the pointers of a
// state map's parts for T rows, and its requests
PyObject* map_in(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!arity("map_in", n, 6)) return nullptr;
    static const char* const names[] = {"cu_seqlens", "seq_of", "slot_of", "init_slot"};
    const at::Tensor* t[4];
    for (int i = 0; i < 4; ++i) {
        if (!THPVariable_Check(a[i])) return PyErr_Format(PyExc_TypeError, "%s must be a tensor", names[i]);
        t[i] = &THPVariable_Unpack(a[i]);
    }
    const int64_t T = PyLong_AsLongLong(a[4]);
    if (T == -1 && PyErr_Occurred()) return nullptr;
    if (!THPDevice_Check(a[5])) return PyErr_Format(PyExc_TypeError, "map_in: a device expected");
    const int64_t nseq = t[0]->numel() - 1;
    const int64_t len[] = {nseq + 1, T, T, nseq};
    for (int i = 0; i < 4; ++i) {
        const auto type = i == 2 ? at::ScalarType::Long : at::ScalarType::Int;
        if (len[i] < 0 || t[i]->scalar_type() != type || t[i]->device() != reinterpret_cast<THPDevice*>(a[5])->device ||
            !has_shape(*t[i], &len[i], 1) || !t[i]->is_contiguous())
            return PyErr_Format(PyExc_ValueError, "%s must be a contiguous torch.%s tensor of shape (%lld,) on %S", names[i],
                                i == 2 ? "int64" : "int32", (long long)len[i], a[5]);
    }
    return Py_BuildValue("(NNNNL)", pointer(*t[0]), pointer(*t[1]), pointer(*t[2]), pointer(*t[3]), (long long)nseq);
    END_HANDLE_TH_ERRORS
}

// map_out(requests, max_blocks, rows, extra, device): a new state map's
// cu_seqlens, seq_of, pos_of, slot_of, init_slot, table and free_head, then the
// address of `extra` more int32: one allocation, each part on 16 bytes.
PyObject* map_out(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!arity("map_out", n, 5)) return nullptr;
    int64_t v[4];
    for (int i = 0; i < 4; ++i) {
        v[i] = PyLong_AsLongLong(a[i]);
        if (v[i] == -1 && PyErr_Occurred()) return nullptr;
        if (v[i] < 0 || v[i] > std::numeric_limits<int>::max()) return PyErr_Format(PyExc_ValueError, "map_out: a size out of range");
    }
    if (!THPDevice_Check(a[4])) return PyErr_Format(PyExc_TypeError, "map_out: a device expected");
    const int64_t reqs = v[0], blocks = v[1], T = v[2];
    const auto on = at::TensorOptions().device(reinterpret_cast<THPDevice*>(a[4])->device);
    const int64_t sizes[] = {reqs + 1, T, T, 2 * T, reqs, reqs * blocks, 1};   // in int32
    int64_t at[8] = {0};
    for (int i = 0; i < 7; ++i) at[i + 1] = at[i] + (sizes[i] + 3) / 4 * 4;
    const at::Tensor whole = at::empty({at[7] + v[3]}, on.dtype(at::kInt));
    auto view = [&](int i, at::IntArrayRef shape, at::IntArrayRef strides) {
        // as detach() makes a second tensor of one storage, at a place and shape of its own
        auto impl = whole.unsafeGetTensorImpl()->shallow_copy_and_detach(c10::VariableVersion(0), /*allow_tensor_metadata_change=*/true);
        if (i == 3) impl->set_storage_and_dtype(whole.storage(), caffe2::TypeMeta::fromScalarType(at::kLong));
        impl->set_sizes_and_strides(shape, strides, i == 3 ? at[i] / 2 : at[i]);
        return THPVariable_Wrap(at::Tensor(std::move(impl)));
    };
    const int64_t row = blocks > 0 ? blocks : 1;
    return Py_BuildValue("(NNNNNNNN)", view(0, {reqs + 1}, {1}), view(1, {T}, {1}), view(2, {T}, {1}), view(3, {T}, {1}),
                         view(4, {reqs}, {1}), view(5, {reqs, blocks}, {row, 1}), view(6, {1}, {1}),
                         PyLong_FromVoidPtr(whole.data_ptr<int>() + at[7]));
    END_HANDLE_TH_ERRORS
}

// empty(shape, dtype, device): torch.empty
PyObject* empty(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!arity("empty", n, 3)) return nullptr;
    int64_t dims[kMaxDims];
    const int nd = as_dims(a[0], dims);
    if (nd < 0) return nullptr;
    if (!THPDtype_Check(a[1]) || !THPDevice_Check(a[2])) {
        PyErr_SetString(PyExc_TypeError, "empty: a dtype and a device expected");
        return nullptr;
    }
    return THPVariable_Wrap(at::empty(at::IntArrayRef(dims, nd), at::TensorOptions()
                                                                     .dtype(reinterpret_cast<THPDtype*>(a[1])->scalar_type)
                                                                     .device(reinterpret_cast<THPDevice*>(a[2])->device)));
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------------
// the entry points: fn(arguments in the header's order), pointers as integers
// or None

template <typename T> bool convert(PyObject* o, T& v)
{
    if constexpr (std::is_pointer_v<T>) {
        v = nullptr;
        if (o == Py_None) return true;
        v = (T)PyLong_AsVoidPtr(o);
        return v || !PyErr_Occurred();
    } else if constexpr (std::is_same_v<T, size_t>) {
        v = PyLong_AsSize_t(o);
        return v != (size_t)-1 || !PyErr_Occurred();
    } else {
        const long long i = PyLong_AsLongLong(o);
        if (i == -1 && PyErr_Occurred()) return false;
        if constexpr (sizeof(T) == 4) {
            if (i < std::numeric_limits<int>::min() || i > std::numeric_limits<int>::max()) {
                PyErr_SetString(PyExc_OverflowError, "argument beyond int");
                return false;
            }
        }
        v = (T)i;
        return true;
    }
}

template <auto F> struct Entry;
template <typename R, typename... A, R (*F)(A...)> struct Entry<F> {
    template <size_t... I> static PyObject* go(PyObject* const* a, std::index_sequence<I...>)
    {
        std::tuple<A...> v;
        if (!(convert(a[I], std::get<I>(v)) && ...)) return nullptr;
        R r;
        Py_BEGIN_ALLOW_THREADS
        r = F(std::get<I>(v)...);
        Py_END_ALLOW_THREADS
        if constexpr (std::is_same_v<R, size_t>) return PyLong_FromSize_t(r);
        else return PyLong_FromLong((long)r);
    }
    static PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n)
    {
        if (!arity("entry point", n, sizeof...(A))) return nullptr;
        return go(a, std::make_index_sequence<sizeof...(A)>{});
    }
};

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) { return (PyCFunction)(void (*)(void))f; }

#define ENTRY(name) {#name, fast(Entry<name>::call), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"dense", fast(dense), METH_FASTCALL, nullptr},
    {"rows", fast(rows), METH_FASTCALL, nullptr},
    {"bc", fast(bc), METH_FASTCALL, nullptr},
    {"empty", fast(empty), METH_FASTCALL, nullptr},
    {"where", fast(where), METH_FASTCALL, nullptr},
    {"map_in", fast(map_in), METH_FASTCALL, nullptr},
    {"map_out", fast(map_out), METH_FASTCALL, nullptr},
    ENTRY(ssd_state_map_workspace_bytes),
    ENTRY(ssd_state_map),
    ENTRY(ssd_conv1d_silu_varlen),
    ENTRY(ssd_conv1d_silu_bwd_workspace_bytes),
    ENTRY(ssd_conv1d_silu_bwd),
    ENTRY(ssd_diag_scan_workspace_bytes),
    ENTRY(ssd_diag_scan_fwd_workspace_bytes),
    ENTRY(ssd_diag_scan_fwd),
    ENTRY(ssd_diag_scan_fwd_varlen),
    ENTRY(ssd_diag_scan_bwd_workspace_bytes),
    ENTRY(ssd_diag_scan_bwd),
    ENTRY(ssd_diag_state_update),
    {nullptr, nullptr, 0, nullptr},
};
#undef ENTRY

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycall", "Tensor checks and direct calls of ssd_diag.h's entry points.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__pycall()
{
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", SSD_BUILT_FOR) < 0) Py_CLEAR(m);
    return m;
}
