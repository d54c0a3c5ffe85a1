// calls.cpp -- the short way of the Python binding into the library, for calls whose kernels take
// less time than Python's checks of their tensors.
//
// A call's checks, and all words of its arguments but the addresses, depend on its tensors' shapes,
// strides, dtypes and devices and on a few numbers.  The binding goes through them in Python, makes
// the call and hands what they came to over here (keep), by exactly these.  The next call
// that is alike (run) then takes: the key, a look-up, the outputs, the addresses put in their
// places, and the library's function.  None says that the call is to go the long way: it is not
// known yet, its tensors are not plain CUDA tensors, its device is not current, it has no workspace
// of this thread, device and stream yet, or it needs one while the stream is being captured; or the library
// refused it (which it does before it launches anything), so that the long way's error is raised.
//
// Host time on the GB300's host, the long way and this one: append, plan and attention of a chunk 36 and
// 16 us (12 of them in the library, four launches); selection and reordering of beams 24 and 12; a fork
// and its copies 24 and 10; a compaction and its copies 22 and 10.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <string.h>

#include <memory>
#include <string>
#include <unordered_map>
#include <unordered_set>
#include <vector>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "spec_verify.h"

namespace {

// How the library's function is called: f(args, stream), f(args, workspace, bytes, stream), or
// with the words of `args` one by one (struct Reorder, struct Plan).
enum Style { ARGS, WORKSPACE, REORDER, PLAN };

struct Reorder {
    const void *in, *beams;
    void *out;
    int32_t lead, B, K, n;
    int64_t row_bytes;
};

struct Plan {
    const void *row_start, *kv_len, *table;
    void *plan;
    uint64_t bytes;
    int32_t B, rows, group, page_size, pages_per_seq, num_pages;
};

struct Output {
    std::vector<int64_t> sizes, strides;
    at::ScalarType dtype;
    int at;  // of its address in args
};

struct Recipe {
    const char *name;  // in `names`, for good
    std::string args;
    std::vector<int> in_at;  // of the inputs' addresses in args (-1: not among them)
    std::vector<Output> outs;
    int style, kind, device;
    size_t need;  // bytes of workspace
    void *fn;
    PyObject *extra;  // returned behind the outputs; null: nothing
    ~Recipe() { Py_XDECREF(extra); }
};

constexpr size_t MOST_ARGS = 512, MOST_OUTS = 4, MOST_KEPT = 4096;

// (All under the interpreter's lock.  Never taken down: a process's end comes after the interpreter's,
// whose objects they hold.)
auto &kept = *new std::unordered_map<std::string, std::unique_ptr<Recipe>>;
auto &names = *new std::unordered_set<std::string>;
PyObject *error_class = nullptr;
const char *(*error_text)(int32_t) = nullptr;

// A thread's workspaces.  Their memory belongs to the binding's own store of the thread, a
// threading.local, which goes when the interpreter's state of the thread goes; so this list lies in
// that state's dictionary (a thread of C++ that calls Python now and then has a new one each time).
struct Workspace {
    int kind, device;
    void *stream, *at;
    size_t bytes;
};
thread_local std::string key;
PyObject *list_name = nullptr;

using List = std::vector<Workspace>;
void drop_list(PyObject *capsule) { delete static_cast<List *>(PyCapsule_GetPointer(capsule, nullptr)); }

// The thread's list; null, where it has none and `make` is not asked for, or for an error.
List *workspaces(bool make)
{
    PyObject *of_thread = PyThreadState_GetDict();  // borrowed
    if (!of_thread)
        return nullptr;
    PyObject *capsule = PyDict_GetItemWithError(of_thread, list_name);  // borrowed
    if (!capsule && make && !PyErr_Occurred()) {
        capsule = PyCapsule_New(new List, nullptr, drop_list);
        if (!capsule || PyDict_SetItem(of_thread, list_name, capsule) < 0)
            return nullptr;
        Py_DECREF(capsule);  // the dictionary has it
    }
    return capsule ? static_cast<List *>(PyCapsule_GetPointer(capsule, nullptr)) : nullptr;
}

Workspace *workspace_of(List *list, int kind, int device, void *stream)
{
    if (list)
        for (Workspace &w : *list)
            if (w.kind == kind && w.device == device && w.stream == stream)
                return &w;
    return nullptr;
}

template <typename T>
void add(const T &x)
{
    key.append(reinterpret_cast<const char *>(&x), sizeof x);
}

// The key of a call: its number, two numbers or byte strings, its tensors (None: none).  False
// where one of them is not what it should be.
bool make_key(PyObject *const *a, Py_ssize_t n)
{
    key.clear();
    const long op = PyLong_AsLong(a[0]);
    if (op == -1 && PyErr_Occurred())
        return false;
    add(op);
    for (int i = 1; i < 3; ++i) {
        if (PyLong_CheckExact(a[i])) {
            const long long x = PyLong_AsLongLong(a[i]);
            if (x == -1 && PyErr_Occurred()) {
                PyErr_Clear();
                return false;
            }
            key.push_back('i');
            add(x);
        } else if (PyBytes_CheckExact(a[i])) {
            key.push_back('b');
            key.append(PyBytes_AS_STRING(a[i]), (size_t)PyBytes_GET_SIZE(a[i]));
        } else {
            return false;
        }
    }
    for (Py_ssize_t i = 3; i < n; ++i) {
        if (a[i] == Py_None) {
            key.push_back('n');
            continue;
        }
        if (!THPVariable_CheckExact(a[i]))
            return false;
        const at::Tensor &t = THPVariable_Unpack(a[i]);
        if (!t.is_cuda() || t.layout() != at::kStrided || t.is_conj() || t.is_neg())
            return false;
        key.push_back('t');
        key.push_back((char)t.scalar_type());
        key.push_back((char)t.get_device());
        key.push_back((char)t.dim());
        for (const int64_t x : t.sizes())
            add(x);
        for (const int64_t x : t.strides())
            add(x);
    }
    return true;
}

// run(number, a, b, tensors ..): the outputs, or None.
PyObject *run(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n < 3 || !make_key(a, n)) {
        if (PyErr_Occurred())
            return nullptr;
        Py_RETURN_NONE;
    }
    const auto found = kept.find(key);
    if (found == kept.end())
        Py_RETURN_NONE;
    const Recipe &r = *found->second;
    if (c10::cuda::current_device() != r.device)
        Py_RETURN_NONE;
    void *stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)r.device).stream();
    void *ws = nullptr;
    size_t ws_bytes = 0;
    if (r.style == WORKSPACE) {
        const Workspace *w = workspace_of(workspaces(false), r.kind, r.device, stream);
        if (!w || w->bytes < r.need ||
            c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
            Py_RETURN_NONE;
        ws = w->at;
        ws_bytes = w->bytes;
    }
    alignas(16) char args[MOST_ARGS];
    memcpy(args, r.args.data(), r.args.size());
    for (size_t i = 0; i < r.in_at.size(); ++i)
        if (r.in_at[i] >= 0 && a[3 + i] != Py_None) {
            void *p = THPVariable_Unpack(a[3 + i]).data_ptr();
            memcpy(args + r.in_at[i], &p, sizeof p);
        }
    at::Tensor outs[MOST_OUTS];
    const size_t count = r.outs.size();
    for (size_t i = 0; i < count; ++i) {
        const Output &o = r.outs[i];
        outs[i] = at::Tensor(at::detail::empty_strided_cuda(
            o.sizes, o.strides, o.dtype,
            c10::Device(c10::DeviceType::CUDA, (c10::DeviceIndex)r.device)));
        void *p = outs[i].data_ptr();
        memcpy(args + o.at, &p, sizeof p);
    }
    // (another thread may have the recipe replaced while the lock is not held)
    const int style = r.style;
    void *fn = r.fn;
    const char *name = r.name;
    PyObject *extra = r.extra;
    Py_XINCREF(extra);
    int32_t rc;
    Py_BEGIN_ALLOW_THREADS
    if (style == ARGS) {
        rc = reinterpret_cast<int32_t (*)(const void *, void *)>(fn)(args, stream);
    } else if (style == WORKSPACE) {
        rc = reinterpret_cast<int32_t (*)(const void *, void *, size_t, void *)>(fn)(
            args, ws, ws_bytes, stream);
    } else if (style == REORDER) {
        const Reorder &x = *reinterpret_cast<const Reorder *>(args);
        rc = reinterpret_cast<int32_t (*)(const void *, const void *, void *, int32_t, int32_t,
                                          int32_t, int32_t, int64_t, void *)>(fn)(
            x.in, x.beams, x.out, x.lead, x.B, x.K, x.n, x.row_bytes, stream);
    } else {
        const Plan &x = *reinterpret_cast<const Plan *>(args);
        rc = reinterpret_cast<int32_t (*)(const void *, const void *, const void *, int32_t, int32_t,
                                          int32_t, int32_t, int32_t, int32_t, void *, size_t,
                                          void *)>(fn)(
            x.row_start, x.kv_len, x.table, x.B, x.rows, x.group, x.page_size, x.pages_per_seq,
            x.num_pages, x.plan, x.bytes, stream);
    }
    Py_END_ALLOW_THREADS
    if (rc != SPEC_OK) {
        Py_XDECREF(extra);
        if (rc == SPEC_EINVAL)
            Py_RETURN_NONE;
        PyErr_Format(error_class, "%s failed: %s (status %d)", name, error_text(rc), (int)rc);
        return nullptr;
    }
    if (count == 1 && !extra)
        return THPVariable_Wrap(std::move(outs[0]));
    if (count == 0 && !extra)
        Py_RETURN_TRUE;
    PyObject *all = PyTuple_New((Py_ssize_t)count + (extra ? 1 : 0));
    if (!all) {
        Py_XDECREF(extra);
        return nullptr;
    }
    if (extra)
        PyTuple_SET_ITEM(all, (Py_ssize_t)count, extra);
    for (size_t i = 0; i < count; ++i) {
        PyObject *o = THPVariable_Wrap(std::move(outs[i]));
        if (!o) {
            Py_DECREF(all);
            return nullptr;
        }
        PyTuple_SET_ITEM(all, (Py_ssize_t)i, o);
    }
    return all;
    END_HANDLE_TH_ERRORS
}

bool read_ints(PyObject *from, std::vector<int64_t> &to)
{
    PyObject *fast = PySequence_Fast(from, "a sequence of integers expected");
    if (!fast)
        return false;
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(fast); ++i)
        to.push_back(PyLong_AsLongLong(PySequence_Fast_GET_ITEM(fast, i)));
    Py_DECREF(fast);
    return !PyErr_Occurred();
}

// keep(call, name, function, style, args, inputs' places, outputs, their places, kind of workspace,
// its bytes, device, extra): what run(*call) does from now on.
PyObject *keep(PyObject *, PyObject *given)
{
    HANDLE_TH_ERRORS
    PyObject *call, *in_at, *outs, *out_at, *extra;
    const char *name, *args;
    Py_ssize_t args_bytes;
    unsigned long long fn, need;
    int style, kind, device;
    if (!PyArg_ParseTuple(given, "O!sKiy#O!O!O!iKiO", &PyTuple_Type, &call, &name, &fn, &style, &args,
                          &args_bytes, &PyTuple_Type, &in_at, &PyTuple_Type, &outs, &PyTuple_Type,
                          &out_at, &kind, &need, &device, &extra))
        return nullptr;
    auto r = std::make_unique<Recipe>();
    r->extra = nullptr;
    r->name = names.insert(name).first->c_str();
    r->args.assign(args, (size_t)args_bytes);
    r->style = style;
    r->kind = kind;
    r->device = device;
    r->need = (size_t)need;
    r->fn = reinterpret_cast<void *>((uintptr_t)fn);
    std::vector<int64_t> places, out_places;
    if (!read_ints(in_at, places) || !read_ints(out_at, out_places))
        return nullptr;
    const Py_ssize_t count = PyTuple_GET_SIZE(outs), words = PyTuple_GET_SIZE(call);
    bool ok = args_bytes <= (Py_ssize_t)MOST_ARGS && count <= (Py_ssize_t)MOST_OUTS && words >= 3 &&
              out_places.size() == (size_t)count && places.size() == (size_t)words - 3 &&
              (style != REORDER || args_bytes == (Py_ssize_t)sizeof(Reorder)) &&
              (style != PLAN || args_bytes == (Py_ssize_t)sizeof(Plan));
    for (const int64_t at : places) {
        ok = ok && at >= -1 && at + 8 <= args_bytes;
        r->in_at.push_back((int)at);
    }
    for (Py_ssize_t i = 0; ok && i < count; ++i) {
        PyObject *t = PyTuple_GET_ITEM(outs, i);
        ok = THPVariable_Check(t) && out_places[i] >= 0 && out_places[i] + 8 <= args_bytes;
        if (ok) {
            const at::Tensor &x = THPVariable_Unpack(t);
            r->outs.push_back({x.sizes().vec(), x.strides().vec(), x.scalar_type(),
                               (int)out_places[i]});
        }
    }
    if (!ok) {
        PyErr_SetString(PyExc_ValueError, "arguments of a call do not fit together");
        return nullptr;
    }
    std::vector<PyObject *> a;
    for (Py_ssize_t i = 0; i < words; ++i)
        a.push_back(PyTuple_GET_ITEM(call, i));
    if (!make_key(a.data(), words)) {
        if (PyErr_Occurred())
            return nullptr;
        Py_RETURN_NONE;
    }
    if (extra != Py_None) {
        Py_INCREF(extra);
        r->extra = extra;
    }
    if (kept.size() >= MOST_KEPT)
        kept.clear();
    kept[key] = std::move(r);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// workspace(kind, device, stream, address, bytes): this thread's, from now on.
PyObject *workspace(PyObject *, PyObject *given)
{
    HANDLE_TH_ERRORS
    int kind, device;
    unsigned long long stream, at, bytes;
    if (!PyArg_ParseTuple(given, "iiKKK", &kind, &device, &stream, &at, &bytes))
        return nullptr;
    void *s = reinterpret_cast<void *>((uintptr_t)stream);
    List *list = workspaces(true);
    if (!list) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_RuntimeError, "no interpreter state of the thread");
        return nullptr;
    }
    Workspace *w = workspace_of(list, kind, device, s);
    if (!w) {
        list->push_back({kind, device, s, nullptr, 0});
        w = &list->back();
    }
    w->at = reinterpret_cast<void *>((uintptr_t)at);
    w->bytes = (size_t)bytes;
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// setup(error class, address of spec_verify_strerror)
PyObject *setup(PyObject *, PyObject *given)
{
    PyObject *error;
    unsigned long long text;
    if (!PyArg_ParseTuple(given, "OK", &error, &text))
        return nullptr;
    Py_INCREF(error);
    Py_XSETREF(error_class, error);
    error_text = reinterpret_cast<const char *(*)(int32_t)>((uintptr_t)text);
    kept.clear();
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"run", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(run)), METH_FASTCALL,
     "run(number, a, b, *tensors): a call that is known, or None"},
    {"keep", keep, METH_VARARGS, "what a call's checks came to"},
    {"workspace", workspace, METH_VARARGS, "this thread's workspace on a device and stream"},
    {"setup", setup, METH_VARARGS, "the class of errors, and their texts"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void)
{
    list_name = PyUnicode_InternFromString("speculative_decoding_verification_65_gb300._calls");
    return list_name ? PyModule_Create(&module) : nullptr;
}
