// tensor_calls.cpp -- the common case of the feed-forward tensor forms in one call from
// Python: tensors that need no other stream and no error message.
//
// A decoded token's product takes the GPU 4 to 6 us and took Python 11, half of it in looking
// up shapes, strides, types and addresses one by one.  Each function here looks at all of
// them, allocates the result, calls the library's C entry point, and returns
//   the result    when the call was made,
//   an int        when the library refused it (the status),
//   None          when anything is out of the ordinary: the Python form then does the whole
//                 call, with its checks, messages and streams.
// So what is checked here decides only which of the two runs; nothing is refused here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <algorithm>
#include <cstdint>

#include <ATen/ops/empty_strided.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "few_tokens.h"
#include "gemm_nt.h"

namespace {

// The entry points of the library that the Python side has loaded.
decltype(&gemm_nt_gated) p_gated;
decltype(&gemm_nt_gated_grad) p_grad;
decltype(&gemm_nt_batched_major) p_major;
decltype(&gemm_nt_w4_quantize) p_quantize;
decltype(&gemm_nt_w4) p_w4;
decltype(&gemm_nt_w4_gated) p_w4_gated;
decltype(&gemm_nt_copy_rows) p_copy;

struct Matrix {
    at::Tensor t;
    int64_t rows = 0, cols = 0, ld = 0;
    void* at = nullptr;
    // rows that start on 16-byte boundaries
    bool on_grid() const { return begin() % 16 == 0 && (ld * t.element_size() % 16 == 0 || rows < 2); }
    uintptr_t begin() const { return reinterpret_cast<uintptr_t>(at); }
    // of the bytes that the matrix touches, pitches counted
    uintptr_t end() const { return begin() + static_cast<uintptr_t>(((rows - 1) * ld + cols) * t.element_size()); }
    bool empty() const { return rows == 0 || cols == 0; }
    bool overlaps(const Matrix& o) const { return !empty() && !o.empty() && begin() < o.end() && o.begin() < end(); }
};

// Whether o is a matrix on the device `index` (taken from it if negative) with rows of
// consecutive elements.
bool matrix(PyObject* o, int& index, Matrix& m)
{
    if (!THPVariable_Check(o))
        return false;
    m.t = THPVariable_Unpack(o);
    if (!m.t.is_cuda() || m.t.dim() != 2 || m.t.layout() != at::kStrided || m.t.stride(1) != 1)
        return false;
    if (index < 0)
        index = m.t.get_device();
    if (m.t.get_device() != index)
        return false;
    m.rows = m.t.size(0);
    m.cols = m.t.size(1);
    m.ld = m.rows > 1 ? m.t.stride(0) : std::max<int64_t>(m.cols, 1);
    m.at = m.t.data_ptr();
    return true;
}

bool real16(const at::Tensor& t) { return t.scalar_type() == at::kHalf || t.scalar_type() == at::kBFloat16; }

gemm_dtype_t code(at::ScalarType t)
{
    return t == at::kHalf ? GEMM_DTYPE_F16 : (t == at::kBFloat16 ? GEMM_DTYPE_BF16 : GEMM_DTYPE_F32);
}

// An int argument; false if it is none, or none of 32 bits.
bool number(PyObject* o, long& v)
{
    if (!PyLong_Check(o))
        return false;
    v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    return v >= INT32_MIN && v <= INT32_MAX;
}

// The truth of a flag; false if it has none (what that raises is left to the Python form).
bool flag(PyObject* o, bool& v)
{
    const int t = PyObject_IsTrue(o);
    if (t < 0)
        PyErr_Clear();
    v = t == 1;
    return t >= 0;
}

int64_t pitch(int64_t cols, int64_t unit) { return (cols + unit - 1) / unit * unit; }

at::Tensor rows_of(int64_t rows, int64_t cols, int64_t ld, const at::Tensor& like, at::ScalarType type)
{
    return at::empty_strided({rows, cols}, {ld, 1}, like.options().dtype(type));
}
at::Tensor rows_of(int64_t rows, int64_t cols, const at::Tensor& like)
{
    return rows_of(rows, cols, pitch(cols, 8), like, like.scalar_type());
}

gemm_stream_t stream_of(int index)
{
    return reinterpret_cast<gemm_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream());
}

// Copies a matrix onto 16-byte boundaries, if it lies off them.
gemm_status_t to_grid(Matrix& m, gemm_stream_t stream)
{
    if (m.on_grid())
        return GEMM_OK;
    const int64_t size = m.t.element_size(), ld = pitch(m.cols, 16 / size);
    const at::Tensor copy = rows_of(m.rows, m.cols, ld, m.t, m.t.scalar_type());
    const gemm_status_t st = p_copy(m.at, size * m.ld, copy.data_ptr(), size * ld, m.rows, size * m.cols, stream);
    m.t = copy;
    m.ld = ld;
    m.at = copy.data_ptr();
    return st;
}

// Whether tokens are to be copied: off 16-byte boundaries, where the stream of the weights,
// which reads them anywhere, does not take them.  (Where it takes them it is faster than a
// copy and the kernels that need one: 16 tokens x 2047 x 4096 gated 11.9 us and 15.7, x 4095 x 4096
// in 4 bits 13.7 and 16.4; the any-layout kernel, which is what is left for the others, takes
// 226 for 16 x 4097 x 8192 gated and 31 is the copied form's.)
bool copied(const Matrix& x, bool codes) { return !x.on_grid() && !gnt::few_tokens_fit(x.rows, x.cols, codes); }

// The caller's own output, or a new one.
bool output(PyObject* o, int64_t rows, int64_t cols, const at::Tensor& like, int index, Matrix& m)
{
    if (o != Py_None)
        return matrix(o, index, m) && m.rows == rows && m.cols == cols && m.t.scalar_type() == like.scalar_type();
    m.t = rows_of(rows, cols, like);
    m.rows = rows;
    m.cols = cols;
    m.ld = pitch(cols, 8);
    m.at = m.t.data_ptr();
    return true;
}
PyObject* given_or(PyObject* o, const Matrix& m) { return o != Py_None ? Py_NewRef(o) : THPVariable_Wrap(m.t); }

// Calls without the interpreter's lock, as ctypes does; a call that throws (an operand's
// copy that finds no memory) takes the lock again on its way out.
struct Unlock {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlock() { PyEval_RestoreThread(state); }
};
template <typename F>
gemm_status_t unlocked(F&& call)
{
    const Unlock hold;
    return call();
}

// gated(X, W13, act, keep, out, path)
PyObject* gated(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    int index = -1;
    Matrix x, w, h, gu;
    long act, path;
    bool keep;
    if (n != 6 || !flag(a[3], keep) || !matrix(a[0], index, x) || !matrix(a[1], index, w) || !number(a[2], act) || !number(a[5], path) ||
        !real16(x.t) || w.t.scalar_type() != x.t.scalar_type() || w.cols != x.cols || w.rows % 2 ||
        index != c10::cuda::current_device())
        Py_RETURN_NONE;
    const int64_t inner = w.rows / 2;
    if (!output(a[4], x.rows, inner, x.t, index, h))
        Py_RETURN_NONE;
    if (keep) {
        gu.t = rows_of(x.rows, 2 * inner, x.t);
        gu.at = gu.t.data_ptr();
        gu.ld = pitch(2 * inner, 8);
    }
    // (the library would see whether the output overlaps the copies, not the operands)
    const bool copy_w = path == 0 && !w.on_grid(), copy_x = path == 0 && copied(x, false);
    if ((copy_w && h.overlaps(w)) || (copy_x && h.overlaps(x)))
        return PyLong_FromLong(GEMM_ERR_OVERLAP);
    const gemm_stream_t stream = stream_of(index);
    const gemm_status_t st = unlocked([&] {
        gemm_status_t s = copy_w ? to_grid(w, stream) : GEMM_OK;
        if (s == GEMM_OK && copy_x)
            s = to_grid(x, stream);
        if (s != GEMM_OK)
            return s;
        return p_gated(x.at, x.ld, w.at, w.ld, h.at, h.ld, gu.at, gu.ld, code(x.t.scalar_type()), static_cast<gemm_act_t>(act),
                       x.rows, x.cols, inner, static_cast<gemm_path_t>(path), stream);
    });
    if (st != GEMM_OK)
        return PyLong_FromLong(st);
    PyObject* first = given_or(a[4], h);
    if (!keep || !first)
        return first;
    PyObject* second = THPVariable_Wrap(gu.t);
    PyObject* both = second ? PyTuple_Pack(2, first, second) : nullptr;
    Py_DECREF(first);
    Py_XDECREF(second);
    return both;
    END_HANDLE_TH_ERRORS
}

// backward(dH, GU, X, W13, act)
PyObject* backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    int index = -1;
    Matrix d, gu, x, w;
    long act;
    if (n != 5 || !matrix(a[0], index, d) || !matrix(a[1], index, gu) || !matrix(a[2], index, x) || !matrix(a[3], index, w) ||
        !number(a[4], act) || !real16(x.t) || w.t.scalar_type() != x.t.scalar_type() ||
        d.t.scalar_type() != x.t.scalar_type() || gu.t.scalar_type() != x.t.scalar_type() || w.cols != x.cols || w.rows % 2 ||
        d.rows != x.rows || 2 * d.cols != w.rows || gu.rows != x.rows || gu.cols != w.rows ||
        index != c10::cuda::current_device())
        Py_RETURN_NONE;
    const at::Tensor dgu = rows_of(x.rows, w.rows, x.t), dx = rows_of(x.rows, x.cols, x.t), dw = rows_of(w.rows, x.cols, x.t);
    const gemm_dtype_t t = code(x.t.scalar_type());
    const int64_t ldg = pitch(w.rows, 8), ldo = pitch(x.cols, 8);
    const gemm_stream_t stream = stream_of(index);
    void *pg = dgu.data_ptr(), *px = dx.data_ptr(), *pw = dw.data_ptr();
    const gemm_status_t st = unlocked([&] {
        gemm_status_t s = to_grid(w, stream);
        if (s == GEMM_OK)
            s = to_grid(x, stream);
        if (s == GEMM_OK)
            s = p_grad(d.at, d.ld, gu.at, gu.ld, pg, ldg, t, static_cast<gemm_act_t>(act), x.rows, d.cols, stream);
        if (s == GEMM_OK)
            s = p_major(pg, GEMM_MAJOR_K, w.at, GEMM_MAJOR_MN, px, t, t, x.rows, x.cols, w.rows, ldg, w.ld, ldo, 0, 0, 0, 1,
                        GEMM_PATH_AUTO, stream);
        if (s == GEMM_OK)
            s = p_major(pg, GEMM_MAJOR_MN, x.at, GEMM_MAJOR_MN, pw, t, t, w.rows, x.cols, x.rows, ldg, x.ld, ldo, 0, 0, 0, 1,
                        GEMM_PATH_AUTO, stream);
        return s;
    });
    if (st != GEMM_OK)
        return PyLong_FromLong(st);
    PyObject *first = THPVariable_Wrap(dx), *second = THPVariable_Wrap(dw);
    PyObject* both = first && second ? PyTuple_Pack(2, first, second) : nullptr;
    Py_XDECREF(first);
    Py_XDECREF(second);
    return both;
    END_HANDLE_TH_ERRORS
}

// quantize(W, group, zeros, scale_dtype or None)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    int index = -1;
    Matrix w;
    long group;
    bool zeros;
    if (n != 4 || !flag(a[2], zeros) || !matrix(a[0], index, w) || !number(a[1], group) || (group != 32 && group != 64 && group != 128) ||
        (!real16(w.t) && w.t.scalar_type() != at::kFloat) || index != c10::cuda::current_device())
        Py_RETURN_NONE;
    at::ScalarType st = real16(w.t) ? w.t.scalar_type() : at::kBFloat16;
    if (a[3] != Py_None) {
        if (!THPDtype_Check(a[3]))
            Py_RETURN_NONE;
        st = reinterpret_cast<THPDtype*>(a[3])->scalar_type;
        if (st != at::kHalf && st != at::kBFloat16)
            Py_RETURN_NONE;
    }
    const int64_t width = (w.cols + 1) / 2, groups = (w.cols + group - 1) / group, ldc = pitch(width, 16);
    const int64_t lds = std::max<int64_t>(groups, 1);
    const at::Tensor q = rows_of(w.rows, width, ldc, w.t, at::kByte), s = rows_of(w.rows, groups, lds, w.t, st);
    at::Tensor z;
    if (zeros)
        z = rows_of(w.rows, groups, lds, w.t, at::kByte);
    const gemm_w4_t into = {static_cast<const uint8_t*>(q.data_ptr()), ldc, s.data_ptr(), groups,
                            zeros ? static_cast<const uint8_t*>(z.data_ptr()) : nullptr, groups, static_cast<int32_t>(group)};
    const gemm_status_t status = unlocked([&] {
        return p_quantize(w.at, code(w.t.scalar_type()), w.rows, w.cols, w.ld, &into, code(st), stream_of(index));
    });
    if (status != GEMM_OK)
        return PyLong_FromLong(status);
    PyObject* out = PyTuple_New(zeros ? 3 : 2);
    if (!out)
        return nullptr;
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(q));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(s));
    if (zeros)
        PyTuple_SET_ITEM(out, 2, THPVariable_Wrap(z));
    return out;
    END_HANDLE_TH_ERRORS
}

// w4(X, Q, S, Z, group, act or None, out, path)
PyObject* w4(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    int index = -1;
    Matrix x, q, s, z, out;
    long group, act = 0, path;
    if (n != 8 || !matrix(a[0], index, x) || !matrix(a[1], index, q) || !matrix(a[2], index, s) || !number(a[4], group) ||
        (group != 32 && group != 64 && group != 128) || !number(a[7], path) || !real16(x.t) ||
        q.t.scalar_type() != at::kByte || s.t.scalar_type() != x.t.scalar_type() || index != c10::cuda::current_device())
        Py_RETURN_NONE;
    const bool is_gated = a[5] != Py_None;
    const int64_t groups = (x.cols + group - 1) / group;
    if ((is_gated && (!number(a[5], act) || q.rows % 2)) || q.cols != (x.cols + 1) / 2 || s.rows != q.rows || s.cols != groups)
        Py_RETURN_NONE;
    if (a[3] != Py_None &&
        (!matrix(a[3], index, z) || z.t.scalar_type() != at::kByte || z.rows != q.rows || z.cols != groups))
        Py_RETURN_NONE;
    const int64_t width = is_gated ? q.rows / 2 : q.rows;
    if (!output(a[6], x.rows, width, x.t, index, out))
        Py_RETURN_NONE;
    const gemm_dtype_t t = code(x.t.scalar_type());
    const gemm_path_t way = static_cast<gemm_path_t>(path);
    // (as in `gated`)
    const bool copy_q = path == 0 && !q.on_grid(), copy_x = path == 0 && copied(x, true);
    if ((copy_q && out.overlaps(q)) || (copy_x && out.overlaps(x)))
        return PyLong_FromLong(GEMM_ERR_OVERLAP);
    const gemm_stream_t stream = stream_of(index);
    const gemm_status_t st = unlocked([&] {
        gemm_status_t status = copy_q ? to_grid(q, stream) : GEMM_OK;
        if (status == GEMM_OK && copy_x)
            status = to_grid(x, stream);
        if (status != GEMM_OK)
            return status;
        const gemm_w4_t w = {static_cast<const uint8_t*>(q.at), q.ld, s.at, s.ld, static_cast<const uint8_t*>(z.at), z.ld,
                             static_cast<int32_t>(group)};
        return is_gated ? p_w4_gated(x.at, x.ld, &w, out.at, out.ld, t, static_cast<gemm_act_t>(act), x.rows, x.cols, width,
                                     way, stream)
                        : p_w4(x.at, x.ld, &w, out.at, out.ld, t, x.rows, width, x.cols, way, stream);
    });
    return st == GEMM_OK ? given_or(a[6], out) : PyLong_FromLong(st);
    END_HANDLE_TH_ERRORS
}

// bind(addresses of the seven entry points, in the order above)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    void* at[7];
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "seven addresses");
        return nullptr;
    }
    for (int i = 0; i < 7; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred())
            return nullptr;
    }
    p_gated = reinterpret_cast<decltype(p_gated)>(at[0]);
    p_grad = reinterpret_cast<decltype(p_grad)>(at[1]);
    p_major = reinterpret_cast<decltype(p_major)>(at[2]);
    p_quantize = reinterpret_cast<decltype(p_quantize)>(at[3]);
    p_w4 = reinterpret_cast<decltype(p_w4)>(at[4]);
    p_w4_gated = reinterpret_cast<decltype(p_w4_gated)>(at[5]);
    p_copy = reinterpret_cast<decltype(p_copy)>(at[6]);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind>("bind"), method<gated>("gated"), method<backward>("backward"),
                         method<quantize>("quantize"), method<w4>("w4"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_calls()
{
    PyObject* m = PyModule_Create(&module);
    // a tensor's layout in memory is this release's: the Python side binds under no other
    PyObject* v = m ? Py_BuildValue("(iii)", TORCH_VERSION_MAJOR, TORCH_VERSION_MINOR, TORCH_VERSION_PATCH) : nullptr;
    if (m && (!v || PyModule_AddObjectRef(m, "torch_release", v) < 0))
        Py_CLEAR(m);
    Py_XDECREF(v);
    return m;
}
