// binding.cpp -- the Python side of the short calls: tables, norm + rotation, 4-bit rows and the attention
// over them.
//
// These kernels run for 3 to 20 us on a decode batch; checking nine tensors, allocating outputs and
// marshalling 28 arguments from Python took as long (14.5 us of an attention call's 24, 17 of the
// tables' 23).  Here a call's checks, allocations and marshalling take 2 to 3 us.  Arguments are positional;
// lsa.py has the signatures and their documentation.  Nothing but marshalling happens here: every
// function ends in one call of liblsa.so.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/lsa.h"

namespace {

PyObject *g_error = nullptr;      // lsa.LSAError

struct Refused {
    int code;
    std::string message;
};

[[noreturn]] void refuse(int code, std::string message) { throw Refused{code, std::move(message)}; }

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must be a CUDA tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must be a CUDA tensor");
    return t;
}

const at::Tensor &tensor_of(PyObject *o, int dims, const char *name) {
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != dims)
        refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must be a CUDA tensor of " + std::to_string(dims) + " dimensions");
    return t;
}

void same_device(const at::Tensor &t, int index, const char *name) {
    if (t.get_device() != index)
        refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must be on cuda:" + std::to_string(index) + ", like the first argument");
}

// Address of a contiguous tensor of that type, shape and device.
void *address(const at::Tensor &t, at::ScalarType type, at::IntArrayRef shape, int index, const char *name) {
    if (t.scalar_type() != type)
        refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (t.sizes() != shape)
        refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
    same_device(t, index, name);
    if (!t.is_contiguous()) refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must be contiguous");
    return t.data_ptr();
}
void *address(PyObject *o, at::ScalarType type, at::IntArrayRef shape, int index, const char *name) {
    return address(tensor(o, name), type, shape, index, name);
}

int dtype_code(at::ScalarType t, const char *name) {
    if (t == at::kBFloat16) return LSA_DTYPE_BF16;
    if (t == at::kHalf) return LSA_DTYPE_F16;
    if (t == at::kFloat) return LSA_DTYPE_F32;
    refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must be bfloat16, float16 or float32, got " + c10::toString(t));
}

bool none(PyObject *o) { return o == Py_None; }

int64_t integer(PyObject *o, const char *name, int64_t lo = INT32_MIN, int64_t hi = INT32_MAX) {
    PyObject *i = PyNumber_Index(o);
    if (!i) throw std::exception();      // Python's own error stands
    int overflow = 0;
    const int64_t v = PyLong_AsLongLongAndOverflow(i, &overflow);
    Py_DECREF(i);
    if (overflow || v < lo || v > hi) refuse(LSA_ERR_INVALID_ARG, std::string(name) + " is out of range");
    return v;
}

float number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw std::exception();
    return (float)v;
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw std::exception();
    return v != 0;
}

int32_t *status_of(PyObject *o, int index) {
    if (none(o)) return nullptr;
    const at::Tensor &t = tensor(o, "status");
    if (t.scalar_type() != at::kInt || t.get_device() != index || t.numel() < 1)
        refuse(LSA_ERR_INVALID_ARG, "status must be an int32 tensor on cuda:" + std::to_string(index));
    return static_cast<int32_t *>(t.data_ptr());
}

// The stream of the call: the handle that was passed, or the current one of the tensors' device.
lsa_stream_t stream_of(PyObject *o, int index) {
    if (!none(o)) {
        void *h = PyLong_AsVoidPtr(o);
        if (PyErr_Occurred()) throw std::exception();
        return static_cast<lsa_stream_t>(h);
    }
    return reinterpret_cast<lsa_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream());
}

// Without the dispatcher: half the time of at::empty, and a call makes up to six.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int index) {
    return at::detail::empty_cuda(shape, type, c10::Device(at::kCUDA, (c10::DeviceIndex)index), std::nullopt);
}

// A caller's workspace, or a new one of `bytes`.
struct Workspace {
    at::Tensor own;
    void *ptr;
    size_t bytes;
    Workspace(PyObject *o, size_t need, int index) {
        if (none(o)) {
            own = fresh({(int64_t)std::max<size_t>(need, 256)}, at::kByte, index);
            ptr = own.data_ptr();
            bytes = own.numel();
            return;
        }
        const at::Tensor &t = tensor(o, "ws");
        if (t.scalar_type() != at::kByte || t.get_device() != index || !t.is_contiguous())
            refuse(LSA_ERR_INVALID_ARG, "ws must be a contiguous uint8 tensor on cuda:" + std::to_string(index));
        ptr = t.data_ptr();
        bytes = t.numel();
    }
};

void check(int rc) {
    if (rc) refuse(rc, lsa_last_error());
}

PyObject *object(PyObject *given, const at::Tensor &made) {
    if (!none(given)) {
        Py_INCREF(given);
        return given;
    }
    return THPVariable_Wrap(made);
}

// Runs a call: nargs is checked, refusals become LSAError, C++ exceptions what torch makes of them.
template <class F>
PyObject *guarded(const char *name, Py_ssize_t nargs, Py_ssize_t want, F f) {
    try {
        if (nargs != want) refuse(LSA_ERR_INVALID_ARG, std::string(name) + ": " + std::to_string(want) + " arguments wanted");
        return f();
    } catch (const Refused &r) {
        if (PyObject *e = PyObject_CallFunction(g_error, "is", r.code, r.message.c_str())) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
    } catch (const std::exception &) {      // torch's own types: torch.OutOfMemoryError for an allocation that failed
        if (!PyErr_Occurred()) torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// Device `index` is current for the rest of the scope.
struct On {
    c10::cuda::OptionalCUDAGuard guard;
    explicit On(int index) {
        if (c10::cuda::current_device() != index) guard.set_index((c10::DeviceIndex)index);
    }
};

// ------------------------------------------------------------------ calls --

// table, cached_len, new_len, n_slots, max_new, table_next, slot_map, position, new_offset, n_free, status, ws, stream
PyObject *build_tables(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("build_tables", n, 13, [&]() -> PyObject * {
        const at::Tensor &table = tensor_of(a[0], 2, "table");
        const int index = table.get_device();
        const int64_t B = table.size(0), stride = table.size(1);
        const int64_t n_slots = integer(a[3], "n_slots", INT64_MIN, INT64_MAX), max_new = integer(a[4], "max_new", 0);
        if (B > INT32_MAX || stride > INT32_MAX) refuse(LSA_ERR_INVALID_ARG, "table is too large");
        On on(index);
        at::Tensor next, slots, pos, off, left;
        if (none(a[5])) next = fresh({B, stride}, at::kInt, index);
        if (none(a[6])) slots = fresh({max_new}, at::kLong, index);
        if (none(a[7])) pos = fresh({max_new}, at::kInt, index);
        if (none(a[8])) off = fresh({B + 1}, at::kInt, index);
        if (none(a[9])) left = fresh({1}, at::kInt, index);
        Workspace ws(a[11], lsa_build_tables_workspace_size((int)B, (int)stride, n_slots), index);
        auto out = [&](PyObject *o, const at::Tensor &made, at::ScalarType type, at::IntArrayRef shape, const char *name) {
            return none(o) ? made.data_ptr() : address(o, type, shape, index, name);
        };
        check(lsa_build_tables(
            (const int32_t *)address(table, at::kInt, {B, stride}, index, "table"), (int)stride,
            (const int32_t *)address(a[1], at::kInt, {B}, index, "cached_len"),
            (const int32_t *)address(a[2], at::kInt, {B}, index, "new_len"), (int)B, n_slots, (int)max_new,
            (int32_t *)out(a[5], next, at::kInt, {B, stride}, "table_next"),
            (int64_t *)out(a[6], slots, at::kLong, {max_new}, "slot_map"),
            (int32_t *)out(a[7], pos, at::kInt, {max_new}, "position"),
            (int32_t *)out(a[8], off, at::kInt, {B + 1}, "new_offset"),
            (int32_t *)out(a[9], left, at::kInt, {1}, "n_free"), status_of(a[10], index), ws.ptr, ws.bytes,
            stream_of(a[12], index)));
        return Py_BuildValue("NNNNN", object(a[5], next), object(a[6], slots), object(a[7], pos), object(a[8], off),
                             object(a[9], left));
    });
}

// Rows [T, heads, D] with contiguous columns.
struct Rows {
    void *ptr = nullptr;
    int64_t token = 0, head = 0;
    Rows() = default;
    Rows(const at::Tensor &t, at::ScalarType type, int64_t T, int64_t heads, int64_t D, int index, const char *name) {
        if (t.scalar_type() != type)
            refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
        same_device(t, index, name);
        if (t.dim() != 3 || t.size(0) != T || t.size(1) != heads || t.size(2) != D)
            refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must be " + shape_text({T, heads, D}) + ", got " + shape_text(t.sizes()));
        if (t.stride(2) != 1 && D > 1 && T * heads > 0) refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must have contiguous columns");
        ptr = t.data_ptr();
        // the stride of a dimension of one row is never used; torch may report anything for it
        token = T > 1 ? t.stride(0) : 0;
        head = heads > 1 ? t.stride(1) : 0;
    }
};

// Norm weight and width: (weight, width), either may be None.
const void *weight_of(PyObject *w, PyObject *width, at::ScalarType type, int index, const char *name, int &n) {
    n = none(width) ? 0 : (int)integer(width, "norm width");
    if (none(w)) return nullptr;
    const at::Tensor &t = tensor(w, name);
    if (none(width)) n = (int)std::min<int64_t>(t.numel(), INT32_MAX);
    return n > 0 ? address(t, type, {n}, index, name) : nullptr;
}

// q, k, position, inv_freq, q_weight, k_weight, q_norm_width, k_norm_width, eps, rot_offset, interleaved, q_out, k_out, stream
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("qk_norm_rope", n, 14, [&]() -> PyObject * {
        const at::Tensor &q = tensor_of(a[0], 3, "q");
        const int index = q.get_device();
        const at::ScalarType type = q.scalar_type();
        const int code = dtype_code(type, "q");
        const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
        const at::Tensor &inv = tensor_of(a[3], 1, "inv_freq");
        const int64_t half = inv.size(0);
        if (Hq > 1 << 20 || D > 1 << 20 || half > 1 << 20) refuse(LSA_ERR_SHAPE, "qk_norm_rope: q or inv_freq is too large");
        int qn, kn;
        const void *qw = weight_of(a[4], a[6], type, index, "q_weight", qn);
        const void *kw = weight_of(a[5], a[7], type, index, "k_weight", kn);
        On on(index);
        at::Tensor qo, ko;
        if (none(a[11])) qo = fresh({T, Hq, D}, type, index);
        const Rows q_rows(q, type, T, Hq, D, index, "q");
        const Rows qo_rows(none(a[11]) ? qo : tensor(a[11], "q_out"), type, T, Hq, D, index, "q_out");
        Rows k_rows, ko_rows;
        int64_t Hk = 0;
        if (!none(a[1])) {
            const at::Tensor &k = tensor_of(a[1], 3, "k");
            Hk = k.size(1);
            if (Hk > 1 << 20) refuse(LSA_ERR_SHAPE, "qk_norm_rope: k is too large");
            k_rows = Rows(k, type, T, Hk, D, index, "k");
            if (none(a[12])) ko = fresh({T, Hk, D}, type, index);
            ko_rows = Rows(none(a[12]) ? ko : tensor(a[12], "k_out"), type, T, Hk, D, index, "k_out");
        }
        check(lsa_qk_norm_rope(code, T, (int)D, q_rows.ptr, q_rows.token, q_rows.head, (int)Hq, qw, qn, qo_rows.ptr,
                               qo_rows.token, qo_rows.head, k_rows.ptr, k_rows.token, k_rows.head, (int)Hk, kw, kn,
                               ko_rows.ptr, ko_rows.token, ko_rows.head, number(a[8]),
                               (const int32_t *)address(a[2], at::kInt, {T}, index, "position"),
                               (const float *)address(inv, at::kFloat, {half}, index, "inv_freq"),
                               (int)integer(a[9], "rot_offset"), (int)(2 * half), truth(a[10]), stream_of(a[13], index)));
        PyObject *k_out = none(a[1]) ? (Py_INCREF(Py_None), Py_None) : object(a[12], ko);
        return Py_BuildValue("NN", object(a[11], qo), k_out);
    });
}

struct PoolShape {
    int64_t slots, heads, width;
    PoolShape(const at::Tensor &t, const char *name) {
        if (t.dim() != 3 || t.size(2) % 576 || t.size(2) == 0)
            refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must be a 4-bit pool on a CUDA device, [n_slots, heads, 36 * width] uint8");
        slots = t.size(0);
        heads = t.size(1);
        width = t.size(2) / 36;
    }
};

uint8_t *pool_address(PyObject *o, int64_t slots, int64_t heads, int64_t width, int index, const char *name) {
    return (uint8_t *)address(o, at::kByte, {slots, heads, 36 * width}, index, name);
}

// Rows of one side; [T, width] is one head.
struct Side {
    Rows rows;
    int64_t T, heads, width;
    at::ScalarType type;
    Side(PyObject *o, int index, const char *name) {
        const at::Tensor &t = tensor(o, name);
        if (t.dim() != 2 && t.dim() != 3)
            refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must be a CUDA tensor of 2 or 3 dimensions");
        type = t.scalar_type();
        T = t.size(0);
        heads = t.dim() == 3 ? t.size(1) : 1;
        width = t.size(-1);
        if (heads > 1 << 20 || width > 1 << 20) refuse(LSA_ERR_SHAPE, std::string(name) + " is too large");
        same_device(t, index, name);
        if (t.stride(-1) != 1 && width > 1 && T * heads > 0) refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must have contiguous columns");
        rows.ptr = t.data_ptr();
        rows.token = T > 1 ? t.stride(0) : 0;
        rows.head = heads > 1 ? t.stride(1) : 0;
    }
};

void pair_of(const Side &k, const Side &v, const char *name) {
    if (v.type != k.type || v.T != k.T || v.heads != k.heads)
        refuse(LSA_ERR_INVALID_ARG, std::string(name) + " must have the type, rows and heads of its partner");
}

// k, k_pool, slot_map, v, v_pool, k_scale, v_scale, status, stream
PyObject *write_q4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("write_q4", n, 9, [&]() -> PyObject * {
        const int index = tensor(a[0], "k").get_device();
        const Side k(a[0], index, "k");
        const int code = dtype_code(k.type, "k");
        const PoolShape pool(tensor(a[1], "k_pool"), "k_pool");
        if (none(a[3]) != none(a[4])) refuse(LSA_ERR_INVALID_ARG, "v and v_pool come together");
        Rows v_rows;
        int64_t vw = 0;
        uint8_t *v_pool = nullptr;
        if (!none(a[3])) {
            const Side v(a[3], index, "v");
            pair_of(k, v, "v");
            v_rows = v.rows;
            vw = v.width;
            v_pool = pool_address(a[4], pool.slots, k.heads, vw, index, "v_pool");
        }
        On on(index);
        check(lsa_write_q4(code, k.T, (int)k.heads, k.rows.ptr, k.rows.token, k.rows.head, (int)k.width,
                           pool_address(a[1], pool.slots, k.heads, k.width, index, "k_pool"), number(a[5]), v_rows.ptr,
                           v_rows.token, v_rows.head, (int)vw, v_pool, number(a[6]), pool.slots,
                           (const int64_t *)address(a[2], at::kLong, {k.T}, index, "slot_map"), status_of(a[7], index),
                           stream_of(a[8], index)));
        Py_RETURN_NONE;
    });
}

// new_k, new_v, new_li, k_pool, v_pool, li_pool, chunk_table, window_start, window_len, k_scale, v_scale, status, stream
PyObject *append_token_q4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("append_token_q4", n, 13, [&]() -> PyObject * {
        const int index = tensor(a[0], "new_k").get_device();
        const Side k(a[0], index, "new_k");
        if (!tensor(a[0], "new_k").is_contiguous()) refuse(LSA_ERR_INVALID_ARG, "new_k must be contiguous");
        const int code = dtype_code(k.type, "new_k");
        const int64_t B = k.T;
        const PoolShape pool(tensor(a[3], "k_pool"), "k_pool");
        if (none(a[1]) != none(a[4])) refuse(LSA_ERR_INVALID_ARG, "new_v and v_pool come together");
        if (none(a[2]) != none(a[5])) refuse(LSA_ERR_INVALID_ARG, "new_li and li_pool come together");
        void *vp = nullptr;
        uint8_t *v_pool = nullptr;
        int64_t vw = 0, dl = 0;
        if (!none(a[1])) {
            const Side v(a[1], index, "new_v");
            pair_of(k, v, "new_v");
            if (!tensor(a[1], "new_v").is_contiguous()) refuse(LSA_ERR_INVALID_ARG, "new_v must be contiguous");
            vw = v.width;
            vp = v.rows.ptr;
            v_pool = pool_address(a[4], pool.slots, k.heads, vw, index, "v_pool");
        }
        void *li = nullptr, *li_pool = nullptr;
        if (!none(a[2])) {
            dl = tensor_of(a[5], 3, "li_pool").size(2);
            li = address(a[2], at::kBFloat16, {B, dl}, index, "new_li");
            li_pool = address(a[5], at::kBFloat16, {pool.slots, LSA_CHUNK, dl}, index, "li_pool");
        }
        const int64_t stride = tensor_of(a[6], 2, "chunk_table").size(1);
        if (B > INT32_MAX || stride > INT32_MAX || dl > INT32_MAX) refuse(LSA_ERR_INVALID_ARG, "append_token_q4: sizes are too large");
        On on(index);
        check(lsa_append_token_q4(code, (int)k.heads, k.rows.ptr, (int)k.width,
                                  pool_address(a[3], pool.slots, k.heads, k.width, index, "k_pool"), number(a[9]), vp, (int)vw,
                                  v_pool, number(a[10]), (const lsa_bf16 *)li, (lsa_bf16 *)li_pool, (int)dl, pool.slots,
                                  (const int32_t *)address(a[6], at::kInt, {B, stride}, index, "chunk_table"), (int)stride,
                                  (const int32_t *)address(a[7], at::kInt, {B}, index, "window_start"),
                                  (int32_t *)address(a[8], at::kInt, {B}, index, "window_len"), (int)B, status_of(a[11], index),
                                  stream_of(a[12], index)));
        Py_RETURN_NONE;
    });
}

at::ScalarType scalar_type(PyObject *o) {
    if (!THPDtype_Check(o)) refuse(LSA_ERR_INVALID_ARG, "out_dtype must be a torch dtype");
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

// pool, slot_map, scale, out, out_dtype, status, stream
PyObject *read_q4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("read_q4", n, 7, [&]() -> PyObject * {
        const at::Tensor &p = tensor(a[0], "pool");
        const PoolShape pool(p, "pool");
        const int index = p.get_device();
        const int64_t T = tensor_of(a[1], 1, "slot_map").size(0);
        if (pool.heads > 1 << 20 || pool.width > 1 << 20) refuse(LSA_ERR_SHAPE, "pool is too large");
        On on(index);
        at::Tensor made;
        if (none(a[3])) {
            dtype_code(scalar_type(a[4]), "out");
            made = fresh({T, pool.heads, pool.width}, scalar_type(a[4]), index);
        }
        const at::Tensor &out = none(a[3]) ? made : tensor(a[3], "out");
        check(lsa_read_q4(pool_address(a[0], pool.slots, pool.heads, pool.width, index, "pool"), pool.slots, (int)pool.heads,
                          (int)pool.width, number(a[2]), (const int64_t *)address(a[1], at::kLong, {T}, index, "slot_map"), T,
                          dtype_code(out.scalar_type(), "out"),
                          address(out, out.scalar_type(), {T, pool.heads, pool.width}, index, "out"), status_of(a[5], index),
                          stream_of(a[6], index)));
        return object(a[3], made);
    });
}

// q, k_pool, v_pool, chunk_table, topk_idx, topk_count, window_start, window_len, max_window_len, dv, scale, k_scale, v_scale,
// out, out_dtype, lse, want_lse, status, ws, stream
PyObject *sparse_decode_q4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("sparse_decode_q4", n, 20, [&]() -> PyObject * {
        const at::Tensor &q = tensor_of(a[0], 3, "q");
        const int index = q.get_device();
        const int64_t B = q.size(0), Hq = q.size(1), dqk = q.size(2);
        const PoolShape pool(tensor(a[1], "k_pool"), "k_pool");
        const int64_t dv = integer(a[9], "dv", 1, 1 << 20), longest = integer(a[8], "max_window_len");
        int64_t k = 0;
        const void *topk = nullptr, *count = nullptr;
        if (!none(a[4])) {
            k = tensor_of(a[4], 2, "topk_idx").size(1);
            if (k) {
                topk = address(a[4], at::kInt, {B, k}, index, "topk_idx");
                count = address(a[5], at::kInt, {B}, index, "topk_count");
            }
        }
        const int64_t stride = tensor_of(a[3], 2, "chunk_table").size(1);
        if (B > INT32_MAX || Hq > 1 << 20 || dqk > 1 << 20 || pool.heads > 1 << 20 || stride > INT32_MAX || k > INT32_MAX)
            refuse(LSA_ERR_INVALID_ARG, "sparse_decode_q4: sizes are too large");
        uint8_t *v_pool = none(a[2]) ? nullptr : pool_address(a[2], pool.slots, pool.heads, dv, index, "v_pool");
        On on(index);
        at::Tensor out_made, lse_made;
        if (none(a[13])) {
            dtype_code(scalar_type(a[14]), "out");
            out_made = fresh({B, Hq, dv}, scalar_type(a[14]), index);
        }
        const at::Tensor &out = none(a[13]) ? out_made : tensor(a[13], "out");
        const bool lse = !none(a[15]) || truth(a[16]);
        if (none(a[15]) && lse) lse_made = fresh({B, Hq}, at::kFloat, index);
        void *lse_ptr = !lse ? nullptr : none(a[15]) ? lse_made.data_ptr() : address(a[15], at::kFloat, {B, Hq}, index, "lse");
        Workspace ws(a[18], lsa_sparse_decode_q4_workspace_size((int)B, (int)Hq, (int)pool.heads, (int)dqk, (int)dv, (int)k, (int)longest), index);
        check(lsa_sparse_decode_q4(
            dtype_code(q.scalar_type(), "q"), address(q, q.scalar_type(), {B, Hq, dqk}, index, "q"),
            pool_address(a[1], pool.slots, pool.heads, dqk, index, "k_pool"), number(a[11]), v_pool, number(a[12]), pool.slots,
            (int)pool.heads, (const int32_t *)address(a[3], at::kInt, {B, stride}, index, "chunk_table"), (int)stride,
            (const int32_t *)topk, (const int32_t *)count, (int)k,
            (const int32_t *)address(a[6], at::kInt, {B}, index, "window_start"),
            (const int32_t *)address(a[7], at::kInt, {B}, index, "window_len"), (int)longest, (int)B, (int)Hq, (int)dqk, (int)dv,
            number(a[10]), dtype_code(out.scalar_type(), "out"), address(out, out.scalar_type(), {B, Hq, dv}, index, "out"),
            (float *)lse_ptr, status_of(a[17], index), ws.ptr, ws.bytes, stream_of(a[19], index)));
        PyObject *l = lse ? object(a[15], lse_made) : (Py_INCREF(Py_None), Py_None);
        return Py_BuildValue("NN", object(a[13], out_made), l);
    });
}

PyObject *set_error_type(PyObject *, PyObject *type) {
    Py_INCREF(type);
    Py_XSETREF(g_error, type);
    Py_RETURN_NONE;
}

#define LSA_CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {LSA_CALL(build_tables), LSA_CALL(qk_norm_rope), LSA_CALL(write_q4), LSA_CALL(append_token_q4),
                         LSA_CALL(read_q4), LSA_CALL(sparse_decode_q4),
                         {"set_error_type", set_error_type, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
