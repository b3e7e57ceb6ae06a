// la_binding.cpp -- the quick half of the Python binding of the linear-attention entries: a CPython
// module that looks whether a call's tensors are what the entry takes, allocates what is returned,
// and makes the C call. It says nothing about a call that does not fit: it returns None, and the
// package's Python checks then name what is wrong. (Through ctypes, with the checks in Python, a
// call took 8 to 12 us of host time; a step for one sequence takes the GPU 3.4 us.)
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "rgdr.h"

namespace {

constexpr int64_t kBlock = 32;  // columns that share a scale byte

// A tensor argument: absent (None), a tensor, or something else (`bad`).
struct Arg {
    const at::Tensor *t = nullptr;
    bool bad = false;
    explicit Arg(PyObject *o) {
        if (o == Py_None) return;
        if (THPVariable_Check(o))
            t = &THPVariable_Unpack(o);
        else
            bad = true;
    }
    bool here() const { return t != nullptr; }
};

bool sizes_are(const at::Tensor &t, std::initializer_list<int64_t> s) {
    return t.dim() == (int64_t)s.size() && std::equal(s.begin(), s.end(), t.sizes().begin());
}
bool on(const Arg &a, at::ScalarType type, c10::Device dev) {
    return a.here() && a.t->scalar_type() == type && a.t->device() == dev &&
           a.t->layout() == at::kStrided && !a.t->is_neg();
}
bool fits(const Arg &a, at::ScalarType type, c10::Device dev, std::initializer_list<int64_t> s) {
    return on(a, type, dev) && sizes_are(*a.t, s) && a.t->is_contiguous();
}
// [.., .., ..] of any strides, or with a contiguous fourth axis
bool fits_rows(const Arg &a, at::ScalarType type, c10::Device dev, std::initializer_list<int64_t> s) {
    return on(a, type, dev) && sizes_are(*a.t, s) && (s.size() == 3 || a.t->stride(3) == 1);
}
bool fits_index(const Arg &a, c10::Device dev, int64_t n) {
    return !a.bad && (!a.here() || fits(a, at::kInt, dev, {n}));
}

void *ptr(const Arg &a) { return a.here() ? a.t->data_ptr() : nullptr; }
la_strides strides(const at::Tensor &t) { return {t.stride(0), t.stride(1), t.stride(2)}; }
la_strides strides_bth(const at::Tensor &t) { return {t.stride(0), t.stride(2), t.stride(1)}; }

int dtype_code(at::ScalarType t) {
    switch (t) {
    case at::kFloat: return RGDR_F32;
    case at::kHalf: return RGDR_F16;
    case at::kBFloat16: return RGDR_BF16;
    case at::kChar: return RGDR_MXI8;
    default: return -1;
    }
}

bool int_sizes(std::initializer_list<int64_t> s) {
    for (int64_t x : s)
        if (x < 0 || x > INT32_MAX) return false;
    return true;
}

PyObject *status_and(rgdr_status rc, const at::Tensor &out) {
    PyObject *o = THPVariable_Wrap(out);
    return o ? Py_BuildValue("(iN)", (int)rc, o) : nullptr;
}

// attention(prefill, query, key, value, g, pool, scales, lens, idx, nacc, scale, out, pool_out,
//           scales_out, workspace, stream) -> (status, out), or None
PyObject *attention(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 16) {
        PyErr_SetString(PyExc_TypeError, "attention takes 16 arguments");
        return nullptr;
    }
    const bool prefill = args[0] == Py_True;
    const Arg q(args[1]), k(args[2]), v(args[3]), g(args[4]), pool(args[5]), scales(args[6]);
    const Arg lens(args[7]), idx(args[8]), nacc(args[9]);
    const double scale = PyFloat_AsDouble(args[10]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    const Arg out(args[11]), pool_out(args[12]), scales_out(args[13]), workspace(args[14]);
    const auto stream = reinterpret_cast<hipStream_t>(PyLong_AsVoidPtr(args[15]));
    if (!stream && PyErr_Occurred()) return nullptr;

    if (!q.here() || !v.here() || !pool.here() || !q.t->is_cuda() || q.t->dim() != 4 ||
        v.t->dim() != 4 || pool.t->dim() != 4)
        Py_RETURN_NONE;
    const c10::Device dev = q.t->device();
    const int64_t B = q.t->size(0), Hq = q.t->size(1), T = q.t->size(2), Dk = q.t->size(3);
    const int64_t Hv = v.t->size(1), Dv = v.t->size(3), N = pool.t->size(0);
    const auto state = pool.t->scalar_type();
    const bool mx = state == at::kChar;
    if (state != at::kFloat && state != at::kBFloat16 && !mx) Py_RETURN_NONE;
    if (!int_sizes({B, Hq, T, Dk, Hv, Dv, N})) Py_RETURN_NONE;
    if (!fits_rows(q, at::kBFloat16, dev, {B, Hq, T, Dk}) ||
        !fits_rows(k, at::kBFloat16, dev, {B, Hq, T, Dk}) ||
        !fits_rows(v, at::kBFloat16, dev, {B, Hv, T, Dv}) ||
        !fits(pool, state, dev, {N, Hv, Dk, Dv}) || !fits(pool_out, state, dev, {N, Hv, Dk, Dv}) ||
        !fits_index(lens, dev, B) || !fits_index(idx, dev, B) || !fits_index(nacc, dev, B))
        Py_RETURN_NONE;
    const bool per_head = fits(g, at::kFloat, dev, {Hv});  // one decay for each head
    if (!per_head && !fits_rows(g, at::kFloat, dev, {B, Hv, T})) Py_RETURN_NONE;
    if (mx ? Dv % kBlock != 0 || !fits(scales, at::kByte, dev, {N, Hv, Dk, Dv / kBlock}) ||
                 !fits(scales_out, at::kByte, dev, {N, Hv, Dk, Dv / kBlock})
           : scales.here() || scales.bad || scales_out.here() || scales_out.bad)
        Py_RETURN_NONE;
    if (out.bad || (out.here() && !fits_rows(out, at::kBFloat16, dev, {B, Hv, T, Dv}))) Py_RETURN_NONE;
    if (workspace.bad || (workspace.here() && (!on(workspace, at::kByte, dev) || !workspace.t->is_contiguous())))
        Py_RETURN_NONE;

    const c10::DeviceGuard guard(dev);  // the launch goes to the tensors' device
    const at::Tensor o = out.here() ? *out.t : at::empty({B, Hv, T, Dv}, q.t->options());
    at::Tensor ws;
    if (prefill) {
        if (workspace.here()) {
            ws = *workspace.t;
        } else {
            size_t bytes = 0;
            const rgdr_status rc = la_prefill_workspace_size((int)B, (int)Hv, (int)T, (int)Dk, (int)Dv, &bytes);
            if (rc != RGDR_OK) return status_and(rc, o);
            if (bytes) ws = at::empty({(int64_t)bytes}, q.t->options().dtype(at::kByte));
        }
    }
    const la_strides sq = strides(*q.t), sk = strides(*k.t), sv = strides(*v.t), so = strides(o);
    const la_strides sg = per_head ? la_strides{0, 1, 0} : strides(*g.t);
    rgdr_status rc;
    Py_BEGIN_ALLOW_THREADS
    if (prefill)
        rc = la_prefill(ptr(q), &sq, ptr(k), &sk, ptr(v), &sv, (const float *)ptr(g), &sg, ptr(pool),
                        (const uint8_t *)ptr(scales), (rgdr_dtype)dtype_code(state),
                        (const int32_t *)ptr(lens), (const int32_t *)ptr(idx),
                        (const int32_t *)ptr(nacc), (float)scale, (int)B, (int)Hq, (int)Hv, (int)T,
                        (int)Dk, (int)Dv, (int)N, o.data_ptr(), &so, ptr(pool_out),
                        (uint8_t *)ptr(scales_out), ws.defined() ? ws.data_ptr() : nullptr,
                        ws.defined() ? (size_t)ws.numel() : 0, stream);
    else
        rc = la_decode(ptr(q), &sq, ptr(k), &sk, ptr(v), &sv, (const float *)ptr(g), &sg, ptr(pool),
                       (const uint8_t *)ptr(scales), (rgdr_dtype)dtype_code(state),
                       (const int32_t *)ptr(lens), (const int32_t *)ptr(idx),
                       (const int32_t *)ptr(nacc), (float)scale, (int)B, (int)Hq, (int)Hv, (int)T,
                       (int)Dk, (int)Dv, (int)N, o.data_ptr(), &so, ptr(pool_out),
                       (uint8_t *)ptr(scales_out), stream);
    Py_END_ALLOW_THREADS
    return status_and(rc, o);
    END_HANDLE_TH_ERRORS
}

// move(back, wide, codes, scales, src, dst, n, stream) -> status, or None
PyObject *move(PyObject *, PyObject *const *args, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (count != 8) {
        PyErr_SetString(PyExc_TypeError, "move takes 8 arguments");
        return nullptr;
    }
    const bool back = args[0] == Py_True;
    const Arg wide(args[1]), codes(args[2]), scales(args[3]), src(args[4]), dst(args[5]);
    const int64_t n = PyLong_AsLongLong(args[6]);
    const auto stream = reinterpret_cast<hipStream_t>(PyLong_AsVoidPtr(args[7]));
    if (PyErr_Occurred()) return nullptr;
    if (!wide.here() || !codes.here() || !wide.t->is_cuda() || wide.t->dim() != 4 || codes.t->dim() != 4)
        Py_RETURN_NONE;
    const c10::Device dev = wide.t->device();
    const auto type = wide.t->scalar_type();
    const int64_t W = wide.t->size(0), N = codes.t->size(0);
    const int64_t H = wide.t->size(1), Dk = wide.t->size(2), Dv = wide.t->size(3);
    if ((type != at::kFloat && type != at::kBFloat16) || Dv % kBlock != 0 || !int_sizes({W, N, H, Dk, Dv, n}) ||
        !fits(wide, type, dev, {W, H, Dk, Dv}) || !fits(codes, at::kChar, dev, {N, H, Dk, Dv}) ||
        !fits(scales, at::kByte, dev, {N, H, Dk, Dv / kBlock}) || !fits_index(src, dev, n) ||
        !fits_index(dst, dev, n))
        Py_RETURN_NONE;
    if (n == 0) return PyLong_FromLong(RGDR_OK);
    const c10::DeviceGuard guard(dev);
    rgdr_status rc;
    Py_BEGIN_ALLOW_THREADS
    if (back)
        rc = la_state_dequantize(ptr(codes), (const uint8_t *)ptr(scales), (int)N, (const int32_t *)ptr(src),
                                 ptr(wide), (rgdr_dtype)dtype_code(type), (int)W, (const int32_t *)ptr(dst),
                                 (int)n, (int)H, (int)Dk, (int)Dv, stream);
    else
        rc = la_state_quantize(ptr(wide), (rgdr_dtype)dtype_code(type), (int)W, (const int32_t *)ptr(src),
                               ptr(codes), (uint8_t *)ptr(scales), (int)N, (const int32_t *)ptr(dst), (int)n,
                               (int)H, (int)Dk, (int)Dv, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
    END_HANDLE_TH_ERRORS
}

// norm_gate(x, weight, gate, eps, flags, lens, out, stream) -> (status, out), or None
PyObject *norm_gate(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8) {
        PyErr_SetString(PyExc_TypeError, "norm_gate takes 8 arguments");
        return nullptr;
    }
    const Arg x(args[0]), weight(args[1]), gate(args[2]), lens(args[5]), out(args[6]);
    const double eps = PyFloat_AsDouble(args[3]);
    const unsigned long flags = PyLong_AsUnsignedLong(args[4]);
    const auto stream = reinterpret_cast<hipStream_t>(PyLong_AsVoidPtr(args[7]));
    if (PyErr_Occurred()) return nullptr;
    if (!x.here() || !x.t->is_cuda() || x.t->dim() != 4) Py_RETURN_NONE;
    const c10::Device dev = x.t->device();
    const auto type = x.t->scalar_type();
    const int64_t B = x.t->size(0), H = x.t->size(1), T = x.t->size(2), D = x.t->size(3);
    if ((type != at::kFloat && type != at::kHalf && type != at::kBFloat16) || !int_sizes({B, H, T, D}) ||
        !fits_rows(x, type, dev, {B, H, T, D}) || gate.bad || out.bad ||
        (gate.here() && !fits_rows(gate, type, dev, {B, T, H, D})) ||
        (out.here() && !fits_rows(out, type, dev, {B, T, H, D})) || !fits_index(lens, dev, B))
        Py_RETURN_NONE;
    const bool per_head = fits(weight, at::kFloat, dev, {H, D});
    if (!per_head && !fits(weight, at::kFloat, dev, {D})) Py_RETURN_NONE;
    const c10::DeviceGuard guard(dev);
    const at::Tensor o = out.here() ? *out.t : at::empty({B, T, H, D}, x.t->options());
    const la_strides sx = strides(*x.t), sg = gate.here() ? strides_bth(*gate.t) : la_strides{0, 0, 0};
    const la_strides so = strides_bth(o);
    rgdr_status rc;
    Py_BEGIN_ALLOW_THREADS
    rc = la_norm_gate(ptr(x), &sx, ptr(gate), &sg, (const float *)ptr(weight), per_head ? D : 0,
                      (rgdr_dtype)dtype_code(type), (const int32_t *)ptr(lens), (float)eps, (uint32_t)flags,
                      (int)B, (int)H, (int)T, (int)D, o.data_ptr(), &so, stream);
    Py_END_ALLOW_THREADS
    return status_and(rc, o);
    END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"attention", (PyCFunction)(void (*)())attention, METH_FASTCALL, "la_decode and la_prefill"},
    {"move", (PyCFunction)(void (*)())move, METH_FASTCALL, "la_state_quantize and la_state_dequantize"},
    {"norm_gate", (PyCFunction)(void (*)())norm_gate, METH_FASTCALL, "la_norm_gate"},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_la_binding", "Quick calls of the linear-attention entries.", -1,
                       kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__la_binding(void) { return PyModule_Create(&kModule); }
