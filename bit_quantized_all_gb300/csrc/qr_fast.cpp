// qr_fast.cpp -- the common form of the calls in layer.py without Python between
// their checks, their outputs and the C ABI, as an extension module.
//
// A call of a few rows takes the GPU two to five microseconds and the interpreter
// eleven to twenty: checks of each tensor, the allocation of the outputs, the
// conversion of twenty arguments.  Here the same checks are a few loads.  A function
// takes what the Python function of that name would accept without a stream or an
// output of the caller's, returns its outputs (or the C ABI's status, as an int,
// where that is not QR_OK), and None for anything else, which the Python function
// then handles or refuses: no error is raised here.
#include <Python.h>

#include <array>
#include <cmath>

#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <c10/core/Allocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/qr.h"

namespace {

// The library's entry points, by bind().
decltype(&::qr_q8_quantize) q8_quantize;
decltype(&::qr_rms_norm) rms_norm;
decltype(&::qr_rms_norm_q8) rms_norm_q8;
decltype(&::qr_rope) rope_call;
decltype(&::qr_w8_matmul) w8_matmul;
decltype(&::qr_w8_matmul_workspace_bytes) w8_workspace_bytes;

PyObject *none() { Py_RETURN_NONE; }

// A plain tensor on a GPU, nullptr otherwise.
const at::Tensor *on_gpu(PyObject *o) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    return t.is_cuda() && t.layout() == at::kStrided ? &t : nullptr;
}
bool half_type(const at::Tensor &t) { return t.scalar_type() == at::kHalf || t.scalar_type() == at::kBFloat16; }
qr_dtype_t type_of(at::ScalarType t) { return t == at::kHalf ? QR_FP16 : QR_BF16; }

// Rows of values without gaps.
bool matrix(const at::Tensor &t) { return t.dim() == 2 && (t.size(1) < 2 || t.stride(1) == 1); }
bool like(const at::Tensor &t, const at::Tensor &x) {
    return matrix(t) && t.scalar_type() == x.scalar_type() && t.sizes() == x.sizes() && t.device() == x.device();
}
// A contiguous list of `n` values (any number if below 0).
bool list_of(const at::Tensor &t, at::ScalarType type, int64_t n, const at::Device &device) {
    return t.dim() == 1 && t.scalar_type() == type && (n < 0 || t.size(0) == n) && t.device() == device && t.is_contiguous();
}
bool heads(const at::Tensor &t) { return t.dim() == 3 && (t.size(2) < 2 || t.stride(2) == 1); }

// A new tensor on the current stream; without the dispatcher, which takes longer than
// the allocator.
at::Tensor empty(at::IntArrayRef sizes, at::IntArrayRef strides, at::ScalarType type, const at::Device &device) {
    const c10::cuda::CUDAGuard on(device);
    return at::detail::empty_strided_generic(sizes, strides, c10::GetAllocator(at::kCUDA),
                                             c10::DispatchKeySet(c10::DispatchKey::CUDA), type);
}
qr_stream_t stream_on(const at::Device &d) {
    return reinterpret_cast<qr_stream_t>(c10::cuda::getCurrentCUDAStream(d.index()).stream());
}

// A tensor in `of`'s memory, `offset` of its values from the start (a view takes
// the dispatcher a microsecond).
at::Tensor inside(const at::Tensor &of, int64_t offset, at::IntArrayRef sizes, at::IntArrayRef strides) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(of.storage()), of.key_set(), of.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(offset);
    t.unsafeGetTensorImpl()->set_sizes_and_strides(sizes, strides);
    return t;
}

// (codes, scales, pitch): what a Q8Rows holds.
struct Rows8 {
    at::Tensor codes, scales;
    int64_t pitch;

    Rows8(int64_t tokens, int64_t cols, const at::Device &d) : pitch((cols + 15) / 16 * 16) {
        codes = empty({tokens, cols}, {pitch, 1}, at::kChar, d);
        scales = empty({tokens}, {1}, at::kFloat, d);
    }
    int8_t *at_codes() const { return static_cast<int8_t *>(codes.data_ptr()); }
    float *at_scales() const { return static_cast<float *>(scales.data_ptr()); }
    PyObject *wrap() const {
        return Py_BuildValue("(NNL)", THPVariable_Wrap(codes), THPVariable_Wrap(scales), static_cast<long long>(pitch));
    }
};

// quantize(x)
PyObject *quantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *x = n == 1 ? on_gpu(args[0]) : nullptr;
    if (!x || !matrix(*x) || !half_type(*x) || x->numel() == 0 || x->size(1) > INT32_MAX) return none();
    const Rows8 y(x->size(0), x->size(1), x->device());
    const int status = q8_quantize(type_of(x->scalar_type()), x->size(0), static_cast<int>(x->size(1)), x->data_ptr(), x->stride(0),
                                   y.at_codes(), y.pitch, y.at_scales(), stream_on(x->device()));
    return status ? PyLong_FromLong(status) : y.wrap();
    END_HANDLE_TH_ERRORS
}

// norm(x, weight, eps, residual, residual_out, eight)
PyObject *norm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *x = n == 6 ? on_gpu(args[0]) : nullptr, *w = x ? on_gpu(args[1]) : nullptr;
    if (!w || !matrix(*x) || !half_type(*x) || x->numel() == 0 || x->size(1) > INT32_MAX || !PyFloat_Check(args[2])) return none();
    const at::Device device = x->device();
    const bool wide = w->scalar_type() == at::kFloat;
    if (!list_of(*w, wide ? at::kFloat : x->scalar_type(), x->size(1), device)) return none();
    const double eps = PyFloat_AS_DOUBLE(args[2]);
    if (!(eps > 0.0) || !std::isfinite(eps)) return none();
    const at::Tensor *r = nullptr, *ro = nullptr;
    if (args[3] != Py_None) {
        r = on_gpu(args[3]);
        ro = args[4] == Py_None ? r : on_gpu(args[4]);
        if (!r || !ro || !like(*r, *x) || !like(*ro, *x)) return none();
    } else if (args[4] != Py_None) {
        return none();
    }
    const qr_dtype_t dt = type_of(x->scalar_type());
    const int cols = static_cast<int>(x->size(1));
    const void *const at_r = r ? r->data_ptr() : nullptr;
    void *const at_ro = ro ? ro->data_ptr() : nullptr;
    const int64_t r_row = r ? r->stride(0) : 0, ro_row = ro ? ro->stride(0) : 0;
    if (args[5] == Py_True) {
        const Rows8 y(x->size(0), cols, device);
        const int status = rms_norm_q8(dt, x->size(0), cols, x->data_ptr(), x->stride(0), at_r, r_row, at_ro, ro_row,
                                       w->data_ptr(), wide, static_cast<float>(eps), y.at_codes(), y.pitch, y.at_scales(),
                                       stream_on(device));
        return status ? PyLong_FromLong(status) : y.wrap();
    }
    const at::Tensor y = empty(x->sizes(), {x->size(1), 1}, x->scalar_type(), device);
    const int status = rms_norm(dt, x->size(0), cols, x->data_ptr(), x->stride(0), at_r, r_row, at_ro, ro_row, w->data_ptr(),
                                wide, static_cast<float>(eps), y.data_ptr(), cols, stream_on(device));
    return status ? PyLong_FromLong(status) : THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// rope(q, k, turns, rot_dim, interleaved, factor, positions, q_offsets, kv_lens, in_place)
PyObject *rope(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *q = n == 10 ? on_gpu(args[0]) : nullptr, *turns = q ? on_gpu(args[2]) : nullptr;
    if (!turns || !heads(*q) || !half_type(*q) || q->numel() == 0 || turns->device() != q->device()) return none();
    const at::Device device = q->device();
    const int64_t tokens = q->size(0), dim = q->size(2), rot = PyLong_AsLongLong(args[3]);
    if (dim > INT32_MAX || rot > dim || q->size(1) > INT32_MAX) return none();
    const at::Tensor *k = nullptr;
    if (args[1] != Py_None) {
        k = on_gpu(args[1]);
        if (!k || !heads(*k) || k->scalar_type() != q->scalar_type() || k->device() != device || k->size(0) != tokens ||
            k->size(2) != dim || k->size(1) < 1 || k->size(1) > INT32_MAX)
            return none();
    }
    const at::Tensor *pos = nullptr, *offsets = nullptr, *lens = nullptr;
    if (args[6] != Py_None) {
        pos = on_gpu(args[6]);
        if (!pos || !list_of(*pos, at::kInt, tokens, device)) return none();
    } else {
        offsets = on_gpu(args[7]), lens = on_gpu(args[8]);
        if (!offsets || !lens || !list_of(*lens, at::kInt, -1, device) || lens->size(0) > INT32_MAX ||
            !list_of(*offsets, at::kInt, lens->size(0) + 1, device))
            return none();
    }
    const bool in_place = args[9] == Py_True;
    const qr_stream_t stream = stream_on(device);
    at::Tensor q_out, k_out;
    if (in_place) {
        q_out = *q;
        if (k) k_out = *k;
    } else {
        auto strides = [&](const at::Tensor &x) { return std::array<int64_t, 3>{x.size(1) * dim, dim, 1}; };
        if (pos) {
            q_out = empty(q->sizes(), strides(*q), q->scalar_type(), device);
            if (k) k_out = empty(k->sizes(), strides(*k), k->scalar_type(), device);
        } else {
            // tokens that a plan leaves out: not what the memory held.  One memset of one
            // allocation, k's part from a 16-byte boundary on (in a graph two memsets take
            // 4.5 us more)
            const int64_t k_at = (q->numel() + 7) / 8 * 8, n = k ? k_at + k->numel() : q->numel();
            const at::Tensor all = empty({n}, {1}, q->scalar_type(), device);
            if (cudaMemsetAsync(all.data_ptr(), 0, static_cast<size_t>(n) * 2, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
                return PyLong_FromLong(QR_ERR_CUDA);
            q_out = inside(all, 0, q->sizes(), strides(*q));
            if (k) k_out = inside(all, k_at, k->sizes(), strides(*k));
        }
    }
    auto data = [](const at::Tensor *t) { return t ? static_cast<const int32_t *>(t->data_ptr()) : nullptr; };
    const int status = rope_call(
        type_of(q->scalar_type()), tokens, static_cast<int>(dim), static_cast<int>(rot), args[4] == Py_True,
        static_cast<const uint64_t *>(turns->data_ptr()), static_cast<float>(PyFloat_AsDouble(args[5])), data(pos),
        lens ? static_cast<int>(lens->size(0)) : 0, data(offsets), data(lens), q->data_ptr(), q->stride(0), q->stride(1),
        static_cast<int>(q->size(1)), q_out.data_ptr(), q_out.stride(0), q_out.stride(1), k ? k->data_ptr() : nullptr,
        k ? k->stride(0) : 0, k ? k->stride(1) : 0, k ? static_cast<int>(k->size(1)) : 0, k ? k_out.data_ptr() : nullptr,
        k ? k_out.stride(0) : 0, k ? k_out.stride(1) : 0, stream);
    if (status) return PyLong_FromLong(status);
    if (in_place) return Py_BuildValue("(OO)", args[0], args[1]);
    if (!k) return Py_BuildValue("(NO)", THPVariable_Wrap(q_out), Py_None);
    return Py_BuildValue("(NN)", THPVariable_Wrap(q_out), THPVariable_Wrap(k_out));
    END_HANDLE_TH_ERRORS
}

// matmul(codes, scales, packed, rows, cols, bf16, workspace)
PyObject *matmul(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *codes = n == 7 ? on_gpu(args[0]) : nullptr, *scales = codes ? on_gpu(args[1]) : nullptr,
                     *packed = scales ? on_gpu(args[2]) : nullptr;
    if (!packed || !matrix(*codes) || codes->scalar_type() != at::kChar || packed->device() != codes->device()) return none();
    const at::Device device = codes->device();
    const int64_t tokens = codes->size(0), rows = PyLong_AsLongLong(args[3]), cols = PyLong_AsLongLong(args[4]);
    if (tokens < 1 || codes->size(1) != cols || !list_of(*scales, at::kFloat, tokens, device)) return none();
    at::Tensor own;
    const at::Tensor *ws = nullptr;
    if (args[6] != Py_None) {
        ws = on_gpu(args[6]);
        if (!ws || ws->scalar_type() != at::kByte || !ws->is_contiguous() || ws->device() != device) return none();
    } else if (tokens > 16) {
        own = empty({static_cast<int64_t>(w8_workspace_bytes(tokens, static_cast<int>(cols)))}, {1}, at::kByte, device);
        ws = &own;
    }
    const at::ScalarType type = args[5] == Py_True ? at::kBFloat16 : at::kHalf;
    const at::Tensor y = empty({tokens, rows}, {rows, 1}, type, device);
    const int status = w8_matmul(type_of(type), tokens, static_cast<const int8_t *>(codes->data_ptr()), codes->stride(0),
                                 static_cast<const float *>(scales->data_ptr()), static_cast<int>(rows), static_cast<int>(cols),
                                 packed->data_ptr(), y.data_ptr(), rows, ws ? ws->data_ptr() : nullptr,
                                 ws ? static_cast<size_t>(ws->numel()) : 0, stream_on(device));
    return status ? PyLong_FromLong(status) : THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// bind(addresses of the entry points, in the order of the pointers above)
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    void **const to[6] = {reinterpret_cast<void **>(&q8_quantize), reinterpret_cast<void **>(&rms_norm),
                          reinterpret_cast<void **>(&rms_norm_q8), reinterpret_cast<void **>(&rope_call),
                          reinterpret_cast<void **>(&w8_matmul), reinterpret_cast<void **>(&w8_workspace_bytes)};
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
        return nullptr;
    }
    for (int i = 0; i < 6; ++i) {
        *to[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    return none();
}

#define QR_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {QR_FAST(quantize), QR_FAST(norm), QR_FAST(rope), QR_FAST(matmul), QR_FAST(bind), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qr_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qr_fast() { return PyModule_Create(&module); }
