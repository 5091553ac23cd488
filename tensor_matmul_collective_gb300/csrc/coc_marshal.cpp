// Argument marshalling of the decode-step and 8-bit calls for Python, over the C ABI.
//
// Those calls' kernels take a few microseconds, less than it takes an
// interpreter to look at 8 ranks' tensors one attribute at a time (51 us for
// kv_cache_append on 8 ranks; the C call itself takes 4).  Each function here
// checks the tensors, allocates outputs that were not given, and calls the C
// entry point whose address it gets.  It returns (status, outputs), or None
// where anything is not as expected: the binding in coc.py then goes through
// its own checks, which word the error.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/coc.h"

namespace {

// R tensors of a list or tuple, all of one type, on one device.
struct Ranks {
    const at::Tensor* t[COC_MAX_RANKS];
    const void* p[COC_MAX_RANKS];
    bool take(PyObject* o, int64_t R, at::ScalarType dt, const at::Device& dev) {
        const bool list = PyList_Check(o), tuple = !list && PyTuple_Check(o);
        if (!list && !tuple) return false;
        if ((list ? PyList_GET_SIZE(o) : PyTuple_GET_SIZE(o)) != R) return false;
        for (int64_t r = 0; r < R; ++r) {
            PyObject* x = list ? PyList_GET_ITEM(o, r) : PyTuple_GET_ITEM(o, r);
            if (!THPVariable_Check(x)) return false;
            t[r] = &THPVariable_Unpack(x);
            if (t[r]->scalar_type() != dt || t[r]->device() != dev) return false;
            p[r] = t[r]->data_ptr();
        }
        return true;
    }
    // Packed tensors of the given shape.
    bool packed(int64_t R, at::IntArrayRef shape) const {
        for (int64_t r = 0; r < R; ++r)
            if (t[r]->sizes() != shape || !t[r]->is_contiguous()) return false;
        return true;
    }
    // tokens x heads x d with the same strides, a head's values adjacent.
    bool heads(int64_t R, int64_t tokens, int64_t d, int64_t* n, int64_t (&stride)[2]) const {
        if (t[0]->dim() != 3 || t[0]->size(0) != tokens || t[0]->size(2) != d || t[0]->stride(2) != 1) return false;
        for (int64_t r = 1; r < R; ++r)
            if (t[r]->sizes() != t[0]->sizes() || t[r]->strides() != t[0]->strides()) return false;
        *n = t[0]->size(1);
        stride[0] = t[0]->stride(0);
        stride[1] = t[0]->stride(1);
        return true;
    }
};

const at::Tensor* tensor_of(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// The first tensor of a list, on the current CUDA device, which is `index` where that is given, and of a 16-bit type (codes: e4m3).
const at::Tensor* first_of(PyObject* o, int64_t* R, int64_t index = -1, bool codes = false) {
    PyObject* x = nullptr;
    if (PyList_Check(o) && PyList_GET_SIZE(o) > 0) {
        *R = PyList_GET_SIZE(o);
        x = PyList_GET_ITEM(o, 0);
    } else if (PyTuple_Check(o) && PyTuple_GET_SIZE(o) > 0) {
        *R = PyTuple_GET_SIZE(o);
        x = PyTuple_GET_ITEM(o, 0);
    }
    const at::Tensor* t = x != nullptr ? tensor_of(x) : nullptr;
    if (t == nullptr || *R > COC_MAX_RANKS || !t->is_cuda() || t->device().index() != c10::cuda::current_device()) return nullptr;
    if (index >= 0 && t->device().index() != index) return nullptr;
    if (codes) return t->scalar_type() == at::kFloat8_e4m3fn ? t : nullptr;
    return t->scalar_type() == at::kHalf || t->scalar_type() == at::kBFloat16 ? t : nullptr;
}

coc_dtype_t code_of(const at::Tensor& t) { return t.scalar_type() == at::kBFloat16 ? COC_BF16 : COC_FP16; }

// A new packed tensor on the current device and stream, straight from the allocator (through the dispatcher it costs half a
// microsecond more).
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType dt) {
    return at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(), c10::DispatchKeySet(c10::DispatchKey::CUDA), dt, c10::nullopt);
}

// A list of R tensors of the given shape that follow each other in `all`'s memory from an offset in bytes.
bool parts(const at::Tensor& all, int64_t R, at::IntArrayRef shape, caffe2::TypeMeta type, int64_t offset, PyObject** list,
           void* (&p)[COC_MAX_RANKS]) {
    int64_t n = 1;
    for (const int64_t x : shape) n *= x;
    const int64_t first = offset / static_cast<int64_t>(type.itemsize());
    if ((*list = PyList_New(R)) == nullptr) return false;
    for (int64_t r = 0; r < R; ++r) {
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA), type);
        t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
        t.unsafeGetTensorImpl()->set_storage_offset(first + r * n);
        p[r] = t.data_ptr();
        PyList_SET_ITEM(*list, r, THPVariable_Wrap(std::move(t)));
    }
    return true;
}

// Outputs: the given list's tensors, or R new ones; `list` is a new reference.
// New ones of a call on another than the current stream are that stream's
// memory (what the current stream has freed may still be in use there), and the
// current stream, on which the caller goes on with them, is noted as a user.
bool outputs(PyObject* given, int64_t R, at::IntArrayRef shape, at::ScalarType dt, const at::Device& dev, coc_stream_t stream,
             PyObject** list, void* (&p)[COC_MAX_RANKS]) {
    if (given != Py_None) {
        Ranks o;
        if (!o.take(given, R, dt, dev) || !o.packed(R, shape)) return false;
        *list = PySequence_List(given);
        for (int64_t r = 0; r < R; ++r) p[r] = const_cast<void*>(o.p[r]);
        return *list != nullptr;
    }
    // (what may throw comes before the list)
    const c10::cuda::CUDAStream now = c10::cuda::getCurrentCUDAStream();
    const bool other = reinterpret_cast<cudaStream_t>(stream) != now.stream();
    c10::cuda::OptionalCUDAStreamGuard on;
    if (other) on.reset_stream(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(stream), dev.index()));
    if (R == 1) {
        at::Tensor t = fresh(shape, dt);
        if (other) t.record_stream(now);
        if ((*list = PyList_New(1)) == nullptr) return false;
        p[0] = t.data_ptr();
        PyList_SET_ITEM(*list, 0, THPVariable_Wrap(std::move(t)));
        return true;
    }
    // one allocation for all ranks, a tensor on each rank's part of it (an
    // allocation, or a view through the dispatcher, costs over a microsecond each)
    int64_t n = 1;
    for (const int64_t x : shape) n *= x;
    const at::Tensor all = fresh({R * n}, dt);
    if (other) all.record_stream(now);
    return parts(all, R, shape, all.dtype(), 0, list, p);
}

// int32 arrays that index the cache.
struct Index {
    int64_t seqs, width;
    const int32_t *table, *lens, *cu;
    bool take(PyObject* table_o, PyObject* lens_o, PyObject* cu_o, int64_t tokens, const at::Device& dev) {
        const at::Tensor *tb = tensor_of(table_o), *ln = tensor_of(lens_o), *cn = cu_o == Py_None ? nullptr : tensor_of(cu_o);
        if (tb == nullptr || ln == nullptr || (cn == nullptr && cu_o != Py_None)) return false;
        for (const at::Tensor* t : {tb, ln, cn})
            if (t != nullptr && (t->scalar_type() != at::kInt || t->device() != dev || !t->is_contiguous())) return false;
        if (ln->dim() != 1 || tb->dim() != 2 || tb->size(0) != ln->size(0)) return false;
        seqs = ln->size(0);
        width = tb->size(1);
        if (cn == nullptr ? tokens != seqs : (cn->dim() != 1 || cn->size(0) != seqs + 1)) return false;
        table = static_cast<const int32_t*>(tb->data_ptr());
        lens = static_cast<const int32_t*>(ln->data_ptr());
        cu = cn == nullptr ? nullptr : static_cast<const int32_t*>(cn->data_ptr());
        return true;
    }
};

bool stream_of(PyObject* o, coc_stream_t* s) {
    if (o == Py_None) {
        *s = reinterpret_cast<coc_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
        return true;
    }
    *s = reinterpret_cast<coc_stream_t>(PyLong_AsVoidPtr(o));
    return PyErr_Occurred() == nullptr;
}

PyObject* none() { Py_RETURN_NONE; }

PyObject* result(coc_status_t st, PyObject* list) {
    PyObject* r = Py_BuildValue("(iN)", static_cast<int>(st), list);
    return r;
}

// (entry point, cache, its device's index, ks, vs, block_table, lens, cos, sin, qs, q_outs, cu_new, interleaved, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 14) return none();
    const auto fn = reinterpret_cast<decltype(&coc_kv_cache_append)>(PyLong_AsVoidPtr(a[0]));
    const auto* cache = static_cast<const coc_kv_cache_t*>(PyLong_AsVoidPtr(a[1]));
    const int64_t index = PyLong_AsLongLong(a[2]);
    if (PyErr_Occurred()) return nullptr;
    if (fn == nullptr || cache == nullptr) return none();
    int64_t R = 0;
    const at::Tensor* k0 = first_of(a[3], &R, index);
    if (k0 == nullptr || R != cache->R || k0->dim() != 3) return none();
    const int64_t T = k0->size(0), d = cache->head_dim;
    const at::ScalarType dt = k0->scalar_type();
    const at::Device dev = k0->device();
    Ranks k, v, q;
    int64_t hk, hv, hq = 0, ks[2], vs[2], qs[2] = {0, 0};
    if (!k.take(a[3], R, dt, dev) || !k.heads(R, T, d, &hk, ks) || !v.take(a[4], R, dt, dev) || !v.heads(R, T, d, &hv, vs)) return none();
    if (hk != cache->kv_heads || hv != hk) return none();
    Index ix;
    if (!ix.take(a[5], a[6], a[11], T, dev)) return none();
    const float *cos = nullptr, *sin = nullptr;
    int64_t positions = 0, rot = 0;
    if (a[7] != Py_None || a[8] != Py_None) {
        const at::Tensor *c = tensor_of(a[7]), *s = tensor_of(a[8]);
        if (c == nullptr || s == nullptr || c->dim() != 2 || c->sizes() != s->sizes()) return none();
        for (const at::Tensor* t : {c, s})
            if (t->scalar_type() != at::kFloat || t->device() != dev || !t->is_contiguous()) return none();
        cos = static_cast<const float*>(c->data_ptr());
        sin = static_cast<const float*>(s->data_ptr());
        positions = c->size(0);
        rot = 2 * c->size(1);
        if (rot > d) return none();
    }
    coc_stream_t stream;
    if (!stream_of(a[13], &stream)) return nullptr;
    const int interleaved = PyObject_IsTrue(a[12]);
    if (interleaved < 0) return nullptr;
    PyObject* list = nullptr;
    void* qo[COC_MAX_RANKS] = {};
    if (a[9] != Py_None) {
        if (!q.take(a[9], R, dt, dev) || !q.heads(R, T, d, &hq, qs)) return none();
        if (!outputs(a[10], R, {T, hq, d}, dt, dev, stream, &list, qo)) return PyErr_Occurred() ? nullptr : none();
    } else {
        if (a[10] != Py_None) return none();
        list = none();
    }
    coc_status_t st;
    Py_BEGIN_ALLOW_THREADS
    st = fn(cache, T, ix.seqs, k.p, ks, v.p, vs, static_cast<int>(hq), q.p, qs, qo, ix.table, ix.width, ix.lens, ix.cu, cos, sin,
            positions, static_cast<int>(rot), interleaved, code_of(*k0), stream);
    Py_END_ALLOW_THREADS
    return result(st, list);
    END_HANDLE_TH_ERRORS
}

// (entry point, cache, its device's index, qs, block_table, lens, cu_new, scale, window, sinks, outs, stream)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 12) return none();
    const auto fn = reinterpret_cast<decltype(&coc_kv_cache_attention)>(PyLong_AsVoidPtr(a[0]));
    const auto* cache = static_cast<const coc_kv_cache_t*>(PyLong_AsVoidPtr(a[1]));
    const int64_t index = PyLong_AsLongLong(a[2]);
    if (PyErr_Occurred()) return nullptr;
    if (fn == nullptr || cache == nullptr) return none();
    int64_t R = 0;
    const at::Tensor* q0 = first_of(a[3], &R, index);
    if (q0 == nullptr || R != cache->R || q0->dim() != 3) return none();
    const int64_t T = q0->size(0), d = cache->head_dim;
    Ranks q;
    int64_t hq, qs[2];
    if (!q.take(a[3], R, q0->scalar_type(), q0->device()) || !q.heads(R, T, d, &hq, qs)) return none();
    Index ix;
    if (!ix.take(a[4], a[5], a[6], T, q0->device())) return none();
    const double scale = PyFloat_AsDouble(a[7]);
    const int64_t window = PyLong_AsLongLong(a[8]), sinks = PyLong_AsLongLong(a[9]);
    if (PyErr_Occurred()) return nullptr;
    coc_stream_t stream;
    if (!stream_of(a[11], &stream)) return nullptr;
    PyObject* list = nullptr;
    void* out[COC_MAX_RANKS];
    if (!outputs(a[10], R, {T, hq, d}, q0->scalar_type(), q0->device(), stream, &list, out)) return PyErr_Occurred() ? nullptr : none();
    coc_status_t st;
    Py_BEGIN_ALLOW_THREADS
    st = fn(cache, T, ix.seqs, static_cast<int>(hq), q.p, qs, out, ix.table, ix.width, ix.lens, ix.cu, static_cast<float>(scale), window,
            sinks, code_of(*q0), stream);
    Py_END_ALLOW_THREADS
    return result(st, list);
    END_HANDLE_TH_ERRORS
}

// (entry point, xs, wqs, scales, group_size, zeros, outs, stream)
PyObject* w4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8) return none();
    const auto fn = reinterpret_cast<decltype(&coc_matmul_all_reduce_w4a16)>(PyLong_AsVoidPtr(a[0]));
    if (fn == nullptr) return none();
    int64_t R = 0;
    const at::Tensor* x0 = first_of(a[1], &R);
    const int64_t group = PyLong_AsLongLong(a[4]);
    if (PyErr_Occurred()) return nullptr;
    if (x0 == nullptr || x0->dim() != 2 || group < 1) return none();
    const int64_t m = x0->size(0), k = x0->size(1);
    const at::ScalarType dt = x0->scalar_type();
    const at::Device dev = x0->device();
    Ranks x, w, s, z;
    if (k % 8 != 0 || k % group != 0 || !x.take(a[1], R, dt, dev) || !x.packed(R, {m, k}) || !w.take(a[2], R, at::kInt, dev)) return none();
    if (w.t[0]->dim() != 2) return none();
    const int64_t cols = w.t[0]->size(1);
    if (!w.packed(R, {k / 8, cols}) || !s.take(a[3], R, dt, dev) || !s.packed(R, {k / group, cols})) return none();
    const bool zero = a[5] != Py_None;
    if (zero && (!z.take(a[5], R, at::kChar, dev) || !z.packed(R, {k / group, cols}))) return none();
    coc_stream_t stream;
    if (!stream_of(a[7], &stream)) return nullptr;
    PyObject* list = nullptr;
    void* out[COC_MAX_RANKS];
    if (!outputs(a[6], R, {m, cols}, dt, dev, stream, &list, out)) return PyErr_Occurred() ? nullptr : none();
    coc_status_t st;
    Py_BEGIN_ALLOW_THREADS
    st = fn(static_cast<int>(R), m, cols, k, x.p, w.p, s.p, zero ? z.p : nullptr, group, out, code_of(*x0), stream);
    Py_END_ALLOW_THREADS
    return result(st, list);
    END_HANDLE_TH_ERRORS
}

// Up to three lists of outputs; those not handed on are dropped.
struct Lists {
    PyObject* l[3] = {nullptr, nullptr, nullptr};
    void* p[3][COC_MAX_RANKS] = {};
    ~Lists() {
        for (PyObject* o : l) Py_XDECREF(o);
    }
    PyObject* done(coc_status_t st, int n) {
        PyObject* r = PyTuple_New(n + 1);
        if (r == nullptr) return nullptr;
        PyTuple_SET_ITEM(r, 0, PyLong_FromLong(static_cast<long>(st)));
        for (int i = 0; i < n; ++i) {
            PyTuple_SET_ITEM(r, i + 1, l[i] != nullptr ? l[i] : none());
            l[i] = nullptr;
        }
        return r;
    }
};

int64_t f8_blocks(int64_t n) { return (n + 127) / 128; }

// Codes (rows x cols) and scales of R ranks, given or new; both new ones are
// one allocation, all ranks' codes and then all ranks' scales.  With `sums`
// (not null: an output of the 16-bit type beside them, None where it is new) small new ones
// of all three are one allocation; larger sums have their own, which does not
// keep the codes' memory for as long as a residual lives.
bool code_outputs(PyObject* codes, PyObject* scales, PyObject* sums, at::ScalarType dt, int64_t R, int64_t rows, int64_t cols,
                  const at::Device& dev, coc_stream_t stream, Lists& o) {
    constexpr int64_t kSmall = 1 << 20;
    const int64_t n = R * rows * cols, scale_n = R * rows * f8_blocks(cols);
    const bool fresh_codes = codes == Py_None && scales == Py_None;
    const bool joint = sums == Py_None && fresh_codes && 3 * n + scale_n <= kSmall;
    if (sums != nullptr && !joint && !outputs(sums, R, {rows, cols}, dt, dev, stream, &o.l[2], o.p[2])) return false;
    if (!fresh_codes)
        return outputs(codes, R, {rows, cols}, at::kFloat8_e4m3fn, dev, stream, &o.l[0], o.p[0]) &&
               outputs(scales, R, {rows, f8_blocks(cols)}, at::kFloat8_e8m0fnu, dev, stream, &o.l[1], o.p[1]);
    const c10::cuda::CUDAStream now = c10::cuda::getCurrentCUDAStream();
    const bool other = reinterpret_cast<cudaStream_t>(stream) != now.stream();
    c10::cuda::OptionalCUDAStreamGuard on;
    if (other) on.reset_stream(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(stream), dev.index()));
    const int64_t first = joint ? 2 * n : 0;        // codes behind the sums: whole 16 bytes where rows of codes are
    const at::Tensor all = fresh({first + n + scale_n}, at::kByte);
    if (other) all.record_stream(now);
    return (!joint || parts(all, R, {rows, cols}, caffe2::TypeMeta::fromScalarType(dt), 0, &o.l[2], o.p[2])) &&
           parts(all, R, {rows, cols}, caffe2::TypeMeta::fromScalarType(at::kFloat8_e4m3fn), first, &o.l[0], o.p[0]) &&
           parts(all, R, {rows, f8_blocks(cols)}, caffe2::TypeMeta::fromScalarType(at::kFloat8_e8m0fnu), first + n, &o.l[1], o.p[1]);
}

// (entry point, xs, outs, scales, stream) -> (status, codes, scales)
PyObject* quantize_f8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 5) return none();
    const auto fn = reinterpret_cast<decltype(&coc_quantize_f8)>(PyLong_AsVoidPtr(a[0]));
    if (fn == nullptr) return none();
    int64_t R = 0;
    const at::Tensor* x0 = first_of(a[1], &R);
    if (x0 == nullptr || x0->dim() != 2) return none();
    const int64_t rows = x0->size(0), h = x0->size(1);
    const at::Device dev = x0->device();
    Ranks x;
    if (!x.take(a[1], R, x0->scalar_type(), dev) || !x.packed(R, {rows, h})) return none();
    coc_stream_t stream;
    if (!stream_of(a[4], &stream)) return nullptr;
    Lists o;
    if (!code_outputs(a[2], a[3], nullptr, at::kByte, R, rows, h, dev, stream, o)) return PyErr_Occurred() ? nullptr : none();
    coc_status_t st;
    Py_BEGIN_ALLOW_THREADS
    st = fn(static_cast<int>(R), rows, h, x.p, o.p[0], o.p[1], code_of(*x0), stream);
    Py_END_ALLOW_THREADS
    return o.done(st, 2);
    END_HANDLE_TH_ERRORS
}

// (entry point, xs, weight, residuals, eps, outs, scales, sums, stream) -> (status, codes, scales, sums)
PyObject* norm_f8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9) return none();
    const auto fn = reinterpret_cast<decltype(&coc_add_rms_norm_f8)>(PyLong_AsVoidPtr(a[0]));
    const double eps = PyFloat_AsDouble(a[4]);
    if (PyErr_Occurred()) return nullptr;
    if (fn == nullptr) return none();
    int64_t R = 0;
    const at::Tensor* x0 = first_of(a[1], &R);
    const at::Tensor* w = tensor_of(a[2]);
    if (x0 == nullptr || x0->dim() != 2 || w == nullptr) return none();
    const int64_t rows = x0->size(0), h = x0->size(1);
    const at::ScalarType dt = x0->scalar_type();
    const at::Device dev = x0->device();
    Ranks x, res;
    if (!x.take(a[1], R, dt, dev) || !x.packed(R, {rows, h})) return none();
    if (w->scalar_type() != dt || w->device() != dev || w->dim() != 1 || w->size(0) != h || !w->is_contiguous()) return none();
    const bool add = a[3] != Py_None;
    if (add ? !res.take(a[3], R, dt, dev) || !res.packed(R, {rows, h}) : a[7] != Py_None) return none();
    coc_stream_t stream;
    if (!stream_of(a[8], &stream)) return nullptr;
    Lists o;
    if (!code_outputs(a[5], a[6], add ? a[7] : nullptr, dt, R, rows, h, dev, stream, o)) return PyErr_Occurred() ? nullptr : none();
    coc_status_t st;
    Py_BEGIN_ALLOW_THREADS
    st = fn(static_cast<int>(R), rows, h, x.p, add ? res.p : nullptr, w->data_ptr(), static_cast<float>(eps), add ? o.p[2] : nullptr, o.p[0],
            o.p[1], code_of(*x0), stream);
    Py_END_ALLOW_THREADS
    return o.done(st, 3);
    END_HANDLE_TH_ERRORS
}

// Operands of an 8-bit product: codes and scales of R ranks.
struct F8Operands {
    Ranks x, xs, w, ws;
    int64_t R = 0, rows = 0, k = 0, n = 0;          // n: columns (gated: of a half)
    c10::optional<at::Device> dev;
    bool take(PyObject* const* a, int64_t halves) {
        const at::Tensor* x0 = first_of(a[0], &R, -1, true);
        if (x0 == nullptr || x0->dim() != 2) return false;
        rows = x0->size(0);
        k = x0->size(1);
        dev = x0->device();
        if (!x.take(a[0], R, at::kFloat8_e4m3fn, *dev) || !x.packed(R, {rows, k}) || !xs.take(a[1], R, at::kFloat8_e8m0fnu, *dev) ||
            !xs.packed(R, {rows, f8_blocks(k)}) || !w.take(a[2], R, at::kFloat8_e4m3fn, *dev) || w.t[0]->dim() != 2 ||
            w.t[0]->size(0) % halves != 0)
            return false;
        n = w.t[0]->size(0) / halves;
        return w.packed(R, {halves * n, k}) && ws.take(a[3], R, at::kFloat8_e8m0fnu, *dev) &&
               ws.packed(R, {halves * f8_blocks(n), f8_blocks(k)});
    }
};

// (entry point, op, xs, x_scales, ws, w_scales, outs, dtype code or None, stream) -> (status, outs)
PyObject* matmul_f8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9) return none();
    const auto fn = reinterpret_cast<decltype(&coc_fused_matmul_f8)>(PyLong_AsVoidPtr(a[0]));
    const long op = PyLong_AsLong(a[1]), code = a[7] == Py_None ? -1 : PyLong_AsLong(a[7]);
    if (PyErr_Occurred()) return nullptr;
    F8Operands in;
    if (fn == nullptr || !in.take(a + 2, 1)) return none();
    if (op == COC_OP_REDUCE_SCATTER && in.rows % in.R != 0) return none();
    coc_dtype_t dt = code == COC_FP16 ? COC_FP16 : COC_BF16;
    if (code < 0 && a[6] != Py_None) {
        int64_t given = 0;
        const at::Tensor* o0 = first_of(a[6], &given);
        if (o0 == nullptr) return none();
        dt = code_of(*o0);
    }
    const int64_t m = op == COC_OP_REDUCE_SCATTER ? in.rows / in.R : op == COC_OP_ALL_GATHER ? in.R * in.rows : in.rows;
    coc_stream_t stream;
    if (!stream_of(a[8], &stream)) return nullptr;
    Lists o;
    if (!outputs(a[6], in.R, {m, in.n}, dt == COC_BF16 ? at::kBFloat16 : at::kHalf, *in.dev, stream, &o.l[0], o.p[0]))
        return PyErr_Occurred() ? nullptr : none();
    coc_status_t st;
    Py_BEGIN_ALLOW_THREADS
    st = fn(static_cast<coc_op_t>(op), static_cast<int>(in.R), in.rows, in.n, in.k, in.x.p, in.xs.p, in.w.p, in.ws.p, o.p[0], dt, stream);
    Py_END_ALLOW_THREADS
    return o.done(st, 1);
    END_HANDLE_TH_ERRORS
}

// (entry point, xs, x_scales, ws, w_scales, outs, scales, stream) -> (status, codes, scales)
PyObject* gated_f8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8) return none();
    const auto fn = reinterpret_cast<decltype(&coc_all_gather_gated_matmul_f8)>(PyLong_AsVoidPtr(a[0]));
    F8Operands in;
    if (fn == nullptr || !in.take(a + 1, 2)) return none();
    coc_stream_t stream;
    if (!stream_of(a[7], &stream)) return nullptr;
    Lists o;
    const int64_t m = in.R * in.rows;
    if (!code_outputs(a[5], a[6], nullptr, at::kByte, in.R, m, in.n, *in.dev, stream, o)) return PyErr_Occurred() ? nullptr : none();
    coc_status_t st;
    Py_BEGIN_ALLOW_THREADS
    st = fn(static_cast<int>(in.R), in.rows, in.n, in.k, in.x.p, in.xs.p, in.w.p, in.ws.p, o.p[0], o.p[1], stream);
    Py_END_ALLOW_THREADS
    return o.done(st, 2);
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"quantize_f8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantize_f8)), METH_FASTCALL, nullptr},
    {"norm_f8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm_f8)), METH_FASTCALL, nullptr},
    {"matmul_f8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(matmul_f8)), METH_FASTCALL, nullptr},
    {"gated_f8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gated_f8)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {"w4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(w4)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_coc_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__coc_marshal() { return PyModule_Create(&module); }
