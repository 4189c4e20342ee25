// The binding's fast path: the calls of the block-scaled cache and of the page plan
// for plain tensors on the current device and its current stream.  A decode step makes
// such calls once a layer, and their checks in Python take longer than the smallest of
// their kernels.
//
// Every function takes the arguments of its namesake in the Python module, in their
// order, and returns the call's status, or None, with nothing done, where an argument is
// not as it has to be or needs more than this (another stream, another device, a subclass):
// the caller then makes the same checks in Python, which say what is wrong, or settle
// it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>

#include "pagedfp8.h"

namespace {

using at::ScalarType;

// The arguments of one call, in order; `ok` falls where one does not fit.
struct Args {
    PyObject *const *v;
    int dev;
    bool ok;

    Args(PyObject *const *args) : v(args), dev(-1), ok(true) {}

    // A contiguous tensor of this type and number of dimensions (-1: any) on the device of
    // the first one.
    const at::Tensor *tensor(int i, ScalarType type, int dims)
    {
        if (!ok || !THPVariable_CheckExact(v[i])) {
            ok = false;
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(v[i]);
        const at::Device d = t.device();
        if (dev < 0)
            dev = d.index();
        ok = d.is_cuda() && d.index() == dev && t.scalar_type() == type && (dims < 0 || t.dim() == dims) && t.is_contiguous();
        return ok ? &t : nullptr;
    }

    template <typename T>
    T *data(int i, ScalarType type, int dims)
    {
        const at::Tensor *t = tensor(i, type, dims);
        return t ? static_cast<T *>(t->data_ptr()) : nullptr;
    }

    // The same, or None.
    template <typename T>
    T *optional(int i, ScalarType type, int dims)
    {
        return v[i] == Py_None ? nullptr : data<T>(i, type, dims);
    }

    // fp32 or bf16 rows of `dims` dimensions.
    const at::Tensor *rows(int i, int dims, int &code)
    {
        if (!ok || !THPVariable_CheckExact(v[i])) {
            ok = false;
            return nullptr;
        }
        const ScalarType t = THPVariable_Unpack(v[i]).scalar_type();
        code = t == ScalarType::Float ? PKV_F32 : PKV_BF16;
        return tensor(i, code == PKV_F32 ? ScalarType::Float : ScalarType::BFloat16, dims);
    }

    int32_t integer(int i, int32_t least)
    {
        int overflow = 0;
        const long long x = ok && PyLong_CheckExact(v[i]) ? PyLong_AsLongLongAndOverflow(v[i], &overflow) : -1;
        ok = ok && PyLong_CheckExact(v[i]) && overflow == 0 && x >= least && x <= INT32_MAX;
        return ok ? static_cast<int32_t>(x) : 0;
    }

    int64_t integer64(int i)
    {
        int overflow = 0;
        const long long x = ok && PyLong_CheckExact(v[i]) ? PyLong_AsLongLongAndOverflow(v[i], &overflow) : -1;
        ok = ok && PyLong_CheckExact(v[i]) && overflow == 0 && x >= 0;
        return x;
    }

    float scale(int i, int64_t head_dim)
    {
        if (v[i] == Py_None)
            return static_cast<float>(1.0 / std::sqrt(static_cast<double>(head_dim)));
        ok = ok && PyFloat_CheckExact(v[i]);
        return ok ? static_cast<float>(PyFloat_AS_DOUBLE(v[i])) : 0.f;
    }

    void need(bool x) { ok = ok && x; }

    // The current stream, if argument i is None and the tensors are on the current device.
    cudaStream_t stream(int i)
    {
        ok = ok && v[i] == Py_None && dev == c10::cuda::current_device();
        return ok ? c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream() : nullptr;
    }
};

// The interpreter's lock, let go for as long as this lives (a full launch queue blocks a call).
struct Unlocked {
    PyThreadState *state;
    Unlocked() : state(PyEval_SaveThread()) {}
    ~Unlocked() { PyEval_RestoreThread(state); }
};

template <typename Call>
PyObject *status(Call call)
{
    pkv_status st;
    {
        const Unlocked unlocked;
        st = call();
    }
    return PyLong_FromLong(st);
}

// K and V pools with their blocks' exponents.
struct Pools {
    uint8_t *k, *v, *ke, *ve;
    int64_t pages;
    int hkv, page;

    Pools(Args &a, int at)
    {
        const at::Tensor *kt = a.tensor(at, ScalarType::Byte, 4), *vt = a.tensor(at + 1, ScalarType::Byte, 4);
        const at::Tensor *ket = a.tensor(at + 2, ScalarType::Byte, 3), *vet = a.tensor(at + 3, ScalarType::Byte, 3);
        if (!a.ok)
            return;
        const at::IntArrayRef s = kt->sizes(), e = ket->sizes();
        a.need(vt->sizes() == s && s[3] == PKV_HEAD_DIM && vet->sizes() == e && e[0] == s[0] && e[1] == s[1] &&
               e[2] == s[2] / 16 && s[1] <= INT32_MAX && s[2] <= INT32_MAX);
        k = static_cast<uint8_t *>(kt->data_ptr());
        v = static_cast<uint8_t *>(vt->data_ptr());
        ke = static_cast<uint8_t *>(ket->data_ptr());
        ve = static_cast<uint8_t *>(vet->data_ptr());
        pages = s[0];
        hkv = static_cast<int>(s[1]);
        page = static_cast<int>(s[2]);
    }
};

// (k_new, v_new, slot_mapping, k_cache, v_cache, k_exp, v_exp, device_error, stream)
PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 9)
        Py_RETURN_NONE;
    Args a(args);
    int kd = 0, vd = 0;
    const at::Tensor *k = a.rows(0, 3, kd), *v = a.rows(1, 3, vd);
    const at::Tensor *slots = a.tensor(2, ScalarType::Long, 1);
    const Pools p(a, 3);
    int32_t *err = a.optional<int32_t>(7, ScalarType::Int, -1);
    const cudaStream_t s = a.stream(8);
    if (!a.ok || kd != vd || v->sizes() != k->sizes() || k->size(1) != p.hkv || slots->size(0) != k->size(0) ||
        k->size(2) > INT32_MAX)
        Py_RETURN_NONE;
    return status([&] {
        return pkv_kv_append_fp8b(k->data_ptr(), v->data_ptr(), kd, k->size(0), p.hkv, static_cast<int>(k->size(2)),
                                     static_cast<const int64_t *>(slots->data_ptr()), p.k, p.v, p.ke, p.ve, p.pages, p.page,
                                     err, s);
    });
}

// (slot_mapping, k_cache, v_cache, k_exp, v_exp, k_out, v_out, device_error, stream)
PyObject *read(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 9)
        Py_RETURN_NONE;
    Args a(args);
    int kd = 0, vd = 0;
    const at::Tensor *slots = a.tensor(0, ScalarType::Long, 1);
    const Pools p(a, 1);
    const at::Tensor *k = a.rows(5, 3, kd), *v = a.rows(6, 3, vd);
    int32_t *err = a.optional<int32_t>(7, ScalarType::Int, -1);
    const cudaStream_t s = a.stream(8);
    if (!a.ok || kd != vd || v->sizes() != k->sizes() || k->size(1) != p.hkv || slots->size(0) != k->size(0) ||
        k->size(2) > INT32_MAX)
        Py_RETURN_NONE;
    return status([&] {
        return pkv_kv_read_fp8b(static_cast<const int64_t *>(slots->data_ptr()), k->size(0), p.hkv,
                                   static_cast<int>(k->size(2)), p.k, p.v, p.ke, p.ve, p.pages, p.page, k->data_ptr(),
                                   v->data_ptr(), kd, err, s);
    });
}

// (q, k_cache, v_cache, k_exp, v_exp, block_table, seq_lens, out, workspace, sm_scale,
// device_error, max_ctas, stream, max_seq_len, seq_page_sizes, window, sinks)
PyObject *decode(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 17)
        Py_RETURN_NONE;
    Args a(args);
    int od = 0;
    const at::Tensor *q = a.tensor(0, ScalarType::BFloat16, 3);
    const Pools p(a, 1);
    const at::Tensor *bt = a.tensor(5, ScalarType::Int, 2), *lens = a.tensor(6, ScalarType::Int, 1);
    const at::Tensor *out = a.rows(7, 3, od), *ws = a.tensor(8, ScalarType::Byte, -1);
    const float sm = a.ok ? a.scale(9, q->size(2)) : 0.f;
    int32_t *err = a.optional<int32_t>(10, ScalarType::Int, -1);
    const int32_t max_ctas = a.integer(11, 0), max_len = a.integer(13, 0), window = a.integer(15, 0), sinks = a.integer(16, 0);
    const at::Tensor *sizes = a.ok && args[14] != Py_None ? a.tensor(14, ScalarType::Int, 1) : nullptr;
    const cudaStream_t s = a.stream(12);
    if (!a.ok || out->sizes() != q->sizes() || bt->size(0) != q->size(0) || lens->size(0) != q->size(0) ||
        (sizes && sizes->size(0) != q->size(0)) || q->size(0) > INT32_MAX || q->size(1) > INT32_MAX || q->size(2) > INT32_MAX ||
        bt->size(1) > INT32_MAX)
        Py_RETURN_NONE;
    return status([&] {
        return pkv_paged_gqa_decode_fp8b(
        q->data_ptr(), p.k, p.v, p.ke, p.ve, static_cast<const int32_t *>(bt->data_ptr()), static_cast<int>(bt->size(1)),
        static_cast<const int32_t *>(lens->data_ptr()), max_len,
        sizes ? static_cast<const int32_t *>(sizes->data_ptr()) : nullptr, static_cast<int>(q->size(0)),
        static_cast<int>(q->size(1)), p.hkv, static_cast<int>(q->size(2)), p.page, p.pages, sm, window, sinks, out->data_ptr(),
        od, ws->data_ptr(), static_cast<size_t>(ws->numel()), err, max_ctas, s);
    });
}

// (q, cu_q, k_cache, v_cache, k_exp, v_exp, block_table, seq_lens, out, max_q_len, max_kv_len, workspace, sm_scale,
// device_error, stream, max_total_kv, seq_page_sizes, window, sinks)
PyObject *prefill(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 19)
        Py_RETURN_NONE;
    Args a(args);
    int od = 0;
    const at::Tensor *q = a.tensor(0, ScalarType::BFloat16, 3), *cu = a.tensor(1, ScalarType::Int, 1);
    const Pools p(a, 2);
    const at::Tensor *bt = a.tensor(6, ScalarType::Int, 2), *lens = a.tensor(7, ScalarType::Int, 1);
    const at::Tensor *out = a.rows(8, 3, od);
    const int32_t max_q = a.integer(9, 0), max_kv = a.integer(10, 0);
    const at::Tensor *ws = a.tensor(11, ScalarType::Byte, -1);
    const float sm = a.ok ? a.scale(12, q->size(2)) : 0.f;
    int32_t *err = a.optional<int32_t>(13, ScalarType::Int, -1);
    const int64_t total = a.integer64(15);
    const at::Tensor *sizes = a.ok && args[16] != Py_None ? a.tensor(16, ScalarType::Int, 1) : nullptr;
    const int32_t window = a.integer(17, 0), sinks = a.integer(18, 0);
    const cudaStream_t s = a.stream(14);
    if (!a.ok || out->sizes() != q->sizes() || bt->size(0) != lens->size(0) || cu->size(0) != lens->size(0) + 1 ||
        (sizes && sizes->size(0) != lens->size(0)) || q->size(0) > INT32_MAX || q->size(1) > INT32_MAX ||
        q->size(2) > INT32_MAX || lens->size(0) > INT32_MAX || bt->size(1) > INT32_MAX)
        Py_RETURN_NONE;
    return status([&] {
        return pkv_paged_prefill_fp8b(
        q->data_ptr(), static_cast<const int32_t *>(cu->data_ptr()), static_cast<int>(q->size(0)), max_q, p.k, p.v, p.ke, p.ve,
        static_cast<const int32_t *>(bt->data_ptr()), static_cast<int>(bt->size(1)),
        static_cast<const int32_t *>(lens->data_ptr()), sizes ? static_cast<const int32_t *>(sizes->data_ptr()) : nullptr,
        static_cast<int>(lens->size(0)), max_kv, total, static_cast<int>(q->size(1)), p.hkv, static_cast<int>(q->size(2)),
        p.page, p.pages, sm, window, sinks, out->data_ptr(), od, ws->data_ptr(), static_cast<size_t>(ws->numel()), err, s);
    });
}

// A block table of `batch` rows and a page pool.
struct Table {
    int32_t *table, *pool;
    int max_pages;
    int64_t pages;

    Table(Args &a, int at, int64_t batch)
    {
        const at::Tensor *t = a.tensor(at, ScalarType::Int, 2), *p = a.tensor(at + 1, ScalarType::Int, 1);
        if (!a.ok)
            return;
        a.need(t->size(0) == batch && t->size(1) <= INT32_MAX && p->size(0) > PKV_PAGE_POOL_HEADER && batch <= INT32_MAX);
        table = static_cast<int32_t *>(t->data_ptr());
        pool = static_cast<int32_t *>(p->data_ptr());
        max_pages = static_cast<int>(t->size(1));
        pages = p->size(0) - PKV_PAGE_POOL_HEADER;
    }
};

// (past_lens, new_lens, block_table, pool, page_size, seq_lens, cu_q, slot_mapping, positions, device_error, stream)
PyObject *plan(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 11)
        Py_RETURN_NONE;
    Args a(args);
    const at::Tensor *past = a.tensor(0, ScalarType::Int, 1), *fresh = a.tensor(1, ScalarType::Int, 1);
    const int64_t batch = a.ok ? past->size(0) : 0;
    const Table t(a, 2, batch);
    const int32_t page = a.integer(4, 0);
    const at::Tensor *lens = a.tensor(5, ScalarType::Int, 1), *cu = a.tensor(6, ScalarType::Int, 1);
    const at::Tensor *slots = a.tensor(7, ScalarType::Long, 1);
    const at::Tensor *pos = a.ok && args[8] != Py_None ? a.tensor(8, ScalarType::Int, 1) : nullptr;
    int32_t *err = a.optional<int32_t>(9, ScalarType::Int, -1);
    const cudaStream_t s = a.stream(10);
    if (!a.ok || fresh->size(0) != batch || lens->size(0) != batch || cu->size(0) != batch + 1 ||
        (pos && pos->size(0) != slots->size(0)) || slots->size(0) > INT32_MAX)
        Py_RETURN_NONE;
    return status([&] {
        return pkv_plan_pages(
        static_cast<const int32_t *>(past->data_ptr()), static_cast<const int32_t *>(fresh->data_ptr()),
        static_cast<int>(batch), t.table, t.max_pages, page, t.pool, t.pages, static_cast<int32_t *>(lens->data_ptr()),
        static_cast<int32_t *>(cu->data_ptr()), static_cast<int64_t *>(slots->data_ptr()),
        pos ? static_cast<int32_t *>(pos->data_ptr()) : nullptr, static_cast<int>(slots->size(0)), err, s);
    });
}

// (seq_lens, block_table, pool, page_size, keep_lens, device_error, stream)
PyObject *release(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 7)
        Py_RETURN_NONE;
    Args a(args);
    const at::Tensor *lens = a.tensor(0, ScalarType::Int, 1);
    const int64_t batch = a.ok ? lens->size(0) : 0;
    const Table t(a, 1, batch);
    const int32_t page = a.integer(3, 0);
    const at::Tensor *keep = a.ok && args[4] != Py_None ? a.tensor(4, ScalarType::Int, 1) : nullptr;
    int32_t *err = a.optional<int32_t>(5, ScalarType::Int, -1);
    const cudaStream_t s = a.stream(6);
    if (!a.ok || (keep && keep->size(0) != batch))
        Py_RETURN_NONE;
    return status([&] {
        return pkv_release_pages(static_cast<const int32_t *>(lens->data_ptr()),
                                    keep ? static_cast<const int32_t *>(keep->data_ptr()) : nullptr, static_cast<int>(batch),
                                    t.table, t.max_pages, page, t.pool, t.pages, err, s);
    });
}

// No C++ exception may cross into the interpreter.
template <PyObject *(*kCall)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    try {
        return kCall(self, args, n);
    } catch (...) {
        Py_RETURN_NONE;
    }
}

#define PKV_METHOD(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&guarded<&name>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {PKV_METHOD(append), PKV_METHOD(read),    PKV_METHOD(decode), PKV_METHOD(prefill),
                         PKV_METHOD(plan),   PKV_METHOD(release), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding()
{
    return PyModule_Create(&module);
}
