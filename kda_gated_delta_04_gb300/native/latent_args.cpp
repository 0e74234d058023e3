// latent_args.cpp -- the latent calls' arguments from torch tensors to the C entry points, for calls
// whose every argument is as it should be.  Returns the entry point's status, or -1 when some
// argument is not: kda.py then checks them one by one and names the one.  Nothing is computed here, and
// nothing is kept between calls.
//
// A call passes eight to eleven tensors, and ctypes with the checks in Python takes 9 us for them, twice
// the time of the entry point itself; this takes under one.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "../../include/kda.h"

namespace {

constexpr long kNo = -1;

struct Args {
    PyObject *const *v;
    bool ok = true;
    int device = -1;
    at::ScalarType type = at::kBFloat16;

    const at::Tensor *tensor(int i) const
    {
        return THPVariable_Check(v[i]) ? &THPVariable_Unpack(v[i]) : nullptr;
    }
    bool given(int i) const { return v[i] != Py_None; }
    // the tensor that decides type and device
    const at::Tensor *like(int i, int dims)
    {
        const at::Tensor *t = tensor(i);
        if (!t || !t->is_cuda() || t->dim() != dims || (t->scalar_type() != at::kBFloat16 && t->scalar_type() != at::kFloat)) {
            ok = false;
            return nullptr;
        }
        device = t->get_device();
        type = t->scalar_type();
        return t;
    }
    // Whether the tensors are where the entry points launch, on the current device (where there is none, the entry
    // point says so).
    bool here() const
    {
        c10::DeviceIndex now = -1;
        return c10::cuda::GetDevice(&now) != cudaSuccess || now == device;
    }
    // a tensor of these sizes, its last dimension contiguous; the leading strides, 0 where there is one entry
    template <size_t D>
    void *rows(int i, at::ScalarType want, const int64_t (&size)[D], int64_t *stride)
    {
        const at::Tensor *t = tensor(i);
        if (!t || !t->is_cuda() || t->get_device() != device || t->scalar_type() != want || t->dim() != (int64_t)D) return fail();
        for (size_t d = 0; d < D; ++d)
            if (t->size(d) != size[d]) return fail();
        if (t->stride(D - 1) != 1 && size[D - 1] > 1) return fail();
        for (size_t d = 0; d + 1 < D; ++d) stride[d] = size[d] > 1 ? t->stride(d) : 0;
        return t->data_ptr();
    }
    template <size_t D>
    void *flat(int i, at::ScalarType want, const int64_t (&size)[D])
    {
        int64_t stride[3];
        void *p = rows(i, want, size, stride);
        return ok && tensor(i)->is_contiguous() ? p : fail();
    }
    bool truth(int i)
    {
        const int x = PyObject_IsTrue(v[i]);
        if (x < 0) {
            PyErr_Clear();
            ok = false;
        }
        return x > 0;
    }
    double number(int i)
    {
        const double x = PyFloat_AsDouble(v[i]);
        if (x == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return x;
    }
    // None: the current stream of the device; else its handle
    void *stream(int i)
    {
        if (!given(i)) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
        void *s = PyLong_AsVoidPtr(v[i]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return s;
    }
    kda_dtype_t code() const { return type == at::kBFloat16 ? KDA_DTYPE_BF16 : KDA_DTYPE_F32; }
    void *fail()
    {
        ok = false;
        return nullptr;
    }
};

// The interpreter's lock let go during the entry point, as ctypes does: a launch waits where the GPU's queue is
// full, maybe for a host function that needs the lock.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

template <class F>
PyObject *answer(F &&f)
{
    long st;
    try {
        st = f();
    } catch (...) {  // (a tensor without storage, for instance)
        st = kNo;
    }
    return PyLong_FromLong(st);
}

// latent, k_pe, cache, slots, norm_weight, norm_eps, cos_sin, positions, interleaved, q_pe, q_pe_out, latent_out,
// k_pe_out, errors, stream
PyObject *append(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    return answer([&]() -> long {
        if (n != 15) return kNo;
        Args a{v};
        const at::Tensor *latent = a.like(0, 2), *cache = a.tensor(2);
        if (!latent || !cache || cache->dim() != 3 || a.given(6) != a.given(7) || (!a.given(9) && a.given(10))) return kNo;
        const int64_t T = latent->size(0), pages = cache->size(0), page = cache->size(1);
        int64_t xs = 0, ks = 0, qs[2] = {}, os[2] = {}, ls = 0, ps = 0, H = 0, M = 0;
        const void *x = a.rows(0, a.type, {T, KDA_LATENT_DIM}, &xs), *k = a.rows(1, a.type, {T, KDA_LATENT_PE_DIM}, &ks);
        void *c = a.flat(2, a.type, {pages, page, KDA_LATENT_DIM + KDA_LATENT_PE_DIM});
        const void *slots = a.flat(3, at::kInt, {T});
        const void *w = a.given(4) ? a.flat(4, a.type, {KDA_LATENT_DIM}) : nullptr;
        const double eps = a.number(5);
        const void *cs = nullptr, *pos = nullptr, *q = nullptr;
        void *qo = nullptr, *lo = nullptr, *ko = nullptr, *err = nullptr;
        if (a.given(6)) {
            const at::Tensor *t = a.tensor(6);
            if (!t || t->dim() != 2) return kNo;
            M = t->size(0);
            cs = a.flat(6, at::kFloat, {M, KDA_LATENT_PE_DIM});
            pos = a.flat(7, at::kInt, {T});
        }
        if (a.given(9)) {
            const at::Tensor *t = a.tensor(9);
            if (!t || t->dim() != 3) return kNo;
            H = t->size(1);
            q = a.rows(9, a.type, {T, H, KDA_LATENT_PE_DIM}, qs);
            qo = a.rows(a.given(10) ? 10 : 9, a.type, {T, H, KDA_LATENT_PE_DIM}, os);
        }
        if (a.given(11)) lo = a.rows(11, a.type, {T, KDA_LATENT_DIM}, &ls);
        if (a.given(12)) ko = a.rows(12, a.type, {T, KDA_LATENT_PE_DIM}, &ps);
        if (a.given(13)) err = a.flat(13, at::kInt, {1});
        const bool inter = a.truth(8);
        void *stream = a.stream(14);
        if (!a.ok || !a.here() || T > INT32_MAX || H > INT32_MAX || M > INT32_MAX) return kNo;
        const Unlocked unlocked;
        return kda_latent_append(x, xs, k, ks, w, (float)eps, static_cast<const float *>(cs), (int32_t)M,
                                 static_cast<const int32_t *>(pos), q, qs[0], qs[1], qo, os[0], os[1], lo, ls, ko, ps,
                                 (int32_t)T, (int32_t)H, KDA_LATENT_DIM, KDA_LATENT_PE_DIM, a.code(), c, pages * page,
                                 static_cast<const int32_t *>(slots), static_cast<uint32_t *>(err), stream,
                                 inter ? KDA_LATENT_INTERLEAVED : 0);
    });
}

// q, cache, page_table, seq_lens, scale, o, lse, workspace, errors, stream
PyObject *decode(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    return answer([&]() -> long {
        if (n != 10) return kNo;
        Args a{v};
        const at::Tensor *q = a.like(0, 3), *cache = a.tensor(1), *table = a.tensor(2), *ws = a.tensor(7);
        if (!q || !cache || cache->dim() != 3 || !table || table->dim() != 2 || !ws || !ws->is_cuda() ||
            ws->get_device() != a.device || !ws->is_contiguous())
            return kNo;
        const int64_t B = q->size(0), H = q->size(1), pages = cache->size(0), page = cache->size(1), W = table->size(1);
        constexpr int64_t C = KDA_LATENT_DIM + KDA_LATENT_PE_DIM;
        int64_t qs[2], ts;
        const void *qp = a.rows(0, a.type, {B, H, C}, qs), *c = a.flat(1, a.type, {pages, page, C});
        const void *tp = a.rows(2, at::kInt, {B, W}, &ts), *lens = a.flat(3, at::kInt, {B});
        const double scale = a.number(4);
        void *o = a.flat(5, a.type, {B, H, KDA_LATENT_DIM}), *lse = a.flat(6, at::kFloat, {B, H});
        void *err = a.given(8) ? a.flat(8, at::kInt, {1}) : nullptr, *stream = a.stream(9);
        if (!a.ok || !a.here() || B > INT32_MAX || H > INT32_MAX || page > INT32_MAX || W > INT32_MAX) return kNo;
        void *scratch = ws->data_ptr();
        const size_t scratch_bytes = ws->nbytes();
        const Unlocked unlocked;
        return kda_latent_decode(qp, qs[0], qs[1], c, pages, (int32_t)page, static_cast<const int32_t *>(tp), ts, (int32_t)W,
                                 static_cast<const int32_t *>(lens), (int32_t)B, (int32_t)H, KDA_LATENT_DIM,
                                 KDA_LATENT_PE_DIM, a.code(), (float)scale, o, static_cast<float *>(lse), scratch, scratch_bytes,
                                 static_cast<uint32_t *>(err), stream);
    });
}

// q, k_nope, k_pe, v, scale, cu_q, cu_k, causal, o, lse, errors, stream
PyObject *prefill(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    return answer([&]() -> long {
        if (n != 12) return kNo;
        Args a{v};
        const at::Tensor *q = a.like(0, 3), *kp = a.tensor(2), *cu = a.given(5) ? a.tensor(5) : nullptr;
        if (!q || !kp || kp->dim() != 2 || (a.given(5) && (!cu || cu->dim() != 1)) || (!a.given(5) && a.given(6))) return kNo;
        const int64_t Tq = q->size(0), H = q->size(1), Tk = kp->size(0), N = cu ? cu->size(0) - 1 : 1;
        constexpr int64_t D = KDA_LATENT_HEAD_DIM, P = KDA_LATENT_PE_DIM;
        int64_t qs[2], ns[2], ps, vs[2];
        const void *qp = a.rows(0, a.type, {Tq, H, D + P}, qs), *kn = a.rows(1, a.type, {Tk, H, D}, ns);
        const void *kpp = a.rows(2, a.type, {Tk, P}, &ps), *vp = a.rows(3, a.type, {Tk, H, D}, vs);
        const double scale = a.number(4);
        const void *cq = cu ? a.flat(5, at::kInt, {N + 1}) : nullptr, *ck = a.given(6) ? a.flat(6, at::kInt, {N + 1}) : nullptr;
        const bool causal = a.truth(7);
        void *o = a.flat(8, a.type, {Tq, H, D}), *lse = a.flat(9, at::kFloat, {Tq, H});
        void *err = a.given(10) ? a.flat(10, at::kInt, {1}) : nullptr, *stream = a.stream(11);
        if (!a.ok || !a.here() || H > INT32_MAX || N > INT32_MAX) return kNo;
        const Unlocked unlocked;
        return kda_latent_prefill(qp, qs[0], qs[1], kn, ns[0], ns[1], kpp, ps, vp, vs[0], vs[1],
                                  static_cast<const int32_t *>(cq), static_cast<const int32_t *>(ck), (int32_t)N, Tq, Tk,
                                  (int32_t)H, D, P, D, a.code(), (float)scale, o, static_cast<float *>(lse),
                                  static_cast<uint32_t *>(err), stream, causal ? 0 : KDA_LATENT_FULL);
    });
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode)), METH_FASTCALL, nullptr},
    {"prefill", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefill)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_latent_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__latent_args()
{
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
