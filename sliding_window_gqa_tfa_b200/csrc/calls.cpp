// calls.cpp -- the usual calls of binding.py's small operators, made natively.
//
// A decoding step's operators run for 2 to 5 us on the GPU, and the Python code that
// checks their tensors, allocates the outputs and fills a C call's arguments took
// longer than that (a rotation 14 us a call, this way 5; an append 9.4, 3.2).  A
// function here takes the wrapper's arguments in order, makes the same checks on the
// tensors' own structures and calls the library.  It returns
//   the outputs;  an int, the call's status where it is not TFA_OK;  or None where
//   the call is not a usual one (a stream of its own, another device than the current
//   one, a tensor of a subclass, an argument that is refused): nothing has been done
//   then, and the wrapper's Python code goes on, which makes the call or says what is
//   wrong with it.
// The library's entry points come as addresses from the loaded library, so that there
// is one copy of it.
#include <climits>
#include <cmath>
#include <initializer_list>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/tfa.h"

namespace {

struct Library {
    decltype(&tfa_qk_norm_rope) rope;
    decltype(&tfa_qk_norm_rope_backward) rope_backward;
    decltype(&tfa_qk_norm_rope_workspace) rope_workspace;
    decltype(&tfa_kv4_append) append;
    decltype(&tfa_kv4_read) read;
    decltype(&tfa_kv4_decode) decode;
    decltype(&tfa_kv4_decode_workspace) decode_workspace;
    decltype(&tfa_prefill_first) first;
    decltype(&tfa_prefill_first_backward) first_backward;
    decltype(&tfa_kv4_prefill) prefill;
    decltype(&tfa_kv4_prefill_workspace) prefill_workspace;
} lib;

// What is not a usual call; the functions turn it into None.
struct Unusual {};
void need(bool ok) {
    if (!ok) throw Unusual{};
}

const at::Tensor &tensor(PyObject *o, at::ScalarType type, int64_t dims) {
    need(THPVariable_CheckExact(o));
    const at::Tensor &t = THPVariable_Unpack(o);
    need(t.is_cuda() && t.layout() == at::kStrided && t.scalar_type() == type && t.dim() == dims);
    return t;
}
// The first tensor of a call, on the current device.
const at::Tensor &leading(PyObject *o, at::ScalarType type, int64_t dims) {
    const at::Tensor &t = tensor(o, type, dims);
    need(t.get_device() == c10::cuda::current_device());
    return t;
}
const at::Tensor &beside(const at::Tensor &first, PyObject *o, at::ScalarType type, int64_t dims) {
    const at::Tensor &t = tensor(o, type, dims);
    need(t.get_device() == first.get_device());
    return t;
}
const at::Tensor &whole(const at::Tensor &t) {
    need(t.is_contiguous());
    return t;
}
const at::Tensor &rows(const at::Tensor &t) {  // any strides, contiguous channels
    need(t.stride(-1) == 1);
    return t;
}
const at::Tensor &sized(const at::Tensor &t, at::IntArrayRef sizes) {
    need(t.sizes() == sizes);
    return t;
}
int small(int64_t n) {
    need(n >= 0 && n <= INT_MAX);
    return static_cast<int>(n);
}
int integer(PyObject *o) {
    need(PyLong_Check(o));
    int overflow = 0;
    const long v = PyLong_AsLongAndOverflow(o, &overflow);
    need(overflow == 0 && v >= INT_MIN && v <= INT_MAX);
    return static_cast<int>(v);
}
float number(PyObject *o) {
    need(PyFloat_Check(o) || PyLong_Check(o));
    const double v = PyFloat_AsDouble(o);
    if (v == -1. && PyErr_Occurred()) {
        PyErr_Clear();
        throw Unusual{};
    }
    return static_cast<float>(v);
}
int truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) {  // (the wrapper's code asks again, and raises)
        PyErr_Clear();
        throw Unusual{};
    }
    return v;
}
float scale_or(PyObject *o, int64_t D) {
    return o == Py_None ? static_cast<float>(1. / std::sqrt(static_cast<double>(D))) : number(o);
}
at::Tensor given_or_empty(PyObject *o, const at::Tensor &like, at::IntArrayRef sizes, bool strided = false) {
    if (o == Py_None) return at::empty(sizes, like.options());
    const at::Tensor &t = sized(beside(like, o, like.scalar_type(), static_cast<int64_t>(sizes.size())), sizes);
    return strided ? rows(t) : whole(t);
}
tfa_stream_t stream_of(const at::Tensor &t) {
    return reinterpret_cast<tfa_stream_t>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
}
struct Strides {  // (batch, token, head) of [B, L, H, D] or [B, H, L, D] tensors
    long long s[18];
    int n = 0;
    void tokens(const at::Tensor &t) { s[n] = t.stride(0), s[n + 1] = t.stride(1), s[n + 2] = t.stride(2), n += 3; }
    void heads(const at::Tensor &t) { s[n] = t.stride(0), s[n + 1] = t.stride(2), s[n + 2] = t.stride(1), n += 3; }
};

PyObject *result(const at::Tensor &t) { return THPVariable_Wrap(t); }
PyObject *result(std::initializer_list<at::Tensor> tensors) {  // a tuple; an undefined tensor is None
    PyObject *all = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
    Py_ssize_t i = 0;
    for (const at::Tensor &t : tensors) {
        PyObject *x = all ? THPVariable_Wrap(t) : nullptr;
        if (!x) {
            Py_XDECREF(all);
            return nullptr;
        }
        PyTuple_SET_ITEM(all, i++, x);
    }
    return all;
}

template <typename F>
int without_gil(F call) {
    PyThreadState *state = PyEval_SaveThread();
    const int rc = call();
    PyEval_RestoreThread(state);
    return rc;
}

// Runs a function's body; its Unusual is None, its other exceptions are Python's.
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t wanted, F body) {
    HANDLE_TH_ERRORS
    if (n != wanted) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, wanted);
        return nullptr;
    }
    try {
        return body();
    } catch (const Unusual &) {
        Py_RETURN_NONE;
    }
    END_HANDLE_TH_ERRORS
}

// What the pass and its gradient share: q, k, positions, inv_freq, q_weight, k_weight.
struct Rope {
    const at::Tensor &q, &k, &freq;
    const void *wq = nullptr, *wk = nullptr;
    const int *pos = nullptr;
    int per_row = 0, first = 0;
    int B, L, Hq, Hkv, D, rot;
    explicit Rope(PyObject *const *a)
        : q(rows(leading(a[0], at::kBFloat16, 4))), k(rows(beside(q, a[1], at::kBFloat16, 4))),
          freq(whole(beside(q, a[3], at::kDouble, 1))) {
        B = small(q.size(0)), L = small(q.size(1)), Hq = small(q.size(2)), D = small(q.size(3)), Hkv = small(k.size(2));
        need(k.size(0) == B && k.size(1) == L && k.size(3) == D && freq.size(0) <= D);
        rot = 2 * static_cast<int>(freq.size(0));
        if (a[4] != Py_None || a[5] != Py_None) {
            wq = sized(whole(beside(q, a[4], at::kBFloat16, 1)), {D}).const_data_ptr();
            wk = sized(whole(beside(q, a[5], at::kBFloat16, 1)), {D}).const_data_ptr();
        }
        if (PyLong_Check(a[2])) {
            first = integer(a[2]);
        } else {
            need(THPVariable_CheckExact(a[2]));
            per_row = THPVariable_Unpack(a[2]).dim() == 2;
            const at::Tensor &p = whole(beside(q, a[2], at::kInt, 1 + per_row));
            need(p.size(0) == B && (!per_row || p.size(1) == L));
            pos = static_cast<const int *>(p.const_data_ptr());
        }
    }
};

// q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, mscale, q_out, k_out
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject * {
        const Rope r(a);
        const float eps = number(a[6]), mscale = number(a[8]);
        const int inter = truth(a[7]);
        const at::Tensor qo = given_or_empty(a[9], r.q, {r.B, r.Hq, r.L, r.D}, true);
        const at::Tensor ko = given_or_empty(a[10], r.k, {r.B, r.Hkv, r.L, r.D}, true);
        Strides s;
        s.tokens(r.q), s.tokens(r.k), s.heads(qo), s.heads(ko);
        const tfa_stream_t stream = stream_of(r.q);
        const int rc = without_gil([&] {
            return lib.rope(r.q.const_data_ptr(), r.k.const_data_ptr(), qo.mutable_data_ptr(), ko.mutable_data_ptr(), s.s,
                            r.wq, r.wk, static_cast<const double *>(r.freq.const_data_ptr()), r.pos, r.per_row, r.first,
                            r.B, r.L, r.Hq, r.Hkv, r.D, r.rot, inter, eps, mscale, stream);
        });
        return rc == TFA_OK ? result({qo, ko}) : PyLong_FromLong(rc);
    });
}

// q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, mscale, dq_out, dk_out; with weights
PyObject *rope_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject * {
        const Rope r(a);
        need(r.wq != nullptr);
        const float eps = number(a[6]), mscale = number(a[8]);
        const int inter = truth(a[7]);
        const at::Tensor &gq = sized(rows(beside(r.q, a[9], at::kBFloat16, 4)), {r.B, r.Hq, r.L, r.D});
        const at::Tensor &gk = sized(rows(beside(r.q, a[10], at::kBFloat16, 4)), {r.B, r.Hkv, r.L, r.D});
        const at::Tensor dq = at::empty({r.B, r.L, r.Hq, r.D}, r.q.options());
        const at::Tensor dk = at::empty({r.B, r.L, r.Hkv, r.D}, r.q.options());
        const at::Tensor dwq = at::empty({r.D}, r.q.options().dtype(at::kFloat)), dwk = at::empty_like(dwq);
        const at::Tensor space = at::empty({static_cast<int64_t>(lib.rope_workspace(r.D))}, r.q.options().dtype(at::kByte));
        Strides s;
        s.heads(gq), s.heads(gk), s.tokens(r.q), s.tokens(r.k), s.tokens(dq), s.tokens(dk);
        const tfa_stream_t stream = stream_of(r.q);
        const int rc = without_gil([&] {
            return lib.rope_backward(gq.const_data_ptr(), gk.const_data_ptr(), r.q.const_data_ptr(), r.k.const_data_ptr(),
                                     dq.mutable_data_ptr(), dk.mutable_data_ptr(),
                                     static_cast<float *>(dwq.mutable_data_ptr()),
                                     static_cast<float *>(dwk.mutable_data_ptr()), s.s, r.wq, r.wk,
                                     static_cast<const double *>(r.freq.const_data_ptr()), r.pos, r.per_row, r.first, r.B,
                                     r.L, r.Hq, r.Hkv, r.D, r.rot, inter, eps, mscale, space.mutable_data_ptr(), stream);
        });
        return rc == TFA_OK ? result({dq, dk, dwq, dwk}) : PyLong_FromLong(rc);
    });
}

// The cache's four tensors.
struct Cache {
    const at::Tensor &kc, &km, &vc, &vm;
    int B, Hkv, cap, D;
    explicit Cache(PyObject *const *a)
        : kc(whole(leading(a[0], at::kByte, 4))), km(whole(beside(kc, a[1], at::kBFloat16, 5))),
          vc(whole(beside(kc, a[2], at::kByte, 4))), vm(whole(beside(kc, a[3], at::kBFloat16, 5))) {
        need(kc.size(3) <= 64);
        B = small(kc.size(0)), Hkv = small(kc.size(1)), cap = small(kc.size(2)), D = 2 * small(kc.size(3));
        sized(vc, kc.sizes());
        sized(km, {B, Hkv, cap, D / 32, 2});
        sized(vm, km.sizes());
    }
    void start(PyObject *o, const int **rows_, int *first) const {
        *rows_ = nullptr;
        *first = 0;
        if (PyLong_Check(o))
            *first = integer(o);
        else
            *rows_ = static_cast<const int *>(sized(whole(beside(kc, o, at::kInt, 1)), {B}).const_data_ptr());
    }
};

// k, v, the cache, start
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject * {
        const Cache c(a + 2);
        const at::Tensor &k = rows(beside(c.kc, a[0], at::kBFloat16, 4)), &v = rows(beside(c.kc, a[1], at::kBFloat16, 4));
        const int L = small(k.size(2));
        sized(k, {c.B, c.Hkv, L, c.D});
        sized(v, k.sizes());
        const int *start;
        int first;
        c.start(a[6], &start, &first);
        const long long s[6] = {k.stride(0), k.stride(1), k.stride(2), v.stride(0), v.stride(1), v.stride(2)};
        const tfa_stream_t stream = stream_of(c.kc);
        const int rc = without_gil([&] {
            return lib.append(k.const_data_ptr(), v.const_data_ptr(), s, c.kc.mutable_data_ptr(), c.km.mutable_data_ptr(),
                              c.vc.mutable_data_ptr(), c.vm.mutable_data_ptr(), start, first, c.B, c.Hkv, L, c.cap, c.D,
                              stream);
        });
        return PyLong_FromLong(rc);
    });
}

// the cache, start, rows
PyObject *read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject * {
        const Cache c(a);
        const int *start;
        int first;
        c.start(a[4], &start, &first);
        const int count = integer(a[5]);
        need(count >= 1 && (start || (first >= 0 && first <= c.cap - count)));
        const at::Tensor k = at::empty({c.B, c.Hkv, count, c.D}, c.km.options()), v = at::empty(k.sizes(), k.options());
        const tfa_stream_t stream = stream_of(c.kc);
        const int rc = without_gil([&] {
            return lib.read(c.kc.const_data_ptr(), c.km.const_data_ptr(), c.vc.const_data_ptr(), c.vm.const_data_ptr(),
                            k.mutable_data_ptr(), v.mutable_data_ptr(), start, first, c.B, c.Hkv, count, c.cap, c.D,
                            stream);
        });
        return rc == TFA_OK ? result({k, v}) : PyLong_FromLong(rc);
    });
}

const float *sinks_of(PyObject *o, const at::Tensor &q) {
    if (o == Py_None) return nullptr;
    return static_cast<const float *>(sized(whole(beside(q, o, at::kFloat, 1)), {q.size(1)}).const_data_ptr());
}

// q, the cache, lens, scale, window, first, softcap, sinks, out, workspace
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject * {
        const Cache c(a + 1);
        const at::Tensor &q = whole(beside(c.kc, a[0], at::kBFloat16, 4));
        need(q.size(0) == c.B && q.size(3) == c.D);
        const int Hq = small(q.size(1)), L = small(q.size(2));
        const at::Tensor &lens = sized(whole(beside(q, a[5], at::kInt, 1)), {c.B});
        const float scale = scale_or(a[6], c.D), softcap = number(a[9]);
        const int window = integer(a[7]), first = integer(a[8]);
        const float *sinks = sinks_of(a[10], q);
        const at::Tensor o = given_or_empty(a[11], q, q.sizes());
        const int64_t bytes = static_cast<int64_t>(lib.decode_workspace(Hq, c.Hkv, L, c.D));
        at::Tensor space;
        if (a[12] == Py_None)
            space = at::empty({bytes}, c.kc.options());
        else
            need((space = whole(beside(q, a[12], at::kByte, 1))).size(0) >= bytes);
        const tfa_stream_t stream = stream_of(q);
        const int rc = without_gil([&] {
            return lib.decode(q.const_data_ptr(), c.kc.const_data_ptr(), c.km.const_data_ptr(), c.vc.const_data_ptr(),
                              c.vm.const_data_ptr(), static_cast<const int *>(lens.const_data_ptr()),
                              o.mutable_data_ptr(), c.B, Hq, c.Hkv, L, c.cap, c.D, scale, window, first, softcap, sinks,
                              space.mutable_data_ptr(), stream);
        });
        return rc == TFA_OK ? result(o) : PyLong_FromLong(rc);
    });
}

// q, the cache, S, scale, window, first, softcap, sinks, out, workspace
PyObject *prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject * {
        const Cache c(a + 1);
        const at::Tensor &q = whole(beside(c.kc, a[0], at::kBFloat16, 4));
        need(q.size(0) == c.B && q.size(3) == c.D);
        const int Hq = small(q.size(1)), L = small(q.size(2)), S = integer(a[5]);
        const float scale = scale_or(a[6], c.D), softcap = number(a[9]);
        const int window = integer(a[7]), first = integer(a[8]);
        const float *sinks = sinks_of(a[10], q);
        const at::Tensor o = given_or_empty(a[11], q, q.sizes());
        const int64_t bytes = static_cast<int64_t>(lib.prefill_workspace(c.B, Hq, c.Hkv, L, S, c.D, window, first));
        at::Tensor space;
        if (a[12] == Py_None)
            space = at::empty({bytes < 16 ? 16 : bytes}, c.kc.options());
        else
            need((space = whole(beside(q, a[12], at::kByte, 1))).size(0) >= bytes && space.size(0) >= 16);
        const tfa_stream_t stream = stream_of(q);
        const int rc = without_gil([&] {
            return lib.prefill(q.const_data_ptr(), c.kc.const_data_ptr(), c.km.const_data_ptr(), c.vc.const_data_ptr(),
                               c.vm.const_data_ptr(), o.mutable_data_ptr(), c.B, Hq, c.Hkv, L, S, c.cap, c.D, scale,
                               window, first, softcap, sinks, space.mutable_data_ptr(), stream);
        });
        return rc == TFA_OK ? result(o) : PyLong_FromLong(rc);
    });
}

// The dense tensors of attention with first tokens.
struct First {
    const at::Tensor &q, &k, &v;
    int B, Hq, Hkv, L, S, D;
    const float *mask = nullptr;
    First(PyObject *q_, PyObject *k_, PyObject *v_, PyObject *mask_)
        : q(whole(leading(q_, at::kBFloat16, 4))), k(whole(beside(q, k_, at::kBFloat16, 4))),
          v(whole(beside(q, v_, at::kBFloat16, 4))) {
        B = small(q.size(0)), Hq = small(q.size(1)), L = small(q.size(2)), D = small(q.size(3));
        Hkv = small(k.size(1)), S = small(k.size(2));
        need(k.size(0) == B && k.size(3) == D);
        sized(v, k.sizes());
        if (mask_ != Py_None)
            mask = static_cast<const float *>(sized(whole(beside(q, mask_, at::kFloat, 2)), {B, S}).const_data_ptr());
    }
};

// q, k, v, scale, window, first, key_mask, softcap, sinks, out, lse, want_lse
PyObject *prefill_first(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject * {
        const First d(a[0], a[1], a[2], a[6]);
        const float scale = scale_or(a[3], d.D), softcap = number(a[7]);
        const int window = integer(a[4]), first = integer(a[5]);
        const float *sinks = sinks_of(a[8], d.q);
        const int want = truth(a[11]);
        const at::Tensor o = given_or_empty(a[9], d.q, d.q.sizes());
        at::Tensor lse;
        if (a[10] != Py_None)
            lse = sized(whole(beside(d.q, a[10], at::kFloat, 3)), {d.B, d.Hq, d.L});
        else if (want)
            lse = at::empty({d.B, d.Hq, d.L}, d.q.options().dtype(at::kFloat));
        const tfa_stream_t stream = stream_of(d.q);
        const int rc = without_gil([&] {
            return lib.first(d.q.const_data_ptr(), d.k.const_data_ptr(), d.v.const_data_ptr(), o.mutable_data_ptr(),
                             lse.defined() ? static_cast<float *>(lse.mutable_data_ptr()) : nullptr, d.B, d.Hq, d.Hkv,
                             d.L, d.S, d.D, scale, window, first, d.mask, softcap, sinks, stream);
        });
        return rc == TFA_OK ? result({o, lse}) : PyLong_FromLong(rc);
    });
}

// q, k, v, dout, o, lse, scale, window, first, key_mask
PyObject *backward_first(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        const First d(a[0], a[1], a[2], a[9]);
        const at::Tensor &dout = sized(whole(beside(d.q, a[3], at::kBFloat16, 4)), d.q.sizes());
        const at::Tensor &o = sized(whole(beside(d.q, a[4], at::kBFloat16, 4)), d.q.sizes());
        const at::Tensor &lse = sized(whole(beside(d.q, a[5], at::kFloat, 3)), {d.B, d.Hq, d.L});
        const float scale = scale_or(a[6], d.D);
        const int window = integer(a[7]), first = integer(a[8]);
        const at::Tensor dq = at::empty(d.q.sizes(), d.q.options());
        const at::Tensor dk = at::empty(d.k.sizes(), d.q.options()), dv = at::empty(d.k.sizes(), d.q.options());
        const tfa_stream_t stream = stream_of(d.q);
        const int rc = without_gil([&] {
            return lib.first_backward(d.q.const_data_ptr(), d.k.const_data_ptr(), d.v.const_data_ptr(),
                                      o.const_data_ptr(), static_cast<const float *>(lse.const_data_ptr()),
                                      dout.const_data_ptr(), dq.mutable_data_ptr(), dk.mutable_data_ptr(),
                                      dv.mutable_data_ptr(), d.B, d.Hq, d.Hkv, d.L, d.S, d.D, scale, window, first,
                                      d.mask, stream);
        });
        return rc == TFA_OK ? result({dq, dk, dv}) : PyLong_FromLong(rc);
    });
}

// The library's addresses, in the order of Library.
PyObject *use(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *at[11];
    if (n != 11) {
        PyErr_SetString(PyExc_TypeError, "11 addresses wanted");
        return nullptr;
    }
    for (int i = 0; i < 11; ++i)
        if ((at[i] = PyLong_AsVoidPtr(a[i])) == nullptr && PyErr_Occurred()) return nullptr;
    lib.rope = reinterpret_cast<decltype(lib.rope)>(at[0]);
    lib.rope_backward = reinterpret_cast<decltype(lib.rope_backward)>(at[1]);
    lib.rope_workspace = reinterpret_cast<decltype(lib.rope_workspace)>(at[2]);
    lib.append = reinterpret_cast<decltype(lib.append)>(at[3]);
    lib.read = reinterpret_cast<decltype(lib.read)>(at[4]);
    lib.decode = reinterpret_cast<decltype(lib.decode)>(at[5]);
    lib.decode_workspace = reinterpret_cast<decltype(lib.decode_workspace)>(at[6]);
    lib.first = reinterpret_cast<decltype(lib.first)>(at[7]);
    lib.first_backward = reinterpret_cast<decltype(lib.first_backward)>(at[8]);
    lib.prefill = reinterpret_cast<decltype(lib.prefill)>(at[9]);
    lib.prefill_workspace = reinterpret_cast<decltype(lib.prefill_workspace)>(at[10]);
    Py_RETURN_NONE;
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(use),     CALL(rope),          CALL(rope_backward),  CALL(append), CALL(read), CALL(decode),
                         CALL(prefill), CALL(prefill_first), CALL(backward_first), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch whose tensors this code reads, and the Python.
PyMODINIT_FUNC PyInit__calls(void) {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", TFA_BUILT_FOR) < 0) Py_CLEAR(m);
    return m;
}
