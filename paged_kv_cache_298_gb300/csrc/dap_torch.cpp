// dap_torch.cpp -- argument marshalling of the calls whose time on the host counts most, as a Python
// extension: it looks at the tensors, checks them, and calls the C ABI (include/dap.h) on their device's
// current stream.  The same checks and conversions written in Python with ctypes took 9 of the 13
// microseconds that such a call took on the host (27 of 31 with three launches); here they take about 1.
// No arithmetic and no launch of its own.  Every function raises ValueError for a tensor of the wrong kind
// or shape and DapError (binding.py) for one on another device and for a status of the library.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "dap.h"

namespace {

PyObject *g_error = nullptr;  // binding.DapError

// Thrown after a Python error has been set.
struct Raised {};

[[noreturn]] void value_error(const char *msg) {
    PyErr_SetString(PyExc_ValueError, msg);
    throw Raised();
}

[[noreturn]] void dap_error(PyObject *status, const std::string &what) {
    if (g_error) {
        PyObject *e = PyObject_CallFunction(g_error, "Os", status, what.c_str());
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
    } else {
        PyErr_SetString(PyExc_RuntimeError, what.c_str());
    }
    throw Raised();
}

void check_status(dap_status st, const char *what) {
    if (st == DAP_OK) return;
    PyObject *code = PyLong_FromLong((long)st);
    struct Drop {
        PyObject *o;
        ~Drop() { Py_XDECREF(o); }
    } drop{code};
    dap_error(code, what);
}

// The call's tensors: each must be a CUDA tensor on the device of the first.
struct Call {
    const char *what;
    int device = -1;
    const at::Tensor &tensor(PyObject *o, const char *name) {
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "%s: %s must be a tensor", what, name);
            throw Raised();
        }
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda()) {
            if (device < 0) dap_error(Py_None, std::string(what) + ": the first tensor must be a CUDA tensor");
            dap_error(Py_None, std::string(what) + ": " + name + " is not a CUDA tensor");
        }
        const int d = (int)t.get_device();
        if (device < 0) device = d;
        if (d != device)
            dap_error(Py_None, std::string(what) + ": " + name + " is on cuda:" + std::to_string(d) +
                                   ", the call's tensors on cuda:" + std::to_string(device));
        return t;
    }
    const at::Tensor *optional(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }
};

long long integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}

int integer32(PyObject *o) {
    const long long v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) value_error("an integer argument does not fit 32 bits");
    return (int)v;
}

// The call's device and stream (a given handle, or the device's current stream) made current: what the call
// allocates belongs to the stream that its kernels run on, so that a workspace freed here is not handed to another
// stream while they run.
struct On {
    c10::cuda::CUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard given;
    void *stream;
    On(PyObject *o, int index) : device((c10::DeviceIndex)index) {
        if (o == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
            return;
        }
        stream = PyLong_AsVoidPtr(o);
        if (!stream && PyErr_Occurred()) throw Raised();
        given.reset_stream(
            c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), (c10::DeviceIndex)index));
    }
};

int fit(int64_t n, const char *msg) {
    if (n > INT32_MAX) value_error(msg);
    return (int)n;
}

void rows3(const at::Tensor &t, const char *msg) {
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.stride(2) != 1) value_error(msg);
}

bool int32s(const at::Tensor &t) { return t.scalar_type() == at::kInt && t.is_contiguous(); }

void table_of(const at::Tensor &t, int64_t B) {
    if (!int32s(t) || t.dim() != 2 || t.size(0) != B) value_error("block_table must be contiguous int32 [B, max_pages]");
}

// A contiguous tensor on the device (straight from its allocator: at::empty's dispatch takes 0.7 us more).
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, int device) {
    return at::Tensor(
        at::detail::empty_cuda(sizes, type, at::Device(at::kCUDA, (c10::DeviceIndex)device), std::nullopt));
}

// The e4m3 cache's four arrays and a run's three, as append and read take them.
struct Runs {
    const uint8_t *codes[2];
    void *scale[2];
    int P, ps, Hkv, D, max_pages, B;
    const int32_t *table, *indptr, *positions;
    Runs(Call &c, PyObject *const *a) {
        const at::Tensor &kc = c.tensor(a[0], "k_codes"), &vc = c.tensor(a[1], "v_codes");
        const at::Tensor &ks = c.tensor(a[2], "k_scale"), &vs = c.tensor(a[3], "v_scale");
        const at::Tensor &bt = c.tensor(a[4], "block_table"), &ip = c.tensor(a[5], "indptr");
        const at::Tensor &po = c.tensor(a[6], "positions");
        if (kc.scalar_type() != at::kByte || kc.dim() != 4 || !kc.is_contiguous() || vc.scalar_type() != at::kByte ||
            vc.sizes() != kc.sizes() || !vc.is_contiguous())
            value_error("k_codes/v_codes must be contiguous uint8 [P, ps, Hkv, D]");
        P = fit(kc.size(0), "too many pages");
        ps = fit(kc.size(1), "page size too large");
        Hkv = fit(kc.size(2), "too many heads");
        D = fit(kc.size(3), "head dim too large");
        for (const at::Tensor *f : {&ks, &vs})
            if (f->scalar_type() != at::kBFloat16 || !f->is_contiguous() || f->dim() != 3 || f->size(0) != P ||
                f->size(1) != Hkv || f->size(2) != ps)
                value_error("k_scale/v_scale must be contiguous bf16 [P, Hkv, ps]");
        B = fit(po.numel(), "too many sequences");
        table_of(bt, B);
        if (!int32s(ip) || ip.numel() != (int64_t)B + 1) value_error("indptr must be contiguous int32 [B + 1]");
        if (!int32s(po)) value_error("positions must be contiguous int32 [B]");
        codes[0] = static_cast<const uint8_t *>(kc.data_ptr());
        codes[1] = static_cast<const uint8_t *>(vc.data_ptr());
        scale[0] = ks.data_ptr();
        scale[1] = vs.data_ptr();
        max_pages = fit(bt.size(1), "block_table too wide");
        table = static_cast<const int32_t *>(bt.data_ptr());
        indptr = static_cast<const int32_t *>(ip.data_ptr());
        positions = static_cast<const int32_t *>(po.data_ptr());
    }
};

// append_runs(k_new, v_new, k_codes, v_codes, k_scale, v_scale, block_table, indptr, positions, stream)
void append_runs(PyObject *const *a) {
    const char *what = "kv_append_paged_fp8_multi";
    Call c{what};
    const at::Tensor &k = c.tensor(a[0], "k_new"), &v = c.tensor(a[1], "v_new");
    const Runs r(c, a + 2);
    rows3(k, "k_new must be a bf16 [*, *, D] tensor with unit stride in D");
    rows3(v, "v_new must be a bf16 [*, *, D] tensor with unit stride in D");
    if (v.sizes() != k.sizes() || k.size(1) != r.Hkv || k.size(2) != r.D)
        value_error("cache heads / dims differ from the new rows");
    const int T = fit(k.size(0), "too many tokens");
    const On on(a[9], c.device);
    dap_status st;
    Py_BEGIN_ALLOW_THREADS;  // (nothing in here may raise)
    st = kv_append_paged_fp8_multi(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                                   const_cast<uint8_t *>(r.codes[0]), const_cast<uint8_t *>(r.codes[1]), r.scale[0],
                                   r.scale[1], r.P, r.ps, r.table, r.max_pages, r.indptr, r.positions, T, r.B, r.Hkv,
                                   r.D, on.stream);
    Py_END_ALLOW_THREADS;
    check_status(st, what);
}

// read_runs(k_codes, v_codes, k_scale, v_scale, block_table, indptr, positions, total_tokens, k_out, v_out,
// stream) -> (k_out, v_out)
PyObject *read_runs(PyObject *const *a) {
    const char *what = "kv_read_paged_fp8";
    Call c{what};
    const Runs r(c, a);
    at::Tensor out[2];
    const at::Tensor *given[2] = {c.optional(a[8], "k_out"), c.optional(a[9], "v_out")};
    int64_t T;
    if (a[7] != Py_None) T = integer32(a[7]);
    else if (given[0] || given[1]) T = (given[0] ? given[0] : given[1])->size(0);
    else value_error("total_tokens is needed when no output is given");
    if (T < 0) value_error("total_tokens must not be negative");
    fit(T, "too many tokens");
    const On on(a[10], c.device);
    for (int i = 0; i < 2; ++i) {
        if (given[i]) {
            rows3(*given[i], "k_out and v_out must be bf16 [*, *, D] tensors with unit stride in D");
            if (given[i]->size(0) != T || given[i]->size(1) != r.Hkv || given[i]->size(2) != r.D)
                value_error("k_out and v_out must be [total_tokens, Hkv, D]");
            out[i] = *given[i];
        } else {
            out[i] = fresh({T, r.Hkv, r.D}, at::kBFloat16, c.device);
        }
    }
    dap_status st;
    Py_BEGIN_ALLOW_THREADS;  // (nothing in here may raise)
    st = kv_read_paged_fp8(r.codes[0], r.codes[1], r.scale[0], r.scale[1], r.P, r.ps, r.table, r.max_pages, r.indptr,
                           r.positions, (int)T, r.B, r.Hkv, r.D, out[0].data_ptr(),
                           out[1].data_ptr(), out[0].stride(0), out[0].stride(1), out[1].stride(0), out[1].stride(1),
                           on.stream);
    Py_END_ALLOW_THREADS;
    check_status(st, what);
    PyObject *k = THPVariable_Wrap(out[0]), *v = THPVariable_Wrap(out[1]);
    PyObject *both = k && v ? PyTuple_Pack(2, k, v) : nullptr;
    Py_XDECREF(k);
    Py_XDECREF(v);
    return both;
}

// decode_shared(q, k_cache, v_cache, block_table, seq_lens, prefix_lens, the plan's map [tiles, then seq_group],
// (B, Hq, Hkv, D, groups, tiles, seqs_per_tile), max_prefix_len, max_suffix_len, (prefix_splits, suffix_splits), scale,
// workspace, out, stream) -> out
PyObject *decode_shared(PyObject *const *a) {
    const char *what = "decode_attn_paged_shared";
    Call c{what};
    const at::Tensor &q = c.tensor(a[0], "q"), &k = c.tensor(a[1], "k_cache"), &v = c.tensor(a[2], "v_cache");
    const at::Tensor &bt = c.tensor(a[3], "block_table"), &sl = c.tensor(a[4], "seq_lens");
    const at::Tensor &pl = c.tensor(a[5], "prefix_lens"), &map = c.tensor(a[6], "plan");
    const at::Tensor *wg = c.optional(a[12], "workspace"), *og = c.optional(a[13], "out");
    int d[7];
    for (int i = 0; i < 7; ++i) d[i] = integer32(PyTuple_GET_ITEM(a[7], i));
    const int B = d[0], Hq = d[1], Hkv = d[2], D = d[3], groups = d[4], tiles = d[5];
    if (!int32s(map) || map.numel() != 4 * (int64_t)tiles + B)
        value_error("the plan's map does not fit its sizes");
    rows3(q, "q must be a bf16 [*, *, D] tensor with unit stride in D");
    if (q.size(0) != B || q.size(1) != Hq || q.size(2) != D)
        value_error("q differs from the plan's batch, heads or head dim");
    if (k.scalar_type() != at::kBFloat16 || k.dim() != 4 || !k.is_contiguous() || v.scalar_type() != at::kBFloat16 ||
        v.sizes() != k.sizes() || !v.is_contiguous())
        value_error("k_cache/v_cache must be contiguous bf16 [P, ps, Hkv, D]");
    if (k.size(2) != Hkv || k.size(3) != D) value_error("the cache's kv heads or head dim differ from the plan's");
    table_of(bt, B);
    if (!int32s(sl) || sl.numel() != B) value_error("seq_lens must be contiguous int32 [B]");
    if (!int32s(pl) || pl.numel() != groups) value_error("prefix_lens must be contiguous int32 [num_groups]");
    const int P = fit(k.size(0), "too many pages"), ps = fit(k.size(1), "page size too large");
    const int max_pages = fit(bt.size(1), "block_table too wide");
    const int max_prefix = integer32(a[8]), max_suffix = integer32(a[9]);
    const int pre = integer32(PyTuple_GET_ITEM(a[10], 0)), suf = integer32(PyTuple_GET_ITEM(a[10], 1));
    const double scale = PyFloat_AsDouble(a[11]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised();
    const On on(a[14], c.device);
    at::Tensor out, ws;
    if (og) {
        rows3(*og, "out must be a bf16 [*, *, D] tensor with unit stride in D");
        if (og->sizes() != q.sizes()) value_error("out must be [B, Hq, D]");
        out = *og;
    } else {
        out = fresh({B, Hq, D}, at::kBFloat16, c.device);
    }
    ws = wg ? *wg : fresh({(int64_t)dap_workspace_bytes_shared(B, Hq, D, pre, suf)}, at::kByte, c.device);
    if (!ws.is_contiguous()) value_error("workspace must be contiguous");
    const int32_t *m = static_cast<const int32_t *>(map.data_ptr());
    dap_status st;
    Py_BEGIN_ALLOW_THREADS;  // (nothing in here may raise)
    st = decode_attn_paged_shared(
        q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(), v.data_ptr(), P, ps,
        static_cast<const int32_t *>(bt.data_ptr()), max_pages, static_cast<const int32_t *>(sl.data_ptr()),
        static_cast<const int32_t *>(pl.data_ptr()), m + 4 * (int64_t)tiles, m, groups, tiles, d[6], max_prefix, max_suffix, B, Hq, Hkv, D, (float)scale, pre, suf, ws.data_ptr(), ws.nbytes(),
        out.data_ptr(), out.stride(0), out.stride(1), on.stream);
    Py_END_ALLOW_THREADS;
    check_status(st, what);
    return THPVariable_Wrap(out);
}

template <class F>
PyObject *entry(Py_ssize_t n, Py_ssize_t want, F f) {
    HANDLE_TH_ERRORS
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *py_append_runs(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry(n, 10, [&]() -> PyObject * {
        append_runs(a);
        Py_RETURN_NONE;
    });
}
PyObject *py_read_runs(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry(n, 11, [&] { return read_runs(a); });
}
PyObject *py_decode_shared(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return entry(n, 15, [&] { return decode_shared(a); });
}
PyObject *py_set_error(PyObject *, PyObject *cls) {
    Py_XINCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

template <class F>
PyCFunction as_function(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f));
}

PyMethodDef g_methods[] = {
    {"append_runs", as_function(py_append_runs), METH_FASTCALL, "kv_append_paged_fp8_multi on tensors"},
    {"read_runs", as_function(py_read_runs), METH_FASTCALL, "kv_read_paged_fp8 on tensors"},
    {"decode_shared", as_function(py_decode_shared), METH_FASTCALL, "decode_attn_paged_shared on tensors"},
    {"set_error", py_set_error, METH_O, "the exception class for library statuses"},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_dap_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dap_torch(void) { return PyModule_Create(&g_module); }
