// sv_bind.cpp -- the short way from Python to the target-step operators.
//
// A decode step makes these calls for every layer on small tensors, where a call's time is
// the host's: taking tensors apart in Python and packing the arguments costs about 10 us on
// top of the launch.  This module does it in C++ for calls whose tensors need no
// conversion (types, device, contiguity, alignment, torch's current device and stream) and
// returns None for any other, which the Python functions in target.py then serve or refuse.
// It calls the same C entry points, through their addresses, and allocates only what those
// functions do.
#include <ATen/ATen.h>
#include <ATen/cuda/CUDAContext.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <map>
#include <utility>

#include "spec_verify_target.h"

namespace {

int (*g_logits)(const sv_logits_args*, void*) = nullptr;
int (*g_rotate)(const sv_rotate_args*, void*) = nullptr;
int (*g_attention)(const sv_attention_args*, void*) = nullptr;
size_t (*g_attention_ws)(int64_t, int64_t, int64_t, int64_t, int64_t) = nullptr;
PyObject* g_error = nullptr;  // raises for a status: g_error(status)

// "not served here" (also for a number that is none: the Python side names the error)
#define SV_NONE                \
    do {                       \
        PyErr_Clear();         \
        Py_RETURN_NONE;        \
    } while (0)

// the tensor of an argument; false: not a tensor
inline bool tensor(PyObject* o, const at::Tensor** t) {
    if (!THPVariable_Check(o)) return false;
    *t = &THPVariable_Unpack(o);
    return true;
}
inline bool on(const at::Tensor& t, const at::Device& d, at::ScalarType s) {
    return t.scalar_type() == s && t.device() == d;
}
// an optional per-sequence vector: its address (None: 0); false where it needs conversion
inline bool vec(PyObject* o, const at::Device& d, at::ScalarType s, int64_t n, const void** p) {
    *p = nullptr;
    if (o == Py_None) return true;
    const at::Tensor* t;
    if (!tensor(o, &t) || !on(*t, d, s) || t->dim() != 1 || t->size(0) != n || !t->is_contiguous()) return false;
    *p = t->data_ptr();
    return true;
}
inline bool table(PyObject* o, const at::Device& d, int64_t rows, int64_t cols, const at::Tensor** t) {
    return tensor(o, t) && on(**t, d, at::kInt) && (*t)->dim() == 2 && (*t)->size(0) == rows &&
           (*t)->size(1) >= cols && ((*t)->stride(1) == 1 || (*t)->size(1) == 1);
}
// a page table with rows of their own
inline bool page_table(PyObject* o, const at::Device& d, int64_t B, const at::Tensor** t) {
    return table(o, d, B, 1, t) && (B < 2 || (*t)->stride(0) >= (*t)->size(1));
}
// rows [B, N, heads, dim] as the kernels take them
inline bool rows(const at::Tensor& t) {
    return t.stride(3) == 1 && !((t.stride(0) | t.stride(1) | t.stride(2)) & 7) && !((uintptr_t)t.data_ptr() & 15);
}
inline bool same_rows(const at::Tensor& t, const at::Device& d, at::ScalarType s, int64_t B, int64_t N, int64_t H,
                      int64_t D) {
    return on(t, d, s) && t.dim() == 4 && t.size(0) == B && t.size(1) == N && t.size(2) == H && t.size(3) == D && rows(t);
}
inline bool current(const at::Device& d) { return d.is_cuda() && d.index() == c10::cuda::current_device(); }

// a status of the C call: the result, or the exception
inline PyObject* done(int status, const at::Tensor& out) {
    if (status != 0) {
        PyObject* r = PyObject_CallFunction(g_error, "i", status);
        Py_XDECREF(r);
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "the call failed");
        return nullptr;
    }
    return THPVariable_Wrap(out);
}

// a PagedCache's keys and values, as they are at this call: [pages, heads, page_size, dim]
inline bool pages(PyObject* ko, PyObject* vo, const at::Device& d, const at::Tensor** k, const at::Tensor** v) {
    if (!tensor(ko, k) || !tensor(vo, v)) return false;
    const at::Tensor &x = **k, &y = **v;
    const at::ScalarType s = x.scalar_type();
    return (s == at::kBFloat16 || s == at::kHalf) && on(x, d, s) && on(y, d, s) && x.dim() == 4 && x.sizes() == y.sizes() &&
           x.size(2) >= 16 && x.size(2) % 16 == 0 && rows(x) && rows(y);
}
inline void fill(sv_paged_cache* c, const at::Tensor& k, const at::Tensor& v, const at::Tensor& pt, const void* lens,
                 const void* fresh) {
    c->k_pages = k.data_ptr(), c->v_pages = v.data_ptr();
    c->pages = k.size(0), c->page_size = k.size(2);
    c->k_stride_page = k.stride(0), c->k_stride_head = k.stride(1), c->k_stride_slot = k.stride(2);
    c->v_stride_page = v.stride(0), c->v_stride_head = v.stride(1), c->v_stride_slot = v.stride(2);
    c->page_table = pt.data_ptr<int32_t>();
    c->page_table_stride = pt.stride(0);
    c->pages_per_seq = pt.size(1);
    c->cache_lens = (const int32_t*)lens;
    c->num_new = (const int32_t*)fresh;
}
inline int64_t code(at::ScalarType s) { return s == at::kBFloat16 ? SV_BF16 : SV_F16; }

// scratch of the calls on one stream, which follow one another
at::Tensor& scratch(const at::Device& d, void* stream, int64_t bytes) {
    static auto* all = new std::map<std::pair<int, void*>, at::Tensor>;  // (kept: the device outlives no destructor)
    at::Tensor& t = (*all)[{d.index(), stream}];
    if (!t.defined() || t.numel() < bytes) t = at::empty({bytes}, at::TensorOptions().device(d).dtype(at::kByte));
    return t;
}

// attention(q, cache's k, v, page_table, cache_lens, num_new, scale (None: the default), window, max_context, out,
//           row_status, wait_limit_ns)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *q, *ck, *cv, *pt, *given = nullptr;
    if (n != 12 || !tensor(a[0], &q) || q->dim() != 4) SV_NONE;
    const at::Device d = q->device();
    const int64_t B = q->size(0), N = q->size(1), Hq = q->size(2), D = q->size(3);
    if (!current(d) || !pages(a[1], a[2], d, &ck, &cv)) SV_NONE;
    const int64_t Hkv = ck->size(1);
    const at::ScalarType s = ck->scalar_type();
    if (q->scalar_type() != s || D != ck->size(3) || !rows(*q) || Hkv < 1 || Hq % Hkv || B == 0) SV_NONE;
    const void *lens, *fresh, *status;
    if (!page_table(a[3], d, B, &pt) || !vec(a[4], d, at::kInt, B, &lens) || !lens || !vec(a[5], d, at::kInt, B, &fresh) ||
        !vec(a[10], d, at::kInt, B, &status))
        SV_NONE;
    if (a[9] != Py_None && (!tensor(a[9], &given) || !same_rows(*given, d, s, B, N, Hq, D))) SV_NONE;
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) SV_NONE;
    sv_attention_args g;
    std::memset(&g, 0, sizeof g);
    fill(&g.cache, *ck, *cv, *pt, lens, fresh);
    g.scale = a[6] == Py_None ? 1.0 / std::sqrt((double)D) : PyFloat_AsDouble(a[6]);
    g.window = PyLong_AsLongLong(a[7]);
    g.max_context = a[8] == Py_None ? 0 : PyLong_AsLongLong(a[8]);
    g.wait_limit_ns = PyLong_AsUnsignedLongLong(a[11]);
    if (PyErr_Occurred() || g.window < 0) SV_NONE;
    void* stream = at::cuda::getCurrentCUDAStream(d.index()).stream();
    const size_t bytes = g_attention_ws(B, N, Hq, Hkv, D);
    if (bytes == 0) SV_NONE;
    at::Tensor& ws = scratch(d, stream, (int64_t)bytes);
    at::Tensor out = given ? *given : at::empty(q->sizes(), q->options());
    g.struct_size = sizeof g;
    g.q = q->data_ptr();
    g.out = out.data_ptr();
    g.dtype = code(s);
    g.B = B, g.N = N, g.q_heads = Hq, g.kv_heads = Hkv, g.dim = D;
    g.q_stride_b = q->stride(0), g.q_stride_n = q->stride(1), g.q_stride_h = q->stride(2);
    g.o_stride_b = out.stride(0), g.o_stride_n = out.stride(1), g.o_stride_h = out.stride(2);
    g.workspace = ws.data_ptr();
    g.workspace_bytes = ws.numel();
    g.row_status = (uint32_t*)status;
    return done(g_attention(&g, stream), out);
    END_HANDLE_TH_ERRORS
}

// rotate(q, k, v, table, cache's k, v, page_table, cache_lens, num_new, interleaved, out, row_status)
PyObject* rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *q, *k, *v, *tab, *ck, *cv, *pt, *given = nullptr;
    if (n != 12 || !tensor(a[0], &q) || !tensor(a[1], &k) || !tensor(a[2], &v) || !tensor(a[3], &tab) || q->dim() != 4)
        SV_NONE;
    const at::Device d = q->device();
    const int64_t B = q->size(0), N = q->size(1), Hq = q->size(2), D = q->size(3);
    if (!current(d) || !pages(a[4], a[5], d, &ck, &cv)) SV_NONE;
    const int64_t Hkv = ck->size(1);
    const at::ScalarType s = ck->scalar_type();
    if (q->scalar_type() != s || D != ck->size(3) || !rows(*q) || B == 0 || !same_rows(*k, d, s, B, N, Hkv, D) ||
        !same_rows(*v, d, s, B, N, Hkv, D))
        SV_NONE;
    if (!on(*tab, d, at::kFloat) || tab->dim() != 3 || tab->size(1) != 2 || !tab->is_contiguous() || tab->size(2) < 8 ||
        tab->size(2) % 8 || 2 * tab->size(2) > D)
        SV_NONE;
    const void *lens, *fresh, *status;
    if (!page_table(a[6], d, B, &pt) || !vec(a[7], d, at::kInt, B, &lens) || !lens || !vec(a[8], d, at::kInt, B, &fresh) ||
        !vec(a[11], d, at::kInt, B, &status))
        SV_NONE;
    if (a[10] != Py_None && (!tensor(a[10], &given) || !same_rows(*given, d, s, B, N, Hq, D))) SV_NONE;
    sv_rotate_args g;
    std::memset(&g, 0, sizeof g);
    fill(&g.cache, *ck, *cv, *pt, lens, fresh);
    const int turn = PyObject_IsTrue(a[9]);
    if (turn < 0) SV_NONE;
    at::Tensor out = given ? *given : at::empty(q->sizes(), q->options());
    g.struct_size = sizeof g;
    g.q = q->data_ptr();
    g.q_out = out.data_ptr();
    g.k = k->data_ptr();
    g.v = v->data_ptr();
    g.dtype = code(s);
    g.B = B, g.N = N, g.q_heads = Hq, g.kv_heads = Hkv, g.dim = D;
    g.q_stride_b = q->stride(0), g.q_stride_n = q->stride(1), g.q_stride_h = q->stride(2);
    g.o_stride_b = out.stride(0), g.o_stride_n = out.stride(1), g.o_stride_h = out.stride(2);
    g.k_stride_b = k->stride(0), g.k_stride_n = k->stride(1), g.k_stride_h = k->stride(2);
    g.v_stride_b = v->stride(0), g.v_stride_n = v->stride(1), g.v_stride_h = v->stride(2);
    g.table = tab->data_ptr<float>();
    g.table_len = tab->size(0);
    g.rot_dim = 2 * tab->size(2);
    g.interleaved = turn;
    g.row_status = (uint32_t*)status;
    return done(g_rotate(&g, at::cuda::getCurrentCUDAStream(d.index()).stream()), out);
    END_HANDLE_TH_ERRORS
}

// logits(logits, seen, counts, slots, draft_tokens, repetition, frequency, presence, bias ids, values, offsets, mask,
//        out, row_status); seen, counts: the history's planes, or None
PyObject* logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *x, *seen = nullptr, *counts = nullptr, *toks = nullptr, *mask = nullptr, *given = nullptr;
    if (n != 14 || !tensor(a[0], &x) || x->dim() != 3) SV_NONE;
    const at::Device d = x->device();
    const int64_t B = x->size(0), N = x->size(1), V = x->size(2);
    if (!current(d) || (x->scalar_type() != at::kFloat && x->scalar_type() != at::kBFloat16) || x->stride(2) != 1 ||
        B == 0)
        SV_NONE;
    sv_logits_args g;
    std::memset(&g, 0, sizeof g);
    if (a[1] != Py_None) {
        if (!tensor(a[1], &seen) || !tensor(a[2], &counts) || !on(*seen, d, at::kInt) || !on(*counts, d, at::kInt) ||
            seen->dim() != 2 || counts->dim() != 2 || seen->size(0) != counts->size(0) || !seen->is_contiguous() ||
            !counts->is_contiguous() || 32 * seen->size(1) < V || counts->size(1) != V || (a[3] == Py_None && B > counts->size(0)))
            SV_NONE;
        g.seen = (const uint32_t*)seen->data_ptr();
        g.counts = counts->data_ptr<int32_t>();
        g.slots = counts->size(0);
        g.words = seen->size(1);
    }
    const void *slots, *rep, *freq, *pres, *status, *ids = nullptr, *vals = nullptr, *offs = nullptr;
    if (!vec(a[3], d, at::kInt, B, &slots) || !vec(a[5], d, at::kFloat, B, &rep) || !vec(a[6], d, at::kFloat, B, &freq) ||
        !vec(a[7], d, at::kFloat, B, &pres) || !vec(a[13], d, at::kInt, B, &status))
        SV_NONE;
    if (a[4] != Py_None && N > 1) {
        if (!table(a[4], d, B, N - 1, &toks)) SV_NONE;
        g.draft_tokens = toks->data_ptr<int32_t>();
        g.draft_stride = toks->stride(0);
        g.draft_len = toks->size(1);
    }
    if (a[8] != Py_None) {
        const at::Tensor* t;
        if (!tensor(a[8], &t) || t->dim() != 1) SV_NONE;
        const int64_t nb = t->size(0);
        if (nb == 0 || !vec(a[8], d, at::kInt, nb, &ids) || !vec(a[9], d, at::kFloat, nb, &vals) ||
            !vec(a[10], d, at::kInt, B + 1, &offs) || !vals || !offs)
            SV_NONE;
        g.bias_total = nb;
    }
    if (a[11] != Py_None) {
        if (!tensor(a[11], &mask) || !on(*mask, d, at::kInt)) SV_NONE;
        const int64_t dims = mask->dim();
        if ((dims != 2 && dims != 3) || mask->size(0) != B || (dims == 3 && mask->size(1) != N) ||
            32 * mask->size(-1) < V || mask->stride(-1) != 1)
            SV_NONE;
        g.mask = (const uint32_t*)mask->data_ptr();
        g.mask_stride_b = mask->stride(0);
        g.mask_stride_n = dims == 3 ? mask->stride(1) : 0;
    }
    if (a[12] != Py_None && (!tensor(a[12], &given) || !on(*given, d, x->scalar_type()) ||
                             given->sizes() != x->sizes() || given->stride(2) != 1))
        SV_NONE;
    at::Tensor out = given ? *given : at::empty(x->sizes(), x->options());
    g.struct_size = sizeof g;
    g.logits = x->data_ptr();
    g.out = out.data_ptr();
    g.dtype = x->scalar_type() == at::kFloat ? SV_F32 : SV_BF16;
    g.B = B, g.N = N, g.V = V;
    g.logits_stride_b = x->stride(0), g.logits_stride_n = x->stride(1);
    g.out_stride_b = out.stride(0), g.out_stride_n = out.stride(1);
    g.slot_of = seen ? (const int32_t*)slots : nullptr;
    g.repetition = (const float*)rep;
    g.frequency = (const float*)freq;
    g.presence = (const float*)pres;
    g.bias_ids = (const int32_t*)ids;
    g.bias_values = (const float*)vals;
    g.bias_offsets = (const int32_t*)offs;
    g.row_status = (uint32_t*)status;
    return done(g_logits(&g, at::cuda::getCurrentCUDAStream(d.index()).stream()), out);
    END_HANDLE_TH_ERRORS
}

// setup(addresses of the four C functions, the function that raises for a status)
PyObject* setup(PyObject*, PyObject* args) {
    unsigned long long l, r, t, w;
    PyObject* e;
    if (!PyArg_ParseTuple(args, "KKKKO", &l, &r, &t, &w, &e)) return nullptr;
    g_logits = (decltype(g_logits))l;
    g_rotate = (decltype(g_rotate))r;
    g_attention = (decltype(g_attention))t;
    g_attention_ws = (decltype(g_attention_ws))w;
    Py_INCREF(e);
    g_error = e;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"setup", setup, METH_VARARGS, nullptr},
                         {"attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, nullptr},
                         {"rotate", (PyCFunction)(void (*)(void))rotate, METH_FASTCALL, nullptr},
                         {"logits", (PyCFunction)(void (*)(void))logits, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "Short way to the target-step operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) { return PyModule_Create(&module); }
