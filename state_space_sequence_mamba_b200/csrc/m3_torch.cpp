// Argument marshalling of linear attention, the gated scan, rotary positions and the norms between torch
// tensors and the C ABI, in C++: a decode step's kernels take a few microseconds, as long as a dozen attribute reads in
// Python. Checks shapes, types and devices, allocates what the caller did not give, and calls the
// library's entry points (whose addresses the Python side hands over, so that both use the library
// that it loaded) on the tensors' device and its current stream. Computes nothing.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "m3.h"

namespace {

using at::Tensor;

struct Api {
    decltype(&m3_linattn_workspace_bytes) linattn_workspace;
    decltype(&m3_linattn_bwd_workspace_bytes) linattn_bwd_workspace;
    decltype(&m3_linattn_fwd) linattn_fwd;
    decltype(&m3_linattn_step) linattn_step;
    decltype(&m3_linattn_bwd) linattn_bwd;
    decltype(&m3_group_norm_fwd) group_norm_fwd;
    decltype(&m3_group_norm_bwd_workspace_bytes) group_norm_bwd_workspace;
    decltype(&m3_group_norm_bwd) group_norm_bwd;
    decltype(&m3_gated_scan_fwd) gated_scan_fwd;
    decltype(&m3_gated_scan_step) gated_scan_step;
    decltype(&m3_gated_scan_bwd_workspace_bytes) gated_scan_bwd_workspace;
    decltype(&m3_gated_scan_bwd) gated_scan_bwd;
    decltype(&m3_rotary) rotary;
    decltype(&m3_block_norm_fwd) block_norm_fwd;
    decltype(&m3_block_norm_bwd_workspace_bytes) block_norm_bwd_workspace;
    decltype(&m3_block_norm_bwd) block_norm_bwd;
} api;

const Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}
// nullptr for None
const Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

void same_device(const Tensor& ref, const Tensor* t, const char* name) {
    if (t) TORCH_CHECK_VALUE(t->device() == ref.device(), name, " is on ", t->device(), ", other tensors on ", ref.device());
}

int32_t dtype_code(const Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return M3_BF16;
    TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat, "unsupported input dtype ", t.scalar_type());
    return M3_F32;
}

// A tensor [b, L, heads, dim] (a step's: [b, heads, dim]) by its strides.
m3_view view(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type) {
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", t.sizes(), ", expected ", shape);
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " is ", t.scalar_type(), ", expected ", type);
    const int64_t n = t.dim();
    TORCH_CHECK_VALUE(t.stride(n - 1) == 1 || shape[n - 1] <= 1, name, ": the last dimension must be contiguous");
    return n == 4 ? m3_view{t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)}
                  : m3_view{t.data_ptr(), t.stride(0), 0, t.stride(1)};
}
m3_view out_view(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type) {
    const m3_view v = view(t, name, shape, type);
    for (int64_t i = 0; i < t.dim(); ++i)
        TORCH_CHECK_VALUE(t.stride(i) != 0 || shape[i] <= 1, name, " is written and must not be expanded");
    return v;
}

float* f32(const Tensor* t, const char* name, at::IntArrayRef shape) {
    if (!t) return nullptr;
    TORCH_CHECK_VALUE(t->sizes() == shape, name, " has shape ", t->sizes(), ", expected ", shape);
    TORCH_CHECK_VALUE(t->scalar_type() == at::kFloat, name, " must be float32");
    TORCH_CHECK_VALUE(t->is_contiguous(), name, " must be contiguous");
    return static_cast<float*>(t->data_ptr());
}
const int32_t* i32(const Tensor* t, const char* name, int64_t n) {
    if (!t) return nullptr;
    TORCH_CHECK_VALUE(t->scalar_type() == at::kInt && t->dim() == 1 && t->is_contiguous(), name,
                      " must be a contiguous int32 vector");
    TORCH_CHECK_VALUE(n < 0 || t->size(0) == n, name, " has ", t->size(0), " values, expected ", n);
    return static_cast<const int32_t*>(t->data_ptr());
}

// the caller's workspace or a new one
Tensor workspace(const Tensor* given, size_t need, const Tensor& ref) {
    if (given) {
        TORCH_CHECK_VALUE(given->device() == ref.device() && given->is_contiguous(),
                          "workspace must be contiguous and on the tensors' device");
        return *given;
    }
    if (need == 0) return Tensor();
    return at::empty({static_cast<int64_t>(need)}, ref.options().dtype(at::kByte));
}
void* data(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
size_t bytes(const Tensor& t) { return t.defined() ? t.nbytes() : 0; }

// What a call wrote into a tensor of the caller's counts as a change of it, so that autograd refuses to use a
// saved one unseen. (Inference tensors have no version.)
void wrote(PyObject* given, const Tensor& t) {
    if (THPVariable_Check(given) && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

PyObject* wrap(const Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject* tuple(std::initializer_list<Tensor> ts) {
    PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (!r) throw python_error();
    Py_ssize_t i = 0;
    for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
    return r;
}

struct LinArgs {
    const Tensor *q, *k, *v, *log_decay, *cu;
    m3_linattn_dims d;
    m3_linattn_inputs in;
};

// q [b, L, Hq, K], k [b, L, Hk, K], v [b, L, Hv, V] (a step: without L), log_decay [H]
LinArgs lin_args(PyObject* const* a, PyObject* scale, PyObject* cu, int64_t nd) {
    LinArgs r{};
    r.q = &tensor(a[0], "q");
    r.k = &tensor(a[1], "k");
    r.v = &tensor(a[2], "v");
    r.log_decay = &tensor(a[3], "log_decay");
    r.cu = maybe(cu, "cu_seqlens");
    const Tensor &q = *r.q, &k = *r.k, &v = *r.v;
    TORCH_CHECK_VALUE(q.is_cuda(), "tensors must be on a CUDA device");
    same_device(q, &k, "k");
    same_device(q, &v, "v");
    same_device(q, r.log_decay, "log_decay");
    same_device(q, r.cu, "cu_seqlens");
    TORCH_CHECK_VALUE(q.dim() == nd && k.dim() == nd && v.dim() == nd, "q, k and v must have ", nd, " dimensions");
    TORCH_CHECK_VALUE(r.log_decay->dim() == 1, "log_decay must be a vector of one value per head");
    const int64_t b = q.size(0), L = nd == 4 ? q.size(1) : 1, K = q.size(nd - 1), V = v.size(nd - 1);
    const int64_t H = r.log_decay->size(0);
    m3_linattn_dims& d = r.d;
    d.nseq = b;
    d.seqlen = L;
    d.nheads = H;
    d.qheads = q.size(nd - 2);
    d.kheads = k.size(nd - 2);
    d.vheads = v.size(nd - 2);
    d.kdim = K;
    d.vdim = V;
    d.in_dtype = dtype_code(q);
    d.scale = static_cast<float>(number(scale));
    const auto type = q.scalar_type();
    const int64_t qs[4] = {b, L, d.qheads, K}, ks[4] = {b, L, d.kheads, K}, vs[4] = {b, L, d.vheads, V};
    const int64_t q3[3] = {b, d.qheads, K}, k3[3] = {b, d.kheads, K}, v3[3] = {b, d.vheads, V};
    const auto shape = [&](const int64_t* four, const int64_t* three) {
        return nd == 4 ? at::IntArrayRef(four, 4) : at::IntArrayRef(three, 3);
    };
    r.in.q = view(q, "q", shape(qs, q3), type);
    r.in.k = view(k, "k", shape(ks, k3), type);
    r.in.v = view(v, "v", shape(vs, v3), type);
    r.in.log_decay = f32(r.log_decay, "log_decay", {H});
    r.in.cu_seqlens = i32(r.cu, "cu_seqlens", -1);
    if (r.cu) {
        TORCH_CHECK_VALUE(b == 1, "packed sequences lie in tensors of batch 1");
        d.nseq = r.cu->size(0) - 1;
        TORCH_CHECK_VALUE(d.nseq >= 0, "cu_seqlens needs at least one value");
    }
    return r;
}

// (q, k, v, log_decay, scale, init, final, o, cu_seqlens, workspace) -> (o, final) or a status
PyObject* linattn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 10, "linattn_fwd takes 10 arguments");
    const LinArgs r = lin_args(a, a[4], a[8], 4);
    const Tensor& q = *r.q;
    const m3_linattn_dims& d = r.d;
    const c10::cuda::CUDAGuard guard(q.device());
    const Tensor* init = maybe(a[5], "init");
    Tensor fin, o;
    const int64_t states[4] = {d.nseq, d.nheads, d.kdim, d.vdim}, shape[4] = {q.size(0), q.size(1), d.nheads, d.vdim};
    if (a[6] == Py_True) fin = at::empty(states, q.options().dtype(at::kFloat));
    else if (a[6] != Py_None && a[6] != Py_False) fin = tensor(a[6], "final");
    if (a[7] != Py_None) o = tensor(a[7], "o");
    else o = r.cu ? at::zeros(shape, q.options()) : at::empty(shape, q.options());
    same_device(q, init, "init");
    same_device(q, fin.defined() ? &fin : nullptr, "final");
    same_device(q, &o, "o");
    const m3_view ov = out_view(o, "o", shape, q.scalar_type());
    const Tensor ws = workspace(maybe(a[9], "workspace"), api.linattn_workspace(&d, r.cu != nullptr), q);
    const int rc = api.linattn_fwd(&d, &r.in, f32(init, "init", states), f32(fin.defined() ? &fin : nullptr, "final", states),
                                   &ov, data(ws), bytes(ws), stream_of(q));
    if (rc != M3_OK) return PyLong_FromLong(rc);
    wrote(a[7], o);
    wrote(a[6], fin);
    return tuple({o, fin});
    END_HANDLE_TH_ERRORS
}

// (q, k, v, log_decay, scale, state, state_out, slots, o) -> (o, state_out) or a status
PyObject* linattn_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 9, "linattn_step takes 9 arguments");
    const LinArgs r = lin_args(a, a[4], Py_None, 3);
    const Tensor& q = *r.q;
    const m3_linattn_dims& d = r.d;
    const c10::cuda::CUDAGuard guard(q.device());
    const Tensor& state = tensor(a[5], "state");
    const Tensor& out = a[6] == Py_None ? state : tensor(a[6], "state_out");
    const Tensor* slots = maybe(a[7], "slots");
    same_device(q, &state, "state");
    same_device(q, &out, "state_out");
    same_device(q, slots, "slots");
    TORCH_CHECK_VALUE(state.dim() == 4, "state must have 4 dimensions");
    const int64_t states[4] = {slots ? state.size(0) : d.nseq, d.nheads, d.kdim, d.vdim}, shape[3] = {d.nseq, d.nheads, d.vdim};
    const Tensor o = a[8] != Py_None ? tensor(a[8], "o") : at::empty(shape, q.options());
    same_device(q, &o, "o");
    const m3_view ov = out_view(o, "o", shape, q.scalar_type());
    const int rc = api.linattn_step(&d, &r.in, f32(&state, "state", states), f32(&out, "state_out", states), states[0],
                                    i32(slots, "slots", d.nseq), &ov, stream_of(q));
    if (rc != M3_OK) return PyLong_FromLong(rc);
    wrote(a[8], o);
    wrote(a[6] == Py_None ? a[5] : a[6], out);
    return tuple({o, out});
    END_HANDLE_TH_ERRORS
}

// (q, k, v, log_decay, scale, do, init, dfinal, cu_seqlens, dq, dk, dv, want_init, workspace)
// -> (dq, dk, dv, dinit) or a status; dq, dk and dv are all None or all tensors
PyObject* linattn_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 14, "linattn_bwd takes 14 arguments");
    const LinArgs r = lin_args(a, a[4], a[8], 4);
    const Tensor& q = *r.q;
    const m3_linattn_dims& d = r.d;
    const c10::cuda::CUDAGuard guard(q.device());
    const Tensor& dout = tensor(a[5], "do");
    const Tensor *init = maybe(a[6], "init"), *dfinal = maybe(a[7], "dfinal");
    const Tensor* ins[3] = {r.q, r.k, r.v};
    const char* names[3] = {"dq", "dk", "dv"};
    Tensor g[3], dinit;
    m3_view gv[3];
    for (int i = 0; i < 3; ++i) {
        if (a[9 + i] != Py_None) g[i] = tensor(a[9 + i], names[i]);
        else g[i] = r.cu ? at::zeros(ins[i]->sizes(), q.options()) : at::empty(ins[i]->sizes(), q.options());
        same_device(q, &g[i], names[i]);
        gv[i] = out_view(g[i], names[i], ins[i]->sizes(), q.scalar_type());
    }
    const int64_t states[4] = {d.nseq, d.nheads, d.kdim, d.vdim}, shape[4] = {q.size(0), q.size(1), d.nheads, d.vdim};
    if (a[12] == Py_True) dinit = at::empty(states, q.options().dtype(at::kFloat));
    else if (a[12] != Py_None && a[12] != Py_False) dinit = tensor(a[12], "want_init");
    same_device(q, &dout, "do");
    same_device(q, init, "init");
    same_device(q, dfinal, "dfinal");
    same_device(q, dinit.defined() ? &dinit : nullptr, "want_init");
    const m3_view dv = view(dout, "do", shape, q.scalar_type());
    const m3_linattn_grads gc{gv[0], gv[1], gv[2]};
    const Tensor ws = workspace(maybe(a[13], "workspace"), api.linattn_bwd_workspace(&d, r.cu != nullptr), q);
    const int rc = api.linattn_bwd(&d, &r.in, f32(init, "init", states), &dv, f32(dfinal, "dfinal", states), &gc,
                                   f32(dinit.defined() ? &dinit : nullptr, "dinit", states), data(ws), bytes(ws), stream_of(q));
    if (rc != M3_OK) return PyLong_FromLong(rc);
    for (int i = 0; i < 3; ++i) wrote(a[9 + i], g[i]);
    wrote(a[12], dinit);
    return tuple({g[0], g[1], g[2], dinit});
    END_HANDLE_TH_ERRORS
}

// ---- grouped norm

// The stride at which the elements of dimensions [lo, hi) lie; false if there is no such.
bool one_stride(const Tensor& t, int64_t lo, int64_t hi, int64_t* step) {
    *step = 0;
    bool any = false;
    int64_t span = 0;
    for (int64_t i = hi - 1; i >= lo; --i) {
        if (t.size(i) == 1) continue;
        if (!any) {
            any = true;
            *step = t.stride(i);
            span = t.stride(i) * t.size(i);
        } else if (t.stride(i) != span) {
            return false;
        } else {
            span *= t.size(i);
        }
    }
    return true;
}

// (batch, rows) and the views of tensors [..., C] of the first one's shape and of the given types: their
// leading dimensions cut where each part of every tensor's lies at one stride. Absent tensors are skipped.
template <int N>
void row_views(const Tensor* const (&ts)[N], const char* const (&names)[N], const at::ScalarType (&types)[N], int64_t D,
               int64_t* batch, int64_t* rows, m3_view (&vs)[N]) {
    const Tensor& x = *ts[0];
    const int64_t lead = x.dim() - 1, C = x.size(lead);
    bool plain = true;
    for (int i = 0; i < N; ++i) {
        if (!ts[i]) continue;
        const Tensor& t = *ts[i];
        same_device(x, &t, names[i]);
        TORCH_CHECK_VALUE(t.sizes() == x.sizes(), names[i], " has shape ", t.sizes(), ", expected ", x.sizes());
        TORCH_CHECK_VALUE(t.scalar_type() == types[i], names[i], " is ", t.scalar_type(), ", expected ", types[i]);
        TORCH_CHECK_VALUE(t.stride(lead) == 1 || C == 1, names[i], ": the channels must be contiguous");
        plain = plain && t.is_contiguous();
    }
    for (int64_t cut = 0; cut <= lead; ++cut) {
        bool ok = true;
        for (int i = 0; i < N && ok; ++i) {
            vs[i] = m3_view{};
            if (!ts[i]) continue;
            int64_t outer = 0, inner = C;
            if (!plain) ok = one_stride(*ts[i], 0, cut, &outer) && one_stride(*ts[i], cut, lead, &inner);
            vs[i] = m3_view{ts[i]->data_ptr(), outer, inner, D};
        }
        if (!ok) continue;
        *batch = *rows = 1;
        for (int64_t i = 0; i < lead; ++i) *(i < cut ? batch : rows) *= x.size(i);
        return;
    }
    TORCH_CHECK_VALUE(false, "rows must lie at one stride, or at one in every batch entry");
}

// the same for tensors of the first one's type
template <int N>
void gn_views(m3_group_norm_dims& d, const Tensor* const (&ts)[N], const char* const (&names)[N], m3_view (&vs)[N]) {
    const Tensor& x = *ts[0];
    TORCH_CHECK_VALUE(x.is_cuda(), "tensors must be on a CUDA device");
    TORCH_CHECK_VALUE(x.dim() >= 1 && x.size(-1) >= 1, "x needs a last dimension of channels");
    d.channels = x.size(-1);
    d.in_dtype = dtype_code(x);
    at::ScalarType types[N];
    for (at::ScalarType& t : types) t = x.scalar_type();
    row_views<N>(ts, names, types, d.groups > 0 ? d.channels / d.groups : d.channels, &d.batch, &d.rows, vs);
}

m3_group_norm_dims gn_dims(PyObject* groups, PyObject* center, PyObject* silu, PyObject* eps) {
    m3_group_norm_dims d{};
    d.groups = integer(groups);
    d.eps = static_cast<float>(number(eps));
    d.flags = (truth(center) ? M3_GN_CENTER : 0u) | (truth(silu) ? M3_GN_SILU : 0u);
    return d;
}

// (x, groups, weight, bias, z, center, silu, eps, out) -> out or a status
PyObject* group_norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 9, "group_norm_fwd takes 9 arguments");
    const Tensor& x = tensor(a[0], "x");
    const Tensor *w = maybe(a[2], "weight"), *b = maybe(a[3], "bias"), *z = maybe(a[4], "z");
    TORCH_CHECK_VALUE(x.is_cuda(), "tensors must be on a CUDA device");
    const c10::cuda::CUDAGuard guard(x.device());
    const Tensor out = a[8] != Py_None ? tensor(a[8], "out") : at::empty(x.sizes(), x.options());
    m3_group_norm_dims d = gn_dims(a[1], a[5], a[6], a[7]);
    m3_view v[3];
    gn_views<3>(d, {&x, z, &out}, {"x", "z", "out"}, v);
    same_device(x, w, "weight");
    same_device(x, b, "bias");
    const int rc = api.group_norm_fwd(&d, &v[0], &v[1], f32(w, "weight", {d.channels}), f32(b, "bias", {d.channels}), &v[2],
                                      stream_of(x));
    if (rc != M3_OK) return PyLong_FromLong(rc);
    wrote(a[8], out);
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

// (dout, x, groups, weight, bias, z, center, silu, eps, dx, dz, workspace) -> (dx, dz, dweight, dbias)
PyObject* group_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 12, "group_norm_bwd takes 12 arguments");
    const Tensor &dout = tensor(a[0], "dout"), &x = tensor(a[1], "x");
    const Tensor *w = maybe(a[3], "weight"), *b = maybe(a[4], "bias"), *z = maybe(a[5], "z");
    TORCH_CHECK_VALUE(x.is_cuda(), "tensors must be on a CUDA device");
    const c10::cuda::CUDAGuard guard(x.device());
    const Tensor dx = a[9] != Py_None ? tensor(a[9], "dx") : at::empty(x.sizes(), x.options());
    Tensor dz, dw, db;
    if (z) dz = a[10] != Py_None ? tensor(a[10], "dz") : at::empty(x.sizes(), x.options());
    m3_group_norm_dims d = gn_dims(a[2], a[6], a[7], a[8]);
    m3_view v[5];
    gn_views<5>(d, {&x, z, &dout, &dx, z ? &dz : nullptr}, {"x", "z", "dout", "dx", "dz"}, v);
    same_device(x, w, "weight");
    same_device(x, b, "bias");
    const float *wp = f32(w, "weight", {d.channels}), *bp = f32(b, "bias", {d.channels});
    if (w) dw = at::empty({d.channels}, w->options());
    if (b) db = at::empty({d.channels}, b->options());
    const Tensor ws = workspace(maybe(a[11], "workspace"), api.group_norm_bwd_workspace(&d), x);
    const int rc = api.group_norm_bwd(&d, &v[0], &v[1], wp, bp, &v[2], &v[3], &v[4],
                                      static_cast<float*>(data(dw)), static_cast<float*>(data(db)), data(ws), bytes(ws),
                                      stream_of(x));
    if (rc != M3_OK) return PyLong_FromLong(rc);
    wrote(a[9], dx);
    if (z) wrote(a[10], dz);
    return tuple({dx, dz, dw, db});
    END_HANDLE_TH_ERRORS
}

// ---- gated scan

// a tensor [b, L, C], or a step's [b, C], by its strides
m3_view rows_view(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, bool written = false) {
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", t.sizes(), ", expected ", shape);
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " is ", t.scalar_type(), ", expected ", type);
    const int64_t n = t.dim();
    TORCH_CHECK_VALUE(t.stride(n - 1) == 1 || shape[n - 1] <= 1, name, ": the channels must be contiguous");
    for (int64_t i = 0; written && i < n; ++i)
        TORCH_CHECK_VALUE(t.stride(i) != 0 || shape[i] <= 1, name, " is written and must not be expanded");
    return m3_view{t.data_ptr(), t.stride(0), n == 3 ? t.stride(1) : 0, 0};
}

struct ScanArgs {
    const Tensor *x, *r, *i, *decay, *cu;
    m3_gated_scan_dims d;
    m3_gated_scan_inputs in;
};

// x, r, i (or None), decay (or None), power, lerp
ScanArgs scan_args(PyObject* const* a, PyObject* cu, int64_t nd) {
    ScanArgs s{};
    s.x = &tensor(a[0], "x");
    s.r = &tensor(a[1], "r");
    s.i = maybe(a[2], "i");
    s.decay = maybe(a[3], "decay");
    s.cu = maybe(cu, "cu_seqlens");
    const Tensor& x = *s.x;
    TORCH_CHECK_VALUE(x.is_cuda(), "tensors must be on a CUDA device");
    TORCH_CHECK_VALUE(x.dim() == nd, "x must have ", nd, " dimensions");
    same_device(x, s.r, "r");
    same_device(x, s.i, "i");
    same_device(x, s.decay, "decay");
    same_device(x, s.cu, "cu_seqlens");
    m3_gated_scan_dims& d = s.d;
    d.nseq = x.size(0);
    d.seqlen = nd == 3 ? x.size(1) : 1;
    d.channels = x.size(nd - 1);
    d.in_dtype = dtype_code(x);
    d.power = static_cast<float>(number(a[4]));
    d.flags = truth(a[5]) ? M3_GS_LERP : 0u;
    const auto type = x.scalar_type();
    s.in.x = rows_view(x, "x", x.sizes(), type);
    s.in.r = rows_view(*s.r, "r", x.sizes(), type);
    if (s.i) s.in.i = rows_view(*s.i, "i", x.sizes(), type);
    s.in.decay = f32(s.decay, "decay", {d.channels});
    TORCH_CHECK_VALUE(s.decay || (d.flags & M3_GS_LERP), "decay is needed without lerp");
    s.in.cu_seqlens = i32(s.cu, "cu_seqlens", -1);
    if (s.cu) {
        TORCH_CHECK_VALUE(d.nseq == 1, "packed sequences lie in tensors of batch 1");
        d.nseq = s.cu->size(0) - 1;
        TORCH_CHECK_VALUE(d.nseq >= 0, "cu_seqlens needs at least one value");
    }
    return s;
}

// True: a new tensor of that shape; None or False: none; else the caller's
Tensor wanted(PyObject* o, const char* name, const Tensor& ref, at::IntArrayRef shape) {
    Tensor t;
    if (o == Py_True) t = at::empty(shape, ref.options().dtype(at::kFloat));
    else if (o != Py_None && o != Py_False) t = tensor(o, name);
    if (t.defined()) same_device(ref, &t, name);
    return t;
}
float* f32(const Tensor& t, const char* name, at::IntArrayRef shape) { return f32(t.defined() ? &t : nullptr, name, shape); }

// the caller's output or a new one (packed: rows of no sequence are zero)
Tensor output(PyObject* o, const char* name, const Tensor& like, bool packed) {
    if (o != Py_None) {
        const Tensor& t = tensor(o, name);
        same_device(like, &t, name);
        return t;
    }
    return packed ? at::zeros(like.sizes(), like.options()) : at::empty(like.sizes(), like.options());
}

// (x, r, i, decay, power, lerp, init, final, y, cu_seqlens, marks) -> (y, final, marks) or a status
PyObject* gated_scan_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 11, "gated_scan_fwd takes 11 arguments");
    const ScanArgs s = scan_args(a, a[9], 3);
    const Tensor& x = *s.x;
    const m3_gated_scan_dims& d = s.d;
    const c10::cuda::CUDAGuard guard(x.device());
    const Tensor* init = maybe(a[6], "init");
    same_device(x, init, "init");
    const int64_t states[2] = {d.nseq, d.channels};
    const int64_t blocks[3] = {s.cu ? 1 : d.nseq, (d.seqlen + M3_GS_BLOCK - 1) / M3_GS_BLOCK, d.channels};
    const Tensor fin = wanted(a[7], "final", x, states), marks = wanted(a[10], "marks", x, blocks);
    const Tensor y = output(a[8], "y", x, s.cu != nullptr);
    const m3_view yv = rows_view(y, "y", x.sizes(), x.scalar_type(), true);
    const int rc = api.gated_scan_fwd(&d, &s.in, f32(init, "init", states), f32(fin, "final", states), &yv,
                                      f32(marks, "marks", blocks), stream_of(x));
    if (rc != M3_OK) return PyLong_FromLong(rc);
    wrote(a[8], y);
    wrote(a[7], fin);
    wrote(a[10], marks);
    return tuple({y, fin, marks});
    END_HANDLE_TH_ERRORS
}

// (x, r, i, decay, power, lerp, state, state_out, slots, y) -> (y, state_out) or a status
PyObject* gated_scan_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 10, "gated_scan_step takes 10 arguments");
    const ScanArgs s = scan_args(a, Py_None, 2);
    const Tensor& x = *s.x;
    const m3_gated_scan_dims& d = s.d;
    const c10::cuda::CUDAGuard guard(x.device());
    const Tensor& state = tensor(a[6], "state");
    const Tensor& out = a[7] == Py_None ? state : tensor(a[7], "state_out");
    const Tensor* slots = maybe(a[8], "slots");
    same_device(x, &state, "state");
    same_device(x, &out, "state_out");
    same_device(x, slots, "slots");
    TORCH_CHECK_VALUE(state.dim() == 2, "state must have 2 dimensions");
    const int64_t states[2] = {slots ? state.size(0) : d.nseq, d.channels};
    const Tensor y = output(a[9], "y", x, false);
    const m3_view yv = rows_view(y, "y", x.sizes(), x.scalar_type(), true);
    const int rc = api.gated_scan_step(&d, &s.in, f32(&state, "state", states), f32(&out, "state_out", states), states[0],
                                       i32(slots, "slots", d.nseq), &yv, stream_of(x));
    if (rc != M3_OK) return PyLong_FromLong(rc);
    wrote(a[9], y);
    wrote(a[7] == Py_None ? a[6] : a[7], out);
    return tuple({y, out});
    END_HANDLE_TH_ERRORS
}

// (x, r, i, decay, power, lerp, dy, init, dfinal, cu_seqlens, marks, dx, dr, di, want_init, workspace)
// -> (dx, dr, di, ddecay, dinit) or a status
PyObject* gated_scan_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 16, "gated_scan_bwd takes 16 arguments");
    const ScanArgs s = scan_args(a, a[9], 3);
    const Tensor& x = *s.x;
    const m3_gated_scan_dims& d = s.d;
    const c10::cuda::CUDAGuard guard(x.device());
    const Tensor& dy = tensor(a[6], "dy");
    const Tensor *init = maybe(a[7], "init"), *dfinal = maybe(a[8], "dfinal"), *marks = maybe(a[10], "marks");
    same_device(x, &dy, "dy");
    same_device(x, init, "init");
    same_device(x, dfinal, "dfinal");
    same_device(x, marks, "marks");
    const int64_t states[2] = {d.nseq, d.channels};
    const int64_t blocks[3] = {s.cu ? 1 : d.nseq, (d.seqlen + M3_GS_BLOCK - 1) / M3_GS_BLOCK, d.channels};
    const bool packed = s.cu != nullptr;
    const Tensor dx = output(a[11], "dx", x, packed), dr = output(a[12], "dr", x, packed);
    Tensor di, dd;
    if (s.i) di = output(a[13], "di", x, packed);
    if (s.decay) dd = at::empty({d.channels}, s.decay->options());
    const Tensor dinit = wanted(a[14], "want_init", x, states);
    const auto type = x.scalar_type();
    const m3_view dyv = rows_view(dy, "dy", x.sizes(), type);
    m3_gated_scan_grads g{};
    g.dx = rows_view(dx, "dx", x.sizes(), type, true);
    g.dr = rows_view(dr, "dr", x.sizes(), type, true);
    if (s.i) g.di = rows_view(di, "di", x.sizes(), type, true);
    const Tensor ws = workspace(maybe(a[15], "workspace"), api.gated_scan_bwd_workspace(&d, packed, marks != nullptr), x);
    const int rc = api.gated_scan_bwd(&d, &s.in, f32(init, "init", states), f32(marks, "marks", blocks), &dyv,
                                      f32(dfinal, "dfinal", states), &g, static_cast<float*>(data(dd)),
                                      f32(dinit, "dinit", states), data(ws), bytes(ws), stream_of(x));
    if (rc != M3_OK) return PyLong_FromLong(rc);
    wrote(a[11], dx);
    wrote(a[12], dr);
    if (s.i) wrote(a[13], di);
    wrote(a[14], dinit);
    return tuple({dx, dr, di, dd, dinit});
    END_HANDLE_TH_ERRORS
}

// ---- rotary positions

// (q, k, freq, positions, offset, cu_seqlens, interleaved, inverse, scale, q_out, k_out) -> (q_out, k_out) or a status
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 11, "rotary takes 11 arguments");
    const Tensor& q = tensor(a[0], "q");
    const Tensor* k = maybe(a[1], "k");
    const Tensor& freq = tensor(a[2], "freq");
    const Tensor *pos = maybe(a[3], "positions"), *cu = maybe(a[5], "cu_seqlens");
    TORCH_CHECK_VALUE(q.is_cuda(), "tensors must be on a CUDA device");
    const c10::cuda::CUDAGuard guard(q.device());
    const int64_t nd = q.dim();
    TORCH_CHECK_VALUE(nd == 3 || nd == 4, "q must have 3 or 4 dimensions");
    TORCH_CHECK_VALUE(!k || k->dim() == nd, "k must have q's dimensions");
    same_device(q, k, "k");
    same_device(q, &freq, "freq");
    same_device(q, pos, "positions");
    same_device(q, cu, "cu_seqlens");
    const int64_t b = q.size(0), L = nd == 4 ? q.size(1) : 1;
    m3_rotary_dims d{};
    d.nseq = b;
    d.seqlen = L;
    d.qheads = q.size(nd - 2);
    d.kheads = k ? k->size(nd - 2) : 0;
    d.headdim = q.size(nd - 1);
    d.offset = integer(a[4]);
    d.in_dtype = dtype_code(q);
    d.scale = static_cast<float>(number(a[8]));
    d.flags = (truth(a[6]) ? M3_ROT_INTERLEAVED : 0u) | (truth(a[7]) ? M3_ROT_INVERSE : 0u);
    TORCH_CHECK_VALUE(freq.dim() == 1 && freq.scalar_type() == at::kDouble && freq.is_contiguous(),
                      "freq must be a contiguous float64 vector");
    d.rotdim = 2 * freq.size(0);
    if (cu) {
        TORCH_CHECK_VALUE(nd == 4 && b == 1, "packed sequences lie in tensors [1, rows, heads, dim]");
        TORCH_CHECK_VALUE(cu->dim() == 1 && cu->size(0) >= 1, "cu_seqlens needs at least one value");
        d.nseq = cu->size(0) - 1;
    }
    int64_t pb = 0, pt = 0;
    if (pos) {
        const bool wide = pos->scalar_type() == at::kLong;
        TORCH_CHECK_VALUE(wide || pos->scalar_type() == at::kInt, "positions must be int32 or int64");
        if (wide) d.flags |= M3_ROT_POS64;
        if (nd == 3) {
            TORCH_CHECK_VALUE(pos->dim() == 1 && pos->size(0) == b, "positions has shape ", pos->sizes(), ", expected [", b, "]");
            pb = pos->stride(0);
        } else if (pos->dim() == 1) {
            TORCH_CHECK_VALUE(pos->size(0) == L, "positions has shape ", pos->sizes(), ", expected [", L, "] or [", b, ", ", L, "]");
            pt = pos->stride(0);
        } else {
            TORCH_CHECK_VALUE(pos->dim() == 2 && pos->size(0) == b && pos->size(1) == L, "positions has shape ", pos->sizes(),
                              ", expected [", L, "] or [", b, ", ", L, "]");
            pb = pos->stride(0);
            pt = pos->stride(1);
        }
    }
    const Tensor qo = output(a[9], "q_out", q, cu != nullptr);
    Tensor ko;
    if (k) ko = output(a[10], "k_out", *k, cu != nullptr);
    const auto type = q.scalar_type();
    const m3_view qv = view(q, "q", q.sizes(), type), qov = out_view(qo, "q_out", q.sizes(), type);
    m3_view kv{}, kov{};
    if (k) {
        const int64_t s4[4] = {b, L, d.kheads, d.headdim}, s3[3] = {b, d.kheads, d.headdim};
        const at::IntArrayRef shape = nd == 4 ? at::IntArrayRef(s4, 4) : at::IntArrayRef(s3, 3);
        kv = view(*k, "k", shape, type);
        kov = out_view(ko, "k_out", shape, type);
    }
    const int rc = api.rotary(&d, &qv, &kv, static_cast<const double*>(freq.data_ptr()), pos ? pos->data_ptr() : nullptr, pb, pt,
                              i32(cu, "cu_seqlens", -1), &qov, &kov, stream_of(q));
    if (rc != M3_OK) return PyLong_FromLong(rc);
    wrote(a[9], qo);
    if (k) wrote(a[10], ko);
    return tuple({qo, ko});
    END_HANDLE_TH_ERRORS
}

// ---- block norm

struct BlockArgs {
    const Tensor *y, *x, *z;
    m3_block_norm_dims d;
    m3_block_norm_inputs in;
};

// (y, residual, z, post_weight, post_bias, pre_weight, pre_bias, alpha, eps, flags)
BlockArgs block_args(PyObject* const* a) {
    BlockArgs s{};
    s.y = &tensor(a[0], "y");
    s.x = &tensor(a[1], "residual");
    s.z = maybe(a[2], "z");
    const Tensor& y = *s.y;
    TORCH_CHECK_VALUE(y.is_cuda(), "tensors must be on a CUDA device");
    TORCH_CHECK_VALUE(y.dim() >= 1 && y.size(-1) >= 1, "y needs a last dimension of channels");
    m3_block_norm_dims& d = s.d;
    d.channels = y.size(-1);
    d.in_dtype = dtype_code(y);
    d.res_dtype = dtype_code(*s.x);
    d.alpha = static_cast<float>(number(a[7]));
    d.eps = static_cast<float>(number(a[8]));
    d.flags = static_cast<uint32_t>(integer(a[9]));
    const char* const names[4] = {"post_weight", "post_bias", "pre_weight", "pre_bias"};
    const float** const to[4] = {&s.in.post_weight, &s.in.post_bias, &s.in.pre_weight, &s.in.pre_bias};
    for (int i = 0; i < 4; ++i) {
        const Tensor* t = maybe(a[3 + i], names[i]);
        same_device(y, t, names[i]);
        *to[i] = f32(t, names[i], {d.channels});
    }
    return s;
}

// (block_args ..., h, out) -> (h, out) or a status
PyObject* block_norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 12, "block_norm_fwd takes 12 arguments");
    BlockArgs s = block_args(a);
    const Tensor &y = *s.y, &x = *s.x;
    const c10::cuda::CUDAGuard guard(y.device());
    const bool pre = s.d.flags & (M3_BN_PRE_RMS | M3_BN_PRE_LAYER);
    same_device(y, &x, "residual");
    const Tensor h = a[10] != Py_None ? tensor(a[10], "h") : at::empty(y.sizes(), x.options());
    Tensor out;
    if (pre) out = a[11] != Py_None ? tensor(a[11], "out") : at::empty(y.sizes(), y.options());
    const auto ty = y.scalar_type(), tx = x.scalar_type();
    m3_view v[5];
    row_views<5>({&y, &x, s.z, &h, pre ? &out : nullptr}, {"y", "residual", "z", "h", "out"}, {ty, tx, ty, tx, ty}, 0,
                 &s.d.batch, &s.d.rows, v);
    s.in.y = v[0];
    s.in.residual = v[1];
    s.in.z = v[2];
    const int rc = api.block_norm_fwd(&s.d, &s.in, &v[3], &v[4], stream_of(y));
    if (rc != M3_OK) return PyLong_FromLong(rc);
    wrote(a[10], h);
    if (pre) wrote(a[11], out);
    return tuple({h, out});
    END_HANDLE_TH_ERRORS
}

// (block_args ..., dh, dout, dy, dresidual, dz, workspace)
// -> (dy, dresidual, dz, dpost_weight, dpost_bias, dpre_weight, dpre_bias) or a status
PyObject* block_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == 16, "block_norm_bwd takes 16 arguments");
    BlockArgs s = block_args(a);
    const Tensor &y = *s.y, &x = *s.x;
    const c10::cuda::CUDAGuard guard(y.device());
    const bool pre = s.d.flags & (M3_BN_PRE_RMS | M3_BN_PRE_LAYER);
    same_device(y, &x, "residual");
    const Tensor *dh = maybe(a[10], "dh"), *dout = maybe(a[11], "dout");
    TORCH_CHECK_VALUE(!pre == !dout, pre ? "dout is needed with a pre norm" : "dout without a pre norm");
    const Tensor dy = a[12] != Py_None ? tensor(a[12], "dy") : at::empty(y.sizes(), y.options());
    const Tensor dx = a[13] != Py_None ? tensor(a[13], "dresidual") : at::empty(y.sizes(), x.options());
    Tensor dz, sums[4];
    if (s.z) dz = a[14] != Py_None ? tensor(a[14], "dz") : at::empty(y.sizes(), y.options());
    const auto ty = y.scalar_type(), tx = x.scalar_type();
    m3_view v[8];
    row_views<8>({&y, &x, s.z, dh, dout, &dy, &dx, s.z ? &dz : nullptr},
                 {"y", "residual", "z", "dh", "dout", "dy", "dresidual", "dz"}, {ty, tx, ty, tx, ty, ty, tx, ty}, 0,
                 &s.d.batch, &s.d.rows, v);
    s.in.y = v[0];
    s.in.residual = v[1];
    s.in.z = v[2];
    m3_block_norm_grads g{};
    g.dy = v[5];
    g.dresidual = v[6];
    g.dz = v[7];
    float** const to[4] = {&g.dpost_weight, &g.dpost_bias, &g.dpre_weight, &g.dpre_bias};
    for (int i = 0; i < 4; ++i)
        if (a[3 + i] != Py_None) {
            sums[i] = at::empty({s.d.channels}, y.options().dtype(at::kFloat));
            *to[i] = static_cast<float*>(sums[i].data_ptr());
        }
    const Tensor ws = workspace(maybe(a[15], "workspace"), api.block_norm_bwd_workspace(&s.d), y);
    const int rc = api.block_norm_bwd(&s.d, &s.in, &v[3], &v[4], &g, data(ws), bytes(ws), stream_of(y));
    if (rc != M3_OK) return PyLong_FromLong(rc);
    wrote(a[12], dy);
    wrote(a[13], dx);
    if (s.z) wrote(a[14], dz);
    return tuple({dy, dx, dz, sums[0], sums[1], sums[2], sums[3]});
    END_HANDLE_TH_ERRORS
}

// bind(addresses of the entry points, in Api's order)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    constexpr Py_ssize_t kCount = sizeof(Api) / sizeof(void*);
    TORCH_CHECK_TYPE(n == kCount, "bind takes ", kCount, " addresses");
    void** slot = reinterpret_cast<void**>(&api);
    for (Py_ssize_t i = 0; i < n; ++i) slot[i] = reinterpret_cast<void*>(integer(a[i]));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<bind>("bind"), method<linattn_fwd>("linattn_fwd"),
                         method<linattn_step>("linattn_step"), method<linattn_bwd>("linattn_bwd"),
                         method<group_norm_fwd>("group_norm_fwd"), method<group_norm_bwd>("group_norm_bwd"),
                         method<gated_scan_fwd>("gated_scan_fwd"), method<gated_scan_step>("gated_scan_step"),
                         method<gated_scan_bwd>("gated_scan_bwd"), method<rotary>("rotary"),
                         method<block_norm_fwd>("block_norm_fwd"), method<block_norm_bwd>("block_norm_bwd"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_m3torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__m3torch(void) {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", M3_BUILT_FOR) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
