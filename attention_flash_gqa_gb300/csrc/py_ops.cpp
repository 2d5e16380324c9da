// Python entry of the calls that are short on the GPU (step plan, head norm, tree attention): argument
// checks, output allocation and the call of the C ABI in native code. In Python the same took longer than
// the kernels: per call 10 to 22 us of interpreter time beside 4 to 9 us for the launches themselves.
//
// The functions take every argument by position; the documented signatures are in __init__.py. Tensors
// come and go as torch tensors; nothing of the computation happens here.
#include <Python.h>
#include <dlfcn.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "../../include/attn.h"

namespace {

// The library's functions, looked up once by load().
struct Api {
    decltype(&attn_paged_plan) paged_plan = nullptr;
    decltype(&attn_qk_norm_rope) norm_rope = nullptr;
    decltype(&attn_qk_norm_rope_bwd) norm_rope_bwd = nullptr;
    decltype(&attn_qk_norm_rope_paged) norm_rope_paged = nullptr;
    decltype(&attn_tree_paged) tree_paged = nullptr;
    decltype(&attn_workspace_size) workspace_size = nullptr;
};
Api g_api;
PyObject* g_error = nullptr;  // AttnError
PyObject* g_plan = nullptr;   // PagedPlan

struct Raised {};  // a Python error is set

[[noreturn]] void refuse(const char* format, const char* name) {
    PyErr_Format(PyExc_ValueError, format, name);
    throw Raised();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        throw Raised();
    }
    return THPVariable_Unpack(o);
}

// Device index of a CUDA tensor.
int index_of(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
    return t.get_device();
}

// A contiguous tensor of that type and shape on GPU idx.
template <class T>
T* checked(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, int idx, const char* name) {
    if (t.scalar_type() == type && t.is_cuda() && t.get_device() == idx && t.sizes() == shape && t.is_contiguous())
        return static_cast<T*>(t.data_ptr());
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous %s tensor of %d dimensions on cuda:%d with the call's sizes", name,
                 type == at::kInt ? "int32" : type == at::kFloat ? "float32" : "bfloat16", (int)shape.size(), idx);
    throw Raised();
}
int32_t* i32(PyObject* o, at::IntArrayRef shape, int idx, const char* name) {
    return checked<int32_t>(tensor(o, name), at::kInt, shape, idx, name);
}
attn_bf16* bf16(const at::Tensor& t, at::IntArrayRef shape, int idx, const char* name) {
    return checked<attn_bf16>(t, at::kBFloat16, shape, idx, name);
}

int as_int(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    if (v < INT32_MIN || v > INT32_MAX) refuse("%s is out of range", name);
    return (int)v;
}
float as_float(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return (float)v;
}
bool as_bool(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised();
    return v != 0;
}

// The device and stream that the call runs on, current for its duration: a torch stream object, or None.
struct Place {
    c10::cuda::OptionalCUDAGuard device;
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    cudaStream_t stream = nullptr;
    int idx;
    Place(PyObject* o, int idx_) : idx(idx_) {
        if (o == Py_None) {
            device.set_index((c10::DeviceIndex)idx);
            stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)idx).stream();
            return;
        }
        long long v[3];
        const char* const names[3] = {"stream_id", "device_index", "device_type"};
        for (int i = 0; i < 3; ++i) {
            PyObject* x = PyObject_GetAttrString(o, names[i]);
            if (!x) throw Raised();
            v[i] = PyLong_AsLongLong(x);
            Py_DECREF(x);
            if (v[i] == -1 && PyErr_Occurred()) throw Raised();
        }
        if (v[1] != idx) refuse("%s is on another device than the tensors", "stream");
        const auto s = c10::cuda::CUDAStream::unpack3(v[0], (c10::DeviceIndex)v[1], (c10::DeviceType)v[2]);
        guard.emplace(s);
        stream = s.stream();
    }
    // A tensor of this stream.
    at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
        return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)idx));
    }
};

void check(int status, const char* what) {
    if (status == ATTN_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", status, what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised();
}

// `count` values of a one-dimensional buffer from `first` on, as a tensor of its storage (made directly: a
// view operation of torch's takes about 1 us).
at::Tensor part_of(const at::Tensor& buf, int64_t first, int64_t count) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(buf.storage()), buf.key_set(),
                                                            buf.dtype());
    const int64_t size[1] = {count}, stride[1] = {1};
    t.unsafeGetTensorImpl()->set_storage_offset(buf.storage_offset() + first);
    t.unsafeGetTensorImpl()->set_sizes_and_strides(size, stride);
    return t;
}

// Runs f, with what it throws as the Python error that torch makes of it (out of memory: torch.OutOfMemoryError).
template <class F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
    if (given != wanted) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %d", (int)wanted, (int)given);
        return nullptr;
    }
    if (!g_error) {
        PyErr_SetString(PyExc_RuntimeError, "the attention library is not loaded");
        return nullptr;
    }
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// The tuple of some results, each a given Python object or a new tensor.
struct Result {
    PyObject* given;  // borrowed, or None
    at::Tensor made;
    PyObject* object() const {
        if (given == Py_None) return THPVariable_Wrap(made);
        Py_INCREF(given);
        return given;
    }
};
template <size_t N>
PyObject* tuple(const Result (&r)[N]) {
    PyObject* t = PyTuple_New(N);
    if (!t) return nullptr;
    for (size_t i = 0; i < N; ++i) {
        PyObject* o = r[i].object();
        if (!o) {
            Py_DECREF(t);
            return nullptr;
        }
        PyTuple_SET_ITEM(t, i, o);
    }
    return t;
}

// ---- step plan ---------------------------------------------------------------------------------
// (kv_lens, new_lens, free_pages, block_table, pages_held, free_used, total_new, num_pages, page_size, out, stream)
PyObject* paged_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject* {
        const at::Tensor& kv = tensor(a[0], "kv_lens");
        const at::Tensor& free_pages = tensor(a[2], "free_pages");
        const at::Tensor& table = tensor(a[3], "block_table");
        const int idx = index_of(kv, "kv_lens");
        const int T = as_int(a[6], "total_new"), num_pages = as_int(a[7], "num_pages"), page_size = as_int(a[8], "page_size");
        if (table.dim() != 2) refuse("%s must be [num_reqs, max_pages]", "block_table");
        if (T < 0) refuse("%s must not be negative", "total_new");
        const int64_t R = kv.numel(), F = free_pages.numel(), maxp = table.size(1);
        if (R > INT32_MAX || F > INT32_MAX || maxp > INT32_MAX) refuse("%s is too large", "the plan");
        const int64_t sR[1] = {R}, sR1[1] = {R + 1}, sT[1] = {T}, s1[1] = {1}, sF[1] = {F}, sTab[2] = {R, maxp};
        const int32_t* in[5] = {i32(a[0], sR, idx, "kv_lens"), i32(a[1], sR, idx, "new_lens"), i32(a[4], sR, idx, "pages_held"),
                                i32(a[2], sF, idx, "free_pages"), i32(a[5], s1, idx, "free_used")};
        int32_t* tab = i32(a[3], sTab, idx, "block_table");
        Place place(a[10], idx);
        // seq_lens, cu_q, positions, slots, pages_held, free_used, admitted
        const at::IntArrayRef shapes[7] = {sR, sR1, sT, sT, sR, s1, s1};
        int32_t* out[7];
        PyObject* plan = a[9];
        if (plan != Py_None) {
            static const char* const names[7] = {"out.seq_lens", "out.cu_q", "out.positions", "out.slots",
                                                 "out.pages_held", "out.free_used", "out.admitted"};
            if (!PyTuple_Check(plan) || PyTuple_GET_SIZE(plan) != 7) refuse("%s must be a PagedPlan", "out");
            for (int i = 0; i < 7; ++i) out[i] = i32(PyTuple_GET_ITEM(plan, i), shapes[i], idx, names[i]);
            check(g_api.paged_plan(in[0], in[1], in[2], in[3], in[4], tab, out[0], out[1], out[2], out[3], out[4], out[5], out[6],
                                   (int)R, T, (int)F, page_size, (int)maxp, num_pages, place.stream),
                  "attn_paged_plan");
            Py_INCREF(plan);
            return plan;
        }
        // one allocation; positions and slots first, each at 16 bytes
        const int64_t Tp = ((int64_t)T + 3) / 4 * 4, at_cu = 2 * Tp;
        const int64_t first[7] = {at_cu + R + 1, at_cu, 0, Tp, at_cu + 2 * R + 1, at_cu + 3 * R + 1, at_cu + 3 * R + 2};
        const int64_t total[1] = {at_cu + 3 * R + 3};
        const at::Tensor buf = place.make(total, at::kInt);
        int32_t* base = static_cast<int32_t*>(buf.data_ptr());
        for (int i = 0; i < 7; ++i) out[i] = base + first[i];
        check(g_api.paged_plan(in[0], in[1], in[2], in[3], in[4], tab, out[0], out[1], out[2], out[3], out[4], out[5], out[6], (int)R,
                               T, (int)F, page_size, (int)maxp, num_pages, place.stream),
              "attn_paged_plan");
        auto* type = reinterpret_cast<PyTypeObject*>(g_plan);  // a named tuple
        PyObject* r = type->tp_alloc(type, 7);
        if (!r) throw Raised();
        for (int i = 0; i < 7; ++i) {
            PyObject* o = THPVariable_Wrap(part_of(buf, first[i], shapes[i][0]));
            if (!o) {
                Py_DECREF(r);
                throw Raised();
            }
            PyTuple_SET_ITEM(r, i, o);
        }
        return r;
    });
}

// ---- head norm ---------------------------------------------------------------------------------
// A [T, H, D] or [B, S, H, D] bfloat16 tensor as T tokens of H x D, `step` elements apart.
struct Rows {
    int64_t T, H, D, step;
    attn_bf16* at;
};
Rows rows(const at::Tensor& t, const char* name, int idx) {
    if (t.scalar_type() != at::kBFloat16 || !t.is_cuda() || t.get_device() != idx)
        refuse("%s must be a bfloat16 tensor on the call's device", name);
    const auto s = t.sizes(), st = t.strides();
    Rows r;
    if (s.size() == 3) {
        r.T = s[0], r.step = st[0];
    } else if (s.size() == 4) {
        r.T = s[0] * s[1], r.step = s[1] > 1 ? st[1] : st[0];
        if (s[0] > 1 && s[1] > 1 && st[0] != s[1] * st[1]) refuse("%s: tokens must be evenly spaced across the batch", name);
    } else {
        refuse("%s must be [T, H, D] or [B, S, H, D]", name);
    }
    const size_t d = s.size() - 1;
    r.H = s[d - 1], r.D = s[d];
    if ((st[d] != 1 && r.D > 1) || (st[d - 1] != r.D && r.H > 1)) refuse("%s: the heads of a token must be contiguous", name);
    if (r.T <= 1) r.step = r.H * r.D;
    if (r.T > INT32_MAX || r.H > INT32_MAX || r.D > INT32_MAX) refuse("%s is too large", name);
    r.at = static_cast<attn_bf16*>(t.data_ptr());
    return r;
}

// What the three head-norm calls share.
struct Norm {
    const at::Tensor &q, &k;
    int idx;
    Rows rq, rk;
    const void* weight[2] = {nullptr, nullptr};
    int fp32 = 0;
    const int32_t* positions = nullptr;
    const float* table = nullptr;
    int rot = 0, max_pos = 0;
    float eps, offset;
    int inter;

    // per-token values: [T], or the tokens' own [B, S]
    int32_t* per_token(PyObject* o, const char* name) const {
        const at::Tensor& t = tensor(o, name);
        const int64_t flat[1] = {rq.T};
        return checked<int32_t>(t, at::kInt, t.dim() == 1 ? at::IntArrayRef(flat) : q.sizes().slice(0, q.dim() - 2), idx, name);
    }
    Norm(PyObject* q_, PyObject* k_, PyObject* qw, PyObject* kw, PyObject* pos, PyObject* cos_sin, PyObject* eps_, PyObject* off,
         PyObject* inter_)
        : q(tensor(q_, "q")), k(tensor(k_, "k")), idx(index_of(q, "q")), rq(rows(q, "q", idx)), rk(rows(k, "k", idx)) {
        if (rk.T != rq.T || rk.D != rq.D || q.dim() != k.dim() || q.size(0) != k.size(0))
            refuse("%s must have the same tokens and head size", "q and k");
        PyObject* const w[2] = {qw, kw};
        int kind = -1;
        for (int i = 0; i < 2; ++i) {
            if (w[i] == Py_None) continue;
            const char* name = i ? "k_weight" : "q_weight";
            const at::Tensor& t = tensor(w[i], name);
            const int64_t sD[1] = {rq.D};
            const bool f = t.scalar_type() == at::kFloat;
            weight[i] = checked<void>(t, f ? at::kFloat : at::kBFloat16, sD, idx, name);
            if (kind >= 0 && kind != (int)f) refuse("%s must both be bfloat16 or both float32", "q_weight and k_weight");
            kind = f;
        }
        fp32 = kind > 0;
        if (cos_sin != Py_None) {
            const at::Tensor& t = tensor(cos_sin, "cos_sin");
            if (t.dim() != 2 || t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) refuse("%s must be [max_pos, rot_dim]", "cos_sin");
            const float* at = checked<float>(t, at::kFloat, t.sizes(), idx, "cos_sin");
            if (t.size(1) > 0) {
                if (pos == Py_None) refuse("%s are needed with cos_sin", "positions");
                positions = per_token(pos, "positions");
                table = at, rot = (int)t.size(1), max_pos = (int)t.size(0);
            }
        }
        eps = as_float(eps_), offset = as_float(off), inter = as_bool(inter_);
    }
};

// A given output of x's shape, contiguous, or a new one.
attn_bf16* like(Result& r, PyObject* o, const at::Tensor& x, const Place& place, const char* name) {
    r.given = o;
    if (o != Py_None) return bf16(tensor(o, name), x.sizes(), place.idx, name);
    r.made = place.make(x.sizes(), at::kBFloat16);
    return static_cast<attn_bf16*>(r.made.data_ptr());
}

// (q, k, q_weight, k_weight, positions, cos_sin, q_out, k_out, eps, weight_offset, interleaved, stream)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const Norm x(a[0], a[1], a[2], a[3], a[4], a[5], a[8], a[9], a[10]);
        Place place(a[11], x.idx);
        Result r[2];
        attn_bf16* qo = like(r[0], a[6], x.q, place, "q_out");
        attn_bf16* ko = like(r[1], a[7], x.k, place, "k_out");
        check(g_api.norm_rope(x.rq.at, x.rk.at, qo, ko, x.weight[0], x.weight[1], x.positions, x.table, (int)x.rq.T, (int)x.rq.H,
                              (int)x.rk.H, (int)x.rq.D, x.rot, x.max_pos, x.rq.step, x.rk.step, x.eps, x.offset, x.fp32, x.inter,
                              place.stream),
              "attn_qk_norm_rope");
        return tuple(r);
    });
}

// The workspace given, or one of the call's own: of its stream, or of the graph being captured, so that calls
// on different streams or in different graphs never share it.
void* scratch(at::Tensor& own, size_t& bytes, PyObject* given, size_t need, const Place& place) {
    if (given == Py_None) {
        const int64_t s[1] = {(int64_t)need};
        own = place.make(s, at::kByte);
        bytes = need;
        return own.data_ptr();
    }
    const at::Tensor& t = tensor(given, "workspace");
    if (!t.is_cuda() || t.get_device() != place.idx || !t.is_contiguous()) refuse("%s must be a contiguous tensor on the call's device", "workspace");
    bytes = t.nbytes();
    return t.data_ptr();
}

// (dq_out, dk_out, q, k, q_weight, k_weight, positions, cos_sin, dq, dk, eps, weight_offset, interleaved, workspace, stream)
PyObject* norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject* {
        const Norm x(a[2], a[3], a[4], a[5], a[6], a[7], a[10], a[11], a[12]);
        attn_bf16* gq = bf16(tensor(a[0], "dq_out"), x.q.sizes(), x.idx, "dq_out");
        attn_bf16* gk = bf16(tensor(a[1], "dk_out"), x.k.sizes(), x.idx, "dk_out");
        Place place(a[14], x.idx);
        Result r[4] = {{a[8], {}}, {a[9], {}}, {Py_None, {}}, {Py_None, {}}};
        attn_bf16* d[2];
        int64_t step[2];
        for (int i = 0; i < 2; ++i) {
            const at::Tensor& in = i ? x.k : x.q;
            const Rows& ri = i ? x.rk : x.rq;
            const char* name = i ? "dk" : "dq";
            if (r[i].given == Py_None) {
                r[i].made = place.make(in.sizes(), at::kBFloat16);
                d[i] = static_cast<attn_bf16*>(r[i].made.data_ptr()), step[i] = ri.H * ri.D;
            } else {
                const at::Tensor& t = tensor(r[i].given, name);
                if (t.sizes() != in.sizes()) refuse("%s must have the shape of its input", name);
                const Rows ro = rows(t, name, x.idx);
                d[i] = ro.at, step[i] = ro.step;
            }
        }
        const int64_t sw[1] = {2 * x.rq.D};
        const at::Tensor dw = place.make(sw, at::kFloat);
        float* dwp = static_cast<float*>(dw.data_ptr());
        at::Tensor own;
        size_t bytes = 0;
        void* ws = scratch(own, bytes, a[13], g_api.workspace_size(ATTN_OP_QK_NORM_ROPE_BWD, 0, 0, 0, 0, (int)x.rq.D, 0, 0), place);
        check(g_api.norm_rope_bwd(gq, gk, x.rq.at, x.rk.at, d[0], d[1], dwp, dwp + x.rq.D, x.weight[0], x.weight[1], x.positions,
                                  x.table, (int)x.rq.T, (int)x.rq.H, (int)x.rk.H, (int)x.rq.D, x.rot, x.max_pos, x.rq.step, x.rk.step,
                                  step[0], step[1], x.eps, x.offset, x.fp32, x.inter, ws, bytes, place.stream),
              "attn_qk_norm_rope_bwd");
        r[2].made = part_of(dw, 0, x.rq.D), r[3].made = part_of(dw, x.rq.D, x.rq.D);
        return tuple(r);
    });
}

// Pointers and [num_pages, page_size, Hkv] of a pair of caches.
struct Caches {
    attn_bf16 *k, *v;
    int num_pages, page_size, heads;
    Caches(PyObject* k_, PyObject* v_, int64_t D, int idx) {
        const at::Tensor& t = tensor(k_, "k_cache");
        if (t.dim() != 4 || t.size(3) != D || t.size(0) > INT32_MAX || t.size(1) > INT32_MAX || t.size(2) > INT32_MAX)
            refuse("%s must be [num_pages, page_size, Hkv, D]", "k_cache");
        k = bf16(t, t.sizes(), idx, "k_cache"), v = bf16(tensor(v_, "v_cache"), t.sizes(), idx, "v_cache");
        num_pages = (int)t.size(0), page_size = (int)t.size(1), heads = (int)t.size(2);
    }
};

// (q, k, v, q_weight, k_weight, positions, slots, cos_sin, k_cache, v_cache, q_out, eps, weight_offset, interleaved, stream)
PyObject* norm_rope_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject* {
        const Norm x(a[0], a[1], a[3], a[4], a[5], a[7], a[11], a[12], a[13]);
        const at::Tensor& v = tensor(a[2], "v");
        if (v.sizes() != x.k.sizes()) refuse("%s must have the shape of k", "v");
        const Rows rv = rows(v, "v", x.idx);
        const Caches c(a[8], a[9], x.rq.D, x.idx);
        if (c.heads != x.rk.H) refuse("%s are not k's", "the caches' heads");
        int32_t* slots = x.per_token(a[6], "slots");
        Place place(a[14], x.idx);
        Result r;
        attn_bf16* qo = like(r, a[10], x.q, place, "q_out");
        check(g_api.norm_rope_paged(x.rq.at, x.rk.at, rv.at, qo, c.k, c.v, x.weight[0], x.weight[1], x.positions, slots, x.table,
                                    (int)x.rq.T, (int)x.rq.H, (int)x.rk.H, (int)x.rq.D, x.rot, x.max_pos, c.page_size, c.num_pages,
                                    x.rq.step, x.rk.step, rv.step, x.eps, x.offset, x.fp32, x.inter, place.stream),
              "attn_qk_norm_rope_paged");
        return r.object();
    });
}

// ---- tree attention ----------------------------------------------------------------------------
// (q, k_cache, v_cache, block_table, seq_lens, cu_q, tree_mask, max_q_len, o, lse, positions, window, scale, workspace, stream)
PyObject* tree_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject* {
        const at::Tensor& q = tensor(a[0], "q");
        const int idx = index_of(q, "q");
        if (q.dim() != 3 || q.size(0) > INT32_MAX || q.size(1) > INT32_MAX || q.size(2) > INT32_MAX)
            refuse("%s must be [T, Hq, D]", "q");
        const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
        attn_bf16* qp = bf16(q, q.sizes(), idx, "q");
        const Caches c(a[1], a[2], D, idx);
        const at::Tensor& table = tensor(a[3], "block_table");
        const at::Tensor& lens = tensor(a[4], "seq_lens");
        const at::Tensor& mask = tensor(a[6], "tree_mask");
        const int64_t R = lens.numel();
        if (table.dim() != 2 || mask.dim() != 2 || R > INT32_MAX || table.size(1) > INT32_MAX || mask.size(1) > INT32_MAX)
            refuse("%s: block_table must be [num_reqs, max_pages] and tree_mask [T, words]", "tree attention");
        const int64_t sR[1] = {R}, sR1[1] = {R + 1}, sT[1] = {T}, sTab[2] = {R, table.size(1)}, sM[2] = {T, mask.size(1)};
        int32_t* tab = i32(a[3], sTab, idx, "block_table");
        int32_t* sl = i32(a[4], sR, idx, "seq_lens");
        int32_t* cu = i32(a[5], sR1, idx, "cu_q");
        int32_t* mw = i32(a[6], sM, idx, "tree_mask");
        int32_t* pos = a[10] == Py_None ? nullptr : i32(a[10], sT, idx, "positions");
        const int top = as_int(a[7], "max_q_len"), window = as_int(a[11], "window");
        const float scale = as_float(a[12]);
        Place place(a[14], idx);
        Result r[2];
        attn_bf16* o = like(r[0], a[8], q, place, "o");
        const int64_t sL[2] = {Hq, T};
        float* lse;
        r[1].given = a[9];
        if (a[9] == Py_None) {
            r[1].made = place.make(sL, at::kFloat);
            lse = static_cast<float*>(r[1].made.data_ptr());
        } else {
            lse = checked<float>(tensor(a[9], "lse"), at::kFloat, sL, idx, "lse");
        }
        at::Tensor own;
        size_t bytes = 0;
        void* ws = scratch(own, bytes, a[13], g_api.workspace_size(ATTN_OP_TREE_PAGED, 0, (int)Hq, c.heads, top, (int)D, 0, 0), place);
        check(g_api.tree_paged(qp, c.k, c.v, tab, sl, cu, mw, pos, o, lse, (int)R, (int)T, top, (int)mask.size(1), (int)Hq, c.heads,
                               (int)D, c.page_size, (int)table.size(1), c.num_pages, scale, window, ws, bytes, place.stream),
              "attn_tree_paged");
        return tuple(r);
    });
}

// load(path of the library, AttnError, PagedPlan)
PyObject* load(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "3 arguments expected");
        return nullptr;
    }
    const char* path = PyUnicode_AsUTF8(a[0]);
    if (!path) return nullptr;
    void* lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!lib) {
        PyErr_SetString(PyExc_RuntimeError, dlerror());
        return nullptr;
    }
    if (!PyType_Check(a[2]) || !PyType_IsSubtype(reinterpret_cast<PyTypeObject*>(a[2]), &PyTuple_Type)) {
        PyErr_SetString(PyExc_TypeError, "PagedPlan must be a named tuple");
        return nullptr;
    }
    Api api;
    auto find = [&](auto& f, const char* name) {
        f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(dlsym(lib, name));
        if (!f && !PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s is missing from the attention library", name);
    };
    find(api.paged_plan, "attn_paged_plan");
    find(api.norm_rope, "attn_qk_norm_rope");
    find(api.norm_rope_bwd, "attn_qk_norm_rope_bwd");
    find(api.norm_rope_paged, "attn_qk_norm_rope_paged");
    find(api.tree_paged, "attn_tree_paged");
    find(api.workspace_size, "attn_workspace_size");
    if (PyErr_Occurred()) return nullptr;
    g_api = api;
    Py_INCREF(a[1]), Py_INCREF(a[2]);
    Py_XSETREF(g_plan, a[2]);
    Py_XSETREF(g_error, a[1]);
    Py_RETURN_NONE;
}

#define ATTN_OP(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {ATTN_OP(load),           ATTN_OP(paged_plan), ATTN_OP(norm_rope), ATTN_OP(norm_rope_bwd),
                          ATTN_OP(norm_rope_paged), ATTN_OP(tree_paged), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops(void) { return PyModule_Create(&kModule); }
