// Tensor side of the binding for the operators with a position bias and the
// eviction: checks shapes, types, strides and devices, allocates results and
// workspaces from torch's allocator on the current stream, and calls the C ABI.
// In Python the same steps cost 12 to 16 us a call, more than the kernels of a
// small batch take.  The functions take all arguments by position (None where
// there is none) and return their results, or the call's status code when the
// library refused it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/clone.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>

#include "ragged.h"

namespace {

using at::Tensor;

struct Library {
    decltype(&ragged_attn_bias_fwd_workspace) fwd_workspace;
    decltype(&ragged_attn_bias_fwd) fwd;
    decltype(&ragged_attn_bias_bwd_workspace) bwd_workspace;
    decltype(&ragged_attn_bias_bwd) bwd;
    decltype(&ragged_attn_weight) weight;
    decltype(&ragged_evict) evict;
} g_lib;

const Tensor& tensor(PyObject* o, const char* what) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), what, " must be a tensor");
    return THPVariable_Unpack(o);
}
Tensor maybe(PyObject* o, const char* what) { return o == Py_None ? Tensor() : tensor(o, what); }
int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

// One device for all tensors, and the current one: the library launches there.
struct Devices {
    c10::DeviceIndex current = -1;
    void add(const Tensor& t) {
        if (!t.defined()) return;
        if (current < 0 && t.is_cuda()) current = c10::cuda::current_device();
        TORCH_CHECK_VALUE(t.is_cuda() && t.get_device() == current, "a tensor is on ", t.device(),
                          ", not on the current CUDA device");
    }
};

void ints(const Tensor& t, int64_t n, const char* what) {
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.dim() == 1 && t.is_contiguous() && (n < 0 || t.size(0) == n), what,
                      " must be contiguous int32", n < 0 ? std::string() : " [" + std::to_string(n) + "]");
}

// The address of a tensor; of one without elements, `other` (never read).
void* address(const Tensor& t, const void* other) {
    void* p = t.data_ptr();
    return p != nullptr ? p : const_cast<void*>(other);
}

Tensor empty(at::IntArrayRef size, const Tensor& like, at::ScalarType type) {
    return at::empty(size, like.options().dtype(type).requires_grad(false));
}

void* current_stream(const Devices& d) { return c10::cuda::getCurrentCUDAStream(d.current).stream(); }

// Scratch of one call: its memory goes back to torch's allocator when the call
// returns, which hands it out again behind this call's work on the same stream.
struct Scratch {
    Tensor t;
    void* p = nullptr;
    int64_t bytes = 0;
    void take(int64_t n, const Tensor& like) {
        bytes = n;
        if (n > 0) {
            t = empty({n}, like, at::kByte);
            p = t.data_ptr();
        }
    }
};

// The arguments that the three attention operators share: their tensors, ...
struct Shared {
    const Tensor &cu_q, &cu_k, &table, &buckets;
    const Tensor pos_q, pos_k;
    explicit Shared(PyObject* const* o)
        : cu_q(tensor(o[0], "cu_seqlens_q")), cu_k(tensor(o[1], "cu_seqlens_k")), table(tensor(o[4], "table")), buckets(tensor(o[5], "buckets")),
          pos_q(maybe(o[6], "pos_q")), pos_k(maybe(o[7], "pos_k")) {}
};
// ... and the library's view of them, checked.
struct Problem {
    ragged_bias_attn a;
    Devices dev;
    int64_t Tq, Tk;

    Problem(const Tensor& q, const Tensor& k, const Tensor& v, PyObject* const* o, const Shared& in, const Tensor& lse) {
        const Tensor &cu_q = in.cu_q, &cu_k = in.cu_k, &table = in.table, &buckets = in.buckets, &pos_q = in.pos_q, &pos_k = in.pos_k;
        TORCH_CHECK_VALUE(q.dim() == 3 && k.dim() == 3, "q must be [Tq, H, head_dim], k and v [Tk, Hkv, head_dim]");
        const auto type = q.scalar_type();
        TORCH_CHECK_VALUE(v.sizes() == k.sizes() && k.size(2) == q.size(2) && k.scalar_type() == type &&
                              v.scalar_type() == type && table.scalar_type() == type,
                          "q [Tq, H, d], k and v [Tk, Hkv, d] and table must have one dtype and head_dim");
        TORCH_CHECK_VALUE(q.stride(2) == 1 && k.stride(2) == 1 && v.strides() == k.strides(),
                          "q, k and v need a unit innermost stride, and k and v the same strides");
        Tq = q.size(0);
        Tk = k.size(0);
        const int64_t H = q.size(1);
        TORCH_CHECK_VALUE(table.dim() == 2 && table.size(1) == H && table.is_contiguous(), "table must be contiguous [num_buckets, H]");
        ints(cu_q, -1, "cu_seqlens_q");
        TORCH_CHECK_VALUE(cu_q.size(0) >= 1, "cu_seqlens_q must hold at least one value");
        ints(cu_k, cu_q.size(0), "cu_seqlens_k");
        ints(buckets, -1, "buckets");
        TORCH_CHECK_VALUE(buckets.size(0) % 2 == 1, "buckets must have an odd length, 2 * max_distance + 1");
        if (pos_q.defined()) ints(pos_q, Tq, "pos_q");
        if (pos_k.defined()) ints(pos_k, Tk, "pos_k");
        TORCH_CHECK_VALUE(lse.scalar_type() == at::kFloat && lse.dim() == 2 && lse.size(0) == H && lse.size(1) == Tq &&
                              (Tq <= 1 || lse.stride(1) == 1),
                          "lse must be float32 [H, Tq] with unit innermost stride");
        TORCH_CHECK_VALUE(H <= 1 || lse.stride(0) >= Tq, "the rows of lse must not overlap");
        for (const Tensor* t : {&q, &k, &v, &cu_q, &cu_k, &table, &buckets, &pos_q, &pos_k, &lse}) dev.add(*t);
        const void* some = cu_q.data_ptr();
        a = ragged_bias_attn{};
        a.q = address(q, some);
        a.k = address(k, some);
        a.v = address(v, some);
        a.q_tok_stride = q.stride(0);
        a.q_head_stride = q.stride(1);
        a.kv_tok_stride = k.stride(0);
        a.kv_head_stride = k.stride(1);
        a.cu_seqlens_q = static_cast<const int32_t*>(some);
        a.cu_seqlens_k = static_cast<const int32_t*>(cu_k.data_ptr());
        a.B = cu_q.size(0) - 1;
        a.max_seqlen_q = integer(o[2]);
        a.max_seqlen_k = integer(o[3]);
        a.H = H;
        a.Hkv = k.size(1);
        a.head_dim = q.size(2);
        a.table = table.data_ptr();
        a.buckets = static_cast<const int32_t*>(buckets.data_ptr());
        a.num_buckets = table.size(0);
        a.max_distance = buckets.size(0) / 2;
        a.pos_q = pos_q.defined() ? static_cast<const int32_t*>(address(pos_q, some)) : nullptr;
        a.pos_k = pos_k.defined() ? static_cast<const int32_t*>(address(pos_k, some)) : nullptr;
        a.lse = static_cast<float*>(address(lse, some));
        a.lse_stride = H > 1 ? lse.stride(0) : Tq;
        if (o[8] == Py_None) {
            a.scale = 1.0f / std::sqrt(static_cast<float>(a.head_dim));
        } else {
            const double s = PyFloat_AsDouble(o[8]);
            if (s == -1.0 && PyErr_Occurred()) throw python_error();
            a.scale = static_cast<float>(s);
        }
        TORCH_CHECK_TYPE(type == at::kHalf || type == at::kBFloat16 || type == at::kFloat, "unsupported dtype ", type);
        a.dtype = type == at::kHalf ? RAGGED_F16 : type == at::kBFloat16 ? RAGGED_BF16 : RAGGED_F32;
    }
};

constexpr int kShared = 9;   // cu_q, cu_k, max_q, max_k, table, buckets, pos_q, pos_k, scale

PyObject* status(ragged_status s) { return PyLong_FromLong(s); }
PyObject* results(std::initializer_list<Tensor> ts) {
    PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (r == nullptr) throw python_error();
    Py_ssize_t i = 0;
    for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None));
    return r;
}
void arguments(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

bool rows_of_heads(const Tensor& t) {
    const int64_t H = t.size(1), d = t.size(2);
    return t.stride(2) == 1 && (H <= 1 || t.stride(1) == d) && (t.size(0) <= 1 || t.stride(0) >= H * d);
}
int64_t row_stride(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2); }

// A given result, checked, or a new one with the shape of `like`.
Tensor result(PyObject* o, const Tensor& like, const char* what) {
    if (o == Py_None) return empty(like.sizes(), like, like.scalar_type());
    const Tensor& t = tensor(o, what);
    TORCH_CHECK_VALUE(t.sizes() == like.sizes() && t.scalar_type() == like.scalar_type() && (t.dim() < 3 || t.stride(2) == 1),
                      what, " must have the shape and dtype of its input and a unit innermost stride");
    return t;
}

// The bytes of a tensor: runs of `len` at base + i * step[0] + j * step[1] + ...
struct Bytes {
    int64_t base, len;
    int dims = 0;
    int64_t size[8], step[8];   // from the smallest step to the largest
    bool itself = false;        // runs that overlap one another
    explicit Bytes(const Tensor& t) : base(reinterpret_cast<int64_t>(t.data_ptr())), len(t.numel() == 0 ? 0 : t.element_size()) {
        int order[8], n = 0;
        TORCH_CHECK_VALUE(t.dim() <= 8, "a tensor has ", t.dim(), " dimensions");
        for (int d = 0; d < t.dim(); ++d) {   // by their strides
            if (t.size(d) <= 1) continue;
            int i = n++;
            for (; i > 0 && t.stride(order[i - 1]) > t.stride(d); --i) order[i] = order[i - 1];
            order[i] = d;
        }
        for (int i = 0; i < n; ++i) {
            const int64_t s = t.stride(order[i]) * static_cast<int64_t>(t.element_size());
            itself |= s < extent();
            if (s == 0) continue;   // the same bytes again
            if (dims == 0 && s == len) {
                len *= t.size(order[i]);
            } else {
                size[dims] = t.size(order[i]);
                step[dims++] = s;
            }
        }
    }
    int64_t extent() const {
        int64_t e = len;
        for (int d = 0; d < dims; ++d) e += (size[d] - 1) * step[d];
        return e;
    }
};
// Whether two tensors share a byte.  `left` bounds the work on layouts that no
// closed form covers; past it they count as sharing.
bool share(const Bytes& a, const Bytes& b, int64_t& left) {
    if (a.len == 0 || b.len == 0 || a.base + a.extent() <= b.base || b.base + b.extent() <= a.base) return false;
    if (a.dims + b.dims == 0 || --left < 0) return true;
    if (a.dims <= 1 && b.dims <= 1 && (a.dims == 0 || b.dims == 0 || a.step[0] == b.step[0])) {
        // Runs i of a and j of b meet where -b.len < distance + (j - i) * step < a.len.
        const int64_t step = a.dims ? a.step[0] : b.step[0], na = a.dims ? a.size[0] : 1, nb = b.dims ? b.size[0] : 1, d = b.base - a.base;
        auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y < 0); };
        return std::min(nb - 1, floor_div(a.len - 1 - d, step)) >= std::max(1 - na, -floor_div(d + b.len - 1, step));
    }
    const bool first = b.dims == 0 || (a.dims > 0 && a.size[a.dims - 1] <= b.size[b.dims - 1]);
    Bytes one = first ? a : b;
    const int64_t n = one.size[one.dims - 1], step = one.step[one.dims - 1];
    --one.dims;
    for (int64_t i = 0; i < n; ++i, one.base += step)
        if (share(one, first ? b : a, left)) return true;
    return false;
}
// A result that the caller gave is written while the inputs are still read, and
// while other results are written: it shares no byte with them or within itself.
void apart(const Tensor& result, std::initializer_list<const Tensor*> others, const char* what) {
    if (result.numel() == 0) return;
    const Bytes r(result);
    TORCH_CHECK_VALUE(!r.itself, what, " must not overlap itself");
    for (const Tensor* t : others) {
        if (!t->defined()) continue;
        int64_t left = 1 << 16;
        TORCH_CHECK_VALUE(!share(r, Bytes(*t), left), what, " must not share its memory with an input or another result");
    }
}

// The calls record no graph: results that would silently lose theirs are refused.
void no_graph(std::initializer_list<const Tensor*> inputs) {
    if (!at::GradMode::is_enabled()) return;
    for (const Tensor* t : inputs)
        TORCH_CHECK_VALUE(!t->defined() || !t->requires_grad(), "an input requires a gradient, and this call records no graph: call it under "
                          "torch.no_grad(), or in a torch.autograd.Function with ragged_attn_bias_bwd as its backward");
}

// q, k, v, shared..., out, lse -> (out, lse)
PyObject* bias_fwd(PyObject*, PyObject* const* o, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 3 + kShared + 2);
    const Tensor &q = tensor(o[0], "q"), &k = tensor(o[1], "k"), &v = tensor(o[2], "v");
    TORCH_CHECK_VALUE(q.dim() == 3, "q must be [Tq, H, head_dim]");
    const Tensor out = result(o[3 + kShared], q, "out");
    TORCH_CHECK_VALUE(rows_of_heads(out), "out must be [T, H, head_dim] with contiguous heads");
    const Tensor lse = o[4 + kShared] == Py_None ? empty({q.size(1), q.size(0)}, q, at::kFloat) : tensor(o[4 + kShared], "lse");
    const Shared in(o + 3);
    no_graph({&q, &k, &v, &in.table});
    if (o[3 + kShared] != Py_None) apart(out, {&q, &k, &v, &lse, &in.cu_q, &in.cu_k, &in.table, &in.buckets, &in.pos_q, &in.pos_k}, "out");
    if (o[4 + kShared] != Py_None) apart(lse, {&q, &k, &v, &in.cu_q, &in.cu_k, &in.table, &in.buckets, &in.pos_q, &in.pos_k}, "lse");
    Problem p(q, k, v, o + 3, in, lse);
    p.dev.add(out);
    int64_t bytes = 0;
    ragged_status s = g_lib.fwd_workspace(&p.a, &bytes);
    if (s != RAGGED_OK) return status(s);
    Scratch ws;
    ws.take(bytes, q);
    s = g_lib.fwd(&p.a, address(out, p.a.cu_seqlens_q), row_stride(out), ws.p, ws.bytes, current_stream(p.dev));
    return s != RAGGED_OK ? status(s) : results({out, lse});
    END_HANDLE_TH_ERRORS
}

// dout, q, k, v, out, lse, shared..., dq, dk, dv, dtable -> (dq, dk, dv, dtable)
PyObject* bias_bwd(PyObject*, PyObject* const* o, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 6 + kShared + 4);
    Tensor dout = tensor(o[0], "dout");
    const Tensor &q = tensor(o[1], "q"), &k = tensor(o[2], "k"), &v = tensor(o[3], "v"), &out = tensor(o[4], "out"), &lse = tensor(o[5], "lse");
    PyObject* const* given = o + 6 + kShared;
    TORCH_CHECK_VALUE(out.sizes() == q.sizes() && out.scalar_type() == q.scalar_type() && q.dim() == 3 && rows_of_heads(out),
                      "out must be [T, H, head_dim] with contiguous heads");
    TORCH_CHECK_VALUE(dout.sizes() == q.sizes() && dout.scalar_type() == q.scalar_type(), "dout must have the shape and dtype of out");
    const Shared in(o + 6);
    const Tensor& table = in.table;
    no_graph({&dout, &q, &k, &v, &out, &lse, &table});
    const Tensor dq = result(given[0], q, "dq"), dk = result(given[1], k, "dk"), dv = result(given[2], v, "dv");
    const Tensor dtable = result(given[3], table, "dtable");
    TORCH_CHECK_VALUE(dk.numel() == 0 || dk.strides() == dv.strides(), "dk and dv must have the same strides");
    auto given_apart = [&](int i, const Tensor& d, std::initializer_list<const Tensor*> results, const char* what) {
        if (given[i] == Py_None) return;
        apart(d, results, what);
        apart(d, {&q, &k, &v, &out, &dout, &lse, &table, &in.cu_q, &in.cu_k, &in.buckets, &in.pos_q, &in.pos_k}, what);
    };
    given_apart(0, dq, {&dk, &dv, &dtable}, "dq");
    given_apart(1, dk, {&dv, &dtable}, "dk");
    given_apart(2, dv, {&dtable}, "dv");
    given_apart(3, dtable, {}, "dtable");
    TORCH_CHECK_VALUE(dtable.is_contiguous(), "dtable must be contiguous with the shape and dtype of table");
    Problem p(q, k, v, o + 6, in, lse);
    p.dev.add(dout);
    p.dev.add(out);
    if (!rows_of_heads(dout) || reinterpret_cast<uintptr_t>(dout.data_ptr()) % 16 != 0 || row_stride(dout) % 8 != 0)
        dout = dout.detach().clone(at::MemoryFormat::Contiguous);   // a broadcast or transposed gradient
    for (const Tensor* t : {&dq, &dk, &dv, &dtable}) p.dev.add(*t);
    int64_t bytes = 0;
    ragged_status s = g_lib.bwd_workspace(&p.a, &bytes);
    if (s != RAGGED_OK) return status(s);
    Scratch ws;
    ws.take(bytes, q);
    const void* some = p.a.cu_seqlens_q;
    s = g_lib.bwd(&p.a, address(out, some), row_stride(out), address(dout, some), row_stride(dout), address(dq, some), dq.stride(0),
                  dq.stride(1), address(dk, some), address(dv, some), dk.stride(0), dk.stride(1), dtable.data_ptr(), ws.p, ws.bytes,
                  current_stream(p.dev));
    return s != RAGGED_OK ? status(s) : results({dq, dk, dv, dtable});
    END_HANDLE_TH_ERRORS
}

// q, k, lse, shared..., prev, weight -> (weight,)
PyObject* attn_weight(PyObject*, PyObject* const* o, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 3 + kShared + 2);
    const Tensor &q = tensor(o[0], "q"), &k = tensor(o[1], "k"), &lse = tensor(o[2], "lse");
    const Shared in(o + 3);
    no_graph({&q, &k, &lse, &in.table});
    TORCH_CHECK_VALUE(q.dim() == 3 && k.dim() == 3, "q must be [Tq, H, head_dim], k [Tk, Hkv, head_dim]");
    const int64_t H = q.size(1), Tk = k.size(0);
    const Tensor prev = maybe(o[3 + kShared], "prev");
    const Tensor weight = o[4 + kShared] == Py_None ? empty({H, Tk}, k, at::kFloat) : tensor(o[4 + kShared], "weight");
    if (o[4 + kShared] != Py_None) {
        const bool in_place = prev.defined() && prev.data_ptr() == weight.data_ptr() && prev.strides() == weight.strides();
        apart(weight, {&q, &k, &lse, &in.cu_q, &in.cu_k, &in.table, &in.buckets, &in.pos_q, &in.pos_k}, "weight");
        if (prev.defined() && !in_place) apart(weight, {&prev}, "weight");
    }
    Problem p(q, k, k, o + 3, in, lse);
    const int64_t stride = H > 1 ? weight.stride(0) : Tk;
    for (const Tensor* t : {&weight, &prev}) {
        if (!t->defined()) continue;
        TORCH_CHECK_VALUE(t->scalar_type() == at::kFloat && t->dim() == 2 && t->size(0) == H && t->size(1) == Tk &&
                              (Tk <= 1 || t->stride(1) == 1) && (H <= 1 || t->stride(0) == stride),
                          "weight and prev must be float32 [H, Tk] with unit innermost stride and the same strides");
        p.dev.add(*t);
    }
    TORCH_CHECK_VALUE(H <= 1 || stride >= Tk, "the rows of weight must not overlap");
    const void* some = p.a.cu_seqlens_q;
    const ragged_status s = g_lib.weight(&p.a, prev.defined() ? static_cast<const float*>(prev.data_ptr()) : nullptr,
                                         static_cast<float*>(address(weight, some)), stride, current_stream(p.dev));
    return s != RAGGED_OK ? status(s) : results({weight});
    END_HANDLE_TH_ERRORS
}

// rows, weight, cu_seqlens, max_seqlen, budget, sinks, recents, pos, total -> (rows_out, cu_out, src_idx, weight_out, pos_out)
PyObject* evict(PyObject*, PyObject* const* o, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 9);
    const Tensor rows = maybe(o[0], "rows"), pos = maybe(o[7], "pos");
    const Tensor &weight = tensor(o[1], "weight"), &cu = tensor(o[2], "cu_seqlens"), &budget = tensor(o[4], "budget");
    no_graph({&rows, &weight});
    TORCH_CHECK_VALUE(weight.scalar_type() == at::kFloat && weight.dim() == 2 && (weight.size(1) <= 1 || weight.stride(1) == 1),
                      "weight must be float32 [H, T] with unit innermost stride");
    const int64_t H = weight.size(0), T = weight.size(1), max_seqlen = integer(o[3]);
    TORCH_CHECK_VALUE(!rows.defined() || (rows.dim() >= 1 && rows.size(0) == T && rows.is_contiguous()), "rows must be contiguous [T, ...]");
    ints(cu, -1, "cu_seqlens");
    TORCH_CHECK_VALUE(cu.size(0) >= 1, "cu_seqlens must hold at least one value");
    const int64_t B = cu.size(0) - 1;
    ints(budget, B, "budget");
    if (pos.defined()) ints(pos, T, "pos");
    Devices dev;
    for (const Tensor* t : {&rows, &weight, &cu, &budget, &pos}) dev.add(*t);
    const int64_t total = o[8] == Py_None ? T : integer(o[8]);
    TORCH_CHECK_VALUE(total >= 0, "total is negative");
    Tensor rows_out;
    int64_t row_bytes = 0;
    if (rows.defined()) {
        auto size = rows.sizes().vec();
        size[0] = total;
        rows_out = empty(size, rows, rows.scalar_type());
        row_bytes = T > 0 ? rows.numel() / T * static_cast<int64_t>(rows.element_size()) : 0;
    }
    const Tensor cu_out = empty({B + 1}, cu, at::kInt), src = empty({total}, cu, at::kInt), pos_out = empty({total}, cu, at::kInt);
    const Tensor weight_out = empty({H, total}, weight, at::kFloat);
    Scratch ws;
    if (max_seqlen > RAGGED_EVICT_ONE_LAUNCH) ws.take(4 * T, weight);
    const bool copy = rows.defined() && total > 0 && T > 0;
    const void* some = cu.data_ptr();
    const ragged_status s = g_lib.evict(
        copy ? rows.data_ptr() : nullptr, row_bytes, static_cast<const float*>(address(weight, some)), H > 1 ? weight.stride(0) : 0, H, T,
        static_cast<const int32_t*>(some), B, max_seqlen, static_cast<const int32_t*>(address(budget, some)), integer(o[5]), integer(o[6]),
        pos.defined() && T > 0 ? static_cast<const int32_t*>(pos.data_ptr()) : nullptr, total, copy ? rows_out.data_ptr() : nullptr,
        static_cast<int32_t*>(cu_out.data_ptr()), static_cast<int32_t*>(src.data_ptr()), total > 0 ? static_cast<float*>(weight_out.data_ptr()) : nullptr, total,
        static_cast<int32_t*>(pos_out.data_ptr()), ws.p, ws.bytes, current_stream(dev));
    return s != RAGGED_OK ? status(s) : results({rows_out, cu_out, src, weight_out, pos_out});
    END_HANDLE_TH_ERRORS
}

// Addresses of the library's functions, in the order of Library.
PyObject* bind(PyObject*, PyObject* const* o, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 6);
    void* p[6];
    for (int i = 0; i < 6; ++i) p[i] = reinterpret_cast<void*>(integer(o[i]));
    g_lib = Library{reinterpret_cast<decltype(Library::fwd_workspace)>(p[0]), reinterpret_cast<decltype(Library::fwd)>(p[1]),
                    reinterpret_cast<decltype(Library::bwd_workspace)>(p[2]), reinterpret_cast<decltype(Library::bwd)>(p[3]),
                    reinterpret_cast<decltype(Library::weight)>(p[4]), reinterpret_cast<decltype(Library::evict)>(p[5])};
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(bias_fwd), METHOD(bias_bwd), METHOD(attn_weight), METHOD(evict), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torchcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// Of the torch that this was built against; the build and the binding look for it in the file.
const char kBuiltFor[] = "_torchcall for torch " RAGGED_TORCH_VERSION;

PyMODINIT_FUNC PyInit__torchcall(void) {
    PyObject* m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "built_for", kBuiltFor + sizeof("_torchcall for torch ") - 1) != 0) Py_CLEAR(m);
    return m;
}
