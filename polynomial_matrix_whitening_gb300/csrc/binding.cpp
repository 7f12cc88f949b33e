// binding.cpp -- the Python calls of the operators around the banks (anvil.py documents
// them): argument checks, allocation of the results and of the scratch, and the C ABI call.
//
// Native because these calls run ahead of kernels that may take two microseconds: the same
// checks and torch.empty calls from Python took 9 us per call on the GB300's host CPU.
// PyTorch's C++ API is used for what the Python binding uses it for elsewhere: tensors'
// pointers and shapes, the allocator, the current stream.  libanvil is loaded by anvil.py;
// set_library hands over its entry points.
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdarg.h>
#include <stdio.h>

#include <vector>

#include "../../include/anvil.h"

namespace {

struct Api {
    anvil_status (*layernorm_forward)(const anvil_layernorm_desc*, void*);
    size_t (*layernorm_backward_workspace_bytes)(const anvil_layernorm_grad_desc*);
    anvil_status (*layernorm_backward)(const anvil_layernorm_grad_desc*, void*, size_t, void*);
    size_t (*linear_workspace_bytes)(const anvil_linear_desc*);
    anvil_status (*linear_forward)(const anvil_linear_desc*, void*, size_t, void*);
    size_t (*linear_backward_workspace_bytes)(const anvil_linear_grad_desc*);
    anvil_status (*linear_backward)(const anvil_linear_grad_desc*, void*, size_t, void*);
    anvil_status (*token_logprobs)(const anvil_logprob_desc*, void*);
    anvil_status (*token_logprobs_backward)(const anvil_logprob_grad_desc*, void*);
    anvil_status (*adamw_step)(const anvil_adamw_tensor*, int, const anvil_adamw_config*, const float*, void*);
    anvil_status (*adamw_values)(const anvil_adamw_state*, int, void*);
    size_t (*gated_linear_workspace_bytes)(const anvil_gated_desc*);
    anvil_status (*gated_linear_forward)(const anvil_gated_desc*, void*, size_t, void*);
    size_t (*gated_linear_backward_workspace_bytes)(const anvil_gated_grad_desc*);
    anvil_status (*gated_linear_backward)(const anvil_gated_grad_desc*, void*, size_t, void*);
    size_t (*linear_cross_entropy_workspace_bytes)(const anvil_head_desc*);
    anvil_status (*linear_cross_entropy)(const anvil_head_desc*, void*, size_t, void*);
    size_t (*linear_cross_entropy_backward_workspace_bytes)(const anvil_head_grad_desc*);
    anvil_status (*linear_cross_entropy_backward)(const anvil_head_grad_desc*, void*, size_t, void*);
};
Api api;
PyObject* g_check = nullptr;          // Python: raises AnvilError(status, where)
PyObject* g_out_of_memory = nullptr;  // torch.OutOfMemoryError

// Thrown where a Python error is already set.
struct PyError {};

[[noreturn]] void refuse(const char* format, ...) {
    char text[256];
    va_list args;
    va_start(args, format);
    vsnprintf(text, sizeof(text), format, args);
    va_end(args);
    PyErr_SetString(PyExc_ValueError, text);
    throw PyError();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) refuse("%s must be a tensor", what);
    return THPVariable_Unpack(o);
}
// An optional tensor: null for None.
const at::Tensor* maybe(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }

int dtype_code(const at::Tensor& t, const char* what) {
    switch (t.scalar_type()) {
        case at::kFloat: return ANVIL_F32;
        case at::kBFloat16: return ANVIL_BF16;
        case at::kHalf: return ANVIL_F16;
        default: refuse("%s must be fp32, bf16 or fp16, not %s", what, c10::toString(t.scalar_type()));
    }
}

// A tensor [..., width] as a matrix of contiguous rows with one stride.
struct Rows {
    int64_t rows, ld;
    int64_t width;
};
Rows rows_of(const at::Tensor& t, const char* what) {
    const auto sizes = t.sizes();
    const auto strides = t.strides();
    const int64_t d = t.dim();
    if (d < 1) refuse("%s must have at least one dimension", what);
    Rows r = {1, 0, sizes[d - 1]};
    for (int64_t i = d - 2; i >= 0; --i) {
        if (sizes[i] == 1) continue;
        if (r.rows == 1) r.ld = strides[i];
        else if (sizes[i] && r.rows && strides[i] != r.ld * r.rows)
            refuse("%s: leading dimensions without one common row stride; use .contiguous()", what);
        r.rows *= sizes[i];
    }
    if (strides[d - 1] != 1 && r.width > 1 && r.rows)
        refuse("%s: rows must be contiguous (last stride 1); use .contiguous()", what);
    if (r.ld < r.width) {
        if (r.rows > 1)
            refuse("%s: rows overlap (row stride %lld, width %lld); use .contiguous()", what, static_cast<long long>(r.ld),
                   static_cast<long long>(r.width));
        r.ld = r.width;
    }
    return r;
}

// A width, row length or column count as the C ABI's int.
int as_int(int64_t v, const char* what) {
    if (v > INT32_MAX) refuse("%s is too large", what);
    return static_cast<int>(v);
}

void* vector(const at::Tensor* t, int64_t n, at::ScalarType a, at::ScalarType b, const char* what) {
    if (!t) return nullptr;
    if ((t->scalar_type() != a && t->scalar_type() != b) || t->dim() != 1 || t->size(0) != n || (n > 1 && t->stride(0) != 1))
        refuse("%s must be a contiguous vector of %lld values of %s%s%s", what, static_cast<long long>(n), c10::toString(a),
               a == b ? "" : " or ", a == b ? "" : c10::toString(b));
    return t->data_ptr();
}

float* per_row(const at::Tensor* t, int64_t rows, const char* what) {
    if (!t) return nullptr;
    if (t->scalar_type() != at::kFloat || t->numel() != rows || !t->is_contiguous())
        refuse("%s must be contiguous fp32, one value per row", what);
    return static_cast<float*>(t->data_ptr());
}

void same_form(const at::Tensor& t, at::IntArrayRef sizes, at::ScalarType type, const char* what, const char* like) {
    if (t.scalar_type() != type || t.sizes() != sizes) refuse("%s must have %s", what, like);
}

// The current stream, after checking that every tensor is on the current GPU, and that none
// asks for a gradient that autograd would not get: the calls record nothing.
struct Here {
    void* stream;
    at::Device device;
    Here(const char* what, std::initializer_list<const at::Tensor*> tensors) : stream(nullptr), device(at::kCUDA, 0) {
        if (c10::GradMode::is_enabled()) {
            for (const at::Tensor* t : tensors)
                if (t && t->requires_grad())
                    refuse("%s: a tensor requires grad, but autograd records nothing of the call; use torch.no_grad() "
                           "(an autograd.Function runs under it) and the backward call", what);
        }
        const at::Tensor* first = *tensors.begin();
        if (!first->is_cuda()) refuse("%s: every tensor must be on the current CUDA device", what);
        device = at::Device(at::kCUDA, c10::cuda::current_device());
        for (const at::Tensor* t : tensors)
            if (t && t->device() != device) refuse("%s: every tensor must be on the current CUDA device", what);
        stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    }
    at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type) const {
        return at::empty(sizes, at::TensorOptions().dtype(type).device(device));
    }
};

// Small results of 4-byte values that share one allocation (an allocation costs the host about
// a microsecond, as much as the smallest kernels).
struct Together {
    at::Tensor all;
    int64_t used = 0;
    Together(int64_t values, const Here& here) : all(here.empty({values}, at::kFloat)) {}
    at::Tensor next(at::IntArrayRef sizes, at::ScalarType type, int64_t values) {
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                                c10::scalarTypeToTypeMeta(type));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
        t.unsafeGetTensorImpl()->set_storage_offset(used);
        used += values;
        return t;
    }
};

// A call's scratch: the caller's, or a new one (kept until the call is queued).
struct Scratch {
    at::Tensor keep;
    void* p = nullptr;
    size_t bytes = 0;
    Scratch(size_t need, const at::Tensor* given, const Here& here) {
        if (given) {
            if (!given->is_contiguous()) refuse("workspace: every tensor must be contiguous");
            p = given->data_ptr();
            bytes = static_cast<size_t>(given->numel()) * given->element_size();
        } else if (need) {
            keep = here.empty({static_cast<int64_t>(need)}, at::kByte);
            p = keep.data_ptr();
            bytes = need;
        }
    }
};

void check(anvil_status st, const char* where) {
    if (st == ANVIL_OK) return;
    PyObject* r = PyObject_CallFunction(g_check, "is", static_cast<int>(st), where);
    Py_XDECREF(r);
    throw PyError();
}

void need_args(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        throw PyError();
    }
}
bool truth(PyObject* o) {
    const int r = PyObject_IsTrue(o);
    if (r < 0) throw PyError();
    return r != 0;
}

PyObject* wrap(at::Tensor t) { return t.defined() ? THPVariable_Wrap(std::move(t)) : Py_NewRef(Py_None); }
template <typename... Ts>
PyObject* tuple_of(Ts... items) {
    PyObject* objs[] = {wrap(std::move(items))...};
    const Py_ssize_t n = sizeof...(Ts);
    PyObject* t = PyTuple_New(n);
    for (Py_ssize_t i = 0; i < n; ++i) PyTuple_SET_ITEM(t, i, objs[i]);
    return t;
}

// The caller's result or a new contiguous one.
at::Tensor result(const at::Tensor* out, at::IntArrayRef sizes, at::ScalarType type, const char* like, int64_t* ld,
                  const Here& here) {
    if (!out) {
        *ld = sizes.back();
        return here.empty(sizes, type);
    }
    same_form(*out, sizes, type, "out", like);
    *ld = rows_of(*out, "out").ld;
    return *out;
}

// ---------------------------------------------------------------- layer norm
// (x, weight, bias, eps, out) -> (y, mean, rstd)
PyObject* layernorm_forward(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor *weight = maybe(a[1], "weight"), *bias = maybe(a[2], "bias"), *out = maybe(a[4], "out");
    anvil_layernorm_desc d = {};
    d.eps = static_cast<float>(PyFloat_AsDouble(a[3]));
    if (PyErr_Occurred()) throw PyError();
    d.dtype = dtype_code(x, "x");
    const Rows r = rows_of(x, "x");
    const at::ScalarType type = x.scalar_type();
    const at::ScalarType wt = weight ? weight->scalar_type() : bias ? bias->scalar_type() : type;
    if (wt != type && wt != at::kFloat) refuse("weight and bias must be fp32 or of x's type");
    d.weight_dtype = wt == type ? d.dtype : ANVIL_F32;
    d.weight = vector(weight, r.width, wt, wt, "weight");
    d.bias = vector(bias, r.width, wt, wt, "bias");
    const Here here("layernorm_forward", {&x, weight, bias, out});
    at::Tensor y = result(out, x.sizes(), type, "x's shape and type", &d.ldy, here);
    const auto lead = x.sizes().slice(0, x.dim() - 1);
    Together stats(2 * r.rows, here);
    at::Tensor mean = stats.next(lead, at::kFloat, r.rows), rstd = stats.next(lead, at::kFloat, r.rows);
    d.x = x.data_ptr();
    d.y = y.data_ptr();
    d.mean = static_cast<float*>(mean.data_ptr());
    d.rstd = static_cast<float*>(rstd.data_ptr());
    d.rows = r.rows;
    d.ldx = r.ld;
    d.width = as_int(r.width, "x's width");
    check(api.layernorm_forward(&d, here.stream), "anvil_layernorm_forward");
    return tuple_of(std::move(y), std::move(mean), std::move(rstd));
}

// (dy, x, mean, rstd, weight, residual_grad, out, weight_grads, workspace) -> (dx, dweight, dbias)
PyObject* layernorm_backward(PyObject* const* a) {
    const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x"), &mean = tensor(a[2], "mean"), &rstd = tensor(a[3], "rstd");
    const at::Tensor *weight = maybe(a[4], "weight"), *res = maybe(a[5], "residual_grad"), *out = maybe(a[6], "out"),
                     *ws = maybe(a[8], "workspace");
    const bool grads = truth(a[7]);
    anvil_layernorm_grad_desc d = {};
    d.dtype = dtype_code(x, "x");
    const Rows r = rows_of(x, "x");
    const at::ScalarType type = x.scalar_type();
    same_form(dy, x.sizes(), type, "dy", "x's shape and type");
    d.lddy = rows_of(dy, "dy").ld;
    if (res) {
        same_form(*res, x.sizes(), type, "residual_grad", "x's shape and type");
        d.ldr = rows_of(*res, "residual_grad").ld;
        d.residual_grad = res->data_ptr();
    }
    d.mean = per_row(&mean, r.rows, "mean");
    d.rstd = per_row(&rstd, r.rows, "rstd");
    d.weight_dtype = d.dtype;
    if (weight) {
        if (weight->scalar_type() != type) {
            if (weight->scalar_type() != at::kFloat) refuse("weight must be fp32 or of x's type");
            d.weight_dtype = ANVIL_F32;
        }
        d.weight = vector(weight, r.width, weight->scalar_type(), weight->scalar_type(), "weight");
    }
    const Here here("layernorm_backward", {&x, &dy, &mean, &rstd, weight, res, out, ws});
    at::Tensor dx = result(out, x.sizes(), type, "x's shape and type", &d.lddx, here), dw, db;
    if (grads) {
        dw = here.empty({r.width}, at::kFloat);
        db = here.empty({r.width}, at::kFloat);
        d.dweight = static_cast<float*>(dw.data_ptr());
        d.dbias = static_cast<float*>(db.data_ptr());
    }
    d.dy = dy.data_ptr();
    d.x = x.data_ptr();
    d.dx = dx.data_ptr();
    d.rows = r.rows;
    d.ldx = r.ld;
    d.width = as_int(r.width, "x's width");
    const Scratch scratch(ws ? 0 : api.layernorm_backward_workspace_bytes(&d), ws, here);
    check(api.layernorm_backward(&d, scratch.p, scratch.bytes, here.stream), "anvil_layernorm_backward");
    return tuple_of(std::move(dx), std::move(dw), std::move(db));
}

// ---------------------------------------------------------------- the linear layer
struct Weight {
    int64_t n, k, ld;
    int transposed;
};
// The leading dimension of w [n, k] stored by rows (by columns: as [k, n]); -1: it is not stored
// so.  A single row or column is stored in both orders, each with its own leading dimension.
int64_t ld_in_order(const at::Tensor& w, int by_columns) {
    const int64_t inner = w.size(by_columns ? 0 : 1), outer = w.size(by_columns ? 1 : 0);
    const int64_t step = w.stride(by_columns ? 0 : 1), ld = w.stride(by_columns ? 1 : 0);
    if ((step != 1 && inner > 1) || (ld < inner && outer > 1)) return -1;
    return ld > inner ? ld : inner;
}
Weight weight_of(const at::Tensor& w, at::ScalarType type, const char* what) {
    if (w.dim() != 2 || w.scalar_type() != type) refuse("%s must be [n, k] of %s", what, c10::toString(type));
    for (int by_columns = 0; by_columns < 2; ++by_columns) {
        const int64_t ld = ld_in_order(w, by_columns);
        if (ld >= 0) return {w.size(0), w.size(1), ld, by_columns};
    }
    refuse("%s must be stored by rows or by columns; use .contiguous()", what);
}

// The weight's gradient: the caller's, in weight's order (m changes to the other one where both are
// stored so too: single rows), or a new one.
at::Tensor dweight_like(const at::Tensor& w, Weight* m, const at::Tensor* given, at::ScalarType type, const Here& here, int64_t* ld) {
    if (!given) {
        *ld = m->transposed ? m->n : m->k;
        return m->transposed ? here.empty({m->k, m->n}, type).t() : here.empty({m->n, m->k}, type);
    }
    const Weight g = weight_of(*given, type, "dweight");
    if (ld_in_order(*given, m->transposed) < 0 && ld_in_order(w, !m->transposed) >= 0) {
        m->transposed = !m->transposed;
        m->ld = ld_in_order(w, m->transposed);
    }
    *ld = ld_in_order(*given, m->transposed);
    if (g.n != m->n || g.k != m->k || *ld < 0) refuse("dweight must have weight's shape and order");
    return *given;
}

// (x, weight, bias, activation, residual, save_preact, out, workspace) -> (y, z or None)
PyObject* linear_forward(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight");
    const at::Tensor *bias = maybe(a[2], "bias"), *res = maybe(a[4], "residual"), *out = maybe(a[6], "out"),
                     *ws = maybe(a[7], "workspace");
    anvil_linear_desc d = {};
    d.activation = static_cast<int>(PyLong_AsLong(a[3]));
    d.dtype = dtype_code(x, "x");
    if (d.dtype == ANVIL_F32) refuse("x must be bf16 or fp16");
    const at::ScalarType type = x.scalar_type();
    const Rows r = rows_of(x, "x");
    const Weight m = weight_of(w, type, "weight");
    if (m.k != r.width) refuse("weight must be [n, %lld]", static_cast<long long>(r.width));
    d.bias = vector(bias, m.n, type, at::kFloat, "bias");
    d.bias_dtype = bias && bias->scalar_type() != type ? ANVIL_F32 : d.dtype;
    c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = m.n;
    if (res) {
        same_form(*res, shape, type, "residual", "the result's shape and type");
        d.ldr = rows_of(*res, "residual").ld;
        d.residual = res->data_ptr();
    }
    const Here here("linear_forward", {&x, &w, bias, res, out, ws});
    at::Tensor y = result(out, shape, type, "the result's shape and type", &d.ldy, here), z;
    if (truth(a[5])) {
        z = here.empty(shape, type);
        d.preact = z.data_ptr();
        d.ldz = m.n;
    }
    d.x = x.data_ptr();
    d.weight = w.data_ptr();
    d.y = y.data_ptr();
    d.rows = r.rows;
    d.ldx = r.ld;
    d.ldw = m.ld;
    d.n = as_int(m.n, "weight");
    d.k = as_int(m.k, "weight");
    d.weight_transposed = m.transposed;
    const Scratch scratch(ws ? 0 : api.linear_workspace_bytes(&d), ws, here);
    check(api.linear_forward(&d, scratch.p, scratch.bytes, here.stream), "anvil_linear_forward");
    return tuple_of(std::move(y), std::move(z));
}

// (dy, x, weight, preact, activation, need_dx, need_dweight, bias_grad, dweight fp32 (None:
// x's type), dweight, dbias, accumulate, workspace, dz in two parts) -> (dx, dweight, dbias)
PyObject* linear_backward(PyObject* const* a) {
    const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x"), &w = tensor(a[2], "weight");
    const at::Tensor *z = maybe(a[3], "preact"), *dw_in = maybe(a[9], "dweight"), *db_in = maybe(a[10], "dbias"),
                     *ws = maybe(a[12], "workspace");
    const bool need_dx = truth(a[5]), need_dw = truth(a[6]), need_db = truth(a[7]);
    anvil_linear_grad_desc d = {};
    d.activation = static_cast<int>(PyLong_AsLong(a[4]));
    d.dtype = dtype_code(x, "x");
    if (d.dtype == ANVIL_F32) refuse("x must be bf16 or fp16");
    const at::ScalarType type = x.scalar_type();
    const Rows r = rows_of(x, "x");
    Weight m = weight_of(w, type, "weight");
    if (m.k != r.width) refuse("weight must be [n, %lld]", static_cast<long long>(r.width));
    c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = m.n;
    same_form(dy, shape, type, "dy", "the forward result's shape and type");
    d.lddy = rows_of(dy, "dy").ld;
    if (d.activation) {
        if (!z) refuse("preact is needed with an activation");
        same_form(*z, shape, type, "preact", "the forward result's shape and type");
        d.ldz = rows_of(*z, "preact").ld;
        d.preact = z->data_ptr();
    }
    d.accumulate = truth(a[11]);
    if (d.accumulate && ((need_dw && !dw_in) || (need_db && !db_in))) refuse("accumulate needs dweight and dbias to add to");
    at::ScalarType wt = type;
    if (dw_in) {
        wt = dw_in->scalar_type();
        if (wt != type && wt != at::kFloat) refuse("dweight must be fp32 or of x's type");
    } else if (truth(a[8])) {
        wt = at::kFloat;
    }
    const Here here("linear_backward", {&x, &dy, &w, z, dw_in, db_in, ws});
    at::Tensor dx, dw, db;
    if (need_dx) {
        dx = here.empty(x.sizes(), type);
        d.dx = dx.data_ptr();
        d.lddx = m.k;
    }
    if (need_dw) {
        dw = dweight_like(w, &m, dw_in, wt, here, &d.lddw);
        d.dweight = dw.data_ptr();
    }
    if (need_db) {
        db = db_in ? *db_in : here.empty({m.n}, at::kFloat);
        d.dbias = static_cast<float*>(vector(&db, m.n, at::kFloat, at::kFloat, "dbias"));
    }
    d.dy = dy.data_ptr();
    d.x = x.data_ptr();
    d.weight = w.data_ptr();
    d.rows = r.rows;
    d.ldx = r.ld;
    d.ldw = m.ld;
    d.n = as_int(m.n, "weight");
    d.k = as_int(m.k, "weight");
    d.dweight_dtype = wt == type ? d.dtype : ANVIL_F32;
    d.weight_transposed = m.transposed;
    if (truth(a[13])) d.activation |= ANVIL_DZ_TWO_PARTS;
    const Scratch scratch(ws ? 0 : api.linear_backward_workspace_bytes(&d), ws, here);
    check(api.linear_backward(&d, scratch.p, scratch.bytes, here.stream), "anvil_linear_backward");
    return tuple_of(std::move(dx), std::move(dw), std::move(db));
}

// A tensor of the caller's that a call has written to: a graph that saved it would use the new values.
void overwritten(const at::Tensor* t) {
    if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// The same for many tensors, known before the call.
struct Written {
    std::vector<c10::TensorImpl*> all;
    explicit Written(Py_ssize_t most) { all.reserve(static_cast<size_t>(most)); }
    void add(const at::Tensor* t) {
        if (t && !t->is_inference()) all.push_back(t->unsafeGetTensorImpl());
    }
    void done() const {
        for (c10::TensorImpl* t : all) t->bump_version();
    }
};

// ---------------------------------------------------------------- the gated layer
// The order (0 by rows, 1 by columns) that every given matrix of gate's shape is stored in.
int common_order(const at::Tensor& gate, at::ScalarType type, int64_t k, std::initializer_list<const at::Tensor*> others) {
    if (gate.dim() != 2 || gate.scalar_type() != type || gate.size(1) != k)
        refuse("gate and up must be [n, %lld] of %s", static_cast<long long>(k), c10::toString(type));
    for (const at::Tensor* t : others)
        if (t && t->sizes() != gate.sizes()) refuse("up, dgate and dup must have gate's shape");
    for (int by_columns = 0; by_columns < 2; ++by_columns) {
        bool all = ld_in_order(gate, by_columns) >= 0;
        for (const at::Tensor* t : others) all = all && (!t || ld_in_order(*t, by_columns) >= 0);
        if (all) return by_columns;
    }
    refuse("gate, up, dgate and dup must be stored all by rows or all by columns");
}

// (x, gate, up, activation, save_preact, out, workspace) -> (y, g or None, u or None)
PyObject* gated_linear_forward(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0], "x"), &gate = tensor(a[1], "gate"), &up = tensor(a[2], "up");
    const at::Tensor *out = maybe(a[5], "out"), *ws = maybe(a[6], "workspace");
    anvil_gated_desc d = {};
    d.activation = static_cast<int>(PyLong_AsLong(a[3]));
    d.dtype = dtype_code(x, "x");
    if (d.dtype == ANVIL_F32) refuse("x must be bf16 or fp16");
    const at::ScalarType type = x.scalar_type();
    const Rows r = rows_of(x, "x");
    if (up.scalar_type() != type) refuse("gate and up must be of x's type");
    d.weight_transposed = common_order(gate, type, r.width, {&up});
    const int64_t n = gate.size(0);
    c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = n;
    const Here here("gated_linear_forward", {&x, &gate, &up, out, ws});
    at::Tensor y = result(out, shape, type, "the result's shape and type", &d.ldy, here), g, u;
    if (truth(a[4])) {
        g = here.empty(shape, type);
        u = here.empty(shape, type);
        d.preact_gate = g.data_ptr();
        d.preact_up = u.data_ptr();
        d.ldzg = d.ldzu = n;
    }
    d.x = x.data_ptr();
    d.gate = gate.data_ptr();
    d.up = up.data_ptr();
    d.y = y.data_ptr();
    d.rows = r.rows;
    d.ldx = r.ld;
    d.ldgate = ld_in_order(gate, d.weight_transposed);
    d.ldup = ld_in_order(up, d.weight_transposed);
    d.n = as_int(n, "gate");
    d.k = as_int(r.width, "gate");
    const Scratch scratch(ws ? 0 : api.gated_linear_workspace_bytes(&d), ws, here);
    check(api.gated_linear_forward(&d, scratch.p, scratch.bytes, here.stream), "anvil_gated_linear_forward");
    overwritten(out);
    return tuple_of(std::move(y), std::move(g), std::move(u));
}

// (dy, x, gate, up, g, u, activation, need_dx, need_dweight, dweight fp32 (None: x's type), dgate, dup, accumulate,
// workspace, dz in two parts) -> (dx, dgate, dup)
PyObject* gated_linear_backward(PyObject* const* a) {
    const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x"), &gate = tensor(a[2], "gate"), &up = tensor(a[3], "up"),
                     &zg = tensor(a[4], "preact_gate"), &zu = tensor(a[5], "preact_up");
    const at::Tensor *dg_in = maybe(a[10], "dgate"), *du_in = maybe(a[11], "dup"), *ws = maybe(a[13], "workspace");
    const bool need_dx = truth(a[7]), need_dw = truth(a[8]);
    anvil_gated_grad_desc d = {};
    d.activation = static_cast<int>(PyLong_AsLong(a[6]));
    d.dtype = dtype_code(x, "x");
    if (d.dtype == ANVIL_F32) refuse("x must be bf16 or fp16");
    const at::ScalarType type = x.scalar_type();
    const Rows r = rows_of(x, "x");
    if (up.scalar_type() != type) refuse("gate and up must be of x's type");
    if ((dg_in != nullptr) != (du_in != nullptr)) refuse("dgate and dup must be given together");
    d.weight_transposed = common_order(gate, type, r.width, {&up, need_dw ? dg_in : nullptr, need_dw ? du_in : nullptr});
    const int64_t n = gate.size(0);
    c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = n;
    same_form(dy, shape, type, "dy", "the forward result's shape and type");
    same_form(zg, shape, type, "preact_gate", "the forward result's shape and type");
    same_form(zu, shape, type, "preact_up", "the forward result's shape and type");
    d.lddy = rows_of(dy, "dy").ld;
    d.ldzg = rows_of(zg, "preact_gate").ld;
    d.ldzu = rows_of(zu, "preact_up").ld;
    d.accumulate = truth(a[12]);
    if (d.accumulate && need_dw && !dg_in) refuse("accumulate needs dgate and dup to add to");
    at::ScalarType wt = type;
    if (dg_in) {
        wt = dg_in->scalar_type();
        if ((wt != type && wt != at::kFloat) || du_in->scalar_type() != wt) refuse("dgate and dup must be both fp32 or both of x's type");
    } else if (truth(a[9])) {
        wt = at::kFloat;
    }
    const Here here("gated_linear_backward", {&x, &dy, &gate, &up, &zg, &zu, dg_in, du_in, ws});
    at::Tensor dx, dg, du;
    if (need_dx) {
        dx = here.empty(x.sizes(), type);
        d.dx = dx.data_ptr();
        d.lddx = r.width;
    }
    if (need_dw) {
        const auto make = [&] { return d.weight_transposed ? here.empty({r.width, n}, wt).t() : here.empty({n, r.width}, wt); };
        dg = dg_in ? *dg_in : make();
        du = du_in ? *du_in : make();
        d.dgate = dg.data_ptr();
        d.dup = du.data_ptr();
        d.lddgate = ld_in_order(dg, d.weight_transposed);
        d.lddup = ld_in_order(du, d.weight_transposed);
    }
    d.dy = dy.data_ptr();
    d.x = x.data_ptr();
    d.gate = gate.data_ptr();
    d.up = up.data_ptr();
    d.preact_gate = zg.data_ptr();
    d.preact_up = zu.data_ptr();
    d.rows = r.rows;
    d.ldx = r.ld;
    d.ldgate = ld_in_order(gate, d.weight_transposed);
    d.ldup = ld_in_order(up, d.weight_transposed);
    d.n = as_int(n, "gate");
    d.k = as_int(r.width, "gate");
    d.dweight_dtype = wt == type ? d.dtype : ANVIL_F32;
    if (truth(a[14])) d.activation |= ANVIL_DZ_TWO_PARTS;
    const Scratch scratch(ws ? 0 : api.gated_linear_backward_workspace_bytes(&d), ws, here);
    check(api.gated_linear_backward(&d, scratch.p, scratch.bytes, here.stream), "anvil_gated_linear_backward");
    if (need_dw) {
        overwritten(dg_in);
        overwritten(du_in);
    }
    return tuple_of(std::move(dx), std::move(dg), std::move(du));
}

// ---------------------------------------------------------------- token log probabilities
const void* targets_of(const at::Tensor* t, int64_t rows, int* wide) {
    if (!t) return nullptr;
    *wide = t->scalar_type() == at::kLong;
    if ((!*wide && t->scalar_type() != at::kInt) || t->numel() != rows || !t->is_contiguous())
        refuse("targets must be contiguous int64 or int32, one per row");
    return t->data_ptr();
}

// (logits, targets, top) -> (logprob, entropy, lse, top_logprob, top_index)
PyObject* token_logprobs(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0], "logits");
    const at::Tensor* t = maybe(a[1], "targets");
    const long top = PyLong_AsLong(a[2]);
    if (top == -1 && PyErr_Occurred()) throw PyError();
    anvil_logprob_desc d = {};
    d.dtype = dtype_code(x, "logits");
    const Rows r = rows_of(x, "logits");
    if (top < 0 || top > ANVIL_MAX_TOP || top > r.width)
        refuse("top must be between 0 and %d and at most the vocabulary", ANVIL_MAX_TOP);
    d.targets = targets_of(t, r.rows, &d.targets_int64);
    const Here here("token_logprobs", {&x, t});
    const auto lead = x.sizes().slice(0, x.dim() - 1);
    const int64_t best = r.rows * top;
    Together results((t ? 3 : 2) * r.rows + 2 * best, here);
    at::Tensor lse = results.next(lead, at::kFloat, r.rows), ent = results.next(lead, at::kFloat, r.rows), lp, tv, ti;
    if (t) {
        lp = results.next(lead, at::kFloat, r.rows);
        d.logprob = static_cast<float*>(lp.data_ptr());
    }
    if (top) {
        c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
        shape.back() = top;
        tv = results.next(shape, at::kFloat, best);
        ti = results.next(shape, at::kInt, best);
        d.top_logprob = static_cast<float*>(tv.data_ptr());
        d.top_index = static_cast<int32_t*>(ti.data_ptr());
    }
    d.logits = x.data_ptr();
    d.entropy = static_cast<float*>(ent.data_ptr());
    d.lse = static_cast<float*>(lse.data_ptr());
    d.rows = r.rows;
    d.ld = r.ld;
    d.vocab = as_int(r.width, "the vocabulary");
    d.top = static_cast<int>(top);
    check(api.token_logprobs(&d, here.stream), "anvil_token_logprobs");
    return tuple_of(std::move(lp), std::move(ent), std::move(lse), std::move(tv), std::move(ti));
}

// (logits, targets, lse, grad_logprob, entropy, grad_entropy, out) -> dlogits
PyObject* token_logprobs_backward(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0], "logits");
    const at::Tensor *t = maybe(a[1], "targets"), *lse = maybe(a[2], "lse"), *gl = maybe(a[3], "grad_logprob"),
                     *ent = maybe(a[4], "entropy"), *gh = maybe(a[5], "grad_entropy"), *out = maybe(a[6], "out");
    anvil_logprob_grad_desc d = {};
    d.dtype = dtype_code(x, "logits");
    const Rows r = rows_of(x, "logits");
    d.targets = targets_of(t, r.rows, &d.targets_int64);
    if (gl && !t) refuse("grad_logprob needs targets");
    if (gh && !ent) refuse("grad_entropy needs entropy");
    if (!lse) refuse("lse is needed");
    d.lse = per_row(lse, r.rows, "lse");
    d.entropy = per_row(ent, r.rows, "entropy");
    d.grad_logprob = per_row(gl, r.rows, "grad_logprob");
    d.grad_entropy = per_row(gh, r.rows, "grad_entropy");
    const Here here("token_logprobs_backward", {&x, t, lse, gl, ent, gh, out});
    at::Tensor dl = result(out, x.sizes(), x.scalar_type(), "the logits' shape and type", &d.ldd, here);
    d.logits = x.data_ptr();
    d.dlogits = dl.data_ptr();
    d.rows = r.rows;
    d.ld = r.ld;
    d.vocab = as_int(r.width, "the vocabulary");
    check(api.token_logprobs_backward(&d, here.stream), "anvil_token_logprobs_backward");
    return wrap(std::move(dl));
}

// ---------------------------------------------------------------- the head's cross entropy
// (x, weight, targets, workspace) -> (loss or None, lse)
PyObject* linear_cross_entropy(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight");
    const at::Tensor *t = maybe(a[2], "targets"), *ws = maybe(a[3], "workspace");
    anvil_head_desc d = {};
    d.dtype = dtype_code(x, "x");
    if (d.dtype == ANVIL_F32) refuse("x must be bf16 or fp16");
    const Rows r = rows_of(x, "x");
    const Weight m = weight_of(w, x.scalar_type(), "weight");
    if (m.k != r.width) refuse("weight must be [vocab, %lld]", static_cast<long long>(r.width));
    d.targets = targets_of(t, r.rows, &d.targets_int64);
    const Here here("linear_cross_entropy", {&x, &w, t, ws});
    const auto lead = x.sizes().slice(0, x.dim() - 1);
    Together results((t ? 2 : 1) * r.rows, here);
    at::Tensor lse = results.next(lead, at::kFloat, r.rows), loss;
    if (t) {
        loss = results.next(lead, at::kFloat, r.rows);
        d.loss = static_cast<float*>(loss.data_ptr());
    }
    d.x = x.data_ptr();
    d.weight = w.data_ptr();
    d.lse = static_cast<float*>(lse.data_ptr());
    d.rows = r.rows;
    d.ldx = r.ld;
    d.ldw = m.ld;
    d.vocab = as_int(m.n, "weight");
    d.k = as_int(m.k, "weight");
    d.weight_transposed = m.transposed;
    const Scratch scratch(ws ? 0 : api.linear_cross_entropy_workspace_bytes(&d), ws, here);
    check(api.linear_cross_entropy(&d, scratch.p, scratch.bytes, here.stream), "anvil_linear_cross_entropy");
    return tuple_of(std::move(loss), std::move(lse));
}

// (x, weight, targets, lse, grad_loss, need_dx, need_dweight, dweight fp32 (None: x's type), dweight, accumulate, workspace)
// -> (dx, dweight)
PyObject* linear_cross_entropy_backward(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight"), &t = tensor(a[2], "targets"), &lse = tensor(a[3], "lse"),
                     &gl = tensor(a[4], "grad_loss");
    const at::Tensor *dw_in = maybe(a[8], "dweight"), *ws = maybe(a[10], "workspace");
    const bool need_dx = truth(a[5]), need_dw = truth(a[6]);
    anvil_head_grad_desc d = {};
    d.dtype = dtype_code(x, "x");
    if (d.dtype == ANVIL_F32) refuse("x must be bf16 or fp16");
    const at::ScalarType type = x.scalar_type();
    const Rows r = rows_of(x, "x");
    Weight m = weight_of(w, type, "weight");
    if (m.k != r.width) refuse("weight must be [vocab, %lld]", static_cast<long long>(r.width));
    d.targets = targets_of(&t, r.rows, &d.targets_int64);
    d.lse = per_row(&lse, r.rows, "lse");
    d.grad_loss = per_row(&gl, r.rows, "grad_loss");
    d.accumulate = truth(a[9]);
    if (d.accumulate && need_dw && !dw_in) refuse("accumulate needs dweight to add to");
    at::ScalarType wt = type;
    if (dw_in) {
        wt = dw_in->scalar_type();
        if (wt != type && wt != at::kFloat) refuse("dweight must be fp32 or of x's type");
    } else if (truth(a[7])) {
        wt = at::kFloat;
    }
    const Here here("linear_cross_entropy_backward", {&x, &w, &t, &lse, &gl, dw_in, ws});
    at::Tensor dx, dw;
    if (need_dx) {
        dx = here.empty(x.sizes(), type);
        d.dx = dx.data_ptr();
        d.lddx = m.k;
    }
    if (need_dw) {
        dw = dweight_like(w, &m, dw_in, wt, here, &d.lddw);
        d.dweight = dw.data_ptr();
    }
    d.x = x.data_ptr();
    d.weight = w.data_ptr();
    d.rows = r.rows;
    d.ldx = r.ld;
    d.ldw = m.ld;
    d.vocab = as_int(m.n, "weight");
    d.k = as_int(m.k, "weight");
    d.weight_transposed = m.transposed;
    d.dweight_dtype = wt == type ? d.dtype : ANVIL_F32;
    const Scratch scratch(ws ? 0 : api.linear_cross_entropy_backward_workspace_bytes(&d), ws, here);
    check(api.linear_cross_entropy_backward(&d, scratch.p, scratch.bytes, here.stream), "anvil_linear_cross_entropy_backward");
    if (need_dw) overwritten(dw_in);
    return tuple_of(std::move(dx), std::move(dw));
}

// ---------------------------------------------------------------- AdamW
// A list or tuple of tensors (of `n`, or any number where n < 0); items may be None where `gaps`.
struct Tensors {
    PyObject* seq;
    Py_ssize_t n;
    bool gaps;
    const char* what;
    Tensors(PyObject* o, Py_ssize_t want, bool may_be_none, const char* name) : seq(nullptr), n(want), gaps(may_be_none), what(name) {
        if (o == Py_None && gaps) return;
        if (!PyList_Check(o) && !PyTuple_Check(o)) refuse("%s must be a list of tensors", what);
        seq = o;
        n = PySequence_Fast_GET_SIZE(o);
        if (want >= 0 && n != want) refuse("%s must have one tensor for each of params", what);
    }
    const at::Tensor* at(Py_ssize_t i) const {
        PyObject* o = seq ? PySequence_Fast_GET_ITEM(seq, i) : Py_None;
        if (o == Py_None && gaps) return nullptr;
        if (!THPVariable_Check(o)) refuse("%s must be a list of tensors", what);
        return &THPVariable_Unpack(o);
    }
};
void plain_tensor(const at::Tensor& t, at::Device device, int64_t count, const char* where, const char* what) {
    if (t.device() != device) refuse("%s: every tensor must be on the current CUDA device", where);
    if (!t.is_contiguous()) refuse("%s: %s must be contiguous", where, what);
    if (t.numel() != count) refuse("%s: %s must have its parameter's size", where, what);
}
// The codes and their scales, checked against a count.
void check_codes(const at::Tensor& m, const at::Tensor& v, const at::Tensor& scales, int64_t count, at::Device device, const char* where) {
    if (m.scalar_type() != at::kFloat8_e4m3fn || v.scalar_type() != at::kByte)
        refuse("%s: with scales exp_avg must be float8_e4m3fn and exp_avg_sq uint8", where);
    const int64_t blocks = (count + ANVIL_ADAMW_BLOCK - 1) / ANVIL_ADAMW_BLOCK;
    plain_tensor(scales, device, 2 * blocks, where, "scales, [2, blocks],");
    if (scales.scalar_type() != at::kFloat) refuse("%s: scales must be fp32", where);
}
at::Device current(const char* where, const at::Tensor* first) {
    if (!first || !first->is_cuda()) refuse("%s: every tensor must be on the current CUDA device", where);
    return at::Device(at::kCUDA, c10::cuda::current_device());
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PyError();
    return v;
}

// (params, grads, exp_avgs, exp_avg_sqs, mantissas, scales, scalars, lr, beta1, beta2, eps, weight_decay, grad_scale, step)
PyObject* adamw_step(PyObject* const* a) {
    static const char* const where = "adamw_step";
    const Tensors params(a[0], -1, false, "params"), grads(a[1], params.n, false, "grads"), ms(a[2], params.n, false, "exp_avgs"),
        vs(a[3], params.n, false, "exp_avg_sqs"), lows(a[4], params.n, true, "mantissas"), scales(a[5], params.n, true, "scales");
    const at::Tensor* scalars = maybe(a[6], "scalars");
    anvil_adamw_config c = {number(a[7]), number(a[8]), number(a[9]), number(a[10]), number(a[11]), number(a[12]), 0};
    c.step = PyLong_AsLongLong(a[13]);
    if (c.step == -1 && PyErr_Occurred()) throw PyError();
    if (params.n > ANVIL_MAX_TENSORS) refuse("adamw_step: too many tensors");
    if (!params.n) return Py_NewRef(Py_None);
    const at::Device device = current(where, params.at(0));
    std::vector<anvil_adamw_tensor> tensors(static_cast<size_t>(params.n));
    Written written(5 * params.n);
    for (Py_ssize_t i = 0; i < params.n; ++i) {
        const at::Tensor &p = *params.at(i), &g = *grads.at(i), &m = *ms.at(i), &v = *vs.at(i);
        const at::Tensor *low = lows.at(i), *sc = scales.at(i);
        const int64_t count = p.numel();
        anvil_adamw_tensor& t = tensors[static_cast<size_t>(i)];
        t = {};
        t.param_dtype = dtype_code(p, "params");
        t.grad_dtype = dtype_code(g, "grads");
        if (t.param_dtype != ANVIL_F32 && t.grad_dtype != ANVIL_F32 && t.grad_dtype != t.param_dtype)
            refuse("adamw_step: grads must be fp32 or of their parameters' types");
        plain_tensor(p, device, count, where, "params");
        plain_tensor(g, device, count, where, "grads");
        plain_tensor(m, device, count, where, "exp_avgs");
        plain_tensor(v, device, count, where, "exp_avg_sqs");
        if (sc) check_codes(m, v, *sc, count, device, where);
        else if (m.scalar_type() != at::kFloat || v.scalar_type() != at::kFloat)
            refuse("adamw_step: exp_avgs and exp_avg_sqs must be fp32, or 8-bit codes with scales");
        if (low) {
            plain_tensor(*low, device, count, where, "mantissas");
            if (t.param_dtype != ANVIL_BF16 || (low->scalar_type() != at::kShort && low->scalar_type() != at::kUInt16))
                refuse("adamw_step: mantissas must be 16-bit integers beside bf16 parameters");
            t.mantissa = static_cast<uint16_t*>(low->data_ptr());
        }
        t.param = p.data_ptr();
        t.grad = g.data_ptr();
        t.exp_avg = m.data_ptr();
        t.exp_avg_sq = v.data_ptr();
        t.scales = sc ? static_cast<float*>(sc->data_ptr()) : nullptr;
        t.count = count;
        for (const at::Tensor* w : {&p, &m, &v, low, sc}) written.add(w);
    }
    const float* ds = nullptr;
    if (scalars) {
        plain_tensor(*scalars, device, 4, where, "scalars, fp32 [4],");
        if (scalars->scalar_type() != at::kFloat) refuse("adamw_step: scalars must be fp32 [4]");
        ds = static_cast<const float*>(scalars->data_ptr());
    }
    void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    check(api.adamw_step(tensors.data(), static_cast<int>(params.n), &c, ds, stream), "anvil_adamw_step");
    written.done();
    return Py_NewRef(Py_None);
}

// (exp_avgs, exp_avg_sqs, scales, m's, v's)
PyObject* adamw_values(PyObject* const* a) {
    static const char* const where = "adamw_values";
    const Tensors ms(a[0], -1, false, "exp_avgs"), vs(a[1], ms.n, false, "exp_avg_sqs"), scales(a[2], ms.n, false, "scales"),
        om(a[3], ms.n, false, "out[0]"), ov(a[4], ms.n, false, "out[1]");
    if (ms.n > ANVIL_MAX_TENSORS) refuse("adamw_values: too many tensors");
    if (!ms.n) return Py_NewRef(Py_None);
    const at::Device device = current(where, ms.at(0));
    std::vector<anvil_adamw_state> states(static_cast<size_t>(ms.n));
    Written written(2 * ms.n);
    for (Py_ssize_t i = 0; i < ms.n; ++i) {
        const at::Tensor &m = *ms.at(i), &v = *vs.at(i), &sc = *scales.at(i), &to_m = *om.at(i), &to_v = *ov.at(i);
        const int64_t count = m.numel();
        plain_tensor(m, device, count, where, "exp_avgs");
        plain_tensor(v, device, count, where, "exp_avg_sqs");
        check_codes(m, v, sc, count, device, where);
        plain_tensor(to_m, device, count, where, "out");
        plain_tensor(to_v, device, count, where, "out");
        if (to_m.scalar_type() != at::kFloat || to_v.scalar_type() != at::kFloat) refuse("adamw_values: out must be fp32");
        states[static_cast<size_t>(i)] = {m.data_ptr(), v.data_ptr(), static_cast<const float*>(sc.data_ptr()),
                                          static_cast<float*>(to_m.data_ptr()), static_cast<float*>(to_v.data_ptr()), count};
        written.add(&to_m);
        written.add(&to_v);
    }
    void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    check(api.adamw_values(states.data(), static_cast<int>(ms.n), stream), "anvil_adamw_values");
    written.done();
    return Py_NewRef(Py_None);
}

// Exceptions end here: a C++ one (out of memory, say) becomes the Python one torch gives it.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        need_args(n, N);
        return F(args);
    } catch (const PyError&) {
        return nullptr;
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(g_out_of_memory, e.what_without_backtrace());
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// set_library(addresses of the entry points in Api's order, check, torch.OutOfMemoryError)
PyObject* set_library(PyObject*, PyObject* const* args, Py_ssize_t n) {
    constexpr Py_ssize_t want = sizeof(Api) / sizeof(void*);
    if (n != 3 || !PyTuple_Check(args[0]) || PyTuple_GET_SIZE(args[0]) != want) {
        PyErr_SetString(PyExc_TypeError, "set_library(addresses, check, out of memory error)");
        return nullptr;
    }
    void** slot = reinterpret_cast<void**>(&api);
    for (Py_ssize_t i = 0; i < want; ++i) {
        slot[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args[0], i));
        if (PyErr_Occurred()) return nullptr;
    }
    Py_XSETREF(g_check, Py_NewRef(args[1]));
    Py_XSETREF(g_out_of_memory, Py_NewRef(args[2]));
    Py_RETURN_NONE;
}

#define ANVIL_ENTRY(name, n) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(entry<name, n>)), METH_FASTCALL, ""}
PyMethodDef methods[] = {
    {"set_library", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(set_library)), METH_FASTCALL, ""},
    ANVIL_ENTRY(layernorm_forward, 5),
    ANVIL_ENTRY(layernorm_backward, 9),
    ANVIL_ENTRY(linear_forward, 8),
    ANVIL_ENTRY(linear_backward, 14),
    ANVIL_ENTRY(token_logprobs, 3),
    ANVIL_ENTRY(token_logprobs_backward, 7),
    ANVIL_ENTRY(adamw_step, 14),
    ANVIL_ENTRY(adamw_values, 5),
    ANVIL_ENTRY(gated_linear_forward, 7),
    ANVIL_ENTRY(gated_linear_backward, 15),
    ANVIL_ENTRY(linear_cross_entropy, 4),
    ANVIL_ENTRY(linear_cross_entropy_backward, 11),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_anvil_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__anvil_binding(void) { return PyModule_Create(&module); }
