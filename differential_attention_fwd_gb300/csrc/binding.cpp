// binding.cpp -- the Python binding of the operators around a paged key/value cache, as a
// CPython module: argument checks, allocation of results and the calls of the C ABI.
//
// A decode step makes these calls for every layer, with kernels of a few microseconds, so
// the host's time a call is what a user sees.  Checking a dozen tensors and packing a
// descriptor from Python took 35 to 60 us on the CPU beside a GB300; this takes 4 to 12.
// The gradient of the norm and rotation is an autograd node in C++ for the same reason.
//
// Every function takes its arguments by position, as _paged.py passes them.
#include <Python.h>

#include <cmath>
#include <mutex>
#include <optional>
#include <string>
#include <unordered_set>
#include <vector>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <c10/core/AutogradState.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/functions/accumulate_grad.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/graph_task.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/saved_variable.h>

#include "diffattn.h"

namespace {

using at::Tensor;

PyObject* g_diffattn_error = nullptr;       // the package's DiffattnError

// A refusal: a Python exception with a text.
struct Refusal {
    PyObject* type;
    std::string what;
};
// A code of the C ABI.
struct Failure {
    int code;
    const char* what;
};

[[noreturn]] void bad_value(const std::string& what) { throw Refusal{PyExc_ValueError, what}; }
[[noreturn]] void bad_type(const std::string& what) { throw Refusal{PyExc_TypeError, what}; }

std::string text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

void check(int code, const char* what) {
    if (code != DIFFATTN_OK) throw Failure{code, what};
}

bool is_none(PyObject* o) { return o == Py_None; }

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

// A CUDA tensor of `dim` dimensions; of this type and on this device where given.
const Tensor& need(PyObject* o, const char* name, int64_t dim, std::optional<at::ScalarType> type = {},
                   std::optional<at::Device> dev = {}) {
    const Tensor& t = tensor(o, name);
    if (!t.is_cuda())
        bad_value(std::string(name) + " must be a CUDA tensor (got " + t.device().str() + "); there is no CPU path");
    if (t.dim() != dim) bad_value(std::string(name) + " must be " + std::to_string(dim) + "-D, got " + text(t.sizes()));
    if (type && t.scalar_type() != *type)
        bad_value(std::string(name) + " must be " + at::toString(*type) + ", got " + at::toString(t.scalar_type()));
    if (dev && t.device() != *dev)
        bad_value(std::string(name) + " must be on " + dev->str() + ", got " + t.device().str());
    return t;
}

bool inner_ok(const Tensor& t) { return t.stride(-1) == 1 || t.size(-1) == 1; }
Tensor inner(const Tensor& t) { return inner_ok(t) ? t : t.contiguous(); }

int32_t dtype_code(const Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return DIFFATTN_BF16;
    if (t.scalar_type() == at::kFloat) return DIFFATTN_F32;
    bad_value(std::string("unsupported dtype ") + at::toString(t.scalar_type()) + "; expected bfloat16 or float32");
}

double number(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        bad_type(std::string(name) + " must be a number");
    }
    return v;
}

bool truth(PyObject* o, const char* name) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        bad_type(std::string(name) + " must be a truth value");
    }
    return v == 1;
}

// The code of a norm's name; `group` where the output epilogue allows it.
int32_t norm_code(PyObject* o, bool group) {
    if (is_none(o)) return DIFFATTN_NORM_NONE;
    if (PyUnicode_Check(o)) {
        if (PyUnicode_CompareWithASCIIString(o, "none") == 0) return DIFFATTN_NORM_NONE;
        if (PyUnicode_CompareWithASCIIString(o, "rms") == 0) return DIFFATTN_NORM_RMS;
        if (group && PyUnicode_CompareWithASCIIString(o, "group") == 0) return DIFFATTN_NORM_GROUP;
    }
    bad_value(group ? "norm must be None, 'none', 'rms' or 'group'" : "norm must be None, 'none' or 'rms'");
}

void strides3(int64_t dst[3], const Tensor& t) {
    const auto s = t.strides();
    for (int i = 0; i < 3; ++i) dst[i] = s[i];
}

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
const float* fptr(const Tensor& t) { return t.defined() ? t.const_data_ptr<float>() : nullptr; }

// An uninitialised dense tensor, without the dispatcher (half of at::empty's 1.5 us).
Tensor fresh_tensor(at::IntArrayRef sizes, at::ScalarType type, at::Device dev) {
    return Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
}

diffattn_stream_t stream_of(at::Device dev) {
    return reinterpret_cast<diffattn_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

// Refuses dual tensors: nothing here has a forward-mode derivative, and a result without a
// tangent would be taken for a constant.
void no_tangent(std::initializer_list<const Tensor*> ts, const char* what) {
    if (!c10::AutogradState::get_tls_state().get_fw_grad_mode()) return;
    for (const Tensor* t : ts)
        if (t->defined() && t->_fw_grad(0).defined()) bad_value(std::string(what) + " has no forward-mode derivative");
}

// float32 and dense.
Tensor plain_f32(const Tensor& t) {
    if (t.scalar_type() == at::kFloat && t.is_contiguous()) return t;
    at::NoGradGuard no_grad;
    return t.to(at::kFloat).contiguous();
}

// A norm weight [D] or [heads, D]: float32 and dense, and its head stride.  With no rows of its
// kind (heads = 0) it is looked at and left out: nothing reads it, and it has no gradient.
Tensor norm_weight(PyObject* o, const char* name, int64_t heads, int64_t D, at::Device dev, Tensor* given, int64_t* stride) {
    *stride = 0;
    if (is_none(o)) return {};
    const Tensor& w = tensor(o, name);
    if (w.device() != dev ||
        !((w.dim() == 1 && w.size(0) == D) || (w.dim() == 2 && (w.size(0) == heads || heads == 0) && w.size(1) == D)))
        bad_value(std::string(name) + " must be [D] = (" + std::to_string(D) + ",) or [heads, D] = (" +
                  (heads ? std::to_string(heads) : "heads") + ", " + std::to_string(D) + ") on the inputs' device, got " +
                  text(w.sizes()));
    if (!at::isFloatingType(w.scalar_type())) bad_value(std::string(name) + " must be a floating tensor");
    if (heads == 0) return {};
    *stride = w.dim() == 2 ? D : 0;
    *given = w;
    return plain_f32(w);
}

// What a node saved, for its backward pass.  A hook of saved tensors (save_on_cpu, or a user's)
// may give it back in another layout, so strides are those of what comes back; of other sizes,
// another type or on another device it is not what was saved.
Tensor restored(const Tensor& t, at::IntArrayRef sizes, at::ScalarType type, at::Device dev, const char* what) {
    TORCH_CHECK(t.defined() && t.sizes() == sizes && t.scalar_type() == type && t.device() == dev, what,
                ": a hook of saved tensors gave back ", t.defined() ? text(t.sizes()) : "nothing",
                t.defined() ? std::string(" ") + at::toString(t.scalar_type()) + " on " + t.device().str() : "", " for ",
                text(sizes), " ", at::toString(type), " on ", dev.str());
    return t;
}
// The same for tensors that the kernels take dense: contiguous, from a 16-byte boundary.
Tensor restored_dense(const Tensor& t, at::IntArrayRef sizes, at::ScalarType type, at::Device dev, const char* what) {
    const Tensor r = restored(t, sizes, type, dev, what);
    return r.is_contiguous() && reinterpret_cast<uintptr_t>(r.const_data_ptr()) % 16 == 0
               ? r
               : r.clone(at::MemoryFormat::Contiguous);
}

bool wants_grad(std::initializer_list<const Tensor*> ts) {
    if (!at::GradMode::is_enabled()) return false;
    for (const Tensor* t : ts)
        if (t->defined() && t->requires_grad()) return true;
    return false;
}

// lambda: a number, or one value on the host or the device.
struct Lambda {
    float host = 0.f;
    Tensor dev;             // float32 (or bf16 where the kernels take that), where it is on the device
    Tensor given;           // the tensor, if it is one
    Lambda(PyObject* o, at::Device on, const char* what, bool bf16 = false) {
        if (!THPVariable_Check(o)) {
            host = (float)number(o, "coefficient");
            return;
        }
        given = THPVariable_Unpack(o);
        if (given.numel() != 1) bad_value("coefficient must be a scalar");
        no_tangent({&given}, what);
        if (given.is_cuda()) {
            if (given.device() != on) bad_value("coefficient tensor must be on the inputs' device");
            dev = bf16 && given.scalar_type() == at::kBFloat16 ? given : plain_f32(given);
        } else {
            host = (float)given.item().toDouble();
        }
    }
};

// ---------------------------------------------------------------------------
// norm and rotation
// ---------------------------------------------------------------------------
// What a call says besides its rows.
struct Rotary {
    int64_t B = 0, T = 0, D = 0, H = 0, Hk = 0, R = 0, rows = 0;
    int32_t dtype = 0, norm = 0, interleaved = 0, pos64 = 0;
    int64_t pos_stride[2] = {0, 0}, qws = 0, kws = 0;
    float eps = 0.f;
    diffattn_axes axes{};                   // n = 0: a position a token
    Tensor cos, sin, pos, qw, kw;           // as the kernels read them
    Tensor qw_given, kw_given;              // as the caller has them

    void tables(PyObject* c, PyObject* s, at::Device dev) {
        if (is_none(c) && is_none(s)) return;
        cos = need(c, "cos", 2, at::kFloat, dev);
        sin = need(s, "sin", 2, at::kFloat, dev);
        if (cos.sizes() != sin.sizes() || cos.size(0) < 1 || cos.size(1) < 1 || 2 * cos.size(1) > D)
            bad_value("cos and sin must be [rows, rotary_dim / 2] with rotary_dim <= D, got " + text(cos.sizes()) + " and " +
                      text(sin.sizes()));
        if (cos.requires_grad() || sin.requires_grad()) bad_value("cos and sin take no gradient");
        if (!cos.is_contiguous()) cos = cos.contiguous();
        if (!sin.is_contiguous()) sin = sin.contiguous();
        R = 2 * cos.size(1);
        rows = cos.size(0);
    }
    void positions(PyObject* o, PyObject* sections, at::Device dev) {
        if (!is_none(sections)) return axis_positions(o, sections, dev);
        if (is_none(o)) return;
        pos = tensor(o, "positions");
        const bool flat = pos.dim() == 1;
        if (pos.device() != dev || (pos.scalar_type() != at::kInt && pos.scalar_type() != at::kLong) ||
            !((flat && pos.size(0) == T) || (pos.dim() == 2 && pos.size(0) == B && pos.size(1) == T)))
            bad_value("positions must be an int32 or int64 tensor [T] or [B, T] = (" + std::to_string(B) + ", " +
                      std::to_string(T) + ") on the inputs' device");
        set_positions(pos);
    }
    // The positions as the kernels read them: [T] or [B, T], with axes [T, axes] or [B, T, axes].
    void set_positions(const Tensor& p) {
        pos = p;
        pos64 = p.scalar_type() == at::kLong;
        const int64_t last = axes.n ? 1 : 0;
        pos_stride[0] = p.dim() == 1 + last ? 0 : p.stride(0);
        pos_stride[1] = p.stride(-1 - last);
        if (axes.n) axes.pos_stride = p.stride(-1);
    }
    // positions [T, axes] or [B, T, axes], and the pairs of each axis
    void axis_positions(PyObject* o, PyObject* sections, at::Device dev) {
        if (!PyTuple_Check(sections) && !PyList_Check(sections)) bad_type("sections must be a tuple or a list of whole numbers");
        const Py_ssize_t n = PySequence_Size(sections);
        if (n < 1 || n > DIFFATTN_MAX_AXES)
            bad_value("sections must name 1 to " + std::to_string(DIFFATTN_MAX_AXES) + " axes, got " + std::to_string(n));
        int64_t sum = 0;
        for (Py_ssize_t i = 0; i < n; ++i) {
            PyObject* item = PyTuple_Check(sections) ? PyTuple_GET_ITEM(sections, i) : PyList_GET_ITEM(sections, i);
            if (!PyLong_Check(item)) bad_type("sections must be a tuple or a list of whole numbers");
            const long v = PyLong_AsLong(item);
            if (v == -1 && PyErr_Occurred()) PyErr_Clear();
            if (v < 1 || v > R / 2) bad_value("sections must be positive and add up to rotary_dim / 2 = " + std::to_string(R / 2));
            axes.pairs[i] = (int32_t)v;
            sum += v;
        }
        if (sum != R / 2) bad_value("sections must add up to rotary_dim / 2 = " + std::to_string(R / 2) + ", got " + std::to_string(sum));
        if (is_none(o)) bad_value("sections need positions [T, axes] or [B, T, axes]");
        pos = tensor(o, "positions");
        const bool flat = pos.dim() == 2;
        if (pos.device() != dev || (pos.scalar_type() != at::kInt && pos.scalar_type() != at::kLong) || pos.dim() < 2 ||
            pos.dim() > 3 || pos.size(-1) != n || pos.size(-2) != T || (!flat && pos.size(0) != B))
            bad_value("with sections, positions must be an int32 or int64 tensor [T, axes] or [B, T, axes] = (" +
                      std::to_string(B) + ", " + std::to_string(T) + ", " + std::to_string(n) + ") on the inputs' device");
        axes.n = (int32_t)n;
        set_positions(pos);
    }
    const diffattn_axes* axes_ptr() const { return axes.n ? &axes : nullptr; }
    void set_norm(PyObject* name, PyObject* e) {
        norm = norm_code(name, false);
        eps = (float)number(e, "norm_eps");
        if (norm && !(std::isfinite(eps) && eps > 0.f)) bad_value("norm_eps must be positive and finite");
    }
    diffattn_rotary_desc desc() const {
        diffattn_rotary_desc d{};
        d.B = B; d.T = T; d.D = D; d.H = H; d.Hk = Hk;
        d.dtype = dtype;
        d.rotary_dim = (int32_t)R;
        d.interleaved = interleaved;
        d.norm = norm;
        d.eps = eps;
        d.pos64 = pos64;
        d.table_rows = rows;
        d.pos_stride[0] = pos_stride[0];
        d.pos_stride[1] = pos_stride[1];
        d.q_weight_stride = qws;
        d.k_weight_stride = kws;
        return d;
    }
};

const char* const kRotary = "qk_norm_rotary";
const char* const kRowNames[4] = {"q1", "k1", "q2", "k2"};

// The strides of a descriptor's i-th tensor, in the order q1, k1, q2, k2.
int64_t* row_stride(diffattn_rotary_desc& d, int i) {
    return i == 0 ? d.q1_stride : i == 1 ? d.k1_stride : i == 2 ? d.q2_stride : d.k2_stride;
}
int64_t* grad_stride(diffattn_rotary_desc& d, int i) {
    return i == 0 ? d.q1_grad_stride : i == 1 ? d.k1_grad_stride : i == 2 ? d.q2_grad_stride : d.k2_grad_stride;
}

void rotary_forward(const Rotary& r, const Tensor (&x)[4], Tensor (&y)[4], at::Device dev) {
    diffattn_rotary_desc d = r.desc();
    for (int i = 0; i < 4; ++i) {
        if (!x[i].defined()) continue;
        strides3(row_stride(d, i), x[i]);
        y[i] = fresh_tensor(x[i].sizes(), x[i].scalar_type(), dev);
    }
    check(diffattn_rotary_axes(&d, r.axes_ptr(), ptr(x[0]), ptr(x[1]), ptr(x[2]), ptr(x[3]), fptr(r.qw), fptr(r.kw), fptr(r.cos), fptr(r.sin),
                          ptr(r.pos), ptr(y[0]), ptr(y[1]), ptr(y[2]), ptr(y[3]), stream_of(dev)),
          "diffattn_rotary");
}

// In a capture: whether this backward pass goes on to add to the .grad of a leaf whose
// accumulation belongs to the default stream, because an eager graph of that leaf made it
// there and still lives.  torch would then make the default stream wait inside the capture,
// which CUDA forbids and the process does not survive.
bool joins_default_stream(const torch::autograd::Node& from) {
    using namespace torch::autograd;
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None) return false;
    const auto* task = get_current_graph_task_exec_info();      // empty: every node runs
    std::unordered_set<const Node*> seen;
    std::vector<const Node*> todo{&from};
    while (!todo.empty()) {
        const Node* n = todo.back();
        todo.pop_back();
        for (const Edge& e : n->next_edges()) {
            Node* next = e.function.get();
            if (!next || !seen.insert(next).second) continue;
            if (task && !task->empty()) {
                const auto it = task->find(next);
                if (it == task->end() || !it->second.needed_) continue;
            }
            if (dynamic_cast<AccumulateGrad*>(next)) {
                const auto stream = next->stream();
                if (stream && stream->id() == 0) return true;
            } else {
                todo.push_back(next);
            }
        }
    }
    return false;
}

// The autograd node: backward through diffattn_rotary_bwd.  Its inputs are the rows that
// were given, then the weights; its outputs the rotated rows.
struct RotaryBackward : public torch::autograd::Node {
    Rotary r;
    torch::autograd::SavedVariable x[4], w[2], tables[3];      // tables: cos, sin, positions
    bool given[4] = {}, weight[2] = {};
    // without the norm the rows themselves are not saved: the gradient does not depend on them
    std::vector<int64_t> sizes[4], pos_sizes, w_sizes[2];
    at::ScalarType w_type[2] = {};
    bool has_pos = false;
    std::optional<at::Device> dev;
    bool released = false;

    torch::autograd::variable_list apply(torch::autograd::variable_list&& grads) override {
        std::lock_guard<std::mutex> lock(mutex_);
        TORCH_CHECK(!released, "qk_norm_rotary: backward a second time through a graph whose saved tensors were freed; "
                               "pass retain_graph=True the first time");
        TORCH_CHECK(!at::GradMode::is_enabled(), "qk_norm_rotary is differentiable once (no create_graph)");
        TORCH_CHECK(!joins_default_stream(*this), "qk_norm_rotary: this captured backward pass would add to the .grad of a "
                    "leaf that a graph made outside the capture, on the default stream, still holds; drop that graph (or "
                    "make it on another stream), or take the gradients with torch.autograd.grad");
        Rotary c = r;
        const c10::cuda::OptionalCUDAGuard guard(*dev);
        // unpacking checks that nothing saved was changed in place
        if (c.R > 0) {
            const int64_t table[2] = {c.rows, c.R / 2};
            c.cos = restored_dense(tables[0].unpack(), table, at::kFloat, *dev, kRotary);
            c.sin = restored_dense(tables[1].unpack(), table, at::kFloat, *dev, kRotary);
        }
        if (has_pos) c.set_positions(restored(tables[2].unpack(), pos_sizes, c.pos64 ? at::kLong : at::kInt, *dev, kRotary));
        Tensor wt[2];
        for (int i = 0; i < 2; ++i)
            if (weight[i]) wt[i] = restored(w[i].unpack(), w_sizes[i], w_type[i], *dev, kRotary);
        if (weight[0]) c.qw = plain_f32(wt[0]);
        if (weight[1]) c.kw = plain_f32(wt[1]);
        diffattn_rotary_desc d = c.desc();
        Tensor xs[4], gs[4], dx[4];
        const at::ScalarType type = c.dtype == DIFFATTN_BF16 ? at::kBFloat16 : at::kFloat;
        int out = 0;
        for (int i = 0; i < 4; ++i) {
            if (!given[i]) continue;
            if (c.norm) {
                xs[i] = inner(restored(x[i].unpack(), sizes[i], type, *dev, kRotary));
                strides3(row_stride(d, i), xs[i]);
            }
            Tensor g = grads[out++];
            if (!g.defined()) g = at::zeros(sizes[i], at::TensorOptions().dtype(type).device(*dev));
            gs[i] = inner(g.scalar_type() == type ? g : g.to(type));
            strides3(grad_stride(d, i), gs[i]);
            dx[i] = fresh_tensor(sizes[i], type, *dev);
        }
        Tensor dw[2];
        for (int i = 0; i < 2; ++i)
            if (weight[i] && task_should_compute_output(out + i - (i == 1 && !weight[0])))
                dw[i] = fresh_tensor((i ? c.kw : c.qw).sizes(), at::kFloat, *dev);
        const size_t bytes = diffattn_rotary_bwd_workspace_bytes(&d);
        const Tensor ws = fresh_tensor({(int64_t)bytes}, at::kByte, *dev);
        const int rc = diffattn_rotary_axes_bwd(
            &d, c.axes_ptr(), ptr(xs[0]), ptr(xs[1]), ptr(xs[2]), ptr(xs[3]), fptr(c.qw), fptr(c.kw), fptr(c.cos), fptr(c.sin), ptr(c.pos),
            ptr(gs[0]), ptr(gs[1]), ptr(gs[2]), ptr(gs[3]), ptr(dx[0]), ptr(dx[1]), ptr(dx[2]), ptr(dx[3]),
            dw[0].defined() ? dw[0].data_ptr<float>() : nullptr, dw[1].defined() ? dw[1].data_ptr<float>() : nullptr,
            ws.data_ptr(), bytes, stream_of(*dev));
        TORCH_CHECK(rc == DIFFATTN_OK, "diffattn_rotary_bwd: ", diffattn_strerror(rc), " (", rc, ")");
        torch::autograd::variable_list result;
        for (int i = 0; i < 4; ++i)
            if (given[i]) result.push_back(dx[i]);
        for (int i = 0; i < 2; ++i)
            if (weight[i])
                result.push_back(dw[i].defined() && dw[i].scalar_type() != wt[i].scalar_type() ? dw[i].to(wt[i].scalar_type())
                                                                                               : dw[i]);
        return result;
    }
    void release_variables() override {
        std::lock_guard<std::mutex> lock(mutex_);
        for (auto& v : x) v.reset_data();
        for (auto& v : w) v.reset_data();
        for (auto& v : tables) v.reset_data();
        released = true;
    }
    std::string name() const override { return "QkNormRotaryBackward"; }
};

PyObject* rotary(PyObject* const* a) {
    // q1, k1, q2, k2, cos, sin, positions, norm, norm_eps, q_weight, k_weight, interleaved, sections
    const bool shared = !is_none(a[3]) && a[3] == a[1];
    Tensor in[4];
    const Tensor* first = nullptr;
    for (int i = 0; i < 4; ++i) {
        if (is_none(a[i]) || (i == 3 && shared)) continue;
        if (first) in[i] = need(a[i], kRowNames[i], 4, first->scalar_type(), first->device());
        else in[i] = need(a[i], kRowNames[i], 4);
        if (!first) first = &in[i];
    }
    if (!first) bad_value("at least one of q1, k1, q2, k2 must be given");
    const at::Device dev = first->device();
    Rotary r;
    r.dtype = dtype_code(*first);
    r.B = first->size(0);
    r.T = first->size(2);
    r.D = first->size(3);
    if (r.B < 1 || r.T < 1 || r.D < 1 || r.D > 128)
        bad_value("rows must be [B, heads, T, D] with B, T >= 1 and D <= 128, got " + text(first->sizes()));
    for (int i = 0; i < 4; ++i) {
        if (!in[i].defined()) continue;
        int64_t& heads = i & 1 ? r.Hk : r.H;
        if (in[i].size(0) != r.B || in[i].size(2) != r.T || in[i].size(3) != r.D || in[i].size(1) < 1 ||
            (heads && heads != in[i].size(1)))
            bad_value("q1, q2 must share one shape [B, H, T, D], and k1, k2 [B, H_kv, T, D]");
        heads = in[i].size(1);
    }
    r.tables(a[4], a[5], dev);
    r.positions(a[6], a[12], dev);
    r.set_norm(a[7], a[8]);
    if (!r.norm && !(is_none(a[9]) && is_none(a[10]))) bad_value("q_weight and k_weight need norm='rms'");
    r.qw = norm_weight(a[9], "q_weight", r.H, r.D, dev, &r.qw_given, &r.qws);
    r.kw = norm_weight(a[10], "k_weight", r.Hk, r.D, dev, &r.kw_given, &r.kws);
    r.interleaved = truth(a[11], "interleaved");
    no_tangent({&in[0], &in[1], &in[2], &in[3], &r.cos, &r.sin, &r.qw_given, &r.kw_given}, "qk_norm_rotary");
    const c10::cuda::OptionalCUDAGuard guard(dev);
    bool grad = false;
    if (at::GradMode::is_enabled()) {
        for (const Tensor& t : in) grad |= t.defined() && t.requires_grad();
        grad |= r.qw_given.defined() && r.qw_given.requires_grad();
        grad |= r.kw_given.defined() && r.kw_given.requires_grad();
    }
    Tensor x[4], y[4];
    {
        at::NoGradGuard no_grad;
        for (int i = 0; i < 4; ++i)
            if (in[i].defined()) x[i] = inner(in[i]);
        rotary_forward(r, x, y, dev);
    }
    if (grad) {
        auto node = std::shared_ptr<RotaryBackward>(new RotaryBackward(), torch::autograd::deleteNode);
        torch::autograd::variable_list from;
        for (int i = 0; i < 4; ++i) {
            node->given[i] = in[i].defined();
            if (!in[i].defined()) continue;
            from.push_back(in[i]);
            node->sizes[i] = in[i].sizes().vec();
            if (r.norm) node->x[i] = torch::autograd::SavedVariable(x[i], false);
        }
        node->dev = dev;
        const Tensor ws[2] = {r.qw_given, r.kw_given};
        for (int i = 0; i < 2; ++i) {
            node->weight[i] = ws[i].defined();
            if (!ws[i].defined()) continue;
            from.push_back(ws[i]);
            node->w_sizes[i] = ws[i].sizes().vec();
            node->w_type[i] = ws[i].scalar_type();
            node->w[i] = torch::autograd::SavedVariable(ws[i], false);
        }
        if (r.R > 0) {
            node->tables[0] = torch::autograd::SavedVariable(r.cos, false);
            node->tables[1] = torch::autograd::SavedVariable(r.sin, false);
        }
        if (r.pos.defined()) {
            node->has_pos = true;
            node->pos_sizes = r.pos.sizes().vec();
            node->tables[2] = torch::autograd::SavedVariable(r.pos, false);
        }
        node->set_next_edges(torch::autograd::collect_next_edges(from));
        for (Tensor& t : y)
            if (t.defined()) torch::autograd::set_history(t, node);
        // the node holds its tensors as saved ones only
        r.cos = r.sin = r.pos = r.qw = r.kw = r.qw_given = r.kw_given = Tensor();
        node->r = r;
    }
    PyObject* out = PyTuple_New(4);
    if (!out) return nullptr;
    for (int i = 0; i < 4; ++i) {
        PyObject* o;
        if (i == 3 && shared) {
            o = PyTuple_GET_ITEM(out, 1);
            Py_INCREF(o);
        } else if (y[i].defined()) {
            o = THPVariable_Wrap(y[i]);
        } else {
            o = Py_None;
            Py_INCREF(o);
        }
        if (!o) {
            Py_DECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i, o);
    }
    return out;
}

// ---------------------------------------------------------------------------
// the norm of each head's output
// ---------------------------------------------------------------------------
// An uninitialised tensor laid out as `t` where that is dense in some order of its dimensions
// (with rows of the innermost one), contiguous else.
Tensor fresh_like(const Tensor& t) {
    if (t.is_contiguous() || !inner_ok(t) || !t.is_non_overlapping_and_dense())
        return fresh_tensor(t.sizes(), t.scalar_type(), t.device());
    return Tensor(at::detail::empty_strided_cuda(t.sizes(), t.strides(), t.scalar_type(), t.device()));
}

// An affine parameter [H, C] or [H * C]: float32 and dense.
Tensor affine(PyObject* o, const char* name, int64_t H, int64_t C, at::Device dev, Tensor* given) {
    if (is_none(o)) return {};
    const Tensor& t = tensor(o, name);
    if (t.device() != dev || !((t.dim() == 2 && t.size(0) == H && t.size(1) == C) || (t.dim() == 1 && t.size(0) == H * C)))
        bad_value(std::string(name) + " must be [H, Dv] = (" + std::to_string(H) + ", " + std::to_string(C) +
                  ") on the inputs' device, got " + text(t.sizes()));
    if (!at::isFloatingType(t.scalar_type())) bad_value(std::string(name) + " must be a floating tensor");
    *given = t;
    return plain_f32(t);
}

const char* const kHeadNorm = "differential_head_norm";

// The autograd node: backward through diffattn_head_norm_bwd.  Its inputs are x, then the
// weight and the bias where they were given.
struct HeadNormBackward : public torch::autograd::Node {
    diffattn_norm_desc d{};
    torch::autograd::SavedVariable x, w;
    bool has[2] = {};                       // weight, bias
    std::vector<int64_t> shape[2];
    at::ScalarType type[2] = {};
    std::optional<at::Device> dev;
    bool released = false;

    torch::autograd::variable_list apply(torch::autograd::variable_list&& grads) override {
        std::lock_guard<std::mutex> lock(mutex_);
        TORCH_CHECK(!released, "differential_head_norm: backward a second time through a graph whose saved tensors were "
                               "freed; pass retain_graph=True the first time");
        TORCH_CHECK(!at::GradMode::is_enabled(), "differential_head_norm is differentiable once (no create_graph)");
        TORCH_CHECK(!joins_default_stream(*this), "differential_head_norm: this captured backward pass would add to the .grad "
                    "of a leaf that a graph made outside the capture, on the default stream, still holds; drop that graph, "
                    "or make it on another stream");
        torch::autograd::variable_list result(1 + has[0] + has[1]);
        if (!grads[0].defined()) return result;
        const c10::cuda::OptionalCUDAGuard guard(*dev);
        const int64_t sizes[4] = {d.B, d.H, d.T, d.C};
        const Tensor xs = inner(restored(x.unpack(), sizes, d.dtype == DIFFATTN_BF16 ? at::kBFloat16 : at::kFloat, *dev, kHeadNorm));
        const Tensor ws = has[0] ? plain_f32(restored(w.unpack(), shape[0], type[0], *dev, kHeadNorm)) : Tensor();
        const Tensor g = inner(grads[0].scalar_type() == xs.scalar_type() ? grads[0] : grads[0].to(xs.scalar_type()));
        diffattn_norm_desc c = d;
        Tensor dx, da[2];
        if (task_should_compute_output(0)) dx = fresh_like(xs);
        for (int i = 0, out = 1; i < 2; ++i)
            if (has[i] && task_should_compute_output(out++)) da[i] = fresh_tensor({c.H, c.C}, at::kFloat, *dev);
        if (!dx.defined() && !da[0].defined() && !da[1].defined()) return result;
        strides3(c.x_stride, xs);
        strides3(c.dy_stride, g);
        if (dx.defined()) strides3(c.dx_stride, dx);
        const size_t bytes = da[0].defined() || da[1].defined() ? diffattn_head_norm_bwd_workspace_bytes(&c) : 0;
        const Tensor space = bytes ? fresh_tensor({(int64_t)bytes}, at::kByte, *dev) : Tensor();
        const int rc = diffattn_head_norm_bwd(&c, ptr(xs), fptr(ws), ptr(g), ptr(dx), (float*)ptr(da[0]), (float*)ptr(da[1]),
                                              ptr(space), bytes, stream_of(*dev));
        TORCH_CHECK(rc == DIFFATTN_OK, "diffattn_head_norm_bwd: ", diffattn_strerror(rc), " (", rc, ")");
        result[0] = dx;
        for (int i = 0, out = 1; i < 2; ++i) {
            if (!has[i]) continue;
            if (da[i].defined()) result[out] = da[i].to(type[i]).view(shape[i]);
            ++out;
        }
        return result;
    }
    void release_variables() override {
        std::lock_guard<std::mutex> lock(mutex_);
        x.reset_data();
        w.reset_data();
        released = true;
    }
    std::string name() const override { return "HeadNormBackward"; }
};

PyObject* head_norm(PyObject* const* a) {
    // x, norm, norm_eps, norm_weight, norm_bias, out_scale
    const Tensor& x = need(a[0], "x", 4);
    const at::Device dev = x.device();
    diffattn_norm_desc d{};
    d.dtype = dtype_code(x);
    d.B = x.size(0);
    d.H = x.size(1);
    d.T = x.size(2);
    d.C = x.size(3);
    if (d.B < 1 || d.H < 1 || d.T < 1 || d.C < 1 || d.C > 256)
        bad_value("x must be [B, H, T, Dv] with B, H, T >= 1 and Dv <= 256, got " + text(x.sizes()));
    d.norm = norm_code(a[1], true);
    if (d.norm == DIFFATTN_NORM_NONE) bad_value("norm must be 'rms' or 'group'");
    d.eps = (float)number(a[2], "norm_eps");
    if (!(std::isfinite(d.eps) && d.eps > 0.f)) bad_value("norm_eps must be positive and finite");
    d.out_scale = (float)number(a[5], "out_scale");
    if (!std::isfinite(d.out_scale)) bad_value("out_scale must be finite");
    const c10::cuda::OptionalCUDAGuard guard(dev);
    Tensor given[2];
    const Tensor w = affine(a[3], "norm_weight", d.H, d.C, dev, &given[0]);
    const Tensor b = affine(a[4], "norm_bias", d.H, d.C, dev, &given[1]);
    no_tangent({&x, &given[0], &given[1]}, "differential_head_norm");
    const bool grad = at::GradMode::is_enabled() && (x.requires_grad() || (given[0].defined() && given[0].requires_grad()) ||
                                                     (given[1].defined() && given[1].requires_grad()));
    Tensor xs, y;
    {
        at::NoGradGuard no_grad;
        xs = inner(x);
        y = fresh_like(xs);
        strides3(d.x_stride, xs);
        strides3(d.y_stride, y);
        check(diffattn_head_norm(&d, ptr(xs), fptr(w), fptr(b), ptr(y), stream_of(dev)), "diffattn_head_norm");
    }
    if (grad) {
        auto node = std::shared_ptr<HeadNormBackward>(new HeadNormBackward(), torch::autograd::deleteNode);
        torch::autograd::variable_list from{x};
        node->d = d;
        node->dev = dev;
        node->x = torch::autograd::SavedVariable(x, false);
        for (int i = 0; i < 2; ++i) {
            node->has[i] = given[i].defined();
            if (!given[i].defined()) continue;
            from.push_back(given[i]);
            node->shape[i] = given[i].sizes().vec();
            node->type[i] = given[i].scalar_type();
        }
        if (given[0].defined()) node->w = torch::autograd::SavedVariable(given[0], false);
        node->set_next_edges(torch::autograd::collect_next_edges(from));
        torch::autograd::set_history(y, node);
    }
    return THPVariable_Wrap(y);
}

// ---------------------------------------------------------------------------
// the paged cache
// ---------------------------------------------------------------------------
struct Cache {
    Tensor k1, k2, v, table;
    bool shared;
    int64_t B, Hk, D, Dv;
    int32_t dtype;
    diffattn_pages pages{};

    Cache(PyObject* k1_, PyObject* k2_, PyObject* v_, PyObject* table_, int64_t batch) : B(batch) {
        k1 = need(k1_, "k1_cache", 4);
        const at::Device dev = k1.device();
        const at::ScalarType type = k1.scalar_type();
        dtype = dtype_code(k1);
        shared = is_none(k2_) || k2_ == k1_;
        k2 = shared ? k1 : need(k2_, "k2_cache", 4, type, dev);
        if (k2.sizes() != k1.sizes())
            bad_value("k1_cache and k2_cache must have one shape, got " + text(k1.sizes()) + ", " + text(k2.sizes()));
        v = need(v_, "v_cache", 4, type, dev);
        table = need(table_, "block_table", 2, at::kInt, dev);
        Hk = k1.size(1);
        D = k1.size(3);
        Dv = v.size(3);
        if (v.size(0) != k1.size(0) || v.size(1) != Hk || v.size(2) != k1.size(2) || k1.numel() == 0 || D > 128 || Dv < 1 ||
            Dv > 256)
            bad_value("expected k1_cache, k2_cache [pages, H_kv, page_size, D], v_cache [pages, H_kv, page_size, Dv], "
                      "D <= 128, Dv <= 256, got " + text(k1.sizes()) + ", " + text(v.sizes()));
        if (table.size(0) != B || table.size(1) < 1)
            bad_value("block_table must be [B, max_pages] with B = " + std::to_string(B) + ", got " + text(table.sizes()));
        // a copy would not be the cache
        if (!inner_ok(k1) || !inner_ok(k2) || !inner_ok(v) || !inner_ok(table))
            bad_value("k1_cache, k2_cache, v_cache and block_table must have a contiguous innermost dimension");
        pages.num_pages = k1.size(0);
        pages.page_size = k1.size(2);
        pages.max_pages = table.size(1);
        pages.block_table_stride = table.stride(0);
        strides3(pages.k1_stride, k1);
        strides3(pages.k2_stride, k2);
        strides3(pages.v_stride, v);
    }
    // An int32 tensor [B].
    Tensor lengths(PyObject* o, const char* name) const {
        const Tensor& t = need(o, name, 1, at::kInt, k1.device());
        if (t.size(0) != B) bad_value(std::string(name) + " must be [B] = (" + std::to_string(B) + ",), got " + text(t.sizes()));
        return t.is_contiguous() ? t : t.contiguous();
    }
    const int32_t* table_ptr() const { return table.const_data_ptr<int32_t>(); }
};

PyObject* append(PyObject* const* a) {
    // k1, k2, value, k1_cache, k2_cache, v_cache, block_table, lengths, new_lengths, cos, sin, positions, norm, norm_eps,
    // k_weight, interleaved, sections
    const Tensor& first = need(a[0], "k1", 4);
    Cache c(a[3], a[4], a[5], a[6], first.size(0));
    const at::Device dev = c.k1.device();
    const at::ScalarType type = c.k1.scalar_type();
    const bool shared = is_none(a[1]) || a[1] == a[0];
    if (c.shared != shared) bad_value("k2 and k2_cache must both be shared with k1 and k1_cache, or neither");
    Tensor k[2] = {need(a[0], "k1", 4, type, dev), shared ? Tensor() : need(a[1], "k2", 4, type, dev)};
    Rotary r;
    r.B = c.B;
    r.T = first.size(2);
    r.D = c.D;
    r.Hk = c.Hk;
    r.dtype = c.dtype;
    for (const Tensor& t : k)
        if (t.defined() && (t.size(0) != c.B || t.size(1) != c.Hk || t.size(2) != r.T || t.size(3) != c.D))
            bad_value("k1, k2 must be [B, H_kv, T, D] with the cache's H_kv and D, got " + text(t.sizes()));
    Tensor v = need(a[2], "value", 4, type, dev);
    if (v.size(0) != c.B || v.size(1) != c.Hk || v.size(2) != r.T || v.size(3) != c.Dv || r.T < 1)
        bad_value("value must be [B, H_kv, T, Dv] with the cache's H_kv and Dv, got " + text(v.sizes()));
    r.tables(a[9], a[10], dev);
    r.positions(a[11], a[16], dev);
    r.set_norm(a[12], a[13]);
    if (!r.norm && !is_none(a[14])) bad_value("k_weight needs norm='rms'");
    r.kw = norm_weight(a[14], "k_weight", r.Hk, r.D, dev, &r.kw_given, &r.kws);
    r.interleaved = truth(a[15], "interleaved");
    no_tangent({&k[0], &k[1], &v, &c.k1, &c.k2, &c.v, &r.cos, &r.sin, &r.kw_given}, "paged_cache_append");
    if (wants_grad({&k[0], &k[1], &v, &c.k1, &c.k2, &c.v, &r.kw_given}))
        bad_value("paged_cache_append is forward only: call it under torch.no_grad() or detach its inputs");
    const c10::cuda::OptionalCUDAGuard guard(dev);
    const Tensor lengths = c.lengths(a[7], "lengths");
    const Tensor fresh = is_none(a[8]) ? Tensor() : c.lengths(a[8], "new_lengths");
    for (Tensor& t : k)
        if (t.defined()) t = inner(t);
    v = inner(v);
    diffattn_rotary_desc d = r.desc();
    strides3(d.k1_stride, k[0]);
    if (!shared) strides3(d.k2_stride, k[1]);
    int64_t vs[3];
    strides3(vs, v);
    // in-place: what autograd saved of the cache before will no longer be it, and an
    // inference tensor outside of inference mode refuses
    c.k1.unsafeGetTensorImpl()->bump_version();
    if (!shared) c.k2.unsafeGetTensorImpl()->bump_version();
    c.v.unsafeGetTensorImpl()->bump_version();
    check(diffattn_paged_append_axes(&d, r.axes_ptr(), c.Dv, vs, &c.pages, ptr(k[0]), ptr(k[1]), ptr(v), fptr(r.kw), fptr(r.cos), fptr(r.sin),
                                ptr(r.pos), lengths.const_data_ptr<int32_t>(),
                                fresh.defined() ? fresh.const_data_ptr<int32_t>() : nullptr, c.table_ptr(), ptr(c.k1),
                                shared ? nullptr : ptr(c.k2), ptr(c.v), stream_of(dev)),
          "diffattn_paged_append");
    Py_RETURN_NONE;
}

const char* const kAttention = "attention over a paged cache";

PyObject* attention(PyObject* const* a) {
    // q1, k1_cache, q2, k2_cache, v_cache, block_table, lengths, q_lengths, tree_mask, coefficient, out, norm, norm_eps,
    // norm_weight, norm_bias, out_scale
    Tensor q1 = need(a[0], "q1", 4);
    Cache c(a[1], a[3], a[4], a[5], q1.size(0));
    const at::Device dev = c.k1.device();
    const at::ScalarType type = c.k1.scalar_type();
    q1 = need(a[0], "q1", 4, type, dev);
    Tensor q2 = need(a[2], "q2", 4, type, dev);
    const int64_t H = q1.size(1), Tq = q1.size(2);
    if (q2.sizes() != q1.sizes() || q1.size(3) != c.D || H < 1 || H % c.Hk != 0 || c.B < 1)
        bad_value("q1, q2 must be [B, H, Tq, D] with the cache's D and H_kv dividing H, got " + text(q1.sizes()) + ", " +
                  text(q2.sizes()));
    if (Tq < 1 || Tq > 1024) bad_value("1 to 1024 new tokens a call, got " + std::to_string(Tq));
    diffattn_paged_desc d{};
    d.B = c.B;
    d.H = H;
    d.Tq = Tq;
    d.D = c.D;
    d.Dv = c.Dv;
    d.dtype = c.dtype;
    d.kv_group = (int32_t)(H / c.Hk);
    const c10::cuda::OptionalCUDAGuard guard(dev);
    const Tensor lengths = c.lengths(a[6], "lengths");
    const Tensor q_lengths = is_none(a[7]) ? Tensor() : c.lengths(a[7], "q_lengths");
    Tensor mask;
    if (!is_none(a[8])) {
        if (Tq > 64) bad_value("a tree holds up to 64 drafted tokens, got " + std::to_string(Tq));
        mask = tensor(a[8], "tree_mask");
        const int64_t n = mask.dim();
        if (mask.device() != dev || mask.scalar_type() != at::kBool || n < 2 || n > 3 || mask.size(n - 1) != Tq ||
            mask.size(n - 2) != Tq || (n == 3 && mask.size(0) != c.B))
            bad_value("tree_mask must be a bool tensor [B, Tq, Tq] or [Tq, Tq] on the cache's device");
        mask = inner(mask);
        d.mask_stride[0] = n == 3 ? mask.stride(0) : 0;
        d.mask_stride[1] = mask.stride(-2);
    }
    const Lambda lam(a[9], dev, kAttention);
    if (wants_grad({&lam.given})) bad_value("attention over a paged cache is forward only: detach the coefficient");
    no_tangent({&q1, &q2, &c.k1, &c.k2, &c.v}, kAttention);
    if (wants_grad({&q1, &q2, &c.k1, &c.k2, &c.v}))
        bad_value("attention over a paged cache is forward only: call it under torch.no_grad() or detach its inputs");
    q1 = inner(q1);
    q2 = inner(q2);
    Tensor out;
    if (is_none(a[10])) {
        out = fresh_tensor({c.B, H, Tq, c.Dv}, type, dev);
        d.zero_rest = 1;                    // rows past a sequence's queries: left alone only in a given output
    } else {
        out = need(a[10], "out", 4, type, dev);
        if (out.size(0) != c.B || out.size(1) != H || out.size(2) != Tq || out.size(3) != c.Dv || !inner_ok(out))
            bad_value("out must be [B, H, Tq, Dv] with a contiguous innermost dimension");
        no_tangent({&out}, kAttention);
        if (wants_grad({&out})) bad_value("out takes no gradient");
        out.unsafeGetTensorImpl()->bump_version();
    }
    strides3(d.q1_stride, q1);
    strides3(d.q2_stride, q2);
    strides3(d.o_stride, out);
    diffattn_epilogue e{};
    e.norm = norm_code(a[11], true);
    e.eps = (float)number(a[12], "norm_eps");
    e.out_scale = (float)number(a[15], "out_scale");
    Tensor affine[2];
    for (int i = 0; i < 2; ++i) {
        if (is_none(a[13 + i])) continue;
        const char* name = i ? "norm_bias" : "norm_weight";
        const Tensor& t = tensor(a[13 + i], name);
        if (t.device() != dev || !((t.dim() == 2 && t.size(0) == H && t.size(1) == c.Dv) || (t.dim() == 1 && t.size(0) == H * c.Dv)))
            bad_value(std::string(name) + " must be [H, Dv] = (" + std::to_string(H) + ", " + std::to_string(c.Dv) +
                      ") on the inputs' device");
        no_tangent({&t}, kAttention);
        if (wants_grad({&t})) bad_value("attention over a paged cache is forward only: detach the norm's weights");
        affine[i] = plain_f32(t);
    }
    e.weight = fptr(affine[0]);
    e.bias = fptr(affine[1]);
    // from torch's allocator for every call: calls on other streams, and graphs captured one
    // after another, never share it
    const size_t bytes = diffattn_paged_workspace_bytes(&d, &c.pages);
    const Tensor ws = fresh_tensor({(int64_t)(bytes ? bytes : 16)}, at::kByte, dev);
    check(diffattn_paged_decode(&d, &c.pages, ptr(q1), ptr(c.k1), ptr(q2), ptr(c.k2), ptr(c.v), c.table_ptr(),
                                lengths.const_data_ptr<int32_t>(),
                                q_lengths.defined() ? q_lengths.const_data_ptr<int32_t>() : nullptr,
                                static_cast<const uint8_t*>(ptr(mask)), lam.host, fptr(lam.dev), &e, ptr(out), ws.data_ptr(),
                                (size_t)ws.numel(), stream_of(dev)),
          "diffattn_paged_decode");
    if (!is_none(a[10])) {
        Py_INCREF(a[10]);
        return a[10];
    }
    return THPVariable_Wrap(out);
}

// ---------------------------------------------------------------------------
// attention over an encoder's states
// ---------------------------------------------------------------------------
const char* const kCross = "differential_cross_attention";

// Rows as the tensor-core kernels take them, copied where TMA does not (a stride of 0 or not of
// whole 16-byte pieces): 16 sequences, 64 rows of 16 heads over 1500 states that all read: 183 us
// with the copies, 945 on the CUDA cores.
bool tma_rows(const Tensor& t) {
    if (!inner_ok(t) || reinterpret_cast<uintptr_t>(t.const_data_ptr()) % 16 != 0) return false;
    for (int i = 0; i < 3; ++i)
        if (t.size(i) > 1 && (t.stride(i) <= 0 || t.stride(i) % 8 != 0)) return false;
    return true;
}
Tensor rows_for(const Tensor& t, bool tensor_cores) {
    if (!tensor_cores) return inner(t);
    return tma_rows(t) ? t : t.clone(at::MemoryFormat::Contiguous);
}
bool on_tensor_cores(const diffattn_cross_desc& d) {
    return d.dtype == DIFFATTN_BF16 && d.Dv == 128 && (d.D == 64 || d.D == 128);
}

// The autograd node: backward through diffattn_cross_bwd.  Its inputs are q1, k1, q2, k2 (not
// where it is k1), value, and the coefficient where that is a tensor.
struct CrossBackward : public torch::autograd::Node {
    diffattn_cross_desc d{};                // its strides are the forward's: what is unpacked has its own
    float host = 0.f;
    bool shared = false, tensor_lambda = false, device_lambda = false, has_lens = false, has_rests = false;
    torch::autograd::SavedVariable x[5], lens, results[4];  // q1, k1, q2, k2, value; out, out2, lse, rests
    torch::autograd::SavedVariable lam, lam_read;                   // as given, and as the kernels read it
    std::vector<int64_t> lam_shape;
    std::optional<at::TensorOptions> lam_options;
    std::optional<at::Device> dev;
    bool released = false;

    torch::autograd::variable_list apply(torch::autograd::variable_list&& grads) override {
        std::lock_guard<std::mutex> lock(mutex_);
        TORCH_CHECK(!released, "differential_cross_attention: backward a second time through a graph whose saved tensors "
                               "were freed; pass retain_graph=True the first time");
        TORCH_CHECK(!at::GradMode::is_enabled(), "differential_cross_attention is differentiable once (no create_graph)");
        TORCH_CHECK(!joins_default_stream(*this), "differential_cross_attention: this captured backward pass would add to the .grad "
                    "of a leaf that a graph made outside the capture, on the default stream, still holds; drop that graph, "
                    "or make it on another stream");
        const int inputs = shared ? 4 : 5;
        torch::autograd::variable_list result(inputs + tensor_lambda);
        if (!grads[0].defined()) return result;
        const at::ScalarType type = d.dtype == DIFFATTN_BF16 ? at::kBFloat16 : at::kFloat;
        const bool tensor_cores = on_tensor_cores(d);
        const c10::cuda::OptionalCUDAGuard guard(*dev);
        const int64_t Hk = d.H / d.kv_group;
        const int64_t rows[5][4] = {{d.B, d.H, d.Tq, d.D}, {d.B, Hk, d.Tk, d.D}, {d.B, d.H, d.Tq, d.D},
                                    {d.B, Hk, d.Tk, d.D}, {d.B, Hk, d.Tk, d.Dv}};
        Tensor t[5];
        for (int i = 0; i < 5; ++i)
            if (!(shared && i == 3)) t[i] = rows_for(restored(x[i].unpack(), rows[i], type, *dev, kCross), tensor_cores);
        if (shared) t[3] = t[1];
        const int64_t result_rows[4] = {d.B, d.H, d.Tq, d.Dv}, sums[4] = {d.B, d.H, d.Tq, 2};
        const Tensor out = restored_dense(results[0].unpack(shared_from_this()), result_rows, type, *dev, kCross);
        const Tensor out2 = restored_dense(results[1].unpack(), result_rows, type, *dev, kCross);
        const Tensor lse = restored_dense(results[2].unpack(), sums, at::kFloat, *dev, kCross);
        const int64_t rest_rows[5] = {2, d.B, d.H, d.Tq, d.Dv};
        const Tensor rests =
            has_rests ? restored_dense(results[3].unpack(), rest_rows, type, *dev, kCross) : Tensor();
        const Tensor n = has_lens ? restored(lens.unpack(), d.B, at::kInt, *dev, kCross).contiguous() : Tensor();
        Tensor l;
        if (device_lambda)
            l = restored(lam_read.unpack(), lam_shape, d.lambda_dtype == DIFFATTN_BF16 ? at::kBFloat16 : at::kFloat, *dev, kCross);
        if (tensor_lambda) lam.unpack();        // checks that it was not changed in place
        const Tensor g = rows_for(grads[0].scalar_type() == type ? grads[0] : grads[0].to(type), tensor_cores);
        diffattn_cross_desc c = d;
        strides3(c.q1_stride, t[0]);
        strides3(c.k1_stride, t[1]);
        strides3(c.q2_stride, t[2]);
        strides3(c.k2_stride, t[3]);
        strides3(c.v_stride, t[4]);
        strides3(c.o_stride, out);
        strides3(c.dout_stride, g);
        // position of each input among the node's
        const int at[5] = {0, 1, 2, shared ? 1 : 3, shared ? 3 : 4};
        Tensor dx[5], dlam;
        for (int i : {0, 2})
            if (task_should_compute_output(at[i])) dx[i] = fresh_tensor(t[i].sizes(), type, *dev);
        if (task_should_compute_output(at[1]) || task_should_compute_output(at[3]) || task_should_compute_output(at[4]))
            for (int i : {1, 3, 4})
                if (!(shared && i == 3)) dx[i] = fresh_tensor(t[i].sizes(), type, *dev);
        if (tensor_lambda && task_should_compute_output(inputs))
            dlam = fresh_tensor({}, d.lambda_dtype == DIFFATTN_BF16 ? at::kBFloat16 : at::kFloat, *dev);
        const size_t bytes = diffattn_cross_bwd_workspace_bytes(&c);
        const Tensor ws = fresh_tensor({(int64_t)bytes}, at::kByte, *dev);
        const int rc = diffattn_cross_bwd_ex(&c, ptr(t[0]), ptr(t[1]), ptr(t[2]), ptr(t[3]), ptr(t[4]),
                                          n.defined() ? n.const_data_ptr<int32_t>() : nullptr, host, ptr(l), ptr(out),
                                          ptr(out2), fptr(lse), ptr(rests), ptr(g), ptr(dx[0]), ptr(dx[1]), ptr(dx[2]), ptr(dx[3]),
                                          ptr(dx[4]), ptr(dlam), ws.data_ptr(), bytes,
                                          stream_of(*dev));
        TORCH_CHECK(rc == DIFFATTN_OK, "diffattn_cross_bwd: ", diffattn_strerror(rc), " (", rc, ")");
        for (int i = 0; i < 5; ++i)
            if (!(shared && i == 3)) result[at[i]] = dx[i];
        if (dlam.defined()) {
            if (lam_options->device() != *dev || lam_options->dtype() != dlam.dtype()) dlam = dlam.to(*lam_options);
            result[inputs] = lam_shape.empty() ? dlam : dlam.view(lam_shape);
        }
        return result;
    }
    void release_variables() override {
        std::lock_guard<std::mutex> lock(mutex_);
        for (auto& v : x) v.reset_data();
        for (auto& v : results) v.reset_data();
        lam.reset_data();
        lam_read.reset_data();
        lens.reset_data();
        released = true;
    }
    std::string name() const override { return "CrossAttentionBackward"; }
};

PyObject* cross(PyObject* const* a) {
    // q1, k1, q2, k2, value, coefficient, kv_lengths, out, norm, norm_eps, norm_weight, norm_bias, out_scale
    const bool shared = is_none(a[3]) || a[3] == a[1];
    Tensor given[5] = {need(a[0], "q1", 4)};
    const at::Device dev = given[0].device();
    const at::ScalarType type = given[0].scalar_type();
    const char* const names[5] = {"q1", "k1", "q2", "k2", "value"};
    for (int i = 1; i < 5; ++i) given[i] = shared && i == 3 ? given[1] : need(a[i], names[i], 4, type, dev);
    const Tensor &q1 = given[0], &k1 = given[1], &v = given[4];
    diffattn_cross_desc d{};
    d.dtype = dtype_code(q1);
    d.B = q1.size(0);
    d.H = q1.size(1);
    d.Tq = q1.size(2);
    d.D = q1.size(3);
    d.Tk = k1.size(2);
    d.Dv = v.size(3);
    const int64_t Hk = k1.size(1);
    if (given[2].sizes() != q1.sizes() || q1.numel() == 0 || d.D > 128)
        bad_value("q1, q2 must be [B, H, Tq, D] with no size of 0 and D <= 128, got " + text(q1.sizes()) + ", " +
                  text(given[2].sizes()));
    if (given[3].sizes() != k1.sizes() || k1.size(0) != d.B || k1.size(3) != d.D || k1.numel() == 0 || d.H % Hk != 0)
        bad_value("k1, k2 must be [B, H_kv, Tk, D] with H_kv dividing H = " + std::to_string(d.H) + ", got " + text(k1.sizes()) +
                  ", " + text(given[3].sizes()));
    if (v.size(0) != d.B || v.size(1) != Hk || v.size(2) != d.Tk || d.Dv < 1 || d.Dv > 256)
        bad_value("value must be [B, H_kv, Tk, Dv] with Dv <= 256, got " + text(v.sizes()));
    d.kv_group = (int32_t)(d.H / Hk);
    const c10::cuda::OptionalCUDAGuard guard(dev);
    Tensor lens;
    if (!is_none(a[6])) {
        lens = need(a[6], "kv_lengths", 1, at::kInt, dev);
        if (lens.size(0) != d.B) bad_value("kv_lengths must be [B] = (" + std::to_string(d.B) + ",), got " + text(lens.sizes()));
        if (!lens.is_contiguous()) lens = lens.contiguous();
    }
    const Lambda lam(a[5], dev, kCross, true);
    d.lambda_dtype = lam.dev.defined() && lam.dev.scalar_type() == at::kBFloat16 ? DIFFATTN_BF16 : DIFFATTN_F32;
    no_tangent({&given[0], &given[1], &given[2], &given[3], &given[4]}, kCross);
    const bool grad = wants_grad({&given[0], &given[1], &given[2], &given[3], &given[4], &lam.given});
    diffattn_epilogue e{};
    e.norm = norm_code(a[8], true);
    e.eps = (float)number(a[9], "norm_eps");
    e.out_scale = (float)number(a[12], "out_scale");
    Tensor w_given, b_given;
    const Tensor w = affine(a[10], "norm_weight", d.H, d.Dv, dev, &w_given);
    const Tensor b = affine(a[11], "norm_bias", d.H, d.Dv, dev, &b_given);
    no_tangent({&w_given, &b_given}, kCross);
    if (e.norm == DIFFATTN_NORM_NONE && (w.defined() || b.defined()))
        bad_value("norm_weight and norm_bias need norm='rms' or 'group'");
    const bool epilogue = e.norm != DIFFATTN_NORM_NONE || w.defined() || b.defined() || e.out_scale != 1.f;
    if ((grad && (epilogue || !is_none(a[7]))) || wants_grad({&w_given, &b_given}))
        bad_value("gradients are available for the bare operation only (no out=, norm or out_scale): apply "
                  "differential_head_norm to its result");
    e.weight = fptr(w);
    e.bias = fptr(b);
    Tensor t[5], out, out2, lse, rests;
    {
        at::NoGradGuard no_grad;
        const bool tensor_cores = on_tensor_cores(d) && (grad || d.kv_group * d.Tq > 4);
        for (int i = 0; i < 5; ++i) t[i] = shared && i == 3 ? t[1] : rows_for(given[i], tensor_cores);
        if (is_none(a[7])) {
            out = fresh_tensor({d.B, d.H, d.Tq, d.Dv}, type, dev);
        } else {
            out = need(a[7], "out", 4, type, dev);
            if (out.size(0) != d.B || out.size(1) != d.H || out.size(2) != d.Tq || out.size(3) != d.Dv || !inner_ok(out))
                bad_value("out must be [B, H, Tq, Dv] with a contiguous innermost dimension");
            no_tangent({&out}, kCross);
            if (out.requires_grad()) bad_value("out takes no gradient");
            out.unsafeGetTensorImpl()->bump_version();
        }
        strides3(d.q1_stride, t[0]);
        strides3(d.k1_stride, t[1]);
        strides3(d.q2_stride, t[2]);
        strides3(d.k2_stride, t[3]);
        strides3(d.v_stride, t[4]);
        strides3(d.o_stride, out);
        if (grad) {
            out2 = fresh_tensor(out.sizes(), type, dev);
            lse = fresh_tensor({d.B, d.H, d.Tq, 2}, at::kFloat, dev);
            // (two key tensors 128 wide have their backward on the CUDA cores, which need none)
            if (on_tensor_cores(d) && (d.D == 64 || ptr(t[1]) == ptr(t[3]))) rests = fresh_tensor({2, d.B, d.H, d.Tq, d.Dv}, type, dev);
        }
        // from torch's allocator for every call: calls on other streams, and graphs captured one
        // after another, never share it
        const size_t bytes = diffattn_cross_workspace_bytes(&d);
        const Tensor ws = fresh_tensor({(int64_t)(bytes ? bytes : 16)}, at::kByte, dev);
        check(diffattn_cross_fwd_ex(&d, ptr(t[0]), ptr(t[1]), ptr(t[2]), ptr(t[3]), ptr(t[4]),
                                 lens.defined() ? lens.const_data_ptr<int32_t>() : nullptr, lam.host, ptr(lam.dev), &e, ptr(out),
                                 ptr(out2), lse.defined() ? lse.data_ptr<float>() : nullptr, ptr(rests), ws.data_ptr(), (size_t)ws.numel(),
                                 stream_of(dev)),
              "diffattn_cross_fwd");
    }
    if (grad) {
        auto node = std::shared_ptr<CrossBackward>(new CrossBackward(), torch::autograd::deleteNode);
        torch::autograd::variable_list from;
        for (int i = 0; i < 5; ++i) {
            if (shared && i == 3) continue;
            from.push_back(given[i]);
            // as the kernels read it: a copy where they do not take its layout
            node->x[i] = torch::autograd::SavedVariable(t[i], false);
        }
        if (lam.given.defined()) {
            from.push_back(lam.given);
            node->tensor_lambda = true;
            node->lam = torch::autograd::SavedVariable(lam.given, false);
            node->device_lambda = lam.dev.defined();
            if (lam.dev.defined()) node->lam_read = torch::autograd::SavedVariable(lam.dev, false);
            node->lam_shape = lam.given.sizes().vec();
            node->lam_options = lam.given.options();
        }
        node->has_lens = lens.defined();
        if (lens.defined()) node->lens = torch::autograd::SavedVariable(lens, false);
        node->d = d;
        node->host = lam.host;
        node->shared = shared;
        node->dev = dev;
        node->set_next_edges(torch::autograd::collect_next_edges(from));
        torch::autograd::set_history(out, node);
        node->results[0] = torch::autograd::SavedVariable(out, true);
        node->results[1] = torch::autograd::SavedVariable(out2, false);
        node->results[2] = torch::autograd::SavedVariable(lse, false);
        node->has_rests = rests.defined();
        if (rests.defined()) node->results[3] = torch::autograd::SavedVariable(rests, false);
    }
    if (!is_none(a[7])) {
        Py_INCREF(a[7]);
        return a[7];
    }
    return THPVariable_Wrap(out);
}

// ---------------------------------------------------------------------------
// the module
// ---------------------------------------------------------------------------
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refusal& r) {
        PyErr_SetString(r.type, r.what.c_str());
        return nullptr;
    } catch (const Failure& f) {
        PyObject* e = PyObject_CallFunction(g_diffattn_error, "is", f.code, f.what);
        if (e) {
            PyErr_SetObject(g_diffattn_error, e);
            Py_DECREF(e);
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XDECREF(g_diffattn_error);
    g_diffattn_error = cls;
    Py_RETURN_NONE;
}

PyCFunction as_function(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"rotary", as_function(entry<rotary, 13>), METH_FASTCALL, nullptr},
    {"cross", as_function(entry<cross, 13>), METH_FASTCALL, nullptr},
    {"head_norm", as_function(entry<head_norm, 6>), METH_FASTCALL, nullptr},
    {"append", as_function(entry<append, 17>), METH_FASTCALL, nullptr},
    {"attention", as_function(entry<attention, 16>), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
