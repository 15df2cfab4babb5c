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

// ---------------------------------------------------------------------------
// norm and rotation
// ---------------------------------------------------------------------------
// What a call says besides its rows.
struct Rotary {
    int64_t B = 0, T = 0, D = 0, H = 0, Hk = 0, R = 0, rows = 0;
    int32_t dtype = 0, norm = 0, interleaved = 0, pos64 = 0;
    int64_t pos_stride[2] = {0, 0}, qws = 0, kws = 0;
    float eps = 0.f;
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
    void positions(PyObject* o, at::Device dev) {
        if (is_none(o)) return;
        pos = tensor(o, "positions");
        const bool flat = pos.dim() == 1;
        if (pos.device() != dev || (pos.scalar_type() != at::kInt && pos.scalar_type() != at::kLong) ||
            !((flat && pos.size(0) == T) || (pos.dim() == 2 && pos.size(0) == B && pos.size(1) == T)))
            bad_value("positions must be an int32 or int64 tensor [T] or [B, T] = (" + std::to_string(B) + ", " +
                      std::to_string(T) + ") on the inputs' device");
        pos64 = pos.scalar_type() == at::kLong;
        pos_stride[0] = flat ? 0 : pos.stride(0);
        pos_stride[1] = pos.stride(-1);
    }
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
    check(diffattn_rotary(&d, ptr(x[0]), ptr(x[1]), ptr(x[2]), ptr(x[3]), fptr(r.qw), fptr(r.kw), fptr(r.cos), fptr(r.sin),
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
    std::vector<int64_t> sizes[4];
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
        // unpacking checks that nothing saved was changed in place
        if (c.R > 0) {
            c.cos = tables[0].unpack();
            c.sin = tables[1].unpack();
        }
        const Tensor pos = tables[2].unpack();
        c.pos = pos;
        Tensor wt[2];
        for (int i = 0; i < 2; ++i)
            if (weight[i]) wt[i] = w[i].unpack();
        if (weight[0]) c.qw = plain_f32(wt[0]);
        if (weight[1]) c.kw = plain_f32(wt[1]);
        diffattn_rotary_desc d = c.desc();
        Tensor xs[4], gs[4], dx[4];
        const at::ScalarType type = c.dtype == DIFFATTN_BF16 ? at::kBFloat16 : at::kFloat;
        int out = 0;
        for (int i = 0; i < 4; ++i) {
            if (!given[i]) continue;
            if (c.norm) {
                xs[i] = x[i].unpack();
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
        const c10::cuda::OptionalCUDAGuard guard(*dev);
        const size_t bytes = diffattn_rotary_bwd_workspace_bytes(&d);
        const Tensor ws = fresh_tensor({(int64_t)bytes}, at::kByte, *dev);
        const int rc = diffattn_rotary_bwd(
            &d, ptr(xs[0]), ptr(xs[1]), ptr(xs[2]), ptr(xs[3]), fptr(c.qw), fptr(c.kw), fptr(c.cos), fptr(c.sin), ptr(c.pos),
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
    // q1, k1, q2, k2, cos, sin, positions, norm, norm_eps, q_weight, k_weight, interleaved
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
    r.positions(a[6], dev);
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
            node->w[i] = torch::autograd::SavedVariable(ws[i], false);
        }
        if (r.R > 0) {
            node->tables[0] = torch::autograd::SavedVariable(r.cos, false);
            node->tables[1] = torch::autograd::SavedVariable(r.sin, false);
        }
        if (r.pos.defined()) node->tables[2] = torch::autograd::SavedVariable(r.pos, false);
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

bool wants_grad(std::initializer_list<const Tensor*> ts) {
    if (!at::GradMode::is_enabled()) return false;
    for (const Tensor* t : ts)
        if (t->defined() && t->requires_grad()) return true;
    return false;
}

PyObject* append(PyObject* const* a) {
    // k1, k2, value, k1_cache, k2_cache, v_cache, block_table, lengths, new_lengths, cos, sin, positions, norm, norm_eps,
    // k_weight, interleaved
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
    r.positions(a[11], dev);
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
    check(diffattn_paged_append(&d, c.Dv, vs, &c.pages, ptr(k[0]), ptr(k[1]), ptr(v), fptr(r.kw), fptr(r.cos), fptr(r.sin),
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
    // lambda: a number, or one value on the host or the device
    float lam = 0.f;
    Tensor lam_dev;
    if (THPVariable_Check(a[9])) {
        const Tensor& t = THPVariable_Unpack(a[9]);
        if (t.numel() != 1) bad_value("coefficient must be a scalar");
        no_tangent({&t}, kAttention);
        if (wants_grad({&t})) bad_value("attention over a paged cache is forward only: detach the coefficient");
        if (t.is_cuda()) {
            if (t.device() != dev) bad_value("coefficient tensor must be on the inputs' device");
            lam_dev = plain_f32(t);
        } else {
            lam = (float)t.item().toDouble();
        }
    } else {
        lam = (float)number(a[9], "coefficient");
    }
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
                                static_cast<const uint8_t*>(ptr(mask)), lam, fptr(lam_dev), &e, ptr(out), ws.data_ptr(),
                                (size_t)ws.numel(), stream_of(dev)),
          "diffattn_paged_decode");
    if (!is_none(a[10])) {
        Py_INCREF(a[10]);
        return a[10];
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
    {"rotary", as_function(entry<rotary, 12>), METH_FASTCALL, nullptr},
    {"append", as_function(entry<append, 16>), METH_FASTCALL, nullptr},
    {"attention", as_function(entry<attention, 16>), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
