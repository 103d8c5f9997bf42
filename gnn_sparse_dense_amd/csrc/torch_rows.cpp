// Differentiable row operators: torch autograd nodes around the C calls of
// spmm.h (route, dispatch, combine, segment product, layer norm, attention
// within segments, dropout, a classifier's loss).  Host code
// only; the module checks tensors, allocates outputs through torch and
// enqueues on torch's current stream.
//
// The nodes are C++ because a small training call is host time: a layer norm
// of 9 x 368 with its gradients takes 71 us, and took 127 us with the backward
// functions in Python (the engine by itself, around an identity: 43 us).
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <c10/hip/HIPGraphsC10Utils.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/functions/accumulate_grad.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/extension.h>

#include <algorithm>
#include <cmath>
#include <stdexcept>
#include <string>
#include <unordered_set>
#include <vector>

#include "spmm.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

// ---- errors and checks: the types the Python binding raises ----

struct LibraryError : std::runtime_error {
    int status;
    std::string message;
    LibraryError(int s, const std::string &m)
        : std::runtime_error("[" + std::to_string(s) + "] " + m), status(s), message(m) {}
};

void check(int status) {
    if (status == SPMM_OK) return;
    char message[512];
    spmm_last_error(message, sizeof(message));
    throw LibraryError(status, message);
}

std::string name_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "float32";
        case at::kDouble: return "float64";
        case at::kHalf: return "float16";
        case at::kBFloat16: return "bfloat16";
        case at::kLong: return "int64";
        case at::kInt: return "int32";
        default: return c10::toString(t);
    }
}

std::string name_of(at::IntArrayRef shape) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + (shape.size() == 1 ? ",)" : ")");
}

int rows_type(const char *name, const Tensor &t, int64_t dim) {
    if (t.dim() != dim)
        throw py::value_error(std::string(name) + " has " + std::to_string(t.dim()) + " dimensions, expected " +
                              std::to_string(dim));
    switch (t.scalar_type()) {
        case at::kFloat: return SPMM_F32;
        case at::kBFloat16: return SPMM_BF16;
        case at::kHalf: return SPMM_F16;
        default: break;
    }
    throw py::type_error(std::string(name) + " must be float32, bfloat16 or float16, got " + name_of(t.scalar_type()));
}

void check_like(const char *name, const Tensor &t, at::IntArrayRef shape, at::Device device) {
    if (t.sizes() != shape)
        throw py::value_error(std::string(name) + " has shape " + name_of(t.sizes()) + ", expected " + name_of(shape));
    if (!t.is_cuda()) throw py::value_error(std::string(name) + " must be a GPU tensor");
    if (t.device() != device)
        throw py::value_error(std::string(name) + " is on " + t.device().str() + ", expected " + device.str());
}

// A weight in fp32 or the rows' own type: its type code.
int weight_type(const char *name, const Tensor &w, const Tensor &rows) {
    if (w.scalar_type() != at::kFloat && w.scalar_type() != rows.scalar_type())
        throw py::type_error(std::string(name) + " must be float32 or " + name_of(rows.scalar_type()) + ", got " +
                             name_of(w.scalar_type()));
    return rows_type(name, w, w.dim());
}

void check_offsets(const Tensor &offsets, int64_t E, at::Device device) {
    if (offsets.scalar_type() != at::kLong)
        throw py::type_error("offsets must be int64, got " + name_of(offsets.scalar_type()));
    check_like("offsets", offsets, {E + 1}, device);
}

template <typename P = void>
P *ptr(const Tensor &t) {
    return t.defined() ? static_cast<P *>(t.data_ptr()) : nullptr;
}

void *stream_of(const Tensor &t) { return c10::hip::getCurrentHIPStream(t.get_device()).stream(); }

Tensor packed(const Tensor &t) { return t.defined() ? t.contiguous() : t; }

Tensor scratch(int64_t bytes, const Tensor &like) {
    return bytes ? at::empty({bytes}, like.options().dtype(at::kByte)) : Tensor();
}

int code(const Tensor &t) {
    return t.scalar_type() == at::kFloat ? SPMM_F32 : t.scalar_type() == at::kBFloat16 ? SPMM_BF16 : SPMM_F16;
}

// A tangent of forward mode takes the node too, which refuses it: the plain
// calls would drop it.
bool wants_grad(const Tensor &a, const Tensor &b = {}, const Tensor &c = {}) {
    const bool backward = at::GradMode::is_enabled();
    for (const Tensor *t : {&a, &b, &c})
        if (t->defined() && ((backward && t->requires_grad()) || t->_fw_grad(/*level=*/0).defined())) return true;
    return false;
}

bool capturing(const c10::hip::HIPStream &stream) {
    if (!stream.stream()) return false;                  // the default stream cannot be captured
    const c10::hip::HIPStreamGuard guard(stream);
    return c10::hip::currentStreamCaptureStatusMayInitCtx() != c10::hip::CaptureStatus::None;
}

// torch hands a gradient over on the stream of the node that takes it, and a
// leaf's on the stream of its first use, as long as a graph of the leaf lives.
// Where this backward pass is captured and that is the default stream, the
// hand-over would tie the capture to a stream that cannot be captured, which
// ends the process: refused before the gradient exists, for every node that this
// pass still leads to from here, torch's among them.  A leaf's stream of another
// kind joins the capture, and torch joins it back at the end of the pass (its
// own graphed callables keep such graphs of their warm-up); other nodes' streams
// it does not join back, so those are refused too.
void refuse_nodes_outside_capture(const Tensor &grad) {
    if (!capturing(c10::hip::getCurrentHIPStream(grad.get_device()))) return;
    const auto node = torch::autograd::get_current_node();
    std::vector<torch::autograd::Node *> todo;
    std::unordered_set<torch::autograd::Node *> seen;
    if (node) todo.push_back(node.get());
    while (!todo.empty()) {
        torch::autograd::Node *from = todo.back();
        todo.pop_back();
        for (size_t i = 0; i < from->num_outputs(); ++i) {
            if (!from->task_should_compute_output(i)) continue;
            torch::autograd::Node *to = from->next_edge(i).function.get();
            if (!seen.insert(to).second) continue;
            if (const auto stream = to->stream()) {
                const auto on = c10::hip::HIPStreamMasqueradingAsCUDA(*stream).hip_stream();
                const bool leaf = dynamic_cast<torch::autograd::AccumulateGrad *>(to);
                if (!(leaf && on.stream()) && !capturing(on))
                    throw std::runtime_error(
                        "backward of a row operator is captured while a graph of the same leaf lives that was built on "
                        "a stream outside the capture: drop that graph first");
            }
            todo.push_back(to);
        }
    }
}

// Gradients that would themselves be differentiated raise when that happens.
// reads[i]: the inputs of the node, by their place among its edges, that output
// i depends on next to the incoming gradients.  What raises stands between the
// output and the graphs of all of these, so that the way to any one of them
// leads through it: a graph of the output alone is not walked where only an
// input's gradient is asked for.
using Reads = std::initializer_list<size_t>;

variable_list once(const variable_list &grads, variable_list outputs, std::initializer_list<Reads> reads) {
    if (!at::GradMode::is_enabled()) return outputs;
    const auto node = torch::autograd::get_current_node();
    size_t i = 0;
    for (const Reads &inputs : reads) {
        Tensor &out = outputs[i++];
        if (!out.defined()) continue;
        torch::autograd::edge_list from;
        for (const Tensor &g : grads)
            if (g.defined() && g.requires_grad()) from.push_back(torch::autograd::impl::gradient_edge(g));
        for (const size_t at : inputs)                           // an input without a gradient has no function
            if (node->next_edge(at).is_valid()) from.push_back(node->next_edge(at));
        if (!from.empty())
            torch::autograd::create_gradient_edge(
                out, std::make_shared<torch::autograd::Error>(
                         "trying to differentiate twice a row operator, which is differentiable once", std::move(from)));
    }
    return outputs;
}

// ---- route ----

py::tuple route_build(const Tensor &expert, int64_t E) {
    if (expert.scalar_type() != at::kLong)
        throw py::type_error("expert must be int64, got " + name_of(expert.scalar_type()));
    if (expert.dim() != 1 && expert.dim() != 2)
        throw py::value_error("expert has " + std::to_string(expert.dim()) + " dimensions, expected 1 or 2");
    if (!expert.is_cuda()) throw py::value_error("expert must be a GPU tensor");
    const int64_t T = expert.size(0), k = expert.dim() == 2 ? expert.size(1) : 1, pairs = T * k;
    if (k < 1) throw py::value_error("expert must have at least one choice per row");
    int64_t bytes;
    check(spmm_route_workspace(pairs, E, &bytes));               // refuses sizes before any allocation
    const Tensor e = expert.contiguous(), work = scratch(bytes, e);
    const Tensor offsets = at::empty({E + 1}, e.options());
    const Tensor order = at::empty({pairs}, e.options().dtype(at::kInt));
    const Tensor position = at::empty({T, k}, e.options().dtype(at::kInt));
    check(spmm_route_build(ptr<int64_t>(e), pairs, E, ptr<int64_t>(offsets), ptr<int32_t>(order),
                           ptr<int32_t>(position), ptr(work), bytes, stream_of(e)));
    return py::make_tuple(offsets, order, position, T, k);
}

struct Route {
    Tensor offsets, order, position;
    int64_t T, k, E;
};

void run_dispatch(const Route &r, const Tensor &x, const Tensor &weight, int wtype, const Tensor &xs) {
    check(spmm_route_dispatch(ptr<int64_t>(r.offsets), ptr<int32_t>(r.order), r.T, r.k, r.E, ptr(x), ptr(weight),
                              wtype, ptr(xs), x.size(1), code(x), stream_of(x)));
}

void run_combine(const Route &r, const Tensor &rows, const Tensor &weight, int wtype, const Tensor &out) {
    check(spmm_route_combine(ptr<int64_t>(r.offsets), ptr<int32_t>(r.position), r.T, r.k, r.E, ptr(rows),
                             ptr(weight), wtype, ptr(out), rows.size(1), code(rows), stream_of(rows)));
}

void keep(AutogradContext *ctx, const Route &r, variable_list more) {
    more.insert(more.end(), {r.offsets, r.order, r.position});
    ctx->save_for_backward(std::move(more));
    ctx->saved_data["T"] = r.T;
    ctx->saved_data["k"] = r.k;
    ctx->saved_data["E"] = r.E;
}

Route kept(AutogradContext *ctx, const variable_list &saved) {
    const size_t n = saved.size();
    return {saved[n - 3], saved[n - 2], saved[n - 1], ctx->saved_data["T"].toInt(), ctx->saved_data["k"].toInt(),
            ctx->saved_data["E"].toInt()};
}

// ---- dispatch ----

Tensor dispatched(const Route &r, const Tensor &x) {
    const Tensor xs = at::empty({r.T * r.k, x.size(1)}, x.options());
    run_dispatch(r, x.contiguous(), {}, SPMM_F32, xs);
    return xs;
}

struct Dispatch : torch::autograd::Function<Dispatch> {
    static Tensor forward(AutogradContext *ctx, const Tensor &x, const Route &r) {
        keep(ctx, r, {});
        return dispatched(r, x);
    }

    static variable_list backward(AutogradContext *ctx, variable_list grads) {
        refuse_nodes_outside_capture(grads[0]);
        const Route r = kept(ctx, ctx->get_saved_variables());
        const Tensor dxs = grads[0].contiguous();
        const Tensor dx = at::empty({r.T, dxs.size(1)}, dxs.options());
        run_combine(r, dxs, {}, SPMM_F32, dx);
        return once(grads, {dx, Tensor()}, {{}});
    }
};

Tensor dispatch(const Tensor &offsets, const Tensor &order, const Tensor &position, int64_t T, int64_t k, int64_t E,
                const Tensor &x) {
    rows_type("x", x, 2);
    check_like("x", x, {T, x.size(1)}, offsets.device());
    const Route r = {offsets, order, position, T, k, E};
    return wants_grad(x) ? Dispatch::apply(x, r) : dispatched(r, x);
}

// ---- combine ----

Tensor combined(const Route &r, const Tensor &rows, const Tensor &weight) {
    const Tensor out = at::empty({r.T, rows.size(1)}, rows.options());
    run_combine(r, rows, weight, weight.defined() ? code(weight) : SPMM_F32, out);
    return out;
}

struct Combine : torch::autograd::Function<Combine> {
    static Tensor forward(AutogradContext *ctx, const Tensor &rows_, const std::optional<Tensor> &weight_,
                          const Route &r) {
        const Tensor rows = rows_.contiguous(), weight = packed(weight_.value_or(Tensor()));
        // rows are read again only for the weights' gradient
        keep(ctx, r, {weight.defined() && weight_->requires_grad() ? rows : Tensor(), weight});
        return combined(r, rows, weight);
    }

    static variable_list backward(AutogradContext *ctx, variable_list grads) {
        refuse_nodes_outside_capture(grads[0]);
        const variable_list saved = ctx->get_saved_variables();
        const Route r = kept(ctx, saved);
        const Tensor &rows = saved[0], &weight = saved[1], dout = grads[0].contiguous();
        const int wtype = weight.defined() ? code(weight) : SPMM_F32;
        Tensor drows, dweight;
        if (ctx->needs_input_grad(0)) drows = at::empty({r.T * r.k, dout.size(1)}, dout.options());
        if (weight.defined() && ctx->needs_input_grad(1)) {
            dweight = at::empty_like(weight);
            check(spmm_route_combine_backward(ptr<int64_t>(r.offsets), ptr<int32_t>(r.order), r.T, r.k, r.E,
                                              ptr(rows), ptr(weight), wtype, ptr(dout), ptr(drows), ptr(dweight),
                                              dout.size(1), code(dout), stream_of(dout)));
        } else if (drows.defined()) {
            run_dispatch(r, dout, weight, wtype, drows);
        }
        const Reads weights = {1}, none = {};
        return once(grads, {drows, dweight, Tensor()}, {weight.defined() ? weights : none, {0}});
    }
};

Tensor combine(const Tensor &offsets, const Tensor &order, const Tensor &position, int64_t T, int64_t k, int64_t E,
               const Tensor &rows, const std::optional<Tensor> &weight) {
    rows_type("rows", rows, 2);
    check_like("rows", rows, {T * k, rows.size(1)}, offsets.device());
    const Tensor w = weight.value_or(Tensor());
    if (w.defined()) {
        weight_type("weight", w, rows);
        check_like("weight", w, {T, k}, offsets.device());
    }
    const Route r = {offsets, order, position, T, k, E};
    return wants_grad(rows, w) ? Combine::apply(rows, weight, r) : combined(r, rows.contiguous(), packed(w));
}

// ---- segment product ----

Tensor product(const Tensor &x, const Tensor &w, const Tensor &offsets) {
    const Tensor y = at::empty({x.size(0), w.size(2)}, x.options());
    check(spmm_segment_product(ptr(x), ptr(w), ptr<int64_t>(offsets), ptr(y), x.size(0), w.size(0), w.size(1),
                               w.size(2), code(x), stream_of(x)));
    return y;
}

struct SegmentMatmul : torch::autograd::Function<SegmentMatmul> {
    static Tensor forward(AutogradContext *ctx, const Tensor &x_, const Tensor &w_, const Tensor &offsets_) {
        const Tensor x = x_.contiguous(), w = w_.contiguous(), offsets = offsets_.contiguous();
        ctx->save_for_backward({w_.requires_grad() ? x : Tensor(), x_.requires_grad() ? w : Tensor(), offsets});
        ctx->saved_data["shape"] = w.sizes();
        return product(x, w, offsets);
    }

    static variable_list backward(AutogradContext *ctx, variable_list grads) {
        refuse_nodes_outside_capture(grads[0]);
        const variable_list saved = ctx->get_saved_variables();
        const Tensor &x = saved[0], &w = saved[1], &offsets = saved[2], dy = grads[0].contiguous();
        const auto shape = ctx->saved_data["shape"].toIntVector();
        const int64_t R = dy.size(0), E = shape[0], I = shape[1], O = shape[2];
        Tensor dx, dw;
        if (ctx->needs_input_grad(0)) {
            dx = at::empty({R, I}, dy.options());
            check(spmm_segment_product_dx(ptr(dy), ptr(w), ptr<int64_t>(offsets), ptr(dx), R, E, I, O, code(dy),
                                          stream_of(dy)));
        }
        if (ctx->needs_input_grad(1)) {
            int64_t bytes;
            check(spmm_segment_workspace(R, E, I, O, code(dy), &bytes));
            const Tensor work = scratch(bytes, dy);
            dw = at::empty(shape, dy.options());
            check(spmm_segment_product_dw(ptr(x), ptr(dy), ptr<int64_t>(offsets), ptr(dw), R, E, I, O, code(dy),
                                          ptr(work), bytes, stream_of(dy)));
        }
        return once(grads, {dx, dw, Tensor()}, {{1}, {0}});
    }
};

Tensor segment_matmul(const Tensor &x, const Tensor &w, const Tensor &offsets) {
    rows_type("x", x, 2);
    rows_type("w", w, 3);
    if (w.scalar_type() != x.scalar_type())
        throw py::type_error("w must be " + name_of(x.scalar_type()) + ", got " + name_of(w.scalar_type()));
    check_like("x", x, {x.size(0), w.size(1)}, x.device());
    check_like("w", w, w.sizes(), x.device());
    check_offsets(offsets, w.size(0), x.device());
    if (wants_grad(x, w)) return SegmentMatmul::apply(x, w, offsets);
    return product(x.contiguous(), w.contiguous(), offsets.contiguous());
}

// ---- layer norm ----

int norm_weight_type(const Tensor &x, const Tensor &weight, const Tensor &bias) {
    return weight.defined() ? code(weight) : bias.defined() ? code(bias) : code(x);
}

// Rows of x [..., N].
int64_t norm_rows(const Tensor &x) { return x.size(-1) ? x.numel() / x.size(-1) : 0; }

// stats: fp32 [2, R], mean and 1 / deviation of each row, or undefined.
Tensor normed(const Tensor &x, const Tensor &weight, const Tensor &bias, double eps, const Tensor &stats) {
    const Tensor y = at::empty(x.sizes(), x.options());
    const int64_t R = norm_rows(x);
    float *mean = ptr<float>(stats);
    check(spmm_layer_norm(ptr(x), ptr(weight), ptr(bias), norm_weight_type(x, weight, bias), ptr(y), mean,
                          mean ? mean + R : nullptr, R, x.size(-1), eps, code(x), stream_of(x)));
    return y;
}

// The node takes x as it was given: no view stands between it and a leaf.
struct LayerNorm : torch::autograd::Function<LayerNorm> {
    static Tensor forward(AutogradContext *ctx, const Tensor &x_, const std::optional<Tensor> &weight_,
                          const std::optional<Tensor> &bias_, double eps) {
        const Tensor x = x_.contiguous();
        const Tensor weight = packed(weight_.value_or(Tensor())), bias = packed(bias_.value_or(Tensor()));
        const Tensor stats = at::empty({2, norm_rows(x)}, x.options().dtype(at::kFloat));
        ctx->save_for_backward({x, weight, stats});
        ctx->saved_data["wtype"] = (int64_t)norm_weight_type(x, weight, bias);
        ctx->saved_data["bias"] = bias.defined();
        return normed(x, weight, bias, eps, stats);
    }

    static variable_list backward(AutogradContext *ctx, variable_list grads) {
        refuse_nodes_outside_capture(grads[0]);
        const variable_list saved = ctx->get_saved_variables();
        const Tensor &x = saved[0], &weight = saved[1], &stats = saved[2], dy = grads[0].contiguous();
        const int wtype = (int)ctx->saved_data["wtype"].toInt();
        const auto wopts = x.options().dtype(wtype == SPMM_F32 ? at::kFloat : x.scalar_type());
        const int64_t R = norm_rows(x), N = x.size(-1);
        Tensor dx, dweight, dbias, work;
        if (ctx->needs_input_grad(0)) dx = at::empty(x.sizes(), x.options());
        // an input that is not given has no place among the edges
        const size_t after = weight.defined() ? 2 : 1;
        if (weight.defined() && ctx->needs_input_grad(1)) dweight = at::empty({N}, wopts);
        if (ctx->saved_data["bias"].toBool() && ctx->needs_input_grad(after)) dbias = at::empty({N}, wopts);
        int64_t bytes = 0;
        if (dweight.defined() || dbias.defined()) {
            check(spmm_layer_norm_workspace(R, N, code(x), &bytes));
            work = scratch(bytes, x);
        }
        float *mean = ptr<float>(stats);
        check(spmm_layer_norm_backward(ptr(dy), ptr(x), ptr(weight), wtype, mean, mean ? mean + R : nullptr, ptr(dx),
                                       ptr(dweight), ptr(dbias), R, N, code(x), ptr(work), bytes, stream_of(x)));
        const Reads both = {0, 1}, first = {0};
        return once(grads, {dx, dweight, dbias, Tensor()}, {weight.defined() ? both : first, {0}, {}});
    }
};

Tensor layer_norm(const Tensor &x, const std::optional<Tensor> &weight_, const std::optional<Tensor> &bias_,
                  double eps) {
    if (x.dim() < 1) throw py::value_error("x must have at least one dimension");
    const int64_t N = x.size(-1);
    rows_type("x", x, x.dim());
    const Tensor weight = weight_.value_or(Tensor()), bias = bias_.value_or(Tensor());
    if (weight.defined()) {
        weight_type("weight", weight, x);
        check_like("weight", weight, {N}, x.device());
    }
    if (bias.defined()) {
        weight_type("bias", bias, x);
        check_like("bias", bias, {N}, x.device());
    }
    if (weight.defined() && bias.defined() && weight.scalar_type() != bias.scalar_type())
        throw py::type_error("weight (" + name_of(weight.scalar_type()) + ") and bias (" +
                             name_of(bias.scalar_type()) + ") must have one type");
    check_like("x", x, x.sizes(), x.device());
    return wants_grad(x, weight, bias) ? LayerNorm::apply(x, weight_, bias_, eps)
                                       : normed(x.contiguous(), packed(weight), packed(bias), eps, {});
}

// ---- attention within segments ----

// Rows whose heads stand next to each other are taken as they are, at any
// distance (the parts of a joint projection); others are packed first.
Tensor rows_apart(const Tensor &t) {
    const bool heads = t.size(2) == 1 || t.stride(2) == 1;
    const bool row = t.size(1) == 1 || t.stride(1) == t.size(2);
    const bool apart = t.size(0) <= 1 || t.stride(0) >= t.size(1) * t.size(2);
    return t.numel() && heads && row && apart && t.stride(0) < INT32_MAX ? t : t.contiguous();
}

int64_t apart(const Tensor &t) {
    const int64_t width = t.size(1) * t.size(2);
    return t.size(0) > 1 ? std::max(t.stride(0), width) : width;
}

struct Heads {
    Tensor q, k, v, offsets, key_offsets;
    bool causal;
    double scale;

    int64_t S() const { return offsets.size(0) - 1; }
};

// rest and lse: what the backward pass reads, or undefined.
Tensor attended(const Heads &h, const Tensor &rest, const Tensor &lse) {
    const int64_t R = h.q.size(0), H = h.q.size(1), D = h.q.size(2), K = h.k.size(0), Hk = h.k.size(1);
    int64_t bytes;
    check(spmm_segment_attention_workspace(R, K, h.S(), H, Hk, D, code(h.q), &bytes));
    const Tensor work = scratch(bytes, h.q), out = at::empty(h.q.sizes(), h.q.options());
    check(spmm_segment_attention(ptr(h.q), apart(h.q), ptr(h.k), apart(h.k), ptr(h.v), apart(h.v),
                                 ptr<int64_t>(h.offsets), ptr<int64_t>(h.key_offsets), ptr(out), ptr(rest),
                                 ptr<float>(lse), R, K, h.S(), H, Hk, D, h.scale, h.causal, code(h.q), ptr(work), bytes,
                                 stream_of(h.q)));
    return out;
}

struct SegmentAttention : torch::autograd::Function<SegmentAttention> {
    static Tensor forward(AutogradContext *ctx, const Tensor &q, const Tensor &k, const Tensor &v, const Heads &given) {
        const Heads h = {rows_apart(q), rows_apart(k), rows_apart(v), given.offsets, given.key_offsets, given.causal,
                         given.scale};
        const Tensor lse = at::empty({q.size(0), q.size(1)}, q.options().dtype(at::kFloat));
        const Tensor rest = q.scalar_type() == at::kFloat ? Tensor() : at::empty(q.sizes(), q.options());
        const Tensor out = attended(h, rest, lse);
        ctx->save_for_backward({h.q, h.k, h.v, h.offsets, h.key_offsets, out, rest, lse});
        ctx->saved_data["causal"] = h.causal;
        ctx->saved_data["scale"] = h.scale;
        return out;
    }

    static variable_list backward(AutogradContext *ctx, variable_list grads) {
        refuse_nodes_outside_capture(grads[0]);
        const variable_list saved = ctx->get_saved_variables();
        const Heads h = {saved[0], saved[1], saved[2], saved[3], saved[4], ctx->saved_data["causal"].toBool(),
                         ctx->saved_data["scale"].toDouble()};
        const Tensor &out = saved[5], &rest = saved[6], &lse = saved[7], dout = grads[0].contiguous();
        const int64_t R = h.q.size(0), H = h.q.size(1), D = h.q.size(2), K = h.k.size(0), Hk = h.k.size(1);
        Tensor dq, dk, dv;
        if (ctx->needs_input_grad(0)) dq = at::empty(h.q.sizes(), h.q.options());
        if (ctx->needs_input_grad(1)) dk = at::empty(h.k.sizes(), h.k.options());
        if (ctx->needs_input_grad(2)) dv = at::empty(h.v.sizes(), h.v.options());
        int64_t bytes;
        check(spmm_segment_attention_backward_workspace(R, K, h.S(), H, Hk, D, code(h.q), &bytes));
        const Tensor work = scratch(bytes, h.q);
        check(spmm_segment_attention_backward(ptr(h.q), apart(h.q), ptr(h.k), apart(h.k), ptr(h.v), apart(h.v),
                                              ptr<int64_t>(h.offsets), ptr<int64_t>(h.key_offsets), ptr(out), ptr(rest),
                                              ptr<float>(lse), ptr(dout), ptr(dq), ptr(dk), ptr(dv), R, K, h.S(), H,
                                              Hk, D, h.scale, h.causal, code(h.q), ptr(work), bytes, stream_of(h.q)));
        return once(grads, {dq, dk, dv, Tensor()}, {{0, 1, 2}, {0, 1, 2}, {0, 1, 2}});
    }
};

Tensor segment_attention(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &offsets_,
                         const std::optional<Tensor> &key_offsets_, bool causal, std::optional<double> scale) {
    rows_type("q", q, 3);
    rows_type("k", k, 3);
    rows_type("v", v, 3);
    if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type())
        throw py::type_error("q (" + name_of(q.scalar_type()) + "), k (" + name_of(k.scalar_type()) + ") and v (" +
                             name_of(v.scalar_type()) + ") must have one type");
    check_like("q", q, q.sizes(), q.device());
    check_like("k", k, {k.size(0), k.size(1), q.size(2)}, q.device());
    check_like("v", v, k.sizes(), q.device());
    if (offsets_.dim() != 1 || offsets_.size(0) < 2)
        throw py::value_error("offsets has shape " + name_of(offsets_.sizes()) + ", expected (segments + 1,)");
    check_offsets(offsets_, offsets_.size(0) - 1, q.device());
    const Tensor offsets = offsets_.contiguous();
    Tensor key_offsets = offsets;
    if (key_offsets_) {
        if (key_offsets_->scalar_type() != at::kLong)
            throw py::type_error("key_offsets must be int64, got " + name_of(key_offsets_->scalar_type()));
        check_like("key_offsets", *key_offsets_, offsets.sizes(), q.device());
        key_offsets = key_offsets_->contiguous();
    } else if (q.size(0) != k.size(0)) {
        throw py::value_error("q has " + std::to_string(q.size(0)) + " rows and k " + std::to_string(k.size(0)) +
                              ": key_offsets are needed");
    }
    const double by = scale.value_or(1.0 / std::sqrt((double)q.size(2)));
    if (wants_grad(q, k, v))
        return SegmentAttention::apply(q, k, v, Heads{{}, {}, {}, offsets, key_offsets, causal, by});
    return attended({rows_apart(q), rows_apart(k), rows_apart(v), offsets, key_offsets, causal, by}, {}, {});
}

// ---- dropout ----

Tensor dropped(const Tensor &x, const Tensor &residual, const Tensor &seed, double p, int64_t offset) {
    const Tensor y = at::empty(x.sizes(), x.options());
    check(spmm_dropout(ptr(x), ptr(residual), ptr(y), x.numel(), p, ptr<int64_t>(seed), offset, code(x),
                       stream_of(x)));
    return y;
}

struct Dropout : torch::autograd::Function<Dropout> {
    static Tensor forward(AutogradContext *ctx, const Tensor &x, const std::optional<Tensor> &residual,
                          const Tensor &seed, double p, int64_t offset) {
        ctx->save_for_backward({seed});
        ctx->saved_data["p"] = p;
        ctx->saved_data["offset"] = offset;
        ctx->saved_data["residual"] = residual.has_value();
        return dropped(x.contiguous(), packed(residual.value_or(Tensor())), seed, p, offset);
    }

    static variable_list backward(AutogradContext *ctx, variable_list grads) {
        refuse_nodes_outside_capture(grads[0]);
        const Tensor seed = ctx->get_saved_variables()[0];
        Tensor dx;
        if (ctx->needs_input_grad(0))
            dx = dropped(grads[0].contiguous(), {}, seed, ctx->saved_data["p"].toDouble(),
                         ctx->saved_data["offset"].toInt());
        // the residual's gradient is dy itself, graph and all
        const Tensor dresidual = ctx->saved_data["residual"].toBool() ? grads[0] : Tensor();
        return once(grads, {dx, dresidual, Tensor(), Tensor(), Tensor()}, {{}});
    }
};

Tensor dropout(const Tensor &x, double p, const Tensor &seed, int64_t offset, const std::optional<Tensor> &residual_) {
    rows_type("x", x, x.dim());
    check_like("x", x, x.sizes(), x.device());
    const Tensor residual = residual_.value_or(Tensor());
    if (residual.defined()) {
        if (residual.scalar_type() != x.scalar_type())
            throw py::type_error("residual must be " + name_of(x.scalar_type()) + ", got " +
                                 name_of(residual.scalar_type()));
        check_like("residual", residual, x.sizes(), x.device());
    }
    if (seed.scalar_type() != at::kLong) throw py::type_error("seed must be int64, got " + name_of(seed.scalar_type()));
    if (seed.numel() != 1) throw py::value_error("seed must have one element, got " + std::to_string(seed.numel()));
    check_like("seed", seed, seed.sizes(), x.device());
    return wants_grad(x, residual) ? Dropout::apply(x, residual_, seed, p, offset)
                                   : dropped(x.contiguous(), packed(residual), seed, p, offset);
}

// ---- the loss of a linear classifier ----

struct LossSizes {
    int64_t state, forward, backward;

    LossSizes(const Tensor &x, const Tensor &w) {
        check(spmm_linear_cross_entropy_workspace(x.size(0), x.size(1), w.size(0), code(x), &state, &forward,
                                                  &backward));
    }
};

Tensor lost(const Tensor &x, const Tensor &w, const Tensor &target, int64_t reduction, const Tensor &state,
            const LossSizes &sizes) {
    const Tensor work = scratch(sizes.forward, x);
    const auto opts = x.options().dtype(at::kFloat);
    const Tensor loss = reduction == SPMM_LOSS_ROWS ? at::empty({x.size(0)}, opts) : at::empty({}, opts);
    check(spmm_linear_cross_entropy(ptr(x), ptr(w), ptr<int64_t>(target), ptr<float>(loss), x.size(0), x.size(1),
                                    w.size(0), (int)reduction, code(x), ptr(state), sizes.state, ptr(work),
                                    sizes.forward, stream_of(x)));
    return loss;
}

struct LinearCrossEntropy : torch::autograd::Function<LinearCrossEntropy> {
    static Tensor forward(AutogradContext *ctx, const Tensor &x_, const Tensor &w_, const Tensor &target,
                          int64_t reduction) {
        const Tensor x = x_.contiguous(), w = w_.contiguous();
        const LossSizes sizes(x, w);
        const Tensor state = scratch(sizes.state, x);
        ctx->save_for_backward({x, w, target, state});
        ctx->saved_data["reduction"] = reduction;
        return lost(x, w, target, reduction, state, sizes);
    }

    static variable_list backward(AutogradContext *ctx, variable_list grads) {
        refuse_nodes_outside_capture(grads[0]);
        const variable_list saved = ctx->get_saved_variables();
        const Tensor &x = saved[0], &w = saved[1], &target = saved[2], &state = saved[3], dloss = grads[0].contiguous();
        const LossSizes sizes(x, w);
        const Tensor work = scratch(sizes.backward, x);
        Tensor dx, dw;
        if (ctx->needs_input_grad(0)) dx = at::empty(x.sizes(), x.options());
        if (ctx->needs_input_grad(1)) dw = at::empty(w.sizes(), w.options());
        check(spmm_linear_cross_entropy_backward(ptr(x), ptr(w), ptr<int64_t>(target), ptr<float>(dloss), ptr(dx),
                                                 ptr(dw), x.size(0), x.size(1), w.size(0),
                                                 (int)ctx->saved_data["reduction"].toInt(), code(x), ptr(state),
                                                 sizes.state, ptr(work), sizes.backward, stream_of(x)));
        return once(grads, {dx, dw, Tensor(), Tensor()}, {{0, 1}, {0, 1}});
    }
};

Tensor linear_cross_entropy(const Tensor &x, const Tensor &w, const Tensor &target_, const std::string &reduction) {
    rows_type("x", x, 2);
    rows_type("w", w, 2);
    if (w.scalar_type() != x.scalar_type())
        throw py::type_error("w must be " + name_of(x.scalar_type()) + ", got " + name_of(w.scalar_type()));
    check_like("x", x, x.sizes(), x.device());
    check_like("w", w, {w.size(0), x.size(1)}, x.device());
    if (target_.scalar_type() != at::kLong)
        throw py::type_error("target must be int64, got " + name_of(target_.scalar_type()));
    check_like("target", target_, {x.size(0)}, x.device());
    const int64_t by = reduction == "none"   ? SPMM_LOSS_ROWS
                       : reduction == "sum"  ? SPMM_LOSS_SUM
                       : reduction == "mean" ? SPMM_LOSS_MEAN
                                             : -1;
    if (by < 0) throw py::value_error("reduction must be 'none', 'sum' or 'mean', got '" + reduction + "'");
    const Tensor target = target_.contiguous();
    if (wants_grad(x, w)) return LinearCrossEntropy::apply(x, w, target, by);
    const Tensor rows = x.contiguous(), classes = w.contiguous();
    const LossSizes sizes(rows, classes);
    return lost(rows, classes, target, by, scratch(sizes.state, rows), sizes);
}

}  // namespace

PYBIND11_MODULE(_rows, m) {
    py::register_exception_translator([](std::exception_ptr p) {
        try {
            if (p) std::rethrow_exception(p);
        } catch (const LibraryError &e) {
            const py::object type = py::module_::import("gnn_sparse_dense_amd").attr("SpmmError");
            const py::object value = type(e.status, e.message);
            PyErr_SetObject(type.ptr(), value.ptr());
        }
    });
    m.def("route_build", &route_build);
    m.def("dispatch", &dispatch);
    m.def("combine", &combine);
    m.def("segment_matmul", &segment_matmul);
    m.def("layer_norm", &layer_norm);
    m.def("segment_attention", &segment_attention);
    m.def("dropout", &dropout);
    m.def("linear_cross_entropy", &linear_cross_entropy);
}
