// The token mixer's calls on PyTorch tensors as a Python extension module: the
// small calls of serving and the differentiable operations with their autograd
// nodes.
//
// Both are bound by the host where they are small.  One token of the convolution
// takes 8.9 us through ctypes (with an output of the caller's) and 3.8 as a function
// of this module, calls back to back, for a kernel of 1.9 (4.1 from cold caches);
// as a registered PyTorch operator it took 1.7 times as long as that way.  A training
// step of a block norm (65536 rows of 128) took 220 us with autograd nodes in Python,
// half of it in the engine's thread, where every Python object is cold, for 43 us of
// kernels, and takes 135.
//
// What a function accepts is exactly what the Python function that calls it
// accepts.  For anything else it returns NotImplemented before it has done
// anything, and the Python function finds out what to say.  What fails later is
// raised as it is, once: the call is not made again.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <stdexcept>
#include <string>

#include "dwconv.h"

namespace {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
using Optional = std::optional<Tensor>;

const void *address(const Tensor &t) { return t.defined() ? t.const_data_ptr() : nullptr; }
void *target(const Tensor &t) { return t.defined() ? t.mutable_data_ptr() : nullptr; }
const float *floats(const Tensor &t) { return static_cast<const float *>(address(t)); }
float *float_target(const Tensor &t) { return static_cast<float *>(target(t)); }
const int *lengths_of(const Tensor &t) { return static_cast<const int *>(address(t)); }
Tensor given(const Optional &t) { return t ? *t : Tensor(); }
dwconv_stream stream_of(const Tensor &t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }
// The caller's tensor is written in place: autograd has to see that.
void written(const Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
Tensor like(const Tensor &t) { return t.defined() ? at::empty(t.sizes(), t.options()) : Tensor(); }
Tensor bytes(size_t n, const Tensor &ref) {
    return n ? at::empty({(int64_t)n}, ref.options().dtype(at::kByte)) : Tensor();
}
// A call that the library refused or that failed.
struct Failed : std::runtime_error {
    dwconv_status status;
    const char *where;
    Failed(dwconv_status st, const char *where_)
        : std::runtime_error(std::string(where_) + ": " + dwconv_status_string(st)), status(st), where(where_) {}
};
void check(dwconv_status st, const char *where) {
    if (st != DWCONV_OK) throw Failed(st, where);
}

// Every requirement on an argument; the words are the Python function's.
struct Refused : std::runtime_error {
    Refused() : std::runtime_error("unsupported arguments") {}
};
void need(bool ok) {
    if (!ok) throw Refused();
}
dwconv_dtype code_of(at::ScalarType t) {
    need(t == at::kFloat || t == at::kHalf || t == at::kBFloat16);
    return t == at::kFloat ? DWCONV_FP32 : t == at::kHalf ? DWCONV_FP16 : DWCONV_BF16;
}
int count(int64_t n) {
    need(n <= INT32_MAX);
    return (int)n;
}
// A view whose last dimension is dense.
void need_rows(const Tensor &t, at::IntArrayRef shape, const Tensor &ref, at::ScalarType type) {
    need(t.is_cuda() && t.device() == ref.device() && t.scalar_type() == type && t.sizes() == shape &&
         (t.stride(-1) == 1 || t.size(-1) <= 1));
}
// An optional dense tensor.
void need_dense(const Tensor &t, at::IntArrayRef shape, const Tensor &ref, at::ScalarType type) {
    if (!t.defined()) return;
    need_rows(t, shape, ref, type);
    need(t.is_contiguous());
}

// Whether a backward pass may follow.  Tangents of forward mode, which goes on
// without gradients, are refused: they would be lost.
bool wants_grad(std::initializer_list<Tensor> in) {
    for (const Tensor &t : in)
        TORCH_CHECK_NOT_IMPLEMENTED(!t.defined() || !t._fw_grad(/*level=*/0).defined(),
                                    "the token mixer's operations have no forward-mode derivatives");
    if (!at::GradMode::is_enabled()) return false;
    for (const Tensor &t : in)
        if (t.defined() && t.requires_grad()) return true;
    return false;
}
// The gradients come out of kernels that have no backward pass of their own: under
// create_graph they would look like constants.  This node says that they are none.
struct Once : torch::autograd::Function<Once> {
    static Tensor forward(AutogradContext *, const Tensor &grad, const Tensor &) { return grad; }
    static variable_list backward(AutogradContext *, variable_list) {
        TORCH_CHECK_NOT_IMPLEMENTED(false, "the token mixer's operations cannot be differentiated twice");
    }
};
// A backward pass's gradients; `in` and `up`: what they depend on.
variable_list once(variable_list grads, const variable_list &in, const variable_list &up) {
    if (!at::GradMode::is_enabled()) return grads;
    for (Tensor &g : grads)
        for (const variable_list *from : {&in, &up})  // on the way to each of them: what is not asked for is not run
            for (const Tensor &t : *from)
                if (g.defined() && t.defined() && t.requires_grad()) g = Once::apply(g, t);
    return grads;
}
// The last dimension dense, as the kernels want it.
Tensor dense_rows(const Tensor &t) { return t.stride(-1) == 1 ? t : t.contiguous(); }

// ---- causal convolution

struct Causal {
    dwconv_dtype dt;
    int B, T, C, W;
    dwconv_activation act;
    Causal(const Tensor &x, const Tensor &w, const Tensor &bias, const Tensor &state, const Tensor &n, int64_t act_)
        : dt(code_of(x.scalar_type())), act((dwconv_activation)act_) {
        need(x.dim() == 3 && w.dim() == 2);
        B = count(x.size(0)); T = count(x.size(1)); C = count(x.size(2)); W = count(w.size(0));
        need_rows(x, x.sizes(), x, x.scalar_type());
        need_dense(w, {W, C}, x, x.scalar_type());
        need_dense(bias, {C}, x, at::kFloat);
        need_dense(state, {B, W - 1, C}, x, x.scalar_type());
        need_dense(n, {B}, x, at::kInt);
    }
    // {y} or {y, window}
    variable_list forward(const Tensor &x, const Tensor &w, const Tensor &bias, const Tensor &state, const Tensor &n,
                          bool with_state) const {
        const Tensor y = at::empty({B, T, C}, x.options());
        const Tensor window = with_state ? at::empty({B, W - 1, C}, x.options()) : Tensor();
        check(dwconv_causal_fwd(B, T, C, W, dt, address(x), x.stride(0), x.stride(1), address(w), floats(bias), act,
                                address(state), lengths_of(n), target(y), target(window), stream_of(x)),
              "dwconv_causal_fwd");
        return with_state ? variable_list{y, window} : variable_list{y};
    }
};

struct CausalNode : torch::autograd::Function<CausalNode> {
    static Tensor forward(AutogradContext *ctx, const Tensor &x, const Tensor &w, const Optional &bias,
                          const Optional &state, const Optional &n, int64_t act) {
        ctx->save_for_backward({x, w, given(bias), given(state), given(n)});
        ctx->saved_data["act"] = act;
        return Causal(x, w, given(bias), given(state), given(n), act)
            .forward(x, w, given(bias), given(state), given(n), false)[0];
    }
    static variable_list backward(AutogradContext *ctx, variable_list up) {
        const variable_list in = ctx->get_saved_variables();
        const Tensor &x = in[0], &w = in[1], &bias = in[2], &state = in[3], dy = dense_rows(up[0]);
        const Causal s(x, w, bias, state, in[4], ctx->saved_data["act"].toInt());
        const auto sums = x.options().dtype(at::kFloat);
        const Tensor dx = at::empty({s.B, s.T, s.C}, x.options()), dw = at::empty({s.W, s.C}, sums), db = like(bias);
        // the node has edges for the tensors that are there: x, w, the bias, the state
        const Tensor ds = state.defined() && ctx->needs_input_grad(2 + bias.defined()) ? like(state) : Tensor();
        const size_t size = dwconv_causal_bwd_workspace_size(s.B, s.T, s.C, s.W, s.dt);
        const Tensor work = bytes(size, x);
        check(dwconv_causal_bwd(s.B, s.T, s.C, s.W, s.dt, address(dy), dy.stride(0), dy.stride(1), address(x),
                                x.stride(0), x.stride(1), address(w), floats(bias), s.act, address(state),
                                lengths_of(in[4]), target(dx), float_target(dw), float_target(db), target(ds),
                                target(work), size, stream_of(x)),
              "dwconv_causal_bwd");
        return once({dx, dw.to(w.scalar_type()), db, ds, Tensor(), Tensor()}, in, up);
    }
};

Tensor causal_conv(const Tensor &x, const Tensor &w, const Optional &bias, const Optional &state, const Optional &n,
                   int64_t act) {
    need(x.is_cuda());
    const c10::DeviceGuard guard(x.device());
    if (wants_grad({x, w, given(bias), given(state)})) return CausalNode::apply(x, w, bias, state, n, act);
    return Causal(x, w, given(bias), given(state), given(n), act)
        .forward(x, w, given(bias), given(state), given(n), false)[0];
}

variable_list causal_fwd(const Tensor &x, const Tensor &w, const Optional &bias, const Optional &state,
                         const Optional &n, int64_t act, bool with_state) {
    need(x.is_cuda());
    const c10::DeviceGuard guard(x.device());
    return Causal(x, w, given(bias), given(state), given(n), act)
        .forward(x, w, given(bias), given(state), given(n), with_state);
}

Tensor causal_step(const Tensor &x, const Tensor &w, const Tensor &state, const Optional &bias, const Optional &slots,
                   int64_t act) {
    need(x.is_cuda());
    const c10::DeviceGuard guard(x.device());
    need(x.dim() == 2 && w.dim() == 2 && state.dim() == 3);
    const int B = count(x.size(0)), C = count(x.size(1)), W = count(w.size(0)), N = count(state.size(0));
    const dwconv_dtype dt = code_of(x.scalar_type());
    const Tensor b = given(bias), at = given(slots);
    need_rows(x, x.sizes(), x, x.scalar_type());
    need_dense(w, {W, C}, x, x.scalar_type());
    need_dense(b, {C}, x, at::kFloat);
    need_dense(state, {N, W - 1, C}, x, x.scalar_type());
    need_dense(at, {B}, x, at::kInt);
    const Tensor y = at::empty({B, C}, x.options());
    check(dwconv_causal_step(B, N, C, W, dt, address(x), x.stride(0), address(w), floats(b), (dwconv_activation)act,
                             target(state), lengths_of(at), target(y), stream_of(x)),
          "dwconv_causal_step");
    written(state);
    return y;
}

// ---- norms around a block

struct Norm {
    dwconv_dtype dt;
    long long outer;
    int inner, C;
    dwconv_norm kind;
    dwconv_gate act;
    float eps;
    bool dense = true;
    long long strides[10];  // of y, residual, gate, dh, dn

    // in: y, residual, gate, w_post, scale, w_pre
    Norm(const variable_list &in, int64_t kind_, int64_t act_, double eps_)
        : dt(code_of(in[0].scalar_type())), kind((dwconv_norm)kind_), act((dwconv_gate)act_), eps((float)eps_) {
        const Tensor &y = in[0];
        const int64_t dims = y.dim();
        need(dims >= 1);
        C = count(y.size(-1));
        inner = dims > 1 ? count(y.size(-2)) : 1;
        outer = 1;
        for (int64_t i = 0; i + 2 < dims; ++i) outer *= y.size(i);
        if (inner == 0) {
            outer = 0;
            inner = 1;
        }
        for (int i = 0; i < 3; ++i) rows(in[i], y, strides + 2 * i);
        for (int i = 3; i < 6; ++i) need_dense(in[i], {C}, y, at::kFloat);
        for (int i = 3; i < 5; ++i) {
            strides[2 * i] = (long long)inner * C;
            strides[2 * i + 1] = C;
        }
    }
    // Strides of t's rows: the dimensions before the last two have to collapse into one.
    void rows(const Tensor &t, const Tensor &y, long long *to) {
        to[0] = (long long)inner * C;
        to[1] = C;
        if (!t.defined()) return;
        need_rows(t, y.sizes(), y, y.scalar_type());
        if (t.is_contiguous()) return;
        dense = false;
        const int64_t dims = t.dim();
        if (dims > 1 && t.size(-2) > 1) to[1] = t.stride(-2);
        bool found = false;
        int64_t span = 0;
        for (int64_t i = dims - 3; i >= 0; --i) {
            const int64_t n = t.size(i), s = t.stride(i);
            if (n == 1) continue;
            if (!found) to[0] = s;
            need(!found || s == span);
            found = true;
            span = n * s;
        }
        if (!found) to[0] = to[1] * inner;
    }
    const long long *steps() const { return dense ? nullptr : strides; }
    // {h} or {h, n}
    variable_list forward(const variable_list &in) const {
        const Tensor h = like(in[0]), n = in[5].defined() ? like(in[0]) : Tensor();
        check(dwconv_block_norm_fwd(outer, inner, C, dt, kind, act, eps, address(in[0]), address(in[1]),
                                    address(in[2]), steps(), floats(in[3]), floats(in[4]), floats(in[5]), target(h),
                                    target(n), stream_of(in[0])),
              "dwconv_block_norm_fwd");
        return n.defined() ? variable_list{h, n} : variable_list{h};
    }
};

struct NormNode : torch::autograd::Function<NormNode> {
    static variable_list forward(AutogradContext *ctx, const Tensor &y, const Optional &residual, const Optional &gate,
                                 const Optional &w_post, const Optional &scale, const Optional &w_pre, int64_t kind,
                                 int64_t act, double eps) {
        const variable_list in{y, given(residual), given(gate), given(w_post), given(scale), given(w_pre)};
        ctx->save_for_backward(in);
        ctx->saved_data["kind"] = kind;
        ctx->saved_data["act"] = act;
        ctx->saved_data["eps"] = eps;
        ctx->set_materialize_grads(false);
        return Norm(in, kind, act, eps).forward(in);
    }
    static variable_list backward(AutogradContext *ctx, variable_list up) {
        const variable_list in = ctx->get_saved_variables();
        const Norm s(in, ctx->saved_data["kind"].toInt(), ctx->saved_data["act"].toInt(),
                     ctx->saved_data["eps"].toDouble());
        const Tensor dh = up[0].defined() ? up[0].contiguous() : Tensor(),
                     dn = up.size() > 1 && up[1].defined() ? up[1].contiguous() : Tensor();
        variable_list grads(9);
        if (!dh.defined() && !dn.defined()) return grads;
        for (int i = 0; i < 6; ++i) grads[i] = like(in[i]);
        const size_t size = dwconv_block_norm_bwd_workspace_size(s.outer, s.inner, s.C, s.dt);
        const Tensor work = bytes(size, in[0]);
        check(dwconv_block_norm_bwd(s.outer, s.inner, s.C, s.dt, s.kind, s.act, s.eps, address(in[0]), address(in[1]),
                                    address(in[2]), address(dh), address(dn), s.steps(), floats(in[3]), floats(in[4]),
                                    floats(in[5]), target(grads[0]), target(grads[1]), target(grads[2]),
                                    float_target(grads[3]), float_target(grads[4]), float_target(grads[5]),
                                    target(work), size, stream_of(in[0])),
              "dwconv_block_norm_bwd");
        return once(std::move(grads), in, up);
    }
};

variable_list block_norm(const Tensor &y, const Optional &residual, const Optional &gate, const Optional &w_post,
                         const Optional &scale, const Optional &w_pre, int64_t kind, int64_t act, double eps) {
    need(y.is_cuda());
    const c10::DeviceGuard guard(y.device());
    const variable_list in{y, given(residual), given(gate), given(w_post), given(scale), given(w_pre)};
    if (wants_grad({in[0], in[1], in[2], in[3], in[4], in[5]}))
        return NormNode::apply(y, residual, gate, w_post, scale, w_pre, kind, act, eps);
    return Norm(in, kind, act, eps).forward(in);
}

variable_list block_norm_fwd(const Tensor &y, const Optional &residual, const Optional &gate, const Optional &w_post,
                             const Optional &scale, const Optional &w_pre, int64_t kind, int64_t act, double eps) {
    need(y.is_cuda());
    const c10::DeviceGuard guard(y.device());
    const variable_list in{y, given(residual), given(gate), given(w_post), given(scale), given(w_pre)};
    return Norm(in, kind, act, eps).forward(in);
}

// ---- gated delta rule

constexpr int kMostGradK = 128;

// Inputs of a call, B x (T x) heads x values, the gates B x (T x) value heads.
struct Delta {
    dwconv_dtype dt, gate_dt;
    int B, T, Hk, Hv, K, V, qk_norm;
    std::vector<long long> strides;  // of q, k, v (without the last dimension), g, beta
    float scale;
    // in: q, k, v, g, beta; lead: dimensions before the heads
    Delta(const variable_list &in, int lead, std::optional<double> scale_, bool qk_norm_)
        : dt(code_of(in[0].scalar_type())), gate_dt(code_of(in[3].scalar_type())), qk_norm(qk_norm_) {
        const Tensor &q = in[0], &v = in[2], &g = in[3];
        need(q.dim() == lead + 2 && v.dim() == lead + 2);
        B = count(q.size(0)); T = lead == 2 ? count(q.size(1)) : 1;
        Hk = count(q.size(lead)); K = count(q.size(lead + 1));
        Hv = count(v.size(lead)); V = count(v.size(lead + 1));
        need(Hk > 0 && Hv % Hk == 0 && (gate_dt == dt || gate_dt == DWCONV_FP32));
        at::DimVector first(q.sizes().begin(), q.sizes().begin() + lead), values(first), gates(first);
        values.append({Hv, V});
        gates.append({Hv});
        need_rows(q, q.sizes(), q, q.scalar_type());
        need_rows(in[1], q.sizes(), q, q.scalar_type());
        need_rows(v, values, q, q.scalar_type());
        for (int i = 3; i < 5; ++i)
            need(in[i].is_cuda() && in[i].device() == q.device() && in[i].scalar_type() == g.scalar_type() &&
                 in[i].sizes() == at::IntArrayRef(gates));
        strides.reserve(18);
        for (int i = 0; i < 5; ++i)
            strides.insert(strides.end(), in[i].strides().begin(), in[i].strides().end() - (i < 3));
        scale = (float)(scale_ ? *scale_ : std::pow((double)K, -0.5));
    }
    // {o} or {o, last state}
    variable_list forward(const variable_list &in, const Tensor &state, const Tensor &n, bool with_state,
                          const Tensor &saved) const {
        const Tensor &q = in[0];
        need_dense(state, {B, Hv, K, V}, q, at::kFloat);
        need_dense(n, {B}, q, at::kInt);
        const Tensor o = at::empty({B, T, Hv, V}, q.options());
        const Tensor last = with_state ? at::empty({B, Hv, K, V}, q.options().dtype(at::kFloat)) : Tensor();
        const size_t size = saved.defined() ? 0 : dwconv_delta_fwd_workspace_size(B, T, Hk, Hv, K, V, dt);
        const Tensor work = bytes(size, q);
        check(dwconv_delta_fwd(B, T, Hk, Hv, K, V, dt, gate_dt, address(q), address(in[1]), address(in[2]),
                               address(in[3]), address(in[4]), strides.data(), scale, qk_norm, floats(state),
                               lengths_of(n), target(o), float_target(last), target(saved), target(work), size,
                               stream_of(q)),
              "dwconv_delta_fwd");
        return with_state ? variable_list{o, last} : variable_list{o};
    }
};

struct DeltaNode : torch::autograd::Function<DeltaNode> {
    static variable_list forward(AutogradContext *ctx, const Tensor &q, const Tensor &k, const Tensor &v,
                                 const Tensor &g, const Tensor &beta, const Optional &state, const Optional &n,
                                 std::optional<double> scale, bool qk_norm, bool with_state) {
        const variable_list in{q, k, v, g, beta};
        const Delta s(in, 2, scale, qk_norm);
        need(s.K <= kMostGradK);  // what the backward pass takes
        const Tensor saved = bytes(dwconv_delta_saved_size(s.B, s.T, s.Hk, s.Hv, s.K, s.V, s.dt), q);
        ctx->save_for_backward({q, k, v, g, beta, given(state), given(n), saved});
        ctx->saved_data["scale"] = scale;
        ctx->saved_data["qk_norm"] = qk_norm;
        ctx->set_materialize_grads(false);
        return s.forward(in, given(state), given(n), with_state, saved);
    }
    static variable_list backward(AutogradContext *ctx, variable_list up) {
        const variable_list in = ctx->get_saved_variables();
        const Tensor last = up.size() > 1 && up[1].defined() ? up[1].contiguous() : Tensor();
        variable_list grads(10);
        if (!up[0].defined() && !last.defined()) return grads;
        Delta s(in, 2, ctx->saved_data["scale"].toOptional<double>(), ctx->saved_data["qk_norm"].toBool());
        const Tensor &q = in[0], &state = in[5], &saved = in[7];
        const Tensor d_out = up[0].defined() ? dense_rows(up[0]) : at::zeros({s.B, s.T, s.Hv, s.V}, q.options());
        s.strides.insert(s.strides.end(), {d_out.stride(0), d_out.stride(1), d_out.stride(2)});
        for (int i = 0; i < 5; ++i) grads[i] = like(in[i]);
        if (state.defined() && ctx->needs_input_grad(5)) grads[5] = like(state);
        const size_t size = dwconv_delta_bwd_workspace_size(s.B, s.T, s.Hk, s.Hv, s.K, s.V, s.dt, saved.defined());
        const Tensor work = bytes(size, q);
        check(dwconv_delta_bwd(s.B, s.T, s.Hk, s.Hv, s.K, s.V, s.dt, s.gate_dt, address(d_out), address(q),
                               address(in[1]), address(in[2]), address(in[3]), address(in[4]), s.strides.data(),
                               s.scale, s.qk_norm, floats(state), lengths_of(in[6]), floats(last), target(grads[0]),
                               target(grads[1]), target(grads[2]), target(grads[3]), target(grads[4]),
                               float_target(grads[5]), address(saved), target(work), size, stream_of(q)),
              "dwconv_delta_bwd");
        return once(std::move(grads), in, up);
    }
};

variable_list gated_delta_rule(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &g, const Tensor &beta,
                               const Optional &state, const Optional &n, std::optional<double> scale, bool qk_norm,
                               bool with_state) {
    need(q.is_cuda());
    const c10::DeviceGuard guard(q.device());
    if (wants_grad({q, k, v, g, beta, given(state)}))
        return DeltaNode::apply(q, k, v, g, beta, state, n, scale, qk_norm, with_state);
    const variable_list in{q, k, v, g, beta};
    return Delta(in, 2, scale, qk_norm).forward(in, given(state), given(n), with_state, Tensor());
}

Tensor delta_step(const Tensor &q, const Tensor &k, const Tensor &v, const Tensor &g, const Tensor &beta,
                  const Tensor &state, const Optional &slots, std::optional<double> scale, bool qk_norm) {
    need(q.is_cuda());
    const c10::DeviceGuard guard(q.device());
    const Delta s({q, k, v, g, beta}, 1, scale, qk_norm);
    const Tensor at = given(slots);
    need(state.dim() == 4);
    need_dense(state, {state.size(0), s.Hv, s.K, s.V}, q, at::kFloat);
    need_dense(at, {s.B}, q, at::kInt);
    const Tensor o = at::empty({s.B, s.Hv, s.V}, q.options());
    check(dwconv_delta_step(s.B, count(state.size(0)), s.Hk, s.Hv, s.K, s.V, s.dt, s.gate_dt, address(q), address(k),
                            address(v), address(g), address(beta), s.strides.data(), s.scale, s.qk_norm,
                            float_target(state), lengths_of(at), target(o), stream_of(q)),
          "dwconv_delta_step");
    written(state);
    return o;
}

// ---- Python

// Positional arguments of a call.
struct Args {
    PyObject *const *at;
    Args(PyObject *const *args, Py_ssize_t given, Py_ssize_t wanted) : at(args) { need(given == wanted); }
    const Tensor &tensor(int i) const {
        need(THPVariable_Check(at[i]));
        return THPVariable_Unpack(at[i]);
    }
    Optional maybe(int i) const { return at[i] == Py_None ? Optional() : Optional(tensor(i)); }
    int64_t integer(int i) const {
        need(PyLong_Check(at[i]));
        return PyLong_AsLongLong(at[i]);
    }
    double number(int i) const {
        const double v = PyFloat_AsDouble(at[i]);
        if (v == -1.0 && PyErr_Occurred()) PyErr_Clear(), need(false);
        return v;
    }
    std::optional<double> maybe_number(int i) const {
        return at[i] == Py_None ? std::optional<double>() : std::optional<double>(number(i));
    }
    bool truth(int i) const { return at[i] == Py_True; }
};

PyObject *wrap(const Tensor &t) { return THPVariable_Wrap(t); }
PyObject *wrap(const variable_list &ts) {
    PyObject *out = PyTuple_New((Py_ssize_t)ts.size());
    for (size_t i = 0; out && i < ts.size(); ++i) PyTuple_SET_ITEM(out, (Py_ssize_t)i, THPVariable_Wrap(ts[i]));
    return out;
}
struct WithoutLock {  // the interpreter's, while memory is found and kernels are launched
    PyThreadState *state = PyEval_SaveThread();
    ~WithoutLock() { PyEval_RestoreThread(state); }
};
template <typename F> auto unlocked(F &&f) {
    const WithoutLock hold;
    return f();
}

// Raises the package's own error.
PyObject *raise(const Failed &e) {
    PyObject *lib = PyImport_ImportModule("depthwise_convolution_gb300._lib");
    PyObject *none = lib ? PyObject_CallMethod(lib, "check", "is", (int)e.status, e.where) : nullptr;
    Py_XDECREF(none);
    Py_XDECREF(lib);
    return nullptr;
}

#define DWCONV_METHOD(name, count, call)                                              \
    PyObject *py_##name(PyObject *, PyObject *const *args, Py_ssize_t given) {        \
        HANDLE_TH_ERRORS                                                              \
        try {                                                                         \
            const Args p(args, given, count);                                         \
            return call;                                                              \
        } catch (const Refused &) {                                                   \
            Py_RETURN_NOTIMPLEMENTED;                                                 \
        } catch (const Failed &e) {                                                   \
            return raise(e);                                                          \
        }                                                                             \
        END_HANDLE_TH_ERRORS                                                          \
    }

PyObject *call_causal_conv(const Args &p) {
    const Tensor &x = p.tensor(0), &w = p.tensor(1);
    const Optional bias = p.maybe(2), state = p.maybe(3), n = p.maybe(4);
    const int64_t act = p.integer(5);
    return wrap(unlocked([&] { return causal_conv(x, w, bias, state, n, act); }));
}
PyObject *call_causal_fwd(const Args &p) {
    const Tensor &x = p.tensor(0), &w = p.tensor(1);
    const Optional bias = p.maybe(2), state = p.maybe(3), n = p.maybe(4);
    const int64_t act = p.integer(5);
    const bool with_state = p.truth(6);
    return wrap(unlocked([&] { return causal_fwd(x, w, bias, state, n, act, with_state); }));
}
PyObject *call_causal_step(const Args &p) {
    const Tensor &x = p.tensor(0), &w = p.tensor(1), &state = p.tensor(2);
    const Optional bias = p.maybe(3), slots = p.maybe(4);
    const int64_t act = p.integer(5);
    return wrap(unlocked([&] { return causal_step(x, w, state, bias, slots, act); }));
}
template <typename F> PyObject *call_norm(const Args &p, F &&f) {
    const Tensor &y = p.tensor(0);
    const Optional residual = p.maybe(1), gate = p.maybe(2), w_post = p.maybe(3), scale = p.maybe(4),
                   w_pre = p.maybe(5);
    const int64_t kind = p.integer(6), act = p.integer(7);
    const double eps = p.number(8);
    return wrap(unlocked([&] { return f(y, residual, gate, w_post, scale, w_pre, kind, act, eps); }));
}
PyObject *call_gated_delta_rule(const Args &p) {
    const Tensor &q = p.tensor(0), &k = p.tensor(1), &v = p.tensor(2), &g = p.tensor(3), &beta = p.tensor(4);
    const Optional state = p.maybe(5), n = p.maybe(6);
    const std::optional<double> scale = p.maybe_number(7);
    const bool qk_norm = p.truth(8), with_state = p.truth(9);
    return wrap(unlocked([&] { return gated_delta_rule(q, k, v, g, beta, state, n, scale, qk_norm, with_state); }));
}
PyObject *call_delta_step(const Args &p) {
    const Tensor &q = p.tensor(0), &k = p.tensor(1), &v = p.tensor(2), &g = p.tensor(3), &beta = p.tensor(4),
                 &state = p.tensor(5);
    const Optional slots = p.maybe(6);
    const std::optional<double> scale = p.maybe_number(7);
    const bool qk_norm = p.truth(8);
    return wrap(unlocked([&] { return delta_step(q, k, v, g, beta, state, slots, scale, qk_norm); }));
}

DWCONV_METHOD(causal_conv, 6, call_causal_conv(p))
DWCONV_METHOD(causal_fwd, 7, call_causal_fwd(p))
DWCONV_METHOD(causal_step, 6, call_causal_step(p))
DWCONV_METHOD(block_norm, 9, call_norm(p, block_norm))
DWCONV_METHOD(block_norm_fwd, 9, call_norm(p, block_norm_fwd))
DWCONV_METHOD(gated_delta_rule, 10, call_gated_delta_rule(p))
DWCONV_METHOD(delta_step, 9, call_delta_step(p))

#define DWCONV_ENTRY(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {DWCONV_ENTRY(causal_conv),      DWCONV_ENTRY(causal_fwd), DWCONV_ENTRY(causal_step),
                         DWCONV_ENTRY(block_norm),       DWCONV_ENTRY(block_norm_fwd),
                         DWCONV_ENTRY(gated_delta_rule), DWCONV_ENTRY(delta_step), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "libdwconv_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_libdwconv_torch() { return PyModule_Create(&module); }
