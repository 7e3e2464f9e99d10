// Python entry points of the sequence operators over torch tensors: checks of
// shapes, types and layouts, allocation of what a call returns, and the call of
// the C ABI (include/sc_seq.h) on the current torch stream.  Compiled code
// because single-token calls take a few microseconds on the GPU, less than the
// same checks take in the interpreter (about 30 against 3 us on a Grace host).
// Names, arguments and meanings: seq.py, whose functions these are.
#include <ATen/Context.h>
#include <ATen/Functions.h>
#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <optional>
#include <string>
#include <vector>

#include "../../include/sc_seq.h"

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;
using Shape = std::vector<int64_t>;

namespace {

void need(bool ok, const char* message) {
    if (!ok) throw py::value_error(message);
}
void need(bool ok, const char* what, const char* message) {
    if (!ok) throw py::value_error(std::string(what) + message);
}

void check(sc_status status, const char* where) {
    if (status == SC_OK) return;
    const py::object error = py::module_::import("stream_compaction_gb300").attr("ScanError");
    const py::object value = error((int)status, where);
    PyErr_SetObject(error.ptr(), value.ptr());
    throw py::error_already_set();
}

sc_stream_t stream() { return reinterpret_cast<sc_stream_t>(c10::cuda::getCurrentCUDAStream().stream()); }

int code(const Tensor& t, const char* what) {
    switch (t.scalar_type()) {
    case at::kFloat: return SC_F32;
    case at::kHalf: return SC_F16;
    case at::kBFloat16: return SC_BF16;
    default: need(false, what, " must be float32, float16 or bfloat16");
    }
    return -1;
}

void on_device(const Tensor& t, const char* what) {
    need(t.is_cuda(), what, ": expected a CUDA tensor");
    need(t.device().index() == c10::cuda::current_device(), what, " must be on the current CUDA device");
}

std::string text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

// No operator carries tangents (forward-mode derivatives) on; a result without them would
// say that they are zero.
void no_tangent(const Tensor& t, const char* what) {
    if (!c10::AutogradState::get_tls_state().get_fw_grad_mode() || !t._fw_grad(0).defined()) return;
    PyErr_Format(PyExc_NotImplementedError, "%s has a tangent: forward-mode derivatives are not recorded", what);
    throw py::error_already_set();
}

// Shape, type and device as given, the last dimension contiguous.
const Tensor& like(const Tensor& t, const char* what, at::IntArrayRef shape, at::ScalarType type,
                   const at::Device& device) {
    if (t.sizes() != shape)
        throw py::value_error(std::string(what) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
    if (t.scalar_type() != type)
        throw py::value_error(std::string(what) + " must be " + c10::toString(type) + ", got " +
                              c10::toString(t.scalar_type()));
    need(t.device() == device, what, ": expected a tensor on the device of the others");
    need(t.dim() == 0 || t.size(-1) <= 1 || t.stride(-1) == 1, what,
         ": elements of the last dimension must be contiguous");
    no_tangent(t, what);
    return t;
}
void* whole(const Tensor& t, const char* what, at::IntArrayRef shape, at::ScalarType type, const at::Device& device) {
    like(t, what, shape, type, device);
    need(t.is_contiguous(), what, " must be contiguous");
    return t.data_ptr();
}
void* whole(const Maybe& t, const char* what, at::IntArrayRef shape, at::ScalarType type, const at::Device& device) {
    return t ? whole(*t, what, shape, type, device) : nullptr;
}

const uint8_t* heads_of(const Maybe& heads, const Tensor& x) {
    if (!heads) return nullptr;
    const auto type = heads->scalar_type();
    need(type == at::kByte || type == at::kBool || type == at::kChar,
         "heads must be a uint8/bool tensor with one flag per token");
    return static_cast<const uint8_t*>(whole(*heads, "heads", x.sizes().slice(0, 2), type, x.device()));
}
const int32_t* slots_of(const Maybe& slots, const Tensor& x) {
    return static_cast<const int32_t*>(whole(slots, "slots", {x.size(0)}, at::kInt, x.device()));
}

// A tensor of the caller's that the call writes to: autograd learns of it, as of any
// operation in place, and refuses a gradient that would read the old values.
void written(const Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(const Maybe& t) {
    if (t) written(*t);
}

// Whether torch records a gradient by one of the tensors: the call is then made through
// an autograd function, and the direct one returns None to say so (cheaper than to ask
// first, from the interpreter).
bool records(std::initializer_list<const Maybe*> some, std::initializer_list<const Tensor*> given) {
    if (!at::GradMode::is_enabled()) return false;
    for (const Maybe* t : some)
        if (*t && (*t)->requires_grad()) return true;
    for (const Tensor* t : given)
        if (t->requires_grad()) return true;
    return false;
}

// Whether a dispatch mode watches what torch allocates, or the deterministic algorithms fill it.
bool watched() {
    const auto& context = at::globalContext();
    return c10::impl::dispatch_mode_enabled() ||
           (context.deterministicAlgorithms() && context.deterministicFillUninitializedMemory());
}
// New tensors, without torch's dispatcher where nobody watches: 0.8 us less each of a
// call's 4 to 9.
Tensor make_as(at::IntArrayRef shape, at::ScalarType type, const Tensor& like_this) {
    if (like_this.is_cuda() && !watched()) return at::detail::empty_cuda(shape, type, like_this.device(), std::nullopt);
    return at::empty(shape, like_this.options().dtype(type));
}
Tensor make(at::IntArrayRef shape, const Tensor& like_this) { return make_as(shape, like_this.scalar_type(), like_this); }
Tensor make_f32(at::IntArrayRef shape, const Tensor& like_this) { return make_as(shape, at::kFloat, like_this); }
// `out` if given (checked), else a new tensor like x.
Tensor out_like(const Maybe& out, const Tensor& x) {
    if (!out) return make(x.sizes(), x);
    return like(*out, "out", x.sizes(), x.scalar_type(), x.device());
}

// ------------------------------------------------------------- embedding
int ids64(const Tensor& ids) {
    on_device(ids, "ids");
    need(ids.scalar_type() == at::kInt || ids.scalar_type() == at::kLong, "ids must be int32 or int64");
    need(ids.is_contiguous(), "ids must be contiguous");
    return ids.scalar_type() == at::kLong;
}

Tensor embed(const Tensor& ids, const Tensor& weight, double scale, const Maybe& out) {
    const int wide = ids64(ids);
    const int type = code(weight, "weight");
    need(weight.dim() == 2, "weight must have shape (vocab, dim)");
    like(weight, "weight", weight.sizes(), weight.scalar_type(), ids.device());
    const int64_t vocab = weight.size(0), dim = weight.size(1);
    Shape shape = ids.sizes().vec();
    shape.push_back(dim);
    Tensor y = out ? *out : make(shape, weight);
    void* to = whole(y, "out", shape, weight.scalar_type(), ids.device());
    check(sc_embed(ids.data_ptr(), wide, ids.numel(), (sc_dtype)type, weight.data_ptr(), vocab, dim,
                   vocab > 1 ? weight.stride(0) : dim, (float)scale, to, dim, stream()),
          "sc_embed");
    written(out);
    return y;
}

Tensor embed_grad(const Tensor& ids, const Tensor& dout, int64_t vocab, double scale, const Maybe& out,
                  bool accumulate) {
    const int wide = ids64(ids);
    const int type = code(dout, "dout");
    need(dout.dim() >= 1 && dout.sizes().slice(0, dout.dim() - 1) == ids.sizes(),
         "dout must have the shape of ids and one dimension more");
    need(vocab >= 0, "vocab must not be negative");
    need(out.has_value() || !accumulate, "accumulate needs `out`");
    like(dout, "dout", dout.sizes(), dout.scalar_type(), ids.device());
    need(dout.is_contiguous() || dout.dim() == 2, "dout must be contiguous, or a matrix of rows");
    const int64_t dim = dout.size(-1);
    Tensor dw = out ? *out : at::empty({vocab, dim}, dout.options());
    need(dw.scalar_type() == dout.scalar_type() || dw.scalar_type() == at::kFloat,
         "out must be of dout's type or float32");
    like(dw, "out", {vocab, dim}, dw.scalar_type(), ids.device());
    const int64_t ldd = dout.is_contiguous() || dout.size(0) <= 1 ? dim : dout.stride(0);
    check(sc_embed_grad(ids.data_ptr(), wide, ids.numel(), (sc_dtype)type, dout.data_ptr(), ldd, vocab, dim,
                        (float)scale, (sc_dtype)code(dw, "out"), dw.data_ptr(), vocab > 1 ? dw.stride(0) : dim,
                        accumulate, stream()),
          "sc_embed_grad");
    written(out);
    return dw;
}

// ----------------------------------------------------------- convolution
sc_conv_desc conv_desc(const Tensor& x, const Tensor& weight, const Maybe& bias,
                       const std::optional<std::string>& activation, bool step) {
    on_device(x, "x");
    sc_conv_desc d{};
    d.dtype = code(x, "x");
    need(x.dim() == (step ? 2 : 3), step ? "x must have shape (batch, channels)"
                                         : "x must have shape (batch, length, channels)");
    like(x, "x", x.sizes(), x.scalar_type(), x.device());
    need(weight.dim() == 2 && weight.size(1) >= 1 && weight.size(1) <= SC_CONV_MAX_WIDTH,
         "weight must have shape (channels, width), width 1 to 8");
    need(!activation || *activation == "silu", "activation must be 'silu' or None");
    d.width = (int32_t)weight.size(1);
    d.silu = activation.has_value();
    d.batch = x.size(0);
    d.length = step ? 1 : x.size(1);
    d.channels = x.size(-1);
    d.x = x.data_ptr();
    d.x_batch = x.stride(0);
    d.x_token = step ? 0 : x.stride(1);
    d.weight = whole(weight, "weight", {d.channels, d.width}, x.scalar_type(), x.device());
    d.bias = whole(bias, "bias", {d.channels}, x.scalar_type(), x.device());
    return d;
}
Shape conv_rest(sc_conv_desc& d, const Tensor& x, const Maybe& heads, const Maybe& state) {
    d.heads = heads_of(heads, x);
    const Shape shape{d.batch, d.width - 1, d.channels};
    d.state = whole(state, "state", shape, x.scalar_type(), x.device());
    return shape;
}

Tensor causal_conv(const Tensor& x, const Tensor& weight, const Maybe& bias,
                   const std::optional<std::string>& activation, const Maybe& heads, const Maybe& state,
                   const Maybe& final_state, const Maybe& out) {
    sc_conv_desc d = conv_desc(x, weight, bias, activation, false);
    const Shape shape = conv_rest(d, x, heads, state);
    void* fs = whole(final_state, "final_state", shape, x.scalar_type(), x.device());
    Tensor y = out_like(out, x);
    check(sc_causal_conv(&d, y.data_ptr(), y.stride(0), y.stride(1), fs, stream()), "sc_causal_conv");
    written(final_state);
    written(out);
    return y;
}

py::dict causal_conv_grad(const Tensor& dy, const Tensor& x, const Tensor& weight, const Maybe& bias,
                          const std::optional<std::string>& activation, const Maybe& heads, const Maybe& state) {
    sc_conv_desc d = conv_desc(x, weight, bias, activation, false);
    const Shape shape = conv_rest(d, x, heads, state);
    like(dy, "dy", x.sizes(), x.scalar_type(), x.device());
    Tensor dx = make(x.sizes(), x), dw = make_f32(weight.sizes(), x), db = make_f32({d.channels}, x), ds;
    if (state) ds = make(shape, x);
    check(sc_causal_conv_grad(&d, dy.data_ptr(), dy.stride(0), dy.stride(1), dx.data_ptr(), dx.stride(0),
                              dx.stride(1), dw.data_ptr<float>(), db.data_ptr<float>(),
                              state ? ds.data_ptr() : nullptr, stream()),
          "sc_causal_conv_grad");
    py::dict g;
    g["x"] = dx;
    g["weight"] = dw;
    g["bias"] = db;
    if (state) g["state"] = ds;
    return g;
}

Tensor causal_conv_step(const Tensor& x, const Tensor& state, const Tensor& weight, const Maybe& bias,
                        const std::optional<std::string>& activation, const Maybe& slots, const Maybe& out) {
    const sc_conv_desc d = conv_desc(x, weight, bias, activation, true);
    need(state.dim() == 3, "state must have shape (rows, width - 1, channels)");
    void* pool = whole(state, "state", {state.size(0), d.width - 1, d.channels}, x.scalar_type(), x.device());
    const int32_t* sl = slots_of(slots, x);
    Tensor y = out_like(out, x);
    check(sc_causal_conv_step(&d, pool, state.size(0), sl, y.data_ptr(), y.stride(0), stream()),
          "sc_causal_conv_step");
    written(state);
    written(out);
    return y;
}

// -------------------------------------------------------- selective scan
sc_ssm_desc ssm_desc(const Tensor& x, const Tensor& dt, const Tensor& A, const Tensor& B, const Tensor& C,
                     const Maybe& D, const Maybe& z, const Maybe& dt_bias, bool softplus, bool step) {
    on_device(x, "x");
    sc_ssm_desc d{};
    const auto type = x.scalar_type();
    const at::Device device = x.device();
    d.dtype = code(x, "x");
    need(x.dim() == (step ? 2 : 3), step ? "x must have shape (batch, channels)"
                                         : "x must have shape (batch, length, channels)");
    like(x, "x", x.sizes(), type, device);
    like(dt, "dt", x.sizes(), type, device);
    need(A.dim() == 2 && A.size(1) >= 1, "A must have shape (channels, states)");
    need(B.dim() == x.dim() + 1 && B.size(-2) >= 1,
         step ? "B must have shape (batch, groups, states)" : "B must have shape (batch, length, groups, states)");
    d.softplus = softplus;
    d.batch = x.size(0);
    d.length = step ? 1 : x.size(1);
    d.channels = x.size(-1);
    d.states = A.size(1);
    d.groups = B.size(-2);
    need(d.channels % d.groups == 0, "channels must be a multiple of the groups of B and C");
    d.A = static_cast<const float*>(whole(A, "A", {d.channels, d.states}, at::kFloat, device));
    const int64_t bc4[] = {d.batch, d.length, d.groups, d.states}, bc3[] = {d.batch, d.groups, d.states};
    const at::IntArrayRef bc = step ? at::IntArrayRef(bc3) : at::IntArrayRef(bc4);
    like(B, "B", bc, type, device);
    like(C, "C", bc, type, device);
    d.x = x.data_ptr();
    d.dt = dt.data_ptr();
    d.B = B.data_ptr();
    d.C = C.data_ptr();
    d.x_batch = x.stride(0);
    d.dt_batch = dt.stride(0);
    d.B_batch = B.stride(0);
    d.C_batch = C.stride(0);
    d.B_group = B.stride(-2);
    d.C_group = C.stride(-2);
    if (!step) {
        d.x_token = x.stride(1);
        d.dt_token = dt.stride(1);
        d.B_token = B.stride(1);
        d.C_token = C.stride(1);
    }
    if (z) {
        like(*z, "z", x.sizes(), type, device);
        d.z = z->data_ptr();
        d.z_batch = z->stride(0);
        d.z_token = step ? 0 : z->stride(1);
    }
    d.D = static_cast<const float*>(whole(D, "D", {d.channels}, at::kFloat, device));
    d.dt_bias = static_cast<const float*>(whole(dt_bias, "dt_bias", {d.channels}, at::kFloat, device));
    return d;
}
const float* state_of(const Maybe& t, const char* what, const sc_ssm_desc& d, const Tensor& x) {
    return static_cast<const float*>(whole(t, what, {d.batch, d.channels, d.states}, at::kFloat, x.device()));
}

Shape saved_shape(const Tensor& x, int64_t states) {
    const int64_t padded = states <= 8 ? 8 : states <= 16 ? 16 : states <= 32 ? 32 : 64;
    return {x.size(0), (x.size(1) + SC_SSM_SAVE - 1) / SC_SSM_SAVE, padded / 4, x.size(2), 4};
}
float* saved_of(const Maybe& saved, const sc_ssm_desc& d, const Tensor& x) {
    return static_cast<float*>(whole(saved, "saved", saved_shape(x, d.states), at::kFloat, x.device()));
}

Tensor selective_scan_saved(const Tensor& x, const Tensor& A) {
    need(x.dim() == 3, "x must have shape (batch, length, channels)");
    need(A.dim() == 2 && A.size(1) >= 1, "A must have shape (channels, states)");
    return make_f32(saved_shape(x, A.size(1)), x);
}

Tensor selective_scan(const Tensor& x, const Tensor& dt, const Tensor& A, const Tensor& B, const Tensor& C,
                      const Maybe& D, const Maybe& z, const Maybe& dt_bias, bool softplus, const Maybe& heads,
                      const Maybe& state, const Maybe& final_state, const Maybe& saved, const Maybe& out) {
    sc_ssm_desc d = ssm_desc(x, dt, A, B, C, D, z, dt_bias, softplus, false);
    d.heads = heads_of(heads, x);
    d.state = state_of(state, "state", d, x);
    float* fs = const_cast<float*>(state_of(final_state, "final_state", d, x));
    float* sv = saved_of(saved, d, x);
    Tensor y = out_like(out, x);
    check(sc_selective_scan(&d, y.data_ptr(), y.stride(0), y.stride(1), fs, sv, stream()), "sc_selective_scan");
    written(final_state);
    written(saved);
    written(out);
    return y;
}

py::dict selective_scan_grad(const Tensor& dy, const Tensor& x, const Tensor& dt, const Tensor& A, const Tensor& B,
                             const Tensor& C, const Maybe& D, const Maybe& z, const Maybe& dt_bias, bool softplus,
                             const Maybe& heads, const Maybe& state, const Maybe& saved, const Maybe& dfinal_state) {
    sc_ssm_desc d = ssm_desc(x, dt, A, B, C, D, z, dt_bias, softplus, false);
    d.heads = heads_of(heads, x);
    d.state = state_of(state, "state", d, x);
    like(dy, "dy", x.sizes(), x.scalar_type(), x.device());
    need(saved.has_value(), "saved: the buffer that selective_scan filled is needed");
    sc_ssm_grads g{};
    g.dy = dy.data_ptr();
    g.dy_batch = dy.stride(0);
    g.dy_token = dy.stride(1);
    g.saved = saved_of(saved, d, x);
    g.dfinal = state_of(dfinal_state, "dfinal_state", d, x);
    py::dict r;
    auto add = [&](const char* name, Tensor t) {
        r[name] = t;
        return t.data_ptr();
    };
    g.dx = add("x", make(x.sizes(), x));
    g.ddt = add("dt", make(x.sizes(), x));
    g.dA = static_cast<float*>(add("A", make_f32(A.sizes(), x)));
    g.dB = add("B", make(B.sizes(), x));
    g.dC = add("C", make(C.sizes(), x));
    if (D) g.dD = static_cast<float*>(add("D", make_f32({d.channels}, x)));
    if (z) g.dz = add("z", make(x.sizes(), x));
    if (dt_bias) g.ddt_bias = static_cast<float*>(add("dt_bias", make_f32({d.channels}, x)));
    if (state) g.dstate = static_cast<float*>(add("state", make_f32(state->sizes(), x)));
    check(sc_selective_scan_grad(&d, &g, stream()), "sc_selective_scan_grad");
    return r;
}

Tensor selective_scan_step(const Tensor& x, const Tensor& dt, const Tensor& A, const Tensor& B, const Tensor& C,
                           const Tensor& state, const Maybe& D, const Maybe& z, const Maybe& dt_bias, bool softplus,
                           const Maybe& slots, const Maybe& out) {
    const sc_ssm_desc d = ssm_desc(x, dt, A, B, C, D, z, dt_bias, softplus, true);
    need(state.dim() == 3, "state must have shape (rows, channels, states)");
    void* pool = whole(state, "state", {state.size(0), d.channels, d.states}, at::kFloat, x.device());
    const int32_t* sl = slots_of(slots, x);
    Tensor y = out_like(out, x);
    check(sc_selective_scan_step(&d, static_cast<float*>(pool), state.size(0), sl, y.data_ptr(), y.stride(0),
                                 stream()),
          "sc_selective_scan_step");
    written(state);
    written(out);
    return y;
}

// ------------------------------------------------------------ gated scan
sc_gated_desc gated_desc(const Tensor& x, const Tensor& gate, const std::optional<std::string>& activation, bool step) {
    on_device(x, "x");
    sc_gated_desc d{};
    d.dtype = code(x, "x");
    need(x.dim() == (step ? 2 : 3), step ? "x must have shape (batch, channels)"
                                         : "x must have shape (batch, length, channels)");
    like(x, "x", x.sizes(), x.scalar_type(), x.device());
    like(gate, "gate", x.sizes(), x.scalar_type(), x.device());
    need(!activation || *activation == "sigmoid", "activation must be 'sigmoid' or None");
    d.sigmoid = activation.has_value();
    d.batch = x.size(0);
    d.length = step ? 1 : x.size(1);
    d.channels = x.size(-1);
    d.x = x.data_ptr();
    d.gate = gate.data_ptr();
    d.x_batch = x.stride(0);
    d.gate_batch = gate.stride(0);
    if (!step) {
        d.x_token = x.stride(1);
        d.gate_token = gate.stride(1);
    }
    return d;
}
const float* gated_state(const Maybe& t, const char* what, const Tensor& x) {
    return static_cast<const float*>(whole(t, what, {x.size(0), x.size(-1)}, at::kFloat, x.device()));
}
Shape gated_saved_shape(const Tensor& x) {
    return {x.size(0), (x.size(1) + SC_GATED_SAVE - 1) / SC_GATED_SAVE, x.size(2)};
}
Tensor gated_scan_saved(const Tensor& x) {
    on_device(x, "x");
    need(x.dim() == 3, "x must have shape (batch, length, channels)");
    return make_f32(gated_saved_shape(x), x);
}

py::object gated_scan(const Tensor& x, const Tensor& gate, const std::optional<std::string>& activation,
                      const Maybe& heads, const Maybe& state, const Maybe& final_state, const Maybe& saved,
                      const Maybe& out) {
    if (records({&state}, {&x, &gate})) return py::none();
    sc_gated_desc d = gated_desc(x, gate, activation, false);
    d.heads = heads_of(heads, x);
    d.state = gated_state(state, "state", x);
    float* fs = const_cast<float*>(gated_state(final_state, "final_state", x));
    float* sv = static_cast<float*>(whole(saved, "saved", gated_saved_shape(x), at::kFloat, x.device()));
    Tensor y = out_like(out, x);
    check(sc_gated_scan(&d, y.data_ptr(), y.stride(0), y.stride(1), fs, sv, stream()), "sc_gated_scan");
    written(final_state);
    written(saved);
    written(out);
    return py::cast(y);
}

py::dict gated_scan_grad(const Tensor& dy, const Tensor& x, const Tensor& gate,
                         const std::optional<std::string>& activation, const Maybe& heads, const Maybe& state,
                         const Maybe& saved, const Maybe& dfinal_state) {
    sc_gated_desc d = gated_desc(x, gate, activation, false);
    d.heads = heads_of(heads, x);
    d.state = gated_state(state, "state", x);
    like(dy, "dy", x.sizes(), x.scalar_type(), x.device());
    need(saved.has_value(), "saved: the buffer that gated_scan filled is needed");
    const float* sv = static_cast<const float*>(whole(saved, "saved", gated_saved_shape(x), at::kFloat, x.device()));
    const float* df = gated_state(dfinal_state, "dfinal_state", x);
    Tensor dx = make(x.sizes(), x), dg = make(x.sizes(), x), ds;
    if (state) ds = make_f32(state->sizes(), x);
    check(sc_gated_scan_grad(&d, dy.data_ptr(), dy.stride(0), dy.stride(1), sv, df, dx.data_ptr(), dg.data_ptr(),
                             state ? ds.data_ptr<float>() : nullptr, stream()),
          "sc_gated_scan_grad");
    py::dict g;
    g["x"] = dx;
    g["gate"] = dg;
    if (state) g["state"] = ds;
    return g;
}

py::object gated_scan_step(const Tensor& x, const Tensor& gate, const Tensor& state,
                           const std::optional<std::string>& activation, const Maybe& slots, const Maybe& out) {
    if (records({}, {&x, &gate, &state})) return py::none();
    const sc_gated_desc d = gated_desc(x, gate, activation, true);
    need(state.dim() == 2, "state must have shape (rows, channels)");
    void* pool = whole(state, "state", {state.size(0), d.channels}, at::kFloat, x.device());
    const int32_t* sl = slots_of(slots, x);
    Tensor y = out_like(out, x);
    check(sc_gated_scan_step(&d, static_cast<float*>(pool), state.size(0), sl, y.data_ptr(), y.stride(0), stream()),
          "sc_gated_scan_step");
    written(state);
    written(out);
    return py::cast(y);
}

// ------------------------------------------------------------------ norm
// A tensor of any number of dimensions as batch x length rows: the dimensions before
// `cut` are the batch, those from there to the last but one the length, each run of
// them with one stride.
struct Rows {
    int64_t batch = 1, length = 1, sb = 0, st = 0;
};
Rows rows_of(const Tensor& t, const char* what, int64_t cut) {
    Rows r;
    auto run = [&](int64_t from, int64_t to, int64_t& n, int64_t& stride) {
        for (int64_t i = to - 1; i >= from; --i) {
            if (t.size(i) == 1) continue;
            if (n == 1) stride = t.stride(i);
            else need(t.stride(i) == n * stride, what, ": its leading dimensions have more than two strides");
            n *= t.size(i);
        }
    };
    run(0, cut, r.batch, r.sb);
    run(cut, t.dim() - 1, r.length, r.st);
    if (t.numel() == 0) r = Rows{0, 0, 0, 0};
    return r;
}
// The first dimension from which on a tensor's rows have one stride.
int64_t cut_of(const Tensor& t) {
    int64_t n = 1, stride = 0, i = t.dim() - 2;
    for (; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (n == 1) stride = t.stride(i);
        else if (t.stride(i) != n * stride) break;
        n *= t.size(i);
    }
    return i + 1;
}

sc_norm_desc norm_desc(const Tensor& x, const Maybe& weight, const Maybe& bias, bool rms) {
    on_device(x, "x");
    sc_norm_desc d{};
    d.dtype = d.wtype = code(x, "x");
    need(x.dim() >= 1, "x must have shape (..., channels)");
    like(x, "x", x.sizes(), x.scalar_type(), x.device());
    d.rms = rms;
    d.channels = x.size(-1);
    d.x = x.data_ptr();
    const Maybe& one = weight ? weight : bias;
    if (one) {
        const auto type = one->scalar_type();
        need(type == x.scalar_type() || type == at::kFloat, "weight and bias must be of x's type or float32");
        d.wtype = code(*one, "weight");
        d.weight = whole(weight, "weight", {d.channels}, type, x.device());
        d.bias = whole(bias, "bias", {d.channels}, type, x.device());
    }
    return d;
}
Shape norm_saved_shape(const Tensor& x) {
    Shape s = x.sizes().vec();
    s.back() = 2;
    return s;
}
Tensor layer_norm_saved(const Tensor& x) {
    on_device(x, "x");
    need(x.dim() >= 1, "x must have shape (..., channels)");
    return make_f32(norm_saved_shape(x), x);
}

py::object layer_norm(const Tensor& x, const Maybe& weight, const Maybe& bias, double eps, bool rms,
                      const Maybe& residual, const Maybe& saved, const Maybe& out) {
    if (records({&weight, &bias, &residual}, {&x})) return py::none();
    sc_norm_desc d = norm_desc(x, weight, bias, rms);
    need(eps >= 0, "eps must not be negative");
    d.eps = (float)eps;
    float* sv = static_cast<float*>(whole(saved, "saved", norm_saved_shape(x), at::kFloat, x.device()));
    Tensor y = out_like(out, x), sum;
    int64_t cut = std::max(cut_of(x), cut_of(y));
    if (residual) {
        like(*residual, "residual", x.sizes(), x.scalar_type(), x.device());
        sum = make(x.sizes(), x);
        cut = std::max(cut, cut_of(*residual));
    }
    const Rows rx = rows_of(x, "x", cut), ry = rows_of(y, "out", cut);
    d.batch = rx.batch;
    d.length = rx.length;
    d.x_batch = rx.sb;
    d.x_token = rx.st;
    Rows rs;
    if (residual) {
        const Rows rr = rows_of(*residual, "residual", cut);
        d.residual = residual->data_ptr();
        d.residual_batch = rr.sb;
        d.residual_token = rr.st;
        rs = rows_of(sum, "sum", cut);
    }
    check(sc_layer_norm(&d, y.data_ptr(), ry.sb, ry.st, residual ? sum.data_ptr() : nullptr, rs.sb, rs.st, sv, stream()),
          "sc_layer_norm");
    written(saved);
    written(out);
    if (!residual) return py::cast(y);
    return py::make_tuple(y, sum);
}

py::dict layer_norm_grad(const Tensor& dy, const Tensor& x, const Maybe& weight, const Maybe& bias, bool rms,
                         const Maybe& saved, const Maybe& dsum, bool by_weight, bool by_bias) {
    sc_norm_desc d = norm_desc(x, weight, bias, rms);
    like(dy, "dy", x.sizes(), x.scalar_type(), x.device());
    need(saved.has_value(), "saved: the buffer that layer_norm filled is needed");
    const float* sv = static_cast<const float*>(whole(saved, "saved", norm_saved_shape(x), at::kFloat, x.device()));
    int64_t cut = std::max(cut_of(x), cut_of(dy));
    if (dsum) {
        like(*dsum, "dsum", x.sizes(), x.scalar_type(), x.device());
        cut = std::max(cut, cut_of(*dsum));
    }
    const Rows rx = rows_of(x, "x", cut), re = rows_of(dy, "dy", cut);
    d.batch = rx.batch;
    d.length = rx.length;
    d.x_batch = rx.sb;
    d.x_token = rx.st;
    const Rows rs = dsum ? rows_of(*dsum, "dsum", cut) : Rows{};
    Tensor dx = make(x.sizes(), x), dw, db;
    by_weight = by_weight && weight.has_value();
    by_bias = by_bias && bias.has_value();
    if (by_weight) dw = make_f32({d.channels}, x);
    if (by_bias) db = make_f32({d.channels}, x);
    check(sc_layer_norm_grad(&d, dy.data_ptr(), re.sb, re.st, dsum ? dsum->data_ptr() : nullptr, rs.sb, rs.st, sv,
                             dx.data_ptr(), by_weight ? dw.data_ptr<float>() : nullptr,
                             by_bias ? db.data_ptr<float>() : nullptr, stream()),
          "sc_layer_norm_grad");
    py::dict g;
    g["x"] = dx;
    if (by_weight) g["weight"] = dw;
    if (by_bias) g["bias"] = db;
    return g;
}

// --------------------------------------------------------------- experts
py::tuple expert_sort(const Tensor& experts, int64_t n_experts) {
    on_device(experts, "experts");
    need(experts.scalar_type() == at::kInt || experts.scalar_type() == at::kLong, "experts must be int32 or int64");
    need(experts.dim() == 2, "experts must have shape (tokens, choices)");
    need(experts.is_contiguous(), "experts must be contiguous");
    need(n_experts >= 1 && n_experts <= SC_EXPERT_MAX, "the number of experts must be 1 to 1024");
    Tensor offsets = make_as({n_experts + 1}, at::kLong, experts);
    Tensor order = make_as({experts.numel()}, at::kInt, experts), place = make_as(experts.sizes(), at::kInt, experts);
    check(sc_expert_sort(experts.data_ptr(), experts.scalar_type() == at::kLong, experts.numel(), n_experts,
                         order.data_ptr<int32_t>(), place.data_ptr<int32_t>(), offsets.data_ptr<int64_t>(), stream()),
          "sc_expert_sort");
    return py::make_tuple(offsets, order, place);
}

// The entries' side of a call, from what expert_sort returned, for rows like `rows`.
sc_expert_desc expert_desc(const Tensor& offsets, const Tensor& place, const Tensor& rows, const char* what) {
    on_device(rows, what);
    sc_expert_desc d{};
    d.dtype = d.wtype = code(rows, what);
    need(rows.dim() == 2, what, " must have two dimensions");
    like(rows, what, rows.sizes(), rows.scalar_type(), rows.device());
    need(place.dim() == 2 && offsets.dim() == 1 && offsets.size(0) >= 2, "the order must be what expert_sort returned");
    d.tokens = place.size(0);
    d.choices = place.size(1);
    d.dim = rows.size(1);
    d.experts = offsets.size(0) - 1;
    d.place = static_cast<const int32_t*>(whole(place, "order.place", place.sizes(), at::kInt, rows.device()));
    d.offsets = static_cast<const int64_t*>(whole(offsets, "order.offsets", offsets.sizes(), at::kLong, rows.device()));
    return d;
}
void expert_weights(sc_expert_desc& d, const Maybe& weights, const Tensor& rows) {
    if (!weights) return;
    need(weights->scalar_type() == rows.scalar_type() || weights->scalar_type() == at::kFloat,
         "weights must be of the rows' type or float32");
    d.wtype = code(*weights, "weights");
    d.weights = whole(weights, "weights", {d.tokens, d.choices}, weights->scalar_type(), rows.device());
}
int64_t ld(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }
Tensor rows_out(const Maybe& out, int64_t rows, const Tensor& like_this) {
    const int64_t shape[] = {rows, like_this.size(1)};
    if (!out) return make(shape, like_this);
    return like(*out, "out", shape, like_this.scalar_type(), like_this.device());
}

py::object expert_gather(const Tensor& x, const Tensor& offsets, const Tensor& place, const Maybe& out) {
    if (records({}, {&x})) return py::none();
    const sc_expert_desc d = expert_desc(offsets, place, x, "x");
    need(x.size(0) == d.tokens, "x must have a row for each token");
    Tensor rows = rows_out(out, d.tokens * d.choices, x);
    check(sc_expert_gather(&d, x.data_ptr(), ld(x), rows.data_ptr(), ld(rows), stream()), "sc_expert_gather");
    written(out);
    return py::cast(rows);
}
Tensor expert_gather_grad(const Tensor& drows, const Tensor& offsets, const Tensor& place, const Maybe& out) {
    const sc_expert_desc d = expert_desc(offsets, place, drows, "drows");
    need(drows.size(0) == d.tokens * d.choices, "drows must have a row for each entry");
    Tensor dx = rows_out(out, d.tokens, drows);
    check(sc_expert_gather_grad(&d, drows.data_ptr(), ld(drows), dx.data_ptr(), ld(dx), stream()), "sc_expert_gather_grad");
    written(out);
    return dx;
}
py::object expert_combine(const Tensor& rows, const Tensor& offsets, const Tensor& place, const Maybe& weights,
                          const Maybe& out) {
    if (records({&weights}, {&rows})) return py::none();
    sc_expert_desc d = expert_desc(offsets, place, rows, "rows");
    need(rows.size(0) == d.tokens * d.choices, "rows must have a row for each entry");
    expert_weights(d, weights, rows);
    Tensor y = rows_out(out, d.tokens, rows);
    check(sc_expert_combine(&d, rows.data_ptr(), ld(rows), y.data_ptr(), ld(y), stream()), "sc_expert_combine");
    written(out);
    return py::cast(y);
}
py::dict expert_combine_grad(const Tensor& dout, const Tensor& rows, const Tensor& offsets, const Tensor& place,
                             const Maybe& weights) {
    sc_expert_desc d = expert_desc(offsets, place, rows, "rows");
    need(rows.size(0) == d.tokens * d.choices, "rows must have a row for each entry");
    like(dout, "dout", {d.tokens, d.dim}, rows.scalar_type(), rows.device());
    expert_weights(d, weights, rows);
    Tensor dr = make(rows.sizes(), rows), dw;
    if (weights) dw = make(weights->sizes(), *weights);
    check(sc_expert_combine_grad(&d, dout.data_ptr(), ld(dout), rows.data_ptr(), ld(rows), dr.data_ptr(), ld(dr),
                                 weights ? dw.data_ptr() : nullptr, stream()),
          "sc_expert_combine_grad");
    py::dict g;
    g["y"] = dr;
    if (weights) g["weights"] = dw;
    return g;
}

}  // namespace

PYBIND11_MODULE(_seqbind, m) {
    m.def("embed", &embed);
    m.def("embed_grad", &embed_grad);
    m.def("causal_conv", &causal_conv);
    m.def("causal_conv_grad", &causal_conv_grad);
    m.def("causal_conv_step", &causal_conv_step);
    m.def("selective_scan_saved", &selective_scan_saved);
    m.def("selective_scan", &selective_scan);
    m.def("selective_scan_grad", &selective_scan_grad);
    m.def("selective_scan_step", &selective_scan_step);
    m.def("gated_scan", &gated_scan);
    m.def("gated_scan_saved", &gated_scan_saved);
    m.def("gated_scan_grad", &gated_scan_grad);
    m.def("gated_scan_step", &gated_scan_step);
    m.def("layer_norm", &layer_norm);
    m.def("layer_norm_saved", &layer_norm_saved);
    m.def("layer_norm_grad", &layer_norm_grad);
    m.def("expert_sort", &expert_sort);
    m.def("expert_gather", &expert_gather);
    m.def("expert_gather_grad", &expert_gather_grad);
    m.def("expert_combine", &expert_combine);
    m.def("expert_combine_grad", &expert_combine_grad);
}
