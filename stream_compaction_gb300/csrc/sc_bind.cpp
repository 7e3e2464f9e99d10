// Python entry points of the sequence operators over torch tensors: checks of
// shapes, types and layouts, allocation of what a call returns, and the call of
// the C ABI (include/sc_seq.h) on the current torch stream.  Compiled code
// because single-token calls take a few microseconds on the GPU, less than the
// same checks take in the interpreter (about 30 against 3 us on a Grace host).
// Names, arguments and meanings: seq.py, whose functions these are.
#include <ATen/Functions.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

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

Tensor make(at::IntArrayRef shape, const Tensor& like_this) { return at::empty(shape, like_this.options()); }
Tensor make_f32(at::IntArrayRef shape, const Tensor& like_this) {
    return at::empty(shape, like_this.options().dtype(at::kFloat));
}
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
}
