// C ABI of the sequence operators (include/sc_seq.h): argument checks, plans and
// scratch, dispatch.  Nothing here throws.
#include <algorithm>
#include <cstring>

#include "sc_seq_launch.h"

namespace {

using namespace scg;

constexpr int64_t kMaxGrid = 2147483647;

int bytes_of(int dtype) { return dtype == SC_F32 ? 4 : dtype == SC_F16 || dtype == SC_BF16 ? 2 : 0; }
bool multiple(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
cudaStream_t cu(sc_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// a * b * c * d, or -1 beyond 2^60 (all at least 0).
int64_t product(int64_t a, int64_t b, int64_t c = 1, int64_t d = 1) {
    const __int128 lim = (__int128)1 << 60;
    __int128 v = (__int128)a * b;
    if (v > lim) return -1;
    v *= c;
    if (v > lim) return -1;
    v *= d;
    return v > lim ? -1 : (int64_t)v;
}

// A batch x tokens x channels tensor with free strides.
struct Tensor {
    const void* p = nullptr;
    int64_t batch = 0, tokens = 0, channels = 0, sb = 0, st = 0;
    int eb = 1;
    int64_t span() const {  // elements from the first to behind the last
        if (!batch || !tokens || !channels) return 0;
        const __int128 n = (__int128)(batch - 1) * sb + (__int128)(tokens - 1) * st + channels;
        return n > ((__int128)1 << 60) ? -1 : (int64_t)n;
    }
    bool ok() const { return p && multiple(p, eb) && sb >= 0 && st >= 0 && span() >= 0; }
    // every element has its own address
    bool distinct() const {
        const bool many_b = batch > 1, many_t = tokens > 1;
        if (many_t && st < channels) return false;
        if (many_b && sb < channels) return false;
        if (!many_b || !many_t) return true;
        return sb >= (__int128)(tokens - 1) * st + channels || st >= (__int128)(batch - 1) * sb + channels;
    }
    bool vec(int elems) const {
        return multiple(p, std::min(16, elems * eb)) && (batch <= 1 || sb % elems == 0) && (tokens <= 1 || st % elems == 0);
    }
};
Tensor flat(const void* p, int64_t n, int eb) { return {p, 1, 1, n, 0, 0, eb}; }

// Whether two tensors share memory; column slices of one joint buffer do not.
bool share(const Tensor& a, const Tensor& b) {
    const int64_t na = a.span(), nb = b.span();
    if (!a.p || !b.p || na <= 0 || nb <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    if (!(x < y + (uintptr_t)nb * b.eb && y < x + (uintptr_t)na * a.eb)) return false;
    const int64_t stride = a.tokens > 1 ? a.st : a.sb;
    if (a.eb == b.eb && stride > 0 && a.tokens == b.tokens && a.batch == b.batch && (a.tokens <= 1 || a.st == b.st) &&
        (a.batch <= 1 || (a.sb == b.sb && a.sb % stride == 0)) && (x - y) % a.eb == 0) {
        const int64_t diff = ((int64_t)(x - y)) / a.eb;            // a's first element behind b's
        const int64_t col = ((diff % stride) + stride) % stride;   // its column in b's rows
        if (col >= b.channels && col + a.channels <= stride) return false;
    }
    return true;
}

// Whether every output has its memory to itself: none shares it with an input or
// with another output.  The ranges of addresses decide nearly always.
template <int kOut, int kIn>
bool apart(const Tensor (&out)[kOut], const Tensor (&in)[kIn]) {
    const Tensor* all[kOut + kIn];
    uintptr_t lo[kOut + kIn], hi[kOut + kIn];
    int n = 0, outs = 0;
    auto add = [&](const Tensor& t) {
        const int64_t span = t.p ? t.span() : 0;
        if (span <= 0) return;
        all[n] = &t;
        lo[n] = reinterpret_cast<uintptr_t>(t.p);
        hi[n] = lo[n] + (uintptr_t)span * t.eb;
        ++n;
    };
    for (const Tensor& t : out) add(t);
    outs = n;
    for (const Tensor& t : in) add(t);
    for (int i = 0; i < outs; ++i)
        for (int j = i + 1; j < n; ++j)
            if (lo[i] < hi[j] && lo[j] < hi[i] && share(*all[i], *all[j])) return false;
    return true;
}

bool vec_row(int64_t dim, int64_t ld, const void* p, int elems, int64_t rows) {
    return multiple(p, 16) && dim % elems == 0 && (rows <= 1 || ld % elems == 0);
}

// ----------------------------------------------------------- embedding
sc_status embed_args(const void* ids, int ids64, int64_t tokens, int64_t vocab, int64_t dim) {
    if (tokens < 0 || tokens >= kMaxGrid || vocab < 0 || vocab >= kMaxGrid - 1 || dim < 0) return SC_ERR_INVALID;
    if (product(std::max<int64_t>(tokens, vocab), dim, 8) < 0) return SC_ERR_INVALID;
    if (tokens > 0 && dim > 0 && (!ids || !multiple(ids, ids64 ? 8 : 4))) return SC_ERR_INVALID;
    return SC_OK;
}

// -------------------------------------------------------- convolution
sc_status conv_args(const sc_conv_desc* d, bool step, ConvParams* p) {
    if (!d) return SC_ERR_INVALID;
    const int eb = bytes_of(d->dtype);
    if (d->dtype < 0 || d->dtype > SC_BF16) return SC_ERR_INVALID;
    if (!eb) return SC_ERR_UNSUPPORTED;
    if (d->width < 1 || d->width > SC_CONV_MAX_WIDTH || d->batch < 0 || d->length < 0 || d->channels < 0 ||
        d->reserved != 0 || (step && d->length != 1))
        return SC_ERR_INVALID;
    if (product(d->batch, std::max<int64_t>(d->length, 1), d->channels, 64) < 0) return SC_ERR_INVALID;
    // the smallest run and channel group of any kernel
    const int64_t runs = (d->length + 7) / 8, blocks = (d->channels + 511) / 512;
    const int64_t grid = product(d->batch, std::max<int64_t>(runs, 1), std::max<int64_t>(blocks, 1));
    if (grid < 0 || grid > kMaxGrid || product(d->channels, d->width + 1) / 128 >= kMaxGrid) return SC_ERR_INVALID;
    const bool any = d->batch > 0 && d->length > 0 && d->channels > 0;
    if (any) {
        const Tensor x{d->x, d->batch, d->length, d->channels, d->x_batch, step ? 0 : d->x_token, eb};
        if (!x.ok() || !d->weight || !multiple(d->weight, eb)) return SC_ERR_INVALID;
    }
    if ((d->bias && !multiple(d->bias, eb)) || (d->state && !multiple(d->state, eb))) return SC_ERR_INVALID;
    *p = ConvParams{};
    p->width = d->width;
    p->silu = d->silu != 0;
    p->batch = d->batch;
    p->length = d->length;
    p->channels = d->channels;
    p->x = d->x;
    p->x_batch = d->x_batch;
    p->x_token = d->x_token;
    p->weight = d->weight;
    p->bias = d->bias;
    p->heads = step ? nullptr : d->heads;
    p->state = step ? nullptr : d->state;
    return SC_OK;
}

Tensor conv_state(const void* p, const sc_conv_desc* d) {
    return flat(p, d->batch * (d->width - 1) * d->channels, bytes_of(d->dtype));
}
Tensor conv_weight(const sc_conv_desc* d) { return flat(d->weight, d->channels * d->width, bytes_of(d->dtype)); }
Tensor conv_bias(const sc_conv_desc* d) { return flat(d->bias, d->channels, bytes_of(d->dtype)); }

// ------------------------------------------------------ selective scan
sc_status ssm_args(const sc_ssm_desc* d, bool step, SsmParams* p) {
    if (!d) return SC_ERR_INVALID;
    const int eb = bytes_of(d->dtype);
    if (d->dtype < 0 || d->dtype > SC_BF16) return SC_ERR_INVALID;
    if (!eb) return SC_ERR_UNSUPPORTED;
    if (d->batch < 0 || d->length < 0 || d->channels < 0 || d->states < 1 || d->groups < 1 || (step && d->length != 1))
        return SC_ERR_INVALID;
    if (d->states > SC_SSM_MAX_STATES) return SC_ERR_UNSUPPORTED;
    if (d->channels % d->groups != 0) return SC_ERR_INVALID;
    if (product(d->batch, std::max<int64_t>(d->length, 1), std::max(d->channels, 2 * d->groups), 8 * SC_SSM_MAX_STATES) < 0)
        return SC_ERR_INVALID;
    // the smallest channel block and chunk of any kernel; the last sums' grids
    const int64_t tiles = (d->length + SC_SSM_SAVE - 1) / SC_SSM_SAVE;
    const int64_t per = d->channels / d->groups, blocks = (per + 7) / 8 * d->groups;
    const int64_t grid = product(d->batch, std::max<int64_t>(blocks, 1), std::max<int64_t>(tiles, 1));
    const int64_t bc = product(d->batch, d->length, d->groups, d->states);
    if (grid < 0 || grid > kMaxGrid || bc / 256 >= kMaxGrid || d->channels * (d->states + 2) / 256 >= kMaxGrid)
        return SC_ERR_INVALID;
    if (d->batch > 0 && d->length > 0 && d->channels > 0) {
        const int64_t bt = d->batch, l = d->length, c = d->channels;
        const int64_t f = step ? 0 : 1;
        if (!Tensor{d->x, bt, l, c, d->x_batch, f * d->x_token, eb}.ok() ||
            !Tensor{d->dt, bt, l, c, d->dt_batch, f * d->dt_token, eb}.ok())
            return SC_ERR_INVALID;
        if (d->z && !Tensor{d->z, bt, l, c, d->z_batch, f * d->z_token, eb}.ok()) return SC_ERR_INVALID;
        if (d->B_group < 0 || d->C_group < 0) return SC_ERR_INVALID;
        const __int128 gb = (__int128)(d->groups - 1) * d->B_group + d->states;
        const __int128 gc = (__int128)(d->groups - 1) * d->C_group + d->states;
        if (gb > ((__int128)1 << 40) || gc > ((__int128)1 << 40)) return SC_ERR_INVALID;
        if (!Tensor{d->B, bt, l, (int64_t)gb, d->B_batch, f * d->B_token, eb}.ok() ||
            !Tensor{d->C, bt, l, (int64_t)gc, d->C_batch, f * d->C_token, eb}.ok())
            return SC_ERR_INVALID;
        if (!d->A || !multiple(d->A, 4)) return SC_ERR_INVALID;
    }
    if (!multiple(d->D, 4) || !multiple(d->dt_bias, 4) || !multiple(d->state, 4)) return SC_ERR_INVALID;
    *p = SsmParams{};
    p->softplus = d->softplus != 0;
    p->batch = d->batch;
    p->length = d->length;
    p->channels = d->channels;
    p->states = d->states;
    p->groups = d->groups;
    p->x = d->x;
    p->dt = d->dt;
    p->B = d->B;
    p->C = d->C;
    p->z = d->z;
    p->x_batch = d->x_batch;
    p->x_token = d->x_token;
    p->dt_batch = d->dt_batch;
    p->dt_token = d->dt_token;
    p->z_batch = d->z_batch;
    p->z_token = d->z_token;
    p->B_batch = d->B_batch;
    p->B_token = d->B_token;
    p->B_group = d->B_group;
    p->C_batch = d->C_batch;
    p->C_token = d->C_token;
    p->C_group = d->C_group;
    p->A = d->A;
    p->D = d->D;
    p->dt_bias = d->dt_bias;
    p->state = step ? nullptr : d->state;
    p->heads = step ? nullptr : d->heads;
    return SC_OK;
}

Tensor ssm_x(const sc_ssm_desc* d, const void* p, int64_t sb, int64_t st) {
    return {p, d->batch, d->length, d->channels, sb, st, bytes_of(d->dtype)};
}

// B or C: a token's groups as one row, up to the last group's end (ssm_args checks it).
Tensor ssm_bc(const sc_ssm_desc* d, const void* p, int64_t sb, int64_t st, int64_t group) {
    return {p, d->batch, d->length, (d->groups - 1) * group + d->states, sb, st, bytes_of(d->dtype)};
}
// What every form of the scan reads, into in[0 .. 7] (a step's token strides are not used).
constexpr int kSsmInputs = 8;
void ssm_inputs(const sc_ssm_desc* d, bool step, Tensor* in) {
    const int64_t f = step ? 0 : 1;
    in[0] = ssm_x(d, d->x, d->x_batch, f * d->x_token);
    in[1] = ssm_x(d, d->dt, d->dt_batch, f * d->dt_token);
    in[2] = ssm_x(d, d->z, d->z_batch, f * d->z_token);
    in[3] = ssm_bc(d, d->B, d->B_batch, f * d->B_token, d->B_group);
    in[4] = ssm_bc(d, d->C, d->C_batch, f * d->C_token, d->C_group);
    in[5] = flat(d->A, d->channels * d->states, 4);
    in[6] = flat(d->D, d->channels, 4);
    in[7] = flat(d->dt_bias, d->channels, 4);
}

// 16-byte accesses for every tensor that the tiled kernels read or write.
bool ssm_vec(const sc_ssm_desc* d, const Tensor* more, int n_more) {
    const int e = 16 / bytes_of(d->dtype);
    if ((d->channels / d->groups) % e != 0 || d->states % e != 0) return false;
    if (!ssm_x(d, d->x, d->x_batch, d->x_token).vec(e) || !ssm_x(d, d->dt, d->dt_batch, d->dt_token).vec(e)) return false;
    if (d->z && !ssm_x(d, d->z, d->z_batch, d->z_token).vec(e)) return false;
    if (!ssm_x(d, d->B, d->B_batch, d->B_token).vec(e) || !ssm_x(d, d->C, d->C_batch, d->C_token).vec(e)) return false;
    if (d->groups > 1 && (d->B_group % e != 0 || d->C_group % e != 0)) return false;
    for (int i = 0; i < n_more; ++i)
        if (!more[i].vec(e)) return false;
    return true;
}

void ssm_place(SsmParams* p, const SsmPlan& g, unsigned char* base) {
    p->chunks = g.chunks;
    p->chunk_tiles = g.chunk_tiles;
    p->runs = g.runs;
    p->run_tiles = g.run_tiles;
    p->carry = reinterpret_cast<float*>(base + g.carry);
    p->sum_d = reinterpret_cast<float*>(base + g.sum_d);
    p->cut = base + g.cut;
    p->part_bc = reinterpret_cast<float*>(base + g.part_bc);
    p->part_a = reinterpret_cast<float*>(base + g.part_a);
    p->part_d = reinterpret_cast<float*>(base + g.part_d);
    p->odd = base + g.odd;
}

sc_status zero(void* p, size_t bytes, cudaStream_t s) {
    if (!p || !bytes) return SC_OK;
    return cudaMemsetAsync(p, 0, bytes, s) == cudaSuccess ? SC_OK : SC_ERR_CUDA;
}
// dst = src, or zeros without one
sc_status copy_or_zero(void* dst, const void* src, size_t bytes, cudaStream_t s) {
    if (!dst || !bytes || dst == src) return SC_OK;
    if (!src) return zero(dst, bytes, s);
    return cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, s) == cudaSuccess ? SC_OK : SC_ERR_CUDA;
}
sc_status status_of(cudaError_t e) { return e == cudaSuccess ? SC_OK : SC_ERR_CUDA; }

bool plan_ok(int64_t batch, int64_t length, int64_t channels, int64_t states, int64_t groups) {
    return batch > 0 && length > 0 && channels > 0 && states > 0 && states <= SC_SSM_MAX_STATES && groups > 0 &&
           channels % groups == 0 && product(batch, length, channels, 8 * SC_SSM_MAX_STATES) >= 0;
}

}  // namespace

extern "C" {

sc_status sc_embed(const void* d_ids, int ids64, int64_t tokens, sc_dtype dtype, const void* d_weight, int64_t vocab,
                   int64_t dim, int64_t ldw, float scale, void* d_out, int64_t ldo, sc_stream_t stream) {
    const sc_status st = embed_args(d_ids, ids64, tokens, vocab, dim);
    if (st != SC_OK) return st;
    if (dtype < 0 || dtype > SC_BF16) return SC_ERR_INVALID;
    const int eb = bytes_of(dtype);
    if (!eb) return SC_ERR_UNSUPPORTED;
    if (ldw < dim || ldo < dim) return SC_ERR_INVALID;
    if (tokens == 0 || dim == 0) return SC_OK;
    const Tensor w{d_weight, 1, vocab, dim, 0, ldw, eb}, o{d_out, 1, tokens, dim, 0, ldo, eb};
    if ((vocab > 0 && !w.ok()) || !o.ok() || share(w, o) || share(o, flat(d_ids, tokens, ids64 ? 8 : 4)))
        return SC_ERR_INVALID;
    const int e = 16 / eb;
    EmbedParams p{};
    p.ids = d_ids;
    p.ids64 = ids64 != 0;
    p.tokens = tokens;
    p.vocab = vocab;
    p.dim = dim;
    p.weight = d_weight;
    p.ldw = ldw;
    p.scale = scale;
    p.out = d_out;
    p.ldo = ldo;
    p.vec = vec_row(dim, ldw, d_weight, e, vocab) && vec_row(dim, ldo, d_out, e, tokens);
    return status_of(launch_embed(dtype, p, cu(stream)));
}

size_t sc_embed_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim) {
    if (embed_args(reinterpret_cast<const void*>(8), 1, tokens, vocab, dim) != SC_OK || !vocab || !dim) return 0;
    return seq_scratch_total(embed_grad_plan(tokens, vocab, dim).total);
}

sc_status sc_embed_grad(const void* d_ids, int ids64, int64_t tokens, sc_dtype dtype, const void* d_dout, int64_t ldd,
                        int64_t vocab, int64_t dim, float scale, sc_dtype wtype, void* d_dweight, int64_t ldw,
                        int accumulate, sc_stream_t stream) {
    sc_status st = embed_args(d_ids, ids64, tokens, vocab, dim);
    if (st != SC_OK) return st;
    if (dtype < 0 || dtype > SC_BF16 || wtype < 0 || wtype > SC_BF16) return SC_ERR_INVALID;
    const int eb = bytes_of(dtype), wb = bytes_of(wtype);
    if (!eb || !wb || (wtype != dtype && wtype != SC_F32)) return SC_ERR_UNSUPPORTED;
    if (ldd < dim || ldw < dim) return SC_ERR_INVALID;
    if (vocab == 0 || dim == 0) return SC_OK;
    const Tensor g{d_dout, 1, tokens, dim, 0, ldd, eb}, w{d_dweight, 1, vocab, dim, 0, ldw, wb};
    if ((tokens > 0 && !g.ok()) || !w.ok() || share(g, w) || share(w, flat(d_ids, tokens, ids64 ? 8 : 4)))
        return SC_ERR_INVALID;
    EmbedParams p{};
    p.ids = d_ids;
    p.ids64 = ids64 != 0;
    p.tokens = tokens;
    p.vocab = vocab;
    p.dim = dim;
    p.weight = d_dout;
    p.ldw = ldd;
    p.scale = scale;
    p.out = d_dweight;
    p.ldo = ldw;
    p.accumulate = accumulate != 0;
    p.vec = (tokens == 0 || vec_row(dim, ldd, d_dout, 16 / eb, tokens)) && vec_row(dim, ldw, d_dweight, 16 / eb, vocab);
    const EmbedGradPlan plan = embed_grad_plan(tokens, vocab, dim);
    unsigned char* base = nullptr;
    st = seq_scratch(cu(stream), plan.total, &base);
    if (st != SC_OK) return st;
    return launch_embed_grad(dtype, wtype, p, plan, base, cu(stream));
}

sc_status sc_causal_conv(const sc_conv_desc* d, void* y, int64_t y_batch, int64_t y_token, void* final_state,
                         sc_stream_t stream) {
    ConvParams p;
    const sc_status st = conv_args(d, false, &p);
    if (st != SC_OK) return st;
    const int eb = bytes_of(d->dtype);
    if (final_state && !multiple(final_state, eb)) return SC_ERR_INVALID;
    if (d->batch == 0 || d->channels == 0) return SC_OK;
    const Tensor fs = conv_state(final_state, d), is = conv_state(d->state, d);
    if (share(fs, is) && final_state != d->state) return SC_ERR_INVALID;
    if (d->length == 0)
        return copy_or_zero(final_state, d->state, (size_t)fs.channels * eb, cu(stream));
    if (final_state && final_state == d->state) return SC_ERR_INVALID;  // other runs of tokens still read it
    const Tensor x{d->x, d->batch, d->length, d->channels, d->x_batch, d->x_token, eb};
    const Tensor o{y, d->batch, d->length, d->channels, y_batch, y_token, eb};
    const Tensor in[] = {x, is, conv_weight(d), conv_bias(d), flat(d->heads, d->batch * d->length, 1)}, out[] = {o, fs};
    if (!o.ok() || !o.distinct() || !apart(out, in)) return SC_ERR_INVALID;
    const int e = 4;  // channels of a thread
    p.y = y;
    p.y_batch = y_batch;
    p.y_token = y_token;
    p.final_state = d->width > 1 ? final_state : nullptr;
    p.vec = d->channels % e == 0 && x.vec(e) && o.vec(e) && multiple(d->state, 4 * eb) && multiple(final_state, 4 * eb);
    return status_of(launch_conv(d->dtype, p, cu(stream)));
}

size_t sc_causal_conv_grad_workspace_bytes(int64_t batch, int64_t length, int64_t channels, int width) {
    if (batch <= 0 || length <= 0 || channels <= 0 || width < 1 || width > SC_CONV_MAX_WIDTH ||
        product(batch, length, channels, 64) < 0)
        return 0;
    return seq_scratch_total(conv_grad_scratch(batch, length, channels, width));
}

sc_status sc_causal_conv_grad(const sc_conv_desc* d, const void* dy, int64_t dy_batch, int64_t dy_token, void* dx,
                              int64_t dx_batch, int64_t dx_token, float* dweight, float* dbias, void* dstate,
                              sc_stream_t stream) {
    ConvParams p;
    sc_status st = conv_args(d, false, &p);
    if (st != SC_OK) return st;
    const int eb = bytes_of(d->dtype);
    if (!multiple(dweight, 4) || !multiple(dbias, 4) || !multiple(dstate, eb)) return SC_ERR_INVALID;
    if (d->channels == 0) return SC_OK;
    const cudaStream_t s = cu(stream);
    if (d->batch == 0 || d->length == 0) {
        st = zero(dweight, (size_t)d->channels * d->width * 4, s);
        if (st == SC_OK) st = zero(dbias, (size_t)d->channels * 4, s);
        return st == SC_OK ? zero(dstate, (size_t)conv_state(dstate, d).channels * eb, s) : st;
    }
    const Tensor x{d->x, d->batch, d->length, d->channels, d->x_batch, d->x_token, eb};
    const Tensor g{dy, d->batch, d->length, d->channels, dy_batch, dy_token, eb};
    const Tensor o{dx, d->batch, d->length, d->channels, dx_batch, dx_token, eb};
    const Tensor in[] = {x, g, conv_state(d->state, d), conv_weight(d), conv_bias(d),
                         flat(d->heads, d->batch * d->length, 1)};
    const Tensor out[] = {o, flat(dweight, d->channels * d->width, 4), flat(dbias, d->channels, 4),
                          conv_state(dstate, d)};
    if (!g.ok() || (dx && (!o.ok() || !o.distinct())) || !apart(out, in)) return SC_ERR_INVALID;
    const int e = 4;  // channels of a thread
    p.dy = dy;
    p.dy_batch = dy_batch;
    p.dy_token = dy_token;
    p.dx = dx;
    p.dx_batch = dx_batch;
    p.dx_token = dx_token;
    p.dweight = dweight;
    p.dbias = dbias;
    p.dstate = d->width > 1 ? dstate : nullptr;
    p.vec = d->channels % e == 0 && x.vec(e) && g.vec(e) && (!dx || o.vec(e)) && multiple(d->state, 4 * eb) &&
            multiple(dstate, 4 * eb);
    if (dweight || dbias) {
        unsigned char* base = nullptr;
        st = seq_scratch(s, conv_grad_scratch(d->batch, d->length, d->channels, d->width), &base);
        if (st != SC_OK) return st;
        p.partials = reinterpret_cast<float*>(base);
    }
    return status_of(launch_conv_grad(d->dtype, p, s));
}

sc_status sc_causal_conv_step(const sc_conv_desc* d, void* pool, int64_t pool_rows, const int32_t* slots, void* y,
                              int64_t y_batch, sc_stream_t stream) {
    ConvParams p;
    const sc_status st = conv_args(d, true, &p);
    if (st != SC_OK) return st;
    const int eb = bytes_of(d->dtype);
    if (pool_rows < 0 || (!slots && pool_rows < d->batch) || !multiple(slots, 4)) return SC_ERR_INVALID;
    if (product(pool_rows, d->width, d->channels, 8) < 0) return SC_ERR_INVALID;
    if (d->batch == 0 || d->channels == 0) return SC_OK;
    const Tensor x{d->x, d->batch, 1, d->channels, d->x_batch, 0, eb}, o{y, d->batch, 1, d->channels, y_batch, 0, eb};
    const Tensor ps = flat(pool, pool_rows * (d->width - 1) * d->channels, eb);
    const Tensor in[] = {x, conv_weight(d), conv_bias(d), flat(slots, d->batch, 4)}, out[] = {o, ps};
    if (!o.ok() || !o.distinct() || (ps.channels > 0 && !ps.ok()) || !apart(out, in)) return SC_ERR_INVALID;
    const int e = 4;  // channels of a thread
    p.y = y;
    p.y_batch = y_batch;
    p.pool = pool;
    p.pool_rows = pool_rows;
    p.slots = slots;
    p.vec = d->channels % e == 0 && x.vec(e) && o.vec(e) && multiple(pool, 4 * eb) && multiple(d->weight, 16);
    return status_of(launch_conv_step(d->dtype, p, cu(stream)));
}

size_t sc_selective_scan_saved_bytes(int64_t batch, int64_t length, int64_t channels, int64_t states) {
    if (!plan_ok(batch, length, channels, states, 1)) return 0;
    const int64_t tiles = (length + SC_SSM_SAVE - 1) / SC_SSM_SAVE;
    return (size_t)batch * tiles * channels * 4 * ssm_lanes(states) * 4;
}

size_t sc_selective_scan_workspace_bytes(int64_t batch, int64_t length, int64_t channels, int64_t states,
                                         int64_t groups) {
    if (!plan_ok(batch, length, channels, states, groups)) return 0;
    const size_t n = ssm_plan(batch, length, channels, states, groups, false).total;
    return n ? seq_scratch_total(n) : 0;
}

sc_status sc_selective_scan(const sc_ssm_desc* d, void* y, int64_t y_batch, int64_t y_token, float* final_state,
                            float* saved, sc_stream_t stream) {
    SsmParams p;
    sc_status st = ssm_args(d, false, &p);
    if (st != SC_OK) return st;
    if (!multiple(final_state, 4) || !multiple(saved, 16)) return SC_ERR_INVALID;
    if (d->batch == 0 || d->channels == 0) return SC_OK;
    const cudaStream_t s = cu(stream);
    const int64_t sn = d->batch * d->channels * d->states;
    const Tensor is = flat(d->state, sn, 4), fs = flat(final_state, sn, 4);
    if (share(is, fs) && (final_state != d->state || d->length > 0)) return SC_ERR_INVALID;
    if (d->length == 0) return copy_or_zero(final_state, d->state, (size_t)sn * 4, s);
    const Tensor o = ssm_x(d, y, y_batch, y_token);
    const Tensor sv = flat(saved, (int64_t)(sc_selective_scan_saved_bytes(d->batch, d->length, d->channels, d->states) / 4), 4);
    Tensor in[kSsmInputs + 2];
    ssm_inputs(d, false, in);
    in[kSsmInputs] = flat(d->heads, d->batch * d->length, 1);
    in[kSsmInputs + 1] = is;
    const Tensor out[] = {o, fs, sv};
    if (!o.ok() || !o.distinct() || !apart(out, in)) return SC_ERR_INVALID;
    const SsmPlan plan = ssm_plan(d->batch, d->length, d->channels, d->states, d->groups, false);
    unsigned char* base = nullptr;
    if (plan.total) {
        st = seq_scratch(s, plan.total, &base);
        if (st != SC_OK) return st;
    }
    ssm_place(&p, plan, base);
    p.y = y;
    p.y_batch = y_batch;
    p.y_token = y_token;
    p.final_state = final_state;
    p.saved = saved;
    p.vec = ssm_vec(d, &o, 1);
    return status_of(launch_ssm(d->dtype, p, plan, s));
}

size_t sc_selective_scan_grad_workspace_bytes(int64_t batch, int64_t length, int64_t channels, int64_t states,
                                              int64_t groups) {
    if (!plan_ok(batch, length, channels, states, groups)) return 0;
    return seq_scratch_total(ssm_plan(batch, length, channels, states, groups, true).total);
}

sc_status sc_selective_scan_grad(const sc_ssm_desc* d, const sc_ssm_grads* g, sc_stream_t stream) {
    SsmParams p;
    sc_status st = ssm_args(d, false, &p);
    if (st != SC_OK) return st;
    if (!g || !multiple(g->dA, 4) || !multiple(g->dD, 4) || !multiple(g->ddt_bias, 4) || !multiple(g->dstate, 4) ||
        !multiple(g->dfinal, 4) || !multiple(g->saved, 16))
        return SC_ERR_INVALID;
    if (d->channels == 0) return SC_OK;
    const cudaStream_t s = cu(stream);
    if (!g->dA) return SC_ERR_INVALID;
    const int64_t sn = d->batch * d->channels * d->states;
    const Tensor dst = flat(g->dstate, sn, 4), df = flat(g->dfinal, sn, 4);
    if (share(dst, df) && (g->dstate != g->dfinal || d->length > 0)) return SC_ERR_INVALID;
    if (d->batch == 0 || d->length == 0) {
        st = zero(g->dA, (size_t)d->channels * d->states * 4, s);
        if (st == SC_OK) st = zero(g->dD, (size_t)d->channels * 4, s);
        if (st == SC_OK) st = zero(g->ddt_bias, (size_t)d->channels * 4, s);
        return st == SC_OK ? copy_or_zero(g->dstate, g->dfinal, (size_t)sn * 4, s) : st;
    }
    const int eb = bytes_of(d->dtype);
    const int64_t row = d->length * d->channels, bcn = d->batch * d->length * d->groups * d->states;
    const Tensor dy = ssm_x(d, g->dy, g->dy_batch, g->dy_token);
    const Tensor out[] = {ssm_x(d, g->dx, row, d->channels), ssm_x(d, g->ddt, row, d->channels),
                          ssm_x(d, g->dz, row, d->channels), flat(g->dB, bcn, eb), flat(g->dC, bcn, eb),
                          flat(g->dA, d->channels * d->states, 4), flat(g->dD, d->channels, 4),
                          flat(g->ddt_bias, d->channels, 4), dst};
    if (!dy.ok() || !out[0].ok() || !out[1].ok() || (d->z ? !out[2].ok() : g->dz != nullptr) || !out[3].ok() ||
        !out[4].ok() || !g->saved)
        return SC_ERR_INVALID;
    const Tensor saved = flat(
        g->saved, (int64_t)(sc_selective_scan_saved_bytes(d->batch, d->length, d->channels, d->states) / 4), 4);
    Tensor in[kSsmInputs + 5];
    ssm_inputs(d, false, in);
    in[kSsmInputs] = flat(d->heads, d->batch * d->length, 1);
    in[kSsmInputs + 1] = flat(d->state, sn, 4);
    in[kSsmInputs + 2] = dy;
    in[kSsmInputs + 3] = saved;
    in[kSsmInputs + 4] = df;
    if (!apart(out, in)) return SC_ERR_INVALID;
    const SsmPlan plan = ssm_plan(d->batch, d->length, d->channels, d->states, d->groups, true);
    unsigned char* base = nullptr;
    st = seq_scratch(s, plan.total, &base);
    if (st != SC_OK) return st;
    ssm_place(&p, plan, base);
    p.dy = g->dy;
    p.dy_batch = g->dy_batch;
    p.dy_token = g->dy_token;
    p.saved = const_cast<float*>(g->saved);
    p.dfinal = g->dfinal;
    p.dx = g->dx;
    p.ddt = g->ddt;
    p.dz = g->dz;
    p.dB = g->dB;
    p.dC = g->dC;
    p.dA = g->dA;
    p.dD = g->dD;
    p.ddt_bias = g->ddt_bias;
    p.dstate = g->dstate;
    const Tensor more[] = {dy, out[0], out[1], d->z ? out[2] : out[0]};
    p.vec = ssm_vec(d, more, 4);
    return status_of(launch_ssm_grad(d->dtype, p, plan, s));
}

sc_status sc_selective_scan_step(const sc_ssm_desc* d, float* pool, int64_t pool_rows, const int32_t* slots, void* y,
                                 int64_t y_batch, sc_stream_t stream) {
    SsmParams p;
    const sc_status st = ssm_args(d, true, &p);
    if (st != SC_OK) return st;
    if (pool_rows < 0 || pool_rows > kMaxGrid || (!slots && pool_rows < d->batch) || !multiple(slots, 4))
        return SC_ERR_INVALID;
    if (product(pool_rows, d->states, d->channels, 8) < 0) return SC_ERR_INVALID;
    if (d->batch == 0 || d->channels == 0) return SC_OK;
    const int eb = bytes_of(d->dtype);
    const Tensor o = ssm_x(d, y, y_batch, 0), ps = flat(pool, pool_rows * d->channels * d->states, 4);
    Tensor in[kSsmInputs + 1];
    ssm_inputs(d, true, in);
    in[kSsmInputs] = flat(slots, d->batch, 4);
    const Tensor out[] = {o, ps};
    if (!o.ok() || !o.distinct() || (ps.channels > 0 && !ps.ok()) || !apart(out, in)) return SC_ERR_INVALID;
    p.y = y;
    p.y_batch = y_batch;
    p.pool = pool;
    p.pool_rows = pool_rows;
    p.slots = slots;
    // four states at a time: 16 bytes of float32, 4 elements of B and C
    p.vec = d->states % 4 == 0 && multiple(pool, 16) && multiple(d->A, 16) && multiple(d->B, 4 * eb) &&
            multiple(d->C, 4 * eb) && (d->batch == 1 || (d->B_batch % 4 == 0 && d->C_batch % 4 == 0)) &&
            (d->groups == 1 || (d->B_group % 4 == 0 && d->C_group % 4 == 0));
    return status_of(launch_ssm_step(d->dtype, p, cu(stream)));
}

}  // extern "C"
