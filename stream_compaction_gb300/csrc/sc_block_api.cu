// C ABI of the operators of a sequence model's block (include/sc_seq.h): the gated
// recurrence, the norm, and the way to experts and back.  Argument checks, plans and
// scratch, dispatch.  Nothing here throws.
#include "sc_seq_args.h"
#include "sc_seq_launch.h"

namespace {

using namespace scg;

sc_status types(int dtype) {
    if (dtype < 0 || dtype > SC_BF16) return SC_ERR_INVALID;
    return bytes_of(dtype) ? SC_OK : SC_ERR_UNSUPPORTED;
}
sc_status types(int dtype, int wtype) {
    const sc_status st = types(dtype);
    if (st != SC_OK) return st;
    if (wtype < 0 || wtype > SC_BF16) return SC_ERR_INVALID;
    return wtype == dtype || wtype == SC_F32 ? SC_OK : SC_ERR_UNSUPPORTED;
}

// ---------------------------------------------------------- gated scan
sc_status gated_args(const sc_gated_desc* d, bool step, GatedParams* p) {
    if (!d) return SC_ERR_INVALID;
    const sc_status st = types(d->dtype);
    if (st != SC_OK) return st;
    const int eb = bytes_of(d->dtype);
    if (d->batch < 0 || d->length < 0 || d->length > kMaxGrid / 2 || d->channels < 0 || (step && d->length != 1))
        return SC_ERR_INVALID;
    if (product(d->batch, std::max<int64_t>(d->length, 1), d->channels, 64) < 0) return SC_ERR_INVALID;
    // the smallest channel block, the largest cluster
    const int64_t grid = product(d->batch, (d->channels + 31) / 32, 16);
    if (grid < 0 || grid > kMaxGrid) return SC_ERR_INVALID;
    if (d->batch > 0 && d->length > 0 && d->channels > 0) {
        const int64_t f = step ? 0 : 1;
        if (!Tensor{d->x, d->batch, d->length, d->channels, d->x_batch, f * d->x_token, eb}.ok() ||
            !Tensor{d->gate, d->batch, d->length, d->channels, d->gate_batch, f * d->gate_token, eb}.ok())
            return SC_ERR_INVALID;
    }
    if (!multiple(d->state, 4)) return SC_ERR_INVALID;
    *p = GatedParams{};
    p->sigmoid = d->sigmoid != 0;
    p->batch = d->batch;
    p->length = d->length;
    p->channels = d->channels;
    p->x = d->x;
    p->gate = d->gate;
    p->x_batch = d->x_batch;
    p->x_token = d->x_token;
    p->gate_batch = d->gate_batch;
    p->gate_token = d->gate_token;
    p->heads = step ? nullptr : d->heads;
    p->state = step ? nullptr : d->state;
    return SC_OK;
}
Tensor gated_x(const sc_gated_desc* d, const void* p, int64_t sb, int64_t st) {
    return {p, d->batch, d->length, d->channels, sb, st, bytes_of(d->dtype)};
}
Tensor gated_state(const sc_gated_desc* d, const float* p) { return flat(p, d->batch * d->channels, 4); }
Tensor gated_saved(const sc_gated_desc* d, const float* p) {
    return flat(p, d->batch * ((d->length + SC_GATED_SAVE - 1) / SC_GATED_SAVE) * d->channels, 4);
}
// Whether the copy engine takes every tensor: rows aligned to 16 bytes, strides below
// 2^40 bytes and not 0, indices of 32 bits.
bool gated_wide(const sc_gated_desc* d, std::initializer_list<Tensor> all) {
    const int eb = bytes_of(d->dtype), e = 16 / eb;
    if (d->channels % e != 0 || d->channels > kMaxGrid || d->batch > kMaxGrid) return false;
    for (const Tensor& t : all) {
        const int64_t most = (((int64_t)1 << 40) - 1) / eb;
        if (!t.vec(e)) return false;
        if ((t.tokens > 1 && (t.st == 0 || t.st > most)) || (t.batch > 1 && (t.sb == 0 || t.sb > most))) return false;
    }
    return true;
}

// ---------------------------------------------------------------- norm
// A tensor's rows follow one another with one stride.
bool one_stride(const Tensor& t) { return !t.p || t.batch <= 1 || t.tokens <= 1 || t.sb == (__int128)t.tokens * t.st; }

sc_status norm_args(const sc_norm_desc* d, NormParams* p) {
    if (!d) return SC_ERR_INVALID;
    const sc_status st = types(d->dtype, d->weight || d->bias ? d->wtype : d->dtype);
    if (st != SC_OK) return st;
    if (d->batch < 0 || d->length < 0 || d->channels < 0 || !(d->eps >= 0.0f)) return SC_ERR_INVALID;
    const int64_t rows = product(d->batch, d->length);
    if (rows < 0 || rows >= kMaxGrid || product(rows, d->channels, 8) < 0 || d->channels >= kMaxGrid)
        return SC_ERR_INVALID;
    const int wb = d->weight || d->bias ? bytes_of(d->wtype) : 1;
    if (!multiple(d->weight, wb) || !multiple(d->bias, wb)) return SC_ERR_INVALID;
    *p = NormParams{};
    p->rms = d->rms != 0;
    p->params_f32 = d->wtype == SC_F32;
    p->eps = d->eps;
    p->rows = (uint32_t)rows;
    p->length = (uint32_t)d->length;
    p->channels = d->channels;
    p->weight = d->weight;
    p->bias = d->bias;
    p->x = d->x;
    p->x_batch = d->x_batch;
    p->x_token = d->x_token;
    return SC_OK;
}
Tensor norm_x(const sc_norm_desc* d, const void* p, int64_t sb, int64_t st) {
    return {p, d->batch, d->length, d->channels, sb, st, bytes_of(d->dtype)};
}
Tensor norm_parameter(const sc_norm_desc* d, const void* p) { return flat(p, d->channels, bytes_of(d->wtype)); }
// Rows by vectors where every tensor has aligned rows; one index where all have one stride.
template <int N>
void norm_rows(const sc_norm_desc* d, const Tensor (&t)[N], NormParams* p) {
    const int e = 16 / bytes_of(d->dtype), pair = 4 / bytes_of(d->dtype);
    bool one = true, dense = true;
    p->vec = d->channels % e == 0;
    p->pairs = d->channels % pair == 0;
    for (const Tensor& v : t) {
        if (!v.p) continue;
        p->vec = p->vec && v.vec(e);
        p->pairs = p->pairs && v.vec(pair);
        one = one && one_stride(v);
        dense = dense && (v.tokens > 1 ? v.st : v.sb) == v.channels;
    }
    // length 1: the batch strides are the rows'
    if (one && d->length > 1) p->length = p->rows;
    p->dense = one && dense;
}

// -------------------------------------------------------------- experts
sc_status expert_args(const sc_expert_desc* d, bool weights, ExpertParams* p) {
    if (!d) return SC_ERR_INVALID;
    const sc_status st = types(d->dtype, weights && d->weights ? d->wtype : d->dtype);
    if (st != SC_OK) return st;
    if (d->tokens < 0 || d->choices < 0 || d->dim < 0 || d->experts < 1 || d->experts > SC_EXPERT_MAX) return SC_ERR_INVALID;
    const int64_t entries = product(d->tokens, d->choices);
    if (entries < 0 || entries >= kMaxGrid || d->tokens >= kMaxGrid || product(std::max(entries, d->tokens), d->dim, 8) < 0)
        return SC_ERR_INVALID;
    if ((entries > 0 && !d->place) || (d->tokens > 0 && !d->offsets)) return SC_ERR_INVALID;
    if (!multiple(d->place, 4) || !multiple(d->offsets, 8)) return SC_ERR_INVALID;
    if (weights && d->weights && !multiple(d->weights, bytes_of(d->wtype))) return SC_ERR_INVALID;
    *p = ExpertParams{};
    p->tokens = d->tokens;
    p->choices = d->choices;
    p->dim = d->dim;
    p->entries = entries;
    p->place = d->place;
    p->kept = d->offsets ? d->offsets + d->experts : nullptr;
    p->weights = weights ? d->weights : nullptr;
    p->weights_f32 = d->wtype == SC_F32;
    return SC_OK;
}
Tensor expert_rows(const sc_expert_desc* d, const void* p, int64_t rows, int64_t ld) {
    return {p, 1, rows, d->dim, 0, ld, bytes_of(d->dtype)};
}
Tensor expert_weights(const sc_expert_desc* d, const void* p) { return flat(p, d->tokens * d->choices, bytes_of(d->wtype)); }
// Whether rows begin and end at multiples of `bytes`.
bool expert_rows_at(const sc_expert_desc* d, int bytes, std::initializer_list<Tensor> rows) {
    const int e = bytes / bytes_of(d->dtype);
    if (d->dim % e != 0) return false;
    for (const Tensor& t : rows)
        if (t.p && !t.vec(e)) return false;
    return true;
}
// A call from rows of tokens or entries to the other (or nothing to do: done).
template <class Launch>
sc_status expert_move(const sc_expert_desc* d, ExpertParams* p, const Tensor& in, const Tensor& out, Launch launch) {
    if (in.st < d->dim || out.st < d->dim) return SC_ERR_INVALID;
    if (d->dim == 0 || out.tokens == 0) return SC_OK;
    const Tensor ins[] = {in, flat(d->place, p->entries, 4), flat(d->offsets, d->experts + 1, 8),
                          expert_weights(d, p->weights)};
    const Tensor outs[] = {out};
    if ((in.tokens > 0 && !in.ok()) || !out.ok() || !apart(outs, ins)) return SC_ERR_INVALID;
    p->in = in.p;
    p->ld_in = in.st;
    p->out = const_cast<void*>(out.p);
    p->ld_out = out.st;
    p->vec = expert_rows_at(d, 16, {in, out});
    p->pairs = expert_rows_at(d, 4, {in, out});
    return status_of(launch());
}

}  // namespace

extern "C" {

// ---------------------------------------------------------- gated scan
size_t sc_gated_scan_saved_bytes(int64_t batch, int64_t length, int64_t channels) {
    if (batch <= 0 || length <= 0 || channels <= 0 || product(batch, length, channels, 64) < 0) return 0;
    return (size_t)batch * ((length + SC_GATED_SAVE - 1) / SC_GATED_SAVE) * channels * sizeof(float);
}

sc_status sc_gated_scan(const sc_gated_desc* d, void* y, int64_t y_batch, int64_t y_token, float* final_state,
                        float* saved, sc_stream_t stream) {
    GatedParams p;
    const sc_status st = gated_args(d, false, &p);
    if (st != SC_OK) return st;
    if (!multiple(final_state, 4) || !multiple(saved, 4)) return SC_ERR_INVALID;
    if (d->batch == 0 || d->channels == 0) return SC_OK;
    const Tensor is = gated_state(d, d->state), fs = gated_state(d, final_state);
    if (share(is, fs) && (final_state != d->state || d->length > 0)) return SC_ERR_INVALID;
    if (d->length == 0) return copy_or_zero(final_state, d->state, (size_t)is.channels * 4, cu(stream));
    const Tensor x = gated_x(d, d->x, d->x_batch, d->x_token), g = gated_x(d, d->gate, d->gate_batch, d->gate_token);
    const Tensor o = gated_x(d, y, y_batch, y_token);
    const Tensor in[] = {x, g, flat(d->heads, d->batch * d->length, 1), is}, out[] = {o, fs, gated_saved(d, saved)};
    if (!o.ok() || !o.distinct() || !apart(out, in)) return SC_ERR_INVALID;
    p.y = y;
    p.y_batch = y_batch;
    p.y_token = y_token;
    p.final_state = final_state;
    p.saved = saved;
    p.pairs = d->channels % 2 == 0 && x.vec(2) && g.vec(2) && o.vec(2);
    p.wide = gated_wide(d, {x, g, o});
    return status_of(launch_gated(d->dtype, p, cu(stream)));
}

sc_status sc_gated_scan_grad(const sc_gated_desc* d, const void* dy, int64_t dy_batch, int64_t dy_token,
                             const float* saved, const float* dfinal, void* dx, void* dgate, float* dstate,
                             sc_stream_t stream) {
    GatedParams p;
    const sc_status st = gated_args(d, false, &p);
    if (st != SC_OK) return st;
    if (!multiple(saved, 4) || !multiple(dfinal, 4) || !multiple(dstate, 4)) return SC_ERR_INVALID;
    if (d->batch == 0 || d->channels == 0) return SC_OK;
    const Tensor df = gated_state(d, dfinal), ds = gated_state(d, dstate);
    if (share(df, ds) && (dfinal != dstate || d->length > 0)) return SC_ERR_INVALID;
    if (d->length == 0) return copy_or_zero(dstate, dfinal, (size_t)df.channels * 4, cu(stream));
    if (!saved) return SC_ERR_INVALID;
    const int64_t row = d->length * d->channels;
    const Tensor x = gated_x(d, d->x, d->x_batch, d->x_token), g = gated_x(d, d->gate, d->gate_batch, d->gate_token);
    const Tensor e = gated_x(d, dy, dy_batch, dy_token);
    const Tensor out[] = {gated_x(d, dx, row, d->channels), gated_x(d, dgate, row, d->channels), ds};
    const Tensor in[] = {x, g, e, flat(d->heads, d->batch * d->length, 1), gated_saved(d, saved), df};
    if (!e.ok() || !out[0].ok() || !out[1].ok() || !apart(out, in)) return SC_ERR_INVALID;
    p.saved = const_cast<float*>(saved);
    p.dy = dy;
    p.dy_batch = dy_batch;
    p.dy_token = dy_token;
    p.dfinal = dfinal;
    p.dx = dx;
    p.dgate = dgate;
    p.dstate = dstate;
    p.pairs = d->channels % 2 == 0 && x.vec(2) && g.vec(2) && e.vec(2) && out[0].vec(2) && out[1].vec(2);
    p.wide = gated_wide(d, {x, g, e, out[0], out[1]});
    return status_of(launch_gated_grad(d->dtype, p, cu(stream)));
}

sc_status sc_gated_scan_step(const sc_gated_desc* d, float* pool, int64_t pool_rows, const int32_t* slots, void* y,
                             int64_t y_batch, sc_stream_t stream) {
    GatedParams p;
    const sc_status st = gated_args(d, true, &p);
    if (st != SC_OK) return st;
    if (pool_rows < 0 || (!slots && pool_rows < d->batch) || !multiple(slots, 4)) return SC_ERR_INVALID;
    if (product(pool_rows, d->channels, 8) < 0) return SC_ERR_INVALID;
    if (d->batch == 0 || d->channels == 0) return SC_OK;
    const Tensor x = gated_x(d, d->x, d->x_batch, 0), g = gated_x(d, d->gate, d->gate_batch, 0), o = gated_x(d, y, y_batch, 0);
    const Tensor ps = flat(pool, pool_rows * d->channels, 4);
    const Tensor in[] = {x, g, flat(slots, d->batch, 4)}, out[] = {o, ps};
    if (!o.ok() || !o.distinct() || (ps.channels > 0 && !ps.ok()) || !apart(out, in)) return SC_ERR_INVALID;
    p.y = y;
    p.y_batch = y_batch;
    p.pool = pool;
    p.pool_rows = pool_rows;
    p.slots = slots;
    p.vec = d->channels % 4 == 0 && x.vec(4) && g.vec(4) && o.vec(4) && multiple(pool, 16);
    return status_of(launch_gated_step(d->dtype, p, cu(stream)));
}

// ---------------------------------------------------------------- norm
sc_status sc_layer_norm(const sc_norm_desc* d, void* y, int64_t y_batch, int64_t y_token, void* sum,
                        int64_t sum_batch, int64_t sum_token, float* saved, sc_stream_t stream) {
    NormParams p;
    const sc_status st = norm_args(d, &p);
    if (st != SC_OK) return st;
    if (!multiple(saved, 8)) return SC_ERR_INVALID;
    if (p.rows == 0 || p.channels == 0) return SC_OK;
    if ((d->residual == nullptr) != (sum == nullptr)) return SC_ERR_INVALID;
    const Tensor x = norm_x(d, d->x, d->x_batch, d->x_token), o = norm_x(d, y, y_batch, y_token);
    const Tensor e = norm_x(d, d->residual, d->residual_batch, d->residual_token), s = norm_x(d, sum, sum_batch, sum_token);
    if (!x.ok() || !o.ok() || !o.distinct()) return SC_ERR_INVALID;
    if (d->residual && (!e.ok() || !s.ok() || !s.distinct())) return SC_ERR_INVALID;
    const Tensor in[] = {x, e, norm_parameter(d, d->weight), norm_parameter(d, d->bias)};
    const Tensor out[] = {o, s, flat(saved, (int64_t)p.rows * 2, 4)};
    if (!apart(out, in)) return SC_ERR_INVALID;
    p.residual = d->residual;
    p.residual_batch = d->residual_batch;
    p.residual_token = d->residual_token;
    p.y = y;
    p.y_batch = y_batch;
    p.y_token = y_token;
    p.sum = sum;
    p.sum_batch = sum_batch;
    p.sum_token = sum_token;
    p.saved = saved;
    const Tensor rows[] = {x, o, e, s};
    norm_rows(d, rows, &p);
    return status_of(launch_norm(d->dtype, p, cu(stream)));
}

size_t sc_layer_norm_grad_workspace_bytes(int64_t batch, int64_t length, int64_t channels, sc_dtype dtype) {
    const int64_t rows = batch > 0 && length > 0 ? product(batch, length) : 0;
    if (types(dtype) != SC_OK || channels <= 0 || rows <= 0 || rows >= kMaxGrid || product(rows, channels, 8) < 0 ||
        channels >= kMaxGrid)
        return 0;
    return seq_scratch_total(norm_grad_scratch(rows, channels));
}

sc_status sc_layer_norm_grad(const sc_norm_desc* d, const void* dy, int64_t dy_batch, int64_t dy_token,
                             const void* dsum, int64_t dsum_batch, int64_t dsum_token, const float* saved, void* dx,
                             float* dweight, float* dbias, sc_stream_t stream) {
    NormParams p;
    sc_status st = norm_args(d, &p);
    if (st != SC_OK) return st;
    if (!multiple(saved, 8) || !multiple(dweight, 4) || !multiple(dbias, 4)) return SC_ERR_INVALID;
    if (p.channels == 0) return SC_OK;
    const cudaStream_t s = cu(stream);
    if (p.rows == 0) {
        st = zero(dweight, (size_t)p.channels * 4, s);
        return st == SC_OK ? zero(dbias, (size_t)p.channels * 4, s) : st;
    }
    const Tensor x = norm_x(d, d->x, d->x_batch, d->x_token), e = norm_x(d, dy, dy_batch, dy_token);
    const Tensor t = norm_x(d, dsum, dsum_batch, dsum_token);
    const Tensor o = norm_x(d, dx, d->length * d->channels, d->channels);
    if (!x.ok() || !e.ok() || !o.ok() || (dsum && !t.ok()) || !saved) return SC_ERR_INVALID;
    const Tensor in[] = {x, e, t, norm_parameter(d, d->weight), flat(saved, (int64_t)p.rows * 2, 4)};
    const Tensor out[] = {o, flat(dweight, p.channels, 4), flat(dbias, p.channels, 4)};
    if (!apart(out, in)) return SC_ERR_INVALID;
    p.dy = dy;
    p.dy_batch = dy_batch;
    p.dy_token = dy_token;
    p.dsum = dsum;
    p.dsum_batch = dsum_batch;
    p.dsum_token = dsum_token;
    p.saved = const_cast<float*>(saved);
    p.dx = dx;
    p.dweight = dweight;
    p.dbias = dbias;
    const Tensor rows[] = {x, e, t, o};
    norm_rows(d, rows, &p);
    if (dweight || dbias) {
        unsigned char* base = nullptr;
        st = seq_scratch(s, norm_grad_scratch(p.rows, p.channels), &base);
        if (st != SC_OK) return st;
        p.partials = reinterpret_cast<float*>(base);
    }
    return status_of(launch_norm_grad(d->dtype, p, s));
}

// -------------------------------------------------------------- experts
sc_status sc_expert_sort(const void* d_ids, int ids64, int64_t entries, int64_t experts, int32_t* d_order,
                         int32_t* d_place, int64_t* d_offsets, sc_stream_t stream) {
    if (entries < 0 || entries >= kMaxGrid || experts < 1) return SC_ERR_INVALID;
    if (experts > SC_EXPERT_MAX) return SC_ERR_UNSUPPORTED;
    if (!d_offsets || !multiple(d_offsets, 8)) return SC_ERR_INVALID;
    if (entries > 0 && (!d_ids || !d_order || !d_place || !multiple(d_ids, ids64 ? 8 : 4) || !multiple(d_order, 4) ||
                        !multiple(d_place, 4)))
        return SC_ERR_INVALID;
    const Tensor in[] = {flat(d_ids, entries, ids64 ? 8 : 4)};
    const Tensor out[] = {flat(d_order, entries, 4), flat(d_place, entries, 4), flat(d_offsets, experts + 1, 8)};
    if (!apart(out, in)) return SC_ERR_INVALID;
    return status_of(launch_expert_sort(d_ids, ids64 != 0, entries, (int)experts, d_order, d_place, d_offsets, cu(stream)));
}

sc_status sc_expert_gather(const sc_expert_desc* d, const void* d_x, int64_t ldx, void* d_rows, int64_t ldr,
                           sc_stream_t stream) {
    ExpertParams p;
    const sc_status st = expert_args(d, false, &p);
    if (st != SC_OK) return st;
    return expert_move(d, &p, expert_rows(d, d_x, d->tokens, ldx), expert_rows(d, d_rows, p.entries, ldr),
                       [&] { return launch_expert_gather(d->dtype, p, cu(stream)); });
}

sc_status sc_expert_gather_grad(const sc_expert_desc* d, const void* d_drows, int64_t ldr, void* d_dx, int64_t ldx,
                                sc_stream_t stream) {
    ExpertParams p;
    const sc_status st = expert_args(d, false, &p);
    if (st != SC_OK) return st;
    return expert_move(d, &p, expert_rows(d, d_drows, p.entries, ldr), expert_rows(d, d_dx, d->tokens, ldx),
                       [&] { return launch_expert_combine(d->dtype, p, cu(stream)); });
}

sc_status sc_expert_combine(const sc_expert_desc* d, const void* d_rows, int64_t ldr, void* d_out, int64_t ldo,
                            sc_stream_t stream) {
    ExpertParams p;
    const sc_status st = expert_args(d, true, &p);
    if (st != SC_OK) return st;
    return expert_move(d, &p, expert_rows(d, d_rows, p.entries, ldr), expert_rows(d, d_out, d->tokens, ldo),
                       [&] { return launch_expert_combine(d->dtype, p, cu(stream)); });
}

sc_status sc_expert_combine_grad(const sc_expert_desc* d, const void* d_dout, int64_t ldo, const void* d_rows,
                                 int64_t ldr, void* d_drows, int64_t ldd, void* d_dweights, sc_stream_t stream) {
    ExpertParams p;
    const sc_status st = expert_args(d, true, &p);
    if (st != SC_OK) return st;
    if (d_dweights) {
        const sc_status wt = types(d->dtype, d->wtype);
        if (wt != SC_OK) return wt;
        if (!multiple(d_dweights, bytes_of(d->wtype))) return SC_ERR_INVALID;
    }
    if (ldo < d->dim || ldd < d->dim || (d_dweights && ldr < d->dim)) return SC_ERR_INVALID;
    if (p.entries == 0) return SC_OK;
    if (d->dim == 0) return zero(d_dweights, (size_t)p.entries * bytes_of(d->wtype), cu(stream));
    const Tensor g = expert_rows(d, d_dout, d->tokens, ldo), o = expert_rows(d, d_drows, p.entries, ldd);
    const Tensor r = expert_rows(d, d_dweights ? d_rows : nullptr, p.entries, ldr), w = expert_weights(d, d_dweights);
    if (!g.ok() || !o.ok() || (d_dweights && !r.ok())) return SC_ERR_INVALID;
    const Tensor in[] = {g, r, flat(d->place, p.entries, 4), flat(d->offsets, d->experts + 1, 8), expert_weights(d, p.weights)};
    const Tensor out[] = {o, w};
    if (!apart(out, in)) return SC_ERR_INVALID;
    p.in = d_dout;
    p.ld_in = ldo;
    p.rows = r.p;
    p.ld_rows = ldr;
    p.out = d_drows;
    p.ld_out = ldd;
    p.dweights = d_dweights;
    p.vec = expert_rows_at(d, 16, {g, o, r});
    p.pairs = expert_rows_at(d, 4, {g, o, r});
    return status_of(launch_expert_combine_grad(d->dtype, p, cu(stream)));
}

}  // extern "C"
