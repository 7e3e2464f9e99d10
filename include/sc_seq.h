/*
 * sc_seq.h -- C ABI of the library's sequence-model operators: token embedding
 * with its gradient by sorted tokens, the short causal convolution, and the
 * selective state space scan (libsc_gb300.so, next to the scans of sc_scan.h,
 * whose types, status codes and conventions it uses).
 *
 * What the calls compute (b row of the batch, t token, e channel, n state; all
 * sums, states and exponentials in float32 whatever the tensors' type, each
 * output rounded once):
 *
 *   embedding    out[t] = scale * weight[ids[t]]; an id outside [0, vocab)
 *                gives a row of zeros (as the histogram skips such entries)
 *                dweight[v] = scale * sum of dout[t] over the t with ids[t] == v,
 *                in a fixed order of parts: bitwise the same on every run of
 *                the same ids (where the parts of a long sum are cut depends on
 *                the other ids)
 *   convolution  pre[t,e] = bias[e] + sum_k weight[e,k] * x[t-W+1+k, e]
 *                y = pre * sigmoid(pre), or pre (silu == 0)
 *   scan         d[t,e] = softplus(dt[t,e] + dt_bias[e])  (softplus == 0: the sum)
 *                h[t,e,n] = exp(d[t,e] * A[e,n]) * h[t-1,e,n] + d[t,e] * x[t,e] * B[t,g,n]
 *                y[t,e] = sum_n C[t,g,n] * h[t,e,n] + D[e] * x[t,e],
 *                         times z[t,e] * sigmoid(z[t,e]) where z is given;
 *                g = e / (channels / groups): each group of B and C serves
 *                channels / groups consecutive channels.
 * It is the scan under the composition of affine maps that sc_scan.h defines
 * for uint32 pairs, over float32, with the maps made on the fly and applied.
 *
 * Segments.  heads (one byte per token, batch x length, contiguous; may be
 * NULL) restarts a row as sc_scan_segmented does: where heads[b,t] != 0 the
 * state before t is zero, and the convolution sees no input before t.  The
 * state before token 0 is `state` (zeros where NULL) unless heads[b,0] != 0.
 *
 * Layout.  Elements of a token are contiguous; batch and token strides
 * (*_batch, *_token, in elements, >= 0) are free, so the halves of a joint
 * projection's output need no copy.  weight, bias, A, D, dt_bias, states and
 * heads are contiguous.  Outputs must not overlap inputs or one another
 * (SC_ERR_INVALID; column slices of one joint buffer do not overlap), except
 * that a step's state is updated in place.  Tensors whose pointers and
 * strides are multiples of 16 bytes take 16-byte accesses; others work, element
 * by element.
 *
 * Types.  SC_F32, SC_F16 or SC_BF16 for the activations (and the convolution's
 * weight, bias and state, the embedding's weight); A, D, dt_bias, the scan's
 * states and the parameters' gradients are float32.
 *
 * Calls are asynchronous and stream-ordered.  Those that need scratch memory
 * (the two gradients that sum over tokens, and a scan whose rows are too few
 * for the machine, which splits the length) take it from the stream's
 * workspace of sc_scan.h, after its look-back part, under the same rules:
 * allocated on first use and grown, or bound by sc_set_workspace (the
 * *_workspace_bytes are for the current device); such a call
 * on a capturing stream returns SC_ERR_UNSUPPORTED.  The others may be
 * captured: sc_embed, sc_causal_conv, both steps, and any call whose
 * *_workspace_bytes is 0.  Empty problems (no tokens, no rows, no channels)
 * succeed; sums over no tokens are zeros.
 */
#ifndef SC_SEQ_H
#define SC_SEQ_H

#include "sc_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SC_CONV_MAX_WIDTH 8
#define SC_SSM_MAX_STATES 64
/* Tokens between the states that a scan saves for its gradient. */
#define SC_SSM_SAVE 16

/* ---- token embedding ----
 * ids: int32 (ids64 == 0) or int64, contiguous.  weight: vocab rows of dim
 * elements, ldw >= dim apart; out rows ldo >= dim apart.  vocab < 2^31 - 1,
 * tokens < 2^31. */
sc_status sc_embed(const void *d_ids, int ids64, int64_t tokens, sc_dtype dtype, const void *d_weight, int64_t vocab,
                   int64_t dim, int64_t ldw, float scale, void *d_out, int64_t ldo, sc_stream_t stream);

/* Gradient of the embedding's weight.  dout: type dtype, rows ldd >= dim
 * apart; dweight: type wtype (dtype or SC_F32), rows ldw >= dim apart.  Every
 * row is written: zeros for an absent token (accumulate != 0: the sums are
 * added to what dweight holds, absent rows stay).  Ids outside [0, vocab) give
 * nothing.  The tokens are sorted by id (stable), then each row sums its own.
 */
sc_status sc_embed_grad(const void *d_ids, int ids64, int64_t tokens, sc_dtype dtype, const void *d_dout, int64_t ldd,
                        int64_t vocab, int64_t dim, float scale, sc_dtype wtype, void *d_dweight, int64_t ldw,
                        int accumulate, sc_stream_t stream);
size_t sc_embed_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim);

/* ---- short causal convolution, one filter per channel ---- */
typedef struct {
    int32_t dtype;             /* sc_dtype of x, y, weight, bias, state */
    int32_t width;             /* 1 .. SC_CONV_MAX_WIDTH */
    int32_t silu;              /* 0: y = pre */
    int32_t reserved;          /* 0 */
    int64_t batch, length, channels;
    const void *x;             /* batch x length x channels */
    int64_t x_batch, x_token;
    const void *weight;        /* channels x width; the last tap meets the current token */
    const void *bias;          /* channels; NULL: zeros */
    const uint8_t *heads;      /* batch x length; NULL: none */
    const void *state;         /* batch x (width - 1) x channels, oldest first; NULL: zeros */
} sc_conv_desc;

/* y (strides y_batch, y_token); final_state (like state; NULL: not wanted)
 * receives the last width - 1 inputs of the open segment, zeros before its
 * start, ready for the next call or for sc_causal_conv_step. */
sc_status sc_causal_conv(const sc_conv_desc *p, void *y, int64_t y_batch, int64_t y_token, void *final_state,
                         sc_stream_t stream);
/* Gradients by x (strides dx_*), weight (float32, channels x width), bias
 * (float32) and state (like state); any may be NULL.  Sums over tokens are
 * taken in a fixed order. */
sc_status sc_causal_conv_grad(const sc_conv_desc *p, const void *dy, int64_t dy_batch, int64_t dy_token, void *dx,
                              int64_t dx_batch, int64_t dx_token, float *dweight, float *dbias, void *dstate,
                              sc_stream_t stream);
size_t sc_causal_conv_grad_workspace_bytes(int64_t batch, int64_t length, int64_t channels, int width);
/* One token for each of `batch` sequences (p->length == 1 and p->x_token,
 * heads, state are not used): row r has its inputs in state row slots[r] of a
 * pool of pool_rows x (width - 1) x channels, which is moved on by one token
 * in place.  slots == NULL: row r itself (pool_rows >= batch).  A slot outside
 * [0, pool_rows) leaves the row out: zeros in y, no state touched.  No slot may
 * appear twice. */
sc_status sc_causal_conv_step(const sc_conv_desc *p, void *pool, int64_t pool_rows, const int32_t *slots, void *y,
                              int64_t y_batch, sc_stream_t stream);

/* ---- selective state space scan ---- */
typedef struct {
    int32_t dtype;             /* sc_dtype of x, dt, B, C, z, y and their gradients */
    int32_t softplus;          /* 0: d = dt + dt_bias */
    int64_t batch, length, channels, states, groups;
    const void *x, *dt;        /* batch x length x channels */
    int64_t x_batch, x_token, dt_batch, dt_token;
    const float *A;            /* channels x states; -infinity acts as the lowest finite value */
    const void *B, *C;         /* batch x length x groups x states, a group's states contiguous */
    int64_t B_batch, B_token, B_group, C_batch, C_token, C_group;
    const float *D;            /* channels; NULL: zeros */
    const void *z;             /* batch x length x channels; NULL: no gate */
    int64_t z_batch, z_token;
    const float *dt_bias;      /* channels; NULL: zeros */
    const uint8_t *heads;      /* batch x length; NULL: none */
    const float *state;        /* batch x channels x states; NULL: zeros */
} sc_ssm_desc;

/* y; final_state (like state; NULL: not wanted): h after the last token.
 * saved (sc_selective_scan_saved_bytes; NULL: not wanted): the state before
 * every SC_SSM_SAVE-th token, for sc_selective_scan_grad. */
sc_status sc_selective_scan(const sc_ssm_desc *p, void *y, int64_t y_batch, int64_t y_token, float *final_state,
                            float *saved, sc_stream_t stream);
size_t sc_selective_scan_saved_bytes(int64_t batch, int64_t length, int64_t channels, int64_t states);
size_t sc_selective_scan_workspace_bytes(int64_t batch, int64_t length, int64_t channels, int64_t states,
                                         int64_t groups);

typedef struct {
    const void *dy;            /* batch x length x channels */
    int64_t dy_batch, dy_token;
    const float *saved;        /* as sc_selective_scan wrote it for the same inputs */
    const float *dfinal;       /* gradient by the final state; NULL: zeros */
    void *dx, *ddt, *dz;       /* batch x length x channels, contiguous; dz NULL exactly where z is */
    void *dB, *dC;             /* batch x length x groups x states, contiguous */
    float *dA;                 /* channels x states */
    float *dD, *ddt_bias;      /* channels; NULL: not wanted */
    float *dstate;             /* like state; NULL: not wanted */
} sc_ssm_grads;

/* Every sum over tokens, rows or channels is taken in a fixed order: bitwise
 * the same on every run. */
sc_status sc_selective_scan_grad(const sc_ssm_desc *p, const sc_ssm_grads *g, sc_stream_t stream);
/* Mostly partial rows of dB and dC: 0.5, 1, 4 or 32 bytes for each token and
 * channel with up to 8, 16, 32 or 64 states (at 4 x 4096 tokens of 4096 channels
 * 2.1 GB with 64 states).  The stream keeps it until a larger call or
 * sc_release_stream. */
size_t sc_selective_scan_grad_workspace_bytes(int64_t batch, int64_t length, int64_t channels, int64_t states,
                                              int64_t groups);

/* One token for each of `batch` sequences (p->length == 1; *_token, heads and
 * state are not used): y, and the state in row slots[r] of a pool of pool_rows x
 * channels x states moved on in place; slots as in sc_causal_conv_step. */
sc_status sc_selective_scan_step(const sc_ssm_desc *p, float *pool, int64_t pool_rows, const int32_t *slots, void *y,
                                 int64_t y_batch, sc_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SC_SEQ_H */
