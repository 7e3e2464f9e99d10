// Host side of the sequence operators: kernel parameters, launchers, and what
// sc_api.cu lends them (the stream's workspace, the launch counter).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/sc_seq.h"

namespace scg {

// `bytes` of scratch from the stream's workspace (256-byte aligned, contents
// undefined).  Refuses a capturing stream.
sc_status seq_scratch(cudaStream_t s, size_t bytes, unsigned char** out);
size_t seq_scratch_total(size_t bytes);  // workspace bytes that hold it
void count_launches(int n);
long long seq_sms();  // multiprocessors of the current device

// ------------------------------------------------------------- embedding
struct EmbedParams {
    const void* ids;
    int ids64;
    long long tokens, vocab, dim;
    const void* weight;  // dout for the gradient
    long long ldw;
    float scale;
    void* out;  // dweight for the gradient
    long long ldo;
    int vec;  // rows in 16-byte words
    int accumulate;
};
cudaError_t launch_embed(int dtype, const EmbedParams& p, cudaStream_t s);

// Scratch of the gradient, all sizes in bytes.
struct EmbedGradPlan {
    int digit_bits, passes;
    long long tiles;  // of the sort
    size_t keys0, keys1, vals0, vals1, first, last, counts, partials, total;  // offsets, then the size
};
EmbedGradPlan embed_grad_plan(long long tokens, long long vocab, long long dim);
sc_status launch_embed_grad(int dtype, int wtype, const EmbedParams& p, const EmbedGradPlan& plan,
                            unsigned char* scratch, cudaStream_t s);

// ----------------------------------------------------------- convolution
struct ConvParams {
    int width, silu;
    long long batch, length, channels;
    const void* x;
    long long x_batch, x_token;
    const void* weight;
    const void* bias;
    const uint8_t* heads;
    const void* state;
    void* y;
    long long y_batch, y_token;
    void* final_state;
    // gradient
    const void* dy;
    long long dy_batch, dy_token;
    void* dx;
    long long dx_batch, dx_token;
    float* dweight;
    float* dbias;
    void* dstate;
    float* partials;
    // step
    void* pool;
    long long pool_rows;
    const int32_t* slots;
    int vec;
};
cudaError_t launch_conv(int dtype, const ConvParams& p, cudaStream_t s);
size_t conv_grad_scratch(long long batch, long long length, long long channels, int width);
cudaError_t launch_conv_grad(int dtype, const ConvParams& p, cudaStream_t s);
cudaError_t launch_conv_step(int dtype, const ConvParams& p, cudaStream_t s);

// -------------------------------------------------------- selective scan
struct SsmParams {
    int softplus, vec;
    long long batch, length, channels, states, groups;
    const void *x, *dt, *B, *C, *z;
    long long x_batch, x_token, dt_batch, dt_token, z_batch, z_token;
    long long B_batch, B_token, B_group, C_batch, C_token, C_group;
    const float *A, *D, *dt_bias, *state;
    const uint8_t* heads;
    void* y;
    long long y_batch, y_token;
    float* final_state;
    float* saved;
    // a length split into `chunks` runs of chunk_tiles tiles of SC_SSM_SAVE tokens
    int chunks;
    long long chunk_tiles;
    // what a run of run_tiles tiles makes of a zero state; a chunk is one run, or
    // some of them in the gradient
    int runs;
    long long run_tiles;
    float* carry;    // [batch][runs][channels][padded states]
    float* sum_d;    // [batch][runs][channels] the run's sum of d
    uint8_t* cut;    // [batch][runs] a segment starts inside the run
    // gradient
    const void* dy;
    long long dy_batch, dy_token;
    const float* dfinal;
    void *dx, *ddt, *dz, *dB, *dC;
    float *dA, *dD, *ddt_bias, *dstate;
    float* part_bc;  // [channel blocks][batch][length][2][padded states]
    float* part_a;   // [batch][chunks][channels][padded states]
    float* part_d;   // [2][batch][chunks][channels]
    uint8_t* odd;    // by CTA, padded states: it met an infinity or NaN and left
    // step
    float* pool;
    long long pool_rows;
    const int32_t* slots;
};
// Lanes that share a channel (4 states each) for a number of states: 2, 4, 8 or 16.
int ssm_lanes(long long states);
struct SsmPlan {
    int lanes, chunks, runs;
    long long chunk_tiles, run_tiles, blocks_per_group;  // channel blocks of one CTA
    size_t carry, sum_d, cut, part_bc, part_a, part_d, odd, total;
};
SsmPlan ssm_plan(long long batch, long long length, long long channels, long long states, long long groups, bool grad);
cudaError_t launch_ssm(int dtype, const SsmParams& p, const SsmPlan& plan, cudaStream_t s);
cudaError_t launch_ssm_grad(int dtype, const SsmParams& p, const SsmPlan& plan, cudaStream_t s);
cudaError_t launch_ssm_step(int dtype, const SsmParams& p, cudaStream_t s);

}  // namespace scg
