// mixer.h -- launch interface and device helpers of the mixer kernels: the
// short causal convolution in front of the recurrence and the norms behind
// and around it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rssm {

// Convolution calls.  Channels are ordered x (H*P), B (G*N), C (G*N).
struct ConvParams {
    const void *u;          // raw inputs, one row of Cc channels per token (in dtype)
    const void *dtr;        // raw dt, one row of H values per token
    int64_t u_pitch, dt_pitch;   // elements between consecutive tokens' rows
    void *x, *B, *C, *dt;   // outputs, dense per token (in dtype)
    void *ring;             // [nslots, R, Cc] recent raw inputs (in dtype)
    int32_t *head;          // [nslots] ring row of the next token
    int32_t *work;          // [nslots] arrival counters (zero between calls)
    int32_t *err;           // sticky device error word (work[nslots])
    const float *w;         // [W, Cc], tap W-1 multiplies the current token
    const float *bias;      // [Cc] or NULL
    const float *dt_bias;   // [H] or NULL
    const int32_t *slot_idx;// [rows] or NULL
    const int32_t *n_keep;  // [rows] (accept)
    const int32_t *cu;      // [rows+1] (packed prompts)
    const int32_t *fresh;   // [rows] or NULL (packed prompts)
    int64_t total;          // packed tokens
    int rows, nslots, H, HP, GN, Cc, R, T;
    int from_zero, silu;
    float dt_min, dt_max;
    int nblk;               // workgroups across the channels of a row
    int tile;               // packed prompts: tokens per workgroup
};

hipError_t launch_conv_tokens(const ConvParams &p, bool in_bf16, int width, bool advance, hipStream_t s);
hipError_t launch_conv_packed(const ConvParams &p, bool in_bf16, int width, hipStream_t s);
hipError_t launch_conv_accept(const ConvParams &p, hipStream_t s);

struct GatedNormParams {
    const void *y;          // [rows, dim] fp32 or bf16, dense
    const void *z;          // [rows, dim], z_pitch elements between rows
    void *out;              // [rows, dim], dense
    const float *w;         // [dim]
    int64_t z_pitch;
    int64_t rows;
    int dim, groups;
    float eps;
    int before;             // norm before the gate
};

struct AddNormParams {
    const void *x;          // [rows, dim] block output, dense
    const void *res;        // [rows, dim] residual, dense
    void *res_out;          // [rows, dim], may be res
    void *out;              // [rows, dim] normed
    const float *w;         // [dim]
    const float *post;      // [dim] weight of the norm of x, or NULL
    int64_t rows;
    int dim;
    float scale, eps;
};

hipError_t launch_gated_norm(const GatedNormParams &p, bool y_bf16, bool z_bf16, bool out_bf16, hipStream_t s);
hipError_t launch_add_norm(const AddNormParams &p, bool x_bf16, bool res_bf16, bool out_bf16, hipStream_t s);

}  // namespace rssm
