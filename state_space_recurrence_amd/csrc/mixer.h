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

// Packed prompts go over tiles of tokens.  The tiles that touch a slot's history
// for the prompt start .. end - 1 (end > start): that of the first token and that
// of the last token whose taps reach before the prompt read it (the head, and ring
// rows behind it), those of the last W - 1 inputs, which are kept, write it.  With
// tiles of at least W - 1 tokens no other tile holds a token between the ends of
// either pair, so the new head may be published when all of these are done.
struct HistoryTiles {
    int first, reach, keep, last;   // not descending, but for keep, which may lie before reach
    __host__ __device__ HistoryTiles(int start, int end, int width, int tile) {
        const int m = end - start < width - 1 ? end - start : width - 1;   // tokens that reach back, and inputs kept
        first = start / tile;
        reach = (start + m - 1) / tile;
        keep = (end - m) / tile;
        last = (end - 1) / tile;
    }
    __host__ __device__ bool has(int t) const { return t == first || t == reach || t == keep || t == last; }
    __host__ __device__ int count() const {
        return 1 + (reach != first) + (keep != first && keep != reach) + (last != first && last != reach && last != keep);
    }
};

// Workgroups across the channels of a row, and tokens of a packed prompt per
// workgroup: 32 tokens read 3 of their neighbour's again; when that leaves
// compute units without work, fewer tokens do (down to 4, more than the W - 1
// that HistoryTiles asks for).
constexpr int kConvThreads = 256, kConvVec = 8;

inline int64_t conv_channel_blocks(int64_t channels) {
    return (channels / kConvVec + kConvThreads - 1) / kConvThreads;
}

inline int conv_tile(int64_t total, int64_t nblk) {
    int tile = 32;
    while (tile > 4 && (total + tile - 1) / tile * nblk < 512) tile >>= 1;
    return tile;
}

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
    uint8_t *out_scales;    // [rows, dim / 32], MX outputs
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
    uint8_t *out_scales;    // [rows, dim / 32], MX outputs
};

struct QuantizeParams {
    const void *x;          // [rows, dim], x_pitch elements between rows
    uint8_t *out;           // [rows, dim] codes, dense
    uint8_t *out_scales;    // [rows, dim / 32]
    int64_t x_pitch;
    int64_t rows;
    int dim;
};

hipError_t launch_gated_norm(const GatedNormParams &p, bool y_bf16, bool z_bf16, bool out_bf16, hipStream_t s);
hipError_t launch_add_norm(const AddNormParams &p, bool x_bf16, bool res_bf16, bool out_bf16, hipStream_t s);
hipError_t launch_gated_norm_mx(const GatedNormParams &p, bool y_bf16, bool z_bf16, hipStream_t s);
hipError_t launch_add_norm_mx(const AddNormParams &p, bool x_bf16, bool res_bf16, hipStream_t s);
hipError_t launch_quantize(const QuantizeParams &p, bool x_bf16, hipStream_t s);

}  // namespace rssm
