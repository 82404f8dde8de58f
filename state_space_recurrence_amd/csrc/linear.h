// linear.h -- launch interface of the matrix product with its epilogue.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rssm {

// out = residual + scale act(x w^T + bias): x [rows, n_in], w [n_out, n_in].
struct LinearParams {
    const void *x, *w;            // bf16, or E4M3 codes (MX)
    const uint8_t *x_scales;      // [rows, n_in / 32], MX operands
    const uint8_t *w_scales;      // [n_out, n_in / 32]
    const float *bias;            // [n_out] or NULL
    const void *res;              // [rows, n_out] or NULL, dense
    void *out;                    // [rows, n_out], dense
    uint8_t *out_scales;          // [rows, n_out / 32], MX outputs
    int64_t rows;
    int64_t x_pitch, w_pitch;     // bytes between rows
    int k_bytes;                  // bytes of a row's n_in elements
    int n_out;
    float scale;
    int act;                      // 0 none, 1 SiLU, 2 GELU, 3 squared ReLU
    int out_type;                 // RSSM_F32, RSSM_BF16 or RSSM_FP8_E4M3 (MX)
    int res_bf16;
};

// fast: MX operands may be multiplied by the scaled 8-bit products.
hipError_t launch_linear(const LinearParams &p, bool mx, bool fast, hipStream_t s);

}  // namespace rssm
