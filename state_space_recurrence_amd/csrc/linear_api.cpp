// linear_api.cpp -- extern "C" entry points of the projections and of rows in
// 8 bits: argument validation on the host, then asynchronous kernel launches.
// See include/replayssm.h for the contract of every call.
#include <hip/hip_runtime.h>

#include <cmath>

#include "api_common.h"
#include "linear.h"
#include "mixer.h"
#include "replayssm.h"

using namespace rssm::host;

namespace {

constexpr int kBlock = 32;          // elements that share a scale
constexpr int kMaxUnit = 16384;     // elements of a norm's group or row
constexpr int kMaxSide = 1 << 20;   // n_in, n_out of a product

bool float_type(int32_t t) { return t == RSSM_F32 || t == RSSM_BF16; }

bool aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Rows that leave in MX: rows of whole blocks, codes in wide stores.
int check_mx_rows(const char *what, int64_t rows, int32_t dim, int32_t groups, int32_t most) {
    if (rows < 0 || rows > (int64_t)1 << 26) return fail(RSSM_E_ARG, "%s: rows outside 0..2^26", what);
    if (dim < 1 || groups < 1 || dim % groups != 0 || dim / groups % kBlock != 0)
        return fail(RSSM_E_ARG, "%s: dim %d over groups %d must be a positive multiple of 32", what, dim, groups);
    if (dim / groups > most)
        return fail(RSSM_E_CAPACITY, "%s: %d elements per norm exceed %d", what, dim / groups, most);
    if (rows * groups > 0x7FFFFFFF) return fail(RSSM_E_ARG, "%s: rows * groups too large", what);
    return RSSM_OK;
}

int check_eps(const char *what, float eps) {
    if (!(eps >= 0.f) || std::isinf(eps)) return fail(RSSM_E_ARG, "%s: eps must be finite and >= 0", what);
    return RSSM_OK;
}

int check_codes(const char *what, const void *codes, const void *scales) {
    if (!codes || !scales) return fail(RSSM_E_ARG, "%s: a pointer is NULL", what);
    if (!aligned(codes)) return fail(RSSM_E_ARG, "%s: MX codes start at a multiple of 16 bytes", what);
    return RSSM_OK;
}

typedef __int128 wide;   // any pitch in bytes

// Whether `bytes` bytes at `out` touch any of `rows` rows of `row` bytes that lie `pitch` apart (none for NULL).
bool touches(const void *in, int64_t rows, int64_t row, wide pitch, const void *out, int64_t bytes) {
    if (!in || !out) return false;
    const wide at = (wide) reinterpret_cast<uintptr_t>(out) - reinterpret_cast<uintptr_t>(in);
    if (at + bytes <= 0 || at >= (rows - 1) * pitch + row) return false;
    if (at < 0) return true;
    const wide in_row = at % pitch;
    return in_row < row || in_row + bytes > pitch;   // in a row, or between two and into the next
}

bool touches(const void *in, int64_t size, const void *out, int64_t bytes) { return touches(in, 1, size, size, out, bytes); }

int64_t size_of(int32_t t) { return t == RSSM_F32 ? 4 : t == RSSM_BF16 ? 2 : 1; }

// What a call writes: up to two buffers (rows in 8 bits: codes and scales).  Other workgroups read the operands while
// they are written.
struct Written {
    const void *a;
    int64_t a_bytes;
    const void *b;
    int64_t b_bytes;
    Written(const void *out, int64_t bytes) : a(out), a_bytes(bytes), b(nullptr), b_bytes(0) {}
    Written(const void *codes, const void *scales, int64_t rows, int64_t dim)
        : a(codes), a_bytes(rows * dim), b(scales), b_bytes(rows * dim / kBlock) {}
    bool over(const void *in, int64_t rows, int64_t row, wide pitch) const {
        return touches(in, rows, row, pitch, a, a_bytes) || (b && touches(in, rows, row, pitch, b, b_bytes));
    }
    bool over(const void *in, int64_t size) const { return over(in, 1, size, size); }
    bool over_itself() const { return b && touches(a, a_bytes, b, b_bytes); }
};

int overlap(const char *what) { return fail(RSSM_E_ARG, "%s: an output overlaps another buffer of the call", what); }

}  // namespace

extern "C" {

int replayssm_quantize_mx(int64_t rows, int32_t dim, const void *x, int32_t x_dtype, int64_t x_pitch, void *codes,
                          uint8_t *scales, hipStream_t stream) {
    RSSM_TRY(check_mx_rows("quantize_mx", rows, dim, 1, 1 << 20));
    if (!float_type(x_dtype)) return fail(RSSM_E_UNSUPPORTED, "quantize_mx: x is F32 or BF16");
    if (rows == 0) return RSSM_OK;
    if (!x) return fail(RSSM_E_ARG, "quantize_mx: a pointer is NULL");
    RSSM_TRY(check_codes("quantize_mx", codes, scales));
    if (x_pitch < dim) return fail(RSSM_E_ARG, "quantize_mx: x_pitch shorter than a row");
    if (rows * (dim / 8) > (int64_t)1 << 38)   // 2^30 threads along the first axis, below 2^16 workgroups along the second
        return fail(RSSM_E_CAPACITY, "quantize_mx: more work than a launch holds");
    const Written out(codes, scales, rows, dim);
    const int64_t size = size_of(x_dtype);
    if (out.over_itself() || out.over(x, rows, dim * size, (wide)x_pitch * size)) return overlap("quantize_mx");
    rssm::QuantizeParams p{x, static_cast<uint8_t *>(codes), scales, x_pitch, rows, dim};
    return hip_status(rssm::launch_quantize(p, x_dtype == RSSM_BF16, stream), "quantize launch");
}

int replayssm_gated_norm_mx(int64_t rows, int32_t dim, int32_t groups, const void *y, int32_t y_dtype, const void *z,
                            int32_t z_dtype, int64_t z_pitch, const float *weight, float eps, int32_t norm_before_gate,
                            void *codes, uint8_t *scales, hipStream_t stream) {
    RSSM_TRY(check_mx_rows("gated_norm_mx", rows, dim, groups, kMaxUnit));
    RSSM_TRY(check_eps("gated_norm_mx", eps));
    if (!float_type(y_dtype) || !float_type(z_dtype))
        return fail(RSSM_E_UNSUPPORTED, "gated_norm_mx: y and z are F32 or BF16");
    if (norm_before_gate != 0 && norm_before_gate != 1)
        return fail(RSSM_E_ARG, "gated_norm_mx: norm_before_gate must be 0 or 1");
    if (rows == 0) return RSSM_OK;
    if (!y || !z || !weight) return fail(RSSM_E_ARG, "gated_norm_mx: a pointer is NULL");
    RSSM_TRY(check_codes("gated_norm_mx", codes, scales));
    if (z_pitch < dim) return fail(RSSM_E_ARG, "gated_norm_mx: z_pitch shorter than a row");
    const Written out(codes, scales, rows, dim);
    const int64_t z_size = size_of(z_dtype);
    if (out.over_itself() || out.over(y, rows * dim * size_of(y_dtype)) || out.over(weight, dim * 4) ||
        out.over(z, rows, dim * z_size, (wide)z_pitch * z_size))
        return overlap("gated_norm_mx");
    rssm::GatedNormParams p{y, z, codes, weight, z_pitch, rows, dim, groups, eps, norm_before_gate, scales};
    return hip_status(rssm::launch_gated_norm_mx(p, y_dtype == RSSM_BF16, z_dtype == RSSM_BF16, stream),
                      "gated norm launch");
}

int replayssm_add_norm_mx(int64_t rows, int32_t dim, const void *x, int32_t x_dtype, const void *residual,
                          void *residual_out, int32_t res_dtype, const float *weight, const float *post_weight,
                          float scale, float eps, void *codes, uint8_t *scales, hipStream_t stream) {
    RSSM_TRY(check_mx_rows("add_norm_mx", rows, dim, 1, kMaxUnit));
    RSSM_TRY(check_eps("add_norm_mx", eps));
    if ((x && !float_type(x_dtype)) || !float_type(res_dtype))
        return fail(RSSM_E_UNSUPPORTED, "add_norm_mx: x and residual are F32 or BF16");
    if (rows == 0) return RSSM_OK;
    if (!residual || !weight) return fail(RSSM_E_ARG, "add_norm_mx: a pointer is NULL");
    if (x ? !residual_out : (residual_out || post_weight))
        return fail(RSSM_E_ARG, "add_norm_mx: residual_out goes with x, and post_weight needs it");
    RSSM_TRY(check_codes("add_norm_mx", codes, scales));
    const Written out(codes, scales, rows, dim);
    const int64_t x_bytes = rows * dim * size_of(x_dtype), res_bytes = rows * dim * size_of(res_dtype);
    const Written sum(residual_out, residual_out ? res_bytes : 0);   // a row is read whole before it is written
    if (out.over_itself() || out.over(x, x_bytes) || out.over(residual, res_bytes) || out.over(residual_out, res_bytes) ||
        out.over(weight, dim * 4) || out.over(post_weight, dim * 4) || sum.over(weight, dim * 4) ||
        sum.over(post_weight, dim * 4) || (residual_out != residual && sum.over(residual, res_bytes)) ||
        ((residual_out != x || x_dtype != res_dtype) && sum.over(x, x_bytes)))
        return overlap("add_norm_mx");
    rssm::AddNormParams p{x, residual, residual_out, codes, weight, post_weight, rows, dim, scale, eps, scales};
    return hip_status(rssm::launch_add_norm_mx(p, x && x_dtype == RSSM_BF16, res_dtype == RSSM_BF16, stream),
                      "add norm launch");
}

int replayssm_linear(const rssm_linear_desc *desc, const rssm_linear_io *io, hipStream_t stream) {
    if (!desc) return fail(RSSM_E_ARG, "linear: desc is NULL");
    const rssm_linear_desc &d = *desc;
    if (d.rows < 0 || d.rows > (int64_t)1 << 26) return fail(RSSM_E_ARG, "linear: rows outside 0..2^26");
    if (d.n_in < 1 || d.n_in > kMaxSide || d.n_out < 1 || d.n_out > kMaxSide)
        return fail(RSSM_E_ARG, "linear: n_in %d or n_out %d outside 1..2^20", d.n_in, d.n_out);
    if (d.in_dtype != RSSM_BF16 && d.in_dtype != RSSM_FP8_E4M3)
        return fail(RSSM_E_UNSUPPORTED, "linear: in_dtype %d: BF16, or FP8_E4M3 with scales", d.in_dtype);
    if (!float_type(d.out_dtype) && d.out_dtype != RSSM_FP8_E4M3)
        return fail(RSSM_E_UNSUPPORTED, "linear: out_dtype %d: F32, BF16, or FP8_E4M3 with scales", d.out_dtype);
    if (d.res_dtype != RSSM_NONE && !float_type(d.res_dtype))
        return fail(RSSM_E_UNSUPPORTED, "linear: res_dtype %d: NONE, F32 or BF16", d.res_dtype);
    if (d.activation < RSSM_ACT_NONE || d.activation > RSSM_ACT_RELU2)
        return fail(RSSM_E_ARG, "linear: activation %d is none of rssm_activation", d.activation);
    if (d.products != RSSM_PRODUCTS_EXACT && d.products != RSSM_PRODUCTS_FAST)
        return fail(RSSM_E_ARG, "linear: products %d is none of rssm_products", d.products);
    const bool mx = d.in_dtype == RSSM_FP8_E4M3, mx_out = d.out_dtype == RSSM_FP8_E4M3, res = d.res_dtype != RSSM_NONE;
    if (mx && d.n_in % kBlock != 0) return fail(RSSM_E_ARG, "linear: MX operands need n_in %d a multiple of 32", d.n_in);
    if (mx_out && d.n_out % kBlock != 0)
        return fail(RSSM_E_ARG, "linear: MX outputs need n_out %d a multiple of 32", d.n_out);
    // Tiles of 64 x 64 and 256 threads: fewer than 2^32 threads (a launch of more runs a part of them).
    if (((d.rows + 63) / 64) * ((d.n_out + 63) / 64) >= (int64_t)1 << 24)
        return fail(RSSM_E_CAPACITY, "linear: %lld rows of %d outputs are more than a launch holds", (long long)d.rows, d.n_out);
    if (d.rows == 0) return RSSM_OK;
    if (!io) return fail(RSSM_E_ARG, "linear: io is NULL");
    if (!io->x || !io->weight || !io->out) return fail(RSSM_E_ARG, "linear: x / weight / out is NULL");
    if (mx) {
        RSSM_TRY(check_codes("linear", io->x, io->x_scales));
        RSSM_TRY(check_codes("linear", io->weight, io->weight_scales));
    }
    if (mx_out) RSSM_TRY(check_codes("linear", io->out, io->out_scales));
    if (res != (io->residual != nullptr)) return fail(RSSM_E_ARG, "linear: residual goes with res_dtype");
    const int size = mx ? 1 : 2;
    if (io->x_pitch < d.n_in || (mx && io->x_pitch != d.n_in))
        return fail(RSSM_E_ARG, "linear: x_pitch shorter than a row, or MX rows that are not dense");
    if (io->x_pitch > (int64_t)1 << 22)   // a tile's rows are addressed in 31 bits
        return fail(RSSM_E_CAPACITY, "linear: x_pitch over 2^22 elements");
    const int64_t k_bytes = (int64_t)d.n_in * size;
    const int64_t out_size = size_of(d.out_dtype);
    const Written out = mx_out ? Written(io->out, io->out_scales, d.rows, d.n_out) : Written(io->out, d.rows * d.n_out * out_size);
    if (out.over_itself() || out.over(io->x, d.rows, k_bytes, io->x_pitch * size) || out.over(io->weight, d.n_out * k_bytes) ||
        out.over(io->bias, (int64_t)d.n_out * 4) ||
        (mx && (out.over(io->x_scales, d.rows * d.n_in / kBlock) || out.over(io->weight_scales, (int64_t)d.n_out * d.n_in / kBlock))) ||
        ((io->residual != io->out || d.res_dtype != d.out_dtype) && out.over(io->residual, d.rows * d.n_out * size_of(d.res_dtype))))
        return overlap("linear");
    rssm::LinearParams p{};
    p.x = io->x;
    p.w = io->weight;
    p.x_scales = io->x_scales;
    p.w_scales = io->weight_scales;
    p.bias = io->bias;
    p.res = io->residual;
    p.out = io->out;
    p.out_scales = io->out_scales;
    p.rows = d.rows;
    p.x_pitch = io->x_pitch * size;
    p.w_pitch = (int64_t)d.n_in * size;
    p.k_bytes = d.n_in * size;
    p.n_out = d.n_out;
    p.scale = d.scale;
    p.act = d.activation;
    p.out_type = d.out_dtype;
    p.res_bf16 = d.res_dtype == RSSM_BF16;
    return hip_status(rssm::launch_linear(p, mx, d.products == RSSM_PRODUCTS_FAST, stream), "linear launch");
}

}  // extern "C"
