// mixer_api.cpp -- extern "C" entry points of the mixer operators around the
// recurrence: argument validation on the host, then asynchronous kernel
// launches.  See include/replayssm.h for the contract of every call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>

#include "api_common.h"
#include "kernels.h"
#include "mixer.h"
#include "replayssm.h"
#include "scan.h"

using namespace rssm::host;

namespace {

constexpr int kMinWidth = 2, kMaxWidth = 4, kMaxDraft = 8;
constexpr int kMaxUnit = 16384;   // elements of a norm's group or row

// A launch holds fewer than 2^32 threads along an axis (one that asks for more
// runs a part of them without an error).
int check_threads(const char *what, int64_t threads) {
    if (threads < (int64_t)1 << 32) return RSSM_OK;
    return fail(RSSM_E_CAPACITY, "%s: %lld threads are more than a launch holds", what, (long long)threads);
}

int conv_slots(const rssm_conv_desc *d) { return d->n_slots > 0 ? d->n_slots : d->batch; }

int64_t conv_channels(const rssm_conv_desc *d) {
    return (int64_t)d->n_heads * d->head_dim + 2 * (int64_t)d->n_groups * d->d_state;
}

int conv_rows(const rssm_conv_desc *d) {
    const int drafts = d->width - 1 + d->max_draft, prompt = 2 * (d->width - 1);
    return drafts > prompt ? drafts : prompt;
}

int check_conv_desc(const rssm_conv_desc *d) {
    if (!d) return fail(RSSM_E_ARG, "conv: desc is NULL");
    if (d->batch < 0) return fail(RSSM_E_ARG, "conv: batch %d < 0", d->batch);
    if (d->n_slots < 0) return fail(RSSM_E_ARG, "conv: n_slots %d < 0", d->n_slots);
    if (d->n_heads <= 0 || d->n_groups <= 0 || d->n_heads % d->n_groups != 0)
        return fail(RSSM_E_ARG, "conv: n_heads %d must be a positive multiple of n_groups %d", d->n_heads, d->n_groups);
    if (d->head_dim != 64 || d->d_state != 128)
        return fail(RSSM_E_UNSUPPORTED, "conv: head_dim %d x d_state %d: only 64 x 128 is built", d->head_dim,
                    d->d_state);
    if (d->width < kMinWidth || d->width > kMaxWidth)
        return fail(RSSM_E_UNSUPPORTED, "conv: width %d outside %d..%d", d->width, kMinWidth, kMaxWidth);
    if (d->max_draft < 1 || d->max_draft > kMaxDraft)
        return fail(RSSM_E_CAPACITY, "conv: max_draft %d outside 1..%d", d->max_draft, kMaxDraft);
    if (d->in_dtype != RSSM_F32 && d->in_dtype != RSSM_BF16)
        return fail(RSSM_E_UNSUPPORTED, "conv: in_dtype %d: only F32 and BF16 inputs", d->in_dtype);
    if (d->activation != 0 && d->activation != 1)
        return fail(RSSM_E_ARG, "conv: activation must be 0 (none) or 1 (SiLU)");
    if (!(d->dt_min <= d->dt_max)) return fail(RSSM_E_ARG, "conv: dt_min must not exceed dt_max");
    if (conv_channels(d) > 1 << 20) return fail(RSSM_E_ARG, "conv: too many channels");
    if ((int64_t)d->batch > 1 << 20 || (int64_t)conv_slots(d) > 1 << 24)
        return fail(RSSM_E_ARG, "conv: batch or n_slots too large");
    return RSSM_OK;
}

int check_conv_state(const rssm_conv_desc *d, const rssm_conv_state *s) {
    if (!s) return fail(RSSM_E_ARG, "conv: state is NULL");
    if (!s->ring || !s->head || !s->work || !s->weight)
        return fail(RSSM_E_ARG, "conv: state ring/head/work/weight is NULL");
    if (!s->slot_idx && d->batch > conv_slots(d))
        return fail(RSSM_E_ARG, "conv: batch %d exceeds n_slots %d without a slot map", d->batch, conv_slots(d));
    return RSSM_OK;
}

rssm::ConvParams conv_params(const rssm_conv_desc *d, const rssm_conv_state *s) {
    rssm::ConvParams p{};
    p.ring = s->ring;
    p.head = s->head;
    p.work = s->work;
    p.err = s->work + conv_slots(d);
    p.w = s->weight;
    p.bias = s->bias;
    p.dt_bias = s->dt_bias;
    p.slot_idx = s->slot_idx;
    p.rows = d->batch;
    p.nslots = conv_slots(d);
    p.H = d->n_heads;
    p.HP = d->n_heads * d->head_dim;
    p.GN = d->n_groups * d->d_state;
    p.Cc = p.HP + 2 * p.GN;
    p.R = conv_rows(d);
    p.T = 1;
    p.silu = d->activation;
    p.dt_min = d->dt_min;
    p.dt_max = d->dt_max;
    return p;
}

int check_conv_io(const rssm_conv_desc *d, const rssm_conv_io *io) {
    if (!io) return fail(RSSM_E_ARG, "conv: io is NULL");
    if (!io->u || !io->dt_raw || !io->x || !io->B || !io->C || !io->dt)
        return fail(RSSM_E_ARG, "conv: an input/output pointer is NULL");
    if (io->u_pitch < conv_channels(d) || io->dt_pitch < d->n_heads)
        return fail(RSSM_E_ARG, "conv: u_pitch / dt_pitch shorter than a token's row");
    return RSSM_OK;
}

void set_conv_io(rssm::ConvParams &p, const rssm_conv_io *io) {
    p.u = io->u;
    p.dtr = io->dt_raw;
    p.u_pitch = io->u_pitch;
    p.dt_pitch = io->dt_pitch;
    p.x = io->x;
    p.B = io->B;
    p.C = io->C;
    p.dt = io->dt;
}

int conv_tokens(const rssm_conv_desc *desc, const rssm_conv_state *st, int32_t T, bool advance,
                const rssm_conv_io *io, hipStream_t stream) {
    RSSM_TRY(check_conv_desc(desc));
    if (T < 1 || T > desc->max_draft)
        return fail(RSSM_E_CAPACITY, "conv: T = %d outside 1..max_draft (%d)", T, desc->max_draft);
    if (desc->batch == 0) return RSSM_OK;
    RSSM_TRY(check_conv_state(desc, st));
    RSSM_TRY(check_conv_io(desc, io));
    RSSM_TRY(check_threads("conv", desc->batch * rssm::conv_channel_blocks(conv_channels(desc)) * rssm::kConvThreads));
    rssm::ConvParams p = conv_params(desc, st);
    set_conv_io(p, io);
    p.T = T;
    return hip_status(rssm::launch_conv_tokens(p, desc->in_dtype == RSSM_BF16, desc->width, advance, stream),
                      "conv token launch");
}

bool float_type(int32_t t) { return t == RSSM_F32 || t == RSSM_BF16; }

int check_unit(const char *what, int64_t rows, int32_t dim, int32_t groups, float eps) {
    if (rows < 0 || rows > (int64_t)1 << 26) return fail(RSSM_E_ARG, "%s: rows outside 0..2^26", what);
    if (dim < 1 || groups < 1 || dim % groups != 0)
        return fail(RSSM_E_ARG, "%s: dim %d must be a positive multiple of groups %d", what, dim, groups);
    if (dim / groups > kMaxUnit)
        return fail(RSSM_E_CAPACITY, "%s: %d elements per norm exceed %d", what, dim / groups, kMaxUnit);
    if (rows * groups > 0x7FFFFFFF) return fail(RSSM_E_ARG, "%s: rows * groups too large", what);
    if (!(eps >= 0.f) || std::isinf(eps)) return fail(RSSM_E_ARG, "%s: eps must be finite and >= 0", what);
    return RSSM_OK;
}

// Packed prompts run on the matrix cores where the state is fp32 on both sides of the call.
bool on_matrix_cores(const rssm_desc *d) { return split_mode(d) < 0; }

}  // namespace

extern "C" {

int replayssm_conv_check_desc(const rssm_conv_desc *desc) {
    clear_error();
    return check_conv_desc(desc);
}

int32_t replayssm_conv_ring_rows(const rssm_conv_desc *desc) {
    return check_conv_desc(desc) == RSSM_OK ? conv_rows(desc) : 0;
}

int replayssm_conv_step(const rssm_conv_desc *desc, const rssm_conv_state *st, const rssm_conv_io *io,
                        hipStream_t stream) {
    return conv_tokens(desc, st, 1, true, io, stream);
}

int replayssm_conv_verify(const rssm_conv_desc *desc, const rssm_conv_state *st, int32_t T,
                          const rssm_conv_io *io, hipStream_t stream) {
    return conv_tokens(desc, st, T, false, io, stream);
}

int replayssm_conv_accept(const rssm_conv_desc *desc, const rssm_conv_state *st, const int32_t *n_keep,
                          int32_t T, hipStream_t stream) {
    RSSM_TRY(check_conv_desc(desc));
    if (T < 1 || T > desc->max_draft)
        return fail(RSSM_E_CAPACITY, "conv accept: T = %d outside 1..max_draft (%d)", T, desc->max_draft);
    if (desc->batch == 0) return RSSM_OK;
    RSSM_TRY(check_conv_state(desc, st));
    if (!n_keep) return fail(RSSM_E_ARG, "conv accept: n_keep is NULL");
    rssm::ConvParams p = conv_params(desc, st);
    p.n_keep = n_keep;
    p.T = T;
    return hip_status(rssm::launch_conv_accept(p, stream), "conv accept launch");
}

int replayssm_conv_prefill(const rssm_conv_desc *desc, const rssm_conv_state *st, int64_t total,
                           const int32_t *cu_seqlens, int32_t from_zero, const int32_t *fresh,
                           const rssm_conv_io *io, hipStream_t stream) {
    RSSM_TRY(check_conv_desc(desc));
    if (total < 0 || total > (int64_t)1 << 30) return fail(RSSM_E_ARG, "conv prefill: total outside 0..2^30");
    if (from_zero != 0 && from_zero != 1) return fail(RSSM_E_ARG, "conv prefill: from_zero must be 0 or 1");
    if (desc->batch == 0 || total == 0) return RSSM_OK;
    RSSM_TRY(check_conv_state(desc, st));
    if (!cu_seqlens) return fail(RSSM_E_ARG, "conv prefill: cu_seqlens is NULL");
    RSSM_TRY(check_conv_io(desc, io));
    const int64_t nblk = rssm::conv_channel_blocks(conv_channels(desc)), tile = rssm::conv_tile(total, nblk);
    RSSM_TRY(check_threads("conv prefill", (total + tile - 1) / tile * nblk * rssm::kConvThreads));
    rssm::ConvParams p = conv_params(desc, st);
    set_conv_io(p, io);
    p.cu = cu_seqlens;
    p.fresh = fresh;
    p.from_zero = from_zero;
    p.total = total;
    return hip_status(rssm::launch_conv_packed(p, desc->in_dtype == RSSM_BF16, desc->width, stream),
                      "conv prefill launch");
}

size_t replayssm_prefill_packed_workspace(const rssm_desc *desc, int64_t total) {
    if (check_desc(desc) != RSSM_OK || total < 0 || total > (int64_t)1 << 30 || !on_matrix_cores(desc)) return 0;
    return rssm::scan_workspace(total, desc->batch, desc->n_heads, desc->n_groups, desc->in_dtype == RSSM_BF16);
}

int replayssm_prefill_packed(const rssm_desc *desc, const rssm_state *st, int64_t total,
                             const int32_t *cu_seqlens, int32_t from_zero, const int32_t *fresh,
                             const void *x, const void *B, const void *C, const void *dt, void *y,
                             int32_t y_dtype, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    RSSM_TRY(check_desc(desc));
    if (total < 0 || total > (int64_t)1 << 30 || total * desc->n_heads > (int64_t)1 << 31)
        return fail(RSSM_E_ARG, "prefill_packed: total outside 0..2^30, or total * n_heads over 2^31");
    if (desc->n_heads > 1 << 15)   // a chunk's rows are addressed in 31 bits
        return fail(RSSM_E_CAPACITY, "prefill_packed: %d heads exceed 32768", desc->n_heads);
    if (from_zero != 0 && from_zero != 1) return fail(RSSM_E_ARG, "prefill_packed: from_zero must be 0 or 1");
    if (y && !float_type(y_dtype)) return fail(RSSM_E_UNSUPPORTED, "prefill_packed: y_dtype %d: F32 or BF16", y_dtype);
    RSSM_TRY(check_state(desc, st));
    if (desc->batch == 0 || total == 0) return RSSM_OK;
    if (!cu_seqlens) return fail(RSSM_E_ARG, "prefill_packed: cu_seqlens is NULL");
    if (!x || !B || !dt) return fail(RSSM_E_ARG, "prefill_packed: x / B / dt is NULL");
    if (y && !C) return fail(RSSM_E_ARG, "prefill_packed: outputs need C");
    if (workspace && workspace_bytes < replayssm_prefill_packed_workspace(desc, total))
        return fail(RSSM_E_ARG, "prefill_packed: a workspace of %zu bytes is smaller than "
                    "replayssm_prefill_packed_workspace", workspace_bytes);
    rssm::ReplayParams p = replay_params(desc, st);
    p.x = x;
    p.Bm = B;
    p.Cm = C;
    p.dt = dt;
    p.y = static_cast<float *>(y);
    p.y_bf16 = y_dtype == RSSM_BF16;
    p.from_zero = from_zero;
    p.cu = cu_seqlens;
    p.fresh = fresh;
    p.total = total;
    if (on_matrix_cores(desc))
        return hip_status(rssm::launch_scan(p, desc->in_dtype == RSSM_BF16, y != nullptr, workspace, stream), "packed prefill launch");
    return hip_status(rssm::launch_prefill_packed(p, desc->in_dtype == RSSM_BF16, y != nullptr, split_mode(desc),
                                                  stream),
                      "packed prefill launch");
}

int replayssm_gated_norm(int64_t rows, int32_t dim, int32_t groups, const void *y, int32_t y_dtype,
                         const void *z, int32_t z_dtype, int64_t z_pitch, const float *weight, float eps,
                         int32_t norm_before_gate, void *out, int32_t out_dtype, hipStream_t stream) {
    RSSM_TRY(check_unit("gated_norm", rows, dim, groups, eps));
    if (!float_type(y_dtype) || !float_type(z_dtype) || !float_type(out_dtype))
        return fail(RSSM_E_UNSUPPORTED, "gated_norm: y, z and out are F32 or BF16");
    if (norm_before_gate != 0 && norm_before_gate != 1)
        return fail(RSSM_E_ARG, "gated_norm: norm_before_gate must be 0 or 1");
    if (rows == 0) return RSSM_OK;
    if (!y || !z || !weight || !out) return fail(RSSM_E_ARG, "gated_norm: a pointer is NULL");
    if (z_pitch < dim) return fail(RSSM_E_ARG, "gated_norm: z_pitch shorter than a row");
    rssm::GatedNormParams p{y, z, out, weight, z_pitch, rows, dim, groups, eps, norm_before_gate};
    return hip_status(rssm::launch_gated_norm(p, y_dtype == RSSM_BF16, z_dtype == RSSM_BF16, out_dtype == RSSM_BF16,
                                              stream),
                      "gated norm launch");
}

int replayssm_add_norm(int64_t rows, int32_t dim, const void *x, int32_t x_dtype, const void *residual,
                       void *residual_out, int32_t res_dtype, const float *weight, const float *post_weight,
                       float scale, float eps, void *out, int32_t out_dtype, hipStream_t stream) {
    RSSM_TRY(check_unit("add_norm", rows, dim, 1, eps));
    if (!float_type(x_dtype) || !float_type(res_dtype) || !float_type(out_dtype))
        return fail(RSSM_E_UNSUPPORTED, "add_norm: x, residual and out are F32 or BF16");
    if (rows == 0) return RSSM_OK;
    if (!x || !residual || !residual_out || !weight || !out) return fail(RSSM_E_ARG, "add_norm: a pointer is NULL");
    rssm::AddNormParams p{x, residual, residual_out, out, weight, post_weight, rows, dim, scale, eps};
    return hip_status(rssm::launch_add_norm(p, x_dtype == RSSM_BF16, res_dtype == RSSM_BF16, out_dtype == RSSM_BF16,
                                            stream),
                      "add norm launch");
}

}  // extern "C"
