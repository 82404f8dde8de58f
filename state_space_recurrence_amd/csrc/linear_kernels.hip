// linear_kernels.hip -- out = residual + scale act(x w^T + bias), x [rows, K]
// and w [N, K] in bf16 or in MX (E4M3 codes, a power of two per 32 elements).
//
// The weights are the matrix instruction's first operand, so an accumulator
// holds 4 consecutive outputs of one row per lane: stores and the residual's
// loads are wide, and a 32 x 32 tile's column of outputs, half in a lane and
// half in lane ^ 32, is one block of an MX output.
//
// A step is 128 bytes of K of every row: 64 bf16 elements (four 32x32x16
// products per 32 x 32 tile) or 128 codes (two scaled 32x32x64 products).  Lane
// l of an operand holds row l % 32; its 16-byte chunk s of a step is chunk
// 2 s + l / 32 of the row's 8 for both types: one MX product takes two of them,
// and its scale is byte 2 t + l / 32 of the row's four of the step (t the
// product).  In LDS chunk c of row r lies at place c ^ (r & 7), so that the 8
// lanes that read at a time touch all banks.
//
// Sums are fp32.  A product of a zero code with a NaN is NaN as elsewhere.
#include "linear.h"

#include "mixer_device.h"
#include "mx.h"
#include "replayssm.h"

namespace rssm {
namespace {

typedef float f16v __attribute__((ext_vector_type(16)));
typedef int i8v __attribute__((ext_vector_type(8)));
typedef uint32_t u2u __attribute__((ext_vector_type(2), aligned(2)));

constexpr int kStep = 128;   // bytes of K per step

// ---------------------------------------------------------------- epilogue --

// v Phi(v), Phi the normal distribution: erfc from Abramowitz and Stegun 7.1.26
// (off by at most 1.5e-7), taken of |v| / sqrt 2 so that nothing cancels below 0.
__device__ __forceinline__ float gelu(float v) {
    const float z = fabsf(v) * 0.70710678f, t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, z, 1.f));
    float c = fmaf(1.061405429f, t, -1.453152027f);
    c = fmaf(c, t, 1.421413741f);
    c = fmaf(c, t, -0.284496736f);
    c = fmaf(c, t, 0.254829592f);
    c = 0.5f * (c * t) * __expf(-z * z);
    return v < 0.f ? v * c : v * (1.f - c);
}

__device__ __forceinline__ float activate(int act, float v) {
    if (act == 1) return silu(v);
    if (act == 2) return gelu(v);
    if (act == 3) return v < 0.f ? 0.f : v * v;   // (a NaN stays one)
    return v;
}

// Four consecutive outputs n .. n + 3 of row m from their sums; `left` of them
// are inside the row (whole: left >= 4).
__device__ __forceinline__ f4v outputs4(const LinearParams &p, int64_t m, int n, f4v v) {
    const int left = p.n_out - n;
    if (p.bias) {
        if (left >= 4) v += *reinterpret_cast<const f4u *>(p.bias + n);
        else
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (i < left) v[i] += p.bias[n + i];
    }
    if (p.act)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = activate(p.act, v[i]);
    if (!p.res) return p.scale * v;
    f4v r = (f4v)0.f;
    const int64_t at = m * p.n_out + n;
    if (p.res_bf16) {
        const uint16_t *s = static_cast<const uint16_t *>(p.res) + at;
        if (left >= 4) {
            const u2u b = *reinterpret_cast<const u2u *>(s);
            r = f4v{__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xFFFF0000u), __uint_as_float(b.y << 16),
                    __uint_as_float(b.y & 0xFFFF0000u)};
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (i < left) r[i] = vec8<uint16_t>::get(s + i);
        }
    } else {
        const float *s = static_cast<const float *>(p.res) + at;
        if (left >= 4) r = *reinterpret_cast<const f4u *>(s);
        else
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (i < left) r[i] = s[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fmaf(p.scale, v[i], r[i]);
    return v;
}

__device__ __forceinline__ void store4(const LinearParams &p, int64_t m, int n, f4v v) {
    const int left = p.n_out - n;
    const int64_t at = m * p.n_out + n;
    if (p.out_type == RSSM_BF16) {
        uint16_t *o = static_cast<uint16_t *>(p.out) + at;
        if (left >= 4) {
            typedef __bf16 b4v __attribute__((ext_vector_type(4)));
            typedef uint32_t u2v __attribute__((ext_vector_type(2)));
            *reinterpret_cast<u2u *>(o) = __builtin_bit_cast(u2v, __builtin_convertvector(v, b4v));
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (i < left) vec8<uint16_t>::put(o + i, v[i]);
        }
    } else {
        float *o = static_cast<float *>(p.out) + at;
        if (left >= 4) *reinterpret_cast<f4u *>(o) = v;
        else
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (i < left) o[i] = v[i];
    }
}

// A wave's 32 x 32 tile of sums: outputs n0 .. n0 + 31 (some of them in the
// row) of rows m0 .. m0 + 31 (the lane's row may lie behind the last).
__device__ __forceinline__ void finish(const LinearParams &p, int64_t m0, int n0, const f16v &acc, int lane) {
    const int64_t m = m0 + (lane & 31);
    const int n = n0 + 4 * (lane >> 5);
    const bool mine = m < p.rows;
    if (p.out_type == RSSM_FP8_E4M3) {   // n_out is a multiple of 32: the block is whole
        f4v v[4];
        uint32_t a = 0;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            v[g] = (f4v)0.f;
            if (mine) v[g] = outputs4(p, m, n + 8 * g, f4v{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]});
#pragma unroll
            for (int i = 0; i < 4; ++i) a = max(a, mx_size(v[g][i]));
        }
        a = max(a, (uint32_t)__shfl_xor((int)a, 32));
        const uint32_t s = mx_scale(a);
        const float inv = mx_inverse(s);
        if (!mine) return;
        uint8_t *o = static_cast<uint8_t *>(p.out) + m * p.n_out + n;
#pragma unroll
        for (int g = 0; g < 4; ++g)
            *reinterpret_cast<uint32_t *>(o + 8 * g) = mx_codes(v[g][0], v[g][1], v[g][2], v[g][3], inv);
        if (lane < 32) p.out_scales[m * (p.n_out / kMxBlock) + n0 / kMxBlock] = (uint8_t)s;
        return;
    }
    if (!mine) return;
#pragma unroll
    for (int g = 0; g < 4; ++g)
        if (n + 8 * g < p.n_out)
            store4(p, m, n + 8 * g,
                   outputs4(p, m, n + 8 * g, f4v{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]}));
}

// ---------------------------------------------------------------- products --

// A lane's operand of 32 rows for one step: chunks 2 s + l / 32, and (MX) the
// row's four scales; chunk 2 s + h lies in block s.
struct operand {
    u4v c[4];
    uint32_t scales;
};

// Half of a chunk of codes as 8 bf16 numbers with their scale (E8M0 as the
// exponent of an fp32 number): exact, E4M3 has 4 significant bits.
__device__ __forceinline__ b8v widen_codes(const u4v &c, int half, uint32_t scale) {
    const float f = __uint_as_float(scale << 23);
    const uint32_t lo = c[2 * half], hi = c[2 * half + 1];
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, true);
    const auto d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, false), e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, true);
    return b8v{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

template <bool MX>
__device__ __forceinline__ void multiply(f16v &acc, const operand &w, const operand &x) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        if constexpr (MX) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_codes(w.c[s], half, (w.scales >> (8 * s)) & 0xFFu),
                                                              widen_codes(x.c[s], half, (x.scales >> (8 * s)) & 0xFFu),
                                                              acc, 0, 0, 0);
        } else {
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8v, w.c[s]), __builtin_bit_cast(b8v, x.c[s]),
                                                          acc, 0, 0, 0);
        }
    }
}

// Rows 0..31 of `tile` (LDS, at a multiple of 8 rows) as an operand.
template <bool MX>
__device__ __forceinline__ operand read_operand(const char *tile, const uint32_t *scales, int lane) {
    operand o;
    const int r = lane & 31, h = lane >> 5;
    const char *p = tile + r * kStep;
#pragma unroll
    for (int s = 0; s < 4; ++s) o.c[s] = *reinterpret_cast<const u4v *>(p + (((2 * s + h) ^ (r & 7)) << 4));
    o.scales = MX ? scales[r] : 0;
    return o;
}

// ----------------------------------------------------- rows of any alignment --

// Tiles of 64 outputs x 64 rows, staged through registers: a row may start at
// any element and end at any.  Four waves of 32 x 32.
template <bool MX>
__global__ void __launch_bounds__(256) linear_any_kernel(LinearParams p) {
    constexpr int B = 64;
    __shared__ __attribute__((aligned(16))) char tile[2][2 * B * kStep];   // w's rows, then x's
    __shared__ uint32_t scales[2][2 * B];
    const int tiles_n = (p.n_out + B - 1) / B;
    const int64_t bm = blockIdx.x / tiles_n;
    const int n0 = (int)(blockIdx.x - bm * tiles_n) * B;
    const int64_t m0 = bm * B;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

    // Thread t stages chunk t % 8 of rows t / 8 + 32 i of the 128, and the scales of row t (t < 128).
    const auto row = [&](int r, bool scale) -> const char * {   // rows behind the last are the last again
        if (r < B) {
            const int64_t n = min(n0 + r, p.n_out - 1);
            return scale ? reinterpret_cast<const char *>(p.w_scales) + n * (p.k_bytes / kMxBlock)
                         : static_cast<const char *>(p.w) + n * p.w_pitch;
        }
        const int64_t m = min(m0 + r - B, p.rows - 1);
        return scale ? reinterpret_cast<const char *>(p.x_scales) + m * (p.k_bytes / kMxBlock)
                     : static_cast<const char *>(p.x) + m * p.x_pitch;
    };
    u4v c[4];
    uint32_t sc = 0;
    const auto load = [&](int k) {
        const int at = k * kStep + (threadIdx.x & 7) * 16, left = p.k_bytes - at;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const char *s = row((threadIdx.x >> 3) + 32 * i, false) + at;
            c[i] = (u4v)0u;
            if (left >= 16) {
                c[i] = *reinterpret_cast<const u4u *>(s);
            } else {   // (bf16 alone: MX rows are whole chunks)
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (2 * e < left) c[i][e >> 1] |= (uint32_t) * reinterpret_cast<const uint16_t *>(s + 2 * e) << (16 * (e & 1));
            }
        }
        if constexpr (MX) {
            if (threadIdx.x < 2 * B) {
                const uint8_t *s = reinterpret_cast<const uint8_t *>(row(threadIdx.x, true)) + 4 * k;
                const int n = p.k_bytes / kMxBlock - 4 * k;
                sc = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < n) sc |= (uint32_t)s[i] << (8 * i);
            }
        }
    };
    const auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (threadIdx.x >> 3) + 32 * i;
            *reinterpret_cast<u4v *>(&tile[buf][r * kStep + (((threadIdx.x & 7) ^ (r & 7)) << 4)]) = c[i];
        }
        if (MX && threadIdx.x < 2 * B) scales[buf][threadIdx.x] = sc;
    };

    f16v acc = (f16v)0.f;
    const int wn = 32 * (wave & 1), wm = B + 32 * (wave >> 1);
    const int steps = (p.k_bytes + kStep - 1) / kStep;
    load(0);
    put(0);
    for (int k = 0; k < steps; ++k) {
        if (k + 1 < steps) load(k + 1);
        __syncthreads();
        const operand w = read_operand<MX>(&tile[k & 1][wn * kStep], &scales[k & 1][wn], lane);
        const operand x = read_operand<MX>(&tile[k & 1][wm * kStep], &scales[k & 1][wm], lane);
        multiply<MX>(acc, w, x);
        if (k + 1 < steps) put((k + 1) & 1);
    }
    if (n0 + wn < p.n_out) finish(p, m0 + wm - B, n0 + wn, acc, lane);
}

}  // namespace

hipError_t launch_linear(const LinearParams &p, bool mx, hipStream_t s) {
    const int64_t tiles = ((p.rows + 63) / 64) * ((p.n_out + 63) / 64);
    if (mx) hipLaunchKernelGGL(linear_any_kernel<true>, dim3((unsigned)tiles), dim3(256), 0, s, p);
    else hipLaunchKernelGGL(linear_any_kernel<false>, dim3((unsigned)tiles), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace rssm
