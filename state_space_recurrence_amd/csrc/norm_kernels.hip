// norm_kernels.hip -- norms behind the recurrence and around the block.
//
// Gated norm, per group of dim / groups elements of a row:
//     v = y z sigmoid(z),  out = v rsqrt(mean(v^2) + eps) w
// or, with the norm before the gate, out = y rsqrt(mean(y^2) + eps) w z sigmoid(z).
//
// Add norm, per row:
//     r = res + scale f(x),  f(x) = x or x rsqrt(mean(x^2) + eps) post
//     res_out = r,  out = r rsqrt(mean(r^2) + eps) w
// with the norm taken of the fp32 sum r, before r is rounded for res_out.
//
// Both are one pass over memory: a unit (a group, a row) is held in registers
// between its sum of squares and its scaling, eight elements a lane and step.
// Sums are fp32 in a fixed order; outputs are rounded once.
//
// Bound by memory.  Gated norm, 16384 rows of 6144 elements in 8 groups, bf16:
// 123 us (604 MB, 4.9 TB/s); half a wave per group of 768 takes 123 us where a
// wave of 64 took 131 and two waves 139, and one persistent workgroup per
// compute unit that walks the rows 160 or more.  Add norm, 16384 rows of 4096,
// bf16: 102 us (537 MB, 5.3 TB/s).  Single rows are bound by the launch: 256
// rows of 6144 take 4.6 us, one row of 4096 2.5 to 3.3.  MX outputs: the gated
// norm 118 us (507 MB, 4.3 TB/s), add norm with an fp32 residual 135 us (740 MB,
// 5.5 TB/s).  Loads and stores past the caches would gain the former 4 %, but
// the product behind reads the codes from there.
#include "mixer.h"
#include "mixer_device.h"
#include "mx.h"

#include <type_traits>

namespace rssm {
namespace {

// A launch may have 2^32 - 1 threads along an axis: more workgroups than 2^20
// (2^30 threads) go over two axes.
constexpr unsigned kGridX = 1u << 20;

inline dim3 grid_of(int64_t blocks) {
    if (blocks <= kGridX) return dim3((unsigned)blocks);
    return dim3(kGridX, (unsigned)((blocks + kGridX - 1) / kGridX));
}

__device__ __forceinline__ int64_t block_index() { return (int64_t)blockIdx.y * kGridX + blockIdx.x; }

// Sum over the THREADS lanes that share a unit (32, 64, or a workgroup).
template <int THREADS>
__device__ __forceinline__ float unit_sum(float v, float *lds) {
    v = row16_sum(v);
    v += __shfl_xor(v, 16);
    if constexpr (THREADS == 32) return v;
    v += __shfl_xor(v, 32);
    if constexpr (THREADS > 64) {
        __syncthreads();   // an earlier sum's reads are done
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < THREADS / 64; ++i) v += lds[i];
    }
    return v;
}

template <int NV>
__device__ __forceinline__ float squares(const f8v (&v)[NV]) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(v[k][i], v[k][i], s);
    return s;
}

// Outputs of a lane's eight elements at column c of row `row`: as numbers, or
// (type mx8) as codes with the scale of the 32 elements that four neighbouring
// lanes hold.  Units of MX outputs are whole blocks, so the four lanes store
// together or not at all.
template <bool FULL, typename TO>
__device__ __forceinline__ void store_out(void *out, uint8_t *scales, int64_t row, int dim, int c, const f8v &o, int left) {
    if constexpr (std::is_same<TO, mx8>::value) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, mx_size(o[i]));
        const uint32_t s = mx_scale(quad_max(m));
        const float inv = mx_inverse(s);
        const uint2 q = make_uint2(mx_codes(o[0], o[1], o[2], o[3], inv), mx_codes(o[4], o[5], o[6], o[7], inv));
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(out) + row * dim + c) = q;
        if ((threadIdx.x & 3) == 0) scales[row * (dim / kMxBlock) + c / kMxBlock] = (uint8_t)s;
    } else {
        store_part<FULL>(static_cast<TO *>(out) + row * dim + c, o, left);
    }
}

// THREADS lanes per unit, NV steps of eight elements a lane: units of up to
// 8 THREADS NV elements.  FULL: units are whole steps of eight (no tail code).
// A workgroup of 256 or more holds one unit, or eight of half a wave each.
template <typename TY, typename TZ, typename TO, int THREADS, int NV, bool FULL>
__global__ void __launch_bounds__(THREADS < 256 ? 256 : THREADS) gated_norm_kernel(GatedNormParams p) {
    __shared__ float lds[16];
    constexpr int kUnits = THREADS < 256 ? 256 / THREADS : 1;
    const int gsize = p.dim / p.groups;
    const int64_t unit = block_index() * kUnits + (kUnits > 1 ? threadIdx.x / THREADS : 0);
    if (unit >= p.rows * p.groups) return;   // all lanes of the unit
    const int64_t row = unit / p.groups;
    const int c0 = (int)(unit - row * p.groups) * gsize;
    const int lane = kUnits > 1 ? threadIdx.x % THREADS : threadIdx.x;
    const TY *y = reinterpret_cast<const TY *>(p.y) + row * p.dim + c0;
    const TZ *z = reinterpret_cast<const TZ *>(p.z) + row * p.z_pitch + c0;
    f8v v[NV], g[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * THREADS + lane) * 8;
        v[k] = load_part<FULL>(y + c, gsize - c);
        g[k] = load_part<FULL>(z + c, gsize - c);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[k][i] = silu(g[k][i]);
            if (!p.before) v[k][i] *= g[k][i];
        }
    const float r = rsqrtf(unit_sum<THREADS>(squares(v), lds) / gsize + p.eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * THREADS + lane) * 8;
        if (c < gsize) {
            f8v o = load_part<FULL>(p.w + c0 + c, gsize - c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i] = v[k][i] * r * o[i];
                if (p.before) o[i] *= g[k][i];
            }
            store_out<FULL, TO>(p.out, p.out_scales, row, p.dim, c0 + c, o, gsize - c);
        }
    }
}

template <typename TX, typename TR, typename TO, int THREADS, int NV, bool FULL>
__global__ void __launch_bounds__(THREADS < 256 ? 256 : THREADS) add_norm_kernel(AddNormParams p) {
    __shared__ float lds[16];
    constexpr int kUnits = THREADS < 256 ? 256 / THREADS : 1;
    const int64_t row = block_index() * kUnits + (kUnits > 1 ? threadIdx.x / THREADS : 0);
    if (row >= p.rows) return;   // all lanes of the unit
    const int lane = kUnits > 1 ? threadIdx.x % THREADS : threadIdx.x;
    const TX *x = reinterpret_cast<const TX *>(p.x) + row * p.dim;
    const TR *res = reinterpret_cast<const TR *>(p.res) + row * p.dim;
    TR *res_out = reinterpret_cast<TR *>(p.res_out) + row * p.dim;
    f8v v[NV], r[NV];
    const bool add = !std::is_same<TO, mx8>::value || p.x;   // without x, the norm alone
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * THREADS + lane) * 8;
        if (add) v[k] = load_part<FULL>(x + c, p.dim - c);
        r[k] = load_part<FULL>(res + c, p.dim - c);
    }
    if (p.post) {
        const float n = rsqrtf(unit_sum<THREADS>(squares(v), lds) / p.dim + p.eps);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * THREADS + lane) * 8;
            const f8v w = load_part<FULL>(p.post + c, p.dim - c);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = v[k][i] * n * w[i];
        }
    }
    if (add) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) r[k][i] = fmaf(p.scale, v[k][i], r[k][i]);
    }
    const float n = rsqrtf(unit_sum<THREADS>(squares(r), lds) / p.dim + p.eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * THREADS + lane) * 8;
        if (c < p.dim) {
            if (add) store_part<FULL>(res_out + c, r[k], p.dim - c);
            const f8v w = load_part<FULL>(p.w + c, p.dim - c);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = r[k][i] * n * w[i];
            store_out<FULL, TO>(p.out, p.out_scales, row, p.dim, c, v[k], p.dim - c);
        }
    }
}

// Rows to MX: eight elements a thread, blocks of four lanes.  Bound by memory:
// 14432 rows of 4096 bf16 elements take 34 us (179 MB, 5.3 TB/s).
template <typename TX>
__global__ void __launch_bounds__(256) quantize_kernel(QuantizeParams p) {
    const int64_t at = block_index() * 256 + threadIdx.x;
    const int per = p.dim / 8;
    if (at >= p.rows * per) return;   // all lanes of a block
    const int64_t row = at / per;
    const int c = (int)(at - row * per) * 8;
    const TX *x = reinterpret_cast<const TX *>(p.x) + row * p.x_pitch + c;
    store_out<true, mx8>(p.out, p.out_scales, row, p.dim, c, vec8<TX>::widen(vec8<TX>::load(x)), 8);
}

template <int TH, int NV, typename F>
hipError_t by_tail(int n, F &&f) {
    if (n % 8 == 0) f(std::integral_constant<int, TH>{}, std::integral_constant<int, NV>{}, std::true_type{});
    else f(std::integral_constant<int, TH>{}, std::integral_constant<int, NV>{}, std::false_type{});
    return hipGetLastError();
}

// MX outputs are whole blocks: no tail code is built for them.
template <int TH, int NV, typename TO, typename F>
hipError_t by_output(int n, F &&f) {
    if constexpr (std::is_same<TO, mx8>::value) {
        f(std::integral_constant<int, TH>{}, std::integral_constant<int, NV>{}, std::true_type{});
        return hipGetLastError();
    } else {
        return by_tail<TH, NV>(n, f);
    }
}

// Lanes of a unit of n elements and steps of eight elements a lane.
template <typename TO, typename F>
hipError_t by_size(int n, F &&f) {
    if (n <= 256) return by_output<32, 1, TO>(n, f);
    if (n <= 512) return by_output<32, 2, TO>(n, f);
    if (n <= 768) return by_output<32, 3, TO>(n, f);
    if (n <= 1024) return by_output<32, 4, TO>(n, f);
    if (n <= 2048) return by_output<256, 1, TO>(n, f);
    if (n <= 4096) return by_output<256, 2, TO>(n, f);
    if (n <= 8192) return by_output<1024, 1, TO>(n, f);
    if (n <= 16384) return by_output<1024, 2, TO>(n, f);
    return hipErrorInvalidValue;
}

template <int TH>
constexpr int kThreadsOf = TH < 256 ? 256 : TH;
template <int TH>
constexpr int kUnitsOf = TH < 256 ? 256 / TH : 1;

template <typename TY, typename TZ, typename TO>
hipError_t gated(const GatedNormParams &p, hipStream_t s) {
    return by_size<TO>(p.dim / p.groups, [&](auto th, auto nv, auto full) {
        constexpr int TH = decltype(th)::value, NV = decltype(nv)::value;
        const int64_t units = p.rows * p.groups;
        const dim3 grid = grid_of((units + kUnitsOf<TH> - 1) / kUnitsOf<TH>), block(kThreadsOf<TH>);
        hipLaunchKernelGGL((gated_norm_kernel<TY, TZ, TO, TH, NV, decltype(full)::value>), grid, block, 0, s, p);
    });
}

template <typename TX, typename TR, typename TO>
hipError_t added(const AddNormParams &p, hipStream_t s) {
    return by_size<TO>(p.dim, [&](auto th, auto nv, auto full) {
        constexpr int TH = decltype(th)::value, NV = decltype(nv)::value;
        const dim3 grid = grid_of((p.rows + kUnitsOf<TH> - 1) / kUnitsOf<TH>), block(kThreadsOf<TH>);
        hipLaunchKernelGGL((add_norm_kernel<TX, TR, TO, TH, NV, decltype(full)::value>), grid, block, 0, s, p);
    });
}

}  // namespace

// The middle type pairs with the first or third as serving uses them; every
// combination is built.
#define RSSM_BY_TYPES(F)                                                          \
    switch ((a ? 4 : 0) | (b ? 2 : 0) | (c ? 1 : 0)) {                            \
        case 0: return F<float, float, float>(p, s);                              \
        case 1: return F<float, float, uint16_t>(p, s);                           \
        case 2: return F<float, uint16_t, float>(p, s);                           \
        case 3: return F<float, uint16_t, uint16_t>(p, s);                        \
        case 4: return F<uint16_t, float, float>(p, s);                           \
        case 5: return F<uint16_t, float, uint16_t>(p, s);                        \
        case 6: return F<uint16_t, uint16_t, float>(p, s);                        \
        default: return F<uint16_t, uint16_t, uint16_t>(p, s);                    \
    }

hipError_t launch_gated_norm(const GatedNormParams &p, bool a, bool b, bool c, hipStream_t s) {
    RSSM_BY_TYPES(gated)
}

hipError_t launch_add_norm(const AddNormParams &p, bool a, bool b, bool c, hipStream_t s) {
    RSSM_BY_TYPES(added)
}

hipError_t launch_gated_norm_mx(const GatedNormParams &p, bool y_bf16, bool z_bf16, hipStream_t s) {
    if (y_bf16) return z_bf16 ? gated<uint16_t, uint16_t, mx8>(p, s) : gated<uint16_t, float, mx8>(p, s);
    return z_bf16 ? gated<float, uint16_t, mx8>(p, s) : gated<float, float, mx8>(p, s);
}

hipError_t launch_add_norm_mx(const AddNormParams &p, bool x_bf16, bool res_bf16, hipStream_t s) {
    if (x_bf16) return res_bf16 ? added<uint16_t, uint16_t, mx8>(p, s) : added<uint16_t, float, mx8>(p, s);
    return res_bf16 ? added<float, uint16_t, mx8>(p, s) : added<float, float, mx8>(p, s);
}

hipError_t launch_quantize(const QuantizeParams &p, bool x_bf16, hipStream_t s) {
    const int64_t threads = p.rows * (p.dim / 8);
    const dim3 grid = grid_of((threads + 255) / 256);
    if (x_bf16) hipLaunchKernelGGL(quantize_kernel<uint16_t>, grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL(quantize_kernel<float>, grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace rssm
