// linear_kernels.hip -- out = residual + scale act(x w^T + bias), x [rows, K]
// and w [N, K] in bf16 or in MX (E4M3 codes, a power of two per 32 elements).
//
// The weights are the matrix instruction's first operand, so an accumulator
// holds 4 consecutive outputs of one row per lane.  A step is 128 bytes of K of
// every row: 64 bf16 elements (four 32x32x16 products per 32 x 32 tile) or 128
// codes.  Lane l of an operand holds row l % 32; its 16-byte chunk s of a step is
// chunk 2 s + l / 32 of the row's 8 for both types.  In LDS chunk c of row r lies
// at place c ^ (r >> 1 & 7): the 16 lanes that read at a time then touch all 64
// banks (with r & 7 half of them: a third of the LDS cycles were conflicts).
//
// MX operands are multiplied in one of two ways; sums are fp32 in both.  Widened
// to bf16, which is exact, their sums are those of bf16 rows.  Scaled 8-bit
// products (two 32x32x64 per tile and step) run at twice the rate, but the matrix
// units cut each product 13 binary places below the largest of those that they
// add at once: sums are off by 2.9e-4 of their norm (256 rows of 14432 outputs, K
// 4096), a sixth of what rounding to bf16 takes (1.7e-3), and where large products
// cancel, what is left of the small ones may be anything below that cut.  So these
// are taken where the caller asks for them, and by the tiles from 64 x 64 on,
// which are the ones that they make faster.
//
// What bounds it (rows of 4096 inputs and 14432 outputs unless said otherwise; MX
// by exact products, by fast ones in parentheses):
//   - one row: the weights' bytes in bf16, 23 us for 118 MB, 5.1 TB/s.  In MX 20 us
//     (14) for 61 MB: a SIMD has one wave, which reads, widens and multiplies a
//     step after the other.
//   - tens of rows: 64 take 26 us in bf16, 20 in MX (15), for the same reasons.
//   - hundreds: 256 rows 46 us in bf16, 39 in MX (25).  In bf16 loads in flight: a
//     compute unit has about 120 of its L1's requests (128 bytes) on their way at
//     any time.  In MX the widening: the vector units issue in half of the cycles,
//     the matrix units work in 40 %, and a wave does one after the other.
//   - thousands: the matrix units, at the clock that their work leaves.  8192^3
//     takes 881 us (1.25 PFLOP/s) in bf16 and 769 (482) in MX, the matrix units busy
//     71 %, 80 % (57 %) of the cycles at 1.7, 1.8 (2.0) GHz.  That is no bound yet: a
//     library's bf16 product takes 691 us.  Tiles that stay with a workgroup, the next
//     one's loads behind the stores of the last, measured the same and were dropped.
#include "linear.h"

#include "mixer_device.h"
#include "mx.h"
#include "replayssm.h"

namespace rssm {
namespace {

typedef float f16v __attribute__((ext_vector_type(16)));
typedef int i8v __attribute__((ext_vector_type(8)));

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

// Eight consecutive outputs n .. n + 7 of row m from their sums, some of them
// in the row (`left`, 1 or more); four neighbouring lanes hold 32 outputs.
__device__ __forceinline__ void put8(const LinearParams &p, int64_t m, int n, int left, f8v v, const f8v &bias) {
    const int64_t at = m * p.n_out + n;
    f8v r = (f8v)0.f;
    if (p.res) {
        if (p.res_bf16) r = load_part<false>(static_cast<const uint16_t *>(p.res) + at, left);
        else r = load_part<false>(static_cast<const float *>(p.res) + at, left);
    }
    v += bias;
    if (p.act)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = activate(p.act, v[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(p.scale, v[i], r[i]);
    if (p.out_type == RSSM_FP8_E4M3) {   // n_out is a multiple of 32: the block is whole
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) a = max(a, mx_size(v[i]));
        a = quad_max(a);
        const uint32_t s = mx_scale(a);
        const float inv = mx_inverse(s);
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.out) + at) =
            make_uint2(mx_codes(v[0], v[1], v[2], v[3], inv), mx_codes(v[4], v[5], v[6], v[7], inv));
        if ((threadIdx.x & 3) == 0) p.out_scales[at / kMxBlock] = (uint8_t)s;
    } else if (p.out_type == RSSM_BF16) {
        store_part<false>(static_cast<uint16_t *>(p.out) + at, v, left);
    } else {
        store_part<false>(static_cast<float *>(p.out) + at, v, left);
    }
}

// What the wave's lanes stored to LDS before can be read by its other lanes
// behind, and what they read before can be overwritten.  Every lane gets here.
__device__ __forceinline__ void wave_exchange() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A wave's sums of 32 TN outputs (from n0, some of them in the row) x 32 rows
// (from m0, some of them there), through 4 TN KB of LDS of its own so that a row
// is stored (and its residual loaded) in one piece.  16 bytes c of row r lie at
// place c ^ (r & 7).
template <int TN>
__device__ __forceinline__ void finish(const LinearParams &p, int64_t m0, int n0, const f16v (&acc)[TN], char *lds, int lane) {
    constexpr int kPitch = 128 * TN, kAcross = 4 * TN;   // bytes and lanes of a row
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            *reinterpret_cast<f4v *>(lds + r * kPitch + (((8 * i + 2 * g + h) ^ (r & 7)) << 4)) =
                f4v{acc[i][4 * g], acc[i][4 * g + 1], acc[i][4 * g + 2], acc[i][4 * g + 3]};
    wave_exchange();
    const int c = lane % kAcross, n = n0 + 8 * c, left = p.n_out - n;   // (1 or more for all four lanes of a block, or none)
    f8v bias = (f8v)0.f;
    if (p.bias) bias = load_part<false>(p.bias + n, left);
#pragma unroll 1
    for (int row = lane / kAcross; row < 32; row += 64 / kAcross)
        if (left > 0 && m0 + row < p.rows) {
            const f4v a = *reinterpret_cast<const f4v *>(lds + row * kPitch + (((2 * c) ^ (row & 7)) << 4));
            const f4v b = *reinterpret_cast<const f4v *>(lds + row * kPitch + (((2 * c + 1) ^ (row & 7)) << 4));
            put8(p, m0 + row, n, left, f8v{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, bias);
        }
    wave_exchange();
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

// How operands are multiplied.
enum Product {
    BF16,       // bf16 rows
    MX_EXACT,   // MX rows, widened to bf16: products and sums as for bf16 rows
    MX_FAST     // MX rows, scaled 8-bit products at twice the rate (few rows: as MX_EXACT)
};

// One step of a wave's TM x TN tiles of 32 x 32.
template <Product PR, int TM, int TN>
__device__ __forceinline__ void multiply(f16v (&acc)[TM][TN], const operand (&w)[TN], const operand (&x)[TM]) {
    if constexpr (PR == MX_FAST) {   // (the lane's scales were moved to bytes 0 and 2)
        const auto pair = [](const operand &o, int s) {
            return i8v{(int)o.c[s].x,     (int)o.c[s].y,     (int)o.c[s].z,     (int)o.c[s].w,
                       (int)o.c[s + 1].x, (int)o.c[s + 1].y, (int)o.c[s + 1].z, (int)o.c[s + 1].w};
        };
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j)
                acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(pair(w[i], 0), pair(x[j], 0), acc[j][i], 0, 0, 0,
                                                                            (int)w[i].scales, 0, (int)x[j].scales);
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j)
                acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(pair(w[i], 2), pair(x[j], 2), acc[j][i], 0, 0, 2,
                                                                            (int)w[i].scales, 2, (int)x[j].scales);
        return;
    }
    constexpr int kParts = PR == BF16 ? 4 : 8;   // products of 16 elements of K each
#pragma unroll
    for (int s = 0; s < kParts; ++s) {
        const auto part = [s](const operand &o) {
            if constexpr (PR == BF16) return __builtin_bit_cast(b8v, o.c[s]);
            else return widen_codes(o.c[s >> 1], s & 1, (o.scales >> (8 * (s >> 1))) & 0xFFu);
        };
        b8v b[TM];
#pragma unroll
        for (int j = 0; j < TM; ++j) b[j] = part(x[j]);
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            const b8v a = part(w[i]);
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b[j], acc[j][i], 0, 0, 0);
        }
    }
}

// A row's four scales of a step: the dword at `at`, or (not WHOLE) bytes shift % 4
// .. + 3 of it and the one a plane behind it, `left` of them inside the row (zeros
// behind it).  shift counts a whole operand's scales, modulo 2^32.
template <bool WHOLE>
__device__ __forceinline__ uint32_t row_scales(const char *at, int plane, uint32_t shift, int left) {
    uint32_t v = *reinterpret_cast<const uint32_t *>(at);
    if constexpr (!WHOLE) {
        v = __builtin_amdgcn_alignbyte(*reinterpret_cast<const uint32_t *>(at + plane), v, shift);
        if (left < 4) v &= (1u << (8 * left)) - 1;
    }
    return v;
}

// Rows 0..31 of `tile` (LDS, at a multiple of 16 rows) as an operand, but for its scales.
__device__ __forceinline__ void read_chunks(operand &o, const char *tile, int lane) {
    const int r = lane & 31, h = lane >> 5;
    const char *p = tile + r * kStep;
#pragma unroll
    for (int s = 0; s < 4; ++s) o.c[s] = *reinterpret_cast<const u4v *>(p + (((2 * s + h) ^ ((r >> 1) & 7)) << 4));
}

// ----------------------------------------------------- rows of any alignment --

// Tiles of 64 outputs x 64 rows, staged through registers: a row may start at
// any element and end at any.  Four waves of 32 x 32.  16, 256 and 2048 rows take
// 2.4, 2.6 and 2.7 times the aligned kernels' time (4095 inputs, 14432 outputs: 57 us
// where 4096 take 23; 122, 46; 6143 inputs, 4096 outputs: 257, 6144: 97).
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
            *reinterpret_cast<u4v *>(&tile[buf][r * kStep + (((threadIdx.x & 7) ^ ((r >> 1) & 7)) << 4)]) = c[i];
        }
        if (MX && threadIdx.x < 2 * B) scales[buf][threadIdx.x] = sc;
    };

    f16v acc[1][1] = {{(f16v)0.f}};
    const int wn = 32 * (wave & 1), wm = B + 32 * (wave >> 1);
    const int steps = (p.k_bytes + kStep - 1) / kStep;
    load(0);
    put(0);
    for (int k = 0; k < steps; ++k) {
        if (k + 1 < steps) load(k + 1);
        __syncthreads();
        operand w[1], x[1];
        read_chunks(w[0], &tile[k & 1][wn * kStep], lane);
        read_chunks(x[0], &tile[k & 1][wm * kStep], lane);
        if constexpr (MX) {
            w[0].scales = scales[k & 1][wn + (lane & 31)];
            x[0].scales = scales[k & 1][wm + (lane & 31)];
        }
        multiply<MX ? MX_EXACT : BF16>(acc, w, x);
        if (k + 1 < steps) put((k + 1) & 1);
    }
    __syncthreads();   // the last step was read
    finish<1>(p, m0 + wm - B, n0 + wn, acc[0], tile[0] + 4096 * wave, lane);
}

// ------------------------------------------------------------ direct loads --

// 16 (or 4) bytes a lane from buffer + off + at to the wave's 1024 (256) bytes
// of LDS at `lds`.  Written out, since the compiler would wait for every such
// load before any read of LDS.  Nothing is loaded to a register; m0, the LDS
// base, is set and used in one block.  The buffers are made at the start of a
// kernel, far enough ahead for their scalar registers.
__device__ __forceinline__ void load_to_lds16(u4v buffer, int off, int at, unsigned lds) {
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(off),
                 "s"(buffer), "s"(at), "s"(lds)
                 : "m0", "memory");
}
__device__ __forceinline__ void load_to_lds4(u4v buffer, int off, int at, unsigned lds) {
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds" ::"v"(off), "s"(buffer),
                 "s"(at), "s"(lds)
                 : "m0", "memory");
}

// A buffer resource over `bytes` bytes at a wave-uniform address.
__device__ __forceinline__ u4v resource(const void *p, int bytes) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    return u4v{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)u),
               (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(u >> 32) & 0xFFFFu),
               (uint32_t)__builtin_amdgcn_readfirstlane(bytes), (uint32_t)kBufferRsrcWord3};
}

// The wave's LDS reads and all but LEFT of its loads are done, and every wave
// of the workgroup got here.
template <int LEFT>
__device__ __forceinline__ void arrive() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void arrive_loading() {   // the same, with loads in flight
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ unsigned lds_offset(const void *p) {
    typedef __attribute__((address_space(3))) const void lds_void;
    return __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)(lds_void *)p);
}

// Which tile a workgroup takes.  Workgroups go to the 8 XCDs in turn, so each
// XCD is given one stretch of the order (its L2 then holds what its tiles
// share), and the order goes through GROUP rows of tiles at a time.
template <int GROUP>
__device__ __forceinline__ void tile_of(unsigned id, unsigned tiles_n, unsigned tiles_m, unsigned &tn, unsigned &tm) {
    const unsigned tiles = tiles_n * tiles_m, each = tiles / 8, more = tiles % 8, x = id % 8;
    const unsigned t = x * each + min(x, more) + id / 8;
    const unsigned band = t / (GROUP * tiles_n), in = t - band * GROUP * tiles_n;
    const unsigned high = min((unsigned)GROUP, tiles_m - band * GROUP);
    tn = in / high;
    tm = band * GROUP + in - tn * high;
}

// A byte offset outside every buffer here: a load from it brings zeros (with a
// scalar offset inside the buffer, as the range check may take that off its size).
constexpr int kNowhere = 0x7FFFFFF0;

// One side's rows of a tile, on their way to LDS: ROWS rows by WAVES waves, a
// load of eight rows each.  Rows behind the last are the last again; chunks
// behind a row's end are zeros.
template <int ROWS, int WAVES>
struct RowLoads {
    static constexpr int kLoads = ROWS / 8 / WAVES;
    u4v rows;
    int off[kLoads];
    __device__ __forceinline__ RowLoads(const void *p, int64_t pitch, int64_t first, int64_t count, int k_bytes, int wave,
                                        int lane) {
        const int last = (int)min((int64_t)ROWS, count - first) - 1;
        rows = resource(static_cast<const char *>(p) + first * pitch, (int)(last * pitch) + k_bytes);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) off[i] = min(row_of(i, wave, lane), last) * (int)pitch + 16 * chunk_of(i, wave, lane);
    }
    static __device__ __forceinline__ int row_of(int i, int wave, int lane) { return 8 * (wave + i * WAVES) + lane / 8; }
    static __device__ __forceinline__ int chunk_of(int i, int wave, int lane) {
        return (lane & 7) ^ ((row_of(i, wave, lane) >> 1) & 7);
    }
    // `left`: bytes of a row from step k on.
    __device__ __forceinline__ void issue(int k, int left, unsigned lds, int wave, int lane) const {
        if (left >= kStep) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) load_to_lds16(rows, off[i], k * kStep, lds + 1024 * (wave + i * WAVES));
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                load_to_lds16(rows, 16 * chunk_of(i, wave, lane) < left ? off[i] : kNowhere, k * kStep,
                              lds + 1024 * (wave + i * WAVES));
        }
    }
};

// The scales of 64 rows of one side (a lane each) on their way to LDS, for four
// steps at a time.  Rows of whole fours: 16 bytes a row, at_row = 16 bytes apart,
// the steps' at_step = 4 bytes within them.  Other rows may start at any byte:
// five planes of a dword a row (at_row = 4, at_step = a plane), of which a step's
// four bytes lie in two neighbouring ones; dwords behind the tile's last are that
// one again.
struct ScaleLoads {
    u4v rows;
    int off, end;
    __device__ __forceinline__ ScaleLoads() {}
    // Lane's row `row` of those from `first` on, of which `last` is the last to be read.
    __device__ __forceinline__ ScaleLoads(const uint8_t *scales, int per, int64_t first, int last, int row) {
        const int64_t start = first * per, base = start & ~(int64_t)3;
        const int shift = (int)(start - base);
        end = (shift + (last + 1) * per - 1) & ~3;
        rows = resource(scales + base, end + 4);
        off = (shift + min(row, last) * per) & ~3;
    }
    template <bool WHOLE>
    __device__ __forceinline__ void issue(int g, int steps, unsigned to, int plane) const {
        if constexpr (WHOLE) {
            load_to_lds16(rows, off, 16 * min(g, steps / 4 - 1), to);
        } else {
#pragma unroll
            for (int s = 0; s < 5; ++s) load_to_lds4(rows, min(off + 16 * g + 4 * s, end), 0, to + s * plane);
        }
    }
};

// ------------------------------------------------------------- wide tiles --

// 256 outputs x 256 rows, eight waves of 128 x 64, four half steps (64 bytes of
// K) in LDS.  The two waves of a SIMD alternate: while one multiplies the half
// step that it holds in registers, the other reads its next operands, so the
// matrix cores always have one of them to work for.  Chunk c of row r of a half
// step lies at place c ^ (r >> 2 & 3) of its 64 bytes.
template <Product PR, bool WHOLE>
__global__ void __launch_bounds__(512) linear_wide_kernel(LinearParams p) {
    constexpr int B = 256, kHalf = kStep / 2, kSide = B * kHalf, kStages = 4;
    constexpr int kLoads = 4;   // of a wave and half step
    constexpr int kGroup = 8;   // half steps whose scales are loaded together
    __shared__ __attribute__((aligned(1024))) char tile[kStages][2 * kSide];
    constexpr int kGroupBytes = PR == BF16 ? 16 : 2 * B * 20;
    __shared__ __attribute__((aligned(1024))) char scales[2][kGroupBytes];
    unsigned tn, tm;
    tile_of<8>(blockIdx.x, (p.n_out + B - 1) / B, (unsigned)((p.rows + B - 1) / B), tn, tm);
    const int n0 = tn * B;
    const int64_t m0 = (int64_t)tm * B;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // A wave loads rows 16 (wave + 8 i) .. + 15 of both sides; rows behind the last are the last again.
    const int last_n = min(B, p.n_out - n0) - 1, last_m = (int)min((int64_t)B, p.rows - m0) - 1;
    const u4v rw = resource(static_cast<const char *>(p.w) + n0 * p.w_pitch, (int)(last_n * p.w_pitch) + p.k_bytes);
    const u4v rx = resource(static_cast<const char *>(p.x) + m0 * p.x_pitch, (int)(last_m * p.x_pitch) + p.k_bytes);
    int ow[2], ox[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = 16 * (wave + 8 * i) + lane / 4, c = (lane & 3) ^ ((lane >> 4) & 3);
        ow[i] = min(r, last_n) * (int)p.w_pitch + 16 * c;
        ox[i] = min(r, last_m) * (int)p.x_pitch + 16 * c;
    }
    const int per = p.k_bytes / kMxBlock;
    ScaleLoads sc;
    if constexpr (PR != BF16) {   // waves 0..3 load the scales of w's rows, 4..7 those of x's
        const int row = 64 * (wave & 3) + lane;
        sc = wave < 4 ? ScaleLoads(p.w_scales, per, n0, last_n, row) : ScaleLoads(p.x_scales, per, m0, last_m, row);
    }
    const unsigned lds = lds_offset(tile), lds_sc = lds_offset(scales);
    const int steps = (p.k_bytes + kStep - 1) / kStep, halves = (p.k_bytes + kHalf - 1) / kHalf;
    constexpr int at_row = WHOLE ? 16 : 4, at_step = WHOLE ? 4 : 8 * B;   // (see ScaleLoads)
    const auto issue_scales = [&](int g) {
        sc.template issue<WHOLE>(g, steps, lds_sc + (g & 1) * kGroupBytes + 64 * at_row * wave, at_step);
    };
    // Behind the end the last half step is loaded again, for nobody: a constant number of loads is in flight.
    const auto issue = [&](int j) {
        const int at = min(j, halves - 1) * kHalf, left = p.k_bytes - at;
        const unsigned to = lds + (j & 3) * 2 * kSide + 1024 * wave;
        const auto load = [&](int w0, int w1, int x0, int x1) {
            load_to_lds16(rw, w0, at, to);
            load_to_lds16(rw, w1, at, to + 8192);
            load_to_lds16(rx, x0, at, to + kSide);
            load_to_lds16(rx, x1, at, to + kSide + 8192);
        };
        if (left >= kHalf) {
            load(ow[0], ow[1], ox[0], ox[1]);
        } else {   // chunks behind a row's end are zeros
            const bool in = 16 * ((lane & 3) ^ ((lane >> 4) & 3)) < left;
            load(in ? ow[0] : kNowhere, in ? ow[1] : kNowhere, in ? ox[0] : kNowhere, in ? ox[1] : kNowhere);
        }
        if constexpr (PR != BF16)   // (in time for half step j - j % 8 + 8; the waits below count four loads a half step and wait for more where these are between)
            if ((j & (kGroup - 1)) == 3) issue_scales(j / kGroup + 1);
    };

    f16v acc[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = (f16v)0.f;
    u4v w[4][2], x[2][2];
    uint32_t sw[4], sx[2];
    const int wn = 128 * (wave >> 2), wm = 64 * (wave & 3);
    const int r = lane & 31, h = lane >> 5, place = (h ^ ((r >> 2) & 3)) << 4;
    const auto read = [&](int j) {
        const char *t = tile[j & 3] + r * kHalf;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                x[i][s] = *reinterpret_cast<const u4v *>(t + kSide + (wm + 32 * i) * kHalf + (place ^ (32 * s)));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i][s] = *reinterpret_cast<const u4v *>(t + (wn + 32 * i) * kHalf + (place ^ (32 * s)));
        }
        if constexpr (PR != BF16) {   // MX_FAST: the lane's one scale in byte 0; MX_EXACT: of chunks s = 0, 1 in bytes 0, 1
            const char *at = scales[(j / kGroup) & 1] + at_step * ((j >> 1) & 3) + r * at_row;
            const int left = per - 2 * (j & ~1), shift = 16 * (j & 1) + (PR == MX_FAST ? 8 * h : 0);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                sx[i] = row_scales<WHOLE>(at + (B + wm + 32 * i) * at_row, at_step, ((uint32_t)m0 + wm + 32 * i + r) * per, left) >> shift;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sw[i] = row_scales<WHOLE>(at + (wn + 32 * i) * at_row, at_step, (uint32_t)(n0 + wn + 32 * i + r) * per, left) >> shift;
        }
    };
    const auto work = [&] {
        if constexpr (PR == MX_FAST) {
            const auto pair = [](const u4v (&c)[2]) {
                return i8v{(int)c[0].x, (int)c[0].y, (int)c[0].z, (int)c[0].w, (int)c[1].x, (int)c[1].y, (int)c[1].z, (int)c[1].w};
            };
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(pair(w[i]), pair(x[j]), acc[j][i], 0, 0, 0,
                                                                                (int)sw[i], 0, (int)sx[j]);
            return;
        }
        constexpr int kParts = PR == BF16 ? 2 : 4;
#pragma unroll
        for (int s = 0; s < kParts; ++s) {
            const auto part = [s](const u4v (&c)[2], uint32_t sc) {
                if constexpr (PR == BF16) return __builtin_bit_cast(b8v, c[s]);
                else return widen_codes(c[s >> 1], s & 1, (sc >> (8 * (s >> 1))) & 0xFFu);
            };
            b8v b[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) b[j] = part(x[j], PR == BF16 ? 0 : sx[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const b8v a = part(w[i], PR == BF16 ? 0 : sw[i]);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b[j], acc[j][i], 0, 0, 0);
            }
        }
    };

    // Slot 2j: waves 0..3 read half step j, slot 2j + 1: they multiply it and 4..7
    // read it, slot 2j + 2: 4..7 multiply it.  A set asks for half step j + 3 when it
    // has asked LDS for j: j - 1, which it replaces, was read by all before slot 2j.
    // j + 1 has to be there at the end of slot 2j + 1, with j + 2 and j + 3 still on
    // their way.
    if constexpr (PR != BF16) issue_scales(0);
    issue(0);
    issue(1);
    issue(2);
    arrive<2 * kLoads>();
    if (wave < 4) {
        for (int j = 0; j < halves; ++j) {
            read(j);
            issue(j + 3);
            arrive_loading();
            __builtin_amdgcn_s_setprio(1);
            work();
            __builtin_amdgcn_s_setprio(0);
            arrive<2 * kLoads>();
        }
        arrive_loading();
    } else {
        arrive_loading();
        for (int j = 0; j < halves; ++j) {
            read(j);
            issue(j + 3);
            arrive<2 * kLoads>();
            __builtin_amdgcn_s_setprio(1);
            work();
            __builtin_amdgcn_s_setprio(0);
            arrive_loading();
        }
    }
    arrive<0>();
#pragma unroll
    for (int j = 0; j < 2; ++j) finish<4>(p, m0 + wm + 32 * j, n0 + wn, acc[j], tile[0] + 16384 * wave, lane);
}

// ------------------------------------------------------------ small tiles --

// BN outputs x BM rows by WN x WM waves, STAGES steps in LDS: every wave asks for
// step k + STAGES - 1 before it multiplies step k.
template <Product PR, bool WHOLE, int BN, int BM, int WN, int WM, int STAGES>
__global__ void __launch_bounds__(64 * WN * WM) linear_tile_kernel(LinearParams p) {
    constexpr int kWaves = WN * WM, TN = BN / WN / 32, TM = BM / WM / 32, kRows = BN + BM, kStage = kRows * kStep;
    constexpr int kLoads = kRows / 8 / kWaves, kScaleLoads = PR == BF16 ? 0 : (kRows / 64 + kWaves - 1) / kWaves;
    constexpr int kScaleFour = PR == BF16 ? 16 : kRows * 20;   // bytes of four steps' scales
    static_assert(STAGES <= 5, "a four's scales are asked for no later than its first step");
    static_assert(kRows / 8 % kWaves == 0 && BN % 64 == 0 && BM % 64 == 0, "whole loads");
    static_assert(STAGES * kStage >= kWaves * TN * 4096, "sums pass through the stages");
    __shared__ __attribute__((aligned(1024))) char tile[STAGES][kStage];
    __shared__ __attribute__((aligned(1024))) char scales[2][kScaleFour];
    unsigned tn, tm;
    tile_of<8>(blockIdx.x, (p.n_out + BN - 1) / BN, (unsigned)((p.rows + BM - 1) / BM), tn, tm);
    const int n0 = tn * BN;
    const int64_t m0 = (int64_t)tm * BM;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const RowLoads<BN, kWaves> lw(p.w, p.w_pitch, n0, p.n_out, p.k_bytes, wave, lane);
    const RowLoads<BM, kWaves> lx(p.x, p.x_pitch, m0, p.rows, p.k_bytes, wave, lane);
    const int steps = (p.k_bytes + kStep - 1) / kStep, per = p.k_bytes / kMxBlock;
    constexpr int at_row = WHOLE ? 16 : 4, at_step = WHOLE ? 4 : 4 * kRows;   // (see ScaleLoads)
    // Few rows: the weights are read once, by tiles side by side, which start 12
    // steps apart and go round, so that they do not all ask the same channels for
    // the same part of K (64 rows of 14432 x 4096: 29.6 -> 27.1 us).  Tiles that share
    // weights stay together (1024 rows of 4096 x 6144: 63 us, apart 70).
    const bool apart = p.k_bytes % (4 * kStep) == 0 && p.rows <= BM;
    const int start = apart ? 4 * (3 * tn % (steps / 4)) : 0;
    ScaleLoads sc[kScaleLoads ? kScaleLoads : 1];
    int sto[kScaleLoads ? kScaleLoads : 1];
    if constexpr (PR != BF16) {   // 64 rows' scales a load: w's, then x's (waves without rows load others' again)
#pragma unroll
        for (int i = 0; i < kScaleLoads; ++i) {
            const int at = 64 * ((wave + i * kWaves) % (kRows / 64));
            const bool ofw = at < BN;
            const int64_t first = ofw ? n0 : m0;
            const int last = (int)min((int64_t)(ofw ? BN : BM), (ofw ? (int64_t)p.n_out : p.rows) - first) - 1;
            sc[i] = ScaleLoads(ofw ? p.w_scales : p.x_scales, per, first, last, at - (ofw ? 0 : BN) + lane);
            sto[i] = at * at_row;
        }
    }
    const unsigned lds = lds_offset(tile), lds_sc = lds_offset(scales);
    const auto issue_scales = [&](int g) {
        int at = min(g, (steps - 1) / 4) + start / 4;
        at = at > (steps - 1) / 4 ? at - steps / 4 : at;
#pragma unroll
        for (int i = 0; i < kScaleLoads; ++i) sc[i].template issue<WHOLE>(at, steps, lds_sc + (g & 1) * kScaleFour + sto[i], at_step);
    };
    // Steps behind the last are the last again (a constant number of loads is in flight); nothing reads them.
    const auto issue = [&](int k, int stage) {
        int at = min(k, steps - 1) + start;
        at = at >= steps ? at - steps : at;
        const int left = p.k_bytes - at * kStep;
        lw.issue(at, left, lds + stage * kStage, wave, lane);
        lx.issue(at, left, lds + stage * kStage + BN * kStep, wave, lane);
    };
    f16v acc[TM][TN];
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int i = 0; i < TN; ++i) acc[j][i] = (f16v)0.f;
    const int wn = BN / WN * (wave % WN), wm = BM / WM * (wave / WN);
    if constexpr (PR != BF16) issue_scales(0);
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) issue(k, k);
    int stage = 0, next = STAGES - 1;
    for (int k = 0; k < steps; ++k) {
        arrive<(STAGES - 2) * kLoads>();   // (scales in between make it wait for more)
        if constexpr (PR != BF16)   // into the place of the four before, which all have read
            if ((k & 3) == 0) issue_scales(k / 4 + 1);
        issue(k + STAGES - 1, next);
        operand w[TN], x[TM];
        const char *t = tile[stage], *s = scales[(k >> 2) & 1] + (k & 3) * at_step;
        const int left = per - 4 * k;   // (rows that start apart are whole)
#pragma unroll
        for (int j = 0; j < TM; ++j) read_chunks(x[j], t + (BN + wm + 32 * j) * kStep, lane);
#pragma unroll
        for (int i = 0; i < TN; ++i) read_chunks(w[i], t + (wn + 32 * i) * kStep, lane);
        if constexpr (PR != BF16) {
            const int r = lane & 31, shift = PR == MX_FAST ? 8 * (lane >> 5) : 0;
#pragma unroll
            for (int j = 0; j < TM; ++j)
                x[j].scales = row_scales<WHOLE>(s + (BN + wm + 32 * j + r) * at_row, at_step,
                                                ((uint32_t)m0 + wm + 32 * j + r) * per, left) >> shift;
#pragma unroll
            for (int i = 0; i < TN; ++i)
                w[i].scales = row_scales<WHOLE>(s + (wn + 32 * i + r) * at_row, at_step, (uint32_t)(n0 + wn + 32 * i + r) * per, left) >> shift;
        }
        multiply<PR>(acc, w, x);
        stage = stage + 1 == STAGES ? 0 : stage + 1;
        next = next + 1 == STAGES ? 0 : next + 1;
    }
    arrive<0>();
#pragma unroll
    for (int j = 0; j < TM; ++j) finish<TN>(p, m0 + wm + 32 * j, n0 + wn, acc[j], tile[0] + 4096 * TN * wave, lane);
}

// ---------------------------------------------------------------- few rows --

// 16 NT outputs x 16 MT rows by a workgroup whose waves share K: each takes every
// WAVES-th step, AHEAD of them at a time, straight from memory to registers, and
// their sums are added in LDS in the order of the waves.  16 x 16 tiles: lane l
// holds row l % 16 of an operand, chunks l / 16 and 4 + l / 16 of a step, and
// those lie in blocks l / 32 and 2 + l / 32.
template <bool MX, int WAVES, int NT, int MT, int AHEAD>
__global__ void __launch_bounds__(64 * WAVES) linear_few_kernel(LinearParams p) {
    __shared__ f4v part[WAVES][MT][NT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
    unsigned tn, tm;
    tile_of<8>(blockIdx.x, (p.n_out + 16 * NT - 1) / (16 * NT), (unsigned)((p.rows + 16 * MT - 1) / (16 * MT)), tn, tm);
    const int n0 = tn * 16 * NT;
    const int64_t m0 = (int64_t)tm * 16 * MT;
    const int per = p.k_bytes / kMxBlock;
    const char *x[MT], *w[NT];
    const uint8_t *xs[MT], *ws[NT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {   // rows behind the last are the last again
        const int64_t m = min(m0 + 16 * j + r, p.rows - 1);
        x[j] = static_cast<const char *>(p.x) + m * p.x_pitch + 16 * q;
        xs[j] = MX ? p.x_scales + m * per : nullptr;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t n = min(n0 + 16 * t + r, p.n_out - 1);
        w[t] = static_cast<const char *>(p.w) + n * p.w_pitch + 16 * q;
        ws[t] = MX ? p.w_scales + n * per : nullptr;
    }
    f4v acc[MT][NT];
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[j][t] = (f4v)0.f;
    struct step {
        u4v c[2];
        uint32_t s;
    };
    const int steps = (p.k_bytes + kStep - 1) / kStep;
    typedef uint32_t u1u __attribute__((aligned(1)));
    const auto load = [&](const char *v, const uint8_t *scales, int k) {   // behind a row's end: zeros
        step o;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = k * kStep + 64 * i;
            o.c[i] = at + 16 * q < p.k_bytes ? *reinterpret_cast<const u4v *>(v + at) : (u4v)0u;
        }
        o.s = 0;
        if constexpr (MX) {
            const int left = per - 4 * k;
            if (left >= 4) o.s = *reinterpret_cast<const u1u *>(scales + 4 * k);
            else
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (i < left) o.s |= (uint32_t)scales[4 * k + i] << (8 * i);
        }
        return o;
    };
    for (int k = wave; k < steps; k += AHEAD * WAVES) {
        step a[AHEAD][NT], b[AHEAD][MT];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
#pragma unroll
            for (int t = 0; t < NT; ++t) a[u][t] = load(w[t], ws[t], k + u * WAVES);
#pragma unroll
            for (int j = 0; j < MT; ++j) b[u][j] = load(x[j], xs[j], k + u * WAVES);
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int half = 0; half < (MX ? 2 : 1); ++half) {
                    const auto part = [&](const step &o) {
                        if constexpr (MX) return widen_codes(o.c[i], half, (o.s >> (16 * i + 8 * (q >> 1))) & 0xFFu);
                        else return __builtin_bit_cast(b8v, o.c[i]);
                    };
                    b8v xb[MT];
#pragma unroll
                    for (int j = 0; j < MT; ++j) xb[j] = part(b[u][j]);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const b8v wa = part(a[u][t]);
#pragma unroll
                        for (int j = 0; j < MT; ++j)
                            acc[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wa, xb[j], acc[j][t], 0, 0, 0);
                    }
                }
    }
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int t = 0; t < NT; ++t) part[wave][j][t][lane] = acc[j][t];
    __syncthreads();
    // Output n0 + 8 c .. of row m0 + row: the sums i of lanes 16 (n % 16 / 4) + row % 16 of tile n / 16.
    static_assert(32 * NT * MT <= 64 * WAVES, "a thread for every eight outputs");
    const int c = threadIdx.x % (2 * NT), row = threadIdx.x / (2 * NT), left = p.n_out - n0 - 8 * c;
    if (row >= 16 * MT || m0 + row >= p.rows || left <= 0) return;
    f8v v = (f8v)0.f, bias = (f8v)0.f;
    if (p.bias) bias = load_part<false>(p.bias + n0 + 8 * c, left);
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
        const f4v *t = part[i][row >> 4][c >> 1] + 32 * (c & 1) + (row & 15);
        const f4v a = t[0], b = t[16];
        v += f8v{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    }
    put8(p, m0 + row, n0 + 8 * c, left, v, bias);
}

// Kernels by their tiles, and what a call costs in each: a part that every call
// has and one for each round of 256 tiles (one per compute unit), fitted to calls
// of 1 to 16384 rows of 256 to 16384 outputs; 1 is what 64 x 64 tiles take for one
// round.  Small tiles keep all units at work, large ones load less for each
// product: of 6144 inputs and 4096 outputs in bf16, 64 rows take 45 us in 16 x 16
// tiles, 26 in 32 x 32, 34 in 64 x 64; 1024 rows 96 in 64 x 64, 63 in 128 x 128, 94 in
// 256 x 128, 144 in 256 x 256; 2048 rows 180, 128, 111 and 147; 8192 rows of 8192 x
// 8192 1560, 1125, 1100 and 862.
enum Tile { T16, T32x16, T32, T64, T64x128, T128, T256x128, T256, kTiles };
struct TileCost {
    int n, m;
    float call[3], round[3];   // by Product
};
constexpr TileCost kTileCosts[kTiles] = {
    {16, 16, {.12f, .19f, .19f}, {.24f, .37f, .37f}},   {32, 16, {.14f, .23f, .23f}, {.42f, .56f, .56f}},
    {32, 32, {.13f, .16f, .16f}, {.48f, .81f, .81f}},   {64, 64, {.55f, .60f, .55f}, {.42f, .55f, .41f}},
    {64, 128, {.45f, 1e9f, .30f}, {.85f, .0f, .95f}}, {128, 128, {.40f, .0f, .45f}, {1.22f, 2.05f, 1.25f}},
    {256, 128, {.0f, .0f, .15f}, {2.4f, 3.7f, 2.15f}},  {256, 256, {.0f, .0f, .15f}, {3.8f, 6.1f, 3.25f}},
};

int64_t tiles_of(const LinearParams &p, int n, int m) { return (p.rows + m - 1) / m * ((p.n_out + n - 1) / n); }

Tile best_tile(const LinearParams &p, Product pr) {
    int best = T64;
    float least = 3e38f;
    // (16 outputs are half a block of an MX output)
    for (int t = p.out_type == RSSM_FP8_E4M3 ? T32x16 : T16; t < kTiles; ++t) {
        const int64_t rounds = (tiles_of(p, kTileCosts[t].n, kTileCosts[t].m) + 255) / 256;
        const float cost = kTileCosts[t].call[pr] + kTileCosts[t].round[pr] * rounds;
        if (cost < least) {
            least = cost;
            best = t;
        }
    }
    return (Tile)best;
}

// WHOLE: rows of whole fours of steps' scales (bf16 rows have none).
template <Product PR, bool WHOLE>
void launch_direct(const LinearParams &p, hipStream_t s) {
    constexpr bool MX = PR != BF16;
    const Tile t = best_tile(p, PR);
    const dim3 grid((unsigned)tiles_of(p, kTileCosts[t].n, kTileCosts[t].m));
    switch (t) {
        case T16: hipLaunchKernelGGL((linear_few_kernel<MX, 8, 1, 1, 2>), grid, dim3(512), 0, s, p); break;
        case T32x16: hipLaunchKernelGGL((linear_few_kernel<MX, 8, 2, 1, 2>), grid, dim3(512), 0, s, p); break;
        case T32: hipLaunchKernelGGL((linear_few_kernel<MX, 8, 2, 2, 2>), grid, dim3(512), 0, s, p); break;
        case T64: hipLaunchKernelGGL((linear_tile_kernel<PR, WHOLE, 64, 64, 2, 2, 4>), grid, dim3(256), 0, s, p); break;
        case T64x128:   // (MX_EXACT: never the least)
            if constexpr (PR != MX_EXACT)
                hipLaunchKernelGGL((linear_tile_kernel<PR, WHOLE, 64, 128, 2, 2, 4>), grid, dim3(256), 0, s, p);
            break;
        case T128: hipLaunchKernelGGL((linear_tile_kernel<PR, WHOLE, 128, 128, 2, 4, 4>), grid, dim3(512), 0, s, p); break;
        case T256x128: hipLaunchKernelGGL((linear_tile_kernel<PR, WHOLE, 256, 128, 4, 2, 3>), grid, dim3(512), 0, s, p); break;
        default: hipLaunchKernelGGL((linear_wide_kernel<PR, WHOLE>), grid, dim3(512), 0, s, p); break;
    }
}

bool multiple(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

}  // namespace

hipError_t launch_linear(const LinearParams &p, bool mx, bool fast, hipStream_t s) {
    // Rows at aligned addresses are loaded straight to LDS or operands.
    const bool direct = p.w_pitch % 16 == 0 && p.x_pitch % 16 == 0 && multiple(p.x, 16) && multiple(p.w, 16) &&
                        (!mx || (multiple(p.x_scales, 4) && multiple(p.w_scales, 4)));
    if (!direct) {
        const dim3 grid((unsigned)tiles_of(p, 64, 64));
        if (mx) hipLaunchKernelGGL(linear_any_kernel<true>, grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL(linear_any_kernel<false>, grid, dim3(256), 0, s, p);
    } else if (!mx) {
        launch_direct<BF16, true>(p, s);
    } else {
        const bool whole = p.k_bytes % (4 * kStep) == 0;
        if (fast) whole ? launch_direct<MX_FAST, true>(p, s) : launch_direct<MX_FAST, false>(p, s);
        else whole ? launch_direct<MX_EXACT, true>(p, s) : launch_direct<MX_EXACT, false>(p, s);
    }
    return hipGetLastError();
}

}  // namespace rssm
