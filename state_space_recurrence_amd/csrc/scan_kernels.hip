// scan_kernels.hip -- packed prompts through the recurrence on the matrix
// cores (bf16 or fp32 inputs, fp32 checkpoints).
//
// A sequence is taken in chunks of 64 tokens.  With l_i = A dt_i, c_t the sum
// of l over the chunk up to t, and S the state before the chunk:
//     M_tj = (C_t . B_j) dt_j exp(c_t - c_j)  for j <= t, else 0
//     y_t  = sum_j M_tj x_j + exp(c_t) S C_t + D x_t
//     S'   = exp(c_63) S + sum_j dt_j exp(c_63 - c_j) x_j (outer) B_j
// One wave owns 32 of the 64 state rows p of a head and keeps its half of the
// state, transposed [n][p], in the accumulators of v_mfma_f32_32x32x16_bf16
// for the whole segment.  An accumulator holds 4 consecutive rows per lane
// half, an operand 8 consecutive inner indices; which n or p a row stands for,
// and the order of the inner index, are free as long as both sides agree, so
// the state's accumulators are the operands of S C straight from registers.
// The Gram tiles C B^T are the same for every head: the workgroup's waves form
// them in pieces of 16 x 16, zero above the diagonal, and share them in LDS
// (each wave forming all of them costs 24 more matrix instructions a chunk and
// the 48 registers that the next step's operands now take).
//
// Staging.  The chunk's B, C and x go from memory to LDS directly (16 bytes a
// lane, no registers), one chunk ahead in the other of two buffers; rows of B
// and C serve as operands of S C and of the Gram tiles as they lie, and the
// transposed operands (B as [n][j], x as [p][j]) come from the same rows by
// transposing LDS reads (4 rows x 16 columns a quarter wave).  Pairs of
// 16-byte pieces are exchanged by row so that both kinds of reads spread over
// the banks.
//
// Precision.  x, B, C are bf16 and exact operands.  Values formed in fp32
// (state, M, weighted x) are split into bf16 parts, v = hi + mid + lo, and
// multiplied part by part into the same fp32 accumulator: three parts carry
// all 24 bits, two carry 16.  The state always uses three, so it is as exact
// as an fp32 update; y uses three for fp32 outputs and two for bf16 ones,
// whose own rounding is 2^-8.  Decay sums run in fp64 and are kept as a whole
// and a fractional power of two: a difference of two long sums would
// otherwise lose the bits of a short one.
//
// What bounds it.  One sequence of 16384 tokens, 96 heads in 8 groups, bf16,
// call after call: 42 us for the first launch and 232 us for the second (the
// median; 35 and 196 us the shortest, before the clock falls), where 479 MB
// would take 97 us at the copy rate.  Of a chunk's 15000 cycles a SIMD's two
// waves need 6400 for matrix instructions, and each wave 5500 to issue its 1250
// vector instructions (most of them split the state and M into parts).  A wave
// issues one instruction at a time, so what counts is that neither products nor
// LDS reads are waited for: operands are read a step ahead, and the next step's
// vector work stands between the products of the last (second launch, shortest:
// without both 214 us, with the reads alone 205).  More than two waves a SIMD
// would need more than the LDS: a chunk is 64 KB, twice.  With fp32 outputs a
// chunk takes 122 products instead of 98, and 20000 cycles.
//
// Order.  Whole segments run first, then the sequences' rests by falling
// length: 23 sequences of 9001 tokens together, 128 heads, fp32 outputs, took
// 254 us a call so and 283 us in the sequences' own order (240 us now).
//
// Long sequences.  When sequences x heads do not fill the card, a sequence is
// cut into segments: a first launch leaves each segment's end state (the first
// from the slot's state, the others from zero), and in the second every
// segment joins the states before it, S = loc_{k-1} + lam_{k-1} (loc_{k-2} +
// ...), before it runs its tokens.  Both sums end where the decay is exactly
// zero in fp32: what lies before cannot change them, unless it is not finite,
// which the recurrence carries on (0 NaN is NaN) however fast the state decays.
// The second launch passes every token, so there each segment marks an end
// state that is not all finite, and a third launch, of a workgroup per segment
// and eight heads, puts NaN where the marked states say (where none is marked,
// the call takes 2.5 us longer for it).
#include "device_common.h"
#include "mixer_device.h"
#include "replay_common.h"
#include "scan.h"

namespace rssm {
namespace {

constexpr int kQ = kScanChunk;

typedef float f16v __attribute__((ext_vector_type(16)));
typedef float f2v __attribute__((ext_vector_type(2)));
typedef unsigned int u2v __attribute__((ext_vector_type(2)));
typedef int i8v __attribute__((ext_vector_type(8)));
typedef int i4v __attribute__((ext_vector_type(4)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef short s8v __attribute__((ext_vector_type(8)));
typedef __bf16 b2v __attribute__((ext_vector_type(2)));

// NH heads and 2 NH waves a workgroup; NP bf16 planes of each input.
template <int NH, int NP>
struct ScanSmem {
    struct Chunk {
        alignas(16) char B[NP][kQ][2 * kN];       // B_j[n]: 32-byte pair k of row j at k ^ (j mod 8)
        alignas(16) char C[NP][kQ][2 * kN];       // C_t[n], the same
        alignas(16) char x[NP][NH][kQ][2 * kP];   // x_j[p]: pair k of row j at k ^ (j / 2 mod 4)
    } chunk[NP == 1 ? 2 : 1];
    // per wave, with c_t / ln 2 = k_t + f_t, k_t whole and 0 <= f_t < 1:
    alignas(16) int k[2 * NH][kQ];
    alignas(16) float cf[2 * NH][kQ];         // dt_j 2^-f_j
    alignas(16) float w[2 * NH][kQ];          // dt_j exp(c_63 - c_j)
    float rf[2 * NH][kQ];                     // 2^f_t
    union {
        // G_tj = C_t . B_j of the lower tiles (t, j) = (0, 0), (1, 0), (1, 1) of 32 x 32, zero for j > t:
        // piece q of 4 j of row t at q ^ (t mod 8)
        alignas(16) float gram[3][32][32];
        int done[2][2 * NH];                  // per wave: nothing before the chunk counts (LOCAL)
    };
};

// Of each four quads the middle two trade places: row r of a 16-row tile
// stands for element 4 swapped(r / 4) + r mod 4, which gives the rows of a lane
// half (4 h .. 4 h + 3 and 8 + 4 h ..) eight consecutive elements.
__device__ __forceinline__ int swapped(int q) { return (q & 1) << 1 | q >> 1; }

__device__ __forceinline__ b8v operand(const char *p) {
    return __builtin_bit_cast(b8v, *reinterpret_cast<const f4v *>(p));
}

// Eight inner indices (rows j .. j + 3 and j + 8 .. j + 11, STEP bytes a row)
// of a transposed operand.
template <int STEP>
__device__ __forceinline__ b8v operand_t(const char *p) {
    typedef __attribute__((address_space(3))) s4v lds_s4;
    const s4v a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)p);
    const s4v b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p + 8 * STEP));
    return __builtin_bit_cast(b8v, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// v = part[0] + part[1] + ... to 8 NP bits (each part one rounding, two values an instruction)
template <int NP>
__device__ __forceinline__ void split(f8v v, b8v (&part)[NP]) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        u4v u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u[i] = __builtin_bit_cast(unsigned, __builtin_convertvector(f2v{v[2 * i], v[2 * i + 1]}, b2v));
            if (k + 1 < NP) {
                v[2 * i] -= __uint_as_float(u[i] << 16);
                v[2 * i + 1] -= __uint_as_float(u[i] & 0xFFFF0000u);
            }
        }
        part[k] = __builtin_bit_cast(b8v, u);
    }
}

__device__ __forceinline__ f16v mfma(b8v a, b8v b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f4v mfma16(b8v a, b8v b, f4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f8v half_of(const f16v &v, int s) {
    f8v r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[8 * s + i];
    return r;
}

__device__ __forceinline__ f8v read8(const float *p) {   // p[0..3], p[8..11]
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 8);
    return f8v{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

__device__ __forceinline__ i8v read8(const int *p) {
    const i4v a = *reinterpret_cast<const i4v *>(p), b = *reinterpret_cast<const i4v *>(p + 8);
    return i8v{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// A state tile from and to memory: values 0..7 at s, 8..15 at s + 16.
__device__ __forceinline__ void add_tile(f16v &v, const float *s, float f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 u = *reinterpret_cast<const float4 *>(s + 4 * i + 8 * (i >> 1));
        v[4 * i] += f * u.x;
        v[4 * i + 1] += f * u.y;
        v[4 * i + 2] += f * u.z;
        v[4 * i + 3] += f * u.w;
    }
}

__device__ __forceinline__ void put_tile(const f16v &v, float *s) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4 *>(s + 4 * i + 8 * (i >> 1)) =
            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

__device__ __forceinline__ void copy_tile(const float *s, float *d, bool write) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 u = *reinterpret_cast<const float4 *>(s + 4 * i + 8 * (i >> 1));
        if (write) *reinterpret_cast<float4 *>(d + 4 * i + 8 * (i >> 1)) = u;
    }
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_d(double v) {   // lanes without a source get 0
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)u, CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xF, false);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ double lane_d(double v, int l) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)u, l), hi = __builtin_amdgcn_readlane((int)(u >> 32), l);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Inclusive sum over lanes 0..l: shifts within rows of 16, then the last lane
// of a row into the next one, and lane 31 into the upper half.
__device__ __forceinline__ double prefix(double v) {
    v += dpp_d<0x111, 0xF>(v);
    v += dpp_d<0x112, 0xF>(v);
    v += dpp_d<0x114, 0xF>(v);
    v += dpp_d<0x118, 0xF>(v);
    v += dpp_d<0x142, 0xA>(v);
    v += dpp_d<0x143, 0xC>(v);
    return v;
}

// The lane number, derived again wherever it is asked for (two instructions):
// a chunk's addresses come from it and are held in no register between chunks,
// where a spilled one would wait for the loads in flight.
__device__ __forceinline__ int lane_again() {
    int l;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(l));
    return l;
}

// 16 bytes a lane from byte offset `off` of the buffer resource (zeros outside
// it) to the wave's 1024 bytes of LDS at `lds`.  Written out rather than by the
// builtin, which makes the compiler wait for it before the transposing reads
// of the other buffer; the kernel waits for it itself (vmcnt) at the end of a
// chunk.  Nothing is loaded to a register; m0, the LDS base, is set and used
// here.
__device__ __forceinline__ void load_to_lds(u4v resource, int off, unsigned lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(resource),
                 "s"(lds)
                 : "m0", "memory");
}

__device__ __forceinline__ u4v resource_of(const void *p, int bytes) {   // a wave-uniform address
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    return u4v{(unsigned)__builtin_amdgcn_readfirstlane((unsigned)u),
               (unsigned)__builtin_amdgcn_readfirstlane((unsigned)(u >> 32)) & 0xFFFFu, (unsigned)bytes,
               (unsigned)kBufferRsrcWord3};
}

__device__ __forceinline__ unsigned lds_offset(const void *p) {
    typedef __attribute__((address_space(3))) const void lds_void;
    return __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)(lds_void *)p);
}

// Exponent all ones in either half of any of the operand's dwords.
__device__ __forceinline__ bool non_finite(b8v v) {
    const u4v u = __builtin_bit_cast(u4v, v);
    unsigned bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) bits |= (u[i] & 0x7F807F80u) + 0x00800080u;
    return (bits & 0x80008000u) != 0;
}

// Full segment e of the call belongs to the last sequence that starts at or
// before it, cu[s] / lseg <= e (of sequences with equal quotients only the last
// can be a segment long, so no two claim the same e; some e have no segment).
__device__ __forceinline__ int full_owner(const ScanParams &a, int e, int lane) {
    int lo = 0, n = a.r.batch;   // the answer is in lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int s = lo + lane * step;
        const bool le = lane * step < n && a.r.cu[s] / a.lseg <= e;
        const uint64_t m = __ballot(le);
        const int k = m ? 63 - __builtin_clzll(m) : 0;
        n = n - k * step < step ? n - k * step : step;
        lo += k * step;
    }
    return lo;
}

// Sequences end in a rest shorter than a segment.  The j-th rest to run: of
// each kRestBlock sequences the longest first, by eighths of a segment.
constexpr int kRestBlock = 256;
__device__ __forceinline__ int rest_owner(const ScanParams &a, int j, int lane) {
    const int s0 = j / kRestBlock * kRestBlock;
    j -= s0;
    int cls[kRestBlock / 64];
#pragma unroll
    for (int i = 0; i < kRestBlock / 64; ++i) {
        const int s = s0 + 64 * i + lane;
        cls[i] = -1;
        if (s < a.r.batch) {
            const int len = (int)((unsigned)a.r.cu[s + 1] - (unsigned)a.r.cu[s]);
            cls[i] = len > 0 ? (int)((unsigned)(len % a.lseg) / (unsigned)(a.lseg / 8)) : 0;
        }
    }
    for (int c = 7; c >= 0; --c)
#pragma unroll
        for (int i = 0; i < kRestBlock / 64; ++i) {
            const uint64_t m = __ballot(cls[i] == c);
            const int n = __popcll(m);
            if (j < n) {
                const int rank = __builtin_amdgcn_mbcnt_hi((unsigned)(m >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)m, 0));
                return s0 + 64 * i + __builtin_ctzll(__ballot(cls[i] == c && rank == j));
            }
            j -= n;
        }
    return 0;   // not reached: every sequence has a class
}

// Four consecutive floats as NP planes of four bf16; a non-finite value goes to
// plane 0 alone.
template <int NP>
__device__ __forceinline__ void planes(f4v v, u2v (&part)[NP]) {
#pragma unroll
    for (int k = 0; k < NP; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            part[k][i] = __builtin_bit_cast(unsigned, __builtin_convertvector(f2v{v[2 * i], v[2 * i + 1]}, b2v));
            const float r0 = v[2 * i] - __uint_as_float(part[k][i] << 16);
            const float r1 = v[2 * i + 1] - __uint_as_float(part[k][i] & 0xFFFF0000u);
            v[2 * i] = fabsf(r0) < __builtin_inff() ? r0 : 0.f;
            v[2 * i + 1] = fabsf(r1) < __builtin_inff() ? r1 : 0.f;
        }
}

// TIn: uint16_t (bf16) or float inputs; YP: bf16 parts of M, the state and fp32
// inputs in y; OUT: outputs wanted; LOCAL: the first launch, which leaves the
// end states of segments with a successor.
template <typename TIn, typename TY, int YP, bool OUT, bool LOCAL, int NH>
__global__ void __launch_bounds__(128 * NH, sizeof(TIn) == 2 && NH == 4 ? 2 : 1) scan_kernel(ScanParams a) {
    constexpr int NP = sizeof(TIn) == 2 ? 1 : 3;
    constexpr int NPY = NP == 1 ? 1 : YP;   // planes that count in y
    __shared__ ScanSmem<NH, NP> sm;
    constexpr int kWaves = 2 * NH, kThreads = 64 * kWaves;
    const ReplayParams &r = a.r;
    const int lane = threadIdx.x & 63, c = lane & 31, hf = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int hpg = r.H / r.G;

    if (!LOCAL && blockIdx.x == 0)   // offsets that do not ascend (the mapping below stays within the tensors)
        for (int i = threadIdx.x; i <= r.batch; i += kThreads)
            if (r.cu[i] < 0 || r.cu[i] > r.total || (i && r.cu[i] < r.cu[i - 1])) atomicOr(r.err, kErrSeq);

    if (LOCAL && blockIdx.x == 0 && threadIdx.x == 0) *a.marked = 0;

    // Workgroups of one (segment, group) read the same B and C: they follow
    // each other on one XCD, and the pairs are dealt to the XCDs in turn.
    const int npair = (LOCAL ? a.nfull : a.nfull + r.batch) * r.G;
    const int xcd = blockIdx.x & 7, at = blockIdx.x >> 3;
    const int pair = (at / a.hb) * 8 + xcd, hblk = at % a.hb;
    if (pair >= npair) return;
    const int entry = pair / r.G, g = pair - entry * r.G;

    // Full segments first, then the rests.
    const bool full = entry < a.nfull;
    const int seq = __builtin_amdgcn_readfirstlane(full ? full_owner(a, entry, lane) : rest_owner(a, entry - a.nfull, lane));
    const int start = __builtin_amdgcn_readfirstlane(r.cu[seq]), end = __builtin_amdgcn_readfirstlane(r.cu[seq + 1]);
    if (start < 0 || end > r.total || end <= start) return;
    const int k = full ? entry - start / a.lseg : (end - start) / a.lseg;
    if (k < 0 || (int64_t)(k + full) * a.lseg > end - start) return;
    const int tok0 = start + k * a.lseg;
    const int len = full ? a.lseg : end - tok0;
    if (len == 0) return;   // a sequence of whole segments has no rest
    const bool last = tok0 + len == end;
    if (LOCAL && last) return;
    const int b = __builtin_amdgcn_readfirstlane(slot_of_row(r, seq));
    if (b < 0) return;   // padding row

    const int hh = wave >> 1;                  // the wave's head among the workgroup's
    const int hl = hblk * NH + hh;             // ... within the group
    const bool live = hl < hpg;                // waves past the group's heads run its last head again, unseen
    const int h = g * hpg + (live ? hl : hpg - 1);
    const int p0 = (wave & 1) * 32;            // the wave's state rows
    const int prow = p0 + (c & 16) + 4 * swapped((c >> 2) & 3) + (c & 3);   // ... and the lane's
    const size_t HP = (size_t)r.H * kP, GN = (size_t)r.G * kN;

    // ---- state before the segment: value i of tile nt is S[prow][32 nt + 16 (i / 8) + 8 hf + i mod 8]
    f16v st0 = (f16v)0.f, st1 = (f16v)0.f, st2 = (f16v)0.f, st3 = (f16v)0.f;
    const size_t cell = (size_t)prow * kN + 8 * hf;
    auto add_state = [&](const float *s, float f) {
        add_tile(st0, s + cell, f);
        add_tile(st1, s + cell + 32, f);
        add_tile(st2, s + cell + 64, f);
        add_tile(st3, s + cell + 96, f);
    };
    auto put_state = [&](float *s) {
        put_tile(st0, s + cell);
        put_tile(st1, s + cell + 32);
        put_tile(st2, s + cell + 64);
        put_tile(st3, s + cell + 96);
    };
    const size_t headN = (size_t)kP * kN;
    float *ckpt = r.ckpt + ((size_t)b * r.H + h) * headN;
    const size_t ent0 = (size_t)(start / a.lseg);   // the sequence's first full segment in the workspace
    const bool fresh = r.fresh ? r.fresh[seq] != 0 : r.from_zero != 0;
    float *start_copy = a.s0 + (ent0 * r.H + h) * headN;
    if (k == 0 && !fresh && (LOCAL || last) && threadIdx.x == 0 && r.pos[b] != 0) atomicOr(r.err, kErrPos);   // buffer not empty
    if (LOCAL) {
        // joined at the end
    } else if (k == 0) {
        if (!fresh) add_state(last ? ckpt : start_copy, 1.f);
    } else {
        // a factor of exactly zero ends the sum: nothing before it counts
        float f = 1.f;
        for (int i = k - 1; i >= 0 && f != 0.f; --i) {
            const size_t e = (ent0 + i) * r.H + h;
            add_state(a.loc + e * headN, f);
            f *= a.lam[e];
        }
    }

    const TIn *xin = reinterpret_cast<const TIn *>(r.x) + (size_t)tok0 * HP + (size_t)h * kP;
    const TIn *Bin = reinterpret_cast<const TIn *>(r.Bm) + (size_t)tok0 * GN + (size_t)g * kN;
    const TIn *Cin = reinterpret_cast<const TIn *>(r.Cm) + (size_t)tok0 * GN + (size_t)g * kN;
    const TIn *dtin = reinterpret_cast<const TIn *>(r.dt) + (size_t)tok0 * r.H + h;
    TY *yout = reinterpret_cast<TY *>(r.y) + (size_t)tok0 * HP + (size_t)h * kP + p0;
    const auto scalar = [](float v) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v))); };
    const float Ah = scalar(r.A[h]), Dh = scalar(r.D[h]);

    // ---- staging: a wave's load covers 4 rows of B or C (lane: row lane / 16,
    // piece lane mod 16) or 8 rows of x (row lane / 8, piece lane mod 8).  The
    // chunk's first row is the (uniform) base; rows past the segment fall
    // outside the buffer resource and arrive as zeros.
    const int bpitch = (int)GN * (int)sizeof(TIn), xpitch = (int)HP * (int)sizeof(TIn);
    auto rows_left = [&](int t0) {   // (a vector clamp would make the resources vector values)
        return __builtin_amdgcn_readfirstlane(t0 < 0 || t0 > len ? 0 : (len - t0 < kQ ? len - t0 : kQ));
    };
    auto fetch_bc = [&](int t0, int buf) {
        const int rem = rows_left(t0);
        const u4v bs = resource_of(Bin + (size_t)t0 * GN, rem * bpitch);
        const u4v cs = resource_of(Cin + (size_t)t0 * GN, OUT ? rem * bpitch : 0);
        auto &ch = sm.chunk[buf];
        const int l = lane_again(), bl = l >> 4;
        const int boff = bl * bpitch + 16 * ((l & 15) ^ (2 * bl));
#pragma unroll
        for (int n = 0; n < 16 / kWaves; ++n) {   // rows 4 i + bl: an odd i turns the pairs by 4 more
            const int i = wave * (16 / kWaves) + n;
            const int off = (boff ^ (128 * (i & 1))) + 4 * i * bpitch;
            load_to_lds(bs, off, lds_offset(ch.B[0][4 * i]));
            if (OUT) load_to_lds(cs, off, lds_offset(ch.C[0][4 * i]));
        }
    };
    auto fetch_x = [&](int t0, int buf, int n0, int n1) {
        const u4v xs = resource_of(xin + (size_t)t0 * HP, rows_left(t0) * xpitch);
        auto &ch = sm.chunk[buf];
        const int l = lane_again(), xl = l >> 3;
        const int xoff = xl * xpitch + 16 * ((l & 7) ^ (2 * ((xl >> 1) & 3)));
#pragma unroll
        for (int n = n0; n < n1; ++n) {   // a head's two waves take half of its rows each
            const int i = (wave & 1) * 4 + n;
            load_to_lds(xs, xoff + 8 * i * xpitch, lds_offset(ch.x[0][hh][8 * i]));
        }
    };
    // fp32 inputs: through registers, one chunk ahead, and split into planes on
    // the way to LDS.  A thread takes pieces of four floats: 2048 of B and of C
    // over the workgroup, 1024 of a head's x over its two waves.
    constexpr int kBC = NP == 1 ? 1 : 2048 / kThreads, kX = NP == 1 ? 1 : 8;
    f4v rB[kBC], rC[kBC], rX[kX];
    auto fetch32 = [&](int t0) {
        const int rem = rows_left(t0);
        const auto bs = uniform_rsrc(Bin + (size_t)t0 * GN, rem * bpitch);
        const auto cs = uniform_rsrc(Cin + (size_t)t0 * GN, OUT ? rem * bpitch : 0);
        const auto xs = uniform_rsrc(xin + (size_t)t0 * HP, rem * xpitch);
#pragma unroll
        for (int n = 0; n < kBC; ++n) {
            const int i = (int)threadIdx.x + n * kThreads, off = (i >> 5) * bpitch + 16 * (i & 31);
            rB[n] = __builtin_amdgcn_raw_buffer_load_b128(bs, off, 0, 0);
            if (OUT) rC[n] = __builtin_amdgcn_raw_buffer_load_b128(cs, off, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < kX; ++n) {
            const int i = ((int)threadIdx.x & 127) + n * 128;
            rX[n] = __builtin_amdgcn_raw_buffer_load_b128(xs, (i >> 4) * xpitch + 16 * (i & 15), 0, 0);
        }
    };
    auto stage32 = [&]() {
        auto &ch = sm.chunk[0];
#pragma unroll
        for (int n = 0; n < kBC; ++n) {
            const int i = (int)threadIdx.x + n * kThreads, row = i >> 5, at = 32 * (((i >> 2) & 7) ^ (row & 7)) + 8 * (i & 3);
            u2v part[NP];
            planes<NP>(rB[n], part);
#pragma unroll
            for (int k = 0; k < NP; ++k) *reinterpret_cast<u2v *>(&ch.B[k][row][at]) = part[k];
            if (OUT) {
                planes<NP>(rC[n], part);
#pragma unroll
                for (int k = 0; k < NPY; ++k) *reinterpret_cast<u2v *>(&ch.C[k][row][at]) = part[k];
            }
        }
#pragma unroll
        for (int n = 0; n < kX; ++n) {
            const int i = ((int)threadIdx.x & 127) + n * 128, row = i >> 4;
            u2v part[NP];
            planes<NP>(rX[n], part);
#pragma unroll
            for (int k = 0; k < NP; ++k)
                *reinterpret_cast<u2v *>(&ch.x[k][hh][row][32 * (((i >> 2) & 3) ^ ((row >> 1) & 3)) + 8 * (i & 3)]) = part[k];
        }
    };
    // dt of the lane's token in the chunk at t0
    auto fetch_dt = [&](int t0) -> unsigned {
        const int pitch = r.H * (int)sizeof(TIn);
        const auto ds = uniform_rsrc(dtin + (size_t)t0 * r.H, rows_left(t0) * pitch);
        if constexpr (NP == 1) return __builtin_amdgcn_raw_buffer_load_b16(ds, lane_again() * pitch, 0, 0);
        else return __builtin_amdgcn_raw_buffer_load_b32(ds, lane_again() * pitch, 0, 0);
    };

    // The first launch takes the chunks from the last to the first, each with
    // its decay to the segment's end (`total`): the accumulators are never
    // rescaled, and once a head's decay is exactly zero in fp32 its earlier
    // tokens are not taken at all.
    constexpr int kStep = LOCAL ? -kQ : kQ;
    const int t_first = LOCAL ? (len - 1) / kQ * kQ : 0;
    double total = 0.0;
    if constexpr (NP == 1) {
        fetch_bc(t_first, 0);
        fetch_x(t_first, 0, 0, 4);
    } else fetch32(t_first);
    unsigned dt_bits = fetch_dt(t_first);
    if (OUT)   // the quarters above the diagonal
        for (int i = threadIdx.x; i < 128; i += kThreads) {
            const int t = (i >> 2) & 15, q = 4 + (i & 3);
            *reinterpret_cast<f4v *>(&sm.gram[2 * (i >> 6)][t][4 * (q ^ (t & 7))]) = (f4v)0.f;
        }
    int buf = 0;
    for (int t0 = t_first; LOCAL ? t0 >= 0 : t0 < len; t0 += kStep, buf ^= NP == 1) {
        const int q = len - t0 < kQ ? len - t0 : kQ;   // tokens of this chunk
        // The chunk has arrived (every wave waits for its own loads) and the
        // other buffer's reads are done: the next chunk goes there.
        const bool done = LOCAL && __builtin_amdgcn_exp2f((float)total) == 0.f;
        if (LOCAL && lane == 0) sm.done[buf][wave] = done;
        asm volatile("s_waitcnt vmcnt(0)" : "+v"(dt_bits)::"memory");   // (dt too: not waited for behind the next loads)
        const float dt = __uint_as_float(NP == 1 ? dt_bits << 16 : dt_bits);
        __syncthreads();
        if (LOCAL) {
            int all = 1;
#pragma unroll
            for (int i = 0; i < kWaves; ++i) all &= sm.done[buf][i];
            if (__builtin_amdgcn_readfirstlane(all)) break;
        }
        if constexpr (NP == 1) {
            fetch_bc(t0 + kStep, buf ^ 1);
            if (!OUT) fetch_x(t0 + kStep, buf ^ 1, 0, 4);   // (with outputs, between their products)
        } else {   // one buffer: its reads are done, and it is written before the next reads
            stage32();
            __syncthreads();
            fetch32(t0 + kStep);
        }
        if (LOCAL && done) {
            dt_bits = 0;
            continue;
        }
        __builtin_amdgcn_sched_barrier(0);
        // A wave's priority falls as it moves through its chunk, so that of the
        // two on a SIMD the one behind, with products to issue, goes first and
        // the other's vector work fills in.
        __builtin_amdgcn_s_setprio(3);
        // ---- operand addresses within the chunk's buffer
        const int ln = lane_again(), col = ln & 31, half = ln >> 5, row4 = 4 * half;
        const int get_r = 256 * col + 16 * half + 32 * (col & 7);   // row col of B, C: ^ 32 ks
        // transposing reads: row tr of a quarter wave's four, column quad tc, 16-column half tg
        const int tr = (ln >> 2) & 3, tc = 8 * swapped(ln & 3), tg = (ln >> 4) & 1, tj = row4 + tr;
        const int get_b = 256 * tj + 32 * (tg ^ tj) + tc;                                       // ^ 64 nt, + 4096 js
        const int get_x = 128 * tj + 32 * ((2 * (wave & 1) + tg) ^ ((tj >> 1) & 3)) + tc;       // + 2048 js
        const int get_y = 128 * col + 32 * ((2 * (wave & 1)) ^ ((col >> 1) & 3)) + 16 * half;   // row col of x: ^ 32 s
        const int yoff = (col * (int)HP + 8 * half) * (int)sizeof(TY);
        const char *ldsB = sm.chunk[buf].B[0][0], *ldsC = sm.chunk[buf].C[0][0], *ldsX = sm.chunk[buf].x[0][hh][0];
        constexpr int kPlane = 2 * kN * kQ, kPlaneX = 2 * kP * kQ * NH;   // bytes from plane to plane

        // ---- decays of the wave's head (both waves of a head compute them).
        // exp(c_t - c_j) = 2^(k_t - k_j) 2^f_t 2^-f_j: the fractions' powers
        // are taken once per token, the whole part moves an exponent exactly.
        float lam;
        auto decays = [&]() {
            float A = Ah;
            asm volatile("" : "+s"(A));   // (its product is not held in vector registers)
            // (a token's decay below 2^-2^20 is zero either way; kept there, the whole parts of 64 tokens fit an int)
            double log2a = (double)A * 1.4426950408889634 * (double)dt;
            log2a = log2a < -0x1p20 && fabsf(dt) < __builtin_inff() ? -0x1p20 : log2a;
            const double cum = prefix(log2a), whole = __builtin_floor(cum);
            const double c63 = lane_d(cum, 63);
            const float f = (float)(cum - whole);
            if (OUT) {
                sm.k[wave][ln] = (int)whole;
                // (from a non-finite dt on 2^f_t is NaN and y with it; its factor stays out of earlier tokens' 0 M)
                const float cf = dt * __builtin_amdgcn_exp2f(-f);
                sm.cf[wave][ln] = fabsf(cf) < __builtin_inff() ? cf : 0.f;
                sm.rf[wave][ln] = __builtin_amdgcn_exp2f(f);
            }
            sm.w[wave][ln] = dt * __builtin_amdgcn_exp2f((float)(total + c63 - cum));   // (total: 0 but in LOCAL)
            lam = __builtin_amdgcn_exp2f((float)c63);
            if (LOCAL) total += c63;
            __builtin_amdgcn_wave_barrier();
        };
        if (!OUT) decays();

        unsigned bad_row = 0;   // the lane's row has a non-finite x in this chunk
        if (OUT) {
            // ---- the Gram tiles, the same for every head: 10 pieces of 16 x 16 over the waves
            const int get_g = 256 * (ln & 15) + 16 * ((ln >> 4) & 1) + 32 * ((ln >> 5) ^ (ln & 7));
            b8v gb[4][NPY], gc[4][NPY];
            auto get_gram = [&](int jt, int tt) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                    for (int k = 0; k < NPY; ++k) {
                        gb[ks][k] = operand(ldsB + (get_g ^ (64 * ks)) + 4096 * jt + k * kPlane);
                        gc[ks][k] = operand(ldsC + (get_g ^ (64 * ks)) + 4096 * tt + k * kPlane);
                    }
                if (NP == 1) __builtin_amdgcn_sched_barrier(0);
            };
            auto put_gram = [&](int jt, int tt) {
                f4v g = (f4v)0.f;
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                    for (int k = NPY - 1; k >= 0; --k)
#pragma unroll
                        for (int i = NPY - 1 - k; i >= 0; --i) g = mfma16(gb[ks][k], gc[ks][i], g);
                const int t = ln & 15, j = 4 * (ln >> 4);   // within the piece: the lane's t, its first j
                if (jt == tt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) g[i] = j + i <= t ? g[i] : 0.f;
                *reinterpret_cast<f4v *>(&sm.gram[(tt >> 1) + (jt >> 1)][16 * (tt & 1) + t][4 * ((4 * (jt & 1) + (ln >> 4)) ^ (t & 7))]) = g;
            };
            for (int u = wave; u < 10; u += kWaves) {
                const int tt = (u >= 1) + (u >= 3) + (u >= 6), jt = u - tt * (tt + 1) / 2;
                if (NP == 1) get_gram(jt, tt);
                if (u == wave) decays();   // while the operands come
                if (NP != 1) get_gram(jt, tt);
                put_gram(jt, tt);
            }
            // ---- y^T[p][t] = sum_n S[p][n] C_t[n]
            f16v y0 = (f16v)0.f, y1 = (f16v)0.f;
            b8v xr[4], cA[2][NPY], cB[2][NPY], sA[YP], sB[YP];   // operands of one step, and of the next
            auto get_c = [&](int ks, b8v (&c)[2][NPY]) {
                const int off = get_r ^ (32 * ks);
#pragma unroll
                for (int k = 0; k < NPY; ++k) {
                    c[0][k] = operand(ldsC + off + k * kPlane);
                    c[1][k] = operand(ldsC + off + k * kPlane + 32 * 256);
                }
                __builtin_amdgcn_sched_barrier(0);
            };
            // of products of parts i and k, those with i + k < the number of parts count
            auto products = [&](const b8v (&part)[YP], const b8v (&c)[2][NPY]) {
#pragma unroll
                for (int i = YP - 1; i >= 0; --i)
#pragma unroll
                    for (int k = NPY - 1; k >= 0; --k)
                        if (i + k < YP) {
                            y0 = mfma(part[i], c[0][k], y0);
                            y1 = mfma(part[i], c[1][k], y1);
                        }
            };
            // (between two products, a share of the next step's splitting)
            auto mixed = [&]() {
#pragma unroll
                for (int i = 0; i < 2 * YP; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x2, YP == 2 ? 7 : 8, 0);
                }
                asm volatile("" : "+v"(y0), "+v"(y1));   // (no product is put off past its step)
                __builtin_amdgcn_sched_barrier(0);
            };
            get_c(0, cA);
            split<YP>(half_of(st0, 0), sA);
            // every wave's Gram pieces are in LDS (no wait for the next chunk's loads)
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            get_c(1, cB);
            products(sA, cA);
            split<YP>(half_of(st0, 1), sB);
            mixed();
            if constexpr (NP == 1) fetch_x(t0 + kStep, buf ^ 1, 0, 2);
            get_c(2, cA);
            products(sB, cB);
            split<YP>(half_of(st1, 0), sA);
            mixed();
            get_c(3, cB);
            products(sA, cA);
            split<YP>(half_of(st1, 1), sB);
            mixed();
            if constexpr (NP == 1) fetch_x(t0 + kStep, buf ^ 1, 2, 4);
            get_c(4, cA);
            products(sB, cB);
            split<YP>(half_of(st2, 0), sA);
            mixed();
            get_c(5, cB);
            products(sA, cA);
            split<YP>(half_of(st2, 1), sB);
            mixed();
            get_c(6, cA);
            products(sB, cB);
            split<YP>(half_of(st3, 0), sA);
            mixed();
            get_c(7, cB);
            products(sA, cA);
            split<YP>(half_of(st3, 1), sB);
            mixed();
#pragma unroll
            for (int i = 0; i < 4; ++i) xr[i] = operand(ldsX + (get_y ^ (32 * (i & 1))) + 32 * 128 * (i >> 1));
            const int k0 = sm.k[wave][col], k1 = sm.k[wave][32 + col];
            const float r0 = sm.rf[wave][col], r1 = sm.rf[wave][32 + col];
            __builtin_amdgcn_sched_barrier(0);
            products(sB, cB);
            bool odd = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) odd |= non_finite(xr[i]);
            __builtin_amdgcn_s_setprio(2);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                y0[i] = __builtin_ldexpf(y0[i], k0);
                y1[i] = __builtin_ldexpf(y1[i], k1);
            }
            // M_tj = 0 for j > t does not keep a non-finite x_j out of y_t.  A
            // wave that meets one marks the outputs of its row from its token on,
            // notes the row for the state and takes the value out of its half of
            // x (which no other wave reads).
            const int upto = col - row4;
            if (__builtin_amdgcn_ballot_w64(odd) != 0) {
                auto mark = [&](f16v &y, int from) {   // from: token of the lane less row4
                    f16v bad = (f16v)0.f;
                    for (int js = 0; js < 4; ++js) {
                        const u4v v = __builtin_bit_cast(u4v, operand_t<128>(ldsX + get_x + 2048 * js));
                        u4v is, up;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {   // 0x3F80 is 1 in bf16
                            is[i] = ((v[i] & 0x7F80u) == 0x7F80u) * 0x3F80u | ((v[i] & 0x7F800000u) == 0x7F800000u) * 0x3F800000u;
                            const int j = 16 * js + 8 * (i >> 1) + 2 * (i & 1);
                            up[i] = (j <= from) * 0x3F80u | (j < from) * 0x3F800000u;
                            bad_row |= is[i];
                        }
                        bad = mfma(__builtin_bit_cast(b8v, is), __builtin_bit_cast(b8v, up), bad);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)   // (added to, a NaN stays one)
                        if (bad[i] != 0.f) y[i] = __builtin_nanf("");
                    __builtin_amdgcn_sched_barrier(0);
                };
                mark(y0, upto);
                mark(y1, upto + 32);
                bad_row |= __shfl_xor(bad_row, 32);   // a row's tokens are spread over both halves
                for (int i = 0; i < 4; ++i) {
                    const char *p = ldsX + (get_y ^ (32 * (i & 1))) + 32 * 128 * (i >> 1);
                    u4v v = __builtin_bit_cast(u4v, operand(p));
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        v[d] &= ~(((v[d] & 0x7F80u) == 0x7F80u) * 0xFFFFu | ((v[d] & 0x7F800000u) == 0x7F800000u) * 0xFFFF0000u);
                    // (a store the compiler sees would make it wait for the next chunk's loads)
                    typedef __attribute__((address_space(3))) const char lds_char;
                    asm volatile("ds_write_b128 %0, %1" ::"v"((unsigned)(uintptr_t)(lds_char *)p), "v"(v) : "memory");
                }
            }
            // ---- y^T += x^T M^T without D and the factor 2^f_t
            const int get_m = 128 * col + 16 * (half ^ (col & 7));   // row col of a Gram tile: ^ 64 s, second half ^ 32
            struct Factors {   // of 16 tokens j
                f8v cf;
                i8v kj;
                b8v x[NPY];
            } fA, fB;
            f8v gA, gB;
            auto get_f = [&](int js, Factors &f) {
                f.cf = read8(&sm.cf[wave][16 * js + row4]);
                f.kj = read8(&sm.k[wave][16 * js + row4]);
#pragma unroll
                for (int k = 0; k < NPY; ++k) f.x[k] = operand_t<128>(ldsX + get_x + 2048 * js + k * kPlaneX);
            };
            auto get_g8 = [&](int tile, int s) {
                const char *gram = reinterpret_cast<const char *>(sm.gram[tile]);
                const f4v a = *reinterpret_cast<const f4v *>(gram + (get_m ^ (64 * s))),
                          b = *reinterpret_cast<const f4v *>(gram + (get_m ^ (64 * s + 32)));
                return f8v{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            };
            b8v mA[YP], mB[YP];
            auto decayed = [&](f8v m, const Factors &f, int kt, b8v (&part)[YP]) {
#pragma unroll
                for (int i = 0; i < 8; ++i) m[i] = __builtin_ldexpf(m[i] * f.cf[i], kt - f.kj[i]);
                split<YP>(m, part);
            };
            auto apply = [&](const b8v (&part)[YP], const Factors &f, f16v &y) {
#pragma unroll
                for (int k = NPY - 1; k >= 0; --k)
#pragma unroll
                    for (int i = YP - 1 - k; i >= 0; --i) y = mfma(f.x[k], part[i], y);
            };
            auto mixed_apply = [&]() {
#pragma unroll
                for (int i = 0; i < YP; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x2, 16, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            };
            get_f(0, fA);
            gA = get_g8(0, 0);
            gB = get_g8(1, 0);
            __builtin_amdgcn_sched_barrier(0);
            decayed(gA, fA, k0, mA);
            __builtin_amdgcn_sched_barrier(0);
            gA = get_g8(0, 1);
            get_f(1, fB);
            __builtin_amdgcn_sched_barrier(0);
            apply(mA, fA, y0);
            decayed(gB, fA, k1, mB);
            mixed_apply();
            gB = get_g8(1, 1);
            __builtin_amdgcn_sched_barrier(0);
            apply(mB, fA, y1);
            decayed(gA, fB, k0, mA);
            mixed_apply();
            gA = get_g8(2, 0);
            get_f(2, fA);
            __builtin_amdgcn_sched_barrier(0);
            apply(mA, fB, y0);
            decayed(gB, fB, k1, mB);
            mixed_apply();
            gB = get_g8(2, 1);
            __builtin_amdgcn_sched_barrier(0);
            apply(mB, fB, y1);
            get_f(3, fB);
            decayed(gA, fA, k1, mA);
            mixed_apply();
            apply(mA, fA, y1);
            decayed(gB, fB, k1, mB);
            mixed_apply();
            apply(mB, fB, y1);
            __builtin_amdgcn_s_setprio(1);
            // ---- out: y = 2^f_t y + D x; rows past the chunk (and an unseen head's) fall outside the resource
            const auto ys = uniform_rsrc(yout + (size_t)t0 * HP, live ? q * (int)HP * (int)sizeof(TY) : 0);
            auto store = [&](const f16v &y, float rt, int tt) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    f8v x = vec8<uint16_t>::widen(__builtin_bit_cast(u4u, operand(ldsX + (get_y ^ (32 * s)) + 32 * 128 * tt)));
#pragma unroll
                    for (int k = 1; k < NPY; ++k)
                        x += vec8<uint16_t>::widen(
                            __builtin_bit_cast(u4u, operand(ldsX + (get_y ^ (32 * s)) + 32 * 128 * tt + k * kPlaneX)));
                    f8v v = half_of(y, s);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = fmaf(Dh, x[i], v[i] * rt);
                    const int at = yoff + (32 * tt * (int)HP + 16 * s) * (int)sizeof(TY);
                    if constexpr (sizeof(TY) == 4) {
                        __builtin_amdgcn_raw_buffer_store_b128(f4v{v[0], v[1], v[2], v[3]}, ys, at, 0, 0);
                        __builtin_amdgcn_raw_buffer_store_b128(f4v{v[4], v[5], v[6], v[7]}, ys, at + 16, 0, 0);
                    } else {
                        b8v o[1];
                        split<1>(v, o);
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4v, o[0]), ys, at, 0, 0);
                    }
                }
            };
            store(y0, r0, 0);
            store(y1, r1, 1);
        }

        __builtin_amdgcn_s_setprio(0);
        // the next chunk's dt, now that the accumulators of y and the Gram tiles are free
        dt_bits = fetch_dt(t0 + kStep);

        // ---- S^T[n][p] = exp(c_63) S^T + sum_j B_j[n] (w_j x_j[p])
        struct Weighted {
            b8v x[NP];
            f8v w;
        } wA, wB;
        struct Rows {
            b8v b[4];
        } rA, rB;
        b8v pA[3], pB[3];
        auto get_w = [&](int js, Weighted &f) {
#pragma unroll
            for (int k = 0; k < NP; ++k) f.x[k] = operand_t<128>(ldsX + get_x + 2048 * js + k * kPlaneX);
            f.w = read8(&sm.w[wave][16 * js + row4]);
        };
        auto get_rows = [&](int js, int k, Rows &f) {
            const char *pb = ldsB + 4096 * js + k * kPlane;
#pragma unroll
            for (int i = 0; i < 4; ++i) f.b[i] = operand_t<256>(pb + (get_b ^ (64 * i)));
        };
        auto weigh = [&](const Weighted &f, b8v (&part)[3]) {
            f8v v = vec8<uint16_t>::widen(__builtin_bit_cast(u4u, f.x[0]));
#pragma unroll
            for (int k = 1; k < NP; ++k) v += vec8<uint16_t>::widen(__builtin_bit_cast(u4u, f.x[k]));
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= f.w[i];
            split<3>(v, part);
        };
        auto add = [&](int k, const b8v (&part)[3], const Rows &f) {
#pragma unroll
            for (int i = 2 - k; i >= 0; --i) {
                st0 = mfma(f.b[0], part[i], st0);
                st1 = mfma(f.b[1], part[i], st1);
                st2 = mfma(f.b[2], part[i], st2);
                st3 = mfma(f.b[3], part[i], st3);
            }
        };
        auto mixed_add = [&]() {   // between two products, a share of the next tokens' weighing
#pragma unroll
            for (int i = 0; i < 12; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x2, 5, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        get_w(0, wA);
        if constexpr (NP == 1) {
            get_rows(0, 0, rA);
            get_w(1, wB);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (!LOCAL)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                st0[i] *= lam;
                st1[i] *= lam;
                st2[i] *= lam;
                st3[i] *= lam;
            }
        weigh(wA, pA);
        if constexpr (NP == 1) {
            get_rows(1, 0, rB);
            get_w(2, wA);
            __builtin_amdgcn_sched_barrier(0);
            add(0, pA, rA);
            weigh(wB, pB);
            mixed_add();
            get_rows(2, 0, rA);
            get_w(3, wB);
            __builtin_amdgcn_sched_barrier(0);
            add(0, pB, rB);
            weigh(wA, pA);
            mixed_add();
            get_rows(3, 0, rB);
            __builtin_amdgcn_sched_barrier(0);
            add(0, pA, rA);
            weigh(wB, pB);
            mixed_add();
            add(0, pB, rB);
        } else {
#pragma unroll
            for (int js = 0; js < 4; ++js) {
                if (js) {
                    get_w(js, wA);
                    weigh(wA, pA);
                }
#pragma unroll
                for (int k = NP - 1; k >= 0; --k) {
                    get_rows(js, k, rA);
                    add(k, pA, rA);
                }
            }
        }
        if (OUT && __builtin_amdgcn_ballot_w64(bad_row != 0) != 0) {
            if (bad_row) st0 = st1 = st2 = st3 = (f16v)__builtin_nanf("");
        }
    }

    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // loads to LDS still in flight
    if (LOCAL) {
        const size_t e = (ent0 + k) * r.H + h;
        const float lam = __builtin_amdgcn_exp2f((float)total);
        if (k == 0 && !fresh) {
            // the second launch rewrites the checkpoint, so its first segment reads a copy
            copy_tile(ckpt + cell, start_copy + cell, live);
            copy_tile(ckpt + cell + 32, start_copy + cell + 32, live);
            copy_tile(ckpt + cell + 64, start_copy + cell + 64, live);
            copy_tile(ckpt + cell + 96, start_copy + cell + 96, live);
            if (lam != 0.f) add_state(ckpt, lam);
        }
        if (live) {
            put_state(a.loc + e * headN);
            if ((wave & 1) == 0 && lane == 0) a.lam[e] = lam;
        }
    } else if (last) {
        if (live) put_state(ckpt);
        publish_position(r, b, 0, true, -1);
    } else if (live) {
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            odd |= !(fabsf(st0[i]) < __builtin_inff()) || !(fabsf(st1[i]) < __builtin_inff()) ||
                   !(fabsf(st2[i]) < __builtin_inff()) || !(fabsf(st3[i]) < __builtin_inff());
        const size_t e = (ent0 + k) * r.H + h;
        const bool mark = __builtin_amdgcn_ballot_w64(odd) != 0;
        if (mark) put_state(a.s0 + e * headN);   // (the copy of the start state there has been read)
        if (lane == 0) {
            a.mark[2 * e + (wave & 1)] = mark;
            if (mark) *a.marked = 1;
        }
    }
}

// The piece behind full segment `entry`, eight heads of it: rows whose state was
// not finite at the end of any of the sequence's segments so far get NaN outputs,
// and where the piece is the last one the state's elements get NaN.
constexpr int kMarkHeads = 8;

template <typename TY>
__global__ void __launch_bounds__(256) carry_non_finite_kernel(ScanParams a) {
    if (*a.marked == 0) return;
    __shared__ int bad[kP];
    const ReplayParams &r = a.r;
    const int nblk = (r.H + kMarkHeads - 1) / kMarkHeads;
    const int entry = blockIdx.x / nblk, h0 = (blockIdx.x - entry * nblk) * kMarkHeads;
    const int h1 = h0 + kMarkHeads < r.H ? h0 + kMarkHeads : r.H;
    const int seq = full_owner(a, entry, threadIdx.x & 63);
    const int start = r.cu[seq], end = r.cu[seq + 1];
    if (start < 0 || end > r.total || end <= start) return;
    const int ent0 = start / a.lseg, k = entry - ent0;
    if (k < 0 || (int64_t)(k + 1) * a.lseg >= end - start) return;   // no such segment, or nothing behind it
    const int b = slot_of_row(r, seq);
    if (b < 0) return;   // padding row
    const int per = 2 * (h1 - h0);   // marks of a segment
    int any = 0;
    for (int i = threadIdx.x; i < (k + 1) * per; i += 256)
        any |= a.mark[2 * ((size_t)(ent0 + i / per) * r.H + h0) + i % per];
    if (!__syncthreads_or(any)) return;

    const int tok0 = start + (k + 1) * a.lseg;
    const int len = end - tok0 < a.lseg ? end - tok0 : a.lseg;
    const bool last = tok0 + len == end;
    for (int h = h0; h < h1; ++h) {
        if (threadIdx.x < kP) bad[threadIdx.x] = 0;
        __syncthreads();
        float *ckpt = r.ckpt + ((size_t)b * r.H + h) * (kP * kN);
        for (int i = 0; i <= k; ++i) {
            const size_t e = (size_t)(ent0 + i) * r.H + h;
            for (int half = 0; half < 2; ++half)
                if (a.mark[2 * e + half])
                    for (int at = half * 32 * kN + threadIdx.x; at < (half + 1) * 32 * kN; at += 256)
                        if (!(fabsf(a.s0[e * (kP * kN) + at]) < __builtin_inff())) {
                            bad[at / kN] = 1;
                            if (last && fabsf(ckpt[at]) < __builtin_inff()) ckpt[at] = __builtin_nanf("");
                        }
        }
        __syncthreads();
        if (r.y) {
            TY *y = reinterpret_cast<TY *>(r.y) + ((size_t)tok0 * r.H + h) * kP;
            for (int64_t i = threadIdx.x; i < (int64_t)len * kP; i += 256)
                if (bad[i % kP]) vec8<TY>::put(y + i / kP * ((size_t)r.H * kP) + i % kP, __builtin_nanf(""));
        }
        __syncthreads();
    }
}

int64_t scan_blocks(const ScanParams &a, int segments) {   // of each (segment, group), in whole rounds over the XCDs
    return ((int64_t)segments * a.r.G + 7) / 8 * 8 * a.hb;
}

template <typename TIn, int NH>
void launch_heads(const ScanParams &a, bool outputs, hipStream_t s) {
    const dim3 block(128 * NH), grid(scan_blocks(a, a.nfull + a.r.batch));
    if (a.nfull)
        hipLaunchKernelGGL((scan_kernel<TIn, float, 3, false, true, NH>), dim3(scan_blocks(a, a.nfull)), block, 0, s, a);
    if (!outputs) hipLaunchKernelGGL((scan_kernel<TIn, float, 3, false, false, NH>), grid, block, 0, s, a);
    else if (a.r.y_bf16) hipLaunchKernelGGL((scan_kernel<TIn, uint16_t, 2, true, false, NH>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((scan_kernel<TIn, float, 3, true, false, NH>), grid, block, 0, s, a);
    if (!a.nfull) return;
    const dim3 marks(a.nfull * ((a.r.H + kMarkHeads - 1) / kMarkHeads));
    if (a.r.y_bf16) hipLaunchKernelGGL(carry_non_finite_kernel<uint16_t>, marks, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(carry_non_finite_kernel<float>, marks, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_scan(const ReplayParams &p, bool in_bf16, bool outputs, void *workspace, hipStream_t s) {
    if (p.batch == 0 || p.total == 0) return hipSuccess;
    ScanParams a{};
    a.r = p;
    a.lseg = scan_segment(p.total, p.batch, p.H, p.G, in_bf16);
    a.nfull = (int)(p.total / a.lseg);
    if (!workspace || a.nfull == 0) {   // one segment per sequence
        a.lseg = (int)((p.total + kScanChunk) / kScanChunk * kScanChunk);
        a.nfull = 0;
    } else {
        a.loc = static_cast<float *>(workspace);
        a.s0 = a.loc + (size_t)a.nfull * p.H * kP * kN;
        a.lam = a.s0 + (size_t)a.nfull * p.H * kP * kN;
        a.mark = reinterpret_cast<int *>(a.lam + (size_t)a.nfull * p.H);
        a.marked = a.mark + (size_t)a.nfull * p.H * 2;
    }
    const int nh = scan_heads(p.H / p.G, in_bf16);
    a.hb = (p.H / p.G + nh - 1) / nh;
    a.r.wg_per_slot = p.G * a.hb;
    if (scan_blocks(a, a.nfull + p.batch) > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (nh == 4) launch_heads<uint16_t, 4>(a, outputs, s);
    else if (nh == 2 && in_bf16) launch_heads<uint16_t, 2>(a, outputs, s);
    else if (nh == 2) launch_heads<float, 2>(a, outputs, s);
    else if (in_bf16) launch_heads<uint16_t, 1>(a, outputs, s);
    else launch_heads<float, 1>(a, outputs, s);
    return hipGetLastError();
}

}  // namespace rssm
