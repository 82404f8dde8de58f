// scan_kernels.hip -- packed prompts through the recurrence on the matrix
// cores (bf16 inputs, fp32 checkpoints).
//
// A sequence is taken in chunks of 64 tokens.  With l_i = A dt_i, c_t the sum
// of l over the chunk up to t, and S the state before the chunk:
//     M_tj = (C_t . B_j) dt_j exp(c_t - c_j)  for j <= t, plus D at j = t
//     y_t  = sum_j M_tj x_j + exp(c_t) S C_t
//     S'   = exp(c_63) S + sum_j dt_j exp(c_63 - c_j) x_j (outer) B_j
// One wave owns 32 of the 64 state rows p of a head and keeps its half of the
// state, transposed [n][p], in the accumulators of v_mfma_f32_32x32x16_bf16
// for the whole segment.  An accumulator holds 4 consecutive rows per lane
// half, a matrix operand 8; the products' inner index may run in any order, so
// every operand in LDS is stored with quads 1 and 2 of each 16 exchanged and
// accumulators (the state for S C, the decayed Gram tile for M x) feed the
// next product straight from registers.
//
// Precision.  x, B, C are bf16 and exact operands.  Values formed in fp32
// (state, M, weighted x) are split into bf16 parts, v = hi + mid + lo, and
// multiplied part by part into the same fp32 accumulator: three parts carry
// all 24 bits, two carry 16.  The state always uses three, so it is as exact
// as an fp32 update; y uses three for fp32 outputs and two for bf16 ones,
// whose own rounding is 2^-8.  Decay sums run in fp64 and are kept as two
// floats: a difference of two long sums would otherwise lose the bits of a
// short one.
//
// Long sequences.  When sequences x heads do not fill the card, a sequence is
// cut into segments: a first launch leaves each segment's end state (the first
// from the slot's state, the others from zero), and in the second every
// segment joins the states before it, S = loc_{k-1} + lam_{k-1} (loc_{k-2} +
// ...), before it runs its tokens.
#include "device_common.h"
#include "mixer_device.h"
#include "replay_common.h"
#include "scan.h"

namespace rssm {
namespace {

constexpr int kQ = kScanChunk;
constexpr int kRowN = 136;   // elements of an LDS row of 128: 16 bytes more, so that 16 rows start in different banks
constexpr int kRowQ = 64;    // elements of an LDS row of 64, its 16-byte pieces exchanged by row (see piece)

typedef float f16v __attribute__((ext_vector_type(16)));
typedef unsigned int u2v __attribute__((ext_vector_type(2)));

struct ScanSmem {
    alignas(16) uint16_t B[kQ][kRowN];    // B_j[n], n exchanged
    alignas(16) uint16_t C[kQ][kRowN];    // C_t[n], n exchanged
    alignas(16) uint16_t BT[kN][kRowQ];   // B_j[n] as [n][j], j exchanged
    alignas(16) uint16_t XT[kScanHeads][kP][kRowQ];   // x_j[p] as [p][j], j exchanged
    // per wave, with c_t / ln 2 = k_t + f_t, k_t whole and 0 <= f_t < 1:
    alignas(16) int k[4][kQ];
    alignas(16) float cf[4][kQ];          // dt_j 2^-f_j
    alignas(16) float w[4][kQ];           // dt_j exp(c_63 - c_j)
    float rf[4][kQ], ri[4][kQ];           // 2^f_t, 2^-f_t
    int bad[2];                           // first token with a non-finite x, of even and odd chunks
};

// Position of quad q (4 elements) among the quads of a row: 1 and 2 of each four exchanged.
__device__ __forceinline__ int quad_at(int q) { return (q & ~3) | ((q & 1) << 1) | ((q >> 1) & 1); }

__device__ __forceinline__ b8v operand(const void *p) {
    return __builtin_bit_cast(b8v, *reinterpret_cast<const f4v *>(p));
}

typedef float f2v __attribute__((ext_vector_type(2)));
typedef __bf16 b2v __attribute__((ext_vector_type(2)));
typedef __bf16 b4v __attribute__((ext_vector_type(4)));

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

__device__ __forceinline__ f8v half_of(const f16v &v, int s) {
    f8v r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[8 * s + i];
    return r;
}

typedef int i8v __attribute__((ext_vector_type(8)));
typedef int i4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i8v read8(const int *p) {   // p[0..3], p[8..11]
    const i4v a = *reinterpret_cast<const i4v *>(p), b = *reinterpret_cast<const i4v *>(p + 8);
    return i8v{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

__device__ __forceinline__ f8v read8(const float *p) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 8);
    return f8v{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// Rows of 64 elements are read 16 consecutive rows at a time (operands) and
// written at every eighth row (transposed staging).  Piece k (16 bytes) of row
// n is kept at k ^ turn(n): both then spread over the banks.  turn(n + 32 m) =
// turn(n) ^ 2 m and, for n a multiple of 8, turn(n + i) = turn(n) ^ (i / 2), so
// an address is one of four lane values plus a constant.
__device__ __forceinline__ int turn(int n) { return ((n >> 1) ^ (n >> 4)) & 7; }

// Byte offset of piece k of row n.
__device__ __forceinline__ int piece_offset(int n, int k) { return 2 * kRowQ * n + 16 * (k ^ turn(n)); }

// Column i of four rows of eight 16-bit values.
template <int I>
__device__ __forceinline__ u2v column(u4v a, u4v b, u4v c, u4v d) {
    constexpr unsigned sel = I & 1 ? 0x07060302 : 0x05040100;
    return u2v{__builtin_amdgcn_perm(b[I / 2], a[I / 2], sel), __builtin_amdgcn_perm(d[I / 2], c[I / 2], sel)};
}

// The four rows' columns 0..7 to LDS rows n .. n + 7; `off` is the offset of
// row n with the quad's position in it.
template <int I = 0>
__device__ __forceinline__ void store_columns(char *m, int off, u4v a, u4v b, u4v c, u4v d) {
    *reinterpret_cast<u2v *>(m + (off ^ (16 * (I / 2))) + 2 * kRowQ * I) = column<I>(a, b, c, d);
    if constexpr (I < 7) store_columns<I + 1>(m, off, a, b, c, d);
}

// A state tile from and to memory: values 4 i .. 4 i + 3 at s + 8 i.
__device__ __forceinline__ void add_tile(f16v &v, const float *s, float f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 u = *reinterpret_cast<const float4 *>(s + 8 * i);
        v[4 * i] += f * u.x;
        v[4 * i + 1] += f * u.y;
        v[4 * i + 2] += f * u.z;
        v[4 * i + 3] += f * u.w;
    }
}

__device__ __forceinline__ void put_tile(const f16v &v, float *s) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4 *>(s + 8 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
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

// An address part that is derived again in every chunk instead of being held
// in a register each (the accumulators need them).
__device__ __forceinline__ int recomputed(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// Last sequence s whose first segment entry, cu[s] / lseg + s, is <= j (the
// entries of a sequence follow it; consecutive sequences never overlap).
__device__ __forceinline__ int segment_owner(const ScanParams &a, int j, int lane) {
    int lo = 0, n = a.r.batch;   // the answer is in lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int s = lo + lane * step;
        const bool le = lane * step < n && a.r.cu[s] / a.lseg + s <= j;
        const uint64_t m = __ballot(le);
        const int k = m ? 63 - __builtin_clzll(m) : 0;
        n = n - k * step < step ? n - k * step : step;
        lo += k * step;
    }
    return lo;
}

// YP: bf16 parts of M and the state in y; OUT: outputs wanted; LOCAL: the
// first launch, which leaves the end states of segments with a successor.
template <typename TY, int YP, bool OUT, bool LOCAL>
__global__ void __launch_bounds__(256, 2) scan_kernel(ScanParams a) {
    __shared__ __attribute__((aligned(16))) ScanSmem sm;
    const ReplayParams &r = a.r;
    const int lane = threadIdx.x & 63, c = lane & 31, hf = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int hpg = r.H / r.G;

    if (!LOCAL && blockIdx.x == 0)   // offsets that do not ascend (the mapping below stays within the tensors)
        for (int i = threadIdx.x; i <= r.batch; i += 256)
            if (r.cu[i] < 0 || r.cu[i] > r.total || (i && r.cu[i] < r.cu[i - 1])) atomicOr(r.err, kErrSeq);

    // Workgroups of one (segment, group) read the same B and C: they follow
    // each other on one XCD, and the pairs are dealt to the XCDs in turn.
    const int npair = a.nseg * r.G;
    const int xcd = blockIdx.x & 7, at = blockIdx.x >> 3;
    const int pair = (at / a.hb) * 8 + xcd, hblk = at % a.hb;
    if (pair >= npair) return;
    const int entry = pair / r.G, g = pair - entry * r.G;

    const int seq = __builtin_amdgcn_readfirstlane(segment_owner(a, entry, lane));
    const int start = __builtin_amdgcn_readfirstlane(r.cu[seq]), end = __builtin_amdgcn_readfirstlane(r.cu[seq + 1]);
    if (start < 0 || end > r.total || end <= start) return;
    const int k = entry - (start / a.lseg + seq);
    if (k < 0 || (int64_t)k * a.lseg >= end - start) return;
    const int tok0 = start + k * a.lseg;
    const int len = end - tok0 < a.lseg ? end - tok0 : a.lseg;
    const bool last = tok0 + len == end;
    if (LOCAL && last) return;
    const int b = __builtin_amdgcn_readfirstlane(slot_of_row(r, seq));
    if (b < 0) return;   // padding row

    const int hh = wave >> 1;                  // the wave's head among the workgroup's
    const int hl = hblk * kScanHeads + hh;     // ... within the group
    const bool live = hl < hpg;                // an odd head count: half a workgroup runs the last head again, unseen
    const int h = g * hpg + (live ? hl : hpg - 1);
    const int p0 = (wave & 1) * 32;            // the wave's state rows
    const size_t HP = (size_t)r.H * kP, GN = (size_t)r.G * kN;

    // ---- state before the segment: st[nt][i] = S[p0 + c][32 nt + 8 (i / 4) + 4 hf + i % 4]
    f16v st0 = (f16v)0.f, st1 = (f16v)0.f, st2 = (f16v)0.f, st3 = (f16v)0.f;
    const size_t cell = (size_t)(p0 + c) * kN + 4 * hf;
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
    if (k == 0) {
        const bool fresh = r.fresh ? r.fresh[seq] != 0 : r.from_zero != 0;
        if (!fresh) {
            add_state(LOCAL || last ? ckpt : a.s0 + (ent0 * r.H + h) * headN, 1.f);
            if ((LOCAL || last) && threadIdx.x == 0 && r.pos[b] != 0) atomicOr(r.err, kErrPos);   // buffer not empty
            // the second launch rewrites the checkpoint, so its first segment reads a copy
            if (LOCAL && live) put_state(a.s0 + (ent0 * r.H + h) * headN);
        }
    } else if (!LOCAL) {
        // a factor of exactly zero ends the sum: nothing before it counts
        float f = 1.f;
        for (int i = k - 1; i >= 0 && f != 0.f; --i) {
            const size_t e = (ent0 + i) * r.H + h;
            add_state(a.loc + e * headN, f);
            f *= a.lam[e];
        }
    }

    const uint16_t *xin = reinterpret_cast<const uint16_t *>(r.x) + (size_t)tok0 * HP;
    const uint16_t *Bin = reinterpret_cast<const uint16_t *>(r.Bm) + (size_t)tok0 * GN + (size_t)g * kN;
    const uint16_t *Cin = reinterpret_cast<const uint16_t *>(r.Cm) + (size_t)tok0 * GN + (size_t)g * kN;
    const uint16_t *dtin = reinterpret_cast<const uint16_t *>(r.dt) + (size_t)tok0 * r.H + h;
    TY *yout = reinterpret_cast<TY *>(r.y) + (size_t)tok0 * HP + (size_t)h * kP + p0;
    const int yoff = (c * (int)HP + 4 * hf) * (int)sizeof(TY);
    const double A2 = (double)r.A[h] * 1.4426950408889634;
    const float Dh = r.D[h];

    // ---- staging roles: 16 quads of tokens x 16 octets of n (B, C); 2 heads x 16 quads x 8 octets of p (x)
    const int bo = threadIdx.x & 15, bq = threadIdx.x >> 4;
    const int xo = threadIdx.x & 7, xq = (threadIdx.x >> 3) & 15, xh = threadIdx.x >> 7;
    const int xhl = hblk * kScanHeads + xh;
    const size_t xcol = (size_t)(g * hpg + (xhl < hpg ? xhl : hpg - 1)) * kP + 8 * xo;
    u4v rB[4], rC[4], rX[4];
    float rdt;
    // Buffer loads: the chunk's first row is the (uniform) base, and rows past
    // the segment fall outside the resource and read as zeros.
    const int bpitch = (int)GN * 2, xpitch = (int)HP * 2;
    const int boff = 16 * bo + 4 * bq * bpitch, xoff = (int)xcol * 2 + 4 * xq * xpitch, doff = 2 * lane * r.H;
    auto fetch = [&](int t0) {
        const int left = len - t0 < 0 ? 0 : (len - t0 < kQ ? len - t0 : kQ);
        const int rem = __builtin_amdgcn_readfirstlane(left);   // (a vector clamp would make the resources vector values)
        const int bv = recomputed(boff), xv = recomputed(xoff);
        const auto bs = uniform_rsrc(Bin + (size_t)t0 * GN, rem * bpitch);
        const auto xs = uniform_rsrc(xin + (size_t)t0 * HP, rem * xpitch);
        const auto ds = uniform_rsrc(dtin + (size_t)t0 * r.H, rem * 2 * r.H);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rB[i] = __builtin_amdgcn_raw_buffer_load_b128(bs, bv + i * bpitch, 0, 0);
            rX[i] = __builtin_amdgcn_raw_buffer_load_b128(xs, xv + i * xpitch, 0, 0);
        }
        if (OUT) {
            const auto cs = uniform_rsrc(Cin + (size_t)t0 * GN, rem * bpitch);
#pragma unroll
            for (int i = 0; i < 4; ++i) rC[i] = __builtin_amdgcn_raw_buffer_load_b128(cs, bv + i * bpitch, 0, 0);
        }
        rdt = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b16(ds, doff, 0, 0) << 16);
    };

    // LDS offsets of the staging and of the operands
    const int at_b = quad_at(bq), at_x = quad_at(xq);
    const int put_b0 = piece_offset(8 * bo, at_b >> 1) + 8 * (at_b & 1);
    const int put_x0 = (int)sizeof(sm.XT[0]) * xh + piece_offset(8 * xo, at_x >> 1) + 8 * (at_x & 1);
    const int put_r = 2 * kRowN * 4 * bq + 8 * quad_at(2 * bo);
    const int get_x0 = (int)sizeof(sm.XT[0]) * hh + piece_offset(p0 + c, hf);
    const int get_b0 = piece_offset(c, hf);
    const int get_r = 2 * kRowN * c + 16 * hf;

    double total = 0.0;   // decay of the segment (LOCAL)
    fetch(0);
    int odd = 0;
    if (threadIdx.x < 2) sm.bad[threadIdx.x] = kQ;
    for (int t0 = 0; t0 < len; odd ^= 1) {
        __syncthreads();   // the previous chunk's LDS reads are done
        {
            const int put_b = recomputed(put_b0), put_x = recomputed(put_x0);
            store_columns(reinterpret_cast<char *>(sm.BT), put_b, rB[0], rB[1], rB[2], rB[3]);
            if (OUT) {   // quads 2 bo and 2 bo + 1 of a row are two positions apart
                char *pb = reinterpret_cast<char *>(sm.B) + put_r, *pc = reinterpret_cast<char *>(sm.C) + put_r;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    *reinterpret_cast<u2v *>(pb + 2 * kRowN * i) = u2v{rB[i].x, rB[i].y};
                    *reinterpret_cast<u2v *>(pb + 2 * kRowN * i + 16) = u2v{rB[i].z, rB[i].w};
                    *reinterpret_cast<u2v *>(pc + 2 * kRowN * i) = u2v{rC[i].x, rC[i].y};
                    *reinterpret_cast<u2v *>(pc + 2 * kRowN * i + 16) = u2v{rC[i].z, rC[i].w};
                }
            }
            store_columns(reinterpret_cast<char *>(sm.XT), put_x, rX[0], rX[1], rX[2], rX[3]);
        }
        int q = len - t0 < kQ ? len - t0 : kQ;   // tokens of this chunk
        if (OUT) {
            // M_tj = 0 for j > t does not keep a non-finite x_j out of y_t: a
            // chunk ends before a token that holds one, which is then taken alone.
            unsigned seen = 0;
            int first = kQ;
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                unsigned bits = 0;
#pragma unroll
                for (int d = 0; d < 4; ++d) bits |= (rX[i][d] & 0x7F807F80u) + 0x00800080u;
                if (bits & 0x80008000u) first = 4 * xq + i;
                seen |= bits;
            }
            if (seen & 0x80008000u) atomicMin(&sm.bad[odd], first);
        }
        __syncthreads();
        if (OUT) {
            const int bad = __builtin_amdgcn_readfirstlane(sm.bad[odd]), stop = bad > 0 ? bad : 1;
            if (threadIdx.x == 0) sm.bad[odd ^ 1] = kQ;   // read in the last chunk, set in the next
            if (stop < q) {
                q = stop;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (4 * xq + i >= q) rX[i] = (u4v)0u;
                store_columns(reinterpret_cast<char *>(sm.XT), recomputed(put_x0), rX[0], rX[1], rX[2], rX[3]);
                if (lane >= q) rdt = 0.f;
                __syncthreads();
            }
        }

        const int t1 = t0 + q;
        const char *xt = reinterpret_cast<const char *>(sm.XT), *bt = reinterpret_cast<const char *>(sm.BT);
        const int get_x = recomputed(get_x0), get_b = recomputed(get_b0);

        // ---- decays of the wave's head (both waves of a head compute them).
        // exp(c_t - c_j) = 2^(k_t - k_j) 2^f_t 2^-f_j: the fractions' powers
        // are taken once per token, the whole part moves an exponent exactly.
        float lam;
        auto decays = [&]() {
            const double cum = prefix(A2 * (double)rdt), whole = __builtin_floor(cum);
            const double c63 = lane_d(cum, 63);
            const float f = (float)(cum - whole), ri = __builtin_amdgcn_exp2f(-f);
            sm.k[wave][lane] = (int)whole;
            sm.cf[wave][lane] = rdt * ri;
            sm.w[wave][lane] = rdt * __builtin_amdgcn_exp2f((float)(c63 - cum));
            sm.rf[wave][lane] = __builtin_amdgcn_exp2f(f);
            sm.ri[wave][lane] = ri;
            lam = __builtin_amdgcn_exp2f((float)c63);
            total += c63;
            __builtin_amdgcn_wave_barrier();
        };
        if (!OUT) decays();

        if (OUT) {
            // ---- y^T[p][t] = sum_n S[p][n] C_t[n] and the Gram tiles G^T[j][t] = B_j . C_t
            f16v y0 = (f16v)0.f, y1 = (f16v)0.f, g00 = (f16v)0.f, g01 = (f16v)0.f, g11 = (f16v)0.f;
            auto step = [&](const f16v &tile, int ks) {
                b8v s[YP];
                split<YP>(half_of(tile, ks & 1), s);
                const char *pb = reinterpret_cast<const char *>(sm.B) + get_r + 32 * ks;
                const char *pc = reinterpret_cast<const char *>(sm.C) + get_r + 32 * ks;
                const b8v b0 = operand(pb), b1 = operand(pb + 64 * kRowN), c0 = operand(pc), c1 = operand(pc + 64 * kRowN);
                g00 = mfma(b0, c0, g00);
                g01 = mfma(b0, c1, g01);
                g11 = mfma(b1, c1, g11);
#pragma unroll
                for (int i = YP - 1; i >= 0; --i) {
                    y0 = mfma(s[i], c0, y0);
                    y1 = mfma(s[i], c1, y1);
                }
            };
            step(st0, 0);
            step(st0, 1);
            step(st1, 2);
            step(st1, 3);
            step(st2, 4);
            step(st2, 5);
            step(st3, 6);
            step(st3, 7);
            decays();
            const int k0 = sm.k[wave][c], k1 = sm.k[wave][32 + c];
            const float r0 = sm.rf[wave][c], r1 = sm.rf[wave][32 + c];
            const float D0 = Dh * sm.ri[wave][c], D1 = Dh * sm.ri[wave][32 + c];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                y0[i] = __builtin_ldexpf(y0[i], k0);
                y1[i] = __builtin_ldexpf(y1[i], k1);
            }
            // ---- y^T += x^T M^T without the factor 2^f_t, M^T as the operand straight from the Gram accumulators
            auto apply = [&](const f16v &gram, int jt, int kt, float Dt, bool diag, f16v &y) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int j0 = 32 * jt + 16 * s + 4 * hf;
                    f8v m = half_of(gram, s);
                    const f8v cf = read8(&sm.cf[wave][j0]);
                    const i8v kj = read8(&sm.k[wave][j0]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        m[i] = __builtin_ldexpf(m[i] * cf[i], kt - kj[i]);
                        if (diag) {
                            const int j = 16 * s + 4 * hf + 8 * (i >> 2) + (i & 3);
                            m[i] = j < c ? m[i] : (j == c ? m[i] + Dt : 0.f);
                        }
                    }
                    b8v part[YP];
                    split<YP>(m, part);
                    const b8v x = operand(xt + (get_x ^ (64 * jt + 32 * s)));
#pragma unroll
                    for (int i = YP - 1; i >= 0; --i) y = mfma(x, part[i], y);
                }
            };
            apply(g00, 0, k0, D0, true, y0);
            apply(g01, 0, k1, 0.f, false, y1);
            apply(g11, 1, k1, D1, true, y1);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                y0[i] *= r0;
                y1[i] *= r1;
            }
            // rows past the chunk (and an unseen head's) fall outside the resource
            const auto ys = uniform_rsrc(yout + (size_t)t0 * HP, live ? q * (int)HP * (int)sizeof(TY) : 0);
            auto store = [&](const f16v &y, int off) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f4v v = {y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]};
                    const int at = off + 8 * i * (int)sizeof(TY);
                    if constexpr (sizeof(TY) == 4)
                        __builtin_amdgcn_raw_buffer_store_b128(v, ys, at, 0, 0);
                    else
                        __builtin_amdgcn_raw_buffer_store_b64(
                            __builtin_bit_cast(u2v, __builtin_convertvector(v, b4v)), ys, at, 0, 0);
                }
            };
            store(y0, yoff);
            store(y1, yoff + 32 * (int)HP * (int)sizeof(TY));
        }
        // The next chunk is requested here, when only the state is held.
        __builtin_amdgcn_sched_barrier(0);
        fetch(t1);

        // ---- S^T[n][p] = exp(c_63) S^T + sum_j B_j[n] (w_j x_j[p])
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            st0[i] *= lam;
            st1[i] *= lam;
            st2[i] *= lam;
            st3[i] *= lam;
        }
#pragma unroll
        for (int js = 0; js < 4; ++js) {
            f8v v = vec8<uint16_t>::widen(*reinterpret_cast<const u4v *>(__builtin_assume_aligned(xt + (get_x ^ (32 * js)), 16)));
            const f8v w = read8(&sm.w[wave][16 * js + 4 * hf]);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= w[i];
            b8v part[3];
            split<3>(v, part);
            const b8v b0 = operand(bt + (get_b ^ (32 * js))), b1 = operand(bt + (get_b ^ (32 * (js ^ 1))) + 64 * kRowQ),
                      b2 = operand(bt + (get_b ^ (32 * (js ^ 2))) + 128 * kRowQ),
                      b3 = operand(bt + (get_b ^ (32 * (js ^ 3))) + 192 * kRowQ);
#pragma unroll
            for (int i = 2; i >= 0; --i) {
                st0 = mfma(b0, part[i], st0);
                st1 = mfma(b1, part[i], st1);
                st2 = mfma(b2, part[i], st2);
                st3 = mfma(b3, part[i], st3);
            }
        }
        t0 = t1;
    }

    if (LOCAL) {
        const size_t e = (ent0 + k) * r.H + h;
        if (live) {
            put_state(a.loc + e * headN);
            if ((wave & 1) == 0 && lane == 0) a.lam[e] = exp2f((float)total);
        }
    } else if (last) {
        if (live) put_state(ckpt);
        publish_position(r, b, 0, true, -1);
    }
}

}  // namespace

hipError_t launch_scan(const ReplayParams &p, bool outputs, void *workspace, hipStream_t s) {
    if (p.batch == 0 || p.total == 0) return hipSuccess;
    ScanParams a{};
    a.r = p;
    a.lseg = scan_segment(p.total, p.H, p.G);
    a.nfull = (int)(p.total / a.lseg);
    if (!workspace || a.nfull == 0) {   // one segment per sequence
        a.lseg = (int)((p.total + kScanChunk) / kScanChunk * kScanChunk);
        a.nfull = 0;
    } else {
        a.loc = static_cast<float *>(workspace);
        a.s0 = a.loc + (size_t)a.nfull * p.H * kP * kN;
        a.lam = a.s0 + (size_t)a.nfull * p.H * kP * kN;
    }
    a.nseg = (int)(p.total / a.lseg) + p.batch;
    a.hb = (p.H / p.G + kScanHeads - 1) / kScanHeads;
    a.r.wg_per_slot = p.G * a.hb;
    const int64_t blocks = ((int64_t)a.nseg * p.G + 7) / 8 * 8 * a.hb;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block(256);
    if (a.nfull) hipLaunchKernelGGL((scan_kernel<float, 3, false, true>), grid, block, 0, s, a);
    if (!outputs) hipLaunchKernelGGL((scan_kernel<float, 3, false, false>), grid, block, 0, s, a);
    else if (p.y_bf16) hipLaunchKernelGGL((scan_kernel<uint16_t, 2, true, false>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((scan_kernel<float, 3, true, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace rssm
