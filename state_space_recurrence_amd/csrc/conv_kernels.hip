// conv_kernels.hip -- short causal convolution in front of the recurrence.
//
// For every channel of a token t (x, B and C of the input projection):
//     c_t = bias + sum_{k<W} w[k] u_{t-W+1+k},  out = c_t or c_t sigmoid(c_t)
// and for every head dt = clamp(softplus(dt_raw + dt_bias), dt_min, dt_max).
// Sums are fp32; outputs are rounded once to the input type, the type in
// which the recurrence reads x, B, C and dt.
//
// History.  A slot keeps its last raw inputs in a ring of R rows; `head` is
// the row of the next token and the W-1 rows before it are its history.  A
// token or draft is written at its own row, nothing is shifted, and rollback
// is a smaller advance of `head`: rejected drafts' rows are overwritten
// later, as in the replay buffer.  R >= W-1 + Tmax keeps the drafts clear of
// the history, R >= 2(W-1) the last rows of a prompt clear of the history
// that other workgroups of the call still read; the new head waits for them
// (HistoryTiles).
//
// All of it is streaming: a thread owns eight channels (16 bytes of bf16) and
// walks down the tokens with the last W-1 inputs in registers, so each input
// is read once.  Bound by memory: 16384 tokens of 8192 channels in bf16 take
// 109 us (544 MB, 5.0 TB/s; with cached instead of streaming loads 15 % more).
// A round of 512 x 5 drafts of 10240 channels moves 190 MB: 38 us at the copy
// rate, 32 us where half of its inputs are still in a cache (87 MB read).
#include "mixer.h"
#include "mixer_device.h"

namespace rssm {
namespace {

constexpr int kThreads = kConvThreads;
constexpr int kVec = kConvVec;

template <typename T>
__device__ __forceinline__ float dt_of(const ConvParams &p, int64_t token, int h) {
    float v = vec8<T>::get(reinterpret_cast<const T *>(p.dtr) + token * p.dt_pitch + h);
    if (p.dt_bias) v += p.dt_bias[h];
    // softplus without overflow or cancellation: max(v, 0) + log(1 + exp(-|v|))
    const float sp = fmaxf(v, 0.f) + log1pf(expf(-fabsf(v)));
    return v != v ? v : fminf(fmaxf(sp, p.dt_min), p.dt_max);
}

// Ring row `r` of a slot, r in (-R, 2R).
__device__ __forceinline__ int wrap(int r, int R) { return r < 0 ? r + R : (r >= R ? r - R : r); }

__device__ __forceinline__ int conv_slot(const ConvParams &p, int row) {
    const int b = p.slot_idx ? p.slot_idx[row] : row;
    if (b >= p.nslots || b < -1) {
        if (threadIdx.x == 0) atomicOr(p.err, kErrSlot);
        return -1;
    }
    return b;
}

__device__ __forceinline__ int conv_head(const ConvParams &p, int b) {
    const int h = p.head[b];
    if (h < 0 || h >= p.R) {
        if (threadIdx.x == 0) atomicOr(p.err, kErrPos);
        return 0;
    }
    return h;
}

template <typename T, int W>
struct Taps {
    f8v w[W], bias;
    __device__ __forceinline__ void load(const ConvParams &p, int ch) {
#pragma unroll
        for (int k = 0; k < W; ++k) w[k] = vec8<float>::widen(vec8<float>::load(p.w + (size_t)k * p.Cc + ch));
        bias = p.bias ? vec8<float>::widen(vec8<float>::load(p.bias + ch)) : (f8v)0.f;
    }
    // win[k] = u_{t-W+1+k}
    __device__ __forceinline__ f8v apply(const f8v (&win)[W], int act) const {
        f8v c = bias;
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int i = 0; i < kVec; ++i) c[i] = fmaf(w[k][i], win[k][i], c[i]);
        if (act)
#pragma unroll
            for (int i = 0; i < kVec; ++i) c[i] = silu(c[i]);
        return c;
    }
};

// Where a thread's eight channels go: one of x, B, C (every boundary is a
// multiple of 64), `pitch` elements per token.
template <typename T>
struct OutChannels {
    T *base;
    int pitch;
    __device__ __forceinline__ OutChannels(const ConvParams &p, int ch) {
        if (ch < p.HP) {
            base = reinterpret_cast<T *>(p.x) + ch;
            pitch = p.HP;
        } else {
            const int c = ch - p.HP;
            base = c < p.GN ? reinterpret_cast<T *>(p.B) + c : reinterpret_cast<T *>(p.C) + (c - p.GN);
            pitch = p.GN;
        }
    }
};

// Last of `want` arrivals at slot b publishes its head.
__device__ __forceinline__ void arrive(const ConvParams &p, int b, int want, int new_head) {
    const int old = want == 1 ? 0 : atomicAdd(&p.work[b], 1);
    if (old >= want) atomicOr(p.err, kErrDup);
    if (old == want - 1) {
        if (want > 1) p.work[b] = 0;
        p.head[b] = new_head;
    }
}

// T tokens of every row: one decode token (ADVANCE) or a round of drafts.
template <typename TIn, int W, int TMAX, bool ADVANCE>
__global__ void __launch_bounds__(kThreads) conv_token_kernel(ConvParams p) {
    typedef vec8<TIn> V;
    const int row = blockIdx.x / p.nblk, blk = blockIdx.x - row * p.nblk;
    const int b = conv_slot(p, row);
    if (b < 0) return;   // padding row
    const int tid = blk * kThreads + threadIdx.x;
    const int ch = tid * kVec;
    const int T = TMAX == 1 ? 1 : p.T;
    const int64_t tok = (int64_t)row * T;
    const bool mine = ch < p.Cc;
    const TIn *u = reinterpret_cast<const TIn *>(p.u) + tok * p.u_pitch + ch;
    typename V::raw8 in[TMAX];
    if (mine)
#pragma unroll
        for (int t = 0; t < TMAX; ++t)
            if (t < T) in[t] = V::load(u + t * p.u_pitch);
    const int head = conv_head(p, b);
    if (mine) {
        TIn *ring = reinterpret_cast<TIn *>(p.ring) + (size_t)b * p.R * p.Cc + ch;
        Taps<TIn, W> taps;
        taps.load(p, ch);
        f8v win[W];
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            win[k] = V::widen(V::load(ring + (size_t)wrap(head - (W - 1) + k, p.R) * p.Cc));
        const OutChannels<TIn> out(p, ch);
#pragma unroll
        for (int t = 0; t < TMAX; ++t) {
            if (t < T) {
                win[W - 1] = V::widen(in[t]);
                V::store(out.base + (tok + t) * out.pitch, taps.apply(win, p.silu));
                V::store_raw(ring + (size_t)wrap(head + t, p.R) * p.Cc, in[t]);
#pragma unroll
                for (int k = 0; k < W - 1; ++k) win[k] = win[k + 1];
            }
        }
    }
    for (int i = tid; i < T * p.H; i += p.nblk * kThreads) {
        const int t = i / p.H, h = i - t * p.H;
        V::put(reinterpret_cast<TIn *>(p.dt) + (tok + t) * p.H + h, dt_of<TIn>(p, tok + t, h));
    }
    if (ADVANCE) {
        __syncthreads();   // every thread has read the head
        if (threadIdx.x == 0) arrive(p, b, p.nblk, wrap(head + 1, p.R));
    }
}

// Sequence of packed token t: the last s with cu[s] <= t, or rows when t lies
// past the last offset.
__device__ __forceinline__ int find_sequence(const int32_t *cu, int rows, int t) {
    int lo = 0, hi = rows + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The packed call's view of the sequence s that holds token t
// (wave-uniform); !ok for tokens of no sequence, or of a padding row.
struct Seq {
    int start, end, b, head, m, fresh;
    bool ok;
};

template <int W>
__device__ __forceinline__ Seq sequence(const ConvParams &p, int s, int t) {
    Seq q;
    q.start = p.cu[s];
    q.end = p.cu[s + 1];
    const bool in = q.start >= 0 && q.start <= t && t < q.end && q.end <= p.total;
    q.b = in ? conv_slot(p, s) : -1;
    q.ok = q.b >= 0;
    q.head = q.ok ? conv_head(p, q.b) : 0;
    q.m = q.end - q.start < W - 1 ? q.end - q.start : W - 1;
    q.fresh = p.fresh ? p.fresh[s] != 0 : p.from_zero;
    if (!in) q.end = t + 1;   // look again at the next token
    return q;
}

// Packed prompts: a workgroup takes `tile` consecutive packed tokens (over
// sequence borders) of 2048 channels.
template <typename TIn, int W>
__global__ void __launch_bounds__(kThreads) conv_packed_kernel(ConvParams p) {
    typedef vec8<TIn> V;
    constexpr int U = 4;   // tokens whose inputs are requested together
    const int tile = blockIdx.x / p.nblk, blk = blockIdx.x - tile * p.nblk;
    const int tid = blk * kThreads + threadIdx.x;
    const int ch = tid * kVec;
    const bool mine = ch < p.Cc;
    const int t0 = tile * p.tile;
    const int t1 = (int64_t)t0 + p.tile < p.total ? t0 + p.tile : (int)p.total;
    const TIn *u = reinterpret_cast<const TIn *>(p.u) + ch;

    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i <= p.rows; i += kThreads)
            if (p.cu[i] < 0 || p.cu[i] > p.total || (i && p.cu[i] < p.cu[i - 1])) atomicOr(p.err, kErrSeq);

    const int s0 = find_sequence(p.cu, p.rows, t0);
    int s = s0;
    if (s < p.rows) {
        unsigned live = 0;   // of the tile's tokens (32 at most), those of a sequence with a slot
        Taps<TIn, W> taps;
        f8v win[W];
        if (mine) taps.load(p, ch);
        Seq q = sequence<W>(p, s, t0);
        TIn *ring = reinterpret_cast<TIn *>(p.ring) + (size_t)(q.ok ? q.b : 0) * p.R * p.Cc + ch;
        const OutChannels<TIn> out(p, ch);
        // window before token t of the current sequence
        auto history = [&](int t) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                const int a = t - (W - 1) + k;   // token of this tap
                if (!q.ok) win[k] = (f8v)0.f;
                else if (a >= q.start) win[k] = V::widen(V::load(u + (int64_t)a * p.u_pitch));
                else if (q.fresh) win[k] = (f8v)0.f;
                else win[k] = V::widen(V::load(ring + (size_t)wrap(q.head + (a - q.start), p.R) * p.Cc));
            }
        };
        if (mine) history(t0);
        for (int tb = t0; tb < t1; tb += U) {
            typename V::raw8 in[U];
            if (mine)
#pragma unroll
                for (int j = 0; j < U; ++j)
                    in[j] = V::load_once(u + (int64_t)(tb + j < t1 ? tb + j : t1 - 1) * p.u_pitch);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int t = tb + j;
                if (t >= t1) continue;
                if (t >= q.end) {   // the next sequence that holds t
                    const int sn = find_sequence(p.cu, p.rows, t);
                    if (sn >= p.rows) {   // past the last offset
                        q.ok = false;
                        continue;
                    }
                    s = sn;
                    q = sequence<W>(p, s, t);
                    ring = reinterpret_cast<TIn *>(p.ring) + (size_t)(q.ok ? q.b : 0) * p.R * p.Cc + ch;
                    if (mine) history(t);
                }
                if (!q.ok) continue;
                live |= 1u << (t - t0);
                if (!mine) continue;
                win[W - 1] = V::widen(in[j]);
                V::store(out.base + (int64_t)t * out.pitch, taps.apply(win, p.silu));
#pragma unroll
                for (int k = 0; k < W - 1; ++k) win[k] = win[k + 1];
                const int keep = t - (q.end - q.m);   // >= 0: one of the last W-1 inputs, kept in the ring
                if (keep >= 0) V::store_raw(ring + (size_t)wrap(q.head + keep, p.R) * p.Cc, in[j]);
                if (t == q.start && q.fresh)          // a short fresh prompt: zeros before its tokens
                    for (int k = q.m; k < W - 1; ++k)
                        V::store_raw(ring + (size_t)wrap(q.head + q.m - 1 - k, p.R) * p.Cc, V::zero());
            }
        }
        for (int i = tid; i < (t1 - t0) * p.H; i += p.nblk * kThreads) {
            const int t = i / p.H, h = i - t * p.H;
            if (live >> t & 1) V::put(reinterpret_cast<TIn *>(p.dt) + (int64_t)t0 * p.H + i, dt_of<TIn>(p, t0 + t, h));
        }
        // Publish the heads of the sequences whose history this tile read or
        // wrote, the last of their tiles to arrive does.
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int k = s0; k <= s; ++k) {
                const int start = p.cu[k], end = p.cu[k + 1];
                if (start < 0 || end <= start || end > p.total) continue;
                const HistoryTiles tiles(start, end, W, p.tile);
                if (!tiles.has(tile)) continue;
                const int b = p.slot_idx ? p.slot_idx[k] : k;
                if (b < 0 || b >= p.nslots) continue;
                const int m = end - start < W - 1 ? end - start : W - 1;
                int head = p.head[b];   // not published before this arrival
                head = head < 0 || head >= p.R ? 0 : head;
                arrive(p, b, tiles.count() * p.nblk, wrap(head + m, p.R));
            }
        }
    }
}

__global__ void conv_accept_kernel(ConvParams p) {
    const int row = blockIdx.x * blockDim.x + threadIdx.x;
    if (row >= p.rows) return;
    const int b = p.slot_idx ? p.slot_idx[row] : row;
    if (b >= p.nslots || b < -1) atomicOr(p.err, kErrSlot);
    if (b < 0 || b >= p.nslots) return;
    int n = p.n_keep[row], h = p.head[b];
    if (n < 0 || n > p.T) {
        atomicOr(p.err, kErrKeep);
        n = n < 0 ? 0 : p.T;
    }
    if (h < 0 || h >= p.R) {
        atomicOr(p.err, kErrPos);
        h = 0;
    }
    p.head[b] = wrap(h + n, p.R);
}

template <typename TIn, int W>
void launch_tokens(const ConvParams &p, bool advance, hipStream_t s) {
    const dim3 grid((unsigned)p.rows * p.nblk), block(kThreads);
    if (advance) hipLaunchKernelGGL((conv_token_kernel<TIn, W, 1, true>), grid, block, 0, s, p);
    else if (p.T == 1) hipLaunchKernelGGL((conv_token_kernel<TIn, W, 1, false>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((conv_token_kernel<TIn, W, 8, false>), grid, block, 0, s, p);
}

}  // namespace

#define RSSM_BY_WIDTH(F, T, ...)                      \
    switch (width) {                                  \
        case 2: F<T, 2> __VA_ARGS__; break;           \
        case 3: F<T, 3> __VA_ARGS__; break;           \
        case 4: F<T, 4> __VA_ARGS__; break;           \
        default: return hipErrorInvalidValue;         \
    }

hipError_t launch_conv_tokens(const ConvParams &p0, bool in_bf16, int width, bool advance, hipStream_t s) {
    ConvParams p = p0;
    p.nblk = (int)conv_channel_blocks(p.Cc);
    if (in_bf16) {
        RSSM_BY_WIDTH(launch_tokens, uint16_t, (p, advance, s))
    } else {
        RSSM_BY_WIDTH(launch_tokens, float, (p, advance, s))
    }
    return hipGetLastError();
}

hipError_t launch_conv_packed(const ConvParams &p0, bool in_bf16, int width, hipStream_t s) {
    ConvParams p = p0;
    p.nblk = (int)conv_channel_blocks(p.Cc);
    p.tile = conv_tile(p.total, p.nblk);
    const dim3 grid((unsigned)((p.total + p.tile - 1) / p.tile * p.nblk)), block(kThreads);
#define RSSM_PACKED(T, W) hipLaunchKernelGGL((conv_packed_kernel<T, W>), grid, block, 0, s, p)
    switch (width * 2 + (in_bf16 ? 1 : 0)) {
        case 4: RSSM_PACKED(float, 2); break;
        case 5: RSSM_PACKED(uint16_t, 2); break;
        case 6: RSSM_PACKED(float, 3); break;
        case 7: RSSM_PACKED(uint16_t, 3); break;
        case 8: RSSM_PACKED(float, 4); break;
        case 9: RSSM_PACKED(uint16_t, 4); break;
        default: return hipErrorInvalidValue;
    }
#undef RSSM_PACKED
    return hipGetLastError();
}

hipError_t launch_conv_accept(const ConvParams &p, hipStream_t s) {
    hipLaunchKernelGGL(conv_accept_kernel, dim3((unsigned)(p.rows + 255) / 256), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace rssm
