// scan.h -- host interface of the matrix-core scan of packed prompts.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "kernels.h"

namespace rssm {

constexpr int kScanChunk = 64;       // tokens per chunk

// Heads per workgroup (of one B/C group): B and C are staged once for all of
// them, and two chunks of four heads, or one of two heads in the three planes
// of fp32 inputs, fill the LDS of a compute unit.
inline int scan_heads(int hpg, bool in_bf16) { return in_bf16 ? (hpg >= 3 ? 4 : hpg) : (hpg >= 2 ? 2 : 1); }

struct ScanParams {
    ReplayParams r;
    float *loc;        // [nfull, H, P, N] end state of each full segment that has a successor
    float *s0;         // [nfull, H, P, N] copy of the start state of a split sequence (at its first segment's entry);
                       // behind the second launch, the end state of each marked half of a head
    float *lam;        // [nfull, H] decay over the segment
    int *mark;         // [nfull, H, 2] end state not all finite, in the head's lower and upper 32 rows
    int *marked;       // [1] any mark set
    int lseg;          // tokens per segment (a multiple of kScanChunk)
    int nfull;         // full segments that fit: total / lseg (the grid: these, then a rest per sequence)
    int hb;            // workgroups per (segment, group)
};

// Tokens per segment for a call: long sequences are cut so that each of the
// 256 compute units has a workgroup, and no finer.  (23 sequences of 9001
// tokens together, 128 heads: in segments of half or a third of that the pieces
// even out and the second launch loses 15 us, but the first one grows from 45
// to 95 us.)  Where there are sequences enough for that, a segment may be a
// third longer: a sequence not much above the mean load is then not cut for the
// price of a first launch (the same, over six sets of lengths: 256 us in
// segments of the mean load, 237 us a third longer, 246 us half as long again).
//
// Few heads would leave segments of a chunk or two.  A segment joins every one
// before it, so n chunks are cut into no more than about 4 sqrt(n) segments; and
// where twice the mean length is not five chunks (only the device knows the
// lengths) segments keep at least four, as a launch more costs as much as two
// chunks.  (8 heads: one sequence of 333 tokens in fp32 90 us in segments of four
// chunks and 53 us in single ones, eight of together 2048 tokens of 16 heads in
// bf16 71 and 64 us; five of together 200 tokens 30 us whole and 50 us cut.)
inline int scan_segment(int64_t total, int batch, int H, int G, bool in_bf16) {
    const int nh = scan_heads(H / G, in_bf16);
    const int64_t hb = (int64_t)G * ((H / G + nh - 1) / nh);
    const int64_t chunks = (total + kScanChunk - 1) / kScanChunk;
    const int64_t pieces = hb < 256 ? 256 / hb : 1;   // segments side by side
    int64_t per = (chunks + pieces - 1) / pieces;
    if (batch >= pieces) per += per / 3;   // sequences fill the card by themselves
    const int64_t likely = batch > 2 ? 2 * total / batch : total;
    const int64_t least = likely > 4 * kScanChunk ? (int64_t)std::ceil(std::sqrt((double)chunks / 16.0)) : 4;
    if (per < least) per = least;
    return (int)(per * kScanChunk);
}

inline size_t scan_workspace(int64_t total, int batch, int H, int G, bool in_bf16) {
    const int64_t nfull = total / scan_segment(total, batch, H, G, in_bf16);
    return nfull ? ((size_t)nfull * H * (2 * 64 * 128 + 3) + 1) * sizeof(float) : 0;
}

// fp32 checkpoints.  Without a workspace every sequence is one segment.
hipError_t launch_scan(const ReplayParams &p, bool in_bf16, bool outputs, void *workspace, hipStream_t s);

}  // namespace rssm
