// kda_decay.cuh -- chains of the decayed linear attention cut into segments.
//
// Over a segment of L tokens the state map is S_out = lambda^L S_in + b, so few
// long chains fill the GPU in three steps: b of every segment but a chain's last
// (from zero states), the start states S(g + 1) = lambda^L S(g) + b(g) of every
// segment in order (decay_segments_kernel, elementwise), and all segments side
// by side from their start states.
#pragma once

#include "kda_layers.cuh"
#include "sm100_ptx.cuh"

namespace kda {

struct DecaySegs {
    const int32_t *cu;
    int N, H;
    int64_t total;
    int len;                    // tokens per segment; 0: every chain is one piece
    int cap;                    // segments that `cells` has room for (there are more only if the offsets overlap)
    float *cells;               // [segment][H][dk dv]: b, then the start state
    uint32_t *status;
};

// Offsets are below 2^31 (the entry point sees to it), so token counts are int.
__device__ __forceinline__ void seq_range(const DecaySegs &p, int seq, int &bos, int &eos, bool tell) {
    bos = p.cu[seq];
    eos = p.cu[seq + 1];
    if (bos < 0 || eos < bos || eos > p.total) {
        if (tell) report_status(p.status, kDevBadSeqlens);
        bos = eos = 0;
    }
}

// Segments of a sequence; an empty one has one empty segment (its state is copied).
__device__ __forceinline__ int segments_of(const DecaySegs &p, int len) {
    return len > 0 ? (int)((unsigned)(len - 1) / (unsigned)p.len) + 1 : 1;
}

// The sequence n and the number g within it of segment `seg` of the batch, with
// the segment's tokens; false past the last one.
struct Segment {
    int n, g, t0, t1;
    bool last;
};
__device__ __forceinline__ bool find_segment(const DecaySegs &p, unsigned seg, Segment &x, bool tell) {
    int before = 0;
#pragma unroll 1
    for (int n = 0; n < p.N; ++n) {
        int bos, eos;
        seq_range(p, n, bos, eos, tell);
        const int segs = segments_of(p, eos - bos), g = (int)seg - before;
        before += segs;
        if (g >= segs) continue;
        if (seg >= (unsigned)p.cap) {
            if (tell) report_status(p.status, kDevBadSeqlens);
            return false;
        }
        x.n = n;
        x.g = g;
        x.t0 = bos + g * p.len;
        x.t1 = eos - x.t0 > p.len ? x.t0 + p.len : eos;
        x.last = g == segs - 1;
        return true;
    }
    return false;
}

// 2^(l2 n) with l2 no lower than -16384: exactly 0 for n >= 1 there, and 1 for n = 0.  A NaN stays one.
__device__ __forceinline__ float decay_log2(const float *log_decay, int head) {
    const float l2 = log_decay[head] * kLog2E;
    return l2 < -16384.f ? -16384.f : l2;
}

// Tokens per segment in whole chunks, or 0 for whole chains.  Segments cost a
// second pass over k and v and two more launches: in units of a chunk's time in a
// whole chain, a segment of m chunks takes per m + fixed.  So they are taken where
// the chains fill at most half of the `slots` (CTAs that run at a time), one
// segment per slot, and only where that is less than the longest chain's chunks,
// guessed at 3/2 of the mean (the lengths are on the device; the mean itself where
// there is one sequence).
//   Measured, in segments / whole (us).  bf16, d = 128, 16 heads: 512 tokens 24.0 /
// 18.6, 1024 25.3 / 32.7, 4096 39.7 / 117; 64 heads: 2048 tokens 63.9 / 62.7, 4096
// 108 / 120; 4 sequences of 1024 tokens, 16 heads, 54.5 / 33.4.  f32, d = 128, 16
// heads: 256 tokens 41.4 / 64.9, 4096 268 / 1056; 64 heads: 4096 tokens 1110 / 1074.
// The guess costs most with few long sequences of one length: 4 of 4096 tokens, 16
// heads, 153 / 119.
struct SegmentCost {
    int chunk, least;           // tokens of a chunk; fewest chunks of a segment
    float per, fixed;
};

inline int decay_segment_tokens(int64_t total, int N, int H, int slots, const SegmentCost &cost) {
    const int64_t chains = (int64_t)N * H, C = cost.chunk;
    if (chains * 2 > slots || N > 64) return 0;
    // sum over the sequences of ceil(len / m) stays within the slots
    const int64_t room = (slots - chains) * C;
    int64_t m = (total * H + room - 1) / room;
    if (N == 1) m = ((total + C - 1) / C + slots / H - 1) / (slots / H);
    if (m < cost.least) m = cost.least;
    const float longest = (float)total / (float)(N * C) * (N > 1 ? 1.5f : 1.f);
    return cost.per * (float)m + cost.fixed < longest ? (int)(m * C) : 0;
}

inline size_t decay_cells_bytes(int64_t total, int N, int H, int len, int dk, int dv) {
    return len ? (size_t)((total / len + N) * H) * dk * dv * sizeof(float) : 0;
}

// Launches the elementwise pass over all segments, as a dependent of the kernel before it.
cudaError_t launch_decay_segments(const DecaySegs &p, const float *log_decay, const float *init, int dk, int dv,
                                  cudaStream_t st);

}  // namespace kda
