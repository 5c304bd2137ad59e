// kda_paged.cuh -- how attention over a paged cache is split over the grid.
#pragma once

#include "kda_layers.cuh"

namespace kda {

// ---------------------------------------------------------------------------
// The split.  An item is a (sequence, key-value head, block of at most HB query
// heads); its cache is cut into tiles of TILE tokens.  All tiles of all items
// in order are dealt out evenly: CTA b of g takes tiles [b W / g, (b + 1) W / g)
// of W, whatever the lengths are, so ragged batches and one long row both fill
// the GPU.  An item that one CTA has whole is finished there; of the others
// each CTA leaves at most two partial results (slot 0: it does not start the
// item, slot 1: it starts it), which the join kernel adds up in order.
// ---------------------------------------------------------------------------
struct Split {
    int64_t W;        // tiles in all
    int g;            // CTAs that have any
    int64_t cum;      // tiles of one head of the sequences before `n`
    int n;            // sequence
};

__device__ __forceinline__ int clamped(const PagedParams &p, int len) {
    const int64_t cap = (int64_t)p.max_pages << p.page_shift;
    return len < 0 ? 0 : (len > cap ? (int)cap : len);
}
__device__ __forceinline__ int clamp_len(const PagedParams &p, int n, bool tell) {
    const int len = p.lens[n], c = clamped(p, len);
    if (tell && c != len) report_status(p.status, KDA_ERR_INVALID_ARG);
    return c;
}

// Tiles of one item of sequence n.
template <int TILE>
__device__ __forceinline__ int64_t tiles_of(const PagedParams &p, int n) {
    return (clamp_len(p, n, false) + TILE - 1) / TILE;
}

// Block-wide (the first 256 threads scan): the totals, and with b >= 0 the sequence in which
// CTA b's first tile lies; with b < 0 the sums before sequence `n`.
template <int TILE>
__device__ Split find_split(const PagedParams &p, int items, int grid, int b, int n, int64_t *s_sum /* 257 */,
                            int *s_n) {
    const int tid = threadIdx.x;
    const int per = (p.N + 255) / 256, n0 = min(p.N, tid * per), n1 = min(p.N, n0 + per);
    int64_t mine = 0;
    for (int i = n0; i < n1; ++i) mine += tiles_of<TILE>(p, i);
    // inclusive scan over the 256 threads: within warps, then over the 8 warp sums
    int64_t x = mine;
    const int lane = tid & 31, w = tid >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_sum[w] = x;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int i = 0; i < 8; ++i) {
        if (i < w) before += s_sum[i];
        total += s_sum[i];
    }
    int64_t c = before + x - mine;                 // tiles of one item of every sequence before n0
    Split r;
    r.W = total * items;
    r.g = (int)(r.W < grid ? r.W : grid);
    r.n = n;
    r.cum = 0;
    if (b >= 0 && b >= r.g) return r;
    const int64_t w0 = b >= 0 ? (int64_t)b * r.W / r.g : 0;
    for (int i = n0; i < n1; ++i) {
        const int64_t ti = tiles_of<TILE>(p, i);
        if (b >= 0 ? (w0 >= c * items && w0 < (c + ti) * items) : i == n) {
            s_sum[256] = c;
            *s_n = i;
        }
        c += ti;
    }
    __syncthreads();
    r.cum = s_sum[256];
    r.n = *s_n;
    __syncthreads();
    return r;
}

// Zero outputs and lse = -inf of sequence n, which has no tokens (block-wide).
template <typename T>
__device__ __forceinline__ void empty_sequence(const PagedParams &p, int n, int D) {
    clamp_len(p, n, threadIdx.x == 0);
    T *out = static_cast<T *>(p.out) + (int64_t)n * p.Hq * D;
    for (int i = threadIdx.x; i < p.Hq * D; i += blockDim.x) out[i] = from_f32<T>(0.f);
    if (p.lse)
        for (int i = threadIdx.x; i < p.Hq; i += blockDim.x) p.lse[(int64_t)n * p.Hq + i] = -INFINITY;
}

// Those of all empty sequences, where no join kernel follows to write them.
template <typename T, int TILE>
__device__ __forceinline__ void empty_sequences(const PagedParams &p, int D) {
    if (p.lone)
        for (int n = blockIdx.x; n < p.N; n += gridDim.x)
            if (tiles_of<TILE>(p, n) == 0) empty_sequence<T>(p, n, D);
}

// One partial result of an item of HB query heads: m, l (base-2 logarithms) per
// head, then a[d] per head.
__host__ __device__ constexpr int part_floats(int d, int HB) { return HB * (d + 2); }

// bf16, d = 64 or 128, pages of at least 8 tokens: the tensor-core form and the
// grid it runs on, with HB query heads per item.
cudaError_t launch_paged_decode_tc(const PagedParams &p, int d, int HB, int grid, cudaStream_t st);
constexpr int kTileTc = 128;

}  // namespace kda
