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

// a / b of numbers >= 0, in 32 bits where they fit (64-bit division is a long loop).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// Tiles of one item of sequence n.
template <int TILE>
__device__ __forceinline__ int64_t tiles_of(const PagedParams &p, int n) {
    return (clamp_len(p, n, false) + TILE - 1) / TILE;
}

// Block-wide (the first SCAN threads scan): the totals, and with b >= 0 the sequence in which
// CTA b's first tile lies; with b < 0 the sums before sequence `n`.
template <int TILE, int SCAN = 256>
__device__ Split find_split(const PagedParams &p, int items, int grid, int b, int n, int64_t *s_sum /* 257 */,
                            int *s_n) {
    const int tid = threadIdx.x;
    const int per = (p.N + SCAN - 1) / SCAN, n0 = min(p.N, tid * per), n1 = min(p.N, n0 + per);
    int64_t mine = 0;
    for (int i = n0; i < n1; ++i) mine += tiles_of<TILE>(p, i);
    // inclusive scan over the threads: within warps, then over the warps' sums
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
#pragma unroll
    for (int i = 0; i < SCAN / 32; ++i) {
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
    const int64_t w0 = b >= 0 ? quotient((int64_t)b * r.W, r.g) : 0;
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

// Zero outputs and lse = -inf of the sequences without tokens, a warp at a time.
template <typename T>
__device__ __forceinline__ void empty_sequences(const PagedParams &p, int D) {
    const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
    // (the last CTAs first: they have no tiles where there are few)
    for (int64_t n0 = ((int64_t)(gridDim.x - 1 - blockIdx.x) * warps + (threadIdx.x >> 5)) * 32; n0 < p.N;
         n0 += (int64_t)gridDim.x * warps * 32) {
        const int len = n0 + lane < p.N ? clamp_len(p, (int)n0 + lane, true) : 1;
        for (uint32_t left = __ballot_sync(0xffffffffu, len == 0); left; left &= left - 1) {
            const int64_t n = n0 + __ffs(left) - 1;
            T *out = static_cast<T *>(p.out) + n * p.Hq * D;
            for (int i = lane; i < p.Hq * D; i += 32) out[i] = from_f32<T>(0.f);
            if (p.lse)
                for (int i = lane; i < p.Hq; i += 32) p.lse[n * p.Hq + i] = -INFINITY;
        }
    }
}

// The same by the whole of a CTA that has one in its turn, before anything else: for kernels that have no registers to
// spare for it at their end.
template <typename T, int TILE>
__device__ __forceinline__ void empty_sequences_first(const PagedParams &p, int D) {
    for (int n = blockIdx.x; n < p.N; n += gridDim.x)
        if (tiles_of<TILE>(p, n) == 0) {
            clamp_len(p, n, threadIdx.x == 0);
            T *out = static_cast<T *>(p.out) + (int64_t)n * p.Hq * D;
            for (int i = threadIdx.x; i < p.Hq * D; i += blockDim.x) out[i] = from_f32<T>(0.f);
            if (p.lse)
                for (int i = threadIdx.x; i < p.Hq; i += blockDim.x) p.lse[(int64_t)n * p.Hq + i] = -INFINITY;
        }
}

// One partial result of an item of HB query heads: m, l (base-2 logarithms) per
// head, then, from 16 bytes on, a[d] per head.
__host__ __device__ constexpr int part_head(int HB) { return (HB * 2 + 3) & ~3; }
__host__ __device__ constexpr int part_floats(int d, int HB) { return part_head(HB) + HB * d; }

// bf16, d = 64 or 128, pages of at least 8 tokens: the tensor-core form and the
// grid it runs on, with HB query heads per item.
cudaError_t launch_paged_decode_tc(const PagedParams &p, int d, int HB, int grid, cudaStream_t st);
constexpr int kTileTc = 128;
// e4m3 caches with bf16 queries; tokens of a row of its tiles, which have 128
constexpr int tokens_per_row(int d, int HB) { return d < 128 && HB <= 16 ? 2 : 1; }
cudaError_t launch_paged_decode_q8_tc(const PagedQ8Params &p, int d, int HB, int grid, cudaStream_t st);

}  // namespace kda
