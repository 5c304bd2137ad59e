// kda_paged.cu -- the paged key-value cache of a full-attention layer: writing
// new tokens into their pages, and softmax attention of one token per sequence
// over the cache, split over its length and joined.
//
// With scores s_t = scale q . k_t over any part of the cache, a part is
// summed up by m = max s_t, l = sum e^{s_t - m} and a = sum e^{s_t - m} v_t; two
// parts join as m = max(m1, m2), l = l1 e^{m1-m} + l2 e^{m2-m}, a likewise, and
// the whole gives out = a / l, lse = m + log l.
#include "kda_paged.cuh"
#include "kda_tc_util.cuh"
#include "kda_testing.h"
#include "sm100_ptx.cuh"

namespace kda {

// ---------------------------------------------------------------------------
// Append: one warp per token.  Reads and writes each byte once: 133k tokens of 8
// heads, d = 128, in 160 us (6.83 TB/s, the rate of a plain copy), 256 in 2.2 us.
// ---------------------------------------------------------------------------
template <typename V>
__global__ void __launch_bounds__(256) paged_append_kernel(const AppendParams p) {
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= p.total) return;
    int seq = (int)t;
    int64_t off = 0;
    if (p.cu_seqlens) {   // the last sequence that starts at or before t
        int lo = 0, hi = p.num_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.cu_seqlens[mid] <= t) lo = mid; else hi = mid;
        }
        seq = lo;
        off = t - p.cu_seqlens[seq];
        if (off < 0 || t >= p.cu_seqlens[seq + 1]) {   // offsets that do not cover t
            if (lane == 0) report_status(p.status, KDA_ERR_INVALID_ARG);
            return;
        }
    }
    const int start = p.start[seq];
    const int64_t pos = start + off;
    const int64_t pi = pos >> p.page_shift;
    const int page = (start < 0 || pi >= p.max_pages) ? -1 : p.table[(int64_t)seq * p.max_pages + pi];
    if (page < 0 || page >= p.num_pages) {
        if (lane == 0) report_status(p.status, KDA_ERR_INVALID_ARG);
        return;
    }
    const int at = (int)(pos & ((1 << p.page_shift) - 1));
    const int per = p.row_bytes / (int)sizeof(V);          // vectors per head
    const int n = p.Hkv * per;
    const V *k = reinterpret_cast<const V *>(static_cast<const uint8_t *>(p.k) + t * p.ldk);
    const V *v = reinterpret_cast<const V *>(static_cast<const uint8_t *>(p.v) + t * p.ldv);
    V *kc = static_cast<V *>(p.kc), *vc = static_cast<V *>(p.vc);
    // loads of eight vectors go before their stores (the compiler may not swap them)
    for (int i0 = lane; i0 < n; i0 += 128) {
        V x[4], y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * 32;
            if (i < n) {
                x[u] = k[i];
                y[u] = v[i];
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * 32;
            if (i >= n) break;
            const int h = i / per;
            const int64_t to = (((((int64_t)page * p.Hkv + h) << p.page_shift) + at) * per) + (i - h * per);
            kc[to] = x[u];
            vc[to] = y[u];
        }
    }
}

cudaError_t launch_paged_append(const AppendParams &p, bool vec16, cudaStream_t st) {
    const unsigned grid = (unsigned)((p.total + 7) / 8);
    return launch_dependent(vec16 ? paged_append_kernel<uint4> : paged_append_kernel<uint16_t>, dim3(grid), 256, 0, st, 1, p);
}

// ---------------------------------------------------------------------------
// CUDA-core form (float32 caches, d = 32, pages of under eight tokens): tiles of
// 64 tokens in shared memory as float32.  Bound by shared memory, from where each
// product takes an operand; it reads a float32 cache at 31 % of the copy rate.
// ---------------------------------------------------------------------------
constexpr int kHB = 16;        // query heads per item
constexpr int kTile = 64;

template <typename T, int D>
__global__ void __launch_bounds__(256) paged_decode_simt_kernel(const PagedParams p) {
    constexpr int TILE = kTile, LD = D + 4, NG = 256 / D, NA = kHB / NG;
    extern __shared__ float sm[];
    float *sK = sm, *sV = sK + TILE * LD, *sQ = sV + TILE * D, *sS = sQ + kHB * D;   // sS [kHB][TILE]
    float *sM = sS + kHB * TILE, *sL = sM + kHB, *sC = sL + kHB;                     // max, sum, correction
    __shared__ int64_t s_sum[257];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, wy = tid >> 5;
    const int nb = (p.G + kHB - 1) / kHB, items = p.Hkv * nb;
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();     // the join kernel may start: it reads lengths before it waits
    const Split sp = find_split<TILE>(p, items, gridDim.x, blockIdx.x, 0, s_sum, &s_n);
    empty_sequences<T, TILE>(p, D);
    if ((int)blockIdx.x >= sp.g) return;
    int64_t w = (int64_t)blockIdx.x * sp.W / sp.g;
    const int64_t w1 = (int64_t)(blockIdx.x + 1) * sp.W / sp.g;
    int n = sp.n;
    int64_t nt = tiles_of<TILE>(p, n);
    int item = (int)((w - sp.cum * items) / nt);
    int64_t tile = (w - sp.cum * items) - item * nt;
    const float sc2 = p.scale * kLog2E;
    const T *kc = static_cast<const T *>(p.kc), *vc = static_cast<const T *>(p.vc);
    const int col = tid % D, hg = tid / D;

    while (w < w1) {
        const int len = clamp_len(p, n, tid == 0 && item == 0 && tile == 0);
        const int kvh = item / nb, g0 = (item % nb) * kHB, hb = min(kHB, p.G - g0);
        const int hq0 = kvh * p.G + g0;
        const int64_t first = tile, last = min(nt, tile + (w1 - w));      // tiles [first, last) of the item
        __syncthreads();
        for (int i = tid; i < hb * D; i += 256)
            sQ[i] = to_f32(static_cast<const T *>(p.q)[(int64_t)n * p.ldq + (int64_t)hq0 * D + i]) * sc2;
        if (tid < kHB) { sM[tid] = -INFINITY; sL[tid] = 0.f; }
        float acc[NA];
#pragma unroll
        for (int i = 0; i < NA; ++i) acc[i] = 0.f;
        for (; tile < last; ++tile) {
            const int t0 = (int)(tile * TILE);
            __syncthreads();
            for (int i = tid; i < TILE * (D / 4); i += 256) {
                const int r = i / (D / 4), c = (i % (D / 4)) * 4;
                float kk[4] = {}, vv[4] = {};
                if (t0 + r < len) {
                    const int pg = p.table[(int64_t)n * p.max_pages + ((t0 + r) >> p.page_shift)];
                    if (pg >= 0 && pg < p.num_pages) {
                        const int64_t at = (((((int64_t)pg * p.Hkv + kvh) << p.page_shift) +
                                             ((t0 + r) & ((1 << p.page_shift) - 1))) * D) + c;
#pragma unroll
                        for (int e = 0; e < 4; ++e) { kk[e] = to_f32(kc[at + e]); vv[e] = to_f32(vc[at + e]); }
                    } else {
                        if (c == 0) report_status(p.status, KDA_ERR_INVALID_ARG);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) { sK[r * LD + c + e] = kk[e]; sV[r * D + c + e] = vv[e]; }
            }
            __syncthreads();
            {   // scores: thread = token x every fourth head
                const int j = tid & 63;
                bool ok = t0 + j < len;
                if (ok) {
                    const int pg = p.table[(int64_t)n * p.max_pages + ((t0 + j) >> p.page_shift)];
                    ok = pg >= 0 && pg < p.num_pages;
                }
                for (int g = tid >> 6; g < hb; g += 4) {
                    float a = 0.f;
#pragma unroll 8
                    for (int c = 0; c < D; c += 4) {
                        float x[4], y[4];
                        tc::ld4(sQ + g * D + c, x);
                        tc::ld4(sK + j * LD + c, y);
                        a = fmaf(x[0], y[0], a); a = fmaf(x[1], y[1], a);
                        a = fmaf(x[2], y[2], a); a = fmaf(x[3], y[3], a);
                    }
                    sS[g * TILE + j] = ok ? a : -INFINITY;
                }
            }
            __syncthreads();
            for (int g = wy; g < hb; g += 8) {   // softmax of one head per warp
                const float s0 = sS[g * TILE + lane], s1 = sS[g * TILE + 32 + lane];
                float m = fmaxf(s0, s1);
#pragma unroll
                for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                const float mo = sM[g], mn = fmaxf(mo, m);
                // a tile with nothing in it leaves everything as it is
                const float mu = mn == -INFINITY ? 0.f : mn;
                const float p0 = exp2f(s0 - mu), p1 = exp2f(s1 - mu);
                float l = p0 + p1;
#pragma unroll
                for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                sS[g * TILE + lane] = p0;
                sS[g * TILE + 32 + lane] = p1;
                __syncwarp();
                if (lane == 0) {
                    const float f = exp2f(mo - mu);
                    sC[g] = f;
                    sM[g] = mn;
                    sL[g] = sL[g] * f + l;
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                const int g = hg + i * NG;
                if (g >= hb) break;
                float a = acc[i] * sC[g];
#pragma unroll 8
                for (int j = 0; j < TILE; ++j) a = fmaf(sS[g * TILE + j], sV[j * D + col], a);
                acc[i] = a;
            }
        }
        __syncthreads();
        if (first == 0 && last == nt) {
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                const int g = hg + i * NG;
                if (g >= hb) break;
                const float l = sL[g];
                static_cast<T *>(p.out)[((int64_t)n * p.Hq + hq0 + g) * D + col] =
                    from_f32<T>(l > 0.f ? acc[i] / l : (l == 0.f ? 0.f : l));
                if (col == 0 && p.lse) p.lse[(int64_t)n * p.Hq + hq0 + g] = (sM[g] + log2f(l)) / kLog2E;
            }
        } else {
            float *part = p.part + ((int64_t)blockIdx.x * 2 + (first == 0 ? 1 : 0)) * part_floats(D, kHB);
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                const int g = hg + i * NG;
                if (g >= hb) break;
                part[kHB * 2 + g * D + col] = acc[i];
                if (col == 0) { part[2 * g] = sM[g]; part[2 * g + 1] = sL[g]; }
            }
        }
        w += last - first;
        if (w < w1) {   // the next item
            tile = 0;
            if (++item == items) {
                item = 0;
                do { ++n; nt = tiles_of<TILE>(p, n); } while (nt == 0);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Join: one warp per sequence and query head, eight heads per CTA.  Heads whose
// item one CTA had whole are done already; a sequence without tokens gets
// zeros.  A long row has a part from nearly every CTA: their maxima and sums
// are read a part per lane and joined by shuffles, then the weighted rows are
// summed in order, with as many loads under way as the unrolling gives.
// ---------------------------------------------------------------------------
template <typename T, int D, int TILE, int HB>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedParams p, int grid) {
    __shared__ int64_t s_sum[257];
    __shared__ int s_n;
    const int n = blockIdx.x, hq = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int nb = (p.G + HB - 1) / HB, items = p.Hkv * nb;
    constexpr int E = D / 32;
    T *out = static_cast<T *>(p.out);
    const int64_t nt = tiles_of<TILE>(p, n);
    if (nt == 0) {
        ptx::pdl_wait();         // this grid's end stands for the one before it too
        if (blockIdx.y == 0) empty_sequence<T>(p, n, D);
        return;
    }
    const Split sp = find_split<TILE>(p, items, grid, -1, n, s_sum, &s_n);
    ptx::pdl_wait();             // the partial results
    if (hq >= p.Hq) return;
    const int kvh = hq / p.G, gi = hq % p.G, item = kvh * nb + gi / HB, g = gi % HB;
    const int64_t s = sp.cum * items + item * nt, e = s + nt;
    const int b0 = (int)(((s + 1) * sp.g - 1) / sp.W), b1 = (int)((e * sp.g - 1) / sp.W);
    if (b0 == b1) return;
    // CTA b0 starts the item (slot 1), the others go on with it (slot 0)
    auto part = [&](int b) { return p.part + ((int64_t)b * 2 + (b == b0 ? 1 : 0)) * part_floats(D, HB); };
    float m = -INFINITY;
    for (int b = b0 + lane; b <= b1; b += 32) m = fmaxf(m, part(b)[2 * g]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float mu = m == -INFINITY ? 0.f : m;
    float l = 0.f, a[E] = {};
    for (int c0 = b0; c0 <= b1; c0 += 32) {
        const int b = c0 + lane;
        const float f = b <= b1 ? exp2f(part(b)[2 * g] - mu) : 0.f;
        l += b <= b1 ? part(b)[2 * g + 1] * f : 0.f;
        const int cnt = min(32, b1 - c0 + 1);
#pragma unroll 8
        for (int i = 0; i < cnt; ++i) {
            const float *x = part(c0 + i) + HB * 2 + g * D + lane * E;
            const float w = __shfl_sync(0xffffffffu, f, i);
#pragma unroll
            for (int j = 0; j < E; ++j) a[j] = fmaf(x[j], w, a[j]);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const int64_t row = (int64_t)n * p.Hq + hq;
#pragma unroll
    for (int i = 0; i < E; ++i) out[row * D + lane * E + i] = from_f32<T>(l > 0.f ? a[i] / l : (l == 0.f ? 0.f : l));
    if (lane == 0 && p.lse) p.lse[row] = (m + log2f(l)) / kLog2E;
}

template <typename T, int D, int TILE, int HB>
static cudaError_t launch_join(const PagedParams &p, int grid, cudaStream_t st) {
    if (p.lone) return cudaSuccess;
    return launch_dependent(paged_join_kernel<T, D, TILE, HB>, dim3((unsigned)p.N, (unsigned)((p.Hq + 7) / 8)), 256, 0, st, 1,
                            p, grid);
}

// Query heads per item of the tensor-core form: one pass over the cache for up to 32 of them.
static int heads_tc(int G) { return G <= 16 ? 16 : 32; }

// The tensor-core form: its TMA copies take whole 8-row groups of a page, and
// their row coordinates are 32-bit.
static bool use_tc(const PagedParams &p, int d, bool bf16) {
    return bf16 && d >= 64 && p.page_shift >= 3 && p.num_pages > 0 && p.max_pages > 0 &&
           ((int64_t)p.num_pages * p.Hkv << p.page_shift) < (int64_t(1) << 31);
}

// CTAs that can have work: at most one per tile of the longest possible batch.
static int grid_for(int N, int64_t max_tokens, int items, int tile, int most) {
    const int64_t tiles = (int64_t)N * items * ((max_tokens + tile - 1) / tile);
    return (int)(tiles < 1 ? 1 : (tiles < most ? tiles : most));
}
static int grid_tc(int N, int64_t max_tokens, int Hkv, int G) {
    const int HB = heads_tc(G);
    return grid_for(N, max_tokens, Hkv * ((G + HB - 1) / HB), kTileTc, sm_count());
}
static int grid_simt(int N, int64_t max_tokens, int Hkv, int G) {
    return grid_for(N, max_tokens, Hkv * ((G + kHB - 1) / kHB), kTile, 2 * sm_count());
}

size_t paged_decode_workspace_bytes(int N, int64_t max_tokens, int Hq, int Hkv, int d) {
    const int G = Hq / Hkv;
    if (max_tokens <= (kTile < kTileTc ? kTile : kTileTc)) return 0;      // one tile: nothing to join
    const size_t tc = (size_t)grid_tc(N, max_tokens, Hkv, G) * 2 * part_floats(d, heads_tc(G));
    const size_t simt = (size_t)grid_simt(N, max_tokens, Hkv, G) * 2 * part_floats(d, kHB);
    return sizeof(float) * (tc > simt ? tc : simt);
}

template <typename T, int D>
static cudaError_t paged_simt(PagedParams p, cudaStream_t st) {
    p.lone = ((int64_t)p.max_pages << p.page_shift) <= kTile;
    const size_t smem = sizeof(float) * (kTile * (D + 4) + kTile * D + kHB * D + kHB * kTile + 3 * kHB);
    cudaError_t e = allow_smem<paged_decode_simt_kernel<T, D>>((uint32_t)smem);
    if (e != cudaSuccess) return e;
    const int grid = grid_simt(p.N, (int64_t)p.max_pages << p.page_shift, p.Hkv, p.G);
    if ((e = launch_dependent(paged_decode_simt_kernel<T, D>, dim3(grid), 256, smem, st, 1, p)) != cudaSuccess) return e;
    return launch_join<T, D, kTile, kHB>(p, grid, st);
}

template <typename T>
static cudaError_t paged_dispatch(const PagedParams &p, int d, cudaStream_t st) {
    switch (d) {
        case 32: return paged_simt<T, 32>(p, st);
        case 64: return paged_simt<T, 64>(p, st);
        case 128: return paged_simt<T, 128>(p, st);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_paged_decode(const PagedParams &p, int d, bool bf16, cudaStream_t st) {
    if (!use_tc(p, d, bf16)) return bf16 ? paged_dispatch<__nv_bfloat16>(p, d, st) : paged_dispatch<float>(p, d, st);
    const int HB = heads_tc(p.G), grid = grid_tc(p.N, (int64_t)p.max_pages << p.page_shift, p.Hkv, p.G);
    PagedParams pt = p;
    pt.expire = take_layers_expire(KDA_TESTING_PAGED);
    pt.lone = ((int64_t)p.max_pages << p.page_shift) <= kTileTc;
    const cudaError_t e = launch_paged_decode_tc(pt, d, HB, grid, st);
    if (e != cudaSuccess) return e;
    if (d == 64)
        return HB == 16 ? launch_join<__nv_bfloat16, 64, kTileTc, 16>(pt, grid, st)
                        : launch_join<__nv_bfloat16, 64, kTileTc, 32>(pt, grid, st);
    return HB == 16 ? launch_join<__nv_bfloat16, 128, kTileTc, 16>(pt, grid, st)
                    : launch_join<__nv_bfloat16, 128, kTileTc, 32>(pt, grid, st);
}

}  // namespace kda
