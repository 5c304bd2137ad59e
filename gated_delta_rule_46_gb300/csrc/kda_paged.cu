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
// Append: 2^lanes_log2 lanes per token, so that each has four vectors of k and of
// v under way.  Reads and writes each byte once: 133k tokens of 8 heads, d = 128,
// in 160 us (6.83 TB/s, the rate of a plain copy), 256 in 2.2 us; of one head in
// 24 us (57 with a warp per token), of 8 heads of 32 channels in 44 (65).
// ---------------------------------------------------------------------------
template <typename V>
__global__ void __launch_bounds__(256) paged_append_kernel(const AppendParams p) {
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int lanes = 1 << p.lanes_log2, lane = threadIdx.x & (lanes - 1);
    const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> p.lanes_log2;
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
    for (int i0 = lane; i0 < n; i0 += 4 * lanes) {
        V x[4], y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * lanes;
            if (i < n) {
                x[u] = k[i];
                y[u] = v[i];
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * lanes;
            if (i >= n) break;
            const int h = i / per;
            const int64_t to = (((((int64_t)page * p.Hkv + h) << p.page_shift) + at) * per) + (i - h * per);
            kc[to] = x[u];
            vc[to] = y[u];
        }
    }
}

cudaError_t launch_paged_append(AppendParams p, bool vec16, cudaStream_t st) {
    const int64_t n = (int64_t)p.Hkv * p.row_bytes / (vec16 ? 16 : 2);       // vectors of a token
    p.lanes_log2 = 5;
    while (p.lanes_log2 > 2 && n < (4 << p.lanes_log2)) --p.lanes_log2;
    const unsigned grid = (unsigned)(((p.total << p.lanes_log2) + 255) / 256);
    return launch_dependent(vec16 ? paged_append_kernel<uint4> : paged_append_kernel<uint16_t>, dim3(grid), 256, 0, st, 1, p);
}

// ---------------------------------------------------------------------------
// CUDA-core form (float32 caches, d = 32, pages of under eight tokens): d / 8
// lanes share a token, eight channels each of its key, its value, the queries
// and the outputs of HB heads, all in registers; a warp works on 256 / d tokens
// at a time and on U such rounds between corrections of its maximum.  A round's
// keys are reloaded as soon as its scores are out, and its values as soon as
// they are summed up, so that loads are always under way.  Lane groups and warps
// keep maxima, sums and outputs of their own, which are joined once per item.
//   64 rows of 8192 float32 tokens, 8 key-value heads of 128 channels, 4 query
// heads each, take 783 us: 5.5 TB/s, 81 % of the copy rate.  With 8 query heads each
// it is 59 %, as then two rounds are all that the registers hold and the FMAs of a
// byte are twice as many; bf16 pages of 4 tokens, 52 %.
// ---------------------------------------------------------------------------
constexpr int kTile = 64;

// Eight channels of a row as they are loaded: of lane l of the d / 8 that share it.
template <typename T, int D>
struct Ch8;
template <int D>
struct Ch8<float, D> {
    float4 a = {}, b = {};
    static __device__ int channel(int l, int e) { return (e & 4) * (D / 8) + l * 4 + (e & 3); }
    __device__ void load(const float *row, int l) {
        a = *reinterpret_cast<const float4 *>(row + l * 4);
        b = *reinterpret_cast<const float4 *>(row + D / 2 + l * 4);
    }
    __device__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
template <int D>
struct Ch8<__nv_bfloat16, D> {
    uint4 u = {};
    static __device__ int channel(int l, int e) { return l * 8 + e; }
    __device__ void load(const __nv_bfloat16 *row, int l) { u = *reinterpret_cast<const uint4 *>(row + l * 8); }
    __device__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

template <typename T, int D, int HB>
struct Simt {
    static constexpr int WARPS = HB == 4 ? 10 : 8;                         // registers for as many
    static constexpr int U = HB == 4 || sizeof(T) == 2 ? 4 : 2;            // rounds between corrections
    static constexpr int LPT = D / 8, TPW = 32 / LPT;                      // lanes per token, tokens per warp
    static constexpr uint32_t smem = sizeof(float) * WARPS * HB * (D + 2);
};

template <typename T, int D, int HB>
__global__ void __launch_bounds__(Simt<T, D, HB>::WARPS * 32, 1) paged_decode_simt_kernel(const PagedParams p) {
    using S = Simt<T, D, HB>;
    constexpr int TILE = kTile, U = S::U, LPT = S::LPT, STEP = S::WARPS * S::TPW, NT = S::WARPS * 32;
    extern __shared__ float sm[];                     // of each warp: m and l [HB], outputs [HB][D]
    __shared__ int64_t s_sum[257];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l8 = lane % LPT;
    const int nb = (p.G + HB - 1) / HB, items = p.Hkv * nb;
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

    while (w < w1) {
        const int len = clamp_len(p, n, tid == 0 && item == 0 && tile == 0);
        const int kvh = item / nb, g0 = (item % nb) * HB, hb = min(HB, p.G - g0);
        const int hq0 = kvh * p.G + g0;
        const int64_t first = tile, last = min(nt, tile + (w1 - w));      // tiles [first, last) of the item
        const int end = (int)min(last * TILE, (int64_t)len);
        const int32_t *table = p.table + (int64_t)n * p.max_pages;
        int t = (int)(first * TILE) + warp * S::TPW + lane / LPT;         // this lane's token of the first round

        float q[HB][8];
#pragma unroll
        for (int h = 0; h < HB; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                q[h][e] = h < hb ? to_f32(static_cast<const T *>(p.q)[(int64_t)n * p.ldq + (int64_t)(hq0 + h) * D +
                                                                      Ch8<T, D>::channel(l8, e)]) * sc2
                                 : 0.f;
        float m[HB], l[HB], acc[HB][8];
#pragma unroll
        for (int h = 0; h < HB; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[h][e] = 0.f;
        }

        // pages of the U rounds from token t on (-1: no token), and rows of a cache on them
        auto pages = [&](int t, int (&pg)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                pg[u] = -1;
                if (t + u * STEP < end) {
                    pg[u] = table[(t + u * STEP) >> p.page_shift];
                    if (pg[u] < 0 || pg[u] >= p.num_pages) {
                        if (l8 == 0) report_status(p.status, KDA_ERR_INVALID_ARG);
                        pg[u] = -1;
                    }
                }
            }
        };
        auto fetch = [&](const T *cache, int t, const int (&pg)[U], Ch8<T, D> (&x)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                x[u] = Ch8<T, D>();
                if (pg[u] >= 0)
                    x[u].load(cache + (((((int64_t)pg[u] * p.Hkv + kvh) << p.page_shift) +
                                        ((t + u * STEP) & ((1 << p.page_shift) - 1))) * D), l8);
            }
        };
        Ch8<T, D> k[U], v[U];
        int pg[U], pn[U];
        pages(t, pg);
        fetch(kc, t, pg, k);
        fetch(vc, t, pg, v);
        pages(t + U * STEP, pn);
        // the rounds of a warp's lanes are the same in number: the shuffles are the whole warp's
        const int t0 = (int)(first * TILE) + warp * S::TPW;
        for (int r = t0; r < end; r += U * STEP, t += U * STEP) {
            float s[U][HB];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[8];
                k[u].get(x);
#pragma unroll
                for (int h = 0; h < HB; ++h) {
                    float a = x[0] * q[h][0];
#pragma unroll
                    for (int e = 1; e < 8; ++e) a = fmaf(x[e], q[h][e], a);
                    s[u][h] = a;
                }
            }
            fetch(kc, t + U * STEP, pn, k);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int h = 0; h < HB; ++h) {
#pragma unroll
                    for (int o = 1; o < LPT; o <<= 1) s[u][h] += __shfl_xor_sync(0xffffffffu, s[u][h], o);
                    if (pg[u] < 0) s[u][h] = -INFINITY;
                }
#pragma unroll
            for (int h = 0; h < HB; ++h) {
                float mn = m[h];
#pragma unroll
                for (int u = 0; u < U; ++u) mn = fmaxf(mn, s[u][h]);
                // rounds without a token leave everything as it is
                const float mu = mn == -INFINITY ? 0.f : mn, f = tc::ex2(m[h] - mu);
                m[h] = mn;
                l[h] *= f;
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[h][e] *= f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    s[u][h] = tc::ex2(s[u][h] - mu);
                    l[h] += s[u][h];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[8];
                v[u].get(x);
#pragma unroll
                for (int h = 0; h < HB; ++h)
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[h][e] = fmaf(s[u][h], x[e], acc[h][e]);
            }
            fetch(vc, t + U * STEP, pn, v);
#pragma unroll
            for (int u = 0; u < U; ++u) pg[u] = pn[u];
            pages(t + 2 * U * STEP, pn);
        }

        // join the warp's lane groups, then the warps
#pragma unroll
        for (int o = LPT; o < 32; o <<= 1)
#pragma unroll
            for (int h = 0; h < HB; ++h) {
                const float mo = __shfl_xor_sync(0xffffffffu, m[h], o), lo = __shfl_xor_sync(0xffffffffu, l[h], o);
                const float mn = fmaxf(m[h], mo), mu = mn == -INFINITY ? 0.f : mn;
                const float f = tc::ex2(m[h] - mu), fo = tc::ex2(mo - mu);
                m[h] = mn;
                l[h] = fmaf(l[h], f, lo * fo);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[h][e] = fmaf(acc[h][e], f, __shfl_xor_sync(0xffffffffu, acc[h][e], o) * fo);
            }
        __syncthreads();                              // the item before is written
        float *mine = sm + warp * HB * (D + 2);
        if (lane < LPT)
#pragma unroll
            for (int h = 0; h < HB; ++h) {
                if (lane == 0) { mine[2 * h] = m[h]; mine[2 * h + 1] = l[h]; }
#pragma unroll
                for (int e = 0; e < 8; ++e) mine[2 * HB + h * D + Ch8<T, D>::channel(l8, e)] = acc[h][e];
            }
        __syncthreads();
        const bool whole = first == 0 && last == nt;
        float *part = p.part + ((int64_t)blockIdx.x * 2 + (first == 0 ? 1 : 0)) * part_floats(D, HB);
        for (int i = tid; i < hb * D; i += NT) {
            const int h = i / D, c = i % D;
            float mx = -INFINITY;
#pragma unroll
            for (int x = 0; x < S::WARPS; ++x) mx = fmaxf(mx, sm[x * HB * (D + 2) + 2 * h]);
            const float mu = mx == -INFINITY ? 0.f : mx;
            float ls = 0.f, a = 0.f;
#pragma unroll
            for (int x = 0; x < S::WARPS; ++x) {
                const float *o = sm + x * HB * (D + 2);
                const float f = tc::ex2(o[2 * h] - mu);
                ls = fmaf(o[2 * h + 1], f, ls);
                a = fmaf(o[2 * HB + h * D + c], f, a);
            }
            if (whole) {
                static_cast<T *>(p.out)[((int64_t)n * p.Hq + hq0 + h) * D + c] =
                    from_f32<T>(ls > 0.f ? a / ls : (ls == 0.f ? 0.f : ls));
                if (c == 0 && p.lse) p.lse[(int64_t)n * p.Hq + hq0 + h] = (mx + log2f(ls)) / kLog2E;
            } else {
                part[HB * 2 + h * D + c] = a;
                if (c == 0) { part[2 * h] = mx; part[2 * h + 1] = ls; }
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

// Query heads per item of the tensor-core form: one pass over the cache for up to 32 of them (64 rows of 8192 tokens, 2
// key-value heads, 32 query heads each: 97 us, 163 in two passes of 16).
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
// Query heads per item of the CUDA-core form: what its registers hold, and four where there are no more (float32, 64 rows
// of 8192 tokens, 2 key-value heads, 4 query heads each: 208 us, 279 in items of eight).
static int heads_simt(int G) { return G <= 4 ? 4 : 8; }
static int grid_simt(int N, int64_t max_tokens, int Hkv, int G) {
    const int HB = heads_simt(G);
    return grid_for(N, max_tokens, Hkv * ((G + HB - 1) / HB), kTile, sm_count());
}

size_t paged_decode_workspace_bytes(int N, int64_t max_tokens, int Hq, int Hkv, int d) {
    const int G = Hq / Hkv;
    if (max_tokens <= (kTile < kTileTc ? kTile : kTileTc)) return 16;     // one tile: nothing to join
    const size_t tc = (size_t)grid_tc(N, max_tokens, Hkv, G) * 2 * part_floats(d, heads_tc(G));
    const size_t simt = (size_t)grid_simt(N, max_tokens, Hkv, G) * 2 * part_floats(d, heads_simt(G));
    return sizeof(float) * (tc > simt ? tc : simt);
}

template <typename T, int D, int HB>
static cudaError_t paged_simt(PagedParams p, cudaStream_t st) {
    using S = Simt<T, D, HB>;
    p.lone = ((int64_t)p.max_pages << p.page_shift) <= kTile;
    auto *kernel = paged_decode_simt_kernel<T, D, HB>;
    cudaError_t e = allow_smem<paged_decode_simt_kernel<T, D, HB>>(S::smem);
    if (e != cudaSuccess) return e;
    const int grid = grid_simt(p.N, (int64_t)p.max_pages << p.page_shift, p.Hkv, p.G);
    if ((e = launch_dependent(kernel, dim3(grid), S::WARPS * 32, S::smem, st, 1, p)) != cudaSuccess) return e;
    return launch_join<T, D, kTile, HB>(p, grid, st);
}

template <typename T>
static cudaError_t paged_dispatch(const PagedParams &p, int d, cudaStream_t st) {
    const bool four = heads_simt(p.G) == 4;
    switch (d) {
        case 32: return four ? paged_simt<T, 32, 4>(p, st) : paged_simt<T, 32, 8>(p, st);
        case 64: return four ? paged_simt<T, 64, 4>(p, st) : paged_simt<T, 64, 8>(p, st);
        case 128: return four ? paged_simt<T, 128, 4>(p, st) : paged_simt<T, 128, 8>(p, st);
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
