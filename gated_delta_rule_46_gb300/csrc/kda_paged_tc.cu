// kda_paged_tc.cu -- attention of one token per sequence over a paged cache on
// the tensor cores (bf16, d = 64 or 128).
//
// The cache is the traffic: 2 d bytes each of K and V per cached token and
// key-value head, read once.  So that it goes from HBM to the MMAs without
// passing through registers, the cached tokens are the M side of both products:
//   S^T [128 tokens x heads] = K Q^T          (K tile as it lies in the page)
//   O^T [d x heads]          = V^T P^T        (V tile read along its tokens)
// and the query heads that share a key-value head (padded to HB = 16 or 32) are
// the N side.  Pages come in by TMA, one copy per page and 64 channels, into
// rings of 128-token tiles of K and of V (up to 192 KB under way per SM).
//
// Roles of the 12 warps: 0 loads, 1 issues the MMAs (the next tile's S^T before
// this tile's O^T), 2 zeroes rows of V that hold no token (a masked weight of 0
// does not silence a NaN there), 3 stages Q, 4-7 run the softmax (thread =
// token), 8-11 keep the running output (thread = channel) in float32 registers,
// rescaling it by e^{m_old - m_new} tile by tile, so that TMEM is only read.
// The weights P are rounded to bf16 for the second product (2^-9 of each, the
// size of the output's own rounding); maxima, sums and outputs are float32.
//
// Bound by reading the cache: a ragged batch with 2.1 GB of it takes 317 us (6.75
// TB/s, the rate of a plain copy), one row of 131072 tokens (537 MB, split over all
// SMs and joined) 88 us (6.1 TB/s; 79 at the copy rate, the rest is the launch, the
// first pages' latency and the join).  With d = 64 a tile is half as large and takes
// the softmax warps about as long: 64 rows of 8192 tokens, 8 key-value heads, 4 query
// heads each, run at 94 % of the copy rate, and at 79 % if the softmax works on all 16
// of the MMA's columns.
#include <cuda.h>

#include "kda_paged.cuh"
#include "kda_tc_util.cuh"
#include "kda_tmap.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int TILE = kTileTc;
constexpr int NSMAX = 6;                          // stages of the K and of the V ring, at most
constexpr long long kWaitBudget = 2000000000LL;   // cycles (about one second)
constexpr long long kDrain = 20000000LL;
constexpr uint32_t kSub = TILE * 128;             // 128 tokens x 64 channels, 128-byte swizzled rows

enum Bar { KFULL, KFREE = KFULL + NSMAX, VFULL = KFREE + NSMAX, VFREE = VFULL + NSMAX, VCLEAN = VFREE + NSMAX, SD = VCLEAN + NSMAX,
           PREADY = SD + 2, PVD = PREADY + 2, OFREE = PVD + 2, QFULL = OFREE + 2, QFREE = QFULL + 2, IREADY = QFREE + 2,
           IFREE = IREADY + 2, NBAR = IFREE + 2 };

template <int D, int HB>
struct Lay {
    static constexpr uint32_t tile = kSub * (D / 64);
    // as many stages as fit 227 KB
    static constexpr int NS = D == 64 ? (HB == 16 ? 6 : 5) : (HB == 16 ? 3 : 2);
    static constexpr uint32_t K = 0, V = NS * tile, Q = 2 * NS * tile, q_bytes = HB * D * 2;
    static constexpr uint32_t P = Q + 2 * q_bytes, p_bytes = HB * TILE * 2;
    static constexpr uint32_t F = P + 2 * p_bytes;                   // float: factors [2][HB]
    static constexpr uint32_t RED = F + 2 * HB * 4;                  // maxima [2][4][HB]
    static constexpr uint32_t SUM = RED + 8 * HB * 4;                // sums [2][4][HB], maxima [2][HB]
    static constexpr uint32_t bytes = SUM + 10 * HB * 4;
};

// The tiles of this CTA in order: (sequence, item, tile); every role walks its
// own copy.  The next sequence's length is read a sequence ahead.
struct Walk {
    int64_t w, w1, nt, tile;
    int n, item, items, len, raw, ahead;      // len: raw, clamped to the table
    __device__ void start(const PagedParams &p, const Split &sp, int items_) {
        items = items_;
        w = (int64_t)blockIdx.x * sp.W / sp.g;
        w1 = (int64_t)(blockIdx.x + 1) * sp.W / sp.g;
        n = sp.n;
        raw = p.lens[n];
        len = clamped(p, raw);
        ahead = n + 1 < p.N ? p.lens[n + 1] : 0;
        nt = (len + TILE - 1) / TILE;
        item = (int)((w - sp.cum * items) / nt);
        tile = (w - sp.cum * items) - item * nt;
    }
    __device__ bool more() const { return w < w1; }
    // end of this CTA's part of the item
    __device__ int64_t last() const { return nt < tile + (w1 - w) ? nt : tile + (w1 - w); }
    __device__ void next_item(const PagedParams &p, int64_t done) {
        w += done;
        if (w >= w1) return;
        tile = 0;
        if (++item == items) {
            item = 0;
            do {
                raw = ahead;
                len = clamped(p, raw);
                ahead = ++n + 1 < p.N ? p.lens[n + 1] : 0;
            } while (len == 0 && n < p.N);
            nt = (len + TILE - 1) / TILE;
        }
    }
};

__device__ __forceinline__ bool warp_wait(uint64_t *bar, int phase) {
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar, phase & 1, kWaitBudget));
}
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar);
}
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t addr, uint32_t lead) {
    return (ptx::sdesc_kmajor_sw128(addr) & ~((uint64_t)0x3FFF << 16)) | ((uint64_t)((lead >> 4) & 0x3FFF) << 16);
}

// Eight bf16 from any even address.
__device__ __forceinline__ uint4 load8(const __nv_bfloat16 *p) {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = __bfloat16_as_ushort(p[i]);
    return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}

// N = 8 or 16 values per lane, combined over the warp: lane i ends with value i / (32 / N).
template <int N, typename Op>
__device__ __forceinline__ float reduce_lanes(float (&v)[N], int lane, Op op) {
#pragma unroll
    for (int n = N / 2, bit = 16; n >= 1; n >>= 1, bit >>= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
            v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, bit));
        }
    }
#pragma unroll
    for (int bit = 16 / N; bit >= 1; bit >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], bit));
    return v[0];
}
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[N]) {
    if constexpr (N == 8) ptx::tmem_ld8(addr, v);
    else ptx::tmem_ld16(addr, v);
}

// HB heads are the MMAs' columns (their least is 16), the first HR of them are worked on: the others' columns hold
// whatever is there and reach no one.
template <int D, int HB, int HR>
__global__ void __launch_bounds__(384, 1)
    paged_decode_tc_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const PagedParams p) {
    using L = Lay<D, HB>;
    constexpr int NS = L::NS;
    constexpr int HALVES = D / 64, W = HR < 16 ? HR : 16;       // heads at a time
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar[NBAR];
    __shared__ int64_t s_sum[257];
    __shared__ int s_n;
    __shared__ uint32_t s_tmem, s_abort, s_mask[8];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t base = ptx::smem_addr(sm);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nb = (p.G + HB - 1) / HB, items = p.Hkv * nb;
    constexpr uint32_t kCols = HB == 16 ? 64 : 128;

    ptx::pdl_wait();
    ptx::pdl_launch_dependents();     // the join kernel may start: it reads lengths before it waits
    const Split sp = find_split<TILE>(p, items, gridDim.x, blockIdx.x, 0, s_sum, &s_n);
    empty_sequences<__nv_bfloat16, TILE>(p, D);
    if ((int)blockIdx.x >= sp.g) return;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NBAR; ++i) {
            const bool four = (i >= PREADY && i < PREADY + 2) || (i >= OFREE && i < OFREE + 2) || i >= IREADY;
            ptx::mbar_init(&bar[i], four ? 4 : 1);
        }
        ptx::fence_mbar_init();
        s_abort = 0;
        ptx::prefetch_tensormap(&mk);
        ptx::prefetch_tensormap(&mv);
    }
    if (warp == 1) {
        ptx::tmem_alloc(&s_tmem, kCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = s_tmem;
    auto tm_s = [&](int b) { return tmem + b * HB; };
    auto tm_o = [&](int b) { return tmem + 2 * HB + b * HB; };
    Walk wk;
    wk.start(p, sp, items);
    const int rows = min(TILE, 1 << p.page_shift);        // tokens of a tile that one page holds
    const int pieces = TILE / rows;
    bool ok = true;

    if (warp == 0) {                                              // ---- loads: lane = page of the tile
        // a tile's page is looked up while the tile before it is loaded
        int64_t i = wk.tile, first = i, last = wk.last();
        auto lookup = [&](int at) {
            return lane < pieces && at < wk.len ? p.table[(int64_t)wk.n * p.max_pages + (at >> p.page_shift)] : 0;
        };
        int told = -1, at = (int)(i * TILE) + lane * rows, id = lookup(at);     // at: this page's first token of the tile
        for (int t = 0; ok && wk.more(); ++t) {
            if (wk.n != told) {
                told = wk.n;
                if (lane == 0 && wk.raw != wk.len) report_status(p.status, KDA_ERR_INVALID_ARG);
            }
            const int kvh = wk.item / nb, at0 = at;
            int page = -1;
            if (lane < pieces && at < wk.len) {
                if (id >= 0 && id < p.num_pages) page = id;
                else report_status(p.status, KDA_ERR_INVALID_ARG);
            }
            if (++i == last) {
                wk.next_item(p, last - first);
                if (wk.more()) { first = i = wk.tile; last = wk.last(); }
            }
            at = (int)(i * TILE) + lane * rows;
            id = wk.more() ? lookup(at) : 0;
            const uint32_t mask = __ballot_sync(0xffffffffu, page >= 0);
            const uint32_t bytes = (uint32_t)__popc(mask) * rows * 128u * HALVES;
            const int y = (int)(((((int64_t)page * p.Hkv) + kvh) << p.page_shift) + (at0 & ((1 << p.page_shift) - 1)));
            const int s = t % NS;
            for (int kv = 0; kv < 2; ++kv) {
                uint64_t *full = &bar[(kv ? VFULL : KFULL) + s], *free = &bar[(kv ? VFREE : KFREE) + s];
                if (t >= NS && !warp_wait(free, t / NS - 1)) { ok = false; break; }
                uint8_t *dst = sm + (kv ? L::V : L::K) + s * L::tile + lane * rows * 128;
                if (lane == 0) {
                    if (kv == 0) s_mask[t & 7] = mask;
                    ptx::mbar_arrive_expect_tx(full, bytes);
                }
                __syncwarp();
                if (page >= 0)
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) ptx::tma_load_2d(dst + h * kSub, kv ? &mv : &mk, h * 64, y, full);
            }
        }
    } else if (warp == 1) {                                       // ---- MMAs
        if (ptx::elect_one()) {
            const int total = (int)(wk.w1 - wk.w);
            // the tile that the S^T products have reached, one ahead of the O^T products
            int item_no = 0;
            int64_t i = wk.tile, last = wk.last(), first = i;
            const uint32_t id_s = ptx::idesc_bf16_f32(128, HB), id_o = ptx::idesc_bf16_f32(128, HB) | (1u << 15);
            auto scores = [&](int t) {
                const int b = t & 1, s = t % NS;
                if (i == first && !ptx::mbar_wait(&bar[QFULL + (item_no & 1)], (item_no >> 1) & 1, kWaitBudget)) return false;
                if (!ptx::mbar_wait(&bar[KFULL + s], (t / NS) & 1, kWaitBudget)) return false;
                if (t >= 2 && !ptx::mbar_wait(&bar[PREADY + b], ((t >> 1) - 1) & 1, kWaitBudget)) return false;
                ptx::tc_fence_after_sync();
                mma_k<D / 16>(tm_s(b), base + L::K + s * L::tile, kSub, base + L::Q + (item_no & 1) * L::q_bytes, HB * 128,
                              id_s, false);
                ptx::mma_commit(&bar[SD + b]);
                ptx::mma_commit(&bar[KFREE + s]);
                if (++i == last) {
                    ptx::mma_commit(&bar[QFREE + (item_no & 1)]);
                    ++item_no;
                    wk.next_item(p, last - first);
                    if (wk.more()) { i = first = wk.tile; last = wk.last(); }
                }
                return true;
            };
            if (p.expire && blockIdx.x == 0) ok = ptx::mbar_wait(&bar[PVD], 0, kTestWait);
            ok = ok && scores(0);
            for (int t = 0; t < total && ok; ++t) {
                if (t + 1 < total && !scores(t + 1)) { ok = false; break; }
                const int b = t & 1, s = t % NS;
                if (!ptx::mbar_wait(&bar[PREADY + b], (t >> 1) & 1, kWaitBudget) ||
                    !ptx::mbar_wait(&bar[VCLEAN + s], (t / NS) & 1, kWaitBudget)) { ok = false; break; }
                ptx::tc_fence_after_sync();
                // (with d = 64 the upper 64 rows of V^T are the next bytes of the ring: rows of O^T that no one reads)
                const uint64_t a = sdesc_mn_sw128(base + L::V + s * L::tile, kSub);
                const uint64_t pb = ptx::sdesc_kmajor_sw128(base + L::P + b * L::p_bytes);
#pragma unroll
                for (int k = 0; k < TILE / 16; ++k)
                    ptx::mma_bf16_ss(tm_o(b), a + k * (2048 >> 4), pb + (((k >> 2) * (HB * 128) + (k & 3) * 32) >> 4), id_o,
                                     k > 0);
                ptx::mma_commit(&bar[PVD + b]);
                ptx::mma_commit(&bar[VFREE + s]);
            }
        }
    } else if (warp == 2) {                                       // ---- rows of V without a token
        int t = 0;
        while (ok && wk.more()) {
            const int len = wk.len;
            const int64_t first = wk.tile, last = wk.last();
            for (int64_t i = first; i < last; ++i, ++t) {
                const int s = t % NS;
                ok = warp_wait(&bar[VFULL + s], t / NS);
                if (!ok) break;
                const uint32_t mask = *static_cast<volatile uint32_t *>(&s_mask[t & 7]);
                const int left = len - (int)(i * TILE);
                if (left < TILE || __popc(mask) < pieces) {
                    // 16 bytes a lane and step, from the first row that may be without a token on
                    const int from = __popc(mask) < pieces ? 0 : min(max(left, 0), TILE);
                    for (int j = from * 8 + lane; j < TILE * 8; j += 32) {
                        const int r = j >> 3;
                        if (r < left && (mask >> (r / rows) & 1)) continue;
#pragma unroll
                        for (int h = 0; h < HALVES; ++h)
                            *reinterpret_cast<uint4 *>(sm + L::V + s * L::tile + h * kSub + j * 16) = make_uint4(0, 0, 0, 0);
                    }
                    ptx::fence_async_smem();
                }
                warp_arrive(&bar[VCLEAN + s]);
            }
            wk.next_item(p, last - first);
        }
    } else if (warp == 3) {                                       // ---- Q
        int item_no = 0;
        const bool q16 = reinterpret_cast<uintptr_t>(p.q) % 16 == 0 && p.ldq % 8 == 0;
        while (ok && wk.more()) {
            const int64_t first = wk.tile, last = wk.last();
            const int kvh = wk.item / nb, g0 = (wk.item % nb) * HB, hb = min(HB, p.G - g0);
            uint8_t *dst = sm + L::Q + (item_no & 1) * L::q_bytes;
            const __nv_bfloat16 *q =
                static_cast<const __nv_bfloat16 *>(p.q) + (int64_t)wk.n * p.ldq + ((int64_t)kvh * p.G + g0) * D;
            // eight channels per lane and step, all loads first
            constexpr int PER = HR * D / 256;
            uint4 u[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int j = lane + i * 32, h = j / (D / 8);
                u[i] = make_uint4(0, 0, 0, 0);
                if (h < hb) {
                    if (q16) u[i] = *reinterpret_cast<const uint4 *>(q + j * 8);
                    else u[i] = load8(q + j * 8);
                }
            }
            if (item_no >= 2) ok = warp_wait(&bar[QFREE + (item_no & 1)], (item_no >> 1) - 1);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int j = lane + i * 32, h = j / (D / 8), c = j % (D / 8);
                *reinterpret_cast<uint4 *>(dst + (c >> 3) * (HB * 128) + swz(h, c & 7)) = u[i];
            }
            ptx::fence_async_smem();
            warp_arrive(&bar[QFULL + (item_no & 1)]);
            ++item_no;
            wk.next_item(p, last - first);
        }
    } else if (warp < 8) {                                        // ---- softmax: thread = token of the tile
        const int q = warp & 3, j = q * 32 + lane;
        const float sc2 = p.scale * kLog2E;
        float *sf = reinterpret_cast<float *>(sm + L::F), *red = reinterpret_cast<float *>(sm + L::RED),
              *sums = reinterpret_cast<float *>(sm + L::SUM), *maxs = sums + 8 * HB;
        int t = 0, item_no = 0;
        while (ok && wk.more()) {
            const int len = wk.len;
            const int64_t first = wk.tile, last = wk.last();
            float m[HR], l[HR];
#pragma unroll
            for (int h = 0; h < HR; ++h) { m[h] = -INFINITY; l[h] = 0.f; }
            for (int64_t i = first; i < last; ++i, ++t) {
                const int b = t & 1;
                // the factors and weights of two tiles ago have been used
                ok = warp_wait(&bar[SD + b], t >> 1) && (t < 2 || warp_wait(&bar[OFREE + b], (t >> 1) - 1));
                float s[HR];
                if (ok) {
                    ptx::tc_fence_after_sync();
#pragma unroll
                    for (int h = 0; h < HR; h += W) {
                        float v[W];
                        tmem_load(tm_s(b) + ((uint32_t)q << 21) + h, v);
                        ptx::tmem_ld_wait(v);
                        const bool in = (int)(i * TILE) + j < len &&
                                        (*static_cast<volatile uint32_t *>(&s_mask[t & 7]) >> (j / rows) & 1);
#pragma unroll
                        for (int e = 0; e < W; ++e) s[h + e] = v[e] = in ? v[e] * sc2 : -INFINITY;
                        const float mx = reduce_lanes(v, lane, [](float x, float y) { return fmaxf(x, y); });
                        if (lane % (32 / W) == 0) red[(b * 4 + q) * HB + h + lane / (32 / W)] = mx;
                    }
                }
                ok = !ptx::bar_any(1, 128, !ok);
                if (!ok) break;
                uint8_t *sp_ = sm + L::P + b * L::p_bytes + (j >> 6) * (HB * 128) + (j & 7) * 2;
#pragma unroll
                for (int h = 0; h < HR; h += 4) {
                    float mt[4], f[4];
                    ld4(red + (b * 4) * HB + h, mt);
#pragma unroll
                    for (int w = 1; w < 4; ++w) {
                        float o[4];
                        ld4(red + (b * 4 + w) * HB + h, o);
#pragma unroll
                        for (int e = 0; e < 4; ++e) mt[e] = fmaxf(mt[e], o[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float mn = fmaxf(m[h + e], mt[e]), mu = mn == -INFINITY ? 0.f : mn;
                        f[e] = ex2(m[h + e] - mu);
                        const float w = ex2(s[h + e] - mu);
                        l[h + e] = fmaf(l[h + e], f[e], w);
                        m[h + e] = mn;
                        *reinterpret_cast<__nv_bfloat16 *>(sp_ + swz(h + e, (j & 63) >> 3)) = __float2bfloat16_rn(w);
                    }
                    if (j == 0) *reinterpret_cast<float4 *>(sf + b * HB + h) = make_float4(f[0], f[1], f[2], f[3]);
                }
                ptx::fence_async_smem();
                ptx::tc_fence_before_sync();
                warp_arrive(&bar[PREADY + b]);
            }
            if (!ok) break;
            const int ib = item_no & 1;
            if (item_no >= 2) ok = warp_wait(&bar[IFREE + ib], (item_no >> 1) - 1);
            if (!ok) break;
#pragma unroll
            for (int h = 0; h < HR; h += W) {
                float v[W];
#pragma unroll
                for (int e = 0; e < W; ++e) v[e] = l[h + e];
                const float sum = reduce_lanes(v, lane, [](float x, float y) { return x + y; });
                if (lane % (32 / W) == 0) sums[(ib * 4 + q) * HB + h + lane / (32 / W)] = sum;
            }
            if (j == 0)
#pragma unroll
                for (int h = 0; h < HR; h += 4)
                    *reinterpret_cast<float4 *>(maxs + ib * HB + h) = make_float4(m[h], m[h + 1], m[h + 2], m[h + 3]);
            warp_arrive(&bar[IREADY + ib]);
            ++item_no;
            wk.next_item(p, last - first);
        }
    } else {                                                      // ---- output: thread = channel
        const int q = warp & 3, d = q * 32 + lane;
        const float *sf = reinterpret_cast<float *>(sm + L::F), *sums = reinterpret_cast<float *>(sm + L::SUM),
                    *maxs = sums + 8 * HB;
        int t = 0, item_no = 0;
        while (ok && wk.more()) {
            const int64_t first = wk.tile, last = wk.last();
            const int kvh = wk.item / nb, g0 = (wk.item % nb) * HB, hb = min(HB, p.G - g0);
            const int64_t row0 = (int64_t)wk.n * p.Hq + (int64_t)kvh * p.G + g0;
            float acc[HR];
#pragma unroll
            for (int h = 0; h < HR; ++h) acc[h] = 0.f;
            for (int64_t i = first; i < last; ++i, ++t) {
                const int b = t & 1;
                ok = warp_wait(&bar[PVD + b], t >> 1);
                if (!ok) break;
                ptx::tc_fence_after_sync();
#pragma unroll
                for (int h = 0; h < HR; h += W) {
                    float v[W], f[W];
                    tmem_load(tm_o(b) + ((uint32_t)q << 21) + h, v);
#pragma unroll
                    for (int e = 0; e < W; e += 8) ld8(sf + b * HB + h + e, f + e);
                    ptx::tmem_ld_wait(v);
#pragma unroll
                    for (int e = 0; e < W; ++e) acc[h + e] = fmaf(acc[h + e], f[e], v[e]);
                }
                ptx::tc_fence_before_sync();
                warp_arrive(&bar[OFREE + b]);
            }
            if (!ok) break;
            const int ib = item_no & 1;
            ok = warp_wait(&bar[IREADY + ib], item_no >> 1);
            if (!ok) break;
            const bool whole = first == 0 && last == wk.nt;
            float *part = p.part + ((int64_t)blockIdx.x * 2 + (first == 0 ? 1 : 0)) * part_floats(D, HB);
            // head d's sum and maximum by thread d; outputs by all, with a sum that is 0 or at least 1 (a maximum's own
            // weight), or infinite or NaN
            if (d < hb) {
                const float l = (sums[ib * 4 * HB + d] + sums[(ib * 4 + 1) * HB + d]) +
                                (sums[(ib * 4 + 2) * HB + d] + sums[(ib * 4 + 3) * HB + d]);
                const float m = maxs[ib * HB + d];
                if (!whole) { part[2 * d] = m; part[2 * d + 1] = l; }
                else if (p.lse) p.lse[row0 + d] = (m + log2f(l)) / kLog2E;
            }
            float l[HR];
            if (whole) {
#pragma unroll
                for (int h = 0; h < HR; h += 4) {
                    float x[4][4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) ld4(sums + (ib * 4 + w) * HB + h, x[w]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) l[h + e] = (x[0][e] + x[1][e]) + (x[2][e] + x[3][e]);
                }
            }
            warp_arrive(&bar[IFREE + ib]);
            if (d < D) {
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + row0 * D + d;
                if (whole) {
#pragma unroll
                    for (int h = 0; h < HR; ++h)
                        if (h < hb)
                            out[h * D] = __float2bfloat16_rn(l[h] > 0.f ? __fdividef(acc[h], l[h])
                                                                        : (l[h] == 0.f ? 0.f : l[h]));
                } else {
#pragma unroll
                    for (int h = 0; h < HR; ++h)
                        if (h < hb) part[HB * 2 + h * D + d] = acc[h];
                }
            }
            ++item_no;
            wk.next_item(p, last - first);
        }
    }
    if (!ok) {
        s_abort = 1;
        report_status(p.status, KDA_ERR_DEVICE_TIMEOUT);
    }
    __syncthreads();
    if (s_abort) {      // every copy and MMA in flight lands before the memory is given back
        const long long t0 = clock64();
        while (clock64() - t0 < kDrain) {}
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, kCols);
    }
}

template <int D, int HB, int HR>
cudaError_t launch(const PagedParams &p, int grid, cudaStream_t st) {
    CUtensorMap mk, mv;
    const uint64_t rows = (uint64_t)p.num_pages * p.Hkv << p.page_shift;
    const uint32_t box = p.page_shift < 7 ? 1u << p.page_shift : TILE;
    if (!make_map_2d(&mk, p.kc, true, rows, D, D * 2, box) || !make_map_2d(&mv, p.vc, true, rows, D, D * 2, box))
        return cudaErrorInvalidValue;
    // (d = 64: the MMA's unread rows reach one sub-tile past the last V tile)
    constexpr uint32_t smem = Lay<D, HB>::bytes + (D == 64 ? kSub : 0) + 1024;
    auto *kernel = paged_decode_tc_kernel<D, HB, HR>;
    static_assert(smem <= 229000, "shared memory");
    const cudaError_t e = allow_smem<paged_decode_tc_kernel<D, HB, HR>>(smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(grid), 384, smem, st, 1, mk, mv, p);
}

}  // namespace

cudaError_t launch_paged_decode_tc(const PagedParams &p, int d, int HB, int grid, cudaStream_t st) {
    if (d == 64) {
        if (p.G <= 8) return launch<64, 16, 8>(p, grid, st);
        return HB == 16 ? launch<64, 16, 16>(p, grid, st) : launch<64, 32, 32>(p, grid, st);
    }
    if (p.G <= 8) return launch<128, 16, 8>(p, grid, st);
    return HB == 16 ? launch<128, 16, 16>(p, grid, st) : launch<128, 32, 32>(p, grid, st);
}

}  // namespace kda
