// kda_paged_q8_tc.cu -- attention of one token per sequence over a paged cache in
// 8 bits on the tensor cores (bf16 queries and outputs).
//
// As in kda_paged_tc.cu the cached tokens are the M side of both products, so that
// the codes go from HBM to the MMAs without passing through registers:
//   S^T [128 rows x N] = K Q^T,    O^T [row bytes x N] = V^T P^T
// on e4m3 operands.  K and V are e4m3 as they lie in the cache, in rows of one token or,
// for up to 64 channels and 16 heads, of F = 2: a tile is 128 rows either way, and what a
// tile costs whatever it holds (waits, maxima, an MMA's 47 cycles of issue) is spent on
// twice the tokens.  Tokens e = 0, 1 of the rows have N columns of their own: S^T of e is
// the product with the e-th half of K's rows, and of O^T's columns of e only the e-th half
// of the rows is looked at, the sum of a token's weights and the other's values being noise.
//
// Q and the weights P, which need more than e4m3's four significant bits, come in two parts,
//   x = hi + lo / f,   hi = e4m3(x),   lo = e4m3(f (x - hi))
// whose products are added up.  For Q f is 1, and they share accumulators, or for up to 8
// heads, where an MMA's 16 columns have room for both parts, are in neighbouring columns.  With
// the largest of a head's channels at 224 or more that is exact for a bf16 query down to 2^-11
// of it, and off by 2^-10, 2^-18 of the largest, below.  For P, at most 128, f is 32, and the
// parts have columns of their own: eight bits of a weight are kept, as bf16 would, down to
// 2^-14 of the largest, and 2^-22 of that (2^-15 of 128) below.
//
// A token's scale of K multiplies its row of S^T.  Its scale of V goes into its
// weight: with the tile's largest scale of V u and largest product of both m,
//   m = max s + log v_scale / u,   P = 128 e^{s - m} v_scale / u,
//   O = O_before e^{m_before - m_now} + u / 128 e^{m - m_now} V^T P
// so that the weights use e4m3's range from the tile's largest on, whatever the rest of the row
// holds and whichever tokens the largest score and the largest scale belong to.  Tiles do not
// wait for each other's maxima: two groups of softmax warps work on tiles in turn.  Where a tile's
// scales are within a factor of 2, as they mostly are, m is its largest score, which is as much
// off at most (an error of 2^-21 of the largest); it is never taken more than 40 (base 2) below
// the largest score, so that sums of e^{s - m} stay finite.  A softmax thread has
// four rows and a quarter of the heads (TMEM's 16 x 256-bit reads), so that what is one for
// all tokens (maxima, their exponentials; worked out by a lane per head) is a vector or two.
//
// Roles of the 20 warps: 0-3 load tiles in turn (pages by TMA, scales by 4-byte copies),
// 4 issues the S^T MMAs, 5 zeroes rows of V that hold no token and issues the O^T MMAs,
// 6 and 7 split and stage Q of items in turn, 8-11 and 12-15 run the softmax of even and odd tiles, 16-19 keep
// the running output (thread = row of O^T) in float32 registers.  Items of 32 heads have one
// warp that loads, as their softmax takes 128 registers a thread.
//
// Measured (8 key-value heads unless said): 64 rows of up to 16384 tokens, 4 query heads of
// 128 channels each, 173 us, 0.91 of the copy rate; one row of 131072, 51 us (0.77), of which
// about 12 are the start, the first loads' latency and the join; with 16 query heads and up
// to 8192 tokens 98 us (0.81), 4 query heads of 64 channels 92 us (0.86), of 32 channels
// 89 (0.45); 128 rows of up to 8192, 4 key-value heads with 16 query heads of 64 channels,
// 74 us (0.53); 64 rows of up to 16384, 2 key-value heads with 32 query heads of 128 channels 67
// (0.59), of 64 channels 62 (0.32); 256 rows of up to 128 tokens 28 us.
// What bounds 16 heads of 64 channels is the softmax: a chain of some 450 instructions a thread and
// tile of 256 tokens, each about seven cycles after the one before with two such warps a
// scheduler (issue slots 49 %, no pipe above 40 %).  A third group of softmax warps spills
// registers (73 -> 85 us), and gains nothing where the scores are read from TMEM twice to need
// fewer (70.5 -> 73.4); moving what is freed from the load and MMA warps to them with setmaxnreg
// makes no difference to the compiler (103 us).  Freeing stages by the consumers instead of a
// second commit: 141 -> 152 us (4 heads, 64 channels, in rows of one token).
// Second parts of the weights with a step and columns of their own, and the largest product
// instead of the two maxima, cost 16 heads of 64 channels 70.6 -> 74.4 us, 4 heads of 32 channels
// 85.8 -> 88.5, short rows 27.4 -> 28.5 and long ones of 128 channels nothing; the reciprocal of u by
// an IEEE division cost 2 to 4 us more, the weights' power of two at the weights 0.5, room for
// large scores per tile instead of in the exponents' offset 1 to 3.5 %.
#include <cuda.h>

#include "kda_paged_tc.cuh"
#include "kda_tmap.cuh"

namespace kda {
namespace {

using namespace tc;
using namespace paged;

constexpr int NSMAX = 12;                         // stages of the K and of the V ring, at most
constexpr int SB = 4, RING = 16;                  // S^T buffers; tiles whose scales and page masks are kept
constexpr int QRING = 16;                         // items whose queries' factors are kept
constexpr int NG = 2;                             // groups of softmax warps
constexpr int LMAX = 4;                           // warps that load, at most
// A page mask or scales of tile t are read before O^T of tile t is issued, which V's stage of tile t + NS waits for; the warp
// that writes them again, for tile t + RING, has loaded tile t + RING - LMAX >= t + NS before.  An item's factors are written
// again once S^T of the item QRING - 2 behind it is done: of its last tiles one for each group of softmax warps waited for an
// S^T buffer that the group gave back after this item.
static_assert(RING >= NSMAX + LMAX && QRING >= SB + NG + 2, "rings");

enum Bar { KFULL, KFREE = KFULL + NSMAX, VFULL = KFREE + NSMAX, VFREE = VFULL + NSMAX, SCALES = VFREE + NSMAX, SD = SCALES + RING,
           SFREE = SD + SB, PREADY = SFREE + SB, PVD = PREADY + NG, OFREE = PVD + NG, QFULL = OFREE + NG, QFREE = QFULL + 2,
           IREADY = QFREE + 2, IFREE = IREADY + 2, NBAR = IFREE + 2 };

template <int D, int HB>
struct Lay {
    static constexpr int F = tokens_per_row(D, HB), RB = D * F;      // tokens and bytes of a row
    static constexpr int TOK = TILE * F, NBK = TOK / 16;             // tokens and, at most, blocks of a tile
    static constexpr bool BOTH = HB == 8;                            // both parts in the columns
    static constexpr int QN = BOTH ? 16 : HB, N = F * QN;            // columns of a token of the rows, of all
    static constexpr int PARTS = BOTH ? 1 : 2, HT = HB / 4;          // rounds of S^T's MMAs; heads of a softmax thread
    static constexpr int ON = BOTH ? N : 2 * N;                      // columns of P and O^T: both parts
    // roles, by their first warps; 32 heads need the registers of 16 warps
    static constexpr int LOADERS = HB == 32 ? 1 : LMAX;
    static constexpr int MMA_S = LOADERS, MMA_O = LOADERS + 1, STAGE_Q = LOADERS + 2, SOFTMAX = LOADERS == 1 ? 4 : 8;
    static constexpr int STAGERS = SOFTMAX - STAGE_Q;                // warps that stage Q, items in turn
    static constexpr int OUT = SOFTMAX + 4 * NG, THREADS = 32 * (OUT + 4);
    static constexpr uint32_t tile = TILE * RB;
    // about 190 KB of stages where there is room for as much
    static constexpr int NS = RB == 128 ? (HB == 32 || (HB == 16 && F == 2) ? 5 : 6) : RB == 64 ? (HB == 8 ? NSMAX : 10) : NSMAX;
    // (V first: with rows of less than 128 bytes the MMA's rows past them read what lies behind a stage, which no one looks at)
    static constexpr uint32_t V = 0, K = NS * tile, Q = 2 * NS * tile, q_part = QN * D, q_bytes = PARTS * q_part;
    static constexpr uint32_t P = Q + 2 * q_bytes, p_bytes = ON * TILE;
    static constexpr uint32_t SC = P + NG * p_bytes;                 // float: scales of K [RING][NBK], of V [RING][NBK]
    static constexpr uint32_t QS = SC + 2 * RING * NBK * 4;          // factors of the queries [QRING][HB]
    static constexpr uint32_t M = QS + QRING * HB * 4;               // maxima of the tile [NG][HB], u [NG] (padded to 4)
    static constexpr uint32_t RED = M + NG * HB * 4 + 16;            // maxima of the warps [NG][2][4][HB]
    static constexpr uint32_t SUM = RED + NG * 8 * HB * 4;           // sums of the item [2][4 NG][HB], maxima [2][NG][HB]
    static constexpr uint32_t STAT = SUM + 10 * NG * HB * 4;         // of each softmax and output warp: [4][HB]
    static constexpr uint32_t X = STAT + (4 * NG + 4) * 4 * HB * 4;  // outputs of an item's tokens e, F == 2: [HB][RB]
    static constexpr uint32_t bytes = X + (F == 2 ? HB * RB * 4 : 0);
    static constexpr uint32_t cols = SB * N + NG * ON <= 128 ? 128 : 256;    // TMEM: SB buffers of S^T, NG of O^T
    static_assert(SB * N + NG * ON <= cols, "tensor memory");
};
// The column of S^T, and the row of Q's stage, of head h: a softmax thread finds its HT heads in a row in its own columns.
template <int HB>
__device__ __forceinline__ int column(int h) {
    return HB == 8 ? h : HB == 16 ? 8 * (h >> 1 & 1) + 2 * (h >> 2) + (h & 1) : 8 * (h >> 1 & 3) + 2 * (h >> 3) + (h & 1);
}

// The column of O^T that the softmax threads write head h to (up to 8 heads: its first part, the second is two behind it).
template <int HB>
__device__ __forceinline__ constexpr int out_column(int h) {
    const int j = h & 3;
    return HB == 8 ? 2 * (h - j) + 4 * (j >> 1) + (j & 1) : HB == 16 ? h : 16 * (h >> 2 & 1) + 4 * (h >> 3) + j;
}

// Byte offset of the 16-byte chunk of a row, swizzled as TMA does it.
template <int D>
__device__ __forceinline__ uint32_t swizzled(int row, int chunk) {
    return (uint32_t)(row * D + ((chunk ^ (D == 128 ? row & 7 : D == 64 ? row >> 1 & 3 : row >> 2 & 1)) << 4));
}

// Two values in two parts each; of weights, which come kLow times too large, the second stays so.  (What the first
// leaves of a weight, at most 256 with all rounding, is at most 8.)
constexpr float kLow = 32.f;
// Exponents of the largest weights, which scales of V then bring to 2^12 = 128 kLow.  (Taken from a score as large as 2^26 a
// 16 leaves no rounding; and where the score itself is off by up to 1, from 2^24 on, a weight of 256 still has both parts.)
constexpr float kTop = 16.f, kShare = 0.0625f;
template <bool WEIGHT>
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    const __half2 w = __floats2half2_rn(x, y), first = WEIGHT ? __hmul2(w, __float2half2_rn(1.f / kLow)) : w;
    const uint16_t h = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(first), __NV_SATFINITE, __NV_E4M3);
    const __half2 r = __hfma2(__half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)), __float2half2_rn(WEIGHT ? -kLow : -1.f), w);
    hi = h;
    lo = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(r), __NV_SATFINITE, __NV_E4M3);
}

// N values per lane, combined over the lanes with the same lane % 4: lane i ends with value `mine` of them.
template <int N, typename Op>
__device__ __forceinline__ float reduce_rows(float (&v)[N], int lane, int &mine, Op op) {
    mine = 0;
#pragma unroll
    for (int n = N, bit = 16; bit >= 4; bit >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool up = lane & bit;
            mine += up ? n : 0;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
                v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, bit));
            }
        } else {
            v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], bit));
        }
    }
    return v[0];
}
template <int N>
__device__ __forceinline__ void ld_heads(const float *p, float (&x)[N]) {
    if constexpr (N == 2) {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        x[0] = v.x; x[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) ld4(p + i, x + i);
    }
}

template <int D, int HB>
__global__ void __launch_bounds__(Lay<D, HB>::THREADS, 1)
    paged_decode_q8_tc_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const PagedQ8Params p) {
    using L = Lay<D, HB>;
    constexpr int NS = L::NS, LOADERS = L::LOADERS, F = L::F, FS = F - 1, TOK = L::TOK;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar[NBAR];
    __shared__ int64_t s_sum[257];
    __shared__ int s_n;
    __shared__ uint32_t s_tmem, s_abort, s_mask[RING];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t base = ptx::smem_addr(sm);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nb = (p.G + HB - 1) / HB, items = p.Hkv * nb;

    if (threadIdx.x < NBAR) {         // what needs nothing of the kernels before overlaps them
        const int i = threadIdx.x;
        int count = 1;
        if (i >= SCALES && i < SD) count = 32;
        else if (i >= IREADY && i < IFREE) count = 4 * NG;
        else if ((i >= SFREE && i < PVD) || (i >= OFREE && i < QFULL) || i >= IFREE) count = 4;
        ptx::mbar_init(&bar[i], count);
        ptx::fence_mbar_init();
    }
    if (threadIdx.x == 0) {
        s_abort = 0;
        ptx::prefetch_tensormap(&mk);
        ptx::prefetch_tensormap(&mv);
    }
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();     // the join kernel may start: it reads lengths before it waits
    const Split sp = find_split<TOK>(p, items, gridDim.x, blockIdx.x, 0, s_sum, &s_n);
    if ((int)blockIdx.x >= sp.g) {
        empty_sequences<__nv_bfloat16>(p, D);
        return;
    }
    if (warp == L::MMA_S) {
        ptx::tmem_alloc(&s_tmem, L::cols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = s_tmem;
    auto tm_s = [&](int b) { return tmem + b * L::N; };
    auto tm_o = [&](int b) { return tmem + SB * L::N + b * L::ON; };
    WalkOf<TOK> wk;
    wk.start(p, sp, items);
    const int rows = min(TILE, 1 << (p.page_shift - FS)); // of a tile that one page holds
    const int pieces = TILE / rows, rows_shift = 31 - __clz(rows);
    float *const sc = reinterpret_cast<float *>(sm + L::SC), *const qs = reinterpret_cast<float *>(sm + L::QS),
                 *const sm_m = reinterpret_cast<float *>(sm + L::M), *const sums = reinterpret_cast<float *>(sm + L::SUM);
    bool ok = true;

    if (warp < LOADERS) {                                         // ---- loads: lane = page of the tile
        const int per = 1 << (p.page_shift - p.block_shift);      // scales of a page and head
        int t0 = 0;                                               // tiles before the item
        while (ok && wk.more()) {
            const int64_t first = wk.tile, last = wk.last();
            const int kvh = nb == 1 ? wk.item : wk.item / nb, len = wk.len;
            const int32_t *table = p.table + (int64_t)wk.n * p.max_pages;
            if (threadIdx.x == 0 && wk.raw != len) report_status(p.status, KDA_ERR_INVALID_ARG);
            for (int64_t i = first + ((warp - t0) & (LOADERS - 1)); i < last; i += LOADERS) {
                const int t = t0 + (int)(i - first), s = t % NS, r = t % RING;
                const int at = (int)(i * TOK) + lane * rows * F;  // this page's first token of the tile
                int page = -1;
                if (lane < pieces && at < len) {
                    page = table[at >> p.page_shift];
                    if (page < 0 || page >= p.num_pages) {
                        report_status(p.status, KDA_ERR_INVALID_ARG);
                        page = -1;
                    }
                }
                const uint32_t mask = __ballot_sync(0xffffffffu, page >= 0);
                // (a page before the first reads as zeros, as one that is missing)
                const int y = (at & ((1 << p.page_shift) - 1)) >> FS;
                // scales: a lane for each block of tokens
                const int off = lane << p.block_shift, from = (int)(i * TOK) + off;
                const int of = __shfl_sync(0xffffffffu, page, (off >> FS >> rows_shift) & 31);
                const bool block = off < TOK && from < len && of >= 0;
                const int64_t at_scale =
                    block ? ((int64_t)of * p.Hkv + kvh) * per + ((from & ((1 << p.page_shift) - 1)) >> p.block_shift) : 0;
                for (int kv = 0; kv < 2; ++kv) {
                    uint64_t *full = &bar[(kv ? VFULL : KFULL) + s], *free = &bar[(kv ? VFREE : KFREE) + s];
                    if (t >= NS && !warp_wait(free, t / NS - 1)) { ok = false; break; }
                    uint8_t *dst = sm + (kv ? L::V : L::K) + s * L::tile + lane * rows * L::RB;
                    if (lane == 0) {
                        if (kv == 0) s_mask[r] = mask;
                        ptx::mbar_arrive_expect_tx(full, L::tile);
                    }
                    __syncwarp();
                    if (lane < pieces) ptx::tma_load_4d(dst, kv ? &mv : &mk, 0, y, kvh, page, full);
                    if (kv == 0) {
                        if (lane < L::NBK) {
                            ptx::cp_async4(sc + r * L::NBK + lane, p.ks + at_scale, block);
                            ptx::cp_async4(sc + (RING + r) * L::NBK + lane, p.vs + at_scale, block);
                        }
                        ptx::cp_async_arrive(&bar[SCALES + r]);
                    }
                }
                if (!ok) break;
            }
            t0 += (int)(last - first);
            wk.next_item(p, last - first);
        }
    } else if (warp == L::MMA_S) {                                // ---- S^T
        if (ptx::elect_one()) {
            int item_no = 0;
            constexpr uint32_t id_s = ptx::idesc_e4m3_f32(128, L::QN, false);
            if (p.expire && blockIdx.x == 0) ok = ptx::mbar_wait(&bar[PVD], 0, kTestWait);
            for (int t = 0; ok && wk.more();) {
                const int64_t first = wk.tile, last = wk.last();
                const int ib = item_no & 1;
                ok = ptx::mbar_wait(&bar[QFULL + ib], (item_no >> 1) & 1, kWaitBudget);
                const uint64_t q = ptx::sdesc_rows<D>(base + L::Q + ib * L::q_bytes);
                constexpr int J = D / 32;
                for (int64_t i = first; i < last && ok; ++i, ++t) {
                    const int s = t % NS, b = t % SB;
                    ok = ptx::mbar_wait(&bar[KFULL + s], (t / NS) & 1, kWaitBudget) &&
                         (t < SB || ptx::mbar_wait(&bar[SFREE + b], (t / SB - 1) & 1, kWaitBudget));
                    if (!ok) break;
                    ptx::tc_fence_after_sync();
                    const uint64_t k = ptx::sdesc_rows<L::RB>(base + L::K + s * L::tile);
#pragma unroll
                    for (int j = 0; j < F * L::PARTS * J; ++j) {
                        const int e = j / (L::PARTS * J), part = j / J % L::PARTS;
                        ptx::mma_f8_ss(tm_s(b) + e * L::QN, k + (e * D >> 4) + j % J * 2, q + part * (L::q_part >> 4) + j % J * 2,
                                       id_s, j % (L::PARTS * J) > 0);
                    }
                    ptx::mma_commit(&bar[SD + b]);
                    ptx::mma_commit(&bar[KFREE + s]);
                }
                ptx::mma_commit(&bar[QFREE + ib]);
                ++item_no;
                wk.next_item(p, last - first);
            }
        }
    } else if (warp == L::MMA_O) {                                // ---- rows of V without a token, O^T
        constexpr uint32_t id_o = ptx::idesc_e4m3_f32(128, L::ON, true);
        for (int t = 0; ok && wk.more();) {
            const int len = wk.len;
            const int64_t first = wk.tile, last = wk.last();
            for (int64_t i = first; i < last; ++i, ++t) {
                const int s = t % NS, b = t % NG;
                ok = warp_wait(&bar[VFULL + s], t / NS);
                if (!ok) break;
                const int left = len - (int)(i * TOK);
                if (left < TOK) {       // (a weight of 0 does not silence a NaN) 16 bytes a lane and step, to the page's end
                    constexpr int C = L::RB / 16;
                    const int end = min(TILE, ((left + F - 1) / F + rows - 1) & ~(rows - 1)) * C;
                    for (int j = left * (D / 16) + lane; j < end; j += 32)
                        *reinterpret_cast<uint4 *>(sm + L::V + s * L::tile + swizzled<L::RB>(j / C, j % C)) = make_uint4(0, 0, 0, 0);
                    ptx::fence_async_smem();
                    __syncwarp();
                }
                ok = warp_wait(&bar[PREADY + b], t / NG);         // (which says that O^T's buffer is free too)
                if (!ok) break;
                if (ptx::elect_one()) {
                    ptx::tc_fence_after_sync();
                    const uint64_t v = ptx::sdesc_rows<L::RB>(base + L::V + s * L::tile, L::tile);
                    const uint64_t w = ptx::sdesc_plain_n(base + L::P + b * L::p_bytes, 8 * L::ON, 128);
                    constexpr int J = TILE / 32;
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        ptx::mma_f8_ss(tm_o(b), v + j * (32 * L::RB >> 4), w + j * (32 * L::ON >> 4), id_o, j > 0);
                    ptx::mma_commit(&bar[PVD + b]);
                    ptx::mma_commit(&bar[VFREE + s]);
                }
                __syncwarp();
            }
            wk.next_item(p, last - first);
        }
    } else if (warp < L::SOFTMAX) {                               // ---- Q
        int item_no = 0;
        const bool q16 = reinterpret_cast<uintptr_t>(p.q) % 16 == 0 && p.ldq % 8 == 0;
        constexpr int LPR = D / 8, RPS = 32 / LPR, STEPS = HB / RPS < 1 ? 1 : HB / RPS;     // lanes per head, heads at a time
        const int c = lane % LPR;
        while (ok && wk.more()) {
            const int64_t first = wk.tile, last = wk.last();
            const int kvh = nb == 1 ? wk.item : wk.item / nb, g0 = (wk.item - kvh * nb) * HB, hb = min(HB, p.G - g0);
            if (item_no % L::STAGERS != warp - L::STAGE_Q) {
                ++item_no;
                wk.next_item(p, last - first);
                continue;
            }
            uint8_t *dst = sm + L::Q + (item_no & 1) * L::q_bytes;
            const __nv_bfloat16 *q =
                static_cast<const __nv_bfloat16 *>(p.q) + (int64_t)wk.n * p.ldq + ((int64_t)kvh * p.G + g0) * D;
            constexpr int U = STEPS < 8 ? STEPS : 8;              // loads under way
            for (int i0 = 0; i0 < STEPS; i0 += U) {
                uint4 u[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int h = (i0 + i) * RPS + lane / LPR;
                    u[i] = make_uint4(0, 0, 0, 0);
                    if (h < hb) {
                        if (q16) u[i] = *reinterpret_cast<const uint4 *>(q + h * D + c * 8);
                        else u[i] = load8(q + h * D + c * 8);
                    }
                }
                if (i0 == 0 && item_no >= 2) ok = warp_wait(&bar[QFREE + (item_no & 1)], (item_no >> 1) - 1);
                if (!ok) break;
                // each head's largest magnitude, by its bits, of two values at a time; what is not finite is larger still
                uint32_t top[U];
                bool odd = false;
#pragma unroll
                for (int i = 0; i < U; ++i)
                    top[i] = __vmaxu2(__vmaxu2(u[i].x & 0x7fff7fffu, u[i].y & 0x7fff7fffu),
                                      __vmaxu2(u[i].z & 0x7fff7fffu, u[i].w & 0x7fff7fffu));
#pragma unroll
                for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
                    for (int i = 0; i < U; ++i) top[i] = __vmaxu2(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    top[i] = max(top[i] << 16, top[i] & 0xffff0000u);
                    odd |= top[i] >= 0x7f800000u;
                }
                if (__any_sync(0xffffffffu, odd))                 // what is not finite becomes NaN, the rest as without it
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w}, m = 0;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t half = w[e >> 1] >> (16 * (e & 1)) & 0x7fffu;
                            if (half >= 0x7f80u) w[e >> 1] |= 0x7fffu << (16 * (e & 1));
                            else m = max(m, half);
                        }
#pragma unroll
                        for (int o = 1; o < LPR; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                        u[i] = make_uint4(w[0], w[1], w[2], w[3]);
                        top[i] = m << 16;
                    }
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int h = (i0 + i) * RPS + lane / LPR;
                    // (a negative scale's sign goes with the queries, so that the largest product is the largest score)
                    const float f = scale_for(__uint_as_float(top[i]));
                    // (a factor below 2^-126, of a scale of 0 too, would leave none to tell masked tokens by: it goes with them)
                    const float factor = f * fabsf(p.scale) * kLog2E, least = factor < 0x1p-126f ? factor * 0x1p126f : 1.f;
                    const float inv = copysignf(inverse(f) * least, p.scale);
                    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)     // (exact in float16 but for what is below 2^-23 of the largest)
                        split2<false>(__uint_as_float(w[e] << 16) * inv, __uint_as_float(w[e] & 0xffff0000u) * inv, hi[e], lo[e]);
                    if (h < HB) {
                        const int n = column<HB>(h);
                        uint8_t *low = dst + (L::BOTH ? swizzled<D>(8 + n, c >> 1) : L::q_part + swizzled<D>(n, c >> 1));
                        *reinterpret_cast<uint2 *>(dst + swizzled<D>(n, c >> 1) + (c & 1) * 8) =
                            make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                        *reinterpret_cast<uint2 *>(low + (c & 1) * 8) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
                        if (c == 0) qs[(item_no % QRING) * HB + h] = factor < 0x1p-126f ? 0x1p-126f : factor;
                    }
                }
            }
            if (!ok) break;
            ptx::fence_async_smem();
            warp_arrive(&bar[QFULL + (item_no & 1)]);
            ++item_no;
            wk.next_item(p, last - first);
        }
    } else if (warp >= L::SOFTMAX && warp < L::OUT) {             // ---- softmax
        // row k of this thread: 32 q + lane / 4 + 8 k; its heads: lane % 4 * HT and on
        constexpr int HT = L::HT, NT = L::N / 8;
        const int wg = (warp - L::SOFTMAX) >> 2, q = warp & 3, row0 = q * 32 + (lane >> 2), h0 = (lane & 3) * HT;
        float *const st = reinterpret_cast<float *>(sm + L::STAT) + (warp - L::SOFTMAX) * 4 * HB;
        const int hl = lane < HB ? lane : 0;                      // this lane's head, of what is one for all tokens
        int t = 0, item_no = 0;
        while (ok && wk.more()) {
            const int len = wk.len;
            const int64_t first = wk.tile, last = wk.last();
            float m = -INFINITY, l[HT];
#pragma unroll
            for (int h = 0; h < HT; ++h) l[h] = 0.f;
            for (int64_t i = first; i < last; ++i, ++t) {
                if (t % NG != wg) continue;
                const int sb = t % SB, r = t % RING, turn = t / NG;
                float *red = reinterpret_cast<float *>(sm + L::RED) + (wg * 2 + (turn & 1)) * 4 * HB;
                ok = warp_wait(&bar[SCALES + r], t / RING) && warp_wait(&bar[SD + sb], t / SB);
                float x[F * HT][4], weight[4], unit = 0.f;        // scores of token e, head h: x[e * HT + h]
                bool apart = false;
                if (ok) {
                    ptx::tc_fence_after_sync();
                    float raw[2][4 * NT];                         // lanes 0-15 and 16-31 of the warp's part of TMEM
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t from = tm_s(sb) + ((uint32_t)q << 21) + ((uint32_t)half << 20);
                        if constexpr (NT == 2) ptx::tmem_ld_tiles2(from, raw[half]);
                        else ptx::tmem_ld_tiles4(from, raw[half]);
                    }
                    const float *fk = sc + r * L::NBK, *fv = sc + (RING + r) * L::NBK;
                    float f[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int at = (row0 + 8 * k) * F >> p.block_shift;
                        f[k] = fk[at];
                        weight[k] = fv[at];
                    }
                    // the tile's largest scale of V, 2^-126 at least (where a block has no token its scale is 0)
                    unit = fmaxf(ptx::warp_max(fabsf(lane < (TOK >> p.block_shift) ? fv[lane] : 0.f)), 0x1p-126f);
                    const float share = __fdividef(kShare, unit);
                    ptx::tmem_ld_wait(raw[0], raw[1]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        weight[k] *= share;
                        auto column = [&](int tile, int b) { return raw[k >> 1][4 * tile + 2 * (k & 1) + b]; };
#pragma unroll
                        for (int e = 0; e < F; ++e)
#pragma unroll
                            for (int h = 0; h < HT; ++h)
                                x[e * HT + h][k] = f[k] * (L::BOTH ? column(2 * e, h) + column(2 * e + 1, h)
                                                                   : column(e * (L::QN / 8) + (h >> 1), h & 1));
                    }
                    const uint32_t mask = *static_cast<volatile uint32_t *>(&s_mask[r]);
                    const int left = len - (int)(i * TOK);
                    {
                        const int token = lane << p.block_shift;  // of a block; does it have one, on a page that is there?
                        const bool is = token < min(left, TOK) && (mask >> (token >> FS >> rows_shift & 31) & 1);
                        apart = __any_sync(0xffffffffu, is && fabsf(fv[lane]) < 0.5f * unit);
                    }
                    if (left < TOK || __popc(mask) < pieces) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int row = row0 + 8 * k;
                            const bool page = mask >> (row >> rows_shift) & 1;
#pragma unroll
                            for (int e = 0; e < F; ++e) {
                                const bool in = page && row * F + e < left;
#pragma unroll
                                for (int h = 0; h < HT; ++h) x[e * HT + h][k] = in ? x[e * HT + h][k] : -INFINITY;
                            }
                            if (!page) weight[k] = 0.f;
                        }
                    }
                    float mx[HT];
#pragma unroll
                    for (int h = 0; h < HT; ++h) mx[h] = -INFINITY;
                    if (!apart) {
#pragma unroll
                        for (int h = 0; h < HT; ++h)
#pragma unroll
                            for (int e = 0; e < F; ++e)
#pragma unroll
                                for (int k = 0; k < 4; ++k) mx[h] = fmaxf(mx[h], x[e * HT + h][k]);
                    } else {                                      // (the queries' factors were there before S^T)
                        float f[HT];
                        ld_heads(qs + (item_no % QRING) * HB + h0, f);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float low = fmaxf(__log2f(fabsf(weight[k]) * (1.f / kShare)), -40.f);
#pragma unroll
                            for (int h = 0; h < HT; ++h)
#pragma unroll
                                for (int e = 0; e < F; ++e) mx[h] = fmaxf(mx[h], fmaf(x[e * HT + h][k], f[h], low));
                        }
                    }
                    int mine;
                    const float top = reduce_rows(mx, lane, mine, [](float a, float b) { return fmaxf(a, b); });
                    red[q * HB + h0 + mine] = top;
                    ptx::tc_fence_before_sync();
                    warp_arrive(&bar[SFREE + sb]);
                    // the weights and maxima of this group's last tile have been used
                    ok = t < NG || warp_wait(&bar[OFREE + wg], turn - 1);
                }
                ok = !ptx::bar_any(1 + wg, 128, !ok);
                if (!ok) break;
                {   // a lane per head: its factor, the tile's maximum, what that is to the sums so far
                    const float mt = fmaxf(fmaxf(red[hl], red[HB + hl]), fmaxf(red[2 * HB + hl], red[3 * HB + hl]));
                    const float f = qs[(item_no % QRING) * HB + hl], top = mt == -INFINITY || apart ? mt : mt * f;
                    const float mn = fmaxf(m, top), mu = mn == -INFINITY ? 0.f : mn, less = ex2(m - mu);
                    if (lane < HB) {
                        st[hl] = f;
                        st[HB + hl] = top == -INFINITY ? 0.f : top - kTop;
                        st[2 * HB + hl] = ex2(top - kTop - mu);
                        st[3 * HB + hl] = less;
                        if (q == 0) sm_m[wg * HB + hl] = top;
                    }
                    const bool any = __any_sync(0xffffffffu, (less != 1.f && m != -INFINITY));
                    m = mn;
                    __syncwarp();
                    if (any) {
                        float y[HT];
                        ld_heads(st + 3 * HB + h0, y);
#pragma unroll
                        for (int h = 0; h < HT; ++h) l[h] *= y[h];
                    }
                }
                float f[HT], top[HT], g[HT];
                ld_heads(st + h0, f);
                ld_heads(st + HB + h0, top);
                ld_heads(st + 2 * HB + h0, g);
                constexpr int WB = L::BOTH ? 1 : HT / 4;          // 16-byte columns of a token, a word of this thread in each
                uint8_t *w8 = sm + L::P + wg * L::p_bytes + (4 * q + (lane >> 3)) * 8 * L::ON + (lane & 7) * 16;
#pragma unroll
                for (int e = 0; e < F; ++e)
#pragma unroll
                    for (int blk = 0; blk < WB; ++blk) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float w[4];
#pragma unroll
                            for (int j = 0; j < (L::BOTH ? 2 : 4); ++j) {
                                const int h = 4 * blk + j;
                                const float own = ex2(fmaf(x[e * HT + h][k], f[h], -top[h]));
                                l[h] = fmaf(own, g[h], l[h]);
                                w[j] = own * weight[k];
                            }
                            uint32_t h0_, l0_, h1_, l1_;
                            split2<true>(w[0], w[1], h0_, l0_);
                            if constexpr (L::BOTH) {
                                hi[k] = h0_ | l0_ << 16;
                            } else {
                                split2<true>(w[2], w[3], h1_, l1_);
                                hi[k] = h0_ | h1_ << 16;
                                lo[k] = l0_ | l1_ << 16;
                            }
                        }
                        uint8_t *to = w8 + (e * WB + blk) * 128;
                        ptx::stmatrix4(ptx::smem_addr(to), hi[0], hi[1], hi[2], hi[3]);
                        if constexpr (!L::BOTH) ptx::stmatrix4(ptx::smem_addr(to + 8 * L::N), lo[0], lo[1], lo[2], lo[3]);
                    }
                if (q == 0 && lane == 0) sm_m[NG * HB + wg] = unit;
                ptx::fence_async_smem();
                warp_arrive(&bar[PREADY + wg]);
            }
            if (!ok) break;
            const int ib = item_no & 1;
            ok = item_no < 2 || warp_wait(&bar[IFREE + ib], (item_no >> 1) - 1);
            ok = !ptx::bar_any(1 + wg, 128, !ok);
            if (!ok) break;
            int mine;
            const float sum = reduce_rows(l, lane, mine, [](float a, float b) { return a + b; });
            sums[((ib * NG + wg) * 4 + q) * HB + h0 + mine] = sum;
            if (q == 0 && lane < HB) sums[(8 * NG + ib * NG + wg) * HB + lane] = m;
            warp_arrive(&bar[IREADY + ib]);
            ++item_no;
            wk.next_item(p, last - first);
        }
    } else if (warp >= L::OUT) {                                  // ---- output: thread = row of O^T
        const int q = warp & 3, row = q * 32 + lane, e = row / D, d = row % D;
        float *const st = reinterpret_cast<float *>(sm + L::STAT) + (warp - L::SOFTMAX) * 4 * HB;
        float *const xch = reinterpret_cast<float *>(sm + L::X);
        const int hl = lane < HB ? lane : 0;
        const bool works = q * 32 < L::RB;                        // (rows of O^T past a row's bytes reach no one)
        int t = 0, item_no = 0;
        while (ok && wk.more()) {
            const int64_t first = wk.tile, last = wk.last();
            const int kvh = nb == 1 ? wk.item : wk.item / nb, g0 = (wk.item - kvh * nb) * HB, hb = min(HB, p.G - g0);
            const int64_t row0 = (int64_t)wk.n * p.Hq + (int64_t)kvh * p.G + g0;
            float acc[HB], m = -INFINITY;
#pragma unroll
            for (int h = 0; h < HB; ++h) acc[h] = 0.f;
            for (int64_t i = first; i < last; ++i, ++t) {
                const int b = t % NG;
                ok = warp_wait(&bar[PVD + b], t / NG);
                if (!ok) break;
                if (works) {
                    ptx::tc_fence_after_sync();
                    const uint32_t from = tm_o(b) + ((uint32_t)q << 21) + (F == 2 ? (uint32_t)e * L::QN : 0u);
                    float v[16], x[16];                           // 16 columns of both parts (up to 8 heads: v has both)
                    auto load = [&](int c) {
                        ptx::tmem_ld16(from + c, v);
                        if constexpr (!L::BOTH) ptx::tmem_ld16(from + L::N + c, x);
                    };
                    load(0);
                    const float top = sm_m[b * HB + hl], mn = fmaxf(m, top), mu = mn == -INFINITY ? 0.f : mn;
                    __syncwarp();                                 // (the factors before have been read)
                    if (lane < HB) {
                        st[hl] = ex2(m - mu);
                        st[HB + hl] = ex2(top - kTop - mu) * (kLow / kShare) * sm_m[NG * HB + b];
                    }
                    m = mn;
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < L::QN; c += 16) {
                        if (c > 0) load(c);
                        if constexpr (L::BOTH) ptx::tmem_ld_wait(v);
                        else ptx::tmem_ld_wait(v, x);
#pragma unroll
                        for (int h = 0; h < HB; h += 4) {
                            if (out_column<HB>(h) / 16 != c / 16) continue;
                            float f[4], g[4];
                            ld4(st + h, f);
                            ld4(st + HB + h, g);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int at = out_column<HB>(h + j) % 16;
                                const float y = fmaf(L::BOTH ? v[at + 2] : x[at], 1.f / kLow, v[at]);
                                acc[h + j] = fmaf(acc[h + j], f[j], y * g[j]);
                            }
                        }
                    }
                    ptx::tc_fence_before_sync();
                }
                warp_arrive(&bar[OFREE + b]);
            }
            const int ib = item_no & 1;
            ok = ok && warp_wait(&bar[IREADY + ib], item_no >> 1);
            if constexpr (F == 2) {      // tokens e = 0 and 1 of the rows together, half of the heads each
                if (ok && works)
#pragma unroll
                    for (int h = 0; h < HB; ++h) xch[h * L::RB + row] = acc[h];
                ok = !ptx::bar_any(1 + NG, 128, !ok);
                if (ok && works)
#pragma unroll
                    for (int h = 0; h < HB / 2; ++h) {
                        const float *x = xch + (e * (HB / 2) + h) * L::RB + d;
                        acc[h] = x[0] + x[D];
                    }
                ptx::bar_any(1 + NG, 128, false);                 // (what is written next has been read)
            }
            if (!ok) break;
            const bool whole = first == 0 && last == wk.nt;
            float *part = p.part + ((int64_t)blockIdx.x * 2 + (first == 0 ? 1 : 0)) * part_floats(D, HB);
            {   // a lane per head: the sum, which every group of softmax warps has a part of
                const float *ms = sums + (8 + ib) * NG * HB + hl;
                float mh = ms[0], l = 0.f;
#pragma unroll
                for (int g = 1; g < NG; ++g) mh = fmaxf(mh, ms[g * HB]);
                const float mu = mh == -INFINITY ? 0.f : mh;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float *x = sums + (ib * NG + g) * 4 * HB + hl;
                    l = fmaf((x[0] + x[HB]) + (x[2 * HB] + x[3 * HB]), ex2(ms[g * HB] - mu), l);
                }
                __syncwarp();
                // (a sum is 0, without a token, or about 1 at least, where m is, or infinite or NaN)
                if (lane < HB) st[2 * HB + hl] = l > 0.f ? __fdividef(1.f, l) : l;
                if (q == 0 && lane < hb) {
                    if (!whole) { part[2 * lane] = mh; part[2 * lane + 1] = l; }
                    else if (p.lse) p.lse[row0 + lane] = (mh + log2f(l)) / kLog2E;
                }
                __syncwarp();
            }
            warp_arrive(&bar[IFREE + ib]);
            if (works) {
                constexpr int HM = HB / F;                        // heads of this thread
                const int h1 = F == 2 ? e * HM : 0;
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + row0 * D + d;
                if (whole) {
#pragma unroll
                    for (int h = 0; h < HM; h += 4) {
                        float l[4];
                        ld4(st + 2 * HB + h1 + h, l);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (h1 + h + j < hb) out[(h1 + h + j) * D] = __float2bfloat16_rn(acc[h + j] * l[j]);
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < HM; ++h)
                        if (h1 + h < hb) part[HB * 2 + (h1 + h) * D + d] = acc[h];
                }
            }
            ++item_no;
            wk.next_item(p, last - first);
        }
    }
    empty_sequences<__nv_bfloat16>(p, D);
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
    if (warp == LOADERS) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, L::cols);
    }
}

template <int D, int HB>
cudaError_t launch(const PagedQ8Params &p, int grid, cudaStream_t st) {
    CUtensorMap mk, mv;
    using L = Lay<D, HB>;
    const int shift = p.page_shift - (L::F - 1);
    const uint32_t box = shift < 7 ? 1u << shift : TILE;
    for (const bool v : {false, true})
        if (!make_map_pages(v ? &mv : &mk, v ? p.vc : p.kc, p.num_pages, p.Hkv, 1ull << shift, L::RB, box)) return cudaErrorInvalidValue;
    constexpr uint32_t smem = L::bytes + 1024;
    static_assert(smem <= 227 * 1024 - 4096, "shared memory");    // (beside the static part)
    const cudaError_t e = allow_smem<paged_decode_q8_tc_kernel<D, HB>>(smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(paged_decode_q8_tc_kernel<D, HB>, dim3(grid), L::THREADS, smem, st, 1, mk, mv, p);
}
template <int D>
cudaError_t launch_h(const PagedQ8Params &p, int HB, int grid, cudaStream_t st) {
    return HB == 8 ? launch<D, 8>(p, grid, st) : HB == 16 ? launch<D, 16>(p, grid, st) : launch<D, 32>(p, grid, st);
}

}  // namespace

cudaError_t launch_paged_decode_q8_tc(const PagedQ8Params &p, int d, int HB, int grid, cudaStream_t st) {
    return d == 32 ? launch_h<32>(p, HB, grid, st) : d == 64 ? launch_h<64>(p, HB, grid, st) : launch_h<128>(p, HB, grid, st);
}

}  // namespace kda
