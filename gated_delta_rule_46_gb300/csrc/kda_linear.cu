// kda_linear.cu -- out = act(x w^T + bias) + residual on the tensor cores.
//
// Two kernels.  `linear_pair_kernel` (many rows): a pair of CTAs works on one
// 256 x 256 tile of out at a time.  `linear_rows_kernel` (few rows): the roles
// of x and w are swapped, so that 128 output features lie on the MMA's rows and
// the rows of x, however few, on its columns; K is split over a cluster.
//
// Many rows are bound by the tensor pipe: 8192 x 16384 x 4096 (M x N x K) takes
// 555-565 us, 1.95-1.98 PFLOP/s, as long as the power cap does not set in (then
// 663); the pipe is 90 % busy at 4096 x 9728 x 4096 (175 us).  Few rows are bound
// by reading w: 64 x 16384 x 8192 takes 46 us (5.9 TB/s), 64 x 4096 x 4096 11.5 us,
// of which the 34 MB are 5; launch, the first load and the join are the rest.
// Every sum is held in float32 (TMEM, and the join of a cluster's parts in order
// of rank, so that results do not depend on timing; a float32 output, and any at very
// long K, in several parts); the one rounding to fewer bits is out's own.
#include <cuda.h>

#include "kda_layers.cuh"
#include "kda_tc_util.cuh"
#include "kda_testing.h"
#include "kda_tmap.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr long long kWaitBudget = 2000000000LL;   // cycles (about one second)
constexpr long long kDrain = 20000000LL;          // cycles (about ten milliseconds)

// GELU's Phi, with its relative precision in the lower tail too, where (1 + erf) / 2
// cancels (5 % off at y = -5, 0 below -5.5).  Phi(-a) = e^{-a^2 / 2} R(a): R, Mills'
// ratio over sqrt(2 pi), is smooth in t = 1 / (1 + 0.26 a) all the way to a = inf, where
// it is a multiple of t; R / t is taken from a polynomial of degree 8 in t, fitted by
// reweighted least squares to a relative error of 3e-8.  Rounding makes that 4e-7 up
// to |y| = 1, 1.5e-6 to 5 and 5e-6 to 10 (the exponent's ulp).  8192 x 8192 x 512 in
// bf16: 117-135 us; 140-163 with erff, 240-296 with erfcf, 65-80 without an activation.
__device__ __forceinline__ float normal_cdf(float y) {
    const float t = rcp(fmaf(0.26f, fabsf(y), 1.f));
    float q = 0.030235235f;
    q = fmaf(q, t, -0.15151833f);
    q = fmaf(q, t, 0.24878243f);
    q = fmaf(q, t, -0.14784548f);
    q = fmaf(q, t, 0.15879746f);
    q = fmaf(q, t, 0.051948357f);
    q = fmaf(q, t, 0.102792896f);
    q = fmaf(q, t, 0.10305038f);
    q = fmaf(q, t, 0.103757054f);
    const float p = q * t * ex2(-0.5f * kLog2E * y * y);
    return y < 0.f ? p : 1.f - p;
}

// The activation on the float32 sum.  sigmoid and silu are written with
// exp(-y): it overflows to +inf for very negative y, where both then give 0.
template <int ACT>
__device__ __forceinline__ float activate(float y) {
    if constexpr (ACT == KDA_ACT_RELU) return y > 0.f ? y : (y != y ? y : 0.f);
    if constexpr (ACT == KDA_ACT_GELU) return y * normal_cdf(y);
    if constexpr (ACT == KDA_ACT_SILU) return __fdividef(y, 1.f + __expf(-y));
    if constexpr (ACT == KDA_ACT_SIGMOID) return __fdividef(1.f, 1.f + __expf(-y));
    return y;
}

// After an expired wait: long enough for every copy and MMA in flight to land
// before shared and tensor memory are given back.
__device__ __forceinline__ void drain() {
    const long long t0 = clock64();
    while (clock64() - t0 < kDrain) {}
}

struct Tail {   // what the epilogue needs
    const float *bias;
    const void *residual;
    void *out;
    int M, N, K;
    uint32_t *status;
    int expire;           // test support
};

Tail tail(const LinearParams &p) {
    return {p.bias, p.residual, p.out, (int)p.M, (int)p.N, (int)p.K, p.status, take_layers_expire(KDA_TESTING_LINEAR)};
}

// ---------------------------------------------------------------------------
// Few rows.  One CTA: 128 features (rows of w, the MMA's M) x NT rows of x (the
// MMA's N, a multiple of 16), over its share of K; the S CTAs of a cluster
// share one tile and add their sums up in order of rank, each for its part of
// the rows.  Warp 0 loads (TMA), warp 1 issues the MMAs, warps 2-5 read TMEM.
// With LOAD = 1 (rows that no TMA copy can start on) warps 6-13 load instead, by
// way of registers, into the same swizzled layout.
// ---------------------------------------------------------------------------
constexpr int kBK = 64;                     // K per stage: one 128-byte swizzled row
constexpr uint32_t kABytes = 128 * 128;     // 128 rows

struct RowsParams {
    Tail t;
    const __nv_bfloat16 *x, *w;   // LOAD = 1
    int64_t ldx;
    int NT, stages, S;
    int per, parts;       // K steps of one part of the sum; accumulators for the parts after the first
};

template <int ACT, bool F32>
__device__ __forceinline__ void put(const Tail &t, int64_t m, int64_t n, float y) {
    y = activate<ACT>(y);
    const int64_t at = m * t.N + n;
    if constexpr (F32) {
        if (t.residual) y += static_cast<const float *>(t.residual)[at];
        static_cast<float *>(t.out)[at] = y;
    } else {
        if (t.residual) y += to_f32(static_cast<const __nv_bfloat16 *>(t.residual)[at]);
        static_cast<__nv_bfloat16 *>(t.out)[at] = __float2bfloat16_rn(y);
    }
}

// The eight elements from address a on, out of the two 16-byte words that hold them.
__device__ __forceinline__ uint4 shifted(const uint4 &x, const uint4 &y, uint32_t a) {
    uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = a & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = a & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __byte_perm(w[i], w[i + 1], a & 2 ? 0x5432 : 0x3210);
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Elements p[0] .. p[n - 1] of eight one by one, zeros for the others.
__device__ __forceinline__ uint4 load8(const __nv_bfloat16 *p, int n) {
    uint32_t e[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) e[c] = c < n ? __bfloat16_as_ushort(p[c]) : 0u;
    return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}

template <int ACT, bool F32, int LOAD>
__global__ void __launch_bounds__(LOAD ? 448 : 192, 1)
    linear_rows_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                       const RowsParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[12], empty[12], done, pfull[2], pfree[2];
    __shared__ uint32_t s_tmem, s_abort;
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t stage_bytes = kABytes + (uint32_t)p.NT * 128u;
    const int rank = p.S > 1 ? (int)ptx::cluster_rank() : 0;
    const int f0 = (int)(blockIdx.x / p.S) * 128, m0 = (int)blockIdx.y * p.NT;
    const int kb_all = (p.t.K + kBK - 1) / kBK;
    const int kb0 = (int)((int64_t)kb_all * rank / p.S), kb1 = (int)((int64_t)kb_all * (rank + 1) / p.S);
    // The sum is taken in parts of `per` K steps: the first in the result's own accumulator, the others in `parts` more by
    // turns, from where the epilogue's warps add them to it.
    const int steps = kb1 - kb0, passes = (steps + p.per - 1) / p.per;
    uint32_t cols = 32;
    while (cols < (uint32_t)(p.NT * (1 + p.parts))) cols <<= 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            ptx::mbar_init(&full[i], LOAD ? 256 : 1);
            ptx::mbar_init(&empty[i], 1);
        }
        ptx::mbar_init(&done, 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&pfull[i], 1);
            ptx::mbar_init(&pfree[i], 4);        // the epilogue's warps
        }
        ptx::fence_mbar_init();
        s_abort = 0;
        if (!LOAD) {
            ptx::prefetch_tensormap(&mw);
            ptx::prefetch_tensormap(&mx);
        }
    }
    if (warp == 1) {
        ptx::tmem_alloc(&s_tmem, cols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = s_tmem;
    bool ok = true;
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();

    if (warp == 0 && !LOAD) {
        if (lane == 0) {
            // Each tile starts at another place of its K range, so that the CTAs do not all read the same columns of rows
            // that lie a power of two apart (64 x 16384 x 8192: 46.0 us, 48.7 in step; 4096 columns: no difference).
            int kb = kb0 + (int)(3 * (blockIdx.x / p.S) % (unsigned)(kb1 - kb0));
            for (int i = 0; i < kb1 - kb0; ++i, kb = kb + 1 == kb1 ? kb0 : kb + 1) {
                const int s = i % p.stages;
                if (i >= p.stages && !ptx::mbar_wait(&empty[s], ((i / p.stages) - 1) & 1, kWaitBudget)) { ok = false; break; }
                uint8_t *a = sm + s * stage_bytes;
                ptx::mbar_arrive_expect_tx(&full[s], stage_bytes);
                ptx::tma_load_2d(a, &mw, kb * kBK, f0, &full[s]);
                ptx::tma_load_2d(a + kABytes, &mx, kb * kBK, m0, &full[s]);
            }
        }
    } else if (warp == 1) {
        if (ptx::elect_one()) {
            const uint32_t idesc = ptx::idesc_bf16_f32(128, p.NT);
            if (p.t.expire && blockIdx.x + blockIdx.y == 0) ok = ptx::mbar_wait(&done, 0, kTestWait);
            for (int pass = 0, i = 0; pass < passes && ok; ++pass) {
                const int b = pass > 0 ? (pass - 1) % p.parts : 0, end = min(steps, i + p.per);
                if (pass > p.parts && !ptx::mbar_wait(&pfree[b], ((pass - 1) / p.parts - 1) & 1, kWaitBudget)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after_sync();
                const uint32_t to = tmem + (pass > 0 ? (1 + b) * p.NT : 0);
                for (bool first = true; i < end; ++i, first = false) {
                    const int s = i % p.stages;
                    if (!ptx::mbar_wait(&full[s], (i / p.stages) & 1, kWaitBudget)) { ok = false; break; }
                    ptx::tc_fence_after_sync();
                    const uint32_t a = ptx::smem_addr(sm + s * stage_bytes);
                    mma_k<4>(to, a, 0, a + kABytes, 0, idesc, !first);
                    ptx::mma_commit(&empty[s]);
                }
                if (ok && pass > 0) ptx::mma_commit(&pfull[b]);
            }
            if (ok) ptx::mma_commit(&done);
        }
    } else if (LOAD && warp >= 6) {
        const int tid = threadIdx.x - 192, chunks = (128 + p.NT) * 8;
        for (int kb = kb0, i = 0; kb < kb1; ++kb, ++i) {
            const int s = i % p.stages;
            uint4 v[12];
            // Eight elements at a time from any even address: where all are there, and the two 16-byte words that hold them
            // lie within x or w, by those words, six pieces' loads at a time; else one by one.  4096^2 x 4095: 801 us (one
            // by one throughout 2479; 81 by TMA with K = 4096), 64 x 4096 x 4095: 30 (68; 10).
            auto piece = [&](int j, int &n, uintptr_t &a, bool &words) {
                const int id = tid + j * 256, row = id >> 3;
                const int64_t k0 = (int64_t)kb * kBK + (id & 7) * 8;
                const bool isw = row < 128;
                const int64_t r = isw ? f0 + row : m0 + row - 128;
                const __nv_bfloat16 *begin = isw ? p.w : p.x;
                const int64_t ld = isw ? p.t.K : p.ldx, rows = isw ? p.t.N : p.t.M;
                n = id < chunks && r < rows ? (int)max((int64_t)0, min((int64_t)8, p.t.K - k0)) : 0;
                a = reinterpret_cast<uintptr_t>(begin + r * ld + k0);
                const uintptr_t lo = a & ~uintptr_t(15);
                words = n == 8 && lo >= reinterpret_cast<uintptr_t>(begin) &&
                        lo + 32 <= reinterpret_cast<uintptr_t>(begin + (rows - 1) * ld + p.t.K);
            };
#pragma unroll
            for (int j0 = 0; j0 < 12; j0 += 6) {
                if (j0 * 256 >= chunks) break;
                uint4 y[6];
#pragma unroll
                for (int j = 0; j < 6; ++j) {
                    int n;
                    uintptr_t a;
                    bool words;
                    piece(j0 + j, n, a, words);
                    const uint4 *lo = reinterpret_cast<const uint4 *>(a & ~uintptr_t(15));
                    if (words) {
                        v[j0 + j] = lo[0];
                        y[j] = lo[1];
                    }
                }
#pragma unroll
                for (int j = 0; j < 6; ++j) {
                    int n;
                    uintptr_t a;
                    bool words;
                    piece(j0 + j, n, a, words);
                    if (words) v[j0 + j] = shifted(v[j0 + j], y[j], (uint32_t)a);
                    else v[j0 + j] = load8(reinterpret_cast<const __nv_bfloat16 *>(a), n);
                }
            }
            if (i >= p.stages && !ptx::mbar_wait(&empty[s], ((i / p.stages) - 1) & 1, kWaitBudget)) { ok = false; break; }
#pragma unroll
            for (int j = 0; j < 12; ++j) {
                const int id = tid + j * 256;
                if (id >= chunks) break;
                const int row = id >> 3;
                uint8_t *dst = row < 128 ? sm + s * stage_bytes + swz(row, id & 7)
                                         : sm + s * stage_bytes + kABytes + swz(row - 128, id & 7);
                *reinterpret_cast<uint4 *>(dst) = v[j];
            }
            ptx::fence_async_smem();
            ptx::mbar_arrive(&full[s]);
        }
    }
    const bool reader = warp >= 2 && warp < 6;
    const int q = warp & 3;                      // TMEM lane quarter of this warp
    float bias = 0.f;
    const int f = f0 + q * 32 + lane;
    const int rows = min(p.NT, p.t.M - m0);
    if (reader) {
        if (p.t.bias && f < p.t.N) bias = p.t.bias[f];
        for (int pass = 1; pass < passes; ++pass) {
            // (a part's barrier stands for all products before it too)
            const int b = (pass - 1) % p.parts;
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(&pfull[b], ((pass - 1) / p.parts) & 1, kWaitBudget));
            if (!ok) break;
            ptx::tc_fence_after_sync();
            const uint32_t at = tmem + ((uint32_t)q << 21);
            for (int c0 = 0; c0 < rows; c0 += 16) {
                float d[16], x[16];
                ptx::tmem_ld16(at + c0, d);
                ptx::tmem_ld16(at + (1 + b) * p.NT + c0, x);
                ptx::tmem_ld_wait(d, x);
#pragma unroll
                for (int e = 0; e < 16; ++e) d[e] += x[e];
                ptx::tmem_st16(at + c0, d);
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&pfree[b]);
        }
        ok = ok && ptx::mbar_wait(&done, 0, kWaitBudget);
        ptx::tc_fence_after_sync();
    }
    if (!ok) {
        s_abort = 1;
        report_status(p.t.status, KDA_ERR_DEVICE_TIMEOUT);
    }
    __syncthreads();
    if (s_abort) drain();
    if (p.S == 1) {
        if (reader && !s_abort) {
            for (int c0 = 0; c0 < rows; c0 += 16) {
                float d[16];
                ptx::tmem_ld16(tmem + ((uint32_t)q << 21) + c0, d);
                ptx::tmem_ld_wait(d);
                if (f < p.t.N)
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (c0 + c < rows) put<ACT, F32>(p.t, m0 + c0 + c, f, d[c] + bias);
            }
        }
    } else {
        // this CTA's sums as [row][128] float32 over the stages (all consumed), then each CTA of the
        // cluster adds up every S-th row over the ranks
        float *part = reinterpret_cast<float *>(sm);
        if (reader) {
            for (int c0 = 0; c0 < rows; c0 += 16) {
                float d[16];
                ptx::tmem_ld16(tmem + ((uint32_t)q << 21) + c0, d);
                ptx::tmem_ld_wait(d);
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    if (c0 + c < rows) part[(c0 + c) * 128 + q * 32 + lane] = d[c];
            }
        }
        ptx::cluster_sync();
        if (!s_abort) {
            float b[4];
            const int n0 = f0 + lane * 4;
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = p.t.bias && n0 + e < p.t.N ? p.t.bias[n0 + e] : 0.f;
            for (int r = rank + p.S * warp; r < rows; r += p.S * (int)(blockDim.x >> 5)) {
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int o = 0; o < p.S; ++o) {
                    const float4 v = ptx::ld_cluster_f4(ptx::map_to_rank(part + r * 128 + lane * 4, (uint32_t)o));
                    a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
                }
                const float y[4] = {a.x + b[0], a.y + b[1], a.z + b[2], a.w + b[3]};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n0 + e < p.t.N) put<ACT, F32>(p.t, m0 + r, n0 + e, y[e]);
            }
        }
        ptx::cluster_sync();     // no CTA leaves while another reads its shared memory
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, cols);
    }
}

// ---------------------------------------------------------------------------
// Many rows.  A pair of CTAs per 256 x BN tile: each loads its 128 rows of x and
// half of the BN rows of w per K step (32 KB for BN = 256; the MMA reads the
// halves of w from both, so each SM fetches half of what a lone CTA would),
// accumulates 128 x BN float32 in TMEM, two tiles' worth, so that the epilogue of one tile
// runs beside the next one's MMAs.  Persistent: pair i takes tiles i, i + pairs, ...
// Warp 0 loads, warp 1 issues (rank 0 of the pair only), warps 2-9 are the
// epilogue: two groups of four, BN / 2 columns each, by way of a 16 KB staging
// tile and TMA stores; a residual tile comes in by TMA through the same buffer.
// ---------------------------------------------------------------------------
constexpr uint32_t kStaging = 16384;
template <int BN>
struct PairLay {
    static constexpr int stages = BN == 256 ? 6 : 8;
    static constexpr uint32_t stage = kABytes + (BN / 2) * 128;
    static constexpr uint32_t staging = stages * stage;
    static constexpr uint32_t bytes = staging + 2 * kStaging + 1024;
};

struct PairParams {
    Tail t;
    int tiles_m, tiles_n, group;    // tiles are walked `group` row tiles at a time, column by column
};

__device__ __forceinline__ void tile_at(const PairParams &p, int i, int &tm, int &tn) {
    const int per = p.group * p.tiles_n, g = i / per, m0 = g * p.group;
    const int h = min(p.group, p.tiles_m - m0), r = i - g * per;
    tm = m0 + r % h;
    tn = r / h;
}

template <int ACT, bool F32, int BN>
__global__ void __launch_bounds__(320)
    linear_pair_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                       const __grid_constant__ CUtensorMap mo, const __grid_constant__ CUtensorMap mr,
                       const PairParams p) {
    using L = PairLay<BN>;
    constexpr int kStages = L::stages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], rbar[2];
    __shared__ uint32_t s_tmem, s_abort;
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_rank();
    const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
    const int tiles = p.tiles_m * p.tiles_n, kbs = (p.t.K + kBK - 1) / kBK;
    // A float32 output is summed in passes of 512 products, which the epilogue adds up: the MMAs' own float32 sums lose up
    // to an ulp at each step, always towards zero (rounding to bf16 hides that).  3812 x 5166 x 2244 in one sum is 1.3e-6
    // off, in passes 5e-7, a float32 product 4e-7; 4096 x 4096 x 8192 takes 240 us, 158 with a bf16 output.
    const int per = F32 ? 8 : kbs, passes = F32 ? (kbs + per - 1) / per : 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&tfull[i], 1);
            ptx::mbar_init(&tempty[i], 16);      // the epilogue warps of both CTAs
            ptx::mbar_init(&rbar[i], 1);
        }
        ptx::fence_mbar_init();
        s_abort = 0;
        ptx::prefetch_tensormap(&mx);
        ptx::prefetch_tensormap(&mw);
        ptx::prefetch_tensormap(&mo);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(&s_tmem, 2 * BN);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before_sync();
    ptx::cluster_sync();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = s_tmem;
    bool ok = true;
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            for (int i = pair; i < tiles && ok; i += pairs) {
                int tm, tn;
                tile_at(p, i, tm, tn);
                const int m0 = tm * 256 + (int)rank * 128, n0 = tn * BN + (int)rank * (BN / 2);
                for (int kb = 0; kb < kbs; ++kb, ++it) {
                    const int s = it % kStages;
                    if (it >= kStages && !ptx::mbar_wait_cluster(&empty[s], ((it / kStages) - 1) & 1, kWaitBudget)) {
                        ok = false;
                        break;
                    }
                    uint8_t *a = sm + s * L::stage;
                    // rank 0's barrier counts the bytes of both CTAs
                    if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], 2 * L::stage);
                    const uint32_t bar = ptx::map_to_rank(&full[s], 0);
                    ptx::tma_load_2d_pair(a, &mx, kb * kBK, m0, bar);
                    ptx::tma_load_2d_pair(a + kABytes, &mw, kb * kBK, n0, bar);
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && ptx::elect_one()) {
            const uint32_t idesc = ptx::idesc_bf16_f32(256, BN);
            int it = 0, n = 0;
            if (p.t.expire && pair == 0) ok = ptx::mbar_wait(&tfull[0], 0, kTestWait);
            // all passes of a tile, then the next tile's
            for (int i = pair * passes; i < tiles * passes && ok; i += (i + 1) % passes ? 1 : (pairs - 1) * passes + 1, ++n) {
                const int b = n & 1;
                if (n >= 2 && !ptx::mbar_wait_cluster(&tempty[b], ((n >> 1) - 1) & 1, kWaitBudget)) { ok = false; break; }
                ptx::tc_fence_after_sync();
                const int k0 = (i % passes) * per, k1 = min(kbs, k0 + per);
                for (int kb = k0; kb < k1; ++kb, ++it) {
                    const int s = it % kStages;
                    if (!ptx::mbar_wait_cluster(&full[s], (it / kStages) & 1, kWaitBudget)) { ok = false; break; }
                    ptx::tc_fence_after_sync();
                    const uint32_t a = ptx::smem_addr(sm + s * L::stage);
                    const uint64_t da = ptx::sdesc_kmajor_sw128(a), db = ptx::sdesc_kmajor_sw128(a + kABytes);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        ptx::mma_bf16_ss_pair(tmem + b * BN, da + k * 2, db + k * 2, idesc, kb > k0 || k > 0);
                    ptx::mma_commit_pair(&empty[s]);
                }
                if (ok) ptx::mma_commit_pair(&tfull[b]);
            }
        }
    } else {
        const int g = (warp - 2) >> 2, q = warp & 3, row = q * 32 + lane;
        const bool lead = ((warp - 2) & 3) == 0 && lane == 0;      // the group's thread for TMA
        uint8_t *st = sm + L::staging + g * kStaging;
        constexpr int CW = F32 ? 32 : 64, CHUNKS = BN / 2 / CW;    // columns of a 128-byte staging row
        int n = 0;
        uint32_t rphase = 0;
        for (int i = pair; i < tiles && ok; i += pairs, ++n) {
            int tm, tn;
            tile_at(p, i, tm, tn);
            const int m0 = tm * 256 + (int)rank * 128, n0 = tn * BN + g * (BN / 2);
            float sum[F32 ? BN / 2 : 1];
            if constexpr (F32) {
                for (int pass = 0; pass + 1 < passes && ok; ++pass, ++n) {
                    const int b = n & 1;
                    ok = !ptx::bar_any(g + 1, 128, !ptx::mbar_wait_cluster(&tfull[b], (n >> 1) & 1, kWaitBudget));
                    if (!ok) break;
                    ptx::tc_fence_after_sync();
#pragma unroll
                    for (int c = 0; c < BN / 2; c += 16) {
                        float d[16];
                        ptx::tmem_ld16(tmem + ((uint32_t)q << 21) + b * BN + g * (BN / 2) + c, d);
                        ptx::tmem_ld_wait(d);
#pragma unroll
                        for (int e = 0; e < 16; ++e) sum[c + e] = pass ? sum[c + e] + d[e] : d[e];
                    }
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster(ptx::map_to_rank(&tempty[b], 0));
                }
                if (!ok) break;
            }
            const int b = n & 1;
            // the group goes on, or gives up, as one
            ok = !ptx::bar_any(g + 1, 128, !ptx::mbar_wait_cluster(&tfull[b], (n >> 1) & 1, kWaitBudget));
            if (!ok) break;
            ptx::tc_fence_after_sync();
            auto chunk = [&](const int c) {
                const int nc = n0 + c * CW;
                // the staging tile is free once its last store has read it
                if (lead) {
                    ptx::bulk_wait_read();
                    if (p.t.residual) {
                        ptx::mbar_arrive_expect_tx(&rbar[g], kStaging);
                        ptx::tma_load_2d(st, &mr, nc, m0, &rbar[g]);
                    }
                }
                float d[CW];
                ptx::tmem_ld32(tmem + ((uint32_t)q << 21) + b * BN + g * (BN / 2) + c * CW, *reinterpret_cast<float(*)[32]>(d));
                if constexpr (!F32)
                    ptx::tmem_ld32(tmem + ((uint32_t)q << 21) + b * BN + g * (BN / 2) + c * CW + 32,
                                   *reinterpret_cast<float(*)[32]>(d + 32));
                ptx::tmem_ld_wait(d);
                if constexpr (F32) {
                    if (passes > 1)
#pragma unroll
                        for (int j = 0; j < CW; ++j) d[j] += sum[c * CW + j];
                }
                if (c == CHUNKS - 1) {
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_cluster(ptx::map_to_rank(&tempty[b], 0));
                }
#pragma unroll
                for (int j = 0; j < CW; j += 4) {
                    float bb[4] = {};
                    if (p.t.bias) {
                        if (nc + j + 4 <= p.t.N) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) bb[e] = __ldg(p.t.bias + nc + j + e);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) bb[e] = nc + j + e < p.t.N ? p.t.bias[nc + j + e] : 0.f;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[j + e] = activate<ACT>(d[j + e] + bb[e]);
                }
                if (p.t.residual) {
                    ok = ptx::mbar_wait(&rbar[g], rphase, kWaitBudget);
                    rphase ^= 1;
                } else {
                    asm volatile("bar.sync %0, 128;" ::"r"(g + 1) : "memory");
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint8_t *at = st + swz(row, j);
                    if constexpr (F32) {
                        float4 v = make_float4(d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]);
                        if (p.t.residual) {
                            const float4 r = *reinterpret_cast<float4 *>(at);
                            v.x += r.x; v.y += r.y; v.z += r.z; v.w += r.w;
                        }
                        *reinterpret_cast<float4 *>(at) = v;
                    } else {
                        if (p.t.residual) {
                            float r[8];
                            ld_chunk(st, swz(row, j), r);
#pragma unroll
                            for (int e = 0; e < 8; ++e) d[8 * j + e] += r[e];
                        }
                        st_chunk(st, swz(row, j), d + 8 * j);
                    }
                }
                ptx::fence_async_smem();
                ok = !ptx::bar_any(g + 1, 128, !ok);
                if (ok && lead) {
                    ptx::tma_store_2d(&mo, nc, m0, st);
                    ptx::bulk_commit();
                }
            };
            if constexpr (F32) {       // the sums are registers: unrolled
                chunk(0);
                if (ok) chunk(1);
            } else {
#pragma unroll 1
                for (int c = 0; c < CHUNKS && ok; ++c) chunk(c);
            }
        }
        if (lead) ptx::bulk_wait_all();
    }
    if (!ok) {
        s_abort = 1;
        report_status(p.t.status, KDA_ERR_DEVICE_TIMEOUT);
    }
    __syncthreads();
    if (s_abort) drain();
    ptx::tc_fence_before_sync();
    ptx::cluster_sync();         // neither CTA leaves while the other's MMAs or barriers use it
    if (warp == 1) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc_pair(tmem, 2 * BN);
    }
}

template <int ACT, bool F32, int BN>
cudaError_t launch_pair(const LinearParams &p, cudaStream_t st) {
    using L = PairLay<BN>;
    CUtensorMap mx, mw, mo, mr;
    const uint64_t eb = F32 ? 4 : 2;
    if (!make_map_2d(&mx, p.x, true, p.M, p.K, p.ldx * 2, 128) || !make_map_2d(&mw, p.w, true, p.N, p.K, p.K * 2, BN / 2) ||
        !make_map_2d(&mo, p.out, !F32, p.M, p.N, p.N * eb, 128) ||
        !make_map_2d(&mr, p.residual ? p.residual : p.out, !F32, p.M, p.N, p.N * eb, 128))
        return cudaErrorInvalidValue;
    PairParams pp{tail(p), (int)((p.M + 255) / 256), (int)((p.N + BN - 1) / BN), 8};
    auto *kernel = linear_pair_kernel<ACT, F32, BN>;
    const cudaError_t e = allow_smem<linear_pair_kernel<ACT, F32, BN>>(L::bytes);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)pp.tiles_m * pp.tiles_n;
    const int pairs = sm_count() / 2;
    return launch_dependent(kernel, dim3(2 * (unsigned)(tiles < pairs ? tiles : pairs)), 320, L::bytes, st, 2, mx, mw, mo, mr,
                            pp);
}

// Most products of one sum in the tensor cores for a bf16 output: each step of 16 loses up to an ulp of it, 2^-23,
// together 2^-11 where the output's rounding takes 2^-9.
constexpr int kPart = 65536;

// Rows of x per CTA.
constexpr int kRowsTile = 256;
int rows_tile(int64_t M) { return M < kRowsTile ? (int)((M + 15) / 16) * 16 : kRowsTile; }

template <int ACT, bool F32, int LOAD>
cudaError_t launch_rows(const LinearParams &p, cudaStream_t st) {
    RowsParams rp{};
    rp.t = tail(p);
    rp.x = p.x;
    rp.w = p.w;
    rp.ldx = p.ldx;
    const int64_t kbs = (p.K + kBK - 1) / kBK;
    rp.NT = rows_tile(p.M);
    const uint32_t stage = kABytes + rp.NT * 128;
    constexpr uint32_t kRoom = 200 * 1024;      // all of an SM's: the weights under way are what hides HBM's latency
    rp.stages = (int)(kRoom / stage) < 12 ? (int)(kRoom / stage) : 12;
    const int64_t tiles = ((p.N + 127) / 128) * ((p.M + rp.NT - 1) / rp.NT);
    const cudaError_t e = allow_smem<linear_rows_kernel<ACT, F32, LOAD>>(kRoom + 1024);
    if (e != cudaSuccess) return e;
    // Split K over the largest cluster of which all tiles' run at a time, one CTA per SM, with at least four steps for
    // each CTA.  64 x 4096 x 4096 (32 tiles): S = 4 takes 10.6 us; with two smaller CTAs per SM S = 4 takes 11.2 and S =
    // 8 11.9.  64 x 5120 x 4096 (40 tiles): S = 3 takes 12.7, S = 2 14.7; 64 x 2560 x 4096 (20 tiles): S = 7, of which
    // no more than 15 run at a time, 16.0, S = 4 9.4.
    rp.S = 8;
    while (rp.S > 1 && (kbs / rp.S < 4 || tiles > cluster_room<linear_rows_kernel<ACT, F32, LOAD>>(
                                                      rp.S, LOAD ? 448 : 192, kRoom + 1024)))
        --rp.S;
    // A float32 output is summed in parts of 512 products (see linear_pair_kernel), up to two of them under way beside the
    // result as far as TMEM holds them; a bf16 output in parts of kPart.
    const int64_t steps = (kbs + rp.S - 1) / rp.S, room = 512 / rp.NT - 1 < 2 ? 512 / rp.NT - 1 : 2;
    rp.per = F32 ? 8 : kPart / kBK;
    const int64_t after = (steps + rp.per - 1) / rp.per - 1;
    rp.parts = (int)(after < room ? after : room);
    uint32_t smem = rp.stages * stage;
    if (rp.S > 1 && smem < (uint32_t)rp.NT * 512u) smem = rp.NT * 512u;
    smem += 1024;
    CUtensorMap mw{}, mx{};
    if (!LOAD && (!make_map_2d(&mw, p.w, true, p.N, p.K, p.K * 2, 128) ||
                  !make_map_2d(&mx, p.x, true, p.M, p.K, p.ldx * 2, rp.NT)))
        return cudaErrorInvalidValue;
    auto *kernel = linear_rows_kernel<ACT, F32, LOAD>;
    const int64_t mt = (p.M + rp.NT - 1) / rp.NT;
    return launch_dependent(kernel, dim3((unsigned)((p.N + 127) / 128 * rp.S), (unsigned)mt), LOAD ? 448 : 192, smem, st,
                            rp.S, mw, mx, rp);
}

template <int ACT, bool F32>
cudaError_t launch_act(const LinearParams &p, cudaStream_t st) {
    const bool tma = p.K % 8 == 0 && p.ldx % 8 == 0 && reinterpret_cast<uintptr_t>(p.x) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(p.w) % 16 == 0;
    if (!tma) return launch_rows<ACT, F32, 1>(p, st);
    const uint64_t eb = F32 ? 4 : 2;
    const bool store = p.N * eb % 16 == 0 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(p.residual) % 16 == 0;
    // Tiles of 256 x 256 where they give more than half of the pairs work (256 x 16384 x 4096: 31 us, 38 by rows; 1024 x
    // 4096 x 4096: 25 us, 32 by rows), of 256 x 128 where those do (512 x 4096 x 4096: 21 us, 24 either way; 1024^3: 8.5
    // us, 10.4 by rows).  With fewer, splitting K beats both (256 x 4096 x 4096: 16 us, 20 in pairs).
    // (A float32 output's epilogue holds its sums in registers, 128 columns' worth.)
    // K past kPart goes by rows, where the sums of a bf16 output too are taken in parts (600 x 2048 x 65600: 200 us, and 281
    // in pairs with 65536 products; 2048 x 4096: 728 and 613).
    const int64_t tiles = ((p.M + 255) / 256) * ((p.N + 255) / 256), pairs = sm_count() / 2;
    if (!F32 && p.K > kPart) return launch_rows<ACT, F32, 0>(p, st);
    if constexpr (!F32)
        if (store && p.M > 128 && tiles * 2 > pairs) return launch_pair<ACT, F32, 256>(p, st);
    if (store && p.M > 256 && tiles * 5 > pairs) return launch_pair<ACT, F32, 128>(p, st);
    return launch_rows<ACT, F32, 0>(p, st);
}

template <int ACT>
cudaError_t launch_type(const LinearParams &p, cudaStream_t st) {
    return p.out_f32 ? launch_act<ACT, true>(p, st) : launch_act<ACT, false>(p, st);
}

cudaError_t launch_slice(const LinearParams &p, cudaStream_t st) {
    switch (p.act) {
        case KDA_ACT_RELU: return launch_type<KDA_ACT_RELU>(p, st);
        case KDA_ACT_GELU: return launch_type<KDA_ACT_GELU>(p, st);
        case KDA_ACT_SILU: return launch_type<KDA_ACT_SILU>(p, st);
        case KDA_ACT_SIGMOID: return launch_type<KDA_ACT_SIGMOID>(p, st);
        default: return launch_type<KDA_ACT_NONE>(p, st);
    }
}

// M is worked on in slices of whole tiles: row tiles are the grid's y, which goes up to 65535.
constexpr int64_t kSlice = int64_t(1) << 22;
static_assert(kSlice / kRowsTile <= 65535 && kSlice % kRowsTile == 0, "slice");

}  // namespace

int64_t linear_row_tiles(int64_t M) {
    const int64_t m = M < kSlice ? M : kSlice, tile = rows_tile(m);
    return (m + tile - 1) / tile;
}

cudaError_t launch_linear(const LinearParams &p, cudaStream_t st) {
    for (int64_t m0 = 0; m0 < p.M; m0 += kSlice) {
        LinearParams s = p;
        s.M = p.M - m0 < kSlice ? p.M - m0 : kSlice;
        s.x = p.x + m0 * p.ldx;
        const int64_t off = m0 * p.N * (p.out_f32 ? 4 : 2);
        s.out = static_cast<uint8_t *>(p.out) + off;
        if (p.residual) s.residual = static_cast<const uint8_t *>(p.residual) + off;
        const cudaError_t e = launch_slice(s, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace kda
