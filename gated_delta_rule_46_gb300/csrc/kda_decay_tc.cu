// kda_decay_tc.cu -- the chunked form of linear attention with one decay per
// head (bf16, dk = dv = 128) on the tensor cores.
//
// Per chain (sequence, head), in chunks of C = 64 tokens with n of them real,
// start state S and lambda = exp(log_decay):
//   P_ij = lambda^{i-j} q_i . k_j  (j <= i, else 0)
//   O^T  = (S^T Q^T) diag(lambda^{i+1}) + V^T P^T
//   S   <- lambda^n S + sum_j (lambda^{n-1-j} k_j) v_j^T
// Only the state links the chunks, and it takes part in one product (S^T Q^T)
// and one update, so everything else of the next chunk runs ahead of it.
//
// Precision.  q, k, v are bf16 and enter the products as they are.  P and the
// copy of S that multiplies q are rounded to bf16 (2^-9 of each, the size of
// the output's own rounding).  The state itself stays in float32 registers, and
// what is added to it must not lose bits: the decayed keys lambda^{n-1-j} k_j
// are split into three bf16 terms (24 bits) whose products accumulate in
// float32, from zero in every chunk, before one float32 addition to the state.
//
// Roles of the 20 warps of a CTA (one CTA per SM): 0 loads by TMA, two chunks
// ahead; 1 issues Q K^T, S^T Q^T and V^T P^T; 2 issues the state's product; 4-7
// take P out of TMEM and later the output; 8-11 split the decayed keys; 12-19
// hold the state, 64 of its columns of one row per thread.  mbarriers link them.
#include <cuda.h>

#include "kda_layers.cuh"
#include "kda_tc_util.cuh"
#include "kda_tmap.cuh"
#include "sm100_ptx.cuh"

namespace kda {

cudaError_t launch_schedule(const int32_t *cu, int num_seqs, int32_t *order, uint32_t *counter, uint32_t *status,
                            cudaStream_t st);

namespace {

using namespace tc;

constexpr int C = 64, D = 128;
constexpr int kThreads = 640;
constexpr long long kWaitBudget = 2000000000LL;   // cycles (about one second)
constexpr long long kDrain = 20000000LL;

// ---- shared memory, bytes from a 1024-aligned base.  Tiles have 128-byte rows
// with the 128-byte swizzle; a 128-channel row is two tiles (halves).
constexpr uint32_t kTile = C * 128;                       // 64 rows x 64 channels
constexpr uint32_t R_STAGE = 0;                           // per stage: [Q0 K0 Q1 K1 V0 V1]
constexpr uint32_t kStage = 6 * kTile, O_Q = 0, O_K = kTile, O_V = 4 * kTile, kHalf = 2 * kTile;
constexpr uint32_t R_T = 2 * kStage;                      // three terms of the decayed keys, [token][channel]
constexpr uint32_t R_P = R_T + 6 * kTile;                 // P [i][j], two buffers
constexpr uint32_t R_S = R_P + 2 * kTile;                 // S bf16 [dk][dv]: two halves of 128 rows
constexpr uint32_t kSHalf = 128 * 128;
constexpr uint32_t R_O = R_S + 2 * kSHalf;                // output staging [token][dv]
constexpr uint32_t R_PW = R_O + 2 * kTile;                // lambda^1 .. lambda^64
constexpr uint32_t kSmem = R_PW + C * 4 + 1024;
static_assert(kSmem <= 231000, "shared memory");

// ---- tensor memory columns (512)
__device__ __forceinline__ uint32_t tm_p(int b) { return b * 64; }            // Q K^T, lanes 0-63
__device__ __forceinline__ uint32_t tm_qs(int b) { return 128 + b * 128; }    // S^T Q^T
__device__ __forceinline__ uint32_t tm_pv(int b) { return 192 + b * 128; }    // V^T P^T
constexpr uint32_t TM_DS = 384;

enum Bar { LD, LD1, FREE, FREE1, QK, QK1, PREADY, PREADY1, OD, OD1, OFREE, OFREE1, QS, SREADY, TFULL, TFULL1, DS, DSFREE, NBAR };

struct Params {
    const float *log_decay;
    const int32_t *cu;
    int N, H;
    int64_t total;
    float scale;
    const float *init;          // initial states, or nullptr
    float *fin;                 // final states, or nullptr
    __nv_bfloat16 *out;
    const int32_t *order;       // longest-first order of the sequences, or nullptr
    uint32_t *status;
    int seg_len;                // 0: a chain is one item; else tokens per segment
    float *seg;                 // [segment][H][D][D]
    int64_t seg_cap;            // segments that seg has room for (more only if the offsets overlap)
};

// One piece of a chain: tokens [t0, t1) of one head.
struct Item {
    int64_t t0, t1;
    int head;
    const float *from;          // start state, nullptr for zeros
    float *to;                  // end state, nullptr for none
};

__device__ __forceinline__ void bounds(const Params &p, int seq, int64_t &bos, int64_t &eos, bool tell) {
    bos = p.cu[seq];
    eos = p.cu[seq + 1];
    if (bos < 0 || eos < bos || eos > p.total) {
        if (tell) report_status(p.status, kDevBadSeqlens);
        bos = eos = 0;
    }
}

// Walks this CTA's items in order; every role walks its own copy.
template <bool OUT>
struct Walk {
    int it = 0;
    __device__ bool next(const Params &p, Item &x, bool tell) {
        const int64_t chain_floats = (int64_t)D * D;
        if (p.seg_len == 0) {
            // rows of gridDim.x chains, dealt out forwards and backwards in turn: with the longest first, every
            // CTA gets about the same number of tokens
            const int64_t i = (int64_t)it * gridDim.x + ((it & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            ++it;
            if ((int64_t)(it - 1) * gridDim.x >= (int64_t)p.N * p.H) return false;
            if (i >= (int64_t)p.N * p.H) {      // the last row is shorter
                x.t0 = x.t1 = 0; x.head = 0; x.from = nullptr; x.to = nullptr;
                return true;
            }
            const int k = (int)(i / p.H), seq = p.order ? p.order[k] : k;
            x.head = (int)(i % p.H);
            bounds(p, seq, x.t0, x.t1, tell);
            const int64_t at = ((int64_t)seq * p.H + x.head) * chain_floats;
            x.from = p.init ? p.init + at : nullptr;
            x.to = p.fin ? p.fin + at : nullptr;
            return true;
        }
        // segments of all sequences in order, heads fastest; the state pass (OUT = false) skips each last one
        int64_t i = (int64_t)it * gridDim.x + blockIdx.x;
        ++it;
        x.head = (int)(i % p.H);
        i /= p.H;
        int64_t before = 0;                     // segments of the sequences before
        for (int n = 0; n < p.N; ++n) {
            int64_t bos, eos;
            bounds(p, n, bos, eos, tell && it == 1);
            // an empty sequence is one empty segment: its state is copied
            const int64_t segs = eos > bos ? (eos - bos + p.seg_len - 1) / p.seg_len : 1;
            if (i < before + segs) {
                if (i >= p.seg_cap) {
                    if (tell) report_status(p.status, kDevBadSeqlens);
                    return false;
                }
                const int64_t g = i - before;
                const int64_t at = ((int64_t)n * p.H + x.head) * chain_floats;
                float *cell = p.seg + (i * p.H + x.head) * chain_floats;
                x.t0 = bos + g * p.seg_len;
                x.t1 = x.t0 + p.seg_len < eos ? x.t0 + p.seg_len : eos;
                if (OUT) {
                    x.from = cell;
                    x.to = g == segs - 1 && p.fin ? p.fin + at : nullptr;
                } else {
                    x.from = nullptr;
                    x.to = cell;
                    if (g == segs - 1) { x.t1 = x.t0; x.to = nullptr; }
                }
                return true;
            }
            before += segs;
        }
        return false;
    }
};

__device__ __forceinline__ float log2_decay(const Params &p, int head) {
    // 2^(l2 n) with l2 no lower than -16384: exactly 0 for n >= 1 there, and 1 for n = 0
    return fmaxf(p.log_decay[head] * kLog2E, -16384.f);
}

// Wait by all lanes of a warp; false for all if it ran out for any.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t phase) {
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar, phase & 1, kWaitBudget));
}
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar);
}

// Descriptor of an operand whose rows run along K (tokens, or state rows) and
// whose contiguous axis is M or N: 64-wide column blocks `lead` bytes apart,
// groups of eight rows 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t addr, uint32_t lead) {
    return (ptx::sdesc_kmajor_sw128(addr) & ~((uint64_t)0x3FFF << 16)) | ((uint64_t)((lead >> 4) & 0x3FFF) << 16);
}
constexpr uint32_t kAMn = 1u << 15, kBMn = 1u << 16;      // instruction descriptor: operand is M- / N-major

template <bool OUT>
__global__ void __launch_bounds__(kThreads, 1)
    decay_chunk_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar[NBAR];
    __shared__ uint32_t s_tmem, s_abort, s_bad[2];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = ptx::smem_addr(sm);

    if (threadIdx.x == 0) {
        const uint8_t counts[NBAR] = {1, 1, OUT ? 3 : 1, OUT ? 3 : 1, 1, 1, 2, 2, 1, 1, 4, 4, 1, 8, 4, 4, 1, 8};
        for (int i = 0; i < NBAR; ++i) ptx::mbar_init(&bar[i], counts[i]);
        ptx::fence_mbar_init();
        s_abort = s_bad[0] = s_bad[1] = 0;
        if (OUT) ptx::prefetch_tensormap(&mq);
        ptx::prefetch_tensormap(&mk);
        ptx::prefetch_tensormap(&mv);
        if (OUT) ptx::prefetch_tensormap(&mo);
    }
    if (warp == 1) {
        ptx::tmem_alloc(&s_tmem, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = s_tmem;
    if (OUT) ptx::pdl_wait();          // the segments' start states
    bool ok = true;
    Walk<OUT> walk;
    Item x;

    if (warp == 0) {                                              // ---- loads
        if (lane == 0) {
            int c = 0;
            while (ok && walk.next(p, x, true)) {
                for (int64_t t = x.t0; t < x.t1; t += C, ++c) {
                    const int s = c & 1;
                    if (c >= 2 && !ptx::mbar_wait(&bar[FREE + s], ((c >> 1) - 1) & 1, kWaitBudget)) { ok = false; break; }
                    uint8_t *st = sm + R_STAGE + s * kStage;
                    ptx::mbar_arrive_expect_tx(&bar[LD + s], (OUT ? 6 : 4) * kTile);
                    for (int h = 0; h < 2; ++h) {
                        const int col = x.head * D + h * 64;
                        if (OUT) ptx::tma_load_2d(st + O_Q + h * kHalf, &mq, col, (int)t, &bar[LD + s]);
                        ptx::tma_load_2d(st + O_K + h * kHalf, &mk, col, (int)t, &bar[LD + s]);
                        ptx::tma_load_2d(st + O_V + h * kTile, &mv, col, (int)t, &bar[LD + s]);
                    }
                }
            }
        }
    } else if (warp == 1) {                                       // ---- Q K^T, S^T Q^T, V^T P^T
        if (OUT && lane == 0) {
            // chunks in all
            int total = 0;
            while (walk.next(p, x, false)) total += (int)((x.t1 - x.t0 + C - 1) / C);
            const uint32_t id_qk = ptx::idesc_bf16_f32(128, 64), id_qs = ptx::idesc_bf16_f32(128, 64) | kAMn;
            auto qk = [&](int c) {
                const int b = c & 1;
                if (!ptx::mbar_wait(&bar[LD + b], (c >> 1) & 1, kWaitBudget)) return false;
                // P's TMEM buffer was read two chunks ago
                if (c >= 2 && !ptx::mbar_wait(&bar[PREADY + b], ((c >> 1) - 1) & 1, kWaitBudget)) return false;
                ptx::tc_fence_after_sync();
                const uint32_t st = base + R_STAGE + b * kStage;
                // rows 0-63: Q K^T; rows 64-127 (K K^T) are not read
                mma_k<8>(tmem + tm_p(b), st + O_Q, kHalf, st + O_K, kHalf, id_qk, false);
                ptx::mma_commit(&bar[QK + b]);
                return true;
            };
            ok = total == 0 || qk(0);
            for (int c = 0; c < total && ok; ++c) {
                if (c + 1 < total && !qk(c + 1)) { ok = false; break; }
                const int b = c & 1;
                const uint32_t st = base + R_STAGE + b * kStage;
                if (!ptx::mbar_wait(&bar[SREADY], c & 1, kWaitBudget) ||
                    (c >= 2 && !ptx::mbar_wait(&bar[OFREE + b], ((c >> 1) - 1) & 1, kWaitBudget))) { ok = false; break; }
                ptx::tc_fence_after_sync();
                {
                    const uint64_t a = sdesc_mn_sw128(base + R_S, kSHalf), q = ptx::sdesc_kmajor_sw128(st + O_Q);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        ptx::mma_bf16_ss(tmem + tm_qs(b), a + k * (2048 >> 4), q + (((k >> 2) * kHalf + (k & 3) * 32) >> 4),
                                         id_qs, k > 0);
                }
                ptx::mma_commit(&bar[QS]);
                if (!ptx::mbar_wait(&bar[PREADY + b], (c >> 1) & 1, kWaitBudget) ||
                    !ptx::mbar_wait(&bar[TFULL + b], (c >> 1) & 1, kWaitBudget)) { ok = false; break; }    // (V's tail is clean)
                ptx::tc_fence_after_sync();
                {
                    const uint64_t a = sdesc_mn_sw128(st + O_V, kTile), q = ptx::sdesc_kmajor_sw128(base + R_P + b * kTile);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        ptx::mma_bf16_ss(tmem + tm_pv(b), a + k * (2048 >> 4), q + k * 2, id_qs, k > 0);
                }
                ptx::mma_commit(&bar[OD + b]);
                ptx::mma_commit(&bar[FREE + b]);
            }
        }
    } else if (warp == 2) {                                       // ---- the state's product
        if (lane == 0) {
            const uint32_t id = ptx::idesc_bf16_f32(128, 128) | kAMn | kBMn;
            int c = 0;
            while (ok && walk.next(p, x, false)) {
                for (int64_t t = x.t0; t < x.t1; t += C, ++c) {
                    const int b = c & 1;
                    if (!ptx::mbar_wait(&bar[TFULL + b], (c >> 1) & 1, kWaitBudget) ||
                        (c >= 1 && !ptx::mbar_wait(&bar[DSFREE], (c - 1) & 1, kWaitBudget))) { ok = false; break; }
                    ptx::tc_fence_after_sync();
                    const uint64_t v = sdesc_mn_sw128(base + R_STAGE + b * kStage + O_V, kTile);
#pragma unroll
                    for (int e = 0; e < 3; ++e) {
                        const uint64_t a = sdesc_mn_sw128(base + R_T + e * 2 * kTile, kTile);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            ptx::mma_bf16_ss(tmem + TM_DS, a + k * (2048 >> 4), v + k * (2048 >> 4), id, e > 0 || k > 0);
                    }
                    ptx::mma_commit(&bar[DS]);
                    ptx::mma_commit(&bar[FREE + b]);
                }
            }
        }
    } else if (warp >= 4 && warp < 8) {                           // ---- P, then the output
        if (OUT) {
            const int tid = threadIdx.x - 128, q = warp & 3;
            float *pw = reinterpret_cast<float *>(sm + R_PW);
            uint8_t *so = sm + R_O;
            // the chunk whose output is still to come
            int64_t ot = 0;
            int on = 0, ohead = 0, head = -1;
            float l2 = 0.f;
            auto output = [&](int c) {      // false: gave up (all 128 threads alike)
                const int b = c & 1;
                bool good = ptx::mbar_wait(&bar[OD + b], (c >> 1) & 1, kWaitBudget);
                if (tid == 0) ptx::bulk_wait_read();                 // the staging tile's last store
                const bool bad = *static_cast<volatile uint32_t *>(&s_bad[b]) != 0;   // an infinity or NaN in V
                if (ptx::bar_any(1, 128, !good || !ok)) return false;
                ptx::tc_fence_after_sync();
                if (!bad && tid == 0) ptx::mbar_arrive(&bar[FREE + b]);
                const int j = q * 32 + lane;                         // value channel
                const uint8_t *sp = sm + R_P + b * kTile, *sv = sm + R_STAGE + b * kStage + O_V + (j >> 6) * kTile;
                auto cell = [](const uint8_t *tile, int row, int col) {
                    return to_f32(*reinterpret_cast<const __nv_bfloat16 *>(tile + swz(row, (col & 63) >> 3) + (col & 7) * 2));
                };
#pragma unroll
                for (int i0 = 0; i0 < C; i0 += 16) {
                    float a[16], o[16];
                    ptx::tmem_ld16(tmem + ((uint32_t)q << 21) + tm_qs(b) + i0, a);
                    ptx::tmem_ld16(tmem + ((uint32_t)q << 21) + tm_pv(b) + i0, o);
                    ptx::tmem_ld_wait();
                    if (bad) {
                        // P's zeros would turn a later token's infinity into NaN: sum the real pairs alone
#pragma unroll 1
                        for (int i = 0; i < 16; ++i) {
                            float y = 0.f;
                            for (int s = 0; s <= i0 + i; ++s) y = fmaf(cell(sp, i0 + i, s), cell(sv, s, j), y);
                            o[0] = i == 0 ? y : o[0];
#pragma unroll
                            for (int e = 1; e < 16; ++e) o[e] = i == e ? y : o[e];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float y = fmaf(a[i], pw[i0 + i], o[i]) * p.scale;
                        *reinterpret_cast<__nv_bfloat16 *>(so + (j >> 6) * kTile + swz(i0 + i, (j & 63) >> 3) + (j & 7) * 2) =
                            __float2bfloat16_rn(y);
                    }
                }
                ptx::tc_fence_before_sync();
                warp_arrive(&bar[OFREE + b]);
                ptx::fence_async_smem();
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (bad && tid == 0) ptx::mbar_arrive(&bar[FREE + b]);
                if (on == C) {
                    if (tid == 0) {
                        ptx::tma_store_2d(&mo, ohead * D, (int)ot, so);
                        ptx::tma_store_2d(&mo, ohead * D + 64, (int)ot, so + kTile);
                        ptx::bulk_commit();
                    }
                } else {
                    for (int i = tid; i < on * 16; i += 128) {
                        const int r = i >> 4, ch = i & 15;
                        *reinterpret_cast<uint4 *>(p.out + ((ot + r) * p.H + ohead) * D + ch * 8) =
                            *reinterpret_cast<const uint4 *>(so + (ch >> 3) * kTile + swz(r, ch & 7));
                    }
                    asm volatile("bar.sync 1, 128;" ::: "memory");   // read before the next chunk's tile
                }
                return true;
            };
            int c = 0;
            while (ok && walk.next(p, x, false)) {
                for (int64_t t = x.t0; t < x.t1; t += C, ++c) {
                    const int b = c & 1;
                    // the chunk before leaves first where its powers differ from this chunk's
                    if (x.head != head && c > 0) {
                        if (!output(c - 1)) { ok = false; break; }
                        on = 0;
                    }
                    if (x.head != head) {
                        head = x.head;
                        l2 = log2_decay(p, head);
                        asm volatile("bar.sync 1, 128;" ::: "memory");
                        if (tid < C) pw[tid] = exp2f(l2 * (float)(tid + 1));
                    }
                    ok = warp_wait(&bar[QK + b], c >> 1);
                    if (ok && q < 2) {
                        ptx::tc_fence_after_sync();
                        const int i = q * 32 + lane;
                        uint8_t *sp = sm + R_P + b * kTile;
#pragma unroll
                        for (int j0 = 0; j0 < C; j0 += 16) {
                            float d[16];
                            ptx::tmem_ld16(tmem + ((uint32_t)q << 21) + tm_p(b) + j0, d);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const int gap = i - (j0 + e);
                                d[e] = gap >= 0 ? d[e] * ex2(l2 * (float)gap) : 0.f;
                            }
                            st_chunk(sp, swz(i, j0 >> 3), d);
                            st_chunk(sp, swz(i, (j0 >> 3) + 1), d + 8);
                        }
                        ptx::fence_async_smem();
                        ptx::tc_fence_before_sync();
                        warp_arrive(&bar[PREADY + b]);
                    }
                    if (c > 0 && on > 0) {
                        if (!output(c - 1)) { ok = false; break; }
                    } else if (ptx::bar_any(1, 128, !ok)) {
                        ok = false;
                        break;
                    }
                    ot = t;
                    on = (int)(x.t1 - t < C ? x.t1 - t : C);
                    ohead = head;
                }
            }
            if (ok && c > 0 && !output(c - 1)) ok = false;
            if (tid == 0) ptx::bulk_wait_all();
        }
    } else if (warp >= 8 && warp < 12) {                          // ---- the decayed keys in three terms
        const int tid = threadIdx.x - 256;
        int c = 0;
        while (ok && walk.next(p, x, false)) {
            const float l2 = log2_decay(p, x.head);
            for (int64_t t = x.t0; t < x.t1; t += C, ++c) {
                const int b = c & 1, n = (int)(x.t1 - t < C ? x.t1 - t : C);
                ok = warp_wait(&bar[LD + b], c >> 1) && (c == 0 || warp_wait(&bar[DS], c - 1));
                if (!ok) break;
                uint8_t *st = sm + R_STAGE + b * kStage;
                uint32_t top = 0;                                 // largest magnitudes of V's pairs
                const int ch = tid & 15;
                const uint32_t half = (ch >> 3), cc = ch & 7;
#pragma unroll 2
                for (int r = tid >> 4; r < C; r += 8) {
                    float k[8], hi[8];
                    ld_chunk(st + O_K + half * kHalf, swz(r, cc), k);
                    const float w = r < n ? exp2f(l2 * (float)(n - 1 - r)) : 0.f;
                    uint8_t *dst = sm + R_T + half * kTile;
                    const uint32_t at = swz(r, cc);
#pragma unroll
                    for (int e = 0; e < 8; ++e) k[e] = r < n ? k[e] * w : 0.f;
#pragma unroll
                    for (int term = 0; term < 3; ++term) {
                        uint4 u;
                        u.x = pack_bf16(k[0], k[1]); u.y = pack_bf16(k[2], k[3]);
                        u.z = pack_bf16(k[4], k[5]); u.w = pack_bf16(k[6], k[7]);
                        *reinterpret_cast<uint4 *>(dst + term * 2 * kTile + at) = u;
                        if (term < 2) {
                            const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 f = bf2_to_f2(uu[e]);
                                hi[2 * e] = f.x; hi[2 * e + 1] = f.y;
                            }
#pragma unroll
                            for (int e = 0; e < 8; ++e) k[e] -= hi[e];
                        }
                    }
                    uint4 *pv = reinterpret_cast<uint4 *>(st + O_V + half * kTile + at);
                    if (r < n) {
                        if (OUT) {
                            const uint4 u = *pv;
                            const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                // a lane of all-ones exponent, in either half
                                const uint32_t m = uu[e] & 0x7f807f80u;
                                top |= (uint32_t)((m & 0xffff0000u) == 0x7f800000u) | (uint32_t)((m & 0xffffu) == 0x7f80u);
                            }
                        }
                    } else {
                        *pv = make_uint4(0, 0, 0, 0);             // rows of the next sequence
                    }
                }
                if (OUT) {
                    // the flag of two chunks ago was read before its stage was handed back
                    const bool any = __any_sync(0xffffffffu, top != 0);
                    if (lane == 0 && any) atomicOr(&s_bad[b], 1u << (warp - 8));
                    if (lane == 0 && !any) atomicAnd(&s_bad[b], ~(1u << (warp - 8)));
                }
                ptx::fence_async_smem();
                warp_arrive(&bar[TFULL + b]);
            }
        }
    } else if (warp >= 12) {                                      // ---- the state
        const int q = warp & 3, col0 = ((warp - 12) >> 2) * 64, row = q * 32 + lane;
        const int64_t mine = (int64_t)row * D + col0;
        int c = 0;
        while (ok && walk.next(p, x, false)) {
            const float l2 = log2_decay(p, x.head);
            float s[64];
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (x.from) f = *reinterpret_cast<const float4 *>(x.from + mine + e);
                s[e] = f.x; s[e + 1] = f.y; s[e + 2] = f.z; s[e + 3] = f.w;
            }
            auto copy_out = [&](int e) {       // 16 columns as bf16
                uint8_t *ss = sm + R_S + (col0 >> 6) * kSHalf;
                st_chunk(ss, swz(row, e >> 3), s + e);
                st_chunk(ss, swz(row, (e >> 3) + 1), s + e + 8);
            };
            if (OUT && x.t1 > x.t0) {
                if (c > 0) ok = warp_wait(&bar[QS], c - 1);
                if (!ok) break;
#pragma unroll
                for (int e = 0; e < 64; e += 16) copy_out(e);
                ptx::fence_async_smem();
                warp_arrive(&bar[SREADY]);
            }
            for (int64_t t = x.t0; t < x.t1; t += C, ++c) {
                const int n = (int)(x.t1 - t < C ? x.t1 - t : C);
                const bool more = t + C < x.t1;
                const float f = exp2f(l2 * (float)n);
                ok = warp_wait(&bar[DS], c) && (!OUT || !more || warp_wait(&bar[QS], c));
                if (!ok) break;
                ptx::tc_fence_after_sync();
#pragma unroll
                for (int e = 0; e < 64; e += 16) {
                    float d[16];
                    ptx::tmem_ld16(tmem + ((uint32_t)q << 21) + TM_DS + col0 + e, d);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[e + i] = fmaf(f, s[e + i], d[i]);
                    if (OUT && more) copy_out(e);
                }
                ptx::tc_fence_before_sync();
                warp_arrive(&bar[DSFREE]);
                if (OUT && more) {
                    ptx::fence_async_smem();
                    warp_arrive(&bar[SREADY]);
                }
            }
            if (!ok) break;
            if (x.to) {
#pragma unroll
                for (int e = 0; e < 64; e += 4)
                    *reinterpret_cast<float4 *>(x.to + mine + e) = make_float4(s[e], s[e + 1], s[e + 2], s[e + 3]);
            }
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
        ptx::tmem_dealloc(tmem, 512);
    }
}

// Start states of the segments: S(0) = initial state, S(g + 1) = lambda^{seg_len}
// S(g) + b(g), in place over the b that the state pass left; one CTA column per
// (sequence, head), one float4 per thread.
__global__ void __launch_bounds__(256) decay_segments_kernel(const Params p) {
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int n = blockIdx.y / p.H, h = blockIdx.y % p.H;
    int64_t bos, eos, before = 0;
    for (int i = 0; i < n; ++i) {
        bounds(p, i, bos, eos, false);
        before += eos > bos ? (eos - bos + p.seg_len - 1) / p.seg_len : 1;
    }
    bounds(p, n, bos, eos, false);
    int64_t segs = eos > bos ? (eos - bos + p.seg_len - 1) / p.seg_len : 1;
    if (before + segs > p.seg_cap) segs = p.seg_cap - before;
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, step = (int64_t)p.H * D * D;
    const float f = exp2f(log2_decay(p, h) * (float)p.seg_len);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.init) s = *reinterpret_cast<const float4 *>(p.init + (int64_t)blockIdx.y * D * D + at);
    float4 *cell = reinterpret_cast<float4 *>(p.seg + (before * p.H + h) * D * D + at);
    // (the first segment's start state is copied too: its buffer may be the one that the last segment writes)
#pragma unroll 4
    for (int64_t g = 0; g + 1 < segs; ++g) {
        const float4 b = cell[g * (step / 4)];
        cell[g * (step / 4)] = s;
        s.x = fmaf(f, s.x, b.x); s.y = fmaf(f, s.y, b.y); s.z = fmaf(f, s.z, b.z); s.w = fmaf(f, s.w, b.w);
    }
    if (segs > 0) cell[(segs - 1) * (step / 4)] = s;
}

constexpr size_t kOrderAt = 256;

// Tokens per segment, or 0 for whole chains.  Segments cost a second pass over
// k and v, so they are taken only where the chains fill at most half of the
// SMs; then one segment per SM, in whole chunks.
int segment_tokens(int64_t total, int N, int H, int sms) {
    const int64_t chains = (int64_t)N * H;
    if (chains * 2 > sms || N > 64) return 0;
    const int64_t per_chain_slots = (sms - chains) * C;           // sum over the sequences of len / m below it
    int64_t m = (total * H + per_chain_slots - 1) / per_chain_slots;
    if (N == 1) m = ((total + C - 1) / C + sms / H - 1) / (sms / H);
    if (m < 4) m = 4;
    const int64_t len = m * C;
    if (len * 2 > total) return 0;
    return (int)len;
}

}  // namespace

size_t decay_prefill_tc_workspace(int64_t total, int N, int H) {
    const int len = segment_tokens(total, N, H, sm_count());
    size_t bytes = kOrderAt + sizeof(int32_t) * (size_t)N;
    bytes = (bytes + 1023) & ~size_t(1023);
    if (len) bytes += (size_t)((total / len + N) * H) * D * D * sizeof(float);
    return bytes;
}

cudaError_t launch_decay_prefill_tc(const DecayParams &d, void *workspace, size_t workspace_bytes, cudaStream_t st) {
    CUtensorMap mq, mk, mv, mo;
    const uint64_t T = (uint64_t)d.total, cols = (uint64_t)d.H * D;
    if (!make_map_2d(&mq, d.q, true, T, cols, d.ldq * 2, C) || !make_map_2d(&mk, d.k, true, T, cols, d.ldk * 2, C) ||
        !make_map_2d(&mv, d.v, true, T, cols, d.ldv * 2, C) || !make_map_2d(&mo, d.out, true, T, cols, cols * 2, C))
        return cudaErrorInvalidValue;
    const int sms = sm_count();
    Params p{d.log_decay, d.cu_seqlens, d.num_seqs, d.H, d.total, d.scale, d.init, d.fin,
             static_cast<__nv_bfloat16 *>(d.out), nullptr, d.status, 0, nullptr, 0};
    cudaError_t e = cudaFuncSetAttribute(decay_chunk_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(decay_chunk_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const bool room = ws && workspace_bytes >= decay_prefill_tc_workspace(d.total, d.num_seqs, d.H);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = &attr;
    const int64_t chains = (int64_t)d.num_seqs * d.H;
    const int len = room ? segment_tokens(d.total, d.num_seqs, d.H, sms) : 0;
    if (len) {
        p.seg_len = len;
        p.seg = reinterpret_cast<float *>(ws + ((kOrderAt + sizeof(int32_t) * (size_t)d.num_seqs + 1023) & ~size_t(1023)));
        p.seg_cap = d.total / len + d.num_seqs;
        const int64_t items = p.seg_cap * d.H;
        cfg.gridDim = dim3((unsigned)(items < sms ? items : sms));
        cfg.numAttrs = 0;
        if ((e = cudaLaunchKernelEx(&cfg, decay_chunk_kernel<false>, mq, mk, mv, mo, p)) != cudaSuccess) return e;
        cudaLaunchConfig_t c2 = cfg;
        c2.gridDim = dim3(D * D / 1024, (unsigned)chains);
        c2.blockDim = dim3(256);
        c2.dynamicSmemBytes = 0;
        c2.numAttrs = 1;
        if ((e = cudaLaunchKernelEx(&c2, decay_segments_kernel, p)) != cudaSuccess) return e;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, decay_chunk_kernel<true>, mq, mk, mv, mo, p);
    }
    if (room && chains > sms && d.num_seqs > 1) {
        int32_t *order = reinterpret_cast<int32_t *>(ws + kOrderAt);
        if ((e = launch_schedule(d.cu_seqlens, d.num_seqs, order, reinterpret_cast<uint32_t *>(ws + 16),
                                 reinterpret_cast<uint32_t *>(ws), st)) != cudaSuccess)
            return e;
        p.order = order;
        cfg.numAttrs = 1;
    }
    cfg.gridDim = dim3((unsigned)(chains < sms ? chains : sms));
    return cudaLaunchKernelEx(&cfg, decay_chunk_kernel<true>, mq, mk, mv, mo, p);
}

}  // namespace kda
