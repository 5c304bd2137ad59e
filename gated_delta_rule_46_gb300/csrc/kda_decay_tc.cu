// kda_decay_tc.cu -- the chunked form of linear attention with one decay per
// head (bf16) on the tensor cores, in tiles of D = 64 or 128 channels for dk, dv <= D.
//
// Per chain (sequence, head), in chunks of C = 64 tokens with n of them real,
// start state S and lambda = exp(log_decay):
//   P_ij = lambda^{i-j} q_i . k_j  (j <= i, else 0)
//   O^T  = (S^T Q^T) diag(lambda^{i+1}) + V^T P^T
//   S^T <- lambda^n S^T + sum_j v_j (lambda^{n-1-j} k_j)^T
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
// Roles of the 20 warps of a CTA (one CTA per SM): 0 and 1 take P out of TMEM, and a
// thread of 0 loads by TMA, up to three chunks ahead; 2 issues the state's product; 3
// issues Q K^T, S^T Q^T and V^T P^T; 4-7 write the output; 8-11 split the decayed
// keys; 12-19 hold the state, 64 key channels of one value channel per thread, and
// leave its bf16 copy in TMEM, where the MMA takes it from.  mbarriers link them.
// The state pass of a segmented batch writes no output: there 4-11 split the keys and
// 3 loads.
//
// What bounds it, of a chunk with 128 channels: its 64 KB from and to HBM are 1.5 us
// at a CTA's share of the copy rate, and its traffic in shared memory about 2,700
// cycles, 1.4 us: the MMAs' operands 1,470 (state's product 770, its V read once per
// term), the keys' terms 510, TMA in and out 510, P and the output 190.  Together they
// take 1.8: 133k ragged tokens of 32 heads run in 803 us, 5.5 TB/s, with the tensor
// pipe 38 % and the issue slots 57 % busy, and the two threads that issue MMAs are
// held up by them nearly all of the time.  d = 64: 635 us for as many tokens and heads.
//   Measured at that batch, where not noted: S's copy in shared memory, which leaves
// room for two stages of loads, 1034 us (917 in TMEM); waits that are calls, 1173; all
// warps at 96 registers, 918 (810); loads by an output warp 884, in pieces between the
// state's products 1079, keys and values in stages of their own 826; the output's
// next part out of TMEM ahead, 811.
#include <cuda.h>

#include "kda_decay.cuh"
#include "kda_tc_util.cuh"
#include "kda_testing.h"
#include "kda_tmap.cuh"
#include "sm100_ptx.cuh"

namespace kda {

cudaError_t launch_schedule(const int32_t *cu, int num_seqs, int32_t *order, uint32_t *counter, uint32_t *status,
                            cudaStream_t st);

namespace {

using namespace tc;

constexpr int C = 64;
constexpr int kThreads = 640;
constexpr long long kWaitBudget = 2000000000LL;   // cycles (about one second)
constexpr long long kDrain = 20000000LL;

// ---- shared memory, bytes from a 1024-aligned base.  Tiles have 128-byte rows
// with the 128-byte swizzle; a row of 128 channels is two tiles (halves).
constexpr uint32_t kTile = C * 128;                       // 64 rows x 64 channels
template <int D, bool OUT>
struct Lay {
    static constexpr int HV = D / 64;                     // halves
    static constexpr int NS = (OUT ? 3 : 4) * (2 / HV);   // stages of loads
    static constexpr int NB = OUT ? 1 : 2;                // buffers of the terms and of their product
    static constexpr uint32_t half = (OUT ? 2 : 1) * kTile;               // from Q0 to Q1, from K0 to K1
    static constexpr uint32_t q = 0, k = OUT ? kTile : 0, v = HV * half;  // in a stage: [(Q0) K0 (Q1) (K1) V0 (V1)]
    static constexpr uint32_t stage = v + HV * kTile;
    static constexpr uint32_t T = NS * stage;             // three terms of the decayed keys, [token][channel]
    static constexpr uint32_t term = HV * kTile;
    static constexpr uint32_t P = T + NB * 3 * term;      // P [i][j], two buffers
    static constexpr uint32_t O = P + 2 * kTile;          // output staging [token][dv]
    static constexpr uint32_t PW = O + HV * kTile;        // lambda^1 .. lambda^64, of two items in turn
    static constexpr uint32_t KW = PW + 2 * C * 4;        // lambda^0 .. lambda^63, one copy for each key warp
    static constexpr uint32_t bytes = (OUT ? KW + 4 * C * 4 : P) + 1024;
    static_assert(bytes <= 232448 - 256, "shared memory");
    // with 64 channels the MMAs' upper 64 rows (M = 128) are whatever lies one tile on: rows that no one reads
    // barriers
    enum Bar { LD, FREE = LD + NS, QK = FREE + NS, PREADY = QK + 2, OD = PREADY + 2, OFREE = OD + 2, QS = OFREE + 2, SREADY,
               TF, DSH = TF + 2 * NS, DS = DSH + 2 * NB, DSFREE = DS + NB, NBAR = DSFREE + NB };
};

// ---- tensor memory columns (512)
constexpr uint32_t TM_P = 0;                                                  // Q K^T, lanes 0-63
constexpr uint32_t TM_S = 64;                                                 // S^T as bf16 pairs: lane = dv, 64 columns
__device__ __forceinline__ uint32_t tm_qs(int b) { return 128 + b * 128; }    // S^T Q^T
__device__ __forceinline__ uint32_t tm_pv(int b) { return 192 + b * 128; }    // V^T P^T
__device__ __forceinline__ uint32_t tm_ds(int b) { return 384 - b * 128; }    // what the chunk adds to S^T

struct Params {
    DecaySegs g;
    const float *log_decay;
    float scale;
    const float *init;          // initial states, or nullptr
    float *fin;                 // final states, or nullptr
    __nv_bfloat16 *out;
    const __nv_bfloat16 *v;     // (the values again, for the rare path)
    int64_t ldv;
    const int32_t *order;       // longest-first order of the sequences, or nullptr
    int expire;                 // test support
    int dk, dv;                 // at most D
};

// One piece of a chain: tokens [t0, t1) of one head.
struct Item {
    int t0, t1;
    int head;
    const float *from;          // start state, nullptr for zeros
    float *to;                  // end state, nullptr for none
};

// Walks this CTA's items in order; every role walks its own copy.
template <int D, bool OUT, bool FULL>
struct Walk {
    unsigned it = 0;
    __device__ __forceinline__ bool next(const Params &p, Item &x, bool tell) {
        const int64_t kState = FULL ? (int64_t)D * D : (int64_t)p.dk * p.dv;
        const unsigned H = (unsigned)p.g.H;
        if (p.g.len == 0) {
            // rows of gridDim.x chains, dealt out forwards and backwards in turn: with the longest first, every
            // CTA gets about the same number of tokens
            const unsigned chains = (unsigned)p.g.N * H, row = it * gridDim.x;
            if (row >= chains) return false;
            const unsigned i = row + ((it & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            ++it;
            x.t0 = x.t1 = x.head = 0;
            x.from = nullptr;
            x.to = nullptr;
            if (i >= chains) return true;       // the last row is shorter
            const unsigned k = i / H;
            const int seq = p.order ? p.order[k] : (int)k;
            x.head = (int)(i - k * H);
            seq_range(p.g, seq, x.t0, x.t1, tell);
            const int64_t at = ((int64_t)seq * H + x.head) * kState;
            if (p.init) x.from = p.init + at;
            if (p.fin) x.to = p.fin + at;
            return true;
        }
        // segments of all sequences in order, heads fastest; the state pass (OUT = false) skips each last one
        const unsigned i = it * gridDim.x + blockIdx.x, seg = i / H;
        ++it;
        x.head = (int)(i - seg * H);
        Segment sg;
        if (!find_segment(p.g, seg, sg, tell && it == 1)) return false;
        x.t0 = sg.t0;
        x.t1 = sg.t1;
        float *cell = p.g.cells + ((int64_t)seg * H + x.head) * kState;
        x.from = OUT ? cell : nullptr;
        x.to = cell;
        if (OUT) x.to = sg.last && p.fin ? p.fin + ((int64_t)sg.n * H + x.head) * kState : nullptr;
        else if (sg.last) { x.t1 = x.t0; x.to = nullptr; }
        return true;
    }
};

// Chunks of all of a CTA's items.
template <int D, bool OUT, bool FULL>
__device__ __forceinline__ int chunks_of(const Params &p, bool tell) {
    Walk<D, OUT, FULL> walk;
    Item x;
    int total = 0;
    while (walk.next(p, x, tell)) total += (x.t1 - x.t0 + C - 1) / C;
    return total;
}

__device__ __forceinline__ float log2_decay(const Params &p, int head) { return decay_log2(p.log_decay, head); }

// x to the nearest of 18 significant bits (24 - 6, by Veltkamp's splitting): its products with counts below 64, and their
// differences, are exact.  As l2 it makes P's diagonal weight lambda^0 exactly 1, however strong the decay; lambda^n
// moves by at most 2^-18 |n l2| ln 2 of itself, 2^-14 where it is 2^-16.  (l2 (i - j) with the difference first is exact
// too, but takes an instruction more per weight: 2 % more time for the ragged batch above.)
__device__ __forceinline__ float round18(float x) {
    const float t = __fmul_rn(x, 65.f);
    return __fsub_rn(t, __fsub_rn(t, x));
}

// The bounded wait in few instructions (about a second on the 32-bit clock).
// The roles' loops run side by side, so what they cost is instruction fetches as
// much as issue slots; and a call would spill the state's registers.
__device__ __forceinline__ bool wait_on(uint64_t *bar, uint32_t phase) {
    const unsigned t0 = (unsigned)clock();
    while (!ptx::mbar_try_wait(bar, phase & 1))
        if ((unsigned)clock() - t0 > (unsigned)kWaitBudget) return false;
    return true;
}

// Wait by all lanes of a warp; false for all if it ran out for any.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t phase) {
    return __all_sync(0xffffffffu, wait_on(bar, phase));
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

// x = k w of eight bf16 k, as three bf16 terms of eight bits each: x cut after
// eight bits of its significand, the exact remainder cut likewise, and the
// rest, which has at most eight bits left.
__device__ __forceinline__ void split3(const uint4 &k, float w, uint4 &t1, uint4 &t2, uint4 &t3) {
    const uint32_t u[4] = {k.x, k.y, k.z, k.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16) * w;
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u) * w;
    }
    auto cut = [&](uint4 &t) {
        uint32_t b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(x[i]);
        t.x = __byte_perm(b[0], b[1], 0x7632);
        t.y = __byte_perm(b[2], b[3], 0x7632);
        t.z = __byte_perm(b[4], b[5], 0x7632);
        t.w = __byte_perm(b[6], b[7], 0x7632);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] -= __uint_as_float(b[i] & 0xffff0000u);
    };
    cut(t1);
    cut(t2);
    cut(t3);
}

// sum_{s <= i} P_is v_sj for token i of the chunk at token t and value channel j
// of a head, v from global memory.
__device__ __forceinline__ float real_pairs(const Params &p, const uint8_t *sp, int t, int t1, int head, int j, int i) {
    float y = 0.f;
    if (t + i >= t1 || j >= p.dv) return y;
    const int at = head * p.dv + j;
#pragma unroll 1
    for (int s = 0; s <= i; ++s)
        y = fmaf(to_f32(*reinterpret_cast<const __nv_bfloat16 *>(sp + swz(i, s >> 3) + (s & 7) * 2)),
                 to_f32(p.v[(int64_t)(t + s) * p.ldv + at]), y);
    return y;
}

// FULL: dk = dv = D, 2-D tensor maps [token][head, channel]; else 3-D maps, which give zeros for the channels that are not
// there, and states of dk x dv (32 x 32, 32 prompts of up to 2048 tokens, 16 heads: 93 us, 501 on the CUDA cores; 64 x
// 128: 122 us, 1418; full heads by 3-D maps: 823 us for the ragged batch above, 803 by 2-D ones).
template <int D, bool OUT, bool FULL>
__global__ void __launch_bounds__(kThreads, 1)
    decay_chunk_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, const Params p) {
    using L = Lay<D, OUT>;
    constexpr int NS = L::NS, HV = L::HV, NB = L::NB;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar[L::NBAR];
    __shared__ uint32_t s_tmem, s_abort;
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = ptx::smem_addr(sm);
    const int dk = FULL ? D : p.dk, dv = FULL ? D : p.dv;

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::NBAR; ++i) {
            int n = 1;
            if (i >= L::FREE && i < L::QK) n = OUT ? 2 : 1;             // the two issuers
            if (i >= L::PREADY && i < L::OD) n = 2;                     // warps 0, 1
            if ((i >= L::OFREE && i < L::QS) || (i >= L::TF && i < L::DSH)) n = 4;   // the output's, the keys' warps
            if (i == L::SREADY || i >= L::DSFREE) n = 4 * HV;           // the state's warps
            ptx::mbar_init(&bar[i], n);
        }
        ptx::fence_mbar_init();
        s_abort = 0;
        if (OUT) ptx::prefetch_tensormap(&mq);
        ptx::prefetch_tensormap(&mk);
        ptx::prefetch_tensormap(&mv);
        if (OUT) ptx::prefetch_tensormap(&mo);
    }
    if (warp == 1) {
        ptx::tmem_alloc(&s_tmem, 512);
        ptx::tmem_relinquish();
    }
    if (OUT)                           // P's masked quarter stays zero
        for (int i = threadIdx.x; i < 2 * (int)kTile / 16; i += kThreads)
            reinterpret_cast<uint4 *>(sm + L::P)[i] = make_uint4(0, 0, 0, 0);
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = s_tmem;
    // In the output pass over segments only the state's warps wait for the kernel before: all that it writes is their
    // start states, and what came before the state pass was complete before any block of that pass let this one start.
    const bool early = OUT && p.g.len > 0;
    if (!early) ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    bool ok = true;
    Walk<D, OUT, FULL> walk;
    Item x;
    // Loads the next chunk (one thread); false at the end, or if its stage does not get free.
    int ls = 0, lround = 0, lt = 0, lt1 = 0, lhead = 0;
    auto load = [&]() -> bool {
        while (lt >= lt1) {
            Item y;
            if (!walk.next(p, y, false)) return false;
            lt = y.t0;
            lt1 = y.t1;
            lhead = y.head;
        }
        if (lround > 0 && !wait_on(&bar[L::FREE + ls], lround - 1)) {
            ok = false;
            return false;
        }
        uint64_t *full = &bar[L::LD + ls];
        uint8_t *st = sm + ls * L::stage;
        ptx::mbar_arrive_expect_tx(full, (OUT ? 3 : 2) * HV * kTile);
#pragma unroll 1
        for (int h = 0; h < HV; ++h) {
            if (FULL) {
                const int col = lhead * D + h * 64;
                ptx::tma_load_2d(st + L::k + h * L::half, &mk, col, lt, full);
                if (OUT) ptx::tma_load_2d(st + L::q + h * L::half, &mq, col, lt, full);
                ptx::tma_load_2d(st + L::v + h * kTile, &mv, col, lt, full);
            } else {
                ptx::tma_load_3d(st + L::k + h * L::half, &mk, h * 64, lhead, lt, full);
                if (OUT) ptx::tma_load_3d(st + L::q + h * L::half, &mq, h * 64, lhead, lt, full);
                ptx::tma_load_3d(st + L::v + h * kTile, &mv, h * 64, lhead, lt, full);
            }
        }
        lt += C;
        if (++ls == NS) { ls = 0; ++lround; }
        return true;
    };
    // 96 registers a thread at launch (61,440); of the five warpgroups' 480 the state's two take 120 each
    if (warp < 4) {
        ptx::regs_dec<80>();
        if (warp == 2) {                                              // ---- the state's product
            const int total = chunks_of<D, OUT, FULL>(p, true);
            if (ptx::elect_one()) {
                const uint32_t id = ptx::idesc_bf16_f32(128, D) | kAMn | kBMn;
                const uint64_t dt = sdesc_mn_sw128(base + L::T, kTile);
                int s = 0, sp = 0, b = 0, bp = 0;                     // the chunk's stage, the product's buffer; their rounds
                for (int c = 0; c < total && ok; ++c) {
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        if (!wait_on(&bar[L::TF + 2 * s + half], sp) ||
                            (half == 0 && bp > 0 && !wait_on(&bar[L::DSFREE + b], bp - 1))) { ok = false; break; }
                        ptx::tc_fence_after_sync();
                        const uint64_t a = dt + (b * 3 * L::term + half * 4096) / 16;
                        const uint64_t v = sdesc_mn_sw128(base + s * L::stage + L::v, kTile) + half * (4096 >> 4);
#pragma unroll 2
                        for (int e = 0; e < 6; ++e)
                            ptx::mma_bf16_ss(tmem + tm_ds(b), v + (e & 1) * (2048 >> 4),
                                             a + ((e >> 1) * L::term + (e & 1) * 2048) / 16, id, half > 0 || e > 0);
                        ptx::mma_commit(&bar[L::DSH + 2 * b + half]);
                    }
                    ptx::mma_commit(&bar[L::DS + b]);
                    ptx::mma_commit(&bar[L::FREE + s]);
                    if (++s == NS) { s = 0; ++sp; }
                    if (++b == NB) { b = 0; ++bp; }
                }
            }
        } else if (!OUT && warp == 3) {                               // ---- loads of the state pass
            if (ptx::elect_one())
                while (load()) {}
        } else if (warp < 2) {                                        // ---- P: thread = token of the chunk
            if (OUT) {
                const int i = threadIdx.x;
                int c = 0;
                Walk<D, OUT, FULL> mine;                                    // (`walk` is the loads')
                if (i == 0)
                    while (lround == 0 && load()) {}
                __syncwarp();
                while (ok && mine.next(p, x, false)) {
                    const float l2 = round18(log2_decay(p, x.head));
                    for (int t = x.t0, t1 = x.t1; t < t1; t += C, ++c) {
                        const int b = c & 1;
                        // P is a chunk ahead of its use: there is time to wait for the stage of two chunks ago
                        if (c >= 2 && i == 0) load();
                        // the output products of two chunks ago have read this buffer, and so has their output if it had to
                        ok = __all_sync(0xffffffffu, ok) && warp_wait(&bar[L::QK + b], c >> 1) &&
                             (c < 2 || warp_wait(&bar[L::OFREE + b], (c >> 1) - 1));
                        if (!ok) break;
                        ptx::tc_fence_after_sync();
                        uint8_t *sp = sm + L::P + b * kTile;
                        // (columns 32-63 of rows 0-31 are never written: zero from the start)
#pragma unroll 1
                        for (int j0 = 0; j0 < 32 * (warp + 1); j0 += 32) {
                            float d[32];
                            ptx::tmem_ld32(tmem + ((uint32_t)warp << 21) + TM_P + j0, d);
                            const float a0 = l2 * (float)(i - j0);               // lambda^{i - j} = 2^{a0 - l2 (j - j0)}, exactly
                            ptx::tmem_ld_wait(d);
#pragma unroll
                            for (int e = 0; e < 32; ++e) d[e] *= ex2(fmaf(-(float)e, l2, a0));
                            if (j0 == 32 * warp)
#pragma unroll
                                for (int e = 0; e < 32; ++e) d[e] = e <= lane ? d[e] : 0.f;
#pragma unroll
                            for (int e = 0; e < 32; e += 8) st_chunk(sp, swz(i, (j0 + e) >> 3), d + e);
                        }
                        ptx::fence_async_smem();
                        ptx::tc_fence_before_sync();
                        warp_arrive(&bar[L::PREADY + b]);
                    }
                }
            }
        } else if (OUT && warp == 3) {                                // ---- Q K^T, S^T Q^T, V^T P^T
            const int total = chunks_of<D, OUT, FULL>(p, false);
            if (ptx::elect_one()) {
                const uint32_t id = ptx::idesc_bf16_f32(128, 64);
                int s = 0, sp = 0, ns = 0, np = 0;                    // this chunk's stage and round, the next one's
                for (int c = -1; c < total && ok; ++c) {              // (step -1: the first chunk's scores alone)
                    const int b = c & 1, phase = (c >> 1) & 1;
                    const uint32_t st = base + s * L::stage;
                    if (c >= 0) {
                        if (!wait_on(&bar[L::SREADY], c & 1) ||
                            (c >= 2 && !wait_on(&bar[L::OFREE + b], phase ^ 1))) { ok = false; break; }
                        ptx::tc_fence_after_sync();
                        const uint64_t q = ptx::sdesc_kmajor_sw128(st + L::q);
#pragma unroll 2
                        for (int k = 0; k < D / 16; ++k)
                            ptx::mma_bf16_ts(tmem + tm_qs(b), tmem + TM_S + k * 8,
                                             q + (((k >> 2) * L::half + (k & 3) * 32) >> 4), id, k > 0);
                        ptx::mma_commit(&bar[L::QS]);
                        if (!wait_on(&bar[L::PREADY + b], phase)) { ok = false; break; }
                        ptx::tc_fence_after_sync();
                    }
                    // The next chunk's scores go ahead of this chunk's output if its tiles are here, else after it: their
                    // load may be waiting for this very chunk's stage.
                    bool todo = c + 1 < total;
#pragma unroll 1
                    for (int pass = 0; pass < 2; ++pass) {
                        if (todo && (pass == 1 || c < 0 || ptx::mbar_test(&bar[L::LD + ns], np & 1))) {
                            todo = false;
                            if (!wait_on(&bar[L::LD + ns], np)) { ok = false; break; }
                            ptx::tc_fence_after_sync();
                            const uint32_t sn = base + ns * L::stage;
                            // rows 0-63: Q K^T; rows 64-127 (K K^T) are not read
                            const uint64_t q = ptx::sdesc_kmajor_sw128(sn + L::q), kd = ptx::sdesc_kmajor_sw128(sn + L::k);
#pragma unroll 2
                            for (int k = 0; k < D / 16; ++k) {
                                const uint32_t at = ((k >> 2) * L::half + (k & 3) * 32) >> 4;
                                ptx::mma_bf16_ss(tmem + TM_P, q + at, kd + at, id, k > 0);
                            }
                            ptx::mma_commit(&bar[L::QK + (b ^ 1)]);
                        }
                        if (c < 0 || pass == 1) continue;
                        if (!wait_on(&bar[L::TF + 2 * s], sp) ||                  // (V's tail is clean)
                            !wait_on(&bar[L::TF + 2 * s + 1], sp)) { ok = false; break; }
                        ptx::tc_fence_after_sync();
                        const uint64_t a = sdesc_mn_sw128(st + L::v, kTile);
                        const uint64_t pb = ptx::sdesc_kmajor_sw128(base + L::P + b * kTile);
#pragma unroll 2
                        for (int k = 0; k < 4; ++k)
                            ptx::mma_bf16_ss(tmem + tm_pv(b), a + k * (2048 >> 4), pb + k * 2, id | kAMn, k > 0);
                        ptx::mma_commit(&bar[L::OD + b]);
                        ptx::mma_commit(&bar[L::FREE + s]);
                    }
                    s = ns;
                    sp = np;
                    if (++ns == NS) { ns = 0; ++np; }
                }
            }
        }
    } else if (OUT && warp < 8) {                                 // ---- the output
        ptx::regs_dec<80>();
        {
            const int tid = threadIdx.x - 128, q = warp & 3;
            float *pw = reinterpret_cast<float *>(sm + L::PW);
            uint8_t *so = sm + L::O;
            int c = 0, item = 0;
            while (ok && walk.next(p, x, false)) {
                const int t1 = x.t1, head = x.head;
                if (t1 > x.t0) {                                     // (read after the first chunk's barrier)
                    ++item;
                    if (tid < C) pw[(item & 1) * C + tid] = exp2f(log2_decay(p, head) * (float)(tid + 1));
                }
                for (int t = x.t0; t < t1; t += C, ++c) {
                    const int b = c & 1;
                    const bool good = wait_on(&bar[L::OD + b], (c >> 1) & 1);
                    if (tid == 0) ptx::bulk_wait_read();             // the staging tile's last store
                    ok = !ptx::bar_any(1, 128, !good);        // all 128 threads go on or give up alike
                    if (!ok) break;
                    ptx::tc_fence_after_sync();
                    const uint8_t *sp = sm + L::P + b * kTile;
                    const float *pwo = pw + (item & 1) * C;
                    // 16 value channels x 32 tokens at a time, as 8 x 8 tiles that are stored transposed
#pragma unroll 1
                    for (int part = q * 32 < D ? 0 : 4; part < 4; ++part) {    // (64 channels: two warps)
                        const int j0 = q * 32 + (part & 1) * 16, i0 = (part >> 1) * 32;
                        const uint32_t at = tmem + ((uint32_t)j0 << 16) + i0;
                        float a[16], o[16];
                        ptx::tmem_ld_tiles4(at + tm_qs(b), a);
                        ptx::tmem_ld_tiles4(at + tm_pv(b), o);
                        ptx::tmem_ld_wait(a, o);
                        const int ic = i0 + 2 * (lane & 3);          // this thread's first token
                        // an infinity or NaN in v shows in its channel at every token, as P's zeros for later tokens turn
                        // it into NaN: there the sums are taken again over the real pairs
                        float probe = 0.f;
#pragma unroll
                        for (int e = 0; e < 16; ++e) probe = fmaf(o[e], 0.f, probe);
                        if (probe != 0.f)
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = real_pairs(p, sp, t, t1, head, j0 + (lane >> 2) + ((e >> 1) & 1) * 8,
                                                  ic + (e >> 2) * 8 + (e & 1));
                        uint32_t u[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = *reinterpret_cast<const float2 *>(pwo + ic + e * 8);
                            u[2 * e] = pack_bf16(fmaf(a[4 * e], f.x, o[4 * e]) * p.scale,
                                                 fmaf(a[4 * e + 1], f.y, o[4 * e + 1]) * p.scale);
                            u[2 * e + 1] = pack_bf16(fmaf(a[4 * e + 2], f.x, o[4 * e + 2]) * p.scale,
                                                     fmaf(a[4 * e + 3], f.y, o[4 * e + 3]) * p.scale);
                        }
                        // tile lane / 8: tokens + 8 (tile / 2), channels + 8 (tile % 2); row lane % 8
                        const int r = i0 + (lane >> 4) * 8 + (lane & 7), ch = (j0 & 63) / 8 + ((lane >> 3) & 1);
                        const uint32_t to = ptx::smem_addr(so) + (j0 >> 6) * kTile;
                        ptx::stmatrix4_trans(to + swz(r, ch), u[0], u[1], u[2], u[3]);
                        ptx::stmatrix4_trans(to + swz(r + 16, ch), u[4], u[5], u[6], u[7]);
                    }
                    ptx::tc_fence_before_sync();
                    warp_arrive(&bar[L::OFREE + b]);
                    ptx::fence_async_smem();
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    const int on = min(t1 - t, C);
                    if (on == C) {
                        if (tid == 0) {
                            if (FULL) {
                                ptx::tma_store_2d(&mo, head * D, t, so);
                                if (HV == 2) ptx::tma_store_2d(&mo, head * D + 64, t, so + kTile);
                            } else {
                                ptx::tma_store_3d(&mo, 0, head, t, so);
                                if (HV == 2 && dv > 64) ptx::tma_store_3d(&mo, 64, head, t, so + kTile);
                            }
                            ptx::bulk_commit();
                        }
                    } else {
                        for (int i = tid; i < on * (D / 8); i += 128) {
                            const int r = i / (D / 8), ch = i % (D / 8);
                            if (ch * 8 >= dv) continue;
                            *reinterpret_cast<uint4 *>(p.out + ((int64_t)(t + r) * p.g.H + head) * dv + ch * 8) =
                                *reinterpret_cast<const uint4 *>(so + (ch >> 3) * kTile + swz(r, ch & 7));
                        }
                        asm volatile("bar.sync 1, 128;" ::: "memory");   // read before the next chunk's tile
                    }
                }
            }
            if (tid == 0) ptx::bulk_wait_all();
        }
    } else if (warp < 12) {                                       // ---- the decayed keys in three terms
        ptx::regs_dec<80>();
        constexpr int RP = 128 / (D / 8), NR = 32 / RP;                       // rows at a time; times per half chunk
        // both halves of a chunk, or (where no output is written) one half by warps 4-7 and one by 8-11
        const int th0 = OUT || warp < 8 ? 0 : 1, th1 = OUT || warp >= 8 ? 2 : 1;
        const int tid = threadIdx.x & 127, r0 = tid / (D / 8), ch = tid % (D / 8);   // rows r0, r0 + RP, ...; 16-byte column
        const uint32_t half = ch >> 3, at0 = swz(r0, ch & 7);                 // (8 rows on: 1024 bytes on)
        float *kw = reinterpret_cast<float *>(sm + L::KW) + (warp & 7) * C;    // lambda^0 .. lambda^63
        int c = 0, s = 0, round = 0;
        if (p.expire && blockIdx.x == 0)
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bar[L::DSH], 0, kTestWait));
        while (ok && walk.next(p, x, false)) {
            const float l2 = log2_decay(p, x.head);
            if (OUT) {
                __syncwarp();
                kw[lane] = exp2f(l2 * (float)lane);
                kw[lane + 32] = exp2f(l2 * (float)(lane + 32));
                __syncwarp();
            }
            for (int t = x.t0, t1 = x.t1; t < t1; t += C, ++c) {
                const int n = min(t1 - t, C);
                ok = warp_wait(&bar[L::LD + s], round);
                if (!ok) break;
                uint8_t *st = sm + s * L::stage;
                uint64_t *full = &bar[L::TF + 2 * s];
                if (++s == NS) { s = 0; ++round; }
                const float *w = kw + max(n - 1 - r0, 0);         // row r0 + RP i: lambda^{n - 1 - r0 - RP i}
                const int most = max(n - 1 - r0, 0) / RP;
                const uint8_t *kp = st + L::k + half * L::half + at0 + th0 * 4096;
                uint8_t *dst = sm + L::T + (c & (NB - 1)) * 3 * L::term + half * kTile + at0 + th0 * 4096;
                if (n < C)                                        // rows of the next sequence
                    for (int i = th0 * NR; i < th1 * NR; ++i)
                        if (r0 + RP * i >= n)
                            *reinterpret_cast<uint4 *>(st + L::v + half * kTile + at0 + i * RP * 128) = make_uint4(0, 0, 0, 0);
                // The loads of the next 32 tokens go before the stores of these: beside the MMAs' own reads a load
                // from shared memory takes some 200 cycles.
                uint4 kn[NR];
#pragma unroll
                for (int i = 0; i < NR; ++i) kn[i] = *reinterpret_cast<const uint4 *>(kp + i * RP * 128);
#pragma unroll 1
                for (int th = th0; th < th1; ++th) {              // 32 tokens at a time
                    uint4 k[NR];
                    float wi[NR];
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        k[i] = kn[i];
                        wi[i] = OUT ? w[-RP * min(th * NR + i, most)]
                                    : exp2f(l2 * (float)max(n - 1 - r0 - RP * (th * NR + i), 0));
                        if (r0 + RP * (th * NR + i) >= n) k[i] = make_uint4(0, 0, 0, 0);
                    }
                    if (OUT && th == 0)
#pragma unroll
                        for (int i = 0; i < NR; ++i) kn[i] = *reinterpret_cast<const uint4 *>(kp + (i + NR) * RP * 128);
                    if (c >= NB && !(ok = warp_wait(&bar[L::DSH + 2 * (c & (NB - 1)) + th], c / NB - 1))) break;
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        uint4 t1, t2, t3;
                        split3(k[i], wi[i], t1, t2, t3);
                        *reinterpret_cast<uint4 *>(dst + i * RP * 128) = t1;
                        *reinterpret_cast<uint4 *>(dst + i * RP * 128 + L::term) = t2;
                        *reinterpret_cast<uint4 *>(dst + i * RP * 128 + 2 * L::term) = t3;
                    }
                    dst += 4096;
                    ptx::fence_async_smem();
                    warp_arrive(full + th);
                }
                if (!ok) break;
            }
        }
    } else {                                                      // ---- the state: lane = value channel
        ptx::regs_inc<120>();
        if (early) ptx::pdl_wait();
        if ((warp & 3) * 32 < D) {
            constexpr int KC = D / 2;                                     // key channels k0 .. k0 + KC - 1 per thread
            const int q = warp & 3, k0 = ((warp - 12) >> 2) * KC;
            const int mine = k0 * dv + q * 32 + lane, rows = q * 32 + lane < dv ? dk - k0 : 0;
            const uint32_t at = tmem + ((uint32_t)q << 21);
            int c = 0;
            while (ok && walk.next(p, x, false)) {
                const float l2 = log2_decay(p, x.head);
                // (the real state's rows and columns only)
                const float *from = x.from + mine;
                const int have = x.from ? rows : 0;
                float s[KC];
#pragma unroll
                for (int e = 0; e < KC; ++e) {
                    s[e] = (FULL ? x.from != nullptr : e < have) ? *from : 0.f;
                    from += dv;
                }
                auto copy_out = [&](int e) {       // 16 channels as bf16 pairs
                    uint32_t u[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[i] = pack_bf16(s[e + 2 * i], s[e + 2 * i + 1]);
                    ptx::tmem_st8(at + TM_S + (k0 + e) / 2, u);
                };
                const int t0 = x.t0, t1 = x.t1;
                if (OUT && t1 > t0) {
                    if (c > 0) ok = warp_wait(&bar[L::QS], c - 1);
                    if (!ok) break;
                    ptx::tc_fence_after_sync();
#pragma unroll
                    for (int e = 0; e < KC; e += 16) copy_out(e);
                    ptx::tmem_st_wait();
                    ptx::tc_fence_before_sync();
                    warp_arrive(&bar[L::SREADY]);
                }
                for (int t = t0; t < t1; t += C, ++c) {
                    const bool more = OUT && t + C < t1;
                    const float f = exp2f(l2 * (float)min(t1 - t, C));
                    ok = warp_wait(&bar[L::DS + (c & (NB - 1))], c / NB);
                    if (!ok) break;
                    ptx::tc_fence_after_sync();
                    const uint32_t ds = at + tm_ds(c & (NB - 1)) + k0;
                    // 32 columns at a time: the next product may overwrite them as soon as the last have been read
#pragma unroll
                    for (int e = 0; e < KC; e += 32) {
                        float d[32];
                        ptx::tmem_ld16(ds + e, *reinterpret_cast<float(*)[16]>(d));
                        ptx::tmem_ld16(ds + e + 16, *reinterpret_cast<float(*)[16]>(d + 16));
                        ptx::tmem_ld_wait(d);
                        if (e + 32 == KC) {
                            ptx::tc_fence_before_sync();
                            warp_arrive(&bar[L::DSFREE + (c & (NB - 1))]);
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) s[e + i] = fmaf(f, s[e + i], d[i]);
                    }
                    if (more) {
                        ok = warp_wait(&bar[L::QS], c);
                        if (!ok) break;
                        ptx::tc_fence_after_sync();
#pragma unroll
                        for (int e = 0; e < KC; e += 16) copy_out(e);
                        ptx::tmem_st_wait();
                        ptx::tc_fence_before_sync();
                        warp_arrive(&bar[L::SREADY]);
                    }
                }
                if (!ok) break;
                if (x.to) {
                    float *to = x.to + mine;
#pragma unroll
                    for (int e = 0; e < KC; ++e) {
                        if (FULL || e < rows) *to = s[e];
                        to += dv;
                    }
                }
            }
        }
    }
    if (!ok) {
        s_abort = 1;
        report_status(p.g.status, KDA_ERR_DEVICE_TIMEOUT);
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

constexpr size_t kOrderAt = 256;
constexpr SegmentCost kCost{C, 4, 1.6f, 9.f};
size_t cells_at(int N) { return (kOrderAt + sizeof(int32_t) * (size_t)N + 1023) & ~size_t(1023); }

}  // namespace

size_t decay_prefill_tc_workspace(int64_t total, int N, int H, int dk, int dv) {
    const int len = decay_segment_tokens(total, N, H, sm_count(), kCost);
    if (len == 0 && (N == 1 || (int64_t)N * H <= sm_count())) return 0;
    return cells_at(N) + decay_cells_bytes(total, N, H, len, dk, dv);
}

template <int D, bool FULL>
static cudaError_t launch_tc(const DecayParams &d, int dk, int dv, void *workspace, size_t workspace_bytes, cudaStream_t st) {
    constexpr uint32_t kSmem = Lay<D, true>::bytes, kSmemState = Lay<D, false>::bytes;
    CUtensorMap mq, mk, mv, mo;
    const uint64_t T = (uint64_t)d.total, H = (uint64_t)d.H;
    auto map = [&](CUtensorMap *m, const void *base, int d, uint64_t row_bytes) {
        return FULL ? make_map_2d(m, base, true, T, H * d, row_bytes, C) : make_map_heads(m, base, T, H, d, row_bytes, C);
    };
    if (!map(&mq, d.q, dk, d.ldq * 2) || !map(&mk, d.k, dk, d.ldk * 2) || !map(&mv, d.v, dv, d.ldv * 2) ||
        !map(&mo, d.out, dv, H * dv * 2))
        return cudaErrorInvalidValue;
    const int sms = sm_count();
    Params p{{d.cu_seqlens, d.num_seqs, d.H, d.total, 0, 0, nullptr, d.status},
             d.log_decay,
             d.scale,
             d.init,
             d.fin,
             static_cast<__nv_bfloat16 *>(d.out),
             static_cast<const __nv_bfloat16 *>(d.v),
             d.ldv,
             nullptr,
             take_layers_expire(KDA_TESTING_DECAY),
             dk,
             dv};
    cudaError_t e = allow_smem<decay_chunk_kernel<D, true, FULL>>(kSmem);
    if (e == cudaSuccess) e = allow_smem<decay_chunk_kernel<D, false, FULL>>(kSmemState);
    if (e != cudaSuccess) return e;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const bool room = ws && workspace_bytes >= decay_prefill_tc_workspace(d.total, d.num_seqs, d.H, dk, dv);
    const int64_t chains = (int64_t)d.num_seqs * d.H;
    const int len = room ? decay_segment_tokens(d.total, d.num_seqs, d.H, sms, kCost) : 0;
    if (len) {
        p.g.len = len;
        p.g.cells = reinterpret_cast<float *>(ws + cells_at(d.num_seqs));
        p.g.cap = (int)(d.total / len) + d.num_seqs;
        const int64_t items = (int64_t)p.g.cap * d.H;
        const dim3 grid((unsigned)(items < sms ? items : sms));
        e = launch_dependent(decay_chunk_kernel<D, false, FULL>, grid, kThreads, kSmemState, st, 1, mq, mk, mv, mo, p);
        if (e != cudaSuccess) return e;
        if ((e = launch_decay_segments(p.g, d.log_decay, d.init, dk, dv, st)) != cudaSuccess) return e;
        return launch_dependent(decay_chunk_kernel<D, true, FULL>, grid, kThreads, kSmem, st, 1, mq, mk, mv, mo, p);
    }
    if (room && chains > sms && d.num_seqs > 1) {
        int32_t *order = reinterpret_cast<int32_t *>(ws + kOrderAt);
        if ((e = launch_schedule(d.cu_seqlens, d.num_seqs, order, reinterpret_cast<uint32_t *>(ws + 16),
                                 reinterpret_cast<uint32_t *>(ws), st)) != cudaSuccess)
            return e;
        p.order = order;
    }
    const dim3 grid((unsigned)(chains < sms ? chains : sms));
    return launch_dependent(decay_chunk_kernel<D, true, FULL>, grid, kThreads, kSmem, st, 1, mq, mk, mv, mo, p);
}

cudaError_t launch_decay_prefill_tc(const DecayParams &d, int dk, int dv, void *workspace, size_t workspace_bytes,
                                    cudaStream_t st) {
    if (dk == dv && dk == 128) return launch_tc<128, true>(d, dk, dv, workspace, workspace_bytes, st);
    if (dk == dv && dk == 64) return launch_tc<64, true>(d, dk, dv, workspace, workspace_bytes, st);
    return dk <= 64 && dv <= 64 ? launch_tc<64, false>(d, dk, dv, workspace, workspace_bytes, st)
                                : launch_tc<128, false>(d, dk, dv, workspace, workspace_bytes, st);
}

}  // namespace kda
