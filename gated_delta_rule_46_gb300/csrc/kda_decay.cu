// kda_decay.cu -- linear attention with one decay per head, lambda_h =
// exp(log_decay[h]):
//   S_t = lambda S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t.
// Over a chunk of n tokens from S_0 (i, j counted from 0):
//   o_i = scale (lambda^{i+1} S_0^T q_i + sum_{j<=i} lambda^{i-j} (q_i . k_j) v_j)
//   S_n = lambda^n S_0 + sum_j lambda^{n-1-j} k_j v_j^T
// Every power has a non-negative exponent, so nothing overflows for lambda <= 1.
#include "kda_decay.cuh"
#include "kda_tc_util.cuh"

namespace kda {

// ---------------------------------------------------------------------------
// Start states of the segments (see kda_decay.cuh), one float4 per thread.  The
// first segment's start state is copied too: its buffer may be the one that the
// last segment writes.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) decay_segments_kernel(const DecaySegs p, const float *__restrict__ log_decay,
                                                             const float *__restrict__ init, int state) {
    ptx::pdl_launch_dependents();
    const int n = (int)((unsigned)blockIdx.y / (unsigned)p.H), h = (int)blockIdx.y - n * p.H;
    int bos, eos, before = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        seq_range(p, i, bos, eos, false);
        before += segments_of(p, eos - bos);
    }
    seq_range(p, n, bos, eos, false);
    int segs = segments_of(p, eos - bos);
    if (before + segs > p.cap) segs = p.cap - before;
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, step = (int64_t)p.H * state;
    const float f = exp2f(decay_log2(log_decay, h) * (float)p.len);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (init) s = *reinterpret_cast<const float4 *>(init + (int64_t)blockIdx.y * state + at);
    float4 *cell = reinterpret_cast<float4 *>(p.cells + ((int64_t)before * p.H + h) * state + at);
    ptx::pdl_wait();        // the cells; the inputs were complete before the state pass let this kernel start
    // eight loads under way at a time: a store may not be overtaken by the loads after it
    constexpr int B = 8;
    for (int g0 = 0; g0 < segs; g0 += B) {
        float4 b[B];
#pragma unroll
        for (int i = 0; i < B; ++i)
            if (g0 + i + 1 < segs) b[i] = cell[(g0 + i) * (step / 4)];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            if (g0 + i >= segs) break;
            cell[(g0 + i) * (step / 4)] = s;
            if (g0 + i + 1 < segs) {
                s.x = fmaf(f, s.x, b[i].x); s.y = fmaf(f, s.y, b[i].y); s.z = fmaf(f, s.z, b[i].z); s.w = fmaf(f, s.w, b[i].w);
            }
        }
    }
}

cudaError_t launch_decay_segments(const DecaySegs &p, const float *log_decay, const float *init, int dk, int dv,
                                  cudaStream_t st) {
    return launch_dependent(decay_segments_kernel, dim3(dk * dv / 1024, (unsigned)(p.N * p.H)), 256, 0, st, 1, p, log_decay,
                            init, dk * dv);
}

// ---------------------------------------------------------------------------
// float32 chunk kernel (float32 inputs, and bf16 rows that no 16-byte copy can
// start on): one CTA per (sequence or segment, head, JB
// value channels), tokens in chunks of C = 32.  The value channels (columns of
// S) do not mix, so a chain splits exactly over them; the C x C products q . k
// are repeated per block.  Per chunk, all sums in float32 registers:
//   P      4 x 4 tiles per thread, the key channels split over 4 lanes
//   O      4 x 4 tiles, key channels (of S^T q) and tokens (of P v) split over
//          256 / (2 JB) thread groups and joined through shared memory
//   S      rows x 4 columns per thread, in registers; a copy in shared memory
//          for the next chunk's S^T q
// The next chunk's q, k and v are loaded into registers meanwhile.  Bound by shared
// memory (its pipe is 80 % busy, the issue slots 62 %, two CTAs per SM): a 16-byte load
// takes four of its cycles however much of it is shared between lanes, and eight of
// them feed 64 FMAs of a thread; tiles twice as large do not fit beside the state.
// 4096 tokens of 16 heads, d = 128, take 268 us in segments, 64 tokens of 2 heads, d =
// 32, 7.5 us.
// ---------------------------------------------------------------------------
struct DecaySimtParams {
    DecaySegs g;
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;
    const float *log_decay, *init;
    float *fin;
    void *out;
    float scale;
    int vec;                    // rows start on boundaries of four elements
};

template <typename T>
__device__ __forceinline__ float4 load4(const T *p, bool vec) {
    if (sizeof(T) == 4) {
        if (vec) return *reinterpret_cast<const float4 *>(p);
    } else if (vec) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        const float2 a = tc::bf2_to_f2(u.x), b = tc::bf2_to_f2(u.y);
        return make_float4(a.x, a.y, b.x, b.y);
    }
    return make_float4(to_f32(p[0]), to_f32(p[1]), to_f32(p[2]), to_f32(p[3]));
}

template <typename T>
__device__ __forceinline__ void store4(T *p, float4 x, bool vec) {
    if (sizeof(T) == 4 && vec) {
        *reinterpret_cast<float4 *>(p) = x;
    } else if (vec) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(tc::pack_bf16(x.x, x.y), tc::pack_bf16(x.z, x.w));
    } else {
        p[0] = from_f32<T>(x.x); p[1] = from_f32<T>(x.y); p[2] = from_f32<T>(x.z); p[3] = from_f32<T>(x.w);
    }
}

template <typename T, int DK, int JB, bool OUT>
__global__ void __launch_bounds__(256, 2) decay_simt_kernel(const DecaySimtParams p, int dv) {
    constexpr int C = 32, LD = DK + 4, LP = C + 4;
    constexpr int NK = C * DK / 1024, NV = C * JB / 1024;      // float4 per thread of q or k, of v
    constexpr int G = 256 / (2 * JB), RS = DK * JB / 1024;     // groups of O; rows of S per thread
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *sk = sq + C * LD, *sv = sk + C * LD;      // [C][LD] twice, [C][JB]
    float *sS = sv + C * JB, *sP = sS + DK * JB, *sR = sP + C * LP;   // [DK][JB], [C][LP], [G - 1][C][JB]
    float *pw = sR + (G - 1) * C * JB;                         // lambda^0 .. lambda^C

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, j0 = blockIdx.y * JB;
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int item = (int)((unsigned)blockIdx.x / (unsigned)p.g.H), h = (int)blockIdx.x - item * p.g.H;
    const int64_t state = (int64_t)DK * dv;
    int t0, t1;
    const float *from = nullptr;
    float *to = nullptr;
    if (p.g.len == 0) {
        seq_range(p.g, item, t0, t1, tid == 0 && blockIdx.y == 0);
        const int64_t at = ((int64_t)item * p.g.H + h) * state;
        if (p.init) from = p.init + at;
        if (p.fin) to = p.fin + at;
    } else {
        Segment sg;
        if (!find_segment(p.g, (unsigned)item, sg, tid == 0 && blockIdx.y == 0)) return;
        float *cell = p.g.cells + ((int64_t)item * p.g.H + h) * state;
        t0 = sg.t0;
        t1 = sg.t1;
        if (OUT) {
            from = cell;
            if (sg.last && p.fin) to = p.fin + ((int64_t)sg.n * p.g.H + h) * state;
        } else {
            if (sg.last) return;
            to = cell;
        }
    }
    const float l2 = decay_log2(p.log_decay, h);
    if (tid <= C) pw[tid] = exp2f(l2 * (float)tid);

    const int sc = (tid % (JB / 4)) * 4, sr = (tid / (JB / 4)) * RS;   // this thread's corner of S
    float s[RS][4];
#pragma unroll
    for (int r = 0; r < RS; ++r) {
        const float4 f = from ? *reinterpret_cast<const float4 *>(from + (int64_t)(sr + r) * dv + j0 + sc)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        s[r][0] = f.x; s[r][1] = f.y; s[r][2] = f.z; s[r][3] = f.w;
        if (OUT) *reinterpret_cast<float4 *>(sS + (sr + r) * JB + sc) = f;
    }
    const T *q = static_cast<const T *>(p.q) + (int64_t)h * DK, *k = static_cast<const T *>(p.k) + (int64_t)h * DK;
    const T *v = static_cast<const T *>(p.v) + (int64_t)h * dv + j0;
    float4 nq[NK], nk[NK], nv[NV];
    auto fetch = [&](int t) {          // rows past the end: zeros
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int r = (tid + i * 256) / (DK / 4), c = (tid + i * 256) % (DK / 4) * 4;
            const bool in = t + r < t1;
            if (OUT) nq[i] = in ? load4(q + (t + r) * p.ldq + c, p.vec) : z;
            nk[i] = in ? load4(k + (t + r) * p.ldk + c, p.vec) : z;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int r = (tid + i * 256) / (JB / 4), c = (tid + i * 256) % (JB / 4) * 4;
            nv[i] = t + r < t1 ? load4(v + (t + r) * p.ldv + c, p.vec) : z;
        }
    };
    // O: rows ti + 8 r, columns tj .. tj + 3, group g
    const int ti = lane & 7, ot = warp * 4 + (lane >> 3), tj = (ot % (JB / 4)) * 4, g = ot / (JB / 4);
    fetch(t0);
    for (int t = t0; t < t1; t += C) {
        const int n = min(t1 - t, C);
        __syncthreads();               // the chunk before is done with everything
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int r = (tid + i * 256) / (DK / 4), c = (tid + i * 256) % (DK / 4) * 4;
            if (OUT) *reinterpret_cast<float4 *>(sq + r * LD + c) = nq[i];
            *reinterpret_cast<float4 *>(sk + r * LD + c) = nk[i];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) *reinterpret_cast<float4 *>(sv + (tid + i * 256) * 4) = nv[i];
        __syncthreads();
        if (t + C < t1) fetch(t + C);
        if (OUT) {
            float a[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) a[i] = 0.f;
            {   // P: rows ti + 8 r, columns warp + 8 c; lane / 8 takes every fourth group of four key channels
                const int ks = (lane >> 3) * 4;
#pragma unroll 2
                for (int c = ks; c < DK; c += 16) {
                    float x[4][4], y[4][4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        tc::ld4(sq + (ti + 8 * r) * LD + c, x[r]);
                        tc::ld4(sk + (warp + 8 * r) * LD + c, y[r]);
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
#pragma unroll
                            for (int e = 0; e < 4; ++e) a[r * 4 + u] = fmaf(x[r][e], y[u][e], a[r * 4 + u]);
                }
                // the four lanes of a tile join their sums: each ends with one row of it
#pragma unroll
                for (int m = 8, bit = 16; m >= 4; m >>= 1, bit >>= 1) {
                    const bool up = lane & bit;
#pragma unroll
                    for (int i = 0; i < m; ++i) {
                        const float keep = up ? a[i + m] : a[i], send = up ? a[i] : a[i + m];
                        a[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
                    }
                }
                const int i = ti + 8 * ((lane & 16 ? 2 : 0) + (lane & 8 ? 1 : 0));
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int j = warp + 8 * u;
                    sP[i * LP + j] = j <= i ? a[u] * pw[i - j] : 0.f;
                }
            }
            float o[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int u = 0; u < 4; ++u) o[r][u] = 0.f;
#pragma unroll 2
            for (int c = g * (DK / G); c < (g + 1) * (DK / G); c += 4) {     // S^T q
                float x[4][4], y[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    tc::ld4(sq + (ti + 8 * r) * LD + c, x[r]);
                    tc::ld4(sS + (c + r) * JB + tj, y[r]);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int u = 0; u < 4; ++u) o[r][u] = fmaf(x[r][e], y[e][u], o[r][u]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int u = 0; u < 4; ++u) o[r][u] *= pw[ti + 8 * r + 1];
            __syncthreads();           // P
#pragma unroll 2
            for (int j = g * (C / G); j < (g + 1) * (C / G); j += 4) {
                float x[4][4], y[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    tc::ld4(sP + (ti + 8 * r) * LP + j, x[r]);
                    tc::ld4(sv + (j + r) * JB + tj, y[r]);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j + e <= ti + 8 * r)       // a later token's infinity must not meet P's zero
#pragma unroll
                            for (int u = 0; u < 4; ++u) o[r][u] = fmaf(x[r][e], y[e][u], o[r][u]);
            }
            if (g > 0)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *reinterpret_cast<float4 *>(sR + ((g - 1) * C + ti + 8 * r) * JB + tj) =
                        make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
            __syncthreads();           // the groups' sums; S may change
            if (g == 0)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = ti + 8 * r;
                    if (i >= n) continue;
#pragma unroll
                    for (int e = 1; e < G; ++e) {
                        float y[4];
                        tc::ld4(sR + ((e - 1) * C + i) * JB + tj, y);
#pragma unroll
                        for (int u = 0; u < 4; ++u) o[r][u] += y[u];
                    }
                    store4(static_cast<T *>(p.out) + ((int64_t)(t + i) * p.g.H + h) * dv + j0 + tj,
                           make_float4(o[r][0] * p.scale, o[r][1] * p.scale, o[r][2] * p.scale, o[r][3] * p.scale), p.vec);
                }
        }
        const float f = pw[n];
#pragma unroll
        for (int r = 0; r < RS; ++r)
#pragma unroll
            for (int u = 0; u < 4; ++u) s[r][u] *= f;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float w = pw[n - 1 - i];
            float y[4], x[RS];
            tc::ld4(sv + i * JB + sc, y);
#pragma unroll
            for (int u = 0; u < 4; ++u) y[u] *= w;
            if constexpr (RS >= 4) {
#pragma unroll
                for (int r = 0; r < RS; r += 4) tc::ld4(sk + i * LD + sr + r, x + r);
            } else {
#pragma unroll
                for (int r = 0; r < RS; ++r) x[r] = sk[i * LD + sr + r];
            }
#pragma unroll
            for (int r = 0; r < RS; ++r)
#pragma unroll
                for (int u = 0; u < 4; ++u) s[r][u] = fmaf(x[r], y[u], s[r][u]);
        }
        if (OUT)
#pragma unroll
            for (int r = 0; r < RS; ++r)
                *reinterpret_cast<float4 *>(sS + (sr + r) * JB + sc) = make_float4(s[r][0], s[r][1], s[r][2], s[r][3]);
    }
    if (to)
#pragma unroll
        for (int r = 0; r < RS; ++r)
            *reinterpret_cast<float4 *>(to + (int64_t)(sr + r) * dv + j0 + sc) = make_float4(s[r][0], s[r][1], s[r][2], s[r][3]);
}

constexpr int kSimtChunk = 32;
constexpr SegmentCost kSimtCost{kSimtChunk, 2, 2.25f, 2.f};
// CTAs that run at a time (two per SM), by blocks of up to 64 value channels
static int simt_slots(int dv) { return 2 * sm_count() / (dv > 64 ? 2 : 1); }

size_t decay_prefill_simt_workspace(int64_t total, int N, int H, int dk, int dv) {
    return decay_cells_bytes(total, N, H, decay_segment_tokens(total, N, H, simt_slots(dv), kSimtCost), dk, dv);
}

template <typename T, int DK, int JB>
static cudaError_t decay_simt(DecaySimtParams &p, int dv, int64_t chains, cudaStream_t st) {
    constexpr int C = kSimtChunk, G = 256 / (2 * JB);
    const size_t smem = sizeof(float) * (2 * C * (DK + 4) + C * JB + DK * JB + C * (C + 4) + (G - 1) * C * JB + C + 1);
    cudaError_t e = allow_smem<decay_simt_kernel<T, DK, JB, true>>((uint32_t)smem);
    if (e != cudaSuccess) return e;
    dim3 grid((unsigned)chains, dv / JB);
    if (p.g.len) {
        e = allow_smem<decay_simt_kernel<T, DK, JB, false>>((uint32_t)smem);
        if (e != cudaSuccess) return e;
        grid.x = (unsigned)((int64_t)p.g.cap * p.g.H);
        if ((e = launch_dependent(decay_simt_kernel<T, DK, JB, false>, grid, 256, smem, st, 1, p, dv)) != cudaSuccess) return e;
        if ((e = launch_decay_segments(p.g, p.log_decay, p.init, DK, dv, st)) != cudaSuccess) return e;
    }
    return launch_dependent(decay_simt_kernel<T, DK, JB, true>, grid, 256, smem, st, 1, p, dv);
}

template <typename T>
static cudaError_t decay_simt_dims(DecaySimtParams &p, int dk, int dv, int64_t chains, cudaStream_t st) {
    if (dv == 32) {
        switch (dk) {
            case 32: return decay_simt<T, 32, 32>(p, dv, chains, st);
            case 64: return decay_simt<T, 64, 32>(p, dv, chains, st);
            case 128: return decay_simt<T, 128, 32>(p, dv, chains, st);
        }
    }
    switch (dk) {
        case 32: return decay_simt<T, 32, 64>(p, dv, chains, st);
        case 64: return decay_simt<T, 64, 64>(p, dv, chains, st);
        case 128: return decay_simt<T, 128, 64>(p, dv, chains, st);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_decay_prefill_simt(const DecayParams &d, int dk, int dv, bool bf16, void *workspace,
                                      size_t workspace_bytes, cudaStream_t st) {
    const int64_t e = bf16 ? 2 : 4;
    auto four = [&](const void *x, int64_t ld) { return reinterpret_cast<uintptr_t>(x) % (4 * e) == 0 && ld % 4 == 0; };
    DecaySimtParams p{{d.cu_seqlens, d.num_seqs, d.H, d.total, 0, 0, nullptr, d.status}, d.q, d.k, d.v, d.ldq, d.ldk, d.ldv,
                      d.log_decay, d.init, d.fin, d.out, d.scale,
                      four(d.q, d.ldq) && four(d.k, d.ldk) && four(d.v, d.ldv) && four(d.out, 4)};
    const int len = decay_segment_tokens(d.total, d.num_seqs, d.H, simt_slots(dv), kSimtCost);
    if (len && workspace && workspace_bytes >= decay_prefill_simt_workspace(d.total, d.num_seqs, d.H, dk, dv)) {
        p.g.len = len;
        p.g.cap = (int)(d.total / len) + d.num_seqs;
        p.g.cells = static_cast<float *>(workspace);
    }
    const int64_t chains = (int64_t)d.num_seqs * d.H;
    return bf16 ? decay_simt_dims<__nv_bfloat16>(p, dk, dv, chains, st) : decay_simt_dims<float>(p, dk, dv, chains, st);
}

// ---------------------------------------------------------------------------
// One new token per sequence: one CTA per (sequence, head), the state read once
// with 16-byte loads, updated, reduced over its rows (S^T q) and written back.
// The state's 8 d^2 bytes are all of the traffic: 256 rows of 32 heads, d = 128,
// take 158 us (6.85 TB/s, the rate of a plain copy); 4 rows of 2 heads, d = 64, 1.9 us.
// ---------------------------------------------------------------------------
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(256) decay_decode_kernel(const DecayStepParams p) {
    constexpr int F = DV / 4, RPP = 256 / F, PASSES = DK / RPP;
    static_assert(DK % RPP == 0, "decode tiling");
    __shared__ float s_k[DK], s_q[DK];
    __shared__ float s_red[RPP][DV + 4];
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int nh = blockIdx.x, n = nh / p.H, h = nh % p.H, tid = threadIdx.x;
    T *out = static_cast<T *>(p.out) + (int64_t)nh * DV;
    int slot = p.slots ? p.slots[n] : n;
    if (slot >= p.pool_size) {   // bad id: reported, row treated as padding
        if (tid == 0) report_status(p.status, KDA_ERR_INVALID_ARG);
        slot = -1;
    }
    if (slot < 0) {
        if (tid < DV) out[tid] = from_f32<T>(0.f);
        return;
    }
    const int col4 = tid % F, r0 = tid / F;
    float4 *S4 = reinterpret_cast<float4 *>(p.pool + ((int64_t)slot * p.H + h) * DK * DV);
    float4 s[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) s[i] = S4[(r0 + i * RPP) * F + col4];
    const T *v = static_cast<const T *>(p.v) + (int64_t)n * p.ldv + (int64_t)h * DV + col4 * 4;
    const float v0 = to_f32(v[0]), v1 = to_f32(v[1]), v2 = to_f32(v[2]), v3 = to_f32(v[3]);
    if (tid < DK) {
        s_k[tid] = to_f32(static_cast<const T *>(p.k)[(int64_t)n * p.ldk + (int64_t)h * DK + tid]);
        s_q[tid] = to_f32(static_cast<const T *>(p.q)[(int64_t)n * p.ldq + (int64_t)h * DK + tid]);
    }
    const float lam = exp2f(p.log_decay[h] * kLog2E);
    __syncthreads();
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int c = r0 + i * RPP;
        const float kc = s_k[c], qc = s_q[c];
        s[i].x = fmaf(kc, v0, lam * s[i].x); s[i].y = fmaf(kc, v1, lam * s[i].y);
        s[i].z = fmaf(kc, v2, lam * s[i].z); s[i].w = fmaf(kc, v3, lam * s[i].w);
        S4[c * F + col4] = s[i];
        a.x = fmaf(qc, s[i].x, a.x); a.y = fmaf(qc, s[i].y, a.y);
        a.z = fmaf(qc, s[i].z, a.z); a.w = fmaf(qc, s[i].w, a.w);
    }
    *reinterpret_cast<float4 *>(&s_red[r0][col4 * 4]) = a;
    __syncthreads();
    if (tid < DV) {
        float o = 0.f;
#pragma unroll 8
        for (int r = 0; r < RPP; ++r) o += s_red[r][tid];
        out[tid] = from_f32<T>(o * p.scale);
    }
}

template <typename T>
static cudaError_t decay_decode_dispatch(const DecayStepParams &p, int dk, int dv, cudaStream_t st) {
    const dim3 grid((unsigned)((int64_t)p.N * p.H));
#define KDA_DECAY_CASE(DK_, DV_) \
    if (dk == DK_ && dv == DV_) return launch_dependent(decay_decode_kernel<T, DK_, DV_>, grid, 256, 0, st, 1, p);
    KDA_DECAY_CASE(32, 32) KDA_DECAY_CASE(32, 64) KDA_DECAY_CASE(32, 128)
    KDA_DECAY_CASE(64, 32) KDA_DECAY_CASE(64, 64) KDA_DECAY_CASE(64, 128)
    KDA_DECAY_CASE(128, 32) KDA_DECAY_CASE(128, 64) KDA_DECAY_CASE(128, 128)
#undef KDA_DECAY_CASE
    return cudaErrorInvalidValue;
}

cudaError_t launch_decay_decode(const DecayStepParams &p, int dk, int dv, bool bf16, cudaStream_t st) {
    return bf16 ? decay_decode_dispatch<__nv_bfloat16>(p, dk, dv, st) : decay_decode_dispatch<float>(p, dk, dv, st);
}

}  // namespace kda
