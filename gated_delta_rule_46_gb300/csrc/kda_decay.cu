// kda_decay.cu -- linear attention with one decay per head, lambda_h =
// exp(log_decay[h]):
//   S_t = lambda S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t.
// Over a chunk of n tokens from S_0 (i, j counted from 0):
//   o_i = scale (lambda^{i+1} S_0^T q_i + sum_{j<=i} lambda^{i-j} (q_i . k_j) v_j)
//   S_n = lambda^n S_0 + sum_j lambda^{n-1-j} k_j v_j^T
// Every power has a non-negative exponent, so nothing overflows for lambda <= 1.
#include "kda_layers.cuh"
#include "kda_tc_util.cuh"

namespace kda {

// ---------------------------------------------------------------------------
// float32 chunk kernel: one CTA per (sequence, head, JB value channels), tokens
// in chunks of C.  The value channels (columns of S) do not mix, so a chain
// splits exactly over them; the C x C products q . k are repeated per block.
// ---------------------------------------------------------------------------
template <typename T, int DK>
__global__ void __launch_bounds__(256) decay_prefill_simt_kernel(const DecayParams p, int dv) {
    constexpr int C = 32, JB = 32, LD = DK + 4;
    extern __shared__ float sm[];
    float *sq = sm, *sk = sq + C * LD, *sS = sk + C * LD;        // [C][LD], [C][LD], [DK][JB]
    float *sv = sS + DK * JB, *sw = sv + C * JB, *sP = sw + C * JB;   // [C][JB] v and w v, [C][C + 1]
    float *pw = sP + C * (C + 1);                                 // lambda^0 .. lambda^C

    const int nh = blockIdx.x, seq = nh / p.H, h = nh % p.H, j0 = blockIdx.y * JB, tid = threadIdx.x;
    const int col = tid & 31, wy = tid >> 5;
    int64_t bos, eos;
    tc::seq_bounds(p.cu_seqlens, seq, p.total, p.status, tid + blockIdx.y, bos, eos);
    const float l2 = p.log_decay[h] * kLog2E;
    if (tid <= C) pw[tid] = decay_pow(l2, tid);
    const int64_t sbase = (int64_t)nh * DK * dv + j0;
#pragma unroll 4
    for (int c = wy; c < DK; c += 8) sS[c * JB + col] = p.init ? p.init[sbase + (int64_t)c * dv + col] : 0.f;

    const T *q = static_cast<const T *>(p.q), *k = static_cast<const T *>(p.k), *v = static_cast<const T *>(p.v);
    T *out = static_cast<T *>(p.out);
    for (int64_t t0 = bos; t0 < eos; t0 += C) {
        const int n = (int)(eos - t0 < C ? eos - t0 : C);
        __syncthreads();
        for (int i = tid; i < C * DK; i += 256) {
            const int t = i / DK, c = i % DK;
            sq[t * LD + c] = t < n ? to_f32(q[(t0 + t) * p.ldq + (int64_t)h * DK + c]) : 0.f;
            sk[t * LD + c] = t < n ? to_f32(k[(t0 + t) * p.ldk + (int64_t)h * DK + c]) : 0.f;
        }
        for (int t = wy; t < C; t += 8) {
            const float x = t < n ? to_f32(v[(t0 + t) * p.ldv + (int64_t)h * dv + j0 + col]) : 0.f;
            sv[t * JB + col] = x;
            sw[t * JB + col] = t < n ? x * pw[n - 1 - t] : 0.f;
        }
        __syncthreads();
        {   // P_ij = lambda^{i-j} q_i . k_j, a 2 x 2 block per thread
            const int i0 = (tid >> 4) * 2, jj = (tid & 15) * 2;
            float a00 = 0.f, a01 = 0.f, a10 = 0.f, a11 = 0.f;
#pragma unroll 4
            for (int c = 0; c < DK; c += 4) {
                float x0[4], x1[4], y0[4], y1[4];
                tc::ld4(sq + i0 * LD + c, x0); tc::ld4(sq + (i0 + 1) * LD + c, x1);
                tc::ld4(sk + jj * LD + c, y0); tc::ld4(sk + (jj + 1) * LD + c, y1);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    a00 = fmaf(x0[e], y0[e], a00); a01 = fmaf(x0[e], y1[e], a01);
                    a10 = fmaf(x1[e], y0[e], a10); a11 = fmaf(x1[e], y1[e], a11);
                }
            }
            auto put = [&](int i, int j, float a) { sP[i * (C + 1) + j] = j <= i ? a * pw[i - j] : 0.f; };
            put(i0, jj, a00); put(i0, jj + 1, a01); put(i0 + 1, jj, a10); put(i0 + 1, jj + 1, a11);
        }
        float o[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {   // lambda^{i+1} S_0^T q_i
            const int i = wy * 4 + r;
            float a = 0.f;
#pragma unroll 8
            for (int c = 0; c < DK; ++c) a = fmaf(sq[i * LD + c], sS[c * JB + col], a);
            o[r] = a * pw[i + 1];
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = wy * 4 + r;
            // the sum ends at j = i: a later token's infinity must not meet a zero here
            for (int j = 0; j <= i; ++j) o[r] = fmaf(sP[i * (C + 1) + j], sv[j * JB + col], o[r]);
            if (i < n) out[((t0 + i) * p.H + h) * dv + j0 + col] = from_f32<T>(o[r] * p.scale);
        }
#pragma unroll 4
        for (int c = wy; c < DK; c += 8) {
            float a = sS[c * JB + col] * pw[n];
#pragma unroll 8
            for (int t = 0; t < C; ++t) a = fmaf(sk[t * LD + c], sw[t * JB + col], a);
            sS[c * JB + col] = a;
        }
    }
    if (p.fin) {
#pragma unroll 4
        for (int c = wy; c < DK; c += 8) p.fin[sbase + (int64_t)c * dv + col] = sS[c * JB + col];
    }
}

template <typename T, int DK>
static cudaError_t decay_simt(const DecayParams &p, int dv, cudaStream_t st) {
    constexpr int C = 32, JB = 32;
    const size_t smem = sizeof(float) * (2 * C * (DK + 4) + DK * JB + 2 * C * JB + C * (C + 1) + C + 1);
    const cudaError_t e = cudaFuncSetAttribute(decay_prefill_simt_kernel<T, DK>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    decay_prefill_simt_kernel<T, DK><<<dim3((unsigned)(p.num_seqs * p.H), dv / JB), 256, smem, st>>>(p, dv);
    return cudaGetLastError();
}

cudaError_t launch_decay_prefill_simt(const DecayParams &p, int dk, int dv, bool bf16, cudaStream_t st) {
    switch (dk) {
        case 32: return bf16 ? decay_simt<__nv_bfloat16, 32>(p, dv, st) : decay_simt<float, 32>(p, dv, st);
        case 64: return bf16 ? decay_simt<__nv_bfloat16, 64>(p, dv, st) : decay_simt<float, 64>(p, dv, st);
        case 128: return bf16 ? decay_simt<__nv_bfloat16, 128>(p, dv, st) : decay_simt<float, 128>(p, dv, st);
    }
    return cudaErrorInvalidValue;
}

// ---------------------------------------------------------------------------
// One new token per sequence: one CTA per (sequence, head), the state read once
// with 16-byte loads, updated, reduced over its rows (S^T q) and written back.
// ---------------------------------------------------------------------------
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(256) decay_decode_kernel(const DecayStepParams p) {
    constexpr int F = DV / 4, RPP = 256 / F, PASSES = DK / RPP;
    static_assert(DK % RPP == 0, "decode tiling");
    __shared__ float s_k[DK], s_q[DK];
    __shared__ float s_red[RPP][DV + 4];
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
    const float lam = decay_pow(p.log_decay[h] * kLog2E, 1);
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
    const unsigned grid = (unsigned)((int64_t)p.N * p.H);
#define KDA_DECAY_CASE(DK_, DV_) \
    if (dk == DK_ && dv == DV_) decay_decode_kernel<T, DK_, DV_><<<grid, 256, 0, st>>>(p);
    KDA_DECAY_CASE(32, 32) KDA_DECAY_CASE(32, 64) KDA_DECAY_CASE(32, 128)
    KDA_DECAY_CASE(64, 32) KDA_DECAY_CASE(64, 64) KDA_DECAY_CASE(64, 128)
    KDA_DECAY_CASE(128, 32) KDA_DECAY_CASE(128, 64) KDA_DECAY_CASE(128, 128)
#undef KDA_DECAY_CASE
    return cudaGetLastError();
}

cudaError_t launch_decay_decode(const DecayStepParams &p, int dk, int dv, bool bf16, cudaStream_t st) {
    return bf16 ? decay_decode_dispatch<__nv_bfloat16>(p, dk, dv, st) : decay_decode_dispatch<float>(p, dk, dv, st);
}

}  // namespace kda
