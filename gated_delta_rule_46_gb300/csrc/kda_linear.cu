// kda_linear.cu -- out = act(x w^T + bias) + residual.
#include "kda_layers.cuh"

namespace kda {

// The activation on the float32 sum.  sigmoid and silu are written with
// exp(-y): it overflows to +inf for very negative y, where both then give 0.
__device__ __forceinline__ float activate(float y, int act) {
    switch (act) {
        case KDA_ACT_RELU: return y > 0.f ? y : (y != y ? y : 0.f);
        case KDA_ACT_GELU: return 0.5f * y * (1.f + erff(y * 0.70710678118654752f));
        case KDA_ACT_SILU: return y / (1.f + expf(-y));
        case KDA_ACT_SIGMOID: return 1.f / (1.f + expf(-y));
        default: return y;
    }
}

// CUDA-core form for rows that no TMA copy can start on (K not a multiple of 8
// or misaligned rows): a 64 x 64 tile per CTA, K in steps of 16, 4 x 4 sums
// per thread in float32.
__global__ void __launch_bounds__(256) linear_simt_kernel(const LinearParams p) {
    constexpr int BK = 16;
    __shared__ float xs[BK][68], ws[BK][68];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < p.K; k0 += BK) {
        for (int i = tid; i < 64 * BK; i += 256) {
            const int r = i / BK, c = i % BK;
            const int64_t kk = k0 + c;
            xs[c][r] = (m0 + r < p.M && kk < p.K) ? to_f32(p.x[(m0 + r) * p.ldx + kk]) : 0.f;
            ws[c][r] = (n0 + r < p.N && kk < p.K) ? to_f32(p.w[(n0 + r) * p.K + kk]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < BK; ++c) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) { a[i] = xs[c][ty * 4 + i]; b[i] = ws[c][tx * 4 + i]; }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m >= p.M || n >= p.N) continue;
            const float y = activate(acc[i][j] + (p.bias ? p.bias[n] : 0.f), p.act);
            const int64_t at = m * p.N + n;
            if (p.out_f32) {
                const float r = p.residual ? static_cast<const float *>(p.residual)[at] : 0.f;
                static_cast<float *>(p.out)[at] = y + r;
            } else {
                const float r = p.residual ? to_f32(static_cast<const __nv_bfloat16 *>(p.residual)[at]) : 0.f;
                static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(y + r);
            }
        }
}

cudaError_t launch_linear_simt(const LinearParams &p, cudaStream_t st) {
    const int64_t gx = (p.N + 63) / 64;
    // M in slices of 65,535 row tiles (the grid's limit in y)
    for (int64_t m0 = 0; m0 < p.M; m0 += 65535 * 64) {
        LinearParams s = p;
        s.M = p.M - m0 < 65535 * 64 ? p.M - m0 : 65535 * 64;
        s.x = p.x + m0 * p.ldx;
        const int64_t off = m0 * p.N * (p.out_f32 ? 4 : 2);
        s.out = static_cast<uint8_t *>(p.out) + off;
        if (p.residual) s.residual = static_cast<const uint8_t *>(p.residual) + off;
        linear_simt_kernel<<<dim3((unsigned)gx, (unsigned)((s.M + 63) / 64)), 256, 0, st>>>(s);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace kda
