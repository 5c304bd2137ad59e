// kda_paged_q8.cu -- new tokens into a paged key-value cache in 8 bits.
//
// A block of B tokens of one head has a scale s and e4m3 codes c; a value is c s.
// Scales are powers of two, the least with amax <= 448 s: the codes have four
// significant bits whatever s is, so nothing is lost by it but the chance of a
// finer last step below 2^-6 s, and every product and quotient with s is exact:
// a code is the value rounded once, and codes whose scale doubles stay as they
// are in value unless they fall below 2^-6 of the new one.
//
// A block that holds earlier tokens keeps its scale unless the new ones need a
// larger one; then its earlier codes are rounded again, to the new scale.
#include "kda_layers.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace {

constexpr int WARPS = 8, ROWS = 16;               // of a CTA; tokens of a block that one warp works on

constexpr float kLeast = 0x1p-126f, kMost = 0x1p126f;                      // scales that an earlier call can have left

// Eight values of a row as they are loaded.
template <typename T, bool VEC>
struct Row8 {
    uint4 u[sizeof(T) / 2] = {};
    __device__ void load(const T *p) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = reinterpret_cast<const uint4 *>(p)[i];
        } else if constexpr (sizeof(T) == 4) {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(p);
            u[0] = make_uint4(w[0], w[1], w[2], w[3]);
            u[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
            u[0] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
        }
    }
    // The largest magnitude's bits, of two values in halves for bf16, and as a float's at the end: what is not finite is
    // larger than what is.  (Two instructions for two bf16, where a comparison with infinity takes six.)
    __device__ void top(uint32_t &m) const {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(u);
#pragma unroll
        for (int i = 0; i < 2 * (int)sizeof(T); ++i) m = sizeof(T) == 4 ? max(m, w[i] & 0x7fffffffu) : __vmaxu2(m, w[i] & 0x7fff7fffu);
    }
    static __device__ uint32_t joined(uint32_t m) { return sizeof(T) == 4 ? m : max(m << 16, m & 0xffff0000u); }
    __device__ void get(float (&x)[8]) const {
        if constexpr (sizeof(T) == 4) {
            const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
        } else {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
};

// ODD: infinities, which a saturating conversion takes for large numbers, become NaN.
template <bool ODD>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = x[2 * i] * inv, b = x[2 * i + 1] * inv;
        if constexpr (ODD) {
            if (!(fabsf(x[2 * i]) < INFINITY)) a = NAN;
            if (!(fabsf(x[2 * i + 1]) < INFINITY)) b = NAN;
        }
        c[i] = f2_to_e4m3x2(a, b);
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
__device__ __forceinline__ void decode8(uint2 u, float (&x)[8]) {
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = e4m3x2_to_f2((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// Tokens and blocks of sequence i; what is malformed has none.
struct Seq {
    int t0, start, n, blocks;
};
__device__ __forceinline__ Seq sequence(const AppendQ8Params &p, int i) {
    Seq s{i, p.start[i], 1, 0};
    bool bad = s.start < 0;
    if (p.cu_seqlens) {
        s.t0 = p.cu_seqlens[i];
        const int end = p.cu_seqlens[i + 1];
        s.n = end - s.t0;
        bad = bad || s.t0 < 0 || end < s.t0 || end > p.total;
    }
    // (positions past 2^31 are past any table)
    if (bad || (int64_t)s.start + s.n > 0x7fffffff) s.n = bad ? 0 : 0x7fffffff - s.start;
    if (s.n > 0) s.blocks = ((s.start + s.n - 1) >> p.block_shift) - (s.start >> p.block_shift) + 1;
    return s;
}

// One unit is a block of a sequence, a head, and keys or values, or both where the registers hold them; the units of all
// sequences in order are dealt out evenly.
// B / 16 warps share a unit, 16 tokens each; the one token of a sequence without cu_seqlens is one warp's.
//
// Instructions bound it next to HBM: what a value costs is kept to two and a half (its share of a maximum over the bits of
// two values at a time, half a multiplication's and a conversion's), and registers to what lets as many CTAs run as these
// need to overlap: 131k tokens of 8 heads of 128 channels take 128 us (6.4 TB/s) with three CTAs of an SM, 145 with two,
// 151 with four; float32 105 with two, 133 with three.  Keys and values in one unit: 73 us instead of 79 with 64 channels,
// 43 instead of 57 with 32.  Copying a warp's next units to shared memory ahead gains nothing.
template <typename T, int D>
constexpr int kBoth = ROWS * D * sizeof(T) > 2048 ? 1 : 2;                // keys, or keys and values, of a unit
template <typename T, int D>
constexpr int kCtas = ROWS * D * sizeof(T) > 4096 ? 2 : ROWS * D * sizeof(T) >= 2048 ? 3 : 4;

template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(WARPS * 32, kCtas<T, D>) paged_append_q8_kernel(const AppendQ8Params p) {
    constexpr int LPR = D / 8, RPS = 32 / LPR, STEPS = ROWS / RPS;        // lanes per row, rows per step, steps
    __shared__ int64_t s_sum[WARPS + 1];
    __shared__ int s_n;
    constexpr int KV = kBoth<T, D>;
    __shared__ float s_max[2][KV][WARPS];
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tasks = 2 / KV * p.Hkv, share = p.cu_seqlens ? (1 << p.block_shift) / ROWS : 1;      // warps of a unit
    const int per = WARPS / share, mine = warp / share, part = warp % share;

    // ---- this CTA's units [u0, u1), the sequence in which they start and the blocks before it
    int64_t total = p.num_seqs, cum = 0;
    int n = 0;
    if (p.cu_seqlens) {
        const int each = (p.num_seqs + WARPS * 32 - 1) / (WARPS * 32);
        const int n0 = min(p.num_seqs, tid * each), n1 = min(p.num_seqs, n0 + each);
        int64_t x = 0;
        for (int i = n0; i < n1; ++i) x += sequence(p, i).blocks;
        const int64_t own = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_sum[warp] = x;
        if (tid == 0) s_n = p.num_seqs;
        __syncthreads();
        int64_t before = 0;
        total = 0;
        for (int i = 0; i < WARPS; ++i) {
            if (i < warp) before += s_sum[i];
            total += s_sum[i];
        }
        const int64_t b0 = (int64_t)blockIdx.x * (total * tasks) / gridDim.x / tasks;
        int64_t c = before + x - own;
        if (b0 >= c && b0 < c + own)
            for (int i = n0; i < n1; ++i) {
                const int b = sequence(p, i).blocks;
                if (b0 < c + b) {
                    s_n = i;
                    s_sum[WARPS] = c;
                    break;
                }
                c += b;
            }
        __syncthreads();
        n = s_n;
        cum = s_sum[WARPS];
        if (blockIdx.x == 0) {
            for (int i = tid; i < p.num_seqs; i += WARPS * 32) {
                const int t0 = p.cu_seqlens[i], end = p.cu_seqlens[i + 1];
                if (p.start[i] < 0 || t0 < 0 || end < t0 || end > p.total || (int64_t)p.start[i] + (end - t0) > 0x7fffffff)
                    report_status(p.status, KDA_ERR_INVALID_ARG);
            }
            if (tid == 0 && (p.cu_seqlens[0] != 0 || p.cu_seqlens[p.num_seqs] != p.total))
                report_status(p.status, KDA_ERR_INVALID_ARG);
        }
    }
    const int64_t units = total * tasks;
    const int64_t u0 = (int64_t)blockIdx.x * units / gridDim.x, u1 = (int64_t)(blockIdx.x + 1) * units / gridDim.x;
    if (u0 >= u1) return;
    int64_t blk = (u0 + mine) / tasks;                // block of all sequences, and the unit within it
    int task = (int)(u0 + mine - blk * tasks);
    if (!p.cu_seqlens) n = (int)blk, cum = blk;
    Seq s{};
    if (blk < total) s = sequence(p, n);
    if (!p.cu_seqlens) s.blocks = 1;                  // (of a malformed one too: a sequence is its own block here)

    const int lane_row = lane / LPR, ch = (lane % LPR) * 8;
    const int ps = 1 << p.page_shift;
    for (int64_t u = u0, round = 0; u < u1; u += per, ++round) {
        // ---- the block: rows [from, to) of it are new, [0, from) hold earlier tokens
        int from = 0, to = 0;
        int64_t at = 0;                               // its first row in the cache
        float was[KV] = {};                           // scales before
        int row0 = part * ROWS + lane_row;            // this lane's first row
        const int h = task >= p.Hkv ? task - p.Hkv : task;
        auto value = [&](int kv) { return KV == 2 ? kv == 1 : task >= p.Hkv; };
        Row8<T, VEC> x[KV][STEPS];
        if (u + mine < u1) {
            while (blk >= cum + s.blocks) {
                cum += s.blocks;
                s = sequence(p, ++n);
                if (!p.cu_seqlens) s.blocks = 1;
            }
            const int pos = ((s.start >> p.block_shift) + (int)(blk - cum)) << p.block_shift;
            const int page_i = pos >> p.page_shift;
            const int page = s.n > 0 && page_i < p.max_pages ? p.table[(int64_t)n * p.max_pages + page_i] : -1;
            if (page >= 0 && page < p.num_pages) {
                from = max(s.start - pos, 0);
                to = min(1 << p.block_shift, s.start + s.n - pos);
                if (!p.cu_seqlens) row0 = (from & ~(ROWS - 1)) + lane_row;
                at = (((int64_t)page * p.Hkv + h) << p.page_shift) + (pos & (ps - 1));
#pragma unroll
                for (int kv = 0; kv < KV; ++kv) {
                    const bool v = value(kv);
                    if (from > 0) was[kv] = (v ? p.vs : p.ks)[at >> p.block_shift];
                    const int64_t ld = v ? p.ldv : p.ldk;
                    const T *src = static_cast<const T *>(v ? p.v : p.k) + ((int64_t)s.t0 + pos - s.start) * ld + (int64_t)h * D + ch;
#pragma unroll
                    for (int i = 0; i < STEPS; ++i) {
                        const int r = row0 + i * RPS;
                        if (r >= from && r < to) x[kv][i].load(src + r * ld);
                    }
                }
            } else if (lane == 0 && part == 0) {
                report_status(p.status, KDA_ERR_INVALID_ARG);
            }
        }
        // ---- the largest finite values, and the scales
        float amax[KV];
        bool odd[KV];                                 // (the same in all lanes)
#pragma unroll
        for (int kv = 0; kv < KV; ++kv) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < STEPS; ++i) x[kv][i].top(top);
            top = __reduce_max_sync(0xffffffffu, Row8<T, VEC>::joined(top));
            odd[kv] = top >= 0x7f800000u;
            amax[kv] = __uint_as_float(top);
            if (odd[kv]) {
                float a = 0.f;
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    float f[8];
                    x[kv][i].get(f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(f[e]) < INFINITY ? fabsf(f[e]) : 0.f);
                }
                amax[kv] = ptx::warp_max(a);
            }
            if (share > 1 && lane == 0) s_max[round & 1][kv][warp] = amax[kv];
        }
        if (share > 1) {
            __syncthreads();
#pragma unroll
            for (int kv = 0; kv < KV; ++kv)
                for (int i = 0; i < share; ++i) amax[kv] = fmaxf(amax[kv], s_max[round & 1][kv][mine * share + i]);
        } else {
            __syncwarp();                             // (every lane has read the scales that one writes)
        }
        if (from < to)
#pragma unroll
            for (int kv = 0; kv < KV; ++kv) {
                const bool v = value(kv);
                float scale = scale_for(amax[kv]);
                bool again = false;                   // earlier codes are rounded to a new scale
                if (from > 0) {
                    if (was[kv] >= kLeast && was[kv] <= kMost) {
                        scale = fmaxf(scale, __uint_as_float((__float_as_uint(was[kv]) + 0x7fffffu) & 0xff800000u));
                        again = scale != was[kv];
                    } else if (lane == 0 && part == 0) {
                        report_status(p.status, KDA_ERR_INVALID_ARG);
                    }
                }
                uint8_t *dst = (v ? p.vc : p.kc) + at * D + ch;
                const float inv = inverse(scale);
                auto round_again = [&](int r) {
                    float f[8];
                    decode8(*reinterpret_cast<const uint2 *>(dst + r * D), f);
                    *reinterpret_cast<uint2 *>(dst + r * D) = encode8<true>(f, was[kv] * inv);
                };
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int r = row0 + i * RPS;
                    if (r >= from && r < to) {
                        float f[8];
                        x[kv][i].get(f);
                        *reinterpret_cast<uint2 *>(dst + r * D) = odd[kv] ? encode8<true>(f, inv) : encode8<false>(f, inv);
                    } else if (again && r < from) {
                        round_again(r);
                    }
                }
                if (again && !p.cu_seqlens)           // what lies before this warp's rows
                    for (int r = lane_row; r < row0 - lane_row; r += RPS) round_again(r);
                if (lane == 0 && part == 0) (v ? p.vs : p.ks)[at >> p.block_shift] = scale;
            }
        for (task += per; task >= tasks; task -= tasks) ++blk;
    }
}

template <typename T, int D, bool VEC>
cudaError_t launch(const AppendQ8Params &p, cudaStream_t st) {
    const int B = 1 << p.block_shift, per = p.cu_seqlens ? WARPS / (B / ROWS) : WARPS;
    // at most two blocks of a sequence are not whole
    const int64_t blocks = p.cu_seqlens ? p.total / B + 2 * (int64_t)min((int64_t)p.num_seqs, p.total) : p.num_seqs;
    const int64_t most = (blocks * (2 / kBoth<T, D>) * p.Hkv + per - 1) / per, room = (int64_t)sm_count() * kCtas<T, D>;
    return launch_dependent(paged_append_q8_kernel<T, D, VEC>, dim3((unsigned)(most < room ? most : room)), WARPS * 32, 0, st, 1,
                            p);
}
template <typename T, bool VEC>
cudaError_t launch_d(const AppendQ8Params &p, int d, cudaStream_t st) {
    return d == 32 ? launch<T, 32, VEC>(p, st) : d == 64 ? launch<T, 64, VEC>(p, st) : launch<T, 128, VEC>(p, st);
}

}  // namespace

cudaError_t launch_paged_append_q8(const AppendQ8Params &p, int d, bool bf16, bool vec16, cudaStream_t st) {
    if (bf16) return vec16 ? launch_d<__nv_bfloat16, true>(p, d, st) : launch_d<__nv_bfloat16, false>(p, d, st);
    return vec16 ? launch_d<float, true>(p, d, st) : launch_d<float, false>(p, d, st);
}

}  // namespace kda
