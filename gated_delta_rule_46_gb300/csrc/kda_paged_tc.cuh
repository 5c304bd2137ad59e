// kda_paged_tc.cuh -- what the tensor-core forms of attention over a paged cache share: a CTA's walk over its tiles,
// waits and reductions of a warp.
#pragma once

#include "kda_paged.cuh"
#include "kda_tc_util.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace paged {

constexpr int TILE = kTileTc;
constexpr long long kWaitBudget = 2000000000LL;   // cycles (about one second)
constexpr long long kDrain = 20000000LL;

// The tiles of this CTA in order: (sequence, item, tile); every role walks its
// own copy.  The next sequence's length is read a sequence ahead.
template <int TILE>
struct WalkOf {
    int64_t w, w1, nt, tile;
    int n, item, items, len, raw, ahead;      // len: raw, clamped to the table
    __device__ void start(const PagedParams &p, const Split &sp, int items_) {
        items = items_;
        w = quotient((int64_t)blockIdx.x * sp.W, sp.g);
        w1 = quotient((int64_t)(blockIdx.x + 1) * sp.W, sp.g);
        n = sp.n;
        raw = p.lens[n];
        len = clamped(p, raw);
        ahead = n + 1 < p.N ? p.lens[n + 1] : 0;
        nt = (len + TILE - 1) / TILE;
        item = (int)quotient(w - sp.cum * items, nt);
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

using Walk = WalkOf<TILE>;

__device__ __forceinline__ bool warp_wait(uint64_t *bar, int phase) {
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar, phase & 1, kWaitBudget));
}
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar);
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

}  // namespace paged
}  // namespace kda
