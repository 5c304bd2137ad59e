// kda_pages.cu -- the pages of a paged cache: handed out to rows of a page table,
// taken back, shared between rows that go on from the same tokens, and moved
// together.
//
// The bookkeeping is a few integers a row and one a page, and a chain of steps that
// each need the one before: what is given back, what is free, what goes where.  One
// cluster of eight CTAs does it in one launch: its barrier stands between the steps,
// and counts go from CTA to CTA through distributed shared memory.  Pages' contents
// are copied by a second kernel over the whole GPU, from the list that the first left.
//
// Free pages are taken lowest first, rows and pairs served in order, so that the
// result depends on the arguments alone.
//
// The chain of steps bounds the bookkeeping: a resize that changes hardly anything takes
// 5 us on the device, one that gives back or hands out 65000 pages 14 (eight SMs' scattered
// atomics and stores); a fork of four rows 9, a compaction of a hundred pages 7.  With their
// copies 192 forks of 1.5 MB take 104 us (0.84 of the copy rate), 870 MB compacted 269 (0.95).
#include "kda_pages.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace {

constexpr int CL = 8, NT = 1024, NW = NT / 32;

__device__ __forceinline__ int ldcg(const int32_t *p) { return __ldcg(p); }

// ---------------------------------------------------------------------------
// Sums over the cluster, in the order of its CTAs and their warps.
// ---------------------------------------------------------------------------
struct Scan {
    int warp_sum[NW];
    int cta_sum[2][CL];             // written by all CTAs of the cluster, in turn
};
struct Ranks {
    int before, total;              // in the warps before this one; in all
    int cta;                        // in the CTAs before this one
};

__device__ __forceinline__ int lanes_before(int x, int lane, int &sum) {
    int y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    sum = __shfl_sync(0xffffffffu, y, 31);
    return y - x;
}

// Block-wide, from a number per warp (the same in all its lanes).
__device__ Ranks scan_cta(Scan &s, int mine) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) s.warp_sum[warp] = mine;
    __syncthreads();
    Ranks r{};
    const int x = lanes_before(s.warp_sum[lane], lane, r.total);
    r.before = __shfl_sync(0xffffffffu, x, warp);
    return r;
}
// Cluster-wide, of a number per warp; `turn` counts these calls.
__device__ Ranks scan_cluster(Scan &s, int mine, int &turn) {
    const int rank = (int)ptx::cluster_rank();
    Ranks r = scan_cta(s, mine);
    int *slot = &s.cta_sum[turn & 1][rank];
    ++turn;
    if (threadIdx.x < CL)
        asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(ptx::map_to_rank(slot, threadIdx.x)), "r"(r.total) : "memory");
    ptx::cluster_sync();
    const int *all = slot - rank;
    r.total = 0;
#pragma unroll
    for (int i = 0; i < CL; ++i) {
        if (i < rank) r.cta += all[i];
        r.total += all[i];
    }
    r.before += r.cta;
    return r;
}

// Sums [0, 1024) before each thread's number, in shared memory, and the row of the i-th of what they count.
struct Flat {
    int before[NT];
    __device__ int fill(Scan &s, int x) {
        int sum;
        const int b = lanes_before(x, threadIdx.x & 31, sum);
        const Ranks r = scan_cta(s, sum);
        before[threadIdx.x] = r.before + b;
        __syncthreads();
        return r.total;
    }
    __device__ int row(int i) const {             // the last with before[row] <= i
        int lo = 0;
#pragma unroll
        for (int step = NT / 2; step; step >>= 1)
            if (before[lo + step] <= i) lo += step;
        return lo;
    }
};

// A list that the whole cluster writes and reads: in its CTAs' shared memory, or in device memory where it is longer.
constexpr int kListShift = 13;                    // entries of a CTA
constexpr int kListMost = CL << kListShift;
struct List {
    int32_t *device, *shared;                     // (shared: at the same place in every CTA, or null)
    __device__ void put(int i, int x) const {
        if (shared)
            asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(
                             ptx::map_to_rank(shared + (i & ((1 << kListShift) - 1)), i >> kListShift)), "r"(x) : "memory");
        else
            device[i] = x;
    }
    __device__ int get(int i) const {
        if (!shared) return ldcg(device + i);
        int x;
        asm volatile("ld.shared::cluster.s32 %0, [%1];"
                     : "=r"(x)
                     : "r"(ptx::map_to_rank(shared + (i & ((1 << kListShift) - 1)), i >> kListShift))
                     : "memory");
        return x;
    }
};

// The lowest pages that no one holds, up to `need` of them, into list; how many there are.  Cluster-wide.  A warp looks
// at up to 1024 pages in a row at a time, and lane j keeps which of the j-th 32 are free: one sum over the cluster for
// up to 262,144 pages.
__device__ int take_free(const PageTable &p, int need, const List &list, Scan &s, int &turn) {
    constexpr int J = 8;                          // loads under way per thread
    const int lane = threadIdx.x & 31, gw = (int)ptx::cluster_rank() * NW + (threadIdx.x >> 5);
    const int groups = min(32, (int)(((int64_t)p.num_pages + CL * NW * 32 - 1) / (CL * NW * 32)));
    int found = 0;
    for (int64_t p0 = 0; p0 < p.num_pages && found < need; p0 += CL * NW * 32 * groups) {
        const int64_t at = p0 + (int64_t)gw * 32 * groups + lane;
        unsigned mine = 0;
        for (int g = 0; g < groups; g += J) {
            bool b[J];
#pragma unroll
            for (int j = 0; j < J; ++j)
                b[j] = g + j < groups && at + (g + j) * 32 < p.num_pages && ldcg(p.refs + at + (g + j) * 32) == 0;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const unsigned x = __ballot_sync(0xffffffffu, b[j]);
                if (lane == g + j) mine = x;
            }
        }
        int sum;
        const int before = lanes_before(__popc(mine), lane, sum);
        const Ranks r = scan_cluster(s, sum, turn);
        for (int g = 0; g < groups; ++g) {
            const unsigned b = __shfl_sync(0xffffffffu, mine, g);
            const int k = found + r.before + __shfl_sync(0xffffffffu, before, g) + __popc(b & ((1u << lane) - 1));
            if ((b >> lane & 1) && k < need) list.put(k, (int)(at + g * 32));
        }
        found += r.total;
    }
    ptx::cluster_sync();                          // the list is written
    return min(found, need);
}

// One holder less for each of the pages; one that had none is left so, and so is a count below 0.  (Loads and atomics go
// ahead of what is done with their results, so that all of a thread's are under way at a time.)
template <int U>
__device__ __forceinline__ void give_back(const PageTable &p, const int (&id)[U]) {
    int count[U];
#pragma unroll
    for (int u = 0; u < U; ++u) count[u] = id[u] >= 0 && id[u] < p.num_pages ? ldcg(p.refs + id[u]) : -1;
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (count[u] >= 0) count[u] = atomicSub(p.refs + id[u], 1);
        else count[u] = id[u] < p.num_pages ? 1 : 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (count[u] <= 0) {
            if (id[u] < p.num_pages) atomicAdd(p.refs + id[u], 1);
            report_status(p.status, KDA_ERR_INVALID_ARG);
        }
}

// ---------------------------------------------------------------------------
// Resize.
// ---------------------------------------------------------------------------
struct Change {
    int held, want;                               // pages; equal where nothing changes
};
__device__ __forceinline__ Change change(const PageTable &p, const int32_t *tokens, int row, bool tell) {
    const int t = tokens[row], held = ldcg(p.held + row);
    const int want = t < 0 ? held : (int)(((int64_t)t + (1 << p.page_shift) - 1) >> p.page_shift);
    if (held < 0 || held > p.max_pages || want > p.max_pages) {
        if (tell) report_status(p.status, KDA_ERR_INVALID_ARG);
        return {0, 0};
    }
    return {held, want};
}

__global__ void __launch_bounds__(NT, 1) pages_resize_kernel(const PageTable p, const int32_t *tokens, int32_t *workspace) {
    constexpr int U = 8;                          // pages under way per thread
    __shared__ Scan s;
    __shared__ Flat flat;
    __shared__ int s_first[NT];                   // each row's first entry that changes
    __shared__ int32_t s_list[1 << kListShift];
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    ptx::cluster_sync();                          // all CTAs are there to be written to
    const int tid = threadIdx.x, rank = (int)ptx::cluster_rank();
    const int each = (int)(((int64_t)p.rows + CL - 1) / CL);
    const int64_t r0 = min((int64_t)p.rows, (int64_t)rank * each), r1 = min((int64_t)p.rows, r0 + each);
    int turn = 0, need = 0;

    // what is given back, and how many pages this CTA's rows need
    for (int64_t c = r0; c < r1; c += NT) {
        Change x{0, 0};
        if (c + tid < r1) x = change(p, tokens, (int)(c + tid), true);
        __syncthreads();                          // (the rows before are done with)
        s_first[tid] = x.want;
        const int total = flat.fill(s, max(0, x.held - x.want));
        for (int i0 = tid; i0 < total; i0 += U * NT) {
            int id[U];
            int32_t *entry[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * NT;
                id[u] = -1;
                entry[u] = nullptr;
                if (i >= total) continue;
                const int row = flat.row(i);
                entry[u] = p.table + (c + row) * p.max_pages + s_first[row] + i - flat.before[row];
                id[u] = *entry[u];
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (entry[u]) *entry[u] = -1;
            give_back(p, id);
        }
        if (x.want < x.held) p.held[c + tid] = x.want;
        int sum;
        lanes_before(max(0, x.want - x.held), tid & 31, sum);
        need += sum;                              // (of this warp)
    }
    const Ranks all = scan_cluster(s, need, turn);
    if (all.total == 0) return;                   // (the same in all CTAs)
    int base = all.cta;                           // needed by the CTAs before this one
    const List list{workspace, min(all.total, p.num_pages) <= kListMost ? s_list : nullptr};
    const int got = take_free(p, all.total, list, s, turn);

    for (int64_t c = r0; c < r1; c += NT) {
        Change x{0, 0};
        if (c + tid < r1) x = change(p, tokens, (int)(c + tid), false);
        __syncthreads();
        s_first[tid] = x.held;
        const int mine = max(0, x.want - x.held), total = flat.fill(s, mine), most = min(total, got - base);
        for (int i0 = tid; i0 < most; i0 += U * NT) {
            int page[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * NT < most) page[u] = list.get(base + i0 + u * NT);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * NT;
                if (i >= most) break;
                const int row = flat.row(i);
                p.table[(c + row) * p.max_pages + s_first[row] + i - flat.before[row]] = page[u];
                p.refs[page[u]] = 1;
            }
        }
        if (mine > 0) {
            const int have = min(mine, max(0, got - base - flat.before[tid]));
            if (have < mine) report_status(p.status, KDA_ERR_NO_PAGES);
            p.held[c + tid] = x.held + have;
        }
        base += total;
    }
    ptx::cluster_sync();                          // (the others read this CTA's part of the list)
}

// ---------------------------------------------------------------------------
// Copies of pages in all pools, a unit of up to 4 KB of one page at a time by each warp,
// all of whose loads are under way at once (units of 16 KB by a CTA leave it waiting for
// a page's scales of a few bytes as long as for its keys: 290 us instead of 273).  Sources
// are pages in use and destinations free ones, so no order is needed.
// ---------------------------------------------------------------------------
constexpr int kUnit = 4096, kCopyThreads = 256;
constexpr int64_t kMostAtOnce = 1 << 19;          // bytes of pages that the planning kernel copies by itself


template <typename V>
__device__ __forceinline__ void copy_unit(uint8_t *dst, const uint8_t *src, int bytes) {
    constexpr int U = 8;                          // loads under way per lane
    const int n = bytes / (int)sizeof(V);
    for (int i0 = threadIdx.x & 31; i0 < n; i0 += U * 32) {
        V x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * 32 < n) x[u] = reinterpret_cast<const V *>(src)[i0 + u * 32];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * 32 < n) reinterpret_cast<V *>(dst)[i0 + u * 32] = x[u];
    }
}

// The part of warp `warp` of `warps`.
__device__ __forceinline__ void copy_pages(const Pools &pools, const int32_t *from, const int32_t *to, int count, int warp,
                                           int warps) {
    const int per = pools.first[pools.n];
    for (int64_t u = warp; u < (int64_t)count * per; u += warps) {
        const int pair = (int)(u / per), at = (int)(u - (int64_t)pair * per);
        int lo = 0, hi = pools.n;                 // the pool of the unit
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pools.first[mid] <= at) lo = mid; else hi = mid;
        }
        const int64_t size = pools.bytes[lo], off = (int64_t)(at - pools.first[lo]) * kUnit;
        uint8_t *base = pools.base[lo];
        uint8_t *dst = base + ldcg(to + pair) * size + off;
        const uint8_t *src = base + ldcg(from + pair) * size + off;
        const int bytes = (int)min((int64_t)kUnit, size - off);
        const uint64_t odd = reinterpret_cast<uint64_t>(base) | (uint64_t)size;
        if (odd % 16 == 0) copy_unit<uint4>(dst, src, bytes);
        else if (odd % 4 == 0) copy_unit<uint32_t>(dst, src, bytes);
        else copy_unit<uint8_t>(dst, src, bytes);
    }
}

// ---------------------------------------------------------------------------
// Fork: which pairs hold, and the free pages for their last pages' copies.
// ---------------------------------------------------------------------------
struct ForkPlan {
    int32_t *mark;                  // [rows]: -1 for a source, else the first pair that has the row as its destination
    int32_t *list;                  // [forks]: free pages
    int4 *rows;                     // [forks]: source row (-1: the pair does not hold), destination, full pages, new page or -1
    int32_t *from, *to, *count;     // [forks], [forks], [1]: pages to copy
};
// Source row (-1: the pair does not hold), destination, tokens, and the source's last page where that is to be copied.
__device__ int4 fork_pair(const PageTable &p, const int32_t *lens, const int32_t *src, const int32_t *dst, const ForkPlan &f, int i) {
    const int a = src[i], b = dst[i];
    if (a < 0 || b < 0) return make_int4(-1, b, 0, -1);                    // padding
    int len = 0, page = -1;
    bool bad = a >= p.rows || b >= p.rows || ldcg(f.mark + b) != i || ldcg(p.held + b) != 0;
    if (!bad) {
        const int held = ldcg(p.held + a);
        len = ldcg(lens + a);
        bad = len < 0 || held < 0 || held > p.max_pages || len > (int64_t)held << p.page_shift;
        if (!bad && (len & ((1 << p.page_shift) - 1))) {
            page = p.table[(int64_t)a * p.max_pages + (len >> p.page_shift)];
            bad = page < 0 || page >= p.num_pages || ldcg(p.refs + page) == 0;
        }
    }
    if (bad) report_status(p.status, KDA_ERR_INVALID_ARG);
    return bad ? make_int4(-1, b, 0, -1) : make_int4(a, b, len, page);
}

// The destinations' rows of the table, an entry at a time.
__device__ __forceinline__ void fork_rows(const PageTable &p, int forks, const ForkPlan &f, int64_t thread, int64_t threads) {
    for (int64_t x = thread; x < (int64_t)forks * p.max_pages; x += threads) {
        const int i = (int)(x / p.max_pages), e = (int)(x - (int64_t)i * p.max_pages);
        const int4 r = __ldcg(f.rows + i);
        if (r.x < 0 || e > r.z || (e == r.z && r.w < 0)) continue;
        int id = r.w;
        if (e < r.z) {
            id = p.table[(int64_t)r.x * p.max_pages + e];
            if (id >= 0 && id < p.num_pages) {
                // (a count below 0 is not kept: it would come to 0, and the page be handed out)
                if (ldcg(p.refs + id) >= 0) atomicAdd(p.refs + id, 1);
            } else {
                report_status(p.status, KDA_ERR_INVALID_ARG);
                id = -1;
            }
        }
        p.table[(int64_t)r.y * p.max_pages + e] = id;
    }
}

// copy: the pools are copied here too.
__global__ void __launch_bounds__(NT, 1)
    pages_fork_kernel(const __grid_constant__ Pools pools, const PageTable p, int32_t *lens, const int32_t *src,
                      const int32_t *dst, int forks, const ForkPlan f, bool copy) {
    __shared__ Scan s;
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    ptx::cluster_sync();
    const int tid = threadIdx.x, lane = tid & 31, rank = (int)ptx::cluster_rank();
    auto rows = [&](auto &&visit) {
        for (int64_t i = rank * NT + tid; i < forks; i += CL * NT) {
            const int a = src[i], b = dst[i];
            if (a >= 0 && b >= 0 && a < p.rows && b < p.rows) visit(a, b, (int)i);
        }
        ptx::cluster_sync();
    };
    rows([&](int a, int b, int) { f.mark[a] = f.mark[b] = 0x7fffffff; });
    rows([&](int a, int b, int i) {
        atomicMin(f.mark + a, -1);
        atomicMin(f.mark + b, i);
    });
    const int each = (int)(((int64_t)forks + CL - 1) / CL);
    const int64_t i0 = min((int64_t)forks, (int64_t)rank * each), i1 = min((int64_t)forks, i0 + each);
    int turn = 0, need = 0;
    for (int64_t c = i0; c < i1; c += NT) {
        int4 x = make_int4(-1, 0, 0, -1);
        if (c + tid < i1) f.rows[c + tid] = x = fork_pair(p, lens, src, dst, f, (int)(c + tid));
        need += __popc(__ballot_sync(0xffffffffu, x.w >= 0));
    }
    const Ranks all = scan_cluster(s, need, turn);
    int base = all.cta;
    const int got = take_free(p, all.total, List{f.list, nullptr}, s, turn);
    if (rank == 0 && tid == 0) *f.count = got;
    for (int64_t c = i0; c < i1; c += NT) {
        int4 x = make_int4(-1, 0, 0, -1);
        if (c + tid < i1) x = f.rows[c + tid];     // (written by this thread)
        const unsigned b = __ballot_sync(0xffffffffu, x.w >= 0);
        const Ranks r = scan_cta(s, __popc(b));
        if (x.x >= 0) {
            const int full = x.z >> p.page_shift;
            int page = -1;
            if (x.w >= 0) {
                const int k = base + r.before + __popc(b & ((1u << lane) - 1));
                if (k < got) {
                    page = ldcg(f.list + k);
                    f.from[k] = x.w;
                    f.to[k] = page;
                    p.refs[page] = 1;
                } else {
                    x.x = -1;
                    report_status(p.status, KDA_ERR_NO_PAGES);
                }
            }
            f.rows[c + tid] = make_int4(x.x, x.y, full, page);
            if (x.x >= 0) {
                p.held[x.y] = full + (page >= 0);
                lens[x.y] = x.z;
            }
        }
        base += r.total;
    }
    if (copy) {
        ptx::cluster_sync();                      // the plan is there for all
        fork_rows(p, forks, f, rank * NT + tid, CL * NT);
        copy_pages(pools, f.from, f.to, got, (rank * NT + tid) / 32, CL * NW);
    }
}

// ---------------------------------------------------------------------------
// Compact: with L pages in use, those at L and above move, in order, to the free
// ones below L, of which there are as many.
// ---------------------------------------------------------------------------
struct CompactPlan {
    int32_t *from, *to, *count;     // [num_pages], [num_pages], [1]: pages to copy
    int32_t *map, *live;            // (the caller's)
};

// The table, an entry at a time.
__device__ __forceinline__ void compact_rows(const PageTable &p, const CompactPlan &f, int64_t thread, int64_t threads) {
    for (int64_t x = thread; x < (int64_t)p.rows * p.max_pages; x += threads) {
        const int id = p.table[x];
        if (id < 0) continue;
        const int to = id < p.num_pages ? ldcg(f.map + id) : -1;
        if (to < 0) report_status(p.status, KDA_ERR_INVALID_ARG);
        if (to != id) p.table[x] = to;
    }
}

// copy: the pools are copied here too.
__global__ void __launch_bounds__(NT, 1)
    pages_compact_kernel(const __grid_constant__ Pools pools, const PageTable p, const CompactPlan f, bool copy) {
    __shared__ Scan s;
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    ptx::cluster_sync();
    const int lane = threadIdx.x & 31, gw = (int)ptx::cluster_rank() * NW + (threadIdx.x >> 5);
    constexpr int J = 8;
    // a warp's pages [w0, w1), 32 J at a time: visit(first page of 32, whether this lane's page exists, its holders)
    const int each = (int)(((int64_t)p.num_pages + CL * NW * 32 - 1) / (CL * NW * 32)) * 32;
    const int64_t w0 = min((int64_t)p.num_pages, (int64_t)gw * each), w1 = min((int64_t)p.num_pages, w0 + each);
    auto pages = [&](auto &&visit) {
        for (int64_t b = w0; b < w1; b += 32 * J) {
            int refs[J];
#pragma unroll
            for (int j = 0; j < J; ++j) refs[j] = b + j * 32 + lane < w1 ? ldcg(p.refs + b + j * 32 + lane) : 0;
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (b + j * 32 < w1) visit((int)(b + j * 32) + lane, b + j * 32 + lane < w1, refs[j]);
        }
    };
    int turn = 0, count = 0;
    pages([&](int, bool, int refs) { count += __popc(__ballot_sync(0xffffffffu, refs != 0)); });
    const int live = scan_cluster(s, count, turn).total;
    int holes = 0, movers = 0;
    pages([&](int id, bool is, int refs) {
        holes += __popc(__ballot_sync(0xffffffffu, is && refs == 0 && id < live));
        movers += __popc(__ballot_sync(0xffffffffu, refs != 0 && id >= live));
    });
    const Ranks h = scan_cluster(s, holes, turn), m = scan_cluster(s, movers, turn);
    const unsigned below = (1u << lane) - 1;
    int k = h.before;
    pages([&](int id, bool is, int refs) {
        const bool hole = is && refs == 0 && id < live;
        const unsigned b = __ballot_sync(0xffffffffu, hole);
        if (hole) f.to[k + __popc(b & below)] = id;
        if (is && (refs == 0 || id < live)) f.map[id] = refs ? id : -1;
        k += __popc(b);
    });
    ptx::cluster_sync();                          // the holes are listed
    k = m.before;
    pages([&](int id, bool, int refs) {
        const bool mover = refs != 0 && id >= live;
        const unsigned b = __ballot_sync(0xffffffffu, mover);
        if (mover) {
            const int i = k + __popc(b & below), to = ldcg(f.to + i);
            f.from[i] = id;
            f.map[id] = to;
            p.refs[to] = refs;
            p.refs[id] = 0;
        }
        k += __popc(b);
    });
    if (gw == 0 && lane == 0) {
        *f.count = m.total;
        *f.live = live;
    }
    if (copy) {
        ptx::cluster_sync();                      // the plan is there for all
        const int thread = (int)ptx::cluster_rank() * NT + threadIdx.x;
        compact_rows(p, f, thread, CL * NT);
        copy_pages(pools, f.from, f.to, m.total, thread / 32, CL * NW);
    }
}

// first: the launch that also writes the rows of the table.
__global__ void __launch_bounds__(kCopyThreads)
    pages_fork_copy_kernel(const __grid_constant__ Pools pools, const PageTable p, int forks, const ForkPlan f, bool first) {
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    if (first) fork_rows(p, forks, f, (int64_t)blockIdx.x * kCopyThreads + threadIdx.x, (int64_t)gridDim.x * kCopyThreads);
    copy_pages(pools, f.from, f.to, *f.count, (blockIdx.x * kCopyThreads + threadIdx.x) / 32, gridDim.x * (kCopyThreads / 32));
}

__global__ void __launch_bounds__(kCopyThreads)
    pages_compact_copy_kernel(const __grid_constant__ Pools pools, const PageTable p, const CompactPlan f, bool first) {
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    if (first) compact_rows(p, f, (int64_t)blockIdx.x * kCopyThreads + threadIdx.x, (int64_t)gridDim.x * kCopyThreads);
    copy_pages(pools, f.from, f.to, *f.count, (blockIdx.x * kCopyThreads + threadIdx.x) / 32, gridDim.x * (kCopyThreads / 32));
}

Pools some_pools(void *const *base, const int64_t *bytes, int n) {
    Pools pools{};
    pools.n = n;
    for (int i = 0; i < n; ++i) {
        pools.base[i] = static_cast<uint8_t *>(base[i]);
        pools.bytes[i] = bytes[i];
        pools.first[i + 1] = pools.first[i] + (int)((bytes[i] + kUnit - 1) / kUnit);
    }
    return pools;
}

// Up to half a megabyte the planning kernel's eight CTAs copy sooner than a second launch would.
bool copied_at_once(const int64_t *bytes, int n, int64_t others, int64_t pairs) {
    if (n > kPoolsPerLaunch || others > (1 << 16)) return false;
    int64_t page = 0;
    for (int i = 0; i < n; ++i) page += bytes[i] < kMostAtOnce ? bytes[i] : kMostAtOnce;
    return page == 0 || pairs <= kMostAtOnce / page;
}

// Calls launch(pools, grid, first) for all pools, at most kPoolsPerLaunch of them at a time, and once where there are none.
// others: threads' worth of other work; pairs: pages to copy, at most; ctas: of an SM, at most (three run at a time).  More
// even out what each takes (half of a batch compacted: 273 us with 8, 267 with 24, 264 with 48); where it is not known how
// many pages move, those that find nothing to do cost as well (two pages of 4000: 11.8, 13.5 and 17.2 us).
template <typename F>
cudaError_t launch_copies(void *const *base, const int64_t *bytes, int n, int64_t others, int64_t pairs, int ctas, F &&launch) {
    for (int at = 0; at == 0 || at < n; at += kPoolsPerLaunch) {
        const Pools pools = some_pools(base + at, bytes + at, n - at < kPoolsPerLaunch ? n - at : kPoolsPerLaunch);
        const int64_t units = (pairs * pools.first[pools.n] + kCopyThreads / 32 - 1) / (kCopyThreads / 32), work = (others + kCopyThreads - 1) / kCopyThreads;
        const int64_t most = units > work ? units : work, room = (int64_t)sm_count() * ctas;
        const cudaError_t e = launch(pools, dim3((unsigned)(most < 1 ? 1 : (most < room ? most : room))), at == 0);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

size_t up16(size_t n) { return (n + 15) & ~size_t(15); }

}  // namespace

size_t pages_resize_workspace_bytes(int num_pages) { return num_pages <= kListMost ? 0 : up16(4 * (size_t)num_pages); }

cudaError_t launch_pages_resize(const PageTable &p, const int32_t *tokens, void *workspace, cudaStream_t st) {
    return launch_dependent(pages_resize_kernel, dim3(CL), NT, 0, st, CL, p, tokens, static_cast<int32_t *>(workspace));
}

size_t pages_fork_workspace_bytes(int rows, int forks) {
    return up16(4 * (size_t)rows) + up16(4 * (size_t)forks) * 3 + 16 * (size_t)forks + 16;
}

cudaError_t launch_pages_fork(void *const *pools, const int64_t *page_bytes, int num_pools, const PageTable &p, int32_t *lens,
                              const int32_t *src, const int32_t *dst, int forks, void *workspace, cudaStream_t st) {
    uint8_t *w = static_cast<uint8_t *>(workspace);
    auto piece = [&](size_t bytes) {
        void *at = w;
        w += up16(bytes);
        return static_cast<int32_t *>(at);
    };
    ForkPlan f;
    f.count = piece(4);
    f.mark = piece(4 * (size_t)p.rows);
    f.list = piece(4 * (size_t)forks);
    f.from = piece(4 * (size_t)forks);
    f.to = piece(4 * (size_t)forks);
    f.rows = reinterpret_cast<int4 *>(piece(16 * (size_t)forks));
    const bool once = copied_at_once(page_bytes, num_pools, (int64_t)forks * p.max_pages, forks);
    const Pools now = some_pools(pools, page_bytes, once ? num_pools : 0);
    const cudaError_t e = launch_dependent(pages_fork_kernel, dim3(CL), NT, 0, st, CL, now, p, lens, src, dst, forks, f, once);
    if (e != cudaSuccess || once) return e;
    return launch_copies(pools, page_bytes, num_pools, (int64_t)forks * p.max_pages, forks, 24,
                         [&](const Pools &some, dim3 grid, bool first) {
                             return launch_dependent(pages_fork_copy_kernel, grid, kCopyThreads, 0, st, 1, some, p, forks, f,
                                                     first);
                         });
}

size_t pages_compact_workspace_bytes(int num_pages) { return 16 + 2 * up16(4 * (size_t)num_pages); }

cudaError_t launch_pages_compact(void *const *pools, const int64_t *page_bytes, int num_pools, const PageTable &p,
                                 int32_t *page_map, int32_t *live, void *workspace, cudaStream_t st) {
    uint8_t *w = static_cast<uint8_t *>(workspace);
    CompactPlan f;
    f.count = reinterpret_cast<int32_t *>(w);
    f.from = reinterpret_cast<int32_t *>(w + 16);
    f.to = reinterpret_cast<int32_t *>(w + 16 + up16(4 * (size_t)p.num_pages));
    f.map = page_map;
    f.live = live;
    // (no more pages move than half of them)
    const bool once = copied_at_once(page_bytes, num_pools, (int64_t)p.rows * p.max_pages, p.num_pages / 2);
    const Pools now = some_pools(pools, page_bytes, once ? num_pools : 0);
    const cudaError_t e = launch_dependent(pages_compact_kernel, dim3(CL), NT, 0, st, CL, now, p, f, once);
    if (e != cudaSuccess || once) return e;
    return launch_copies(pools, page_bytes, num_pools, (int64_t)p.rows * p.max_pages, p.num_pages / 2, 16,
                         [&](const Pools &some, dim3 grid, bool first) {
                             return launch_dependent(pages_compact_copy_kernel, grid, kCopyThreads, 0, st, 1, some, p, f, first);
                         });
}

}  // namespace kda
