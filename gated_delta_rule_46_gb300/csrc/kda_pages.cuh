// kda_pages.cuh -- parameter blocks and launchers of include/kda_pages.h.
#pragma once

#include "kda_layers.cuh"
#include "kda_pages.h"

namespace kda {

struct PageTable {
    int32_t *table;                 // [rows][max_pages]
    int rows, max_pages;
    int32_t *held;                  // [rows]
    int32_t *refs;                  // [num_pages]
    int num_pages, page_shift;
    uint32_t *status;
};

// What a page is in each of several pools.
constexpr int kPoolsPerLaunch = 128;
struct Pools {
    uint8_t *base[kPoolsPerLaunch];
    int64_t bytes[kPoolsPerLaunch]; // of a page
    int first[kPoolsPerLaunch + 1]; // copy units of a page before this pool's
    int n;
};

size_t pages_resize_workspace_bytes(int num_pages);
cudaError_t launch_pages_resize(const PageTable &p, const int32_t *tokens, void *workspace, cudaStream_t st);

size_t pages_fork_workspace_bytes(int rows, int forks);
cudaError_t launch_pages_fork(void *const *pools, const int64_t *page_bytes, int num_pools, const PageTable &p, int32_t *lens,
                              const int32_t *src, const int32_t *dst, int forks, void *workspace, cudaStream_t st);

size_t pages_compact_workspace_bytes(int num_pages);
cudaError_t launch_pages_compact(void *const *pools, const int64_t *page_bytes, int num_pools, const PageTable &p,
                                 int32_t *page_map, int32_t *live, void *workspace, cudaStream_t st);

}  // namespace kda
