// kda_layers.cuh -- what the translation units of the layer operators
// (include/kda_layers.h) share: parameter blocks, launchers, small helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kda_common.cuh"
#include "kda_layers.h"

namespace kda {

struct LinearParams {
    const __nv_bfloat16 *x;
    int64_t ldx;
    const __nv_bfloat16 *w;
    const float *bias;
    const void *residual;
    void *out;
    int64_t M, N, K;
    kda_act_t act;
    bool out_f32;
    uint32_t *status;
};
cudaError_t launch_linear(const LinearParams &p, cudaStream_t st);
// gridDim.y of the largest launch of its few-rows kernel
int64_t linear_row_tiles(int64_t M);

struct DecayParams {
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;          // row strides, elements
    const float *log_decay;         // [H]
    const int32_t *cu_seqlens;
    int num_seqs, H;
    int64_t total;
    float scale;
    const float *init;
    float *fin;
    void *out;
    uint32_t *status;
};
// bf16, total > 0, rows that start on 16-byte boundaries
size_t decay_prefill_tc_workspace(int64_t total, int N, int H, int dk, int dv);
cudaError_t launch_decay_prefill_tc(const DecayParams &p, int dk, int dv, void *workspace, size_t workspace_bytes,
                                    cudaStream_t st);
size_t decay_prefill_simt_workspace(int64_t total, int N, int H, int dk, int dv);
cudaError_t launch_decay_prefill_simt(const DecayParams &p, int dk, int dv, bool bf16, void *workspace,
                                      size_t workspace_bytes, cudaStream_t st);

struct DecayStepParams {
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;
    const float *log_decay;
    float *pool;
    int pool_size;
    const int32_t *slots;
    void *out;
    int N, H;
    float scale;
    uint32_t *status;
};
cudaError_t launch_decay_decode(const DecayStepParams &p, int dk, int dv, bool bf16, cudaStream_t st);

struct AppendParams {
    const void *k, *v;
    int64_t ldk, ldv;               // row strides, bytes
    void *kc, *vc;
    int num_pages, page_shift;
    const int32_t *table;
    int max_pages;
    const int32_t *start, *cu_seqlens;
    int num_seqs, Hkv;
    int64_t total;
    int row_bytes;                  // d x element size: one head of one token
    int lanes_log2;                 // lanes per token (of the launch's choosing)
    uint32_t *status;
};
cudaError_t launch_paged_append(AppendParams p, bool vec16, cudaStream_t st);

struct PagedParams {
    const void *q;
    int64_t ldq;
    const void *kc, *vc;
    int num_pages, page_shift;
    const int32_t *table;
    int max_pages;
    const int32_t *lens;
    int N, Hq, Hkv, G;              // G = Hq / Hkv query heads per key-value head
    float scale;
    void *out;
    float *lse;
    float *part;                    // partial results (workspace)
    bool lone;                      // no item has more than one tile: nothing to join
    int expire;                     // test support
    uint32_t *status;
};
size_t paged_decode_workspace_bytes(int N, int64_t max_tokens, int Hq, int Hkv, int d);
cudaError_t launch_paged_decode(const PagedParams &p, int d, bool bf16, cudaStream_t st);

// Number of SMs of the current device.
int sm_count();

// Test support: whether kda_testing_expire_next_wait armed this operator's bit,
// which is cleared; a kernel so called has CTA 0 fail one wait.
bool take_layers_expire(int bit);
constexpr long long kTestWait = 1LL << 21;    // cycles (about a millisecond)

// Opts `Kernel` in to dynamic shared memory of up to `bytes` on the current device, once (the call takes 2 us).
template <auto Kernel>
inline cudaError_t allow_smem(uint32_t bytes) {
    static std::atomic<uint64_t> done{0};         // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// Clusters of S <= 8 CTAs of `Kernel` that run at a time on the current device, always asked for with the same block and
// shared memory: it depends on how many SMs each of the GPU's clusters of SMs has, so the runtime is asked.
template <auto Kernel>
inline int cluster_room(int S, unsigned block, uint32_t smem) {
    static std::atomic<int> known[64][9];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 64 && (n = known[dev][S].load(std::memory_order_relaxed)) > 0) return n;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = S;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(S);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) != cudaSuccess) return 0;
    if (dev < 64) known[dev][S].store(n, std::memory_order_relaxed);
    return n;
}

// Launches `kernel` so that its start may overlap the end of the kernel before
// it in the stream: the kernel calls griddepcontrol.wait before it touches
// anything that another kernel writes, and so does every one of its blocks
// before it ends.  cluster: CTAs of a cluster along x, or 1.
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t st,
                                    unsigned cluster, const A &...args) {
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr float kLog2E = 1.4426950408889634f;

}  // namespace kda
