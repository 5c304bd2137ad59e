/*
 * kda_testing.h -- test support of the GB300 KDA library.  The pages have no
 * counterpart to anything here: it exists so that a test can exercise the
 * library's failure handling without faulting, trapping or hanging a GPU, and
 * look at a launch without making it.
 */
#ifndef KDA_GB300_TESTING_H
#define KDA_GB300_TESTING_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits of kda_testing_expire_next_wait(): the kernels whose first CTA is to see
 * a wait run out; of the tensor-core prefill: */
#define KDA_TESTING_FUSED 1        /* one-kernel plan (many chains) */
#define KDA_TESTING_INTRA 2        /* chunk-parallel kernel of the few-chain plans */
#define KDA_TESTING_SEGMENT 4      /* segment maps of the segment-scan plan */
#define KDA_TESTING_SCAN 8         /* the scan over segments */
#define KDA_TESTING_STATE 16       /* state pass of the few-chain plans */
/* and of the operators in kda_layers.h, where they run on the tensor cores: */
#define KDA_TESTING_LINEAR 32      /* kda_linear */
#define KDA_TESTING_DECAY 64       /* kda_decay_prefill */
#define KDA_TESTING_PAGED 128      /* kda_paged_decode, kda_paged_decode_q8 */

/*
 * kda_testing_expire_next_wait -- arms a simulated wait expiry for the next
 * bf16 d = 128 kda_chunk_prefill or kda_chunk_prefill_logdecay call in this
 * process (any thread, any device), which consumes and clears it.  In each
 * kernel named by `kernels` (a mask of the bits above) that the call
 * launches, CTA 0 waits, with a budget of about a millisecond, on a barrier
 * that nothing arrives at, before its first chunk.  The wait runs out and the
 * kernel takes the same path as a real expired wait: it records
 * KDA_ERR_DEVICE_TIMEOUT in the call's status word, lets its copies and
 * tensor-core operations in flight complete, frees its tensor memory and
 * returns, leaving that call's outputs incomplete and the CUDA context
 * usable.  kernels = 0 disarms.  Not for production use.
 * The last three bits are consumed, each by itself, by the next tensor-core
 * call of their operator; there one role of the kernel gives up and the others'
 * waits for it run out in earnest, after about a second.
 */
void kda_testing_expire_next_wait(int kernels);

/*
 * kda_testing_linear_row_tiles -- the largest gridDim.y of the launches that
 * kda_linear makes for M rows and K products where it takes them by rows: at
 * most 65535.  Touches no device.
 */
int64_t kda_testing_linear_row_tiles(int64_t M, int64_t K, kda_dtype_t out_dtype);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GB300_TESTING_H */
