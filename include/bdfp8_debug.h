/*
 * bdfp8_debug.h -- test hook of the 8-bit cache's decode: so that a test can
 * exercise a path that a correct run never takes.
 */
#ifndef BDFP8_DEBUG_H
#define BDFP8_DEBUG_H

#include "bdfp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* what goes wrong in every block of bdfp8_debug_decode_wait_test */
#define BDFP8_STALL_NONE 0
#define BDFP8_STALL_TILE 1 /* its first key tile is never announced: every wait for it runs out    */
#define BDFP8_STALL_WARP 2 /* one softmax warp gives up on its first tile; the others see it arrive */

/*
 * bdfp8_decode with E4M3, d = 128 and either five to eight query heads per KV
 * head and T_q = 1 or more than 16 rows H_q / H_kv * T_q (the shapes compiled
 * with this switch; others return BDFP4_ERR_UNSUPPORTED), every in-kernel wait
 * bounded by wait_limit_cycles clock cycles (at most the usual two seconds).  With a
 * stall, blocks unwind: their warps leave together, their producers wait
 * (bounded) until every copy they started has landed, their MMA warps until
 * every tensor-core operation they issued has finished, tensor memory is freed
 * and BDFP4_DEV_TIMEOUT is OR-ed into *dev_status.  The output is then
 * undefined; the device context stays usable.  BDFP8_STALL_NONE is bdfp8_decode.
 * Returns BDFP4_ERR_ARG for a bound that is not positive or another stall.
 */
BDFP4_API int bdfp8_debug_decode_wait_test(const void* q, const void* k_pages, const void* v_pages,
                                           const float* kv_scales, const int32_t* block_table,
                                           const int32_t* seq_lens, int B, int T_q, int H_q, int H_kv, int d,
                                           int max_pages_per_seq, int64_t num_pages, bdfp8_fmt fmt, int window,
                                           int sinks, float sm_scale, int chunk_tiles, void* workspace,
                                           size_t workspace_bytes, void* out, int32_t* dev_status,
                                           long long wait_limit_cycles, int stall, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BDFP8_DEBUG_H */
