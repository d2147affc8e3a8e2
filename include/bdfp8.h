/*
 * bdfp8.h -- an 8-bit paged KV cache beside the FP4 one of bdfp4.h: appending
 * keys and values to it with the position rotation applied on the way, and
 * decode attention over it, to the whole context or through a sliding window
 * with a few first tokens that stay visible.
 *
 * An FP4 cache quarters the bytes of a BF16 one and pays in error ("FP4 KV Cache
 * Done Right: What BitDecoding-FP4 Changes for Long-Context Serving", How good
 * are the results, really?); 8-bit floats halve them, with no calibration, no
 * smoothing and no rotation of channels.
 *
 * Conventions are those of bdfp4.h: device pointers, caller-owned memory, no
 * allocation and no state in the library, work asynchronous on `stream` (a
 * cudaStream_t, NULL = the legacy default stream) of the current device, host
 * errors as return codes before any launch, device-found errors OR-ed into
 * *dev_status (which may be NULL), no traps.  Every call can be captured into a
 * CUDA graph.  Queries, keys, values and outputs are bf16.
 *
 * Cache layout (pages of 64 token slots; one byte per element, E4M3 or E5M2):
 *   k_pages   [num_pages][H_kv][64 * d]: [slot/8][elem/16][slot%8][16 elements]
 *   v_pages   [num_pages][H_kv][d * 64]: [chan/8][slot/16][chan%8][16 slots]
 *   kv_scales [num_pages][H_kv][2][4] fp32: [0][i] the scale of the keys, [1][i] of
 *             the values in slots 16 i .. 16 i + 15 of that page and head
 * A value is its code times its block's scale.  The pages are tcgen05 operands as
 * they stand (K-major, no swizzle: the key tile is the A operand of S^T = K q^T,
 * the value tile that of O^T = V^T P^T), so they go to shared memory with one bulk
 * copy each and are never converted.  Scales are not negative and below 2^127, or
 * NaN; bdfp8_append writes powers of two, or NaN with codes of 0.
 *
 * Supported: d in {64, 128}, any H_q that is a multiple of H_kv; other head
 * dims return BDFP4_ERR_UNSUPPORTED.  Pages, the open rows and the workspace are
 * 128-byte aligned, kv_scales 32-byte, q / k / v / outputs and cos_sin 16-byte,
 * with token strides that are multiples of 8 elements (BDFP4_ERR_ALIGN).
 */
#ifndef BDFP8_H
#define BDFP8_H

#include "bdfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { BDFP8_E4M3 = 0, BDFP8_E5M2 = 1 } bdfp8_fmt;

/* a bit of *dev_status beside those of bdfp4.h: a position outside [0, max_pos) */
#define BDFP8_DEV_BAD_POSITION 16

/* bdfp8_append's pairing of rotated elements */
#define BDFP8_ROTATE_HALVES 0   /* element i with element i + rot_dim / 2 */
#define BDFP8_ROTATE_ADJACENT 1 /* element 2 i with element 2 i + 1       */

/*
 * Append the new tokens of B sequences to the cache, rotating their keys (and,
 * with q, their queries) by position.
 *
 * Tokens of all sequences stand one after another: sequence b has rows
 * cu_tokens[b] .. cu_tokens[b+1]-1 of k, v (and q, q_out), possibly none, and
 * they become its tokens seq_lens[b] - n .. seq_lens[b] - 1, n = cu_tokens[b+1] -
 * cu_tokens[b] (seq_lens counts them).  Rows from cu_tokens[B] on are not
 * touched.  k [T][H_kv][d], v [T][H_kv][d], q [T][H_q][d] with token strides of
 * k_stride, v_stride, q_stride elements (heads contiguous: column ranges of one
 * projection's output); q_out [T][H_q][d] contiguous, apart from q; q = q_out =
 * NULL rotates no queries.
 *
 * Rotation: row p of cos_sin [max_pos][rot_dim] fp32 holds rot_dim / 2 cosines,
 * then as many sines, of position p: positions[t] where positions [T] is given,
 * else the token's index in its sequence.  A pair (x, y) becomes
 * (x cos - y sin, y cos + x sin); elements from rot_dim on stay.  rot_dim is a
 * multiple of 16 from 16 to d, or 0 for no rotation (cos_sin may then be NULL).
 * Rotated queries are rounded to bf16 once; rotated keys stay fp32 until they
 * become codes.
 *
 * Quantization, per KV head and 16 consecutive tokens of a sequence: s = the
 * smallest power of two, at least 2^-126, with amax <= top s (top = 448 or
 * 57344; s = 1 for a block of zeros), code = x / s to nearest, ties to even.
 * Slots of a written block past the sequence's end become code 0.  A block with
 * an infinity or a NaN gets scale NaN and codes 0: rows that see it are NaN.
 *
 * A block that is not full is quantized again when tokens join it, from the
 * caller-owned open rows, so that a block's bytes do not depend on how its
 * tokens arrived: k_open [B][16][H_kv][d] fp32 (rotated keys) and v_open
 * [B][16][H_kv][d] bf16, row i = token with index % 16 == i of the sequence's
 * last block.  The call reads rows 0 .. (first new index % 16) - 1 and writes the
 * rows of its new tokens in the last block.  A sequence that starts at a whole
 * block (a new prompt) needs nothing in them.
 *
 * Errors on the device: cu_tokens out of order or out of [0, T] or seq_lens out of
 * [n, 64 max_pages_per_seq] (BDFP4_DEV_BAD_SEQLEN: the sequence is skipped,
 * its q_out rows too; entries of cu_tokens that are not in order also leave it open
 * which tokens of the call's other sequences are appended), a block_table entry out of range (BDFP4_DEV_BAD_PAGE: the block
 * is not written, its open rows are), a position out of range
 * (BDFP8_DEV_BAD_POSITION: the token counts as unrotated).  Sequences must not
 * share a page that the call writes.
 */
BDFP4_API int bdfp8_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const void* q,
                           int64_t q_stride, void* q_out, const int32_t* cu_tokens, const int32_t* seq_lens,
                           const int32_t* positions, const float* cos_sin, int rot_dim, int max_pos, int pairing,
                           float* k_open, void* v_open, const int32_t* block_table, int B, int T, int H_q, int H_kv,
                           int d, int max_pages_per_seq, int64_t num_pages, bdfp8_fmt fmt, void* k_pages,
                           void* v_pages, float* kv_scales, int32_t* dev_status, void* stream);

/*
 * Split plan for bdfp8_decode: tiles (128 tokens) per split, from the host's
 * copy of the lengths.  The arguments are those of the decode call.  Returns
 * chunk_tiles >= 1, or a negative status.
 */
BDFP4_API int bdfp8_decode_plan(const int32_t* host_seq_lens, int B, int T_q, int H_q, int H_kv, int d, int window,
                                int sinks, int num_sms);

/* Bytes of workspace bdfp8_decode needs for this shape and chunk_tiles (> 0): the
 * splits' fp32 partial outputs and (m, l) pairs; 0 where every row has one split.
 * Contents need no initialisation; calls that run at the same time must not
 * share a workspace. */
BDFP4_API size_t bdfp8_decode_workspace_size(int B, int T_q, int H_q, int H_kv, int d, int max_pages_per_seq,
                                             int window, int sinks, int chunk_tiles);

/*
 * Decode attention over the 8-bit cache for the T_q >= 1 newest tokens of each
 * sequence (already appended), causally:
 *   out[b][i][h] = sum_t softmax_t(sm_scale q[b][i][h] . k_t) v_t
 * over the tokens t that query token i, at index p = N_b - T_q + i (N_b =
 * seq_lens[b]), sees: t <= p and, with window > 0, t > p - window or t < sinks.
 * window = 0 sees the whole context (sinks is then unused).
 * q, out [B][T_q][H_q][d] bf16; query head h reads KV head h / (H_q / H_kv);
 * block_table [B][max_pages_per_seq] int32.  Entries of pages that no query
 * token of the sequence sees are never read as pages (a streaming cache may have given
 * them back; write -1 or leave them).  Tokens that a row does not see, slots past
 * the end and pages with a bad entry (BDFP4_DEV_BAD_PAGE) have no influence,
 * whatever their bytes and scales; but a value code that is an infinity or a NaN, in a
 * token that some row of the sequence sees, may reach its other rows too.
 *
 * Arithmetic: a query row is split into two E4M3 terms, exact for a bf16 element
 * down to 2^-9 of the row's largest (2^-13 with up to 16 rows), to 2^-17 of the
 * largest below; logits, softmax and sums are fp32; a probability times its value
 * block's scale (rounded up to a power of two, 2^-92 at the least) goes into the value
 * product as three E5M2 terms: relative error 2^-9, a floor of 2^-28 of the largest such
 * product among the tokens of a split that the row sees.  (A token whose product is
 * below 2^-148 of that one's leaves the sum of probabilities too.)  A value block of
 * scale 1 whose codes in tokens that a row sees are all zeros, as bdfp8_append leaves a
 * block of zeros, counts as one of scale 0 in this.  Up to 16 G T_q rows
 * of a KV head take one kernel, more another that works on 128 rows at a time.
 *
 * An empty sequence and a row that sees no token give zeros; 0 < N_b < T_q also
 * sets BDFP4_DEV_BAD_SEQLEN (rows at negative indexes see nothing), N_b outside
 * [0, 64 max_pages_per_seq] sets it and gives zeros.  chunk_tiles <= 0 plans
 * from max_pages_per_seq.  workspace as bdfp8_decode_workspace_size says (NULL
 * where that is 0; what it says of chunk_tiles = 1 covers every plan), else
 * BDFP4_ERR_WORKSPACE.
 */
BDFP4_API int bdfp8_decode(const void* q, const void* k_pages, const void* v_pages, const float* kv_scales,
                           const int32_t* block_table, const int32_t* seq_lens, int B, int T_q, int H_q, int H_kv,
                           int d, int max_pages_per_seq, int64_t num_pages, bdfp8_fmt fmt, int window, int sinks,
                           float sm_scale, int chunk_tiles, void* workspace, size_t workspace_bytes, void* out,
                           int32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BDFP8_H */
