/*
 * moe_attn.h -- C ABI of the attention half of a decoder layer in 8 bits, the
 * work that runs between two MoE layers (moe_fp4.h) of a serving step:
 *
 *   b1  block tables   blocks of a paged cache given out to the requests of a
 *                      step, and the cache slot of every new token
 *   b2  append         new keys and values into the E4M3 cache
 *   b3  attention      of the new tokens over the cache
 *   b4  projection     y = x W^T with E4M3 operands, block-scaled
 *
 * Conventions are those of moe_fp4.h: row-major tensors, DEVICE pointers owned
 * by the caller, calls that enqueue kernels on `stream` and return without
 * synchronising, argument errors found on the host before anything is
 * enqueued, device-side errors recorded in the status word of the workspace
 * (moe_check_device_status), a workspace that is zero-filled or passed through
 * moe_workspace_init once before its first use, and calls that share one
 * workspace not overlapping on the GPU.  One workspace may serve these calls
 * and the MoE layer's.  All calls can be captured in CUDA graphs.
 *
 * The 8-bit format.  A group of values whose largest finite magnitude is a
 * is stored as E4M3 codes (OCP: bias 7, largest 448, no infinities) with one
 * E8M0 byte s: code = E4M3 nearest-even of v / 2^e, s = e + 127, where e is
 * the smallest exponent with a <= 448 * 2^e, at least -126.  Nothing
 * saturates, and v / 2^e is exact: a power-of-two scale moves a value's
 * exponent only, so it costs a floating-point code no precision (other than in
 * its subnormal range) and needs no division.  Values that are not finite are stored as the NaN
 * code 0x7F and do not count towards a.  Groups: a token's 128
 * consecutive x (b4), a 128 x 128 block of W (b4), the tokens of one cache
 * block and head (b2).
 *
 * The cache.  Blocks of block_size tokens (16, 32, 64 or 128).  With sub-blocks
 * of 16 tokens:
 *   k        uint8 [num_blocks][kv_heads][block_size/16][head_dim/16][16 tokens][16 dims]
 *   v        uint8 [num_blocks][kv_heads][block_size/16][head_dim][16 tokens]
 *   k_scale, v_scale  uint8 [num_blocks][kv_heads]
 * so a sub-block is 16 * head_dim consecutive bytes, and the innermost 16 bytes
 * run along the axis that the product over that operand sums (dims for the
 * scores, tokens for the values): 8 such rows are one tensor-core operand tile.
 * Slots past a request's length may hold anything.
 */
#ifndef MOE_ATTN_H
#define MOE_ATTN_H

#include "moe_fp4.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    uint8_t *k;             /* 16-byte aligned */
    uint8_t *v;             /* 16-byte aligned */
    uint8_t *k_scale;
    uint8_t *v_scale;
    int32_t num_blocks;     /* 1 .. 2^31-1 */
    int32_t kv_heads;       /* 1 .. 1024 */
    int32_t head_dim;       /* 64 or 128 */
    int32_t block_size;     /* 16, 32, 64 or 128 */
} moe_kv_cache_t;

/*
 * b1: the tables of one step of B requests.  Request b has ctx_lens[b] tokens
 * in the cache and brings new_lens[b] >= 0 new ones; it holds
 * ceil(ctx / block_size) blocks, the first entries of its row of block_table
 * [B, max_blocks].  The blocks it lacks are taken, in request order, from
 * free_blocks [num_free] at *free_head onwards and written behind them (the
 * other entries of the row are left alone); *free_head_out = *free_head +
 * blocks taken.  Further outputs: kv_lens [B] = ctx + new, q_offsets [B+1] the
 * exclusive sums of new_lens, slot_map int64 [T] = block * block_size + offset
 * and positions int32 [T] = position in the request, of the new tokens in
 * request order; both are -1 past the last new token (T >= their number, so
 * that a captured step can be replayed with fewer).  The inputs stay as they are, so
 * the call can be repeated.  free_head_out must not be free_head.
 * Device-side errors (MOE_ERR_DEVICE_ASSERT; nothing is written): a negative
 * length, a request longer than max_blocks * block_size, more than T new
 * tokens, a free list that is too short.  B <= 8192, T <= 2^24.  ws: 512 bytes or more.
 */
moe_status_t moe_kv_build_tables(const int32_t *ctx_lens, const int32_t *new_lens, int B, int T, int block_size,
                                 const int32_t *free_blocks, int num_free, const int32_t *free_head,
                                 int32_t *block_table, int max_blocks, int32_t *kv_lens, int32_t *q_offsets,
                                 int64_t *slot_map, int32_t *positions, int32_t *free_head_out, void *ws,
                                 size_t ws_bytes, cudaStream_t stream);

/*
 * b2: writes T tokens' keys and values (bf16; element (t, h, i) at
 * t * stride_t + h * stride_h + i, strides in elements and multiples of 8,
 * pointers 16-byte aligned) into the cache at slot_map [T] (as moe_kv_build_tables makes
 * it: the tokens of a block follow one another in slot_map, with no other slot
 * between them, and in the block; a negative slot is skipped; the range-checked build reports slots that break this).  Each (block, head) has one exponent for its keys
 * and one for its values.  A token at offset 0 starts the block anew.  Where
 * the block holds earlier tokens, its exponent becomes the larger of its own and
 * what the new tokens need, and if it grew the earlier tokens' codes are
 * rounded to it (exact, but for codes that reach the subnormal range).  A slot
 * past the cache is skipped and recorded (MOE_ERR_DEVICE_ASSERT).  The result
 * does not depend on the order of execution.  ws: 512 bytes or more.
 */
moe_status_t moe_kv_append(const uint16_t *k, int64_t k_stride_t, int64_t k_stride_h, const uint16_t *v,
                           int64_t v_stride_t, int64_t v_stride_h, const int64_t *slot_map, int T,
                           const moe_kv_cache_t *cache, void *ws, size_t ws_bytes, cudaStream_t stream);

/* Bytes of workspace of moe_kv_attention for up to T new tokens of up to B
 * requests; 0 for sizes that it does not take. */
size_t moe_kv_attention_workspace_size(int T, int B, int q_heads, int kv_heads, int head_dim);

/*
 * b3: softmax attention of the new tokens over the cache, which holds them
 * already (b2 comes first).  q bf16 (element (t, h, i) at t * stride_t +
 * h * stride_h + i; strides multiples of 4, pointer 8-byte aligned); query head h reads
 * key/value head h / (q_heads / kv_heads).  Request b's tokens are rows
 * q_offsets[b] .. q_offsets[b+1] of q, the last positions of its kv_lens[b]
 * tokens: row i of n is at position p = kv_len - n + i and sees the positions
 * j < kv_len with j <= p if causal, and j > p - window if window > 0.
 *   out [T, q_heads, head_dim] bf16 = sum_j softmax_j(softmax_scale q.k_j) v_j
 *   lse [T, q_heads] fp32 or NULL   = log sum_j exp(softmax_scale q.k_j)
 * A row that sees nothing gives zeros and -infinity.  What it does not see has no
 * influence, NaN included, and table entries of blocks that no row sees (past the request's
 * end, before its window) are not read.  Rows of q past q_offsets[B] give no output.  Products of bf16 q and
 * E4M3 codes are exact (of q down to 2^-39 of its row's largest element), sums and softmax statistics fp32.  The softmax weights
 * are rounded to f16: a weight times its block's 2^exponent to 2^-11 of itself or 2^-29 of the row's largest such product, which is one for
 * all dims.  So a block whose exponent lies more than about 20 binades above the others' costs those precision in every dim, also
 * where it is small itself.  The same arguments give the same bits on the same device.
 * Scores may be of any size that fp32 holds; a row whose largest score leaves that range is NaN.
 * Device-side errors (MOE_ERR_DEVICE_ASSERT): q_offsets that decrease or leave 0..T, a
 * kv_len outside 0..max_blocks * block_size (out stays untouched); a block id outside the
 * cache (that block is read as block 0).  B <= 8192, T <= 2^20,
 * q_heads / kv_heads <= 256.  Two
 * launches at most.
 */
moe_status_t moe_kv_attention(const uint16_t *q, int64_t q_stride_t, int64_t q_stride_h, int T, int q_heads,
                              const moe_kv_cache_t *cache, const int32_t *block_table, int max_blocks,
                              const int32_t *q_offsets, const int32_t *kv_lens, int B, float softmax_scale,
                              int causal, int window, uint16_t *out, float *lse, void *ws, size_t ws_bytes,
                              cudaStream_t stream);

/*
 * Weights of b4 from bf16 (load-time): w [N, K] bf16 -> codes [N, K] E4M3 and
 * scale [ceil(N/128), ceil(K/128)] E8M0 bytes, one for each 128 x 128 block.
 * K a multiple of 16.  w, codes 16-byte aligned.
 */
moe_status_t moe_quantize_fp8_weight(const uint16_t *w, int N, int K, uint8_t *codes, uint8_t *scale,
                                     cudaStream_t stream);

/* Bytes of workspace of moe_linear_fp8 for up to T tokens; 0 for sizes that it does not take. */
size_t moe_linear_fp8_workspace_size(int T, int N, int K);

/*
 * b4: y [T, N] bf16 = X^ W^T.  X^ is x [T, K] (bf16, rows ldx elements apart)
 * quantised in groups of 128 along K, inside the call; W the codes and scales above.
 * The products are exact, summed in fp32 by the tensor cores, rounded
 * once.  A token with a value that is not finite gives NaN.  K a multiple of 16, ldx a
 * multiple of 8; x, codes, y 16-byte aligned; T <= 2^20, N <= 2^20, K <= 65536.
 */
moe_status_t moe_linear_fp8(const uint16_t *x, int64_t ldx, int T, const uint8_t *codes, const uint8_t *scale, int N,
                            int K, uint16_t *y, void *ws, size_t ws_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ATTN_H */
