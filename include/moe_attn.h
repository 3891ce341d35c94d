/*
 * moe_attn.h -- C ABI of the attention half of a decoder layer in 8 bits, the
 * work that runs between two MoE layers (moe_fp4.h) of a serving step:
 *
 *   b1  block tables   blocks of a paged cache given out to the requests of a
 *                      step, and the cache slot of every new token
 *   b2  append         new keys and values into the E4M3 cache
 *   b3  attention      of the new tokens over the cache
 *   b4  projection     y = x W^T with E4M3 operands, block-scaled
 *   b5  norm           residual sum and root-mean-square norm before and after a block
 *   b6  rotary         rotary positions on query and key heads
 *   b7  latent append  a latent vector and a rotary key for each new token into a paged cache
 *   b8  latent attention  of the new tokens over that cache, in its absorbed form
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

/*
 * b5: rows of H, for each of T tokens
 *   u = x, or x * rms(x) * post_weight if post_weight is given   (the norm after a block)
 *   h = residual + scale * gate * u                              (residual, gate: none is 0, 1)
 *   residual_out = h,  y = h * rms(h) * weight                   (the norm before the next block)
 * with rms(v) = 1 / sqrt(mean of v^2 + eps).  All in fp32, h for y not rounded first.  x bf16, rows ldx elements apart;
 * post_weight, weight bf16 [H]; gate bf16, rows ld_gate elements apart, or 0 for one row for all tokens; residual and residual_out [T, H]
 * bf16, or fp32 if residual_f32; y bf16 [T, H].  residual, residual_out, gate and post_weight may be NULL; y and weight may
 * be NULL together, if residual_out is given.  residual_out may be residual, y may be x where ldx is H (refused otherwise).  A row with a value that is not
 * finite, or whose squares overflow, is as the formulas give it in fp32; no other row is touched by it.
 * H a multiple of 8 up to 32768, T <= 2^20; pointers 16-byte aligned, ldx and ld_gate multiples of 8.
 */
moe_status_t moe_rms_norm(const uint16_t *x, int64_t ldx, int T, int H, const uint16_t *post_weight, const uint16_t *gate,
                          int64_t ld_gate, float scale, const void *residual, void *residual_out, int residual_f32,
                          const uint16_t *weight, float eps, uint16_t *y, cudaStream_t stream);

/*
 * b6: rotary positions.  A head's dims offset .. offset + 2 pairs - 1 are `pairs` pairs (a_i, b_i): halves (a_i = dim i, b_i = dim
 * pairs + i of them) or, if interleaved, neighbours (dims 2i, 2i + 1).  At position p
 *   a' = amplitude (a cos t - b sin t),  b' = amplitude (b cos t + a sin t),  t = 2 pi p turns[i] 2^-64
 * turns[i] being the pair's frequency in units of 2^-64 turns a position: p turns[i] modulo 2^64 is the exact angle, at any position.
 * With q_norm (k_norm), bf16 [head_dim], a head v is v * rms(v) * norm first, all of its dims; other dims are as they were.
 * fp32, rounded once.  q, q_out bf16, element (t, h, i) at t * stride_t + h * stride_h + i; k the same with k_heads heads (0: none).
 * q_out may be q and k_out k, with the same strides; otherwise outputs overlap no input.  An output's rows share no value (strides that
 * would have them do so are refused).  A token whose position is negative (as moe_kv_build_tables marks those behind the last) is left
 * out: nothing is written.
 * head_dim a multiple of 8 up to 256; pairs and offset multiples of 8, offset + 2 pairs <= head_dim; up to 1024 heads each; T <= 2^20;
 * pointers 16-byte aligned (positions 4, turns 8), strides multiples of 8.
 */
moe_status_t moe_rotary(const uint16_t *q, int64_t q_stride_t, int64_t q_stride_h, uint16_t *q_out, int64_t q_out_stride_t,
                        int64_t q_out_stride_h, int q_heads, const uint16_t *k, int64_t k_stride_t, int64_t k_stride_h,
                        uint16_t *k_out, int64_t k_out_stride_t, int64_t k_out_stride_h, int k_heads, int T, int head_dim,
                        const int32_t *positions, const uint64_t *turns, int pairs, float amplitude, int interleaved, int offset,
                        const uint16_t *q_norm, const uint16_t *k_norm, float eps, cudaStream_t stream);

/* The paged cache of b7 and b8: a token's latent vector c (latent_dim values) and its rotary key (64) side by side,
 *   data  bf16 [num_blocks][block_size][latent_dim + 64]
 * Slots past a request's length may hold anything. */
typedef struct {
    uint16_t *data;         /* 16-byte aligned */
    int32_t num_blocks;     /* 1 .. 2^31-1, num_blocks * block_size <= 2^31-1 */
    int32_t latent_dim;     /* 256 or 512 */
    int32_t block_size;     /* 16, 32, 64 or 128 */
} moe_latent_cache_t;

/*
 * b7: writes T tokens' latent vectors c (bf16, rows ldc elements apart) and rotary keys k (bf16 [64], rows ldk apart) to the slots
 * slot_map [T] (block * block_size + offset; a negative one is skipped) of the cache.  With norm (bf16 [latent_dim])
 * c * rms(c) * norm is written; with turns (32 of them) k is rotated to positions [T] as b6 does, and a token whose position is negative is
 * left out as there, its latent vector too; without, k as it is.  Both NULL or neither of positions and turns.  A slot past the cache is skipped and recorded (MOE_ERR_DEVICE_ASSERT).  Where two tokens
 * have one slot, either's values may be there afterwards.  T <= 2^24; c, k, norm 16-byte aligned, ldc and ldk multiples of 8.
 * ws: 512 bytes or more.
 */
moe_status_t moe_latent_append(const uint16_t *c, int64_t ldc, const uint16_t *k, int64_t ldk, const int64_t *slot_map, int T,
                               const int32_t *positions, const uint64_t *turns, float amplitude, int interleaved,
                               const uint16_t *norm, float eps, const moe_latent_cache_t *cache, void *ws, size_t ws_bytes,
                               cudaStream_t stream);

/* Bytes of workspace of moe_latent_attention for any step of up to T new tokens of up to B requests; 0 for sizes that it does not take. */
size_t moe_latent_attention_workspace_size(int T, int B, int heads, int latent_dim);

/*
 * b8: softmax attention of the new tokens over the latent cache, which holds them already.  All heads share a token's latent vector
 * c_j and rotary key r_j; the products with the matrices that make a head's keys and values from c_j are absorbed into the
 * query (before) and the output (after), so that
 *   x_j = softmax_scale (q_latent.c_j + q_rope.r_j)
 *   out [T, heads, latent_dim] bf16 = sum_j softmax_j(x) c_j
 *   lse [T, heads] fp32 or NULL     = log sum_j exp(x_j)
 * q_latent [T, heads, latent_dim] and q_rope [T, heads, 64] bf16, element (t, h, i) at t * stride_t + h * stride_h + i.  Rows of a request,
 * what they see (causal or not), rows that see nothing, rows past q_offsets[B], table entries that are not read and device-side errors are as in
 * moe_kv_attention.  What a row does not see has no influence, NaN included; a row that sees a token with a value that is not finite is
 * not finite in those dims at least.  Products are exact, sums and softmax statistics fp32; the weights are
 * rounded to bf16, relative to themselves, and divided by the sum of the rounded ones (lse is of the others).  Scores may be of any size that fp32 holds; a row whose largest score leaves that range is NaN.  Latent
 * values may be of magnitudes up to 2^70.  The same arguments give the same bits on the same device.
 * heads <= 256, B <= 8192, T <= 2^20, T * heads < 2^31; q and out 16-byte aligned, strides multiples of 8; out overlaps no input.  Two
 * launches; three where T and B allow more than 152 units of rows (64 rows; where T <= B a token's heads, up to 128), with more than 256 requests,
 * or with tables of more than 2^29 tokens a request.
 */
moe_status_t moe_latent_attention(const uint16_t *q_latent, int64_t ql_stride_t, int64_t ql_stride_h, const uint16_t *q_rope,
                                  int64_t qr_stride_t, int64_t qr_stride_h, int T, int heads, const moe_latent_cache_t *cache,
                                  const int32_t *block_table, int max_blocks, const int32_t *q_offsets, const int32_t *kv_lens,
                                  int B, float softmax_scale, int causal, uint16_t *out, float *lse, void *ws, size_t ws_bytes,
                                  cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ATTN_H */
