// attn_capi.cu -- the extern "C" boundary of the attention half (moe_attn.h):
// argument checks and launches.
#include "attn.h"

using namespace moe;

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

moe_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool block_size_ok(int bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }

moe_status_t check_ws(const void *ws, size_t ws_bytes, size_t need) {
    if (!ws)
        return MOE_ERR_INVALID_ARG;
    if (!aligned(ws, 256))
        return MOE_ERR_MISALIGNED;
    return ws_bytes < need ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

moe_status_t check_device(int *sms) {
    const moe_status_t st = current_device_sms(sms);
    if (st == MOE_OK)
        (void)cudaGetLastError();
    return st;
}

moe_status_t check_cache(const moe_kv_cache_t *c) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || c->num_blocks <= 0 || c->kv_heads <= 0)
        return MOE_ERR_INVALID_ARG;
    if ((c->head_dim != 64 && c->head_dim != 128) || !block_size_ok(c->block_size) || c->kv_heads > 1024)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16))
        return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

moe_status_t check_attention_sizes(int T, int B, int q_heads, int kv_heads, int head_dim) {
    if (T < 0 || B < 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0)
        return MOE_ERR_INVALID_ARG;
    if (T > kMaxAttnTokens || B > kMaxRequests || kv_heads > 1024 || q_heads / kv_heads > 256 ||
        (head_dim != 64 && head_dim != 128))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

moe_status_t check_linear_sizes(int T, int N, int K) {
    if (T < 0 || N <= 0 || K <= 0)
        return MOE_ERR_INVALID_ARG;
    if (T > kMaxAttnTokens || N > (1 << 20) || K > 65536 || K % 16 != 0)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_kv_build_tables(const int32_t *ctx_lens, const int32_t *new_lens, int B, int T, int block_size,
                                 const int32_t *free_blocks, int num_free, const int32_t *free_head,
                                 int32_t *block_table, int max_blocks, int32_t *kv_lens, int32_t *q_offsets,
                                 int64_t *slot_map, int32_t *positions, int32_t *free_head_out, void *ws,
                                 size_t ws_bytes, cudaStream_t stream) {
    if (B < 0 || T < 0 || num_free < 0 || max_blocks < 0 || !free_head || !q_offsets || !free_head_out ||
        free_head == free_head_out)
        return MOE_ERR_INVALID_ARG;
    if (B > 0 && (!ctx_lens || !new_lens || !kv_lens || (max_blocks > 0 && !block_table)))
        return MOE_ERR_INVALID_ARG;
    if ((T > 0 && (!slot_map || !positions)) || (num_free > 0 && !free_blocks))
        return MOE_ERR_INVALID_ARG;
    if (!block_size_ok(block_size) || B > kMaxRequests || T > kMaxTableTokens ||
        (long long)max_blocks * block_size > 0x7FFFFFFFll)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(free_blocks, 4) || !aligned(free_head, 4) ||
        !aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(q_offsets, 4) || !aligned(slot_map, 8) ||
        !aligned(positions, 4) || !aligned(free_head_out, 4))
        return MOE_ERR_MISALIGNED;
    moe_status_t st = check_ws(ws, ws_bytes, kHdrWords * sizeof(uint32_t));
    int sms = 0;
    if (st != MOE_OK || (st = check_device(&sms)) != MOE_OK)
        return st;
    int shift = 4;
    while ((1 << shift) < block_size)
        ++shift;
    const TablesProblem p{ctx_lens, new_lens, B, T, shift, free_blocks, num_free, free_head, block_table, max_blocks,
                          kv_lens, q_offsets, slot_map, positions, free_head_out, ws_at<uint32_t>(ws, 0)};
    return from_cuda(launch_kv_tables(p, stream));
}

moe_status_t moe_kv_append(const uint16_t *k, int64_t k_stride_t, int64_t k_stride_h, const uint16_t *v,
                           int64_t v_stride_t, int64_t v_stride_h, const int64_t *slot_map, int T,
                           const moe_kv_cache_t *cache, void *ws, size_t ws_bytes, cudaStream_t stream) {
    moe_status_t st = check_cache(cache);
    if (st != MOE_OK)
        return st;
    if (T < 0 || k_stride_t < 0 || k_stride_h < 0 || v_stride_t < 0 || v_stride_h < 0)
        return MOE_ERR_INVALID_ARG;
    if (T > kMaxTableTokens)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0)
        return MOE_OK;
    if (!k || !v || !slot_map)
        return MOE_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 8) || k_stride_t % 8 || k_stride_h % 8 ||
        v_stride_t % 8 || v_stride_h % 8)
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((st = check_ws(ws, ws_bytes, kHdrWords * sizeof(uint32_t))) != MOE_OK || (st = check_device(&sms)) != MOE_OK)
        return st;
    const AppendProblem p{k, v, k_stride_t, k_stride_h, v_stride_t, v_stride_h, slot_map, T, *cache, ws_at<uint32_t>(ws, 0)};
    return from_cuda(launch_kv_append(p, stream));
}

size_t moe_kv_attention_workspace_size(int T, int B, int q_heads, int kv_heads, int head_dim) {
    if (check_attention_sizes(T, B, q_heads, kv_heads, head_dim) != MOE_OK)
        return 0;
    return AttnLayout::make(T, B, q_heads, kv_heads, head_dim).total;
}

moe_status_t moe_kv_attention(const uint16_t *q, int64_t q_stride_t, int64_t q_stride_h, int T, int q_heads,
                              const moe_kv_cache_t *cache, const int32_t *block_table, int max_blocks,
                              const int32_t *q_offsets, const int32_t *kv_lens, int B, float softmax_scale,
                              int causal, int window, uint16_t *out, float *lse, void *ws, size_t ws_bytes,
                              cudaStream_t stream) {
    moe_status_t st = check_cache(cache);
    if (st != MOE_OK || (st = check_attention_sizes(T, B, q_heads, cache->kv_heads, cache->head_dim)) != MOE_OK)
        return st;
    if (max_blocks < 0 || window < 0 || (causal != 0 && causal != 1) || q_stride_t < 0 || q_stride_h < 0 ||
        !(softmax_scale >= 0.0f) || softmax_scale > 3.0e38f)
        return MOE_ERR_INVALID_ARG;
    if ((long long)max_blocks * cache->block_size > 0x7FFFFFFFll - 256)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || B == 0)
        return MOE_OK;
    if (!q || !out || !q_offsets || !kv_lens || (max_blocks > 0 && !block_table))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(q, 8) || !aligned(out, 8) || !aligned(lse, 4) || !aligned(q_offsets, 4) || !aligned(kv_lens, 4) ||
        !aligned(block_table, 4) || q_stride_t % 4 || q_stride_h % 4)
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((st = check_ws(ws, ws_bytes, AttnLayout::make(T, B, q_heads, cache->kv_heads, cache->head_dim).total)) != MOE_OK ||
        (st = check_device(&sms)) != MOE_OK)
        return st;
    const AttnProblem p{q, q_stride_t, q_stride_h, T, q_heads, *cache, block_table, max_blocks, q_offsets, kv_lens, B,
                        softmax_scale, causal, window, out, lse};
    return from_cuda(launch_kv_attention(p, ws, sms, stream));
}

moe_status_t moe_quantize_fp8_weight(const uint16_t *w, int N, int K, uint8_t *codes, uint8_t *scale,
                                     cudaStream_t stream) {
    moe_status_t st = check_linear_sizes(0, N, K);
    if (st != MOE_OK)
        return st;
    if (!w || !codes || !scale)
        return MOE_ERR_INVALID_ARG;
    if (!aligned(w, 16) || !aligned(codes, 16))
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((st = check_device(&sms)) != MOE_OK)
        return st;
    return from_cuda(launch_quantize_fp8_weight(w, N, K, codes, scale, stream));
}

size_t moe_linear_fp8_workspace_size(int T, int N, int K) {
    return check_linear_sizes(T, N, K) == MOE_OK ? linear_fp8_workspace(T, N, K) : 0;
}

moe_status_t moe_linear_fp8(const uint16_t *x, int64_t ldx, int T, const uint8_t *codes, const uint8_t *scale, int N,
                            int K, uint16_t *y, void *ws, size_t ws_bytes, cudaStream_t stream) {
    moe_status_t st = check_linear_sizes(T, N, K);
    if (st != MOE_OK)
        return st;
    if (T == 0)
        return MOE_OK;
    if (!x || !codes || !scale || !y || (T > 1 && ldx < K))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(y, 16) || ldx % 8)
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((st = check_ws(ws, ws_bytes, linear_fp8_workspace(T, N, K))) != MOE_OK || (st = check_device(&sms)) != MOE_OK)
        return st;
    const LinearProblem p{x, ldx, codes, scale, y, T, N, K};
    return from_cuda(launch_linear_fp8(p, ws, sms, stream));
}

}  // extern "C"
