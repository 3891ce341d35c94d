// attn_capi.cu -- the extern "C" boundary of the attention half (moe_attn.h):
// argument checks and launches.
#include <mutex>

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

// Tensor maps are made by the driver, which refuses a host thread without a context, as a thread has none before its first CUDA call that
// needs one.  (A context that is there stays, whoever made it.)
bool bind_context() {
    typedef CUresult (*CurrentFn)(CUcontext *);
    static CurrentFn current = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess)
            current = reinterpret_cast<CurrentFn>(p);
    });
    CUcontext context = nullptr;
    int dev = 0;
    return current && current(&context) == CUDA_SUCCESS && (context || (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess));
}

moe_status_t check_device(int *sms) {
    const moe_status_t st = current_device_sms(sms);
    if (st != MOE_OK)
        return st;
    (void)cudaGetLastError();
    return bind_context() ? MOE_OK : MOE_ERR_CUDA;
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

moe_status_t check_latent_cache(const moe_latent_cache_t *c) {
    if (!c || !c->data || c->num_blocks <= 0)
        return MOE_ERR_INVALID_ARG;
    if ((c->latent_dim != 256 && c->latent_dim != 512) || !block_size_ok(c->block_size) ||
        (long long)c->num_blocks * c->block_size > 0x7FFFFFFFll)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return aligned(c->data, 16) ? MOE_OK : MOE_ERR_MISALIGNED;
}

moe_status_t check_latent_sizes(int T, int B, int heads, int latent_dim) {
    if (T < 0 || B < 0 || heads <= 0)
        return MOE_ERR_INVALID_ARG;
    if (T > kMaxAttnTokens || B > kMaxRequests || heads > 256 || (long long)T * heads > 0x7FFFFFFFll ||
        (latent_dim != 256 && latent_dim != 512))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

bool real_eps(float eps) { return eps >= 0.0f && eps <= 3.0e38f; }

bool finite(float v) { return v >= -3.0e38f && v <= 3.0e38f; }

// Whether rows of `dim` values of T tokens and `heads` heads, st and sh apart, share no value.
bool rows_apart(int64_t T, int64_t heads, int64_t dim, int64_t st, int64_t sh) {
    if ((T > 1 && st < dim) || (heads > 1 && sh < dim))
        return false;
    if (T == 1 || heads == 1 || (st - dim) / (heads - 1) >= sh || (sh - dim) / (T - 1) >= st)
        return true;                             // the usual ones: a token's heads lie before the next token, or a head's tokens before the next head
    for (int64_t h = 1; h < heads; ++h) {        // h heads on lies between tokens t and t + 1
        const __int128 at = (__int128)h * sh, t = at / st;
        if ((t < T && at - t * st < dim) || (t + 1 < T && (t + 1) * st - at < dim))
            return false;
    }
    return true;
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

moe_status_t moe_rms_norm(const uint16_t *x, int64_t ldx, int T, int H, const uint16_t *post_weight, const uint16_t *gate,
                          int64_t ld_gate, float scale, const void *residual, void *residual_out, int residual_f32,
                          const uint16_t *weight, float eps, uint16_t *y, cudaStream_t stream) {
    if (T < 0 || H <= 0 || !real_eps(eps) || !finite(scale) || (residual_f32 != 0 && residual_f32 != 1))
        return MOE_ERR_INVALID_ARG;
    if (T > kMaxAttnTokens || H > kMaxNormDims || H % 8 != 0)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0)
        return MOE_OK;
    if (!x || !y != !weight || (!y && !residual_out) || (T > 1 && ldx < H) || (gate && T > 1 && ld_gate != 0 && ld_gate < H))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(post_weight, 16) || !aligned(gate, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) ||
        !aligned(weight, 16) || !aligned(y, 16) || ldx % 8 || ld_gate % 8)
        return MOE_ERR_MISALIGNED;
    if (y == x && T > 1 && ldx != H)             // rows of y would lie on other rows of x, which may not have been read
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    const moe_status_t st = check_device(&sms);
    if (st != MOE_OK)
        return st;
    const NormProblem p{x, ldx, T, H, post_weight, gate, ld_gate, scale, residual, residual_out, residual_f32, weight, eps, y};
    return from_cuda(launch_rms_norm(p, sms, stream));
}

moe_status_t moe_rotary(const uint16_t *q, int64_t q_stride_t, int64_t q_stride_h, uint16_t *q_out, int64_t q_out_stride_t,
                        int64_t q_out_stride_h, int q_heads, const uint16_t *k, int64_t k_stride_t, int64_t k_stride_h,
                        uint16_t *k_out, int64_t k_out_stride_t, int64_t k_out_stride_h, int k_heads, int T, int head_dim,
                        const int32_t *positions, const uint64_t *turns, int pairs, float amplitude, int interleaved, int offset,
                        const uint16_t *q_norm, const uint16_t *k_norm, float eps, cudaStream_t stream) {
    if (T < 0 || q_heads <= 0 || k_heads < 0 || head_dim <= 0 || pairs <= 0 || offset < 0 || !finite(amplitude) || !real_eps(eps) ||
        (interleaved != 0 && interleaved != 1))
        return MOE_ERR_INVALID_ARG;
    const int64_t strides[] = {q_stride_t, q_stride_h, q_out_stride_t, q_out_stride_h, k_stride_t, k_stride_h, k_out_stride_t, k_out_stride_h};
    bool odd = false;
    for (int i = 0; i < (k_heads > 0 ? 8 : 4); ++i) {
        if (strides[i] < 0)
            return MOE_ERR_INVALID_ARG;
        odd |= strides[i] % 8 != 0;
    }
    if (T > kMaxAttnTokens || q_heads > 1024 || k_heads > 1024 || head_dim > 256 || head_dim % 8 || pairs % 8 || offset % 8 ||
        offset + 2 * (int64_t)pairs > head_dim)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0)
        return MOE_OK;
    if (!q || !q_out || !positions || !turns || (k_heads > 0 && (!k || !k_out)))
        return MOE_ERR_INVALID_ARG;
    if ((q == q_out && (q_stride_t != q_out_stride_t || q_stride_h != q_out_stride_h)) ||
        (k_heads > 0 && k == k_out && (k_stride_t != k_out_stride_t || k_stride_h != k_out_stride_h)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(q_out, 16) || (k_heads > 0 && (!aligned(k, 16) || !aligned(k_out, 16))) || !aligned(positions, 4) ||
        !aligned(turns, 8) || !aligned(q_norm, 16) || (k_heads > 0 && !aligned(k_norm, 16)) || odd)
        return MOE_ERR_MISALIGNED;
    if (!rows_apart(T, q_heads, head_dim, q_out_stride_t, q_out_stride_h) ||
        (k_heads > 0 && !rows_apart(T, k_heads, head_dim, k_out_stride_t, k_out_stride_h)))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    const moe_status_t st = check_device(&sms);
    if (st != MOE_OK)
        return st;
    const RotaryProblem p{{q, q_stride_t, q_stride_h, q_out, q_out_stride_t, q_out_stride_h, q_heads, q_norm},
                          {k, k_stride_t, k_stride_h, k_out, k_out_stride_t, k_out_stride_h, k_heads, k_norm},
                          T, head_dim, positions, turns, pairs, amplitude, interleaved, offset, eps};
    return from_cuda(launch_rotary(p, sms, stream));
}

moe_status_t moe_latent_append(const uint16_t *c, int64_t ldc, const uint16_t *k, int64_t ldk, const int64_t *slot_map, int T,
                               const int32_t *positions, const uint64_t *turns, float amplitude, int interleaved,
                               const uint16_t *norm, float eps, const moe_latent_cache_t *cache, void *ws, size_t ws_bytes,
                               cudaStream_t stream) {
    moe_status_t st = check_latent_cache(cache);
    if (st != MOE_OK)
        return st;
    if (T < 0 || ldc < 0 || ldk < 0 || !finite(amplitude) || !real_eps(eps) || (interleaved != 0 && interleaved != 1))
        return MOE_ERR_INVALID_ARG;
    if (T > kMaxTableTokens)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0)
        return MOE_OK;
    if (!c || !k || !slot_map || !positions != !turns)
        return MOE_ERR_INVALID_ARG;
    if (!aligned(c, 16) || !aligned(k, 16) || !aligned(slot_map, 8) || !aligned(positions, 4) || !aligned(turns, 8) || !aligned(norm, 16) ||
        ldc % 8 || ldk % 8)
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((st = check_ws(ws, ws_bytes, kHdrWords * sizeof(uint32_t))) != MOE_OK || (st = check_device(&sms)) != MOE_OK)
        return st;
    const LatentAppendProblem p{c, ldc, k, ldk, slot_map, T, positions, turns, amplitude, interleaved, norm, eps, *cache, ws_at<uint32_t>(ws, 0)};
    return from_cuda(launch_latent_append(p, sms, stream));
}

size_t moe_latent_attention_workspace_size(int T, int B, int heads, int latent_dim) {
    return check_latent_sizes(T, B, heads, latent_dim) == MOE_OK ? latent_attention_workspace(T, B, heads, latent_dim) : 0;
}

moe_status_t moe_latent_attention(const uint16_t *q_latent, int64_t ql_stride_t, int64_t ql_stride_h, const uint16_t *q_rope,
                                  int64_t qr_stride_t, int64_t qr_stride_h, int T, int heads, const moe_latent_cache_t *cache,
                                  const int32_t *block_table, int max_blocks, const int32_t *q_offsets, const int32_t *kv_lens,
                                  int B, float softmax_scale, int causal, uint16_t *out, float *lse, void *ws, size_t ws_bytes,
                                  cudaStream_t stream) {
    moe_status_t st = check_latent_cache(cache);
    if (st != MOE_OK || (st = check_latent_sizes(T, B, heads, cache->latent_dim)) != MOE_OK)
        return st;
    if (max_blocks < 0 || (causal != 0 && causal != 1) || ql_stride_t < 0 || ql_stride_h < 0 || qr_stride_t < 0 || qr_stride_h < 0 ||
        !(softmax_scale >= 0.0f) || softmax_scale > 3.0e38f)
        return MOE_ERR_INVALID_ARG;
    if ((long long)max_blocks * cache->block_size > 0x7FFFFFFFll - 256)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || B == 0)
        return MOE_OK;
    if (!q_latent || !q_rope || !out || !q_offsets || !kv_lens || (max_blocks > 0 && !block_table))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(q_latent, 16) || !aligned(q_rope, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(q_offsets, 4) ||
        !aligned(kv_lens, 4) || !aligned(block_table, 4) || ql_stride_t % 8 || ql_stride_h % 8 || qr_stride_t % 8 || qr_stride_h % 8)
        return MOE_ERR_MISALIGNED;
    int sms = 0;
    if ((st = check_ws(ws, ws_bytes, latent_attention_need(T, B, heads, cache->latent_dim))) != MOE_OK || (st = check_device(&sms)) != MOE_OK)
        return st;
    const LatentProblem p{q_latent, ql_stride_t, ql_stride_h, q_rope, qr_stride_t, qr_stride_h, T, heads, *cache, block_table, max_blocks,
                          q_offsets, kv_lens, B, softmax_scale, causal, out, lse};
    return from_cuda(launch_latent_attention(p, ws, sms, stream));
}

}  // extern "C"
