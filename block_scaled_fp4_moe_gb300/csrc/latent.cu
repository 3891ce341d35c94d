// latent.cu -- attention over a cache of one latent vector and one rotary key a token (moe_attn.h, b8).
//
//   x_j = softmax_scale (q_latent.c_j + q_rope.r_j),   out = sum_j p_j c_j / sum_j p_j,   p_j = exp(x_j - max x)
//
// The plain form: a CTA has a token's sixteen heads and walks the cache in tiles of 32 tokens in shared memory, with running maxima and
// sums; two dims of every head's sum in a thread's registers.
#include "attn.h"

namespace moe {
namespace {

constexpr int kHeads = 16, kTokens = 32, kThreads = 256;

template <int L>
__global__ void __launch_bounds__(kThreads) latent_plain_kernel(const LatentProblem p, uint32_t *hdr) {
    constexpr int W = L + kRopeDims, P = W + 2;            // a row's pitch: its threads read other banks
    constexpr int D = L / kThreads;
    extern __shared__ uint16_t rows[];                     // queries [kHeads][P], tokens [kTokens][P]
    __shared__ float s_x[kHeads][kTokens], s_m[kHeads], s_l[kHeads], s_by[kHeads];
    __shared__ int s_request;
    const int tid = threadIdx.x, t = blockIdx.x, h0 = blockIdx.y * kHeads;
    pdl_wait();
    pdl_trigger();
    if (tid == 0)
        s_request = -1;
    int bad = 0;
    __syncthreads();
    for (int b = tid; b < p.B; b += kThreads) {
        const int lo = p.q_offsets[b], hi = p.q_offsets[b + 1], kv = p.kv_lens[b];
        bad |= lo < 0 || hi < lo || hi > p.T || kv < 0 || kv > (long long)p.max_blocks * p.cache.block_size;
        if (t >= lo && t < hi)
            s_request = b;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0)
            record_status(hdr, MOE_ERR_DEVICE_ASSERT);
        return;
    }
    const int b = s_request;
    if (b < 0)
        return;
    const int kv = p.kv_lens[b], last = p.causal ? kv - (p.q_offsets[b + 1] - t) + 1 : kv, seen = min(kv, last);
    uint16_t *qs = rows, *ks = rows + kHeads * P;
    for (int i = tid; i < kHeads * W; i += kThreads) {
        const int h = i / W, d = i % W;
        uint16_t v = 0;
        if (h0 + h < p.heads)
            v = d < L ? p.ql[t * p.ql_st + (h0 + h) * p.ql_sh + d] : p.qr[t * p.qr_st + (h0 + h) * p.qr_sh + d - L];
        qs[h * P + d] = v;
    }
    if (tid < kHeads) {
        s_m[tid] = -INFINITY;
        s_l[tid] = 0.0f;
    }
    float o[kHeads][D];
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
#pragma unroll
        for (int d = 0; d < D; ++d)
            o[h][d] = 0.0f;
    auto wide = [](uint16_t v) { return __uint_as_float((uint32_t)v << 16); };
    for (int j0 = 0; j0 < seen; j0 += kTokens) {
        __syncthreads();
        for (int i = tid; i < kTokens * W; i += kThreads) {
            const int j = j0 + i / W, d = i % W;
            uint16_t v = 0;
            if (j < seen) {
                int page = p.table[(size_t)b * p.max_blocks + j / p.cache.block_size];
                if (page < 0 || page >= p.cache.num_blocks) {
                    record_status(hdr, MOE_ERR_DEVICE_ASSERT);
                    page = 0;
                }
                v = p.cache.data[((size_t)page * p.cache.block_size + j % p.cache.block_size) * W + d];
            }
            ks[(i / W) * P + d] = v;
        }
        __syncthreads();
        for (int i = tid; i < kHeads * kTokens; i += kThreads) {
            const int h = i / kTokens, j = i % kTokens;
            float s = 0.0f;
            for (int d = 0; d < W; ++d)
                s = fmaf(wide(qs[h * P + d]), wide(ks[j * P + d]), s);
            s_x[h][j] = j0 + j < seen ? s * p.scale : -INFINITY;
        }
        __syncthreads();
        if (tid < kHeads) {
            float m = s_m[tid];
            for (int j = 0; j < kTokens; ++j)
                m = s_x[tid][j] > m || isnan(s_x[tid][j]) ? s_x[tid][j] : m;
            const float z = m == -INFINITY ? 0.0f : m;
            s_by[tid] = expf(s_m[tid] - z);
            float l = s_l[tid] * s_by[tid];
            for (int j = 0; j < kTokens; ++j) {
                s_x[tid][j] = expf(s_x[tid][j] - z);
                l += s_x[tid][j];
            }
            s_m[tid] = m;
            s_l[tid] = l;
        }
        __syncthreads();
        const int n = min(kTokens, seen - j0);
#pragma unroll
        for (int d = 0; d < D; ++d) {
#pragma unroll
            for (int h = 0; h < kHeads; ++h)
                o[h][d] *= s_by[h];
            for (int j = 0; j < n; ++j) {
                const float c = wide(ks[j * P + tid + d * kThreads]);
#pragma unroll
                for (int h = 0; h < kHeads; ++h)
                    o[h][d] = fmaf(s_x[h][j], c, o[h][d]);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        if (h0 + h >= p.heads)
            break;
        const float l = s_l[h];
        const size_t at = (size_t)t * p.heads + h0 + h;
        for (int d = 0; d < D; ++d) {
            uint16_t v;
            asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(v) : "f"(seen > 0 ? o[h][d] / l : 0.0f));
            p.out[at * L + tid + d * kThreads] = v;
        }
        if (tid == 0 && p.lse)
            p.lse[at] = seen > 0 ? s_m[h] + logf(l) : -INFINITY;
    }
}

}  // namespace

size_t latent_attention_workspace(int, int, int, int) { return align_up(kInitBytes, 256); }

cudaError_t launch_latent_attention(const LatentProblem &p, void *ws, int, cudaStream_t stream) {
    const dim3 grid(p.T, (p.heads + kHeads - 1) / kHeads);
    auto go = [&](auto kernel, int W) {
        const size_t smem = (size_t)(kHeads + kTokens) * (W + 2) * 2;
        cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        return r != cudaSuccess ? r : launch_pdl(kernel, grid, dim3(kThreads), smem, stream, p, ws_at<uint32_t>(ws, 0));
    };
    return p.cache.latent_dim == 256 ? go(latent_plain_kernel<256>, 256 + kRopeDims) : go(latent_plain_kernel<512>, 512 + kRopeDims);
}

}  // namespace moe
