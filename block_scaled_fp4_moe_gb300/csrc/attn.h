// attn.h -- shared definitions of the attention-half kernels: the 8-bit format
// of moe_attn.h and the launch functions (internal to the library).
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "moe_attn.h"

namespace moe {

constexpr int kMaxRequests = 8192;      // B
constexpr int kMaxAttnTokens = 1 << 20; // T of the attention and the projection
constexpr int kMaxTableTokens = 1 << 24;

// ------------------------------------------------------- the 8-bit format

// E8M0 byte of a group whose largest finite magnitude has these fp32 bits:
// e + 127 for the smallest e >= -126 with a <= 448 * 2^e.  With a = 1.f *
// 2^(E-127) and 448 = 1.75 * 2^8, e = E - 127 - 8, plus one where 1.f > 1.75.
__device__ __forceinline__ int fp8_scale_byte(uint32_t amax_bits) {
    return max(1, (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u));
}

// The magnitude bits of v where it is finite, 0 where it is not.
__device__ __forceinline__ uint32_t finite_abs_bits(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
    return b < 0x7F800000u ? b : 0u;
}

// Two values times 2^-e to E4M3 (lo in the low byte); not finite -> NaN.
__device__ __forceinline__ uint32_t fp8_pair(float lo, float hi, float inv) {
    // inf * 0 = NaN, finite * 0 = 0: one FMA turns infinities into NaN and leaves
    // every finite product as it is
    lo = __fmaf_rn(lo, 0.0f, lo * inv);
    hi = __fmaf_rn(hi, 0.0f, hi * inv);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// 8 bf16 (16 bytes) times 2^-e to 8 codes.
__device__ __forceinline__ uint2 fp8_from_bf16x8(uint4 v, float inv) {
    auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
    auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
    return make_uint2(fp8_pair(lo(v.x), hi(v.x), inv) | fp8_pair(lo(v.y), hi(v.y), inv) << 16,
                      fp8_pair(lo(v.z), hi(v.z), inv) | fp8_pair(lo(v.w), hi(v.w), inv) << 16);
}

// Largest finite magnitude bits of 8 bf16: as pairs of 16-bit integers, which
// order as the magnitudes do; where an infinity or NaN is among them, one by one.
__device__ __forceinline__ uint32_t amax_bf16x8(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const uint32_t two = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    uint32_t m = max(two << 16, two & 0xFFFF0000u);
    if (m >= 0x7F800000u) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m = max(m, max(finite_abs_bits(__uint_as_float(w[i] << 16)), finite_abs_bits(__uint_as_float(w[i] & 0xFFFF0000u))));
    }
    return m;
}

// Two E4M3 codes (low 16 bits) to f16x2, exact (NaN codes to NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}

// ------------------------------------------------------- launch functions

struct TablesProblem {
    const int32_t *ctx, *fresh;      // [B] tokens cached, tokens new
    int B, T, block_shift;
    const int32_t *free_blocks;
    int num_free;
    const int32_t *free_head;
    int32_t *table;
    int max_blocks;
    int32_t *kv_lens, *q_offsets;
    int64_t *slot_map;
    int32_t *positions, *free_head_out;
    uint32_t *hdr;
};
cudaError_t launch_kv_tables(const TablesProblem &p, cudaStream_t stream);

struct AppendProblem {
    const uint16_t *k, *v;
    int64_t k_st, k_sh, v_st, v_sh;
    const int64_t *slots;
    int T;
    moe_kv_cache_t cache;
    uint32_t *hdr;
};
cudaError_t launch_kv_append(const AppendProblem &p, cudaStream_t stream);

struct AttnProblem {
    const uint16_t *q;
    int64_t q_st, q_sh;
    int T, q_heads;
    moe_kv_cache_t cache;
    const int32_t *table;
    int max_blocks;
    const int32_t *q_offsets, *kv_lens;
    int B;
    float scale;
    int causal, window;
    uint16_t *out;
    float *lse;
};
// Workspace regions of the attention.
struct AttnLayout {
    size_t plan, recs, part, part_sum, nans, total;
    static AttnLayout make(int T, int B, int q_heads, int kv_heads, int head_dim);
};
// The tensor-memory form (attn_tc.cu) for requests of more than this many rows on average, its units' rows, and the
// bytes of a CTA's list of NaN values.
constexpr int kAttnTcMinRows = 24;
constexpr int kAttnTcRows = 256;
constexpr size_t kAttnNanBytes = 2048 * 32;
cudaError_t launch_attn_tc(const void *args, int head_dim, int ctas, cudaStream_t stream);
cudaError_t launch_kv_attention(const AttnProblem &p, void *ws, int sms, cudaStream_t stream);

size_t linear_fp8_workspace(int T, int N, int K);
struct LinearProblem {
    const uint16_t *x;
    int64_t ldx;
    const uint8_t *codes, *scale;
    uint16_t *y;
    int T, N, K;
};
cudaError_t launch_linear_fp8(const LinearProblem &p, void *ws, int sms, cudaStream_t stream);
cudaError_t launch_quantize_fp8_weight(const uint16_t *w, int N, int K, uint8_t *codes, uint8_t *scale,
                                       cudaStream_t stream);

}  // namespace moe
