// rotary.cu -- rotary positions on query and key heads, and the append to the latent cache (moe_attn.h, b6 and b7).
//
//   a' = m (a cos t - b sin t),  b' = m (b cos t + a sin t),  t = 2 pi p f
//
// The angle of a far position needs more bits than fp32 has: f is held in units of 2^-64 turns, p f modulo 2^64 is one
// integer product and is exact, and its upper 32 bits, as a signed fraction of a turn rounded to fp32, are within 2^-26 turns.
//
// Lanes.  A head has D / 8 lanes (rounded up to a power of two) with eight dims each, so that a norm's sum is a few shuffles.
// With halves a pair's other half is in the lane 2 pairs / 16 away.  Cosines and sines are made once for a token
// and CTA, in shared memory, for all heads.
#include "attn.h"

namespace moe {
namespace {

__device__ __forceinline__ void widen(float (&f)[8], uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// (cos, sin) of a pair's angle at a position, times the amplitude.
__device__ __forceinline__ float2 turn_of(int position, uint64_t turns, float amplitude) {
    const int64_t at = (int64_t)((uint64_t)(uint32_t)position * turns);
    float s, c;
    sincospif((float)(int32_t)(at >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c * amplitude, s * amplitude);
}

// Eight dims of a head, `c` the chunk of the rotated part that they are (of 2 pairs / 8), to their rotated values.  cs: the pairs'.
// The lane of the other half is lane + or - span.  All lanes of the warp take part.
__device__ __forceinline__ void rotate8(float (&v)[8], int c, bool in, int span, int interleaved, const float2 *cs) {
    if (interleaved) {
        if (!in)
            return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = cs[4 * c + i];
            const float a = v[2 * i], b = v[2 * i + 1];
            v[2 * i] = a * t.x - b * t.y;
            v[2 * i + 1] = b * t.x + a * t.y;
        }
        return;
    }
    const bool second = c >= span;
    const int lane = threadIdx.x & 31, other = in ? (second ? lane - span : lane + span) : lane;
    const int first = 8 * (second ? c - span : c);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(0xffffffffu, v[i], other);
        if (in) {
            const float2 t = cs[first + i];
            v[i] = second ? v[i] * t.x + o * t.y : v[i] * t.x - o * t.y;
        }
    }
}

constexpr int kRotaryThreads = 256;

// One CTA: a token's heads blockIdx.y, + gridDim.y, ... (in sets of as many as the CTA holds).
template <int LANES>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryProblem p) {
    __shared__ float2 cs[128];
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x, pos = p.positions[t];
    if (pos < 0)
        return;
    if ((int)threadIdx.x < p.pairs)
        cs[threadIdx.x] = turn_of(pos, __ldg(p.turns + threadIdx.x), p.amplitude);
    __syncthreads();
    const int c = threadIdx.x % LANES, set = kRotaryThreads / LANES;
    const int first = p.offset / 8, span = p.pairs / 8;
    const bool in = c >= first && c < first + 2 * span, live = c < p.D / 8;
    const int heads = p.q.heads + p.k.heads;
    for (int h0 = blockIdx.y * set; h0 < heads; h0 += gridDim.y * set) {      // the same trips for all lanes
        const int h = h0 + threadIdx.x / LANES;
        const bool is_q = h < p.q.heads, mine = live && h < heads;
        const HeadSet &x = is_q ? p.q : p.k;
        const int at = is_q ? h : h - p.q.heads;
        const uint16_t *src = x.in + t * x.st + at * x.sh + 8 * c;
        uint16_t *dst = x.out + t * x.ost + at * x.osh + 8 * c;
        float v[8];
        widen(v, mine ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0));
        if (p.q.norm || p.k.norm) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s = fmaf(v[i], v[i], s);
#pragma unroll
            for (int d = LANES / 2; d > 0; d >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, d);
            if (mine && x.norm) {
                const float by = rsqrtf(s / (float)p.D + p.eps);
                float w[8];
                widen(w, __ldg(reinterpret_cast<const uint4 *>(x.norm) + c));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = v[i] * by * w[i];
            }
        }
        rotate8(v, c - first, in, span, p.interleaved, cs);
        if (mine && (in || x.norm || dst != src))
            *reinterpret_cast<uint4 *>(dst) = narrow(v);
    }
}

// ------------------------------------------------------------ latent append

constexpr int kAppendWarps = 4;

// A warp has a token: its latent vector in L / 256 chunks of eight values a lane, its rotary key in the first eight lanes.
template <int L>
__global__ void __launch_bounds__(kAppendWarps * 32) latent_append_kernel(const LatentAppendProblem p) {
    __shared__ float2 cs[kAppendWarps][kRopeDims / 2];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kAppendWarps + warp;
    if (t >= p.T)
        return;
    const int64_t slot = p.slots[t];
    if (slot < 0)
        return;
    if (slot >= (int64_t)p.cache.num_blocks * p.cache.block_size) {
        if (lane == 0)
            record_status(p.hdr, MOE_ERR_DEVICE_ASSERT);
        return;
    }
    constexpr int PER = L / 256;
    float v[PER][8], k[8];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        widen(v[i], *(reinterpret_cast<const uint4 *>(p.c + t * p.ldc) + lane + 32 * i));
    const bool key = lane < kRopeDims / 8;
    widen(k, key ? *(reinterpret_cast<const uint4 *>(p.k + t * p.ldk) + lane) : make_uint4(0, 0, 0, 0));
    uint16_t *row = p.cache.data + slot * (L + kRopeDims);
    if (p.turns) {
        cs[warp][lane] = turn_of(p.positions[t], __ldg(p.turns + lane), p.amplitude);
        __syncwarp();
        rotate8(k, lane, key, kRopeDims / 16, p.interleaved, cs[warp]);
    }
    if (key)
        *(reinterpret_cast<uint4 *>(row + L) + lane) = narrow(k);
    if (p.norm) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s = fmaf(v[i][e], v[i][e], s);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, d);
        const float by = rsqrtf(s / (float)L + p.eps);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            float w[8];
            widen(w, __ldg(reinterpret_cast<const uint4 *>(p.norm) + lane + 32 * i));
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i][e] = v[i][e] * by * w[e];
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
        *(reinterpret_cast<uint4 *>(row) + lane + 32 * i) = narrow(v[i]);
}

}  // namespace

cudaError_t launch_rotary(const RotaryProblem &p, int sms, cudaStream_t stream) {
    const int lanes = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32, set = kRotaryThreads / lanes;
    const int sets = (p.q.heads + p.k.heads + set - 1) / set;
    const int split = p.T >= 4 * sms ? 1 : sets;           // a CTA for a token's heads, or for as many as it holds
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(p.T, split), dim3(kRotaryThreads), 0, stream, p); };
    return lanes == 8 ? go(rotary_kernel<8>) : lanes == 16 ? go(rotary_kernel<16>) : go(rotary_kernel<32>);
}

cudaError_t launch_latent_append(const LatentAppendProblem &p, int, cudaStream_t stream) {
    const dim3 grid((p.T + kAppendWarps - 1) / kAppendWarps), block(kAppendWarps * 32);
    return p.cache.latent_dim == 256 ? launch_pdl(latent_append_kernel<256>, grid, block, 0, stream, p)
                                     : launch_pdl(latent_append_kernel<512>, grid, block, 0, stream, p);
}

}  // namespace moe
