// rotary.cu -- rotary positions on query and key heads, and the append to the latent cache (moe_attn.h, b6 and b7).
//
//   a' = m (a cos t - b sin t),  b' = m (b cos t + a sin t),  t = 2 pi p f
//
// The angle of a far position needs more bits than fp32 has: f is held in units of 2^-64 turns, p f modulo 2^64 is one
// integer product and is exact, and its upper 32 bits, as a signed fraction of a turn rounded to fp32, are within 2^-26 turns.
//
// Lanes.  A lane has 16 dims of a head: where pairs are halves, eight of each half, so that no values pass between lanes; a norm's
// sum is a few shuffles over the head's lanes (a power of two of them).  A warp has a token and a few sets of heads, whose loads are all
// in flight before it makes the token's cosines and sines (in shared memory; a lane keeps its eight): no warp waits for another.
//
// Bound by memory, 4 bytes a value, and in part by its way there: 4,000 tokens of 48 heads of 128, halves, in 20.0 us (4.9 TB/s), 25.5 with norms
// (a warp's sums and the norm's weights); neighbours 26 with norms, and 24.4 where half of each head is rotated.  (Three sets of tensors in turn; one set,
// which L2 holds in part, takes 16.1, and 22.8 with norms.)  Forms before, on tensors that L2 held in part, when this one took 18.0: a CTA a token, with a
// lane for eight dims and shuffles between halves 37 us; without shuffles 22; CTAs that go from token to token, loads a step ahead, 21.5.
// The append: 7,900 tokens of 576 values in 4.0 us (4.6 TB/s; launch and one chain of loads).
#include <type_traits>

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

// Eight pairs in two times eight dims.
template <bool INTER>
__device__ __forceinline__ void rotate16_as(float (&u)[8], float (&v)[8], const float2 (&cs)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float &a = INTER ? (i < 4 ? u[2 * i & 7] : v[2 * i & 7]) : u[i];
        float &b = INTER ? (i < 4 ? u[(2 * i & 7) + 1] : v[(2 * i & 7) + 1]) : v[i];
        const float x = a, y = b;
        a = x * cs[i].x - y * cs[i].y;
        b = y * cs[i].x + x * cs[i].y;
    }
}
__device__ __forceinline__ void rotate16(float (&u)[8], float (&v)[8], int interleaved, const float2 (&cs)[8]) {
    if (interleaved)
        rotate16_as<true>(u, v, cs);
    else
        rotate16_as<false>(u, v, cs);
}

constexpr int kRotaryWarps = 4;

// A warp: a token and SETS sets of 32 / LANES heads.  Item i of a head: pairs 8 i .. 8 i + 7, or, behind those, two chunks of eight dims
// that are not rotated.
template <int LANES, int SETS, bool NORM>
__global__ void __launch_bounds__(kRotaryWarps * 32) rotary_kernel(const RotaryProblem p) {
    __shared__ float2 s_cs[kRotaryWarps][128];
    pdl_wait();
    pdl_trigger();
    constexpr int kSet = 32 / LANES;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, heads = p.q.heads + p.k.heads;
    const int segments = (heads + SETS * kSet - 1) / (SETS * kSet);
    const int64_t job = (int64_t)blockIdx.x * kRotaryWarps + warp;
    const int t = (int)(job / segments), h0 = (int)(job % segments) * (SETS * kSet) + lane / LANES;
    if (t >= p.T)
        return;
    const int pos = p.positions[t];
    if (pos < 0)
        return;
    const int item = lane % LANES, first = p.offset / 8, span = p.pairs / 8, rest = p.D / 8 - 2 * span;
    const bool in = item < span;
    // the lane's chunks: neither, one or both exist
    int c0 = 2 * (item - span), c1 = c0 + 1;
    const bool has0 = in || c0 < rest, has1 = in || c1 < rest;
    if (in) {
        c0 = first + (p.interleaved ? 2 * item : item);
        c1 = p.interleaved ? c0 + 1 : c0 + span;
    } else {
        c0 += c0 < first ? 0 : 2 * span;
        c1 += c1 < first ? 0 : 2 * span;
    }
    uint4 raw[SETS][2];
#pragma unroll
    for (int u = 0; u < SETS; ++u) {
        const int h = h0 + u * kSet;
        const bool is_q = h < p.q.heads;
        const uint16_t *src = is_q ? p.q.in + t * p.q.st + h * p.q.sh : p.k.in + t * p.k.st + (h - p.q.heads) * p.k.sh;
        raw[u][0] = has0 && h < heads ? *reinterpret_cast<const uint4 *>(src + 8 * c0) : make_uint4(0, 0, 0, 0);
        raw[u][1] = has1 && h < heads ? *reinterpret_cast<const uint4 *>(src + 8 * c1) : make_uint4(0, 0, 0, 0);
    }
    for (int i = lane; i < p.pairs; i += 32)
        s_cs[warp][i] = turn_of(pos, __ldg(p.turns + i), p.amplitude);
    __syncwarp();
    float2 cs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        cs[i] = in ? s_cs[warp][8 * item + i] : make_float2(1.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < SETS; ++u) {
        const int h = h0 + u * kSet;
        const bool is_q = h < p.q.heads;
        const uint16_t *src = is_q ? p.q.in + t * p.q.st + h * p.q.sh : p.k.in + t * p.k.st + (h - p.q.heads) * p.k.sh;
        uint16_t *dst = is_q ? p.q.out + t * p.q.ost + h * p.q.osh : p.k.out + t * p.k.ost + (h - p.q.heads) * p.k.osh;
        const uint16_t *norm = is_q ? p.q.norm : p.k.norm;
        float a[8], b[8];
        widen(a, raw[u][0]);
        widen(b, raw[u][1]);
        if (NORM) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s = fmaf(a[i], a[i], fmaf(b[i], b[i], s));
#pragma unroll
            for (int d = LANES / 2; d > 0; d >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, d);
            if (norm) {
                const float by = rsqrtf(s / (float)p.D + p.eps);
                float w[8];
                widen(w, has0 ? __ldg(reinterpret_cast<const uint4 *>(norm) + c0) : make_uint4(0, 0, 0, 0));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    a[i] = a[i] * by * w[i];
                widen(w, has1 ? __ldg(reinterpret_cast<const uint4 *>(norm) + c1) : make_uint4(0, 0, 0, 0));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    b[i] = b[i] * by * w[i];
            }
        }
        if (in)
            rotate16(a, b, p.interleaved, cs);
        if (h < heads && (in || (NORM && norm) || dst != src)) {
            if (has0)
                *reinterpret_cast<uint4 *>(dst + 8 * c0) = narrow(a);
            if (has1)
                *reinterpret_cast<uint4 *>(dst + 8 * c1) = narrow(b);
        }
    }
}

// ------------------------------------------------------------ latent append

constexpr int kAppendWarps = 4;

// A warp has a token: its latent vector in L / 256 chunks of eight values a lane, a pair of its rotary key in each.
template <int L>
__global__ void __launch_bounds__(kAppendWarps * 32) latent_append_kernel(const LatentAppendProblem p) {
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kAppendWarps + warp;
    if (t >= p.T)
        return;
    const int64_t slot = p.slots[t];
    const int pos = p.turns ? p.positions[t] : 0;
    if (slot < 0 || pos < 0)                     // positions as in rotary_kernel
        return;
    if (slot >= (int64_t)p.cache.num_blocks * p.cache.block_size) {
        if (lane == 0)
            record_status(p.hdr, MOE_ERR_DEVICE_ASSERT);
        return;
    }
    constexpr int PER = L / 256;
    float v[PER][8];
    uint4 raw[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        raw[i] = *(reinterpret_cast<const uint4 *>(p.c + t * p.ldc) + lane + 32 * i);
    const int ka = p.interleaved ? 2 * lane : lane, kb = p.interleaved ? ka + 1 : ka + kRopeDims / 2;
    const uint16_t *key = p.k + t * p.ldk;
    uint16_t a = key[ka], b = key[kb];
    uint16_t *row = p.cache.data + slot * (L + kRopeDims);
    if (p.turns) {
        const float2 cs = turn_of(pos, __ldg(p.turns + lane), p.amplitude);
        const float x = __uint_as_float((uint32_t)a << 16), y = __uint_as_float((uint32_t)b << 16);
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(a) : "f"(x * cs.x - y * cs.y));
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(y * cs.x + x * cs.y));
    }
    row[L + ka] = a;
    row[L + kb] = b;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        widen(v[i], raw[i]);
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
        *(reinterpret_cast<uint4 *>(row) + lane + 32 * i) = p.norm ? narrow(v[i]) : raw[i];             // without a norm the bits as they are
}

}  // namespace

cudaError_t launch_rotary(const RotaryProblem &p, int sms, cudaStream_t stream) {
    const int items = p.pairs / 8 + (p.D / 8 - p.pairs / 4 + 1) / 2, lanes = items <= 4 ? 4 : items <= 8 ? 8 : 16;
    const int heads = p.q.heads + p.k.heads, set = 32 / lanes;
    // Sets of a warp: one while that many warps fit on the GPU at once (64 tokens of 72 heads of 128 in a graph, 2.4 us; with four, 2.7); else four or
    // three, as fewer lanes go without a head (4,000 tokens of 48 heads 20.0 and 21.2 us, with two 22.1; 8,192 of 18 heads of 256 32.4 and 31.0).
    auto waste = [&](int sets) { return (sets * set - heads % (sets * set)) % (sets * set); };
    const bool norm = p.q.norm || p.k.norm;                // (it takes more registers: 25.5 us with three, 27.1 with four)
    const int sets = (int64_t)p.T * heads * lanes <= (int64_t)sms * 512 ? 1 : waste(3) < waste(4) + norm ? 3 : 4;
    const int64_t jobs = (int64_t)p.T * ((heads + sets * set - 1) / (sets * set));
    const dim3 grid((unsigned)((jobs + kRotaryWarps - 1) / kRotaryWarps));
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kRotaryWarps * 32), 0, stream, p); };
    auto form = [&](auto lanes_of) {
        constexpr int N = decltype(lanes_of)::value;
        if (norm)
            return sets == 1 ? go(rotary_kernel<N, 1, true>) : sets == 3 ? go(rotary_kernel<N, 3, true>) : go(rotary_kernel<N, 4, true>);
        return sets == 1 ? go(rotary_kernel<N, 1, false>) : sets == 3 ? go(rotary_kernel<N, 3, false>) : go(rotary_kernel<N, 4, false>);
    };
    return lanes == 4 ? form(std::integral_constant<int, 4>()) : lanes == 8 ? form(std::integral_constant<int, 8>())
                                                                            : form(std::integral_constant<int, 16>());
}

cudaError_t launch_latent_append(const LatentAppendProblem &p, int, cudaStream_t stream) {
    const dim3 grid((p.T + kAppendWarps - 1) / kAppendWarps), block(kAppendWarps * 32);
    return p.cache.latent_dim == 256 ? launch_pdl(latent_append_kernel<256>, grid, block, 0, stream, p)
                                     : launch_pdl(latent_append_kernel<512>, grid, block, 0, stream, p);
}

}  // namespace moe
