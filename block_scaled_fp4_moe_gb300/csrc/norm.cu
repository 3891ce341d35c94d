// norm.cu -- residual sum and root-mean-square norm before and after a block (moe_attn.h, b5).
//
//   u = x, or x / sqrt(mean x^2 + eps) * post;   h = r + scale * gate * u;   y = h / sqrt(mean h^2 + eps) * weight
//
// One pass: a row stays in registers from the loads of x and r to the stores of h and y, the sums of squares
// join its threads in between (one join, two with a norm of x).  A thread has PER chunks of eight values, so that the loads
// of a row are in flight together.  Rows of up to 1,024 values have a warp each and need no barrier.
//
// Bound by memory, a row's 8 bytes a value (12 with a 32-bit residual): 4,000 rows of 7168 in 35.9 us, 6.4 TB/s, 94 % of a copy's rate (two chunks a
// thread: 38.2; one row's loads are then a smaller part of its time).  Few rows are a launch: one of 5,120 takes 1.8 us in a graph.
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

// The sum over a row's threads, in an order that depends on their number alone.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float *red) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    if (WARP)
        return v;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? red[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

template <int PER, bool WARP, bool WIDE>
__global__ void __launch_bounds__(WARP ? 256 : 1024) rms_norm_kernel(const NormProblem p) {
    __shared__ float red[2][32];
    const int group = WARP ? 32 : blockDim.x, me = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int t = WARP ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    pdl_wait();
    pdl_trigger();
    if (t >= p.T)
        return;
    const int chunks = p.H / 8;
    const uint4 *x = reinterpret_cast<const uint4 *>(p.x + (int64_t)t * p.ldx);
    const int64_t row = (int64_t)t * chunks;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 xv[PER], rv[PER][WIDE ? 2 : 1];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = me + i * group;
        xv[i] = c < chunks ? __ldg(x + c) : zero;
#pragma unroll
        for (int k = 0; k < (WIDE ? 2 : 1); ++k)
            rv[i][k] = c < chunks && p.residual ? *(reinterpret_cast<const uint4 *>(p.residual) + (row + c) * (WIDE ? 2 : 1) + k) : zero;
    }
    float by = 1.0f;
    if (p.post) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            float f[8];
            widen(f, xv[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s = fmaf(f[e], f[e], s);
        }
        by = rsqrtf(row_sum<WARP>(s, red[0]) / (float)p.H + p.eps);
    }
    float h[PER][8], s = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = me + i * group;
        const bool in = c < chunks;
        widen(h[i], xv[i]);
        if (p.post) {
            float w[8];
            widen(w, in ? __ldg(reinterpret_cast<const uint4 *>(p.post) + c) : zero);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[i][e] = h[i][e] * by * w[e];
        }
        if (p.gate) {
            float g[8];
            widen(g, in ? __ldg(reinterpret_cast<const uint4 *>(p.gate + (int64_t)t * p.ld_gate) + c) : zero);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[i][e] *= g[e];
        }
        float r[8];
        if (WIDE) {
            r[0] = __uint_as_float(rv[i][0].x), r[1] = __uint_as_float(rv[i][0].y), r[2] = __uint_as_float(rv[i][0].z), r[3] = __uint_as_float(rv[i][0].w);
            const uint4 b = rv[i][WIDE ? 1 : 0];
            r[4] = __uint_as_float(b.x), r[5] = __uint_as_float(b.y), r[6] = __uint_as_float(b.z), r[7] = __uint_as_float(b.w);
        } else {
            widen(r, rv[i][0]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            h[i][e] = fmaf(p.scale, h[i][e], r[e]);
            s = fmaf(h[i][e], h[i][e], s);
        }
        if (in && p.residual_out) {
            uint4 *to = reinterpret_cast<uint4 *>(p.residual_out) + (row + c) * (WIDE ? 2 : 1);
            if (WIDE) {
                to[0] = make_uint4(__float_as_uint(h[i][0]), __float_as_uint(h[i][1]), __float_as_uint(h[i][2]), __float_as_uint(h[i][3]));
                to[1] = make_uint4(__float_as_uint(h[i][4]), __float_as_uint(h[i][5]), __float_as_uint(h[i][6]), __float_as_uint(h[i][7]));
            } else {
                to[0] = narrow(h[i]);
            }
        }
    }
    if (!p.y)
        return;
    by = rsqrtf(row_sum<WARP>(s, red[1]) / (float)p.H + p.eps);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = me + i * group;
        if (c < chunks) {
            float w[8];
            widen(w, __ldg(reinterpret_cast<const uint4 *>(p.weight) + c));
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[i][e] = h[i][e] * by * w[e];
            reinterpret_cast<uint4 *>(p.y)[row + c] = narrow(h[i]);
        }
    }
}

template <int PER, bool WARP>
cudaError_t launch(const NormProblem &p, int threads, cudaStream_t stream) {
    const unsigned grid = WARP ? (unsigned)((p.T + 7) / 8) : (unsigned)p.T;
    return p.wide ? launch_pdl(rms_norm_kernel<PER, WARP, true>, dim3(grid), dim3(threads), 0, stream, p)
                  : launch_pdl(rms_norm_kernel<PER, WARP, false>, dim3(grid), dim3(threads), 0, stream, p);
}

}  // namespace

cudaError_t launch_rms_norm(const NormProblem &p, int sms, cudaStream_t stream) {
    const int chunks = p.H / 8;
    auto threads = [&](int per) { return (((chunks + per - 1) / per) + 31) / 32 * 32; };
    if (chunks <= 32)
        return launch<1, true>(p, 256, stream);
    if (chunks <= 64)
        return launch<2, true>(p, 256, stream);
    if (chunks <= 128)
        return launch<4, true>(p, 256, stream);
    if (chunks <= 1024 && p.T <= sms)
        return launch<1, false>(p, threads(1), stream);
    if (chunks <= 256 || (chunks <= 2048 && p.T <= 4 * sms))
        return launch<2, false>(p, threads(2), stream);
    return launch<4, false>(p, threads(4), stream);
}

}  // namespace moe
