// linear.cu -- y = X^ W^T with E4M3 operands and one power-of-two scale for each block of 128.
//
//   y[t, n] = sum_kb 2^(sx[t, kb] + sw[n / 128, kb]) sum_{k in kb} cx[t, k] cw[n, k]
//
// Because the scales are powers of two, the tensor core applies them
// (kind::mxf8f6f4, one E8M0 byte for 32 K elements: a block's byte is given
// for its four quarters) and the sum over all of K stays in tensor
// memory: no rescaling of partial sums in registers.
//
// fp8_quant_kernel turns x into codes and scale words, fp8_gemm_kernel
// multiplies.  W's rows are the MMA's M (128 of them) and the tokens its N, so that
// a few tokens waste no tensor-core rows and W is streamed once.  Few output
// tiles: the K stages of a tile are shared by a cluster of up to eight CTAs, whose
// sums are added in K order through distributed shared memory, so that one token's
// projection keeps every SM streaming W, without sums in global memory.  Many:
// a persistent grid walks the tiles.
//
// CTA: warp 0 copies stages (128 K) of W, x and x's scales into a shared-memory
// ring with TMA, and writes W's scale; warp 1 issues tcgen05.cp (scales to
// tensor memory) and the MMAs; warps 2..5 drain the accumulators, of
// which a persistent CTA has two, while the next tile is summed.
//
// Measured (W in memory, not in L2): 7168 x 5120 with one token 8.9 us (4.1 TB/s: starting the stream, and the cluster's join, are a
// third of it), 7168 x 8192 with 61 tokens 17.2 us, of which 2.7 quantise x (3.5 TB/s); 7168 x 5120 with 4,000 tokens 148 us, of which
// 10 quantise x (1.99 PFLOP/s).  Weights are quantised at 4.8 TB/s (7168 x 5120 in 23 us; 16 at the rate of a copy).  Many tokens are bound by shared memory: a stage of 128 x 192 x 128 is written to it and read from it in
// about 640 cycles and multiplied in 408, and no more than four fit.
#include <cuda.h>

#include "attn.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kStageK = 128;
constexpr int kABytes = 128 * kStageK;
constexpr int kMaxSplit = 8;       // CTAs of a cluster
constexpr unsigned long long kWaitLimitNs = 200ull * 1000 * 1000;

// Per token tile NN: ring stages, shared memory, tensor-memory columns.  A
// stage has scale-factor columns of its own (A on a 32-column boundary, B 16
// further), so that its empty barrier covers them too.  The persistent form has one
// CTA on an SM and two accumulators; the split form two CTAs with one accumulator
// each, whose shared memory holds its sums when the ring is done.
template <int NN, bool SPLIT>
struct Tile {
    static constexpr int kStages = !SPLIT ? 4 : NN == 128 ? 3 : NN == 64 ? 4 : 5;
    static constexpr int kB = NN * kStageK;
    static constexpr int kBlobs = (NN + 127) / 128;           // 512-byte scale blobs of a stage's tokens
    static constexpr int kSf = 512 * (1 + kBlobs);            // W's scale blob, then x's
    static constexpr size_t kOffB = (size_t)kStages * kABytes;
    static constexpr size_t kOffSf = kOffB + (size_t)kStages * kB;
    static constexpr size_t kOffBars = kOffSf + (size_t)kStages * kSf;
    static constexpr size_t kSmem = kOffBars + (2 * kStages + 5) * 8 + 1024;   // + alignment of the ring
    static constexpr int kDCols = NN < 32 ? 32 : NN;
    static constexpr int kSfCol = (SPLIT ? 1 : 2) * kDCols;
    static constexpr int kCols = SPLIT ? 256 : 512;
    static_assert(kSfCol + 32 * kStages <= kCols, "tensor memory");
    static_assert(!SPLIT || (size_t)NN * 128 * 4 <= kOffBars, "sums fit in the ring");
    static_assert(!SPLIT || 2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
};

struct GemmArgs {
    const uint8_t *wscale;        // [ceil(N/128)][KB]
    const uint8_t *xscale;        // [token tiles][KB][kBlobs] blobs of 512 bytes
    uint16_t *y;
    uint32_t *hdr;
    int T, N, KB, n_tiles, tiles;
    int split;                    // CTAs of a cluster
    const uint16_t *x;            // fused form
    int64_t ldx;
    int K;
};

__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity))
        return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > kWaitLimitNs)
            return false;
    return true;
}

// K-major operand rows of 128 bytes in 128-byte-swizzled atoms of 8 rows.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

// Rows of 16 bytes, 8-row groups 128 bytes apart, no swizzle (scale blobs).
__device__ __forceinline__ uint64_t desc_rows16(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(128 >> 4) << 16 | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// A and B E4M3 (0), K-major, UE8M0 scales (bit 23), scale-factor ids 0.
template <int NN>
__host__ __device__ constexpr uint32_t idesc() {
    return ((uint32_t)(NN >> 3) << 17) | (1u << 23) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// The tensor-core instructions are issued by a converged warp, one elected
// lane of it doing so: their operands stay warp-uniform.  (From a branch of one lane an MMA took
// about 200 cycles to issue: 880 a stage instead of the 384 of its products at N = 192.)
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile(
        "{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\n"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
        : "memory");
}

// 512 bytes of scales to four columns of every lane quarter.
__device__ __forceinline__ void copy_scales(uint32_t col, uint32_t blob) {
    asm volatile(
        "{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\n"
        "@p tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n}\n" ::"r"(col),
        "l"(desc_rows16(blob))
        : "memory");
}

template <int NN>
__device__ __forceinline__ void mma(uint32_t d, uint64_t da, uint64_t db, uint32_t sfa, uint32_t sfb, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p, q;\nelect.sync _|p, 0xffffffff;\nsetp.ne.b32 q, %4, 0;\n"
        "@p tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], q;\n}\n" ::"r"(d),
        "l"(da), "l"(db), "n"(idesc<NN>()), "r"(acc), "r"(sfa), "r"(sfb)
        : "memory");
}

// The K stages of one tile that a CTA sums; the tiles of a CTA, one after the other.
struct Range {
    int tile, kb0, kb1, step;
    __device__ __forceinline__ Range(const GemmArgs &a) {
        const int rank = blockIdx.x % a.split;
        tile = blockIdx.x / a.split;
        step = gridDim.x / a.split;
        kb0 = (int)((long long)a.KB * rank / a.split);
        kb1 = (int)((long long)a.KB * (rank + 1) / a.split);
    }
};

__device__ __forceinline__ void store_bf16(uint16_t *dst, float v) {
    uint16_t b;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(v));
    *dst = b;
}

// FUSED (split form, up to 8 tokens): the warps that drain the accumulators first
// quantise x, each cluster for itself, straight into the operand's
// shared-memory layout: no quantisation kernel before this one.
template <int NN, bool SPLIT, bool FUSED>
__global__ void __launch_bounds__(kThreads, SPLIT ? 2 : 1) fp8_gemm_kernel(const __grid_constant__ GemmArgs a,
                                                                           const __grid_constant__ CUtensorMap wmap,
                                                                           const __grid_constant__ CUtensorMap xmap) {
    static_assert(SPLIT || !FUSED, "form");
    using S = Tile<NN, SPLIT>;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t raw_smem[];
    __shared__ uint32_t s_taddr;
    uint8_t *sm = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + S::kOffBars), *empty = full + kStages;
    uint64_t *d_full = empty + kStages, *d_empty = d_full + 2, *spare = d_empty + 2;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + i, FUSED ? 6 : 2);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(d_full + i, 1);
            mbar_init(d_empty + i, 4);
        }
        mbar_init(spare, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_taddr)), "n"(S::kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = s_taddr;
    const Range r0(a);

    if (warp == 0) {
        // ---- copies.  W does not depend on the quantisation of x: the first stages' W goes out before the wait for that
        // kernel, which itself waited for all that came before.  Without one (fused) the kernel before may be the one that
        // writes W: then it is only asked into L2 ahead of the wait.
        auto stage_w = [&](int st, int tile, int kb) {
            mbar_arrive_expect_tx(full + st, kABytes + (FUSED ? 0 : S::kB + 512 * S::kBlobs));
            tma_2d(smem_u32(sm + (size_t)st * kABytes), &wmap, kb * kStageK, tile % a.n_tiles * 128, full + st);
        };
        auto stage_x = [&](int st, int tile, int kb) {
            if (FUSED)
                return;
            const int tt = tile / a.n_tiles;
            tma_2d(smem_u32(sm + S::kOffB + (size_t)st * S::kB), &xmap, kb * kStageK, tt * NN, full + st);
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                    smem_u32(sm + S::kOffSf + (size_t)st * S::kSf + 512)),
                "l"(a.xscale + ((size_t)tt * a.KB + kb) * (512 * S::kBlobs)), "r"(512 * S::kBlobs), "r"(smem_u32(full + st))
                : "memory");
        };
        long long it = 0;                   // stages issued
        bool dead = false, waited = FUSED;
        if (FUSED) {
            if (lane < kStages && r0.kb0 + lane < r0.kb1)
                asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(&wmap)),
                             "r"((r0.kb0 + lane) * kStageK), "r"(r0.tile % a.n_tiles * 128)
                             : "memory");
            pdl_wait();
            pdl_trigger();
        }
        for (int tile = r0.tile; tile < a.tiles && !dead; tile += r0.step) {
            for (int kb = r0.kb0; kb < r0.kb1; ++kb, ++it) {
                const int st = (int)(it % kStages);
                if (it >= kStages) {
                    if (!waited) {          // the ring is full of W: now x's part of it
                        pdl_wait();
                        pdl_trigger();
                        waited = true;
                        if (lane == 0)
                            for (int i = 0; i < kStages; ++i)
                                stage_x(i, r0.tile + i / (r0.kb1 - r0.kb0) * r0.step, r0.kb0 + i % (r0.kb1 - r0.kb0));
                        __syncwarp();
                    }
                    if (!__all_sync(0xffffffffu, wait_phase(empty + st, (uint32_t)((it / kStages - 1) & 1)))) {
                        dead = true;
                        if (lane == 0)
                            record_status(a.hdr, MOE_ERR_DEVICE_TIMEOUT);
                        break;
                    }
                }
                if (lane == 0) {
                    stage_w(st, tile, kb);
                    if (waited)
                        stage_x(st, tile, kb);
                }
                __syncwarp();
            }
        }
        if (!waited) {                      // the whole range fits in the ring
            pdl_wait();
            pdl_trigger();
            if (lane == 0)
                for (int i = 0; i < (int)it; ++i)
                    stage_x(i, r0.tile + i / (r0.kb1 - r0.kb0) * r0.step, r0.kb0 + i % (r0.kb1 - r0.kb0));
            __syncwarp();
        }
        // nothing may be in flight when the CTA ends
        for (long long i = max(0ll, it - kStages); i < it && !dead; ++i)
            wait_phase(full + i % kStages, (uint32_t)((i / kStages) & 1));
    } else if (warp == 1) {
        // ---- MMAs.  Fused: the kernel before may run for long yet, and its time is none of the waits' limit.
        if (FUSED)
            pdl_wait();
        bool dead = false;
        int it = 0, piece = 0;
        for (int tile = r0.tile; tile < a.tiles && !dead; tile += r0.step, ++piece) {
            const int buf = SPLIT ? 0 : piece & 1;
            if (piece >= 2)
                dead = !__all_sync(0xffffffffu, wait_phase(d_empty + buf, (uint32_t)((piece / 2 - 1) & 1)));
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t d = tmem + buf * S::kDCols;
            for (int kb = r0.kb0; kb < r0.kb1 && !dead; ++kb, ++it) {
                const int st = it % kStages;
                if (!__all_sync(0xffffffffu, wait_phase(full + st, (uint32_t)((it / kStages) & 1)))) {
                    dead = true;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t sfa = tmem + S::kSfCol + 32 * st, sfb = sfa + 16;
                const uint32_t sf = smem_u32(sm + S::kOffSf + (size_t)st * S::kSf);
                copy_scales(sfa, sf);
#pragma unroll
                for (int j = 0; j < S::kBlobs; ++j)
                    copy_scales(sfb + 4 * j, sf + 512 * (j + 1));
                const uint64_t da = desc_sw128(smem_u32(sm + (size_t)st * kABytes)), db = desc_sw128(smem_u32(sm + S::kOffB + (size_t)st * S::kB));
#pragma unroll
                for (int j = 0; j < 4; ++j)              // 32 elements of K: 32 bytes, 2 in the descriptor's unit
                    mma<NN>(d, da + 2 * j, db + 2 * j, sfa, sfb, kb > r0.kb0 || j > 0);
                commit(empty + st);
            }
            commit(d_full + buf);
        }
        if (dead) {
            if (lane == 0)
                record_status(a.hdr, MOE_ERR_DEVICE_TIMEOUT);
            commit(spare);                     // issued MMAs end before the CTA's memory goes away
            wait_phase(spare, 0);
        }
        __syncwarp();
    } else if (warp >= 6) {
        // ---- W's scale, warps in turn: a stage's blob is one byte throughout
        if (FUSED)
            pdl_wait();
        long long it = 0;
        bool dead = false;
        for (int tile = r0.tile; tile < a.tiles && !dead; tile += r0.step) {
            const uint8_t *wsrow = a.wscale + (size_t)(tile % a.n_tiles) * a.KB;
            uint32_t wsc = 0;               // of 32 stages, a byte a lane
            for (int kb = r0.kb0; kb < r0.kb1; ++kb, ++it) {
                const int st = (int)(it % kStages), o = (kb - r0.kb0) & 31;
                if (o == 0)
                    wsc = kb + lane < r0.kb1 ? __ldg(wsrow + kb + lane) : 0;
                if ((it & 1) != (warp & 1))
                    continue;
                if (it >= kStages && !__all_sync(0xffffffffu, wait_phase(empty + st, (uint32_t)((it / kStages - 1) & 1)))) {
                    dead = true;
                    break;
                }
                const uint32_t w = __shfl_sync(0xffffffffu, wsc, o) * 0x01010101u;
                *reinterpret_cast<uint4 *>(sm + S::kOffSf + (size_t)st * S::kSf + lane * 16) = make_uint4(w, w, w, w);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(full + st);
            }
        }
    } else {
        // ---- accumulators to y (split: to shared memory, joined below)
        pdl_wait();
        if (FUSED) {
            // half a warp for each token and stage, four loads in flight
            const int l = lane & 15, r = (warp - 2) * 2 + (lane >> 4), tok0 = r0.tile / a.n_tiles * NN;
            constexpr int kPasses = 1, kAhead = 4;      // 8 tokens a pass
            const int jobs = (r0.kb1 - r0.kb0) * kPasses;
            bool dead = false;
            for (int j0 = 0; j0 < jobs; j0 += kAhead) {
                uint4 v[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int j = j0 + u, t = tok0 + j % kPasses * 8 + r, k = (r0.kb0 + j / kPasses) * 128 + l * 8;
                    v[u] = j < jobs && t < a.T && k < a.K ? __ldg(reinterpret_cast<const uint4 *>(a.x + t * a.ldx + k)) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int j = j0 + u, s = j / kPasses, row = j % kPasses * 8 + r, st = s % kStages;
                    if (j >= jobs)
                        break;
                    if (s >= kStages && j % kPasses == 0 && !dead) {
                        dead = !__all_sync(0xffffffffu, wait_phase(empty + st, (uint32_t)((s / kStages - 1) & 1)));
                        if (dead && lane == 0)
                            record_status(a.hdr, MOE_ERR_DEVICE_TIMEOUT);
                    }
                    uint32_t m = amax_bf16x8(v[u]);
#pragma unroll
                    for (int d = 8; d > 0; d >>= 1)
                        m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
                    const int sc = fp8_scale_byte(m);
                    if (tok0 + row < a.T) {
                        // 128-byte rows, their 16-byte chunks permuted by the row within an atom of 8
                        uint8_t *dst = sm + S::kOffB + (size_t)st * S::kB + row * 128 + (((l >> 1) ^ (row & 7)) << 4) + (l & 1) * 8;
                        *reinterpret_cast<uint2 *>(dst) = fp8_from_bf16x8(v[u], exp2i(127 - sc));
                        if (l == 0)
                            reinterpret_cast<uint32_t *>(sm + S::kOffSf + (size_t)st * S::kSf + 512)[(row % 32) * 4 + row / 32] = sc * 0x01010101u;
                    }
                    if (j % kPasses == kPasses - 1) {
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(full + st);
                    }
                }
            }
        }
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        int piece = 0;
        bool dead = false;
        for (int tile = r0.tile; tile < a.tiles && !dead; tile += r0.step, ++piece) {
            const int buf = SPLIT ? 0 : piece & 1;
            const int n = tile % a.n_tiles * 128 + row, tok0 = tile / a.n_tiles * NN, toks = min(NN, a.T - tok0);
            if (!__all_sync(0xffffffffu, wait_phase(d_full + buf, (uint32_t)((SPLIT ? piece : piece / 2) & 1)))) {
                dead = true;
                if (lane == 0)
                    record_status(a.hdr, MOE_ERR_DEVICE_TIMEOUT);
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
            for (int q = 0; q < NN; q += 16) {
                if (q < toks) {
                    uint32_t v[16];
                    asm volatile(
                        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
                        "tcgen05.wait::ld.sync.aligned;"
                        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                        : "r"(tmem + lanes + buf * S::kDCols + q)
                        : "memory");
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        if (q + j >= toks)
                            break;
                        if (SPLIT && a.split > 1)
                            reinterpret_cast<float *>(sm)[(q + j) * 128 + row] = __uint_as_float(v[j]);
                        else if (n < a.N)
                            store_bf16(a.y + (size_t)(tok0 + q + j) * a.N + n, __uint_as_float(v[j]));
                    }
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                mbar_arrive(d_empty + buf);
        }
    }
    if (SPLIT && a.split > 1) {
        // the cluster's sums of the tile, each CTA adding every split-th token's; K ascends with the rank
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        const int rank = blockIdx.x % a.split, tok0 = r0.tile / a.n_tiles * NN, toks = min(NN, a.T - tok0);
        for (int i = tid; i < 32 * ((toks - rank + a.split - 1) / a.split); i += kThreads) {
            const int row = (i & 31) * 4, q = rank + (i >> 5) * a.split, n = r0.tile % a.n_tiles * 128 + row;
            const uint32_t at = smem_u32(reinterpret_cast<float *>(sm) + q * 128 + row);
            float4 v[kMaxSplit];
#pragma unroll
            for (int c = 0; c < kMaxSplit; ++c)
                if (c < a.split) {
                    uint32_t remote;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(c));
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[c].x), "=f"(v[c].y), "=f"(v[c].z), "=f"(v[c].w) : "r"(remote));
                }
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < kMaxSplit; ++c)
                if (c < a.split) {
                    s[0] += v[c].x;
                    s[1] += v[c].y;
                    s[2] += v[c].z;
                    s[3] += v[c].w;
                }
            uint16_t *dst = a.y + (size_t)(tok0 + q) * a.N + n;
            if (n + 4 <= a.N && a.N % 4 == 0) {
                uint32_t lo, hi;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(s[1]), "f"(s[0]));
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(s[3]), "f"(s[2]));
                *reinterpret_cast<uint2 *>(dst) = make_uint2(lo, hi);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < a.N)
                        store_bf16(dst + e, s[e]);
            }
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kCols));
}

constexpr int kQuantGroups = 4;

// x to codes [T][KB * 128] and scale blobs: half a warp for each group of 128, four loads in flight a thread.
// A token tile's blob for a K stage holds token r's byte, four times, in word
// (r % 32) * 4 + r / 32: the order in which tensor memory keeps the scales of 128 rows.
__global__ void __launch_bounds__(256) fp8_quant_kernel(const uint16_t *__restrict__ x, int64_t ldx, int T, int K, int KB,
                                                        int tile, int blobs, uint8_t *__restrict__ codes,
                                                        uint32_t *__restrict__ scales) {
    pdl_wait();
    pdl_trigger();
    const int l = threadIdx.x & 15, groups = T * KB, first = blockIdx.x * (16 * kQuantGroups) + (threadIdx.x >> 4);
    uint4 v[kQuantGroups];
#pragma unroll
    for (int u = 0; u < kQuantGroups; ++u) {
        const int i = first + 16 * u, t = i / KB, k = (i - t * KB) * 128 + l * 8;
        v[u] = i < groups && k < K ? __ldg(reinterpret_cast<const uint4 *>(x + t * ldx + k)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kQuantGroups; ++u) {
        const int i = first + 16 * u;
        uint32_t m = amax_bf16x8(v[u]);
#pragma unroll
        for (int d = 8; d > 0; d >>= 1)
            m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        const int s = fp8_scale_byte(m);
        if (i < groups) {
            const int t = i / KB, kb = i - t * KB;
            *reinterpret_cast<uint2 *>(codes + (size_t)i * 128 + l * 8) = fp8_from_bf16x8(v[u], exp2i(127 - s));
            if (l == 0) {
                const int tt = t / tile, r = t - tt * tile;
                scales[(((size_t)tt * KB + kb) * blobs + r / 128) * 128 + (r % 32) * 4 + (r % 128) / 32] = s * 0x01010101u;
            }
        }
    }
}

// One CTA for each 128 x 128 block of W, held in registers.
__global__ void __launch_bounds__(256) fp8_weight_kernel(const uint16_t *__restrict__ w, int N, int K,
                                                         uint8_t *__restrict__ codes, uint8_t *__restrict__ scale) {
    __shared__ uint32_t red[8];
    pdl_wait();
    pdl_trigger();
    const int k = blockIdx.x * 128 + (threadIdx.x & 15) * 8, r0 = blockIdx.y * 128 + (threadIdx.x >> 4);
    uint4 v[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        v[i] = r < N && k < K ? __ldg(reinterpret_cast<const uint4 *>(w + (size_t)r * K + k)) : make_uint4(0, 0, 0, 0);
        m = max(m, amax_bf16x8(v[i]));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, red[i]);
    const int s = fp8_scale_byte(m);
    if (threadIdx.x == 0)
        scale[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = (uint8_t)s;
    const float inv = exp2i(127 - s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        if (r < N && k < K)
            *reinterpret_cast<uint2 *>(codes + (size_t)r * K + k) = fp8_from_bf16x8(v[i], inv);
    }
}

// Token tile and form for T tokens and the tiles of N.  The split form's tile is the least
// width that holds the tokens, up to 128, two CTAs to an SM; the persistent form's is 192, one CTA.
struct Form {
    bool split_form;
    int tile, split;
    static Form make(int T, int N, int KB, int sms) {
        Form f{};
        const int n_tiles = (N + 127) / 128;
        f.tile = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
        // The split form for a token tile or less (us of it and of the persistent form: one token and W 45056 x 5120 45.5 and 84.0, 64 and
        // 131072 x 4096 98.8 and 105.3, 100 110.1 and 108.0); for more while its tiles have an SM each, or share one where the persistent
        // form would walk twice (7168 x 5120: 200 tokens, 112 tiles, 20.4 and 25.6; 384, 168 tiles against 112, 28.0 and 26.4; 576, 280
        // against 168, 30.3 and 42.0; 700, 336 against 224, 49.7 and 42.1).
        const long long split_tiles = (long long)n_tiles * ((T + f.tile - 1) / f.tile), wide_tiles = (long long)n_tiles * ((T + 191) / 192);
        f.split_form = T <= 128 || split_tiles <= sms || (wide_tiles > sms && split_tiles <= 2 * sms);
        if (!f.split_form)
            f.tile = 192;
        f.split = 1;
        if (f.split_form) {
            const int tiles = n_tiles * ((T + f.tile - 1) / f.tile);
            // the largest cluster of which all run at once: two CTAs on an SM, a cluster within one of the eight
            // groups of SMs, a tenth to spare (7168 x 5120, 17 tokens: 10.9 us with 4, 16.4 with 5, whose 56 clusters
            // just do not fit)
            for (int s = 1; s <= kMaxSplit && s <= KB; ++s)
                if (tiles * 11 <= 10 * 8 * (2 * (sms / 8) / s))
                    f.split = s;
        }
        return f;
    }
};

// x quantised in the GEMM, each cluster for itself, or by a kernel before it (7168 x 5120, one token 8.9 and 9.6 us, 8 tokens 9.6
// and 10.9; a second pass of 8 over x costs a stage more than its copies hide)
constexpr int kFusedTokens = 8;

struct Layout {
    size_t codes, scales, total;
    // scale blobs for any form: tiles of at least min(T, 192) tokens in blobs of 128 rows
    static Layout make(int T, int K) {
        Layout L{};
        const size_t KB = (size_t)(K + 127) / 128;
        size_t blobs = 0;
        for (int tile : {16, 32, 64, 128, 192})
            if (tile >= T || tile >= 128) {
                const size_t n = (size_t)((T + tile - 1) / tile) * ((tile + 127) / 128);
                blobs = n > blobs ? n : blobs;
            }
        size_t o = kInitBytes;
        auto take = [&](size_t bytes) { o = align_up(o, 256); size_t r = o; o += bytes; return r; };
        L.codes = take((size_t)T * KB * 128);
        L.scales = take(blobs * KB * 512);
        L.total = align_up(o, 256);
        return L;
    }
};

template <int NN, bool SPLIT, bool FUSED>
cudaError_t launch_gemm(const GemmArgs &a, const CUtensorMap &wmap, const uint8_t *codes, int ctas, cudaStream_t stream) {
    using S = Tile<NN, SPLIT>;
    CUtensorMap xmap = wmap;                        // not read by the fused form
    const uint64_t dims[2] = {(uint64_t)a.KB * 128, (uint64_t)a.T}, str[1] = {(uint64_t)a.KB * 128};
    const uint32_t box[2] = {128, NN};
    cudaError_t e = FUSED ? cudaSuccess
                          : encode_tiled(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fp8_gemm_kernel<NN, SPLIT, FUSED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
    if (e == cudaSuccess && SPLIT)
        e = cudaFuncSetAttribute(fp8_gemm_kernel<NN, SPLIT, FUSED>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)a.split, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<NN, SPLIT, FUSED>, a, wmap, xmap);
}

}  // namespace

size_t linear_fp8_workspace(int T, int N, int K) {
    (void)N;
    return Layout::make(T, K).total;
}

cudaError_t launch_linear_fp8(const LinearProblem &p, void *ws, int sms, cudaStream_t stream) {
    const int KB = (p.K + 127) / 128;
    const Form f = Form::make(p.T, p.N, KB, sms);
    const Layout L = Layout::make(p.T, p.K);
    uint8_t *codes = ws_at<uint8_t>(ws, L.codes);
    uint32_t *scales = ws_at<uint32_t>(ws, L.scales);
    GemmArgs a{};
    a.wscale = p.scale;
    a.xscale = reinterpret_cast<const uint8_t *>(scales);
    a.y = p.y;
    a.hdr = ws_at<uint32_t>(ws, 0);
    a.T = p.T;
    a.N = p.N;
    a.KB = KB;
    a.n_tiles = (p.N + 127) / 128;
    a.tiles = a.n_tiles * ((p.T + f.tile - 1) / f.tile);
    a.split = f.split;
    CUtensorMap wmap;
    const uint64_t dims[2] = {(uint64_t)p.K, (uint64_t)p.N}, str[1] = {(uint64_t)p.K};
    const uint32_t box[2] = {128, 128};
    cudaError_t e = encode_tiled(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.codes, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess)
        return e;
    a.x = p.x;
    a.ldx = p.ldx;
    a.K = p.K;
    const int ctas = a.tiles * f.split;
    if (f.split_form && p.T <= kFusedTokens)
        return launch_gemm<16, true, true>(a, wmap, codes, ctas, stream);
    const int groups = p.T * KB, per = 16 * kQuantGroups;       // at most 2^29
    e = launch_pdl(fp8_quant_kernel, dim3((groups + per - 1) / per), dim3(256), 0, stream, p.x, p.ldx, p.T, p.K, KB,
                   f.tile, (f.tile + 127) / 128, codes, scales);
    if (e != cudaSuccess)
        return e;
    if (!f.split_form)
        return launch_gemm<192, false, false>(a, wmap, codes, a.tiles < sms ? a.tiles : sms, stream);
    switch (f.tile) {
    case 16: return launch_gemm<16, true, false>(a, wmap, codes, ctas, stream);
    case 32: return launch_gemm<32, true, false>(a, wmap, codes, ctas, stream);
    case 64: return launch_gemm<64, true, false>(a, wmap, codes, ctas, stream);
    default: return launch_gemm<128, true, false>(a, wmap, codes, ctas, stream);
    }
}

cudaError_t launch_quantize_fp8_weight(const uint16_t *w, int N, int K, uint8_t *codes, uint8_t *scale,
                                       cudaStream_t stream) {
    return launch_pdl(fp8_weight_kernel, dim3((K + 127) / 128, (N + 127) / 128), dim3(256), 0, stream, w, N, K, codes, scale);
}

}  // namespace moe
