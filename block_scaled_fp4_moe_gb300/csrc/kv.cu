// kv.cu -- the paged E4M3 cache's bookkeeping: block tables and slot maps from
// request lengths, and the append of new keys and values.
#include "attn.h"

namespace moe {
namespace {

constexpr int kTablesThreads = 512;

// Inclusive sum over the block of a pair of 64-bit counts; *total is the
// block's sum.  red: 2 * 32 words of shared memory.
__device__ __forceinline__ ulonglong2 block_scan2(ulonglong2 v, ulonglong2 *red, ulonglong2 *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long a = __shfl_up_sync(0xffffffffu, v.x, d), b = __shfl_up_sync(0xffffffffu, v.y, d);
        if (lane >= d) {
            v.x += a;
            v.y += b;
        }
    }
    if (lane == 31)
        red[warp] = v;
    __syncthreads();
    if (warp == 0) {
        ulonglong2 w = lane < nw ? red[lane] : make_ulonglong2(0, 0);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned long long a = __shfl_up_sync(0xffffffffu, w.x, d), b = __shfl_up_sync(0xffffffffu, w.y, d);
            if (lane >= d) {
                w.x += a;
                w.y += b;
            }
        }
        red[lane] = w;
    }
    __syncthreads();
    if (warp > 0) {
        v.x += red[warp - 1].x;
        v.y += red[warp - 1].y;
    }
    *total = red[nw - 1];
    return v;
}

// Tables of a step.  Every CTA sums the B requests' new tokens and new blocks
// itself (8 B bytes from L2, one block-wide scan: cheaper than a second
// launch or a wait between CTAs) and so agrees on the checks; then each
// thread finds its token's request by bisection in shared memory and derives
// block, slot and position.  A token at a block boundary writes the block's
// table entry: every block that a step adds holds one such token.  Bound by
// latency: one chain of length loads, scan, bisection, free-list load.
__global__ void __launch_bounds__(kTablesThreads) kv_tables_kernel(TablesProblem p) {
    extern __shared__ int32_t sm[];
    __shared__ ulonglong2 red[32];
    int32_t *s_ctx = sm, *s_off = sm + p.B, *s_blk = s_off + p.B + 1;   // cached tokens, first token, first new block
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, sh = p.block_shift, bs = 1 << sh;
    const long long cap = (long long)p.max_blocks << sh;
    const int per = (p.B + kTablesThreads - 1) / kTablesThreads;
    const int head = *p.free_head;
    int bad = head < 0;
    for (int b = tid; b < p.B; b += kTablesThreads) {
        const int c = p.ctx[b], n = p.fresh[b];
        bad |= c < 0 || n < 0 || (long long)c + n > cap;
        s_ctx[b] = c;
        s_off[b] = n;
    }
    if (__syncthreads_or(bad)) {
        if (blockIdx.x == 0 && tid == 0)
            record_status(p.hdr, MOE_ERR_DEVICE_ASSERT);
        return;
    }
    // held and new blocks; lengths are at most max_blocks * block_size < 2^31
    auto before = [&](int c) { return (int)(((long long)c + bs - 1) >> sh); };
    auto made = [&](int c, int n) { return (int)(((long long)c + n + bs - 1) >> sh) - before(c); };
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    ulonglong2 mine = make_ulonglong2(0, 0), total;
    for (int b = b0; b < b1; ++b) {
        mine.x += s_off[b];
        mine.y += made(s_ctx[b], s_off[b]);
    }
    const ulonglong2 incl = block_scan2(mine, red, &total);
    if (total.x > (unsigned long long)p.T || (unsigned long long)head + total.y > (unsigned long long)p.num_free) {
        if (blockIdx.x == 0 && tid == 0)
            record_status(p.hdr, MOE_ERR_DEVICE_ASSERT);
        return;
    }
    int off = (int)(incl.x - mine.x), blk = (int)(incl.y - mine.y);
    for (int b = b0; b < b1; ++b) {
        const int n = s_off[b];
        s_off[b] = off;
        s_blk[b] = blk;
        off += n;
        blk += made(s_ctx[b], n);
    }
    const int n_tok = (int)total.x;
    if (tid == 0)
        s_off[p.B] = n_tok;
    __syncthreads();
    const int stride = gridDim.x * kTablesThreads;
    for (int b = blockIdx.x * kTablesThreads + tid; b <= p.B; b += stride) {
        p.q_offsets[b] = s_off[b];
        if (b < p.B)
            p.kv_lens[b] = s_ctx[b] + s_off[b + 1] - s_off[b];
        else
            *p.free_head_out = head + (int)total.y;
    }
    for (int t = blockIdx.x * kTablesThreads + tid; t < p.T; t += stride) {
        if (t >= n_tok) {
            p.slot_map[t] = -1;
            p.positions[t] = -1;
            continue;
        }
        int lo = 0, hi = p.B;                    // s_off[lo] <= t < s_off[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_off[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        const int c = s_ctx[lo], pos = c + t - s_off[lo], idx = pos >> sh, held = before(c);
        const int taken = head + s_blk[lo] + idx - held;        // place in the free list of a block that is new
        if (!MOE_DBG_IN_RANGE(idx, p.max_blocks, p.hdr) || (idx >= held && !MOE_DBG_IN_RANGE(taken, p.num_free, p.hdr)))
            continue;
        int32_t *entry = p.table + (size_t)lo * p.max_blocks + idx;
        int id;
        if (idx < held) {
            id = *entry;
        } else {
            id = p.free_blocks[taken];
            if ((pos & (bs - 1)) == 0)
                *entry = id;
        }
        p.slot_map[t] = ((int64_t)id << sh) + (pos & (bs - 1));
        p.positions[t] = pos;
    }
}

// ----------------------------------------------------------------- append

constexpr int kAppendThreads = 256, kAppendWarps = kAppendThreads / 32;
constexpr int kAppendWindow = 32;       // tokens a CTA looks at, at most
constexpr int kShortRun = 4;            // tokens of a run that one warp appends
#ifdef MOE_DEBUG_BOUNDS
constexpr int kLookBack = 128;          // skipped tokens over which a run's predecessor is looked for
#endif

// 16 codes of a block whose exponent grew, rounded to the new one (f = 2^-growth);
// the first `held` of them are the block's, the rest stays as it is.
__device__ __forceinline__ uint4 recode(uint4 c, float f, int held) {
    uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t o = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t h2 = e4m3x2_to_f16x2((uint16_t)(w[q] >> (16 * e)));
            const float2 f2 = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
            o |= fp8_pair(f2.x, f2.y, f) << (16 * e);
        }
        const int n = held - 4 * q;
        const uint32_t keep = n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (8 * n)) - 1;
        w[q] = (o & keep) | (w[q] & ~keep);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The codes of a block's first off0 tokens, by threads `first` of `count`: 16
// bytes are a token's 16 dims (keys) or a dim's 16 tokens (values).  kFlight
// of them at a time: the stores may alias the loads, which otherwise wait.
template <int D, int kFlight>
__device__ __forceinline__ void recode_block(uint8_t *codes, bool is_v, int off0, float f, int first, int count) {
    const int units = (off0 + 15) / 16 * D;
    for (int u0 = first; u0 < units; u0 += kFlight * count) {
        uint4 c[kFlight];
        int held[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const int u = u0 + i * count, token = is_v ? u / D * 16 : u / (16 * (D / 16)) * 16 + u % 16;
            held[i] = u >= units || token >= off0 ? 0 : is_v ? off0 - token : 16;
            if (held[i])
                c[i] = reinterpret_cast<const uint4 *>(codes)[u];
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i)
            if (held[i])
                reinterpret_cast<uint4 *>(codes)[u0 + i * count] = recode(c[i], f, held[i]);
    }
}

// A CTA looks at `window` consecutive tokens, for one head of the keys
// (blockIdx.z = 0) or values (1), and works for those that begin a run of
// tokens in one block (a run may reach past the window).  Runs of up to
// kShortRun tokens, the decode steps', are a warp's work each; a longer one is
// the whole CTA's, which holds the block's new tokens in registers (at most
// 128 x 128 bf16 = 8 x 16 bytes a thread).  Both take the run's largest magnitude,
// settle the exponent, re-round the codes that the block held where the exponent grew, and
// write the new codes: one pass over the input, no atomics on global memory.
//
// Bound: latency, of the chain slots -> input -> exponent -> codes.  64 requests of
// one token (8 heads of 128) take 3.4 us, 256 take 6.6 and 400 take 8.6; with a CTA for
// every run they took 5.8, 17.4 and 26.6, since few CTAs fit an SM.  5,000 prompt tokens in blocks of
// 64 take 15.1 us (2.1 TB/s in and out); four CTAs an SM at 64 registers are ahead of three (22 us)
// and of five that spill (20 us).
template <int D>
__global__ void __launch_bounds__(kAppendThreads, 4) kv_append_kernel(AppendProblem p, int window) {
    constexpr int kLanes = D / 8;                       // threads per token (16 bytes each)
    constexpr int kTok = kAppendThreads / kLanes;       // tokens per step
    constexpr int kSteps = 128 / kTok;
    __shared__ __align__(16) uint8_t s_code[128 * D];   // values: codes [token][dim] before the transpose
    __shared__ uint32_t s_max[kAppendWarps];
    __shared__ int64_t s_slot[kAppendWindow + 128];     // of the tokens from the one before the window on; < 0: none
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const int bs = p.cache.block_size, sh = 31 - __clz(bs);
    const uint16_t *src = (is_v ? p.v + h * p.v_sh : p.k + h * p.k_sh);
    const int64_t st = is_v ? p.v_st : p.k_st;
    const int64_t n_slots = (int64_t)p.cache.num_blocks << sh;
    const int t0 = blockIdx.x * window;
    for (int i = tid; i < window + bs; i += kAppendThreads) {
        const int t = t0 - 1 + i;
        int64_t slot = t >= 0 && t < p.T ? p.slots[t] : -1;
        if (slot >= n_slots) {
            record_status(p.hdr, MOE_ERR_DEVICE_ASSERT);
            slot = -1;
        }
        s_slot[i] = slot;
    }
    __syncthreads();
    // which tokens of the window begin a run (their block is not that of the token before), and which of
    // these runs are short
    const int64_t here = lane < window ? s_slot[1 + lane] : -1;
    bool begins = false, brief = false;
    if (here >= 0) {
        const int64_t prev = s_slot[lane];
        begins = prev < 0 || (prev >> sh) != (here >> sh);
#ifdef MOE_DEBUG_BOUNDS
        // What the caller must not do (a look at it costs a decode step's append a tenth of its time): a block's tokens that do not follow one
        // another in it, or go on behind skipped ones, where another warp settles the block's scale already.
        bool apart = !begins && here != prev + 1;
        if (prev < 0) {
            int64_t last = -1;
            for (int t = t0 + lane - 1, left = kLookBack; last < 0 && t > 0 && left > 0; --left) {
                last = p.slots[--t];
                if (last >= n_slots)
                    last = -1;
            }
            if (last >= 0 && (last >> sh) == (here >> sh)) {
                begins = false;
                apart = true;
            }
        }
        if (apart)
            record_status(p.hdr, MOE_ERR_DEVICE_ASSERT);
#endif
        brief = bs - (int)(here & (bs - 1)) <= kShortRun;
#pragma unroll
        for (int j = 1; j <= kShortRun; ++j)            // kShortRun < bs: within s_slot
            brief = brief || (s_slot[1 + lane + j] >> sh) != (here >> sh);
    }
    const uint32_t all = __ballot_sync(0xffffffffu, begins), shorts = __ballot_sync(0xffffffffu, begins && brief);

    uint8_t *scales = is_v ? p.cache.v_scale : p.cache.k_scale, *pool = is_v ? p.cache.v : p.cache.k;
    int turn = 0;
    for (uint32_t left = shorts; left; left &= left - 1, ++turn) {
        if (turn % kAppendWarps != warp)
            continue;
        constexpr int kHold = kShortRun * kLanes / 32;  // 16-byte pieces a lane
        const int w0 = __ffs(left), t = t0 + w0 - 1;
        const int64_t slot = s_slot[w0], blk = slot >> sh;
        const int off0 = (int)(slot & (bs - 1));
        const int n = min(bs - off0,
                          __ffs(__ballot_sync(0xffffffffu, lane >= kShortRun || (s_slot[w0 + lane] >> sh) != blk)) - 1);
        uint8_t *scale = scales + blk * p.cache.kv_heads + h;
        uint8_t *codes = pool + ((size_t)blk * p.cache.kv_heads + h) * bs * D;
        const int was = off0 > 0 ? *scale : 0;
        const int dim = lane % kLanes * 8;
        uint4 x[kHold];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int r = (i * 32 + lane) / kLanes;
            x[i] = r < n ? __ldg(reinterpret_cast<const uint4 *>(src + (t + r) * st + dim)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kHold; ++i)
            m = max(m, amax_bf16x8(x[i]));
        m = __reduce_max_sync(0xffffffffu, m);
        const int s = max(fp8_scale_byte(m), was);
        if (off0 > 0 && was < s)
            recode_block<D, 4>(codes, is_v, off0, exp2i(max(was - s, -126)), lane, 32);
        __syncwarp();                                   // old scale read, old codes rewritten
        if (lane == 0)
            *scale = (uint8_t)s;
        const float inv = exp2i(max(127 - s, -126));
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int r = (i * 32 + lane) / kLanes, o = off0 + r;
            if (r >= n)
                continue;
            const uint2 c = fp8_from_bf16x8(x[i], inv);
            if (is_v) {
                uint8_t *dst = codes + (size_t)((o >> 4) * D + dim) * 16 + (o & 15);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    dst[16 * j] = (uint8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
            } else {
                *reinterpret_cast<uint2 *>(codes + (o >> 4) * 16 * D + (dim >> 4) * 256 + (o & 15) * 16 + (dim & 15)) = c;
            }
        }
    }

    for (uint32_t left = all & ~shorts; left; left &= left - 1) {
        const int w0 = __ffs(left), t = t0 + w0 - 1;
        const int64_t slot = s_slot[w0], blk = slot >> sh;
        // run length: up to the first token that lies elsewhere, or the block's end
        const int off0 = (int)(slot & (bs - 1));
        int n = bs - off0;
        for (int j = 0; j < n; j += 32) {
            const uint32_t ends = __ballot_sync(0xffffffffu, j + lane >= n || (s_slot[w0 + j + lane] >> sh) != blk);
            if (ends) {
                n = min(n, j + __ffs(ends) - 1);
                break;
            }
        }
        uint8_t *scale = scales + blk * p.cache.kv_heads + h;
        uint8_t *codes = pool + ((size_t)blk * p.cache.kv_heads + h) * bs * D;
        const int was = off0 > 0 ? *scale : 0;
        // the new tokens, and their largest magnitude
        const int dim = (tid % kLanes) * 8, row = tid / kLanes;
        uint4 x[kSteps];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            if (i * kTok < n) {
                const int r = i * kTok + row;
                x[i] = r < n ? __ldg(reinterpret_cast<const uint4 *>(src + (t + r) * st + dim)) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            if (i * kTok < n)
                m = max(m, amax_bf16x8(x[i]));
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0)
            s_max[warp] = m;
        __syncthreads();
        m = __reduce_max_sync(0xffffffffu, s_max[lane % kAppendWarps]);
        const int s = max(fp8_scale_byte(m), was);
        if (off0 > 0 && was < s)
            recode_block<D, 1>(codes, is_v, off0, exp2i(max(was - s, -126)), tid, kAppendThreads);
        __syncthreads();                                // old scale read, old codes rewritten
        if (tid == 0)
            *scale = (uint8_t)s;
        const float inv = exp2i(max(127 - s, -126));
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = i * kTok + row;
            if (i * kTok < n && r < n) {
                const uint2 c = fp8_from_bf16x8(x[i], inv);
                if (is_v) {
                    *reinterpret_cast<uint2 *>(s_code + r * D + dim) = c;
                } else {
                    const int o = off0 + r;
                    *reinterpret_cast<uint2 *>(codes + (o >> 4) * 16 * D + (dim >> 4) * 256 + (o & 15) * 16 + (dim & 15)) = c;
                }
            }
        }
        if (is_v) {
            __syncthreads();
            // transposed: 16 tokens of one dim are 16 bytes
            const int sub0 = off0 >> 4, subs = ((off0 + n - 1) >> 4) - sub0 + 1;
            for (int u = tid; u < subs * D; u += kAppendThreads) {
                const int sub = sub0 + u / D, d = u % D;
                uint8_t *dst = codes + (size_t)(sub * D + d) * 16;
                const int r0 = sub * 16 - off0;         // row of the sub-block's first token
                if (r0 >= 0 && r0 + 16 <= n) {
                    uint32_t w[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        w[q] = s_code[(r0 + 4 * q) * D + d] | s_code[(r0 + 4 * q + 1) * D + d] << 8 |
                               s_code[(r0 + 4 * q + 2) * D + d] << 16 | (uint32_t)s_code[(r0 + 4 * q + 3) * D + d] << 24;
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    for (int j = max(0, -r0); j < 16 && r0 + j < n; ++j)
                        dst[j] = s_code[(r0 + j) * D + d];
                }
            }
        }
        __syncthreads();                                // s_code, s_max free for the next run
    }
}

}  // namespace

cudaError_t launch_kv_tables(const TablesProblem &p, cudaStream_t stream) {
    const size_t smem = (size_t)(3 * p.B + 1) * sizeof(int32_t);
    if (smem > 40 * 1024) {             // 48 KB without asking, of which the kernel's static memory takes its part
        // a limit of the whole process: the same one from every thread's call
        const cudaError_t e = cudaFuncSetAttribute(kv_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (3 * kMaxRequests + 1) * (int)sizeof(int32_t));
        if (e != cudaSuccess)
            return e;
    }
    const int items = p.T > p.B + 1 ? p.T : p.B + 1;
    int grid = (items + kTablesThreads - 1) / kTablesThreads;
    if (grid > 304)                     // two CTAs per SM; more would repeat the scan without need
        grid = 304;
    return launch_pdl(kv_tables_kernel, dim3(grid), dim3(kTablesThreads), smem, stream, p);
}

cudaError_t launch_kv_append(const AppendProblem &p, cudaStream_t stream) {
    // few tokens: a run for each warp, were all of them short; many: fewer CTAs that find no run to begin
    // (us with 8 and with 32 tokens a CTA: 5,000 prompt tokens 23.4 and 16.0, 600 prompt tokens 5.1 and 9.2,
    // 600 tokens of as many requests 11.0 and 12.5)
    const int window = p.T <= 1024 ? kAppendWarps : kAppendWindow;
    const dim3 grid((p.T + window - 1) / window, p.cache.kv_heads, 2);
    return p.cache.head_dim == 64 ? launch_pdl(kv_append_kernel<64>, grid, dim3(kAppendThreads), 0, stream, p, window)
                                  : launch_pdl(kv_append_kernel<128>, grid, dim3(kAppendThreads), 0, stream, p, window);
}

}  // namespace moe
