// attn_plan.cuh -- what the two attention kernels share: units of work, the
// plan that lists them, and a CTA's walk through its range (attn.cu says how).
#pragma once

#include "attn.h"

namespace moe {
namespace {

constexpr int kTile = 128;             // tokens of a tile
constexpr int kSubs = kTile / 16;      // sub-blocks of a tile
constexpr int kUnitCost = 2;           // a unit's fixed work, in tiles
// Least range of a CTA, in tiles (us with 2, 4 and 6: one request of 1,000 tokens 9.8, 10.8 and 13.4, four of 2,000 12.2, 14.5 and 15.4).
constexpr int kMinCost = 2;
constexpr int kPlanThreads = 1024;
constexpr unsigned long long kWaitLimitNs = 200ull * 1000 * 1000;

// A row tile of a request.
struct RowTile {
    long long before;         // work of the row tiles before it (all heads), in tiles
    int request, q0, n, kv;   // its first row of q, new tokens, tokens
    int row0;                 // first row (of new tokens x group)
    int tile0, tiles;         // cache tiles it sees
};

struct Plan {
    long long work;        // of all units
    long long per;         // of a CTA
    int row_tiles, ctas;
};

struct AttnArgs {
    AttnProblem p;
    int group, shift;                    // query heads of a key/value head; log2(block_size)
    int rows, part_rows;                 // of a unit; of a part in the workspace
    int ctas, max_tiles;
    float scale_log2;
    Plan *plan;
    RowTile *recs;
    uint32_t *tickets;
    float *part;                         // parts of cut units: their rows,
    float2 *part_sum;                    // and their m and l (attn.cu: l 2^-31)
    void *nans;                          // lists of NaN values (attn_tc.cu)
    uint32_t *hdr;
};

// The positions that a row of a request with n new of kv tokens sees: [lo, hi).
__device__ __forceinline__ void row_range(const AttnProblem &p, int group, int kv, int n, int row, int &lo, int &hi) {
    const int pos = kv - n + row / group;
    lo = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
    hi = p.causal ? max(0, min(kv, pos + 1)) : kv;
    if (lo > hi)
        lo = hi;
}

// ------------------------------------------------------------------- plan

template <typename T>
__device__ __forceinline__ T block_scan(T v, T *red, T *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T a = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d)
            v += a;
    }
    __syncthreads();
    if (lane == 31)
        red[warp] = v;
    __syncthreads();
    T sum = 0, total_sum = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < warp)
            sum += red[w];
        total_sum += red[w];
    }
    *total = total_sum;
    return v + sum;
}

__device__ __forceinline__ RowTile row_tile(const AttnArgs &a, int request, int q0, int n, int kv, int row0) {
    RowTile r{};
    r.request = request;
    r.q0 = q0;
    r.n = n;
    r.kv = kv;
    r.row0 = row0;
    const int last = min(row0 + a.rows, n * a.group) - 1;
    int l0, h0, l1, h1;
    row_range(a.p, a.group, kv, n, row0, l0, h0);
    row_range(a.p, a.group, kv, n, last, l1, h1);
    // the first row sees furthest back, the last one furthest on
    r.tile0 = l0 / kTile;
    r.tiles = h1 > l0 ? (h1 + kTile - 1) / kTile - r.tile0 : 0;
    return r;
}

__device__ __forceinline__ Plan plan_of(const AttnArgs &a, long long work, int row_tiles) {
    const long long most = (work + kMinCost - 1) / kMinCost;
    const int used = (int)min((long long)a.ctas, most);
    return Plan{work, used > 0 ? (work + used - 1) / used : 1, row_tiles, used};
}

// The plan of no more requests than threads: a thread lists its request's row tiles.  red: 2 x 32 words of shared memory.
__device__ __forceinline__ void make_small_plan(const AttnArgs &a, long long *red, RowTile *recs, Plan *plan, bool report) {
    const AttnProblem &p = a.p;
    const int tid = threadIdx.x;
    int lo = 0, n = 0, kv = 0, bad = 0;
    if (tid < p.B) {
        const int hi = p.q_offsets[tid + 1];
        lo = p.q_offsets[tid];
        kv = p.kv_lens[tid];
        n = hi - lo;
        bad = lo < 0 || hi < lo || hi > p.T || kv < 0 || kv > ((long long)p.max_blocks << a.shift);
    }
    bad = __syncthreads_or(bad);
    const int count = bad ? 0 : (int)(((long long)n * a.group + a.rows - 1) / a.rows);     // at most a.max_tiles in all
    long long cost = 0, total;
    for (int i = 0; i < count; ++i)
        cost += (long long)(row_tile(a, tid, lo, n, kv, i * a.rows).tiles + kUnitCost) * p.cache.kv_heads;
    // row tiles in the upper bits, work (below 2^48) in the lower
    const long long mine = ((long long)count << 48) + cost, incl = block_scan(mine, red, &total);
    const int tiles = (int)(total >> 48), first = (int)((incl - mine) >> 48);
    const bool fits = tiles <= a.max_tiles;
    if (fits) {
        long long before = (incl - mine) & ((1ll << 48) - 1);
        for (int i = 0; i < count; ++i) {
            RowTile r = row_tile(a, tid, lo, n, kv, i * a.rows);
            r.before = before;
            before += (long long)(r.tiles + kUnitCost) * p.cache.kv_heads;
            recs[first + i] = r;
        }
    }
    if (tid == 0) {
        if ((bad || !fits) && report)
            record_status(a.hdr, MOE_ERR_DEVICE_ASSERT);
        *plan = bad || !fits ? Plan{0, 1, 0, 0} : plan_of(a, total & ((1ll << 48) - 1), tiles);
    }
    __syncthreads();
}

// The plan, by all threads of a CTA.  first: B ints, red: 32 words of shared
// memory; recs in shared or global memory.
__device__ __forceinline__ void make_plan(const AttnArgs &a, int *first, long long *red, RowTile *recs, Plan *plan, bool report) {
    const AttnProblem &p = a.p;
    const int tid = threadIdx.x, nt = blockDim.x;
    const long long cap = (long long)p.max_blocks << a.shift;
    int bad = 0;
    long long carry = 0, total;
    for (int b0 = 0; b0 < p.B; b0 += nt) {
        const int b = b0 + tid;
        long long c = 0;
        if (b < p.B) {
            const int lo = p.q_offsets[b], hi = p.q_offsets[b + 1], kv = p.kv_lens[b];
            if (lo < 0 || hi < lo || hi > p.T || kv < 0 || kv > cap)
                bad = 1;
            else
                c = ((long long)(hi - lo) * a.group + a.rows - 1) / a.rows;
        }
        const long long incl = block_scan(c, red, &total);
        if (b < p.B)
            first[b] = (int)min(carry + incl - c, (long long)a.max_tiles);
        carry += total;
    }
    if (__syncthreads_or(bad) || carry > a.max_tiles) {
        if (tid == 0) {
            if (report)
                record_status(a.hdr, MOE_ERR_DEVICE_ASSERT);
            *plan = Plan{0, 1, 0, 0};
        }
        __syncthreads();
        return;
    }
    const int n_recs = (int)carry;
    carry = 0;
    for (int i0 = 0; i0 < n_recs; i0 += nt) {
        const int i = i0 + tid;
        RowTile r{};
        long long c = 0;
        if (i < n_recs) {
            int lo = 0, hi = p.B;               // the last request with first <= i
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= i)
                    lo = mid;
                else
                    hi = mid;
            }
            const int q0 = p.q_offsets[lo];
            r = row_tile(a, lo, q0, p.q_offsets[lo + 1] - q0, p.kv_lens[lo], (i - first[lo]) * a.rows);
            c = (long long)(r.tiles + kUnitCost) * p.cache.kv_heads;
        }
        const long long incl = block_scan(c, red, &total);
        r.before = carry + incl - c;
        if (i < n_recs)
            recs[i] = r;
        carry += total;
    }
    if (tid == 0)
        *plan = plan_of(a, carry, n_recs);
    __syncthreads();
}

// Wait for a phase; false after kWaitLimitNs.
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity))
        return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > kWaitLimitNs)
            return false;
    return true;
}

// References of a softmax further from zero than this take the rounded form of their differences; half of its last place is 2^-4.
constexpr float kFar = 0x1p20f;

// A maximum as what is subtracted: 0 where nothing has been seen.
__device__ __forceinline__ float seen(float v) { return v == -INFINITY ? 0.0f : v; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One unit's piece, as producers and consumers walk through it.
struct Piece {
    int request, head, row0, rows, q0, n, kv;
    int tile0, t0, t1;            // cache tiles tile0 + [t0, t1)
    int first, last;              // CTAs of the unit's first and last tile
    int first_tiles, last_tiles;  // the unit's tiles in those
};

// Walks a CTA's range.
struct Walk {
    const AttnArgs &a;
    const RowTile *recs;
    long long pos, end, base, per;
    int rt, head, n_recs;
    RowTile r;
    __device__ Walk(const AttnArgs &args, const Plan &pl, const RowTile *tiles) : a(args), recs(tiles) {
        n_recs = pl.row_tiles;
        per = pl.per;
        pos = (long long)blockIdx.x * per;
        end = min(pos + per, pl.work);
        rt = n_recs;
        if ((int)blockIdx.x >= pl.ctas || pos >= pl.work)
            return;
        int lo = 0, hi = n_recs;                // the last row tile with before <= pos
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (recs[mid].before <= pos)
                lo = mid;
            else
                hi = mid;
        }
        rt = lo;
        r = recs[rt];
        head = pos - r.before < 0x7FFFFFFF ? (int)((uint32_t)(pos - r.before) / (uint32_t)(r.tiles + kUnitCost))
                                           : (int)((pos - r.before) / (r.tiles + kUnitCost));
        base = r.before + (long long)head * (r.tiles + kUnitCost);
    }
    // The next piece; false at the end of the range.
    __device__ bool next(Piece &pc) {
        while (rt < n_recs && base < end) {
            const int lo = (int)min(max(pos - base - kUnitCost, 0ll), (long long)r.tiles);
            const int hi = (int)max(min(end - base - kUnitCost, (long long)r.tiles), 0ll);
            const bool mine = r.tiles == 0 ? base >= pos : hi > lo;
            if (mine) {
                pc.request = r.request;
                pc.head = head;
                pc.row0 = r.row0;
                pc.q0 = r.q0;
                pc.n = r.n;
                pc.kv = r.kv;
                pc.rows = min(a.rows, r.n * a.group - r.row0);
                pc.tile0 = r.tile0;
                pc.t0 = lo;
                pc.t1 = hi;
                pc.first = pc.last = (int)blockIdx.x;
                pc.first_tiles = pc.last_tiles = r.tiles;
                const long long t0 = base + kUnitCost, t1 = t0 + r.tiles - 1;
                if (r.tiles > 0 && (t0 < pos || t1 >= end)) {      // cut
                    if (t1 < 0x7FFFFFFF) {                         // the usual sizes: 32-bit divisions
                        pc.first = (int)((uint32_t)t0 / (uint32_t)per);
                        pc.last = (int)((uint32_t)t1 / (uint32_t)per);
                    } else {
                        pc.first = (int)(t0 / per);
                        pc.last = (int)(t1 / per);
                    }
                    pc.first_tiles = (int)min((pc.first + 1) * per - t0, (long long)r.tiles);
                    pc.last_tiles = (int)(t1 + 1 - pc.last * per);
                }
            }
            base += r.tiles + kUnitCost;
            if (++head == a.p.cache.kv_heads) {
                head = 0;
                if (++rt < n_recs)
                    r = recs[rt];
            }
            if (mine)
                return true;
        }
        return false;
    }
};

}  // namespace
}  // namespace moe
