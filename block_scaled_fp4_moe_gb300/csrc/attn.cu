// attn.cu -- attention of a step's new tokens over the paged E4M3 cache.
//
//   o_i = sum_j p_ij v_j / l_i,   p_ij = 2^(x_ij - m_i),   l_i = sum_j p_ij,
//   x_ij = softmax_scale * log2(e) * q_i.k_j,              m_i = max_j x_ij
//
// with k_j = 2^a c_j and v_j = 2^b d_j, c and d E4M3 codes and a, b the
// exponents of the block that holds j.
//
// Numbers.  A row of q is scaled by a power of two into f16's range (bf16's 8
// significant bits fit f16's 11) and a code is exact in f16, so the products
// q.c are exact and summed in fp32 by f16 MMAs; 2^a multiplies the sum.
// The weight of d_j is w_ij = 2^(x_ij + b_j - M_i), M_i = max_j (x_ij + b_j): the
// block's exponent is inside the power, so that the f16 rounding of w (2^-12
// of itself, or 2^-25 of the row's largest) is relative to what the row's
// largest contribution can be, however far the blocks' exponents lie apart.
// l is summed from the unrounded fp32 p with its own maximum m.
//
// Work.  A unit is (request, up to 64 rows, key/value head), a row being a
// (token, query head of the group) pair, so that a key is read once for the
// whole group.  A plan kernel lists the row tiles with the 128-token tiles of
// cache that each sees; the units' tiles, laid end to end, are cut into
// equal ranges, one for each CTA of a persistent grid (one per SM).  A range that
// cuts a unit writes its part (sum and log-sum) to the workspace, and the last of
// the unit's CTAs to arrive joins the parts in the order of the cache.
//
// CTA: a producer warp streams tiles (16-token sub-blocks, 16 * D consecutive
// bytes of a block, by bulk copies) into a ring of shared-memory stages;
// eight consumer warps take 16 rows each and share a tile's sub-blocks among
// the warps of the same rows: 1 x 8, 2 x 4 or 4 x 2 (row groups x token groups),
// whichever the unit's rows need.  A sub-block's 8 x 16 byte
// operand tiles come by ldmatrix (32 bits = 4 codes of a thread's row) and
// are converted in registers: 16 dims of 8 keys are the B operand of one
// MMA.  Thread (g, c) of a warp holds codes 4c .. 4c+3, as K positions 2c, 2c+1,
// 2c+8, 2c+9: q's dims (and, for the values, the weights' tokens) are taken in
// that order.
#include "attn.h"

namespace moe {
namespace {

constexpr int kTile = 128;             // tokens of a tile
constexpr int kSubs = kTile / 16;      // sub-blocks of a tile
constexpr int kRows = 64;              // rows of a unit
constexpr int kConsumers = 8;          // consumer warps
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kUnitCost = 2;           // a unit's fixed work, in tiles
constexpr int kMinCost = 4;            // least range of a CTA, in tiles
constexpr int kPlanThreads = 1024;
constexpr unsigned long long kWaitLimitNs = 200ull * 1000 * 1000;

// A row tile of a request.
struct RowTile {
    long long before;      // work of the row tiles before it (all heads), in tiles
    int request, q0, n, kv;   // its first row of q, new tokens, tokens
    int row0;                 // first row (of new tokens x group)
    int tile0, tiles;         // cache tiles it sees
};

struct Plan {
    long long work;        // of all units
    long long per;         // of a CTA
    int row_tiles, ctas;
};

// Where a CTA begins.
struct Start {
    long long pos;
    int row_tile, head;
};

struct AttnArgs {
    AttnProblem p;
    int group, shift;                    // query heads of a key/value head; log2(block_size)
    float scale_log2;
    const Plan *plan;
    const Start *starts;
    const RowTile *recs;
    uint32_t *tickets;
    float *part, *part_lse;
    uint32_t *hdr;
};

// The positions that the rows row0 .. row0 + rows - 1 of a request with n new
// of kv tokens see: [lo, hi).
__device__ __forceinline__ void row_range(const AttnProblem &p, int group, int kv, int n, int row, int &lo, int &hi) {
    const int pos = kv - n + row / group;
    lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
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
    if (warp == 0) {
        T w = lane < nw ? red[lane] : (T)0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const T a = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d)
                w += a;
        }
        red[lane] = w;
    }
    __syncthreads();
    *total = red[nw - 1];
    return warp > 0 ? v + red[warp - 1] : v;
}

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(AttnArgs a, Plan *plan, Start *starts, RowTile *recs,
                                                                 int ctas, int max_recs) {
    extern __shared__ int s_first[];            // first row tile of a request
    __shared__ long long red[32];
    pdl_wait();
    pdl_trigger();
    const AttnProblem &p = a.p;
    const int tid = threadIdx.x;
    for (int i = tid; i < ctas; i += kPlanThreads)
        a.tickets[i] = 0;
    const long long cap = (long long)p.max_blocks << a.shift;
    int bad = 0;
    long long carry = 0, total;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        long long c = 0;
        if (b < p.B) {
            const int lo = p.q_offsets[b], hi = p.q_offsets[b + 1], kv = p.kv_lens[b];
            if (lo < 0 || hi < lo || hi > p.T || kv < 0 || kv > cap)
                bad = 1;
            else
                c = ((long long)(hi - lo) * a.group + kRows - 1) / kRows;
        }
        const long long incl = block_scan(c, red, &total);
        if (b < p.B)
            s_first[b] = (int)min(carry + incl - c, (long long)max_recs);
        carry += total;
    }
    if (__syncthreads_or(bad) || carry > max_recs) {
        if (tid == 0) {
            record_status(a.hdr, MOE_ERR_DEVICE_ASSERT);
            plan->work = 0;
            plan->per = 1;
            plan->row_tiles = 0;
            plan->ctas = 0;
        }
        return;
    }
    const int n_recs = (int)carry;
    carry = 0;
    for (int i0 = 0; i0 < n_recs; i0 += kPlanThreads) {
        const int i = i0 + tid;
        RowTile r{};
        long long c = 0;
        if (i < n_recs) {
            int lo = 0, hi = p.B;               // the last request with s_first <= i
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_first[mid] <= i)
                    lo = mid;
                else
                    hi = mid;
            }
            const int q0 = p.q_offsets[lo], n = p.q_offsets[lo + 1] - q0, kv = p.kv_lens[lo];
            r.request = lo;
            r.q0 = q0;
            r.n = n;
            r.kv = kv;
            r.row0 = (i - s_first[lo]) * kRows;
            const int last = min(r.row0 + kRows, n * a.group) - 1;
            int l0, h0, l1, h1;
            row_range(p, a.group, kv, n, r.row0, l0, h0);
            row_range(p, a.group, kv, n, last, l1, h1);
            // the first row sees furthest back, the last one furthest on
            r.tile0 = l0 / kTile;
            r.tiles = h1 > l0 ? (h1 + kTile - 1) / kTile - r.tile0 : 0;
            c = (long long)(r.tiles + kUnitCost) * p.cache.kv_heads;
        }
        const long long incl = block_scan(c, red, &total);
        r.before = carry + incl - c;
        if (i < n_recs)
            recs[i] = r;
        carry += total;
    }
    __syncthreads();
    const long long most = (carry + kMinCost - 1) / kMinCost;
    const int used = (int)min((long long)ctas, most);
    const long long per = used > 0 ? (carry + used - 1) / used : 1;
    for (int i = tid; i < used; i += kPlanThreads) {
        const long long pos = i * per;
        Start s{pos, n_recs, 0};
        if (pos < carry) {
            int lo = 0, hi = n_recs;            // the last row tile with before <= pos
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (recs[mid].before <= pos)
                    lo = mid;
                else
                    hi = mid;
            }
            s.row_tile = lo;
            s.head = (int)((pos - recs[lo].before) / (recs[lo].tiles + kUnitCost));
        }
        starts[i] = s;
    }
    if (tid == 0) {
        plan->work = carry;
        plan->per = per;
        plan->row_tiles = n_recs;
        plan->ctas = used;
    }
}

// -------------------------------------------------------------- attention

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

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// 4 codes -> the two B registers of an f16 MMA.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &b0, uint32_t &b1) {
    b0 = e4m3x2_to_f16x2((uint16_t)w);
    b1 = e4m3x2_to_f16x2((uint16_t)(w >> 16));
}

template <int D>
struct Smem {
    static constexpr int kSubBytes = 16 * D;
    static constexpr int kTileBytes = kTile * D;
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kPad = D + 8;                                   // floats of a row of the join buffer
    static constexpr size_t kJoin = (size_t)kStages * kStageBytes;       // [token group][row][D] sums
    static constexpr size_t kStats = kJoin + (size_t)128 * kPad * 4;     // [token group][row] m, M, l
    static constexpr size_t kExps = kStats + 3 * 128 * 4;                // [stage][2][kSubs]
    static constexpr size_t kBars = kExps + (size_t)kStages * 2 * kSubs * 4;
    static constexpr size_t kBytes = kBars + 2 * kStages * 8 + 16;
};

// One unit's piece, as producer and consumers walk through it.
struct Piece {
    int request, head, row0, rows, q0, n, kv;
    int tile0, t0, t1;            // cache tiles tile0 + [t0, t1)
    int first, last;              // CTAs of the unit's first and last tile
};

// Walks a CTA's range.
struct Walk {
    const AttnArgs &a;
    long long pos, end, base, per;
    int rt, head, n_recs;
    RowTile r;
    __device__ Walk(const AttnArgs &args) : a(args) {
        const Plan pl = *a.plan;
        n_recs = pl.row_tiles;
        per = pl.per;
        if ((int)blockIdx.x >= pl.ctas) {
            rt = n_recs;
            return;
        }
        const Start s = a.starts[blockIdx.x];
        pos = s.pos;
        end = min(pos + per, pl.work);
        rt = s.row_tile;
        head = s.head;
        if (rt < n_recs) {
            r = a.recs[rt];
            base = r.before + (long long)head * (r.tiles + kUnitCost);
        }
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
                pc.rows = min(kRows, r.n * a.group - r.row0);
                pc.tile0 = r.tile0;
                pc.t0 = lo;
                pc.t1 = hi;
                pc.first = pc.last = (int)blockIdx.x;
                if (r.tiles > 0) {
                    pc.first = (int)((base + kUnitCost) / per);
                    pc.last = (int)((base + kUnitCost + r.tiles - 1) / per);
                }
            }
            base += r.tiles + kUnitCost;
            if (++head == a.p.cache.kv_heads) {
                head = 0;
                if (++rt < n_recs)
                    r = a.recs[rt];
            }
            if (mine)
                return true;
        }
        return false;
    }
};

template <int D>
__device__ void produce(const AttnArgs &a, uint8_t *sm, uint64_t *full, uint64_t *empty) {
    using S = Smem<D>;
    const AttnProblem &p = a.p;
    const int lane = threadIdx.x & 31, sub = lane & (kSubs - 1);
    const bool is_v = lane >= kSubs;             // lanes 0..7: keys, 8..15: values
    const uint8_t *codes = is_v ? p.cache.v : p.cache.k, *scales = is_v ? p.cache.v_scale : p.cache.k_scale;
    const uint64_t policy = l2_evict_first_policy();
    Walk walk(a);
    Piece pc;
    long long it = 0;
    bool dead = false;
    while (walk.next(pc)) {
        const int hi = p.causal ? min(pc.kv, pc.kv - pc.n + (pc.row0 + pc.rows - 1) / a.group + 1) : pc.kv;
        const int32_t *row = p.table + (size_t)pc.request * p.max_blocks;
        for (int t = pc.t0; t < pc.t1; ++t, ++it) {
            const int st = (int)(it % S::kStages);
            const long long tok = (long long)(pc.tile0 + t) * kTile + sub * 16;
            const bool live = lane < 2 * kSubs && tok < hi;
            int page = 0, e = 0;
            if (live) {
                page = __ldg(row + (tok >> a.shift));
                if (page < 0 || page >= p.cache.num_blocks) {
                    record_status(a.hdr, MOE_ERR_DEVICE_ASSERT);
                    page = 0;
                }
            }
            const size_t unit = (size_t)page * p.cache.kv_heads + pc.head;
            if (live)
                e = (int)__ldg(scales + unit) - 127;
            if (!dead && it >= S::kStages)
                dead = !__all_sync(0xffffffffu, wait_phase(empty + st, (uint32_t)((it / S::kStages - 1) & 1)));
            if (dead) {
                if (lane == 0)
                    record_status(a.hdr, MOE_ERR_DEVICE_TIMEOUT);
                continue;                        // no further copies; the consumers' waits run out
            }
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, live)) * S::kSubBytes;
            uint8_t *dst = sm + (size_t)st * S::kStageBytes + (is_v ? S::kTileBytes : 0) + sub * S::kSubBytes;
            if (lane < 2 * kSubs)
                reinterpret_cast<float *>(sm + S::kExps)[st * 2 * kSubs + lane] = is_v ? (float)e : exp2i(min(max(e, -126), 127));
            __syncwarp();
            if (lane == 0)
                mbar_arrive_expect_tx(full + st, bytes);
            __syncwarp();
            if (live) {
                const uint8_t *src = codes + (unit << a.shift) * D + (size_t)(tok & ((1 << a.shift) - 1)) * D;
                asm volatile(
                    "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, "
                    "[%3], %4;" ::"r"(smem_u32(dst)), "l"(src), "r"(S::kSubBytes), "r"(smem_u32(full + st)), "l"(policy)
                    : "memory");
            }
        }
    }
    // copies still in flight must land before the CTA's shared memory goes away
    const long long from = it > S::kStages ? it - S::kStages : 0;
    for (long long i = from; i < it && !dead; ++i)
        wait_phase(full + i % S::kStages, (uint32_t)((i / S::kStages) & 1));
}

// The state of a warp: 16 rows, row g and row g + 8 of thread (g, c).
template <int D>
struct Acc {
    float o[D / 8][4];
    float m[2], big[2], l[2];       // m_i, M_i, l_i (l: this thread's columns)
};

// One piece's tiles with RG row groups x TG token groups.
template <int D, int RG>
__device__ __forceinline__ void attend(const AttnArgs &a, const Piece &pc, uint8_t *sm, uint64_t *full, uint64_t *empty,
                                       long long &it, bool &dead, Acc<D> &acc) {
    using S = Smem<D>;
    constexpr int TG = kConsumers / RG, NS = kSubs / TG;    // sub-blocks of a warp in a tile
    const AttnProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int rg = warp % RG, tg = warp / RG;
    // the rows: their query in operand order, scaled into f16, and their limits
    uint32_t q[D / 16][4];
    float f[2];
    int lo[2], hi[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int rr = rg * 16 + g + 8 * s;
        const bool live = rr < pc.rows;
        const int row = pc.row0 + (live ? rr : 0);
        const uint16_t *src = p.q + (int64_t)(pc.q0 + row / a.group) * p.q_st + (int64_t)(pc.head * a.group + row % a.group) * p.q_sh + 4 * c;
        uint2 raw[D / 16];
        float mx = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            raw[j] = live ? __ldg(reinterpret_cast<const uint2 *>(src + 16 * j)) : make_uint2(0, 0);
            mx = fmaxf(mx, fmaxf(fmaxf(fabsf(__uint_as_float(raw[j].x << 16)), fabsf(__uint_as_float(raw[j].x & 0xFFFF0000u))),
                                 fmaxf(fabsf(__uint_as_float(raw[j].y << 16)), fabsf(__uint_as_float(raw[j].y & 0xFFFF0000u)))));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int sh = f16_shift_for_max(mx);
        const float sc = exp2i(sh);
        f[s] = a.scale_log2 * exp2i(-sh);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            const __half2 u = __floats2half2_rn(__uint_as_float(raw[j].x << 16) * sc, __uint_as_float(raw[j].x & 0xFFFF0000u) * sc);
            const __half2 v = __floats2half2_rn(__uint_as_float(raw[j].y << 16) * sc, __uint_as_float(raw[j].y & 0xFFFF0000u) * sc);
            q[j][s] = *reinterpret_cast<const uint32_t *>(&u);
            q[j][2 + s] = *reinterpret_cast<const uint32_t *>(&v);
        }
        lo[s] = 0;
        hi[s] = pc.kv;
        if (live)
            row_range(p, a.group, pc.kv, pc.n, row, lo[s], hi[s]);
    }
    const int min_hi = __reduce_min_sync(0xffffffffu, min(hi[0], hi[1])), max_lo = __reduce_max_sync(0xffffffffu, max(lo[0], lo[1]));
    const bool idle = rg * 16 >= pc.rows;                    // no rows: only keeps the ring going
    const uint32_t base = smem_u32(sm);
    // ldmatrix rows: matrix lane / 8, row i = lane % 8.  Keys of the MMA's column i: token 4 (i / 2) + i % 2, plus 2 in the
    // second half; values: dim i.
    const int mi = lane >> 3, ri = lane & 7;
    const uint32_t k_off = (uint32_t)(mi * 256 + (4 * (ri >> 1) + (ri & 1)) * 16), v_off = (uint32_t)(lane * 16);

    for (int t = pc.t0; t < pc.t1; ++t, ++it) {
        const int st = (int)(it % S::kStages);
        if (!dead) {
            dead = !__all_sync(0xffffffffu, wait_phase(full + st, (uint32_t)((it / S::kStages) & 1)));
            if (dead && lane == 0)
                record_status(a.hdr, MOE_ERR_DEVICE_TIMEOUT);
        }
        const int tok0 = (pc.tile0 + t) * kTile;
        const uint32_t ks = base + (uint32_t)(st * S::kStageBytes), vs = ks + S::kTileBytes;
        const float *ex = reinterpret_cast<const float *>(sm + S::kExps) + st * 2 * kSubs;
        if (!idle) {
            const bool edge = tok0 + kTile > min_hi || tok0 < max_lo;
            float x[NS][2][4];
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int sub = i * TG + tg;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[i][h][e] = 0.0f;
#pragma unroll
                for (int j = 0; j < D / 16; j += 4)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t w[4];
                        ldmatrix4(w, ks + (uint32_t)(sub * S::kSubBytes + j * 256 + h * 32) + k_off);
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            uint32_t b0, b1;
                            codes_to_f16(w[u], b0, b1);
                            mma_m16n8k16_f16(x[i][h], q[j + u][0], q[j + u][1], q[j + u][2], q[j + u][3], b0, b1, x[i][h]);
                        }
                    }
                const float kf = ex[sub], f0 = f[0] * kf, f1 = f[1] * kf;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    x[i][h][0] *= f0;
                    x[i][h][1] *= f0;
                    x[i][h][2] *= f1;
                    x[i][h][3] *= f1;
                }
                if (edge) {
                    const int tk = tok0 + sub * 16 + 4 * c;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = tk + 2 * h + (e & 1);
                            if (j < lo[e >> 1] || j >= hi[e >> 1])
                                x[i][h][e] = -INFINITY;
                        }
                }
            }
            // maxima: m over x, M over x + b
            float nm[2] = {acc.m[0], acc.m[1]}, nb[2] = {acc.big[0], acc.big[1]};
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const float b = ex[kSubs + i * TG + tg];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const float v = fmaxf(fmaxf(x[i][0][2 * s], x[i][0][2 * s + 1]), fmaxf(x[i][1][2 * s], x[i][1][2 * s + 1]));
                    nm[s] = fmaxf(nm[s], v);
                    nb[s] = fmaxf(nb[s], v + b);
                }
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                nm[s] = fmaxf(nm[s], __shfl_xor_sync(0xffffffffu, nm[s], 1));
                nb[s] = fmaxf(nb[s], __shfl_xor_sync(0xffffffffu, nb[s], 1));
                nm[s] = fmaxf(nm[s], __shfl_xor_sync(0xffffffffu, nm[s], 2));
                nb[s] = fmaxf(nb[s], __shfl_xor_sync(0xffffffffu, nb[s], 2));
            }
            float mz[2], bz[2];                               // maxima to subtract (0 where nothing is seen yet)
            const bool grew = nb[0] > acc.big[0] || nb[1] > acc.big[1];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                mz[s] = nm[s] == -INFINITY ? 0.0f : nm[s];
                bz[s] = nb[s] == -INFINITY ? 0.0f : nb[s];
                acc.l[s] *= ex2(acc.m[s] - mz[s]);
                acc.m[s] = nm[s];
            }
            if (__any_sync(0xffffffffu, grew)) {
                const float r0 = ex2(acc.big[0] - bz[0]), r1 = ex2(acc.big[1] - bz[1]);
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    acc.o[n][0] *= r0;
                    acc.o[n][1] *= r0;
                    acc.o[n][2] *= r1;
                    acc.o[n][3] *= r1;
                }
            }
            acc.big[0] = nb[0];
            acc.big[1] = nb[1];
            uint32_t nan_seen = 0;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int sub = i * TG + tg;
                const float b = ex[kSubs + sub], d0 = b - bz[0], d1 = b - bz[1];
                uint32_t w[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    acc.l[0] += ex2(x[i][h][0] - mz[0]) + ex2(x[i][h][1] - mz[0]);
                    acc.l[1] += ex2(x[i][h][2] - mz[1]) + ex2(x[i][h][3] - mz[1]);
                    const __half2 u = __floats2half2_rn(ex2(x[i][h][0] + d0), ex2(x[i][h][1] + d0));
                    const __half2 v = __floats2half2_rn(ex2(x[i][h][2] + d1), ex2(x[i][h][3] + d1));
                    w[2 * h] = *reinterpret_cast<const uint32_t *>(&u);
                    w[2 * h + 1] = *reinterpret_cast<const uint32_t *>(&v);
                }
#pragma unroll
                for (int n = 0; n < D / 8; n += 4) {
                    uint32_t vc[4];
                    ldmatrix4(vc, vs + (uint32_t)(sub * S::kSubBytes + n * 128) + v_off);
                    if (edge) {
                        // some row does not see some token here: NaN codes (of unused slots, or of tokens past a
                        // row) must not meet its zero weight.  They are left out, and added below to the rows that see them.
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const uint32_t nan = __vcmpeq4(vc[u] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                            vc[u] &= ~nan;
                            nan_seen |= nan;
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t b0, b1;
                        codes_to_f16(vc[u], b0, b1);
                        mma_m16n8k16_f16(acc.o[n + u], w[0], w[1], w[2], w[3], b0, b1, acc.o[n + u]);
                    }
                }
            }
            if (edge && __any_sync(0xffffffffu, nan_seen != 0)) {
                const uint8_t *vb = sm + (size_t)st * S::kStageBytes + S::kTileBytes;
#pragma unroll 1
                for (int i = 0; i < NS; ++i) {
                    const int sub = i * TG + tg;
#pragma unroll 1
                    for (int k = 0; k < 16; ++k) {
                        const int j = tok0 + sub * 16 + k;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int d = 8 * n + 2 * c + (e & 1);
                                if ((vb[sub * S::kSubBytes + d * 16 + k] & 0x7F) == 0x7F && j >= lo[e >> 1] && j < hi[e >> 1])
                                    acc.o[n][e] = __uint_as_float(0x7FFFFFFFu);
                            }
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(empty + st);
    }
}

__device__ __forceinline__ void store_bf16x4(uint16_t *dst, float4 v) {
    uint32_t a, b;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(a) : "f"(v.y), "f"(v.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(v.w), "f"(v.z));
    *reinterpret_cast<uint2 *>(dst) = make_uint2(a, b);
}

// Joins the token groups of a piece and writes the rows: to the output, or,
// where the unit has other pieces, to the workspace, the last CTA joining those.
template <int D, int RG>
__device__ __forceinline__ void finish(const AttnArgs &a, const Piece &pc, uint8_t *sm, Acc<D> &acc, int *s_last) {
    using S = Smem<D>;
    constexpr int TG = kConsumers / RG, R = RG * 16;
    const AttnProblem &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int rg = warp % RG, tg = warp / RG;
    float *sum = reinterpret_cast<float *>(sm + S::kJoin), *st = reinterpret_cast<float *>(sm + S::kStats);
    float *s_m = st, *s_b = st + 128, *s_l = st + 256;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        acc.l[s] += __shfl_xor_sync(0xffffffffu, acc.l[s], 1);
        acc.l[s] += __shfl_xor_sync(0xffffffffu, acc.l[s], 2);
        if (c == 0) {
            const int i = tg * R + rg * 16 + g + 8 * s;
            s_m[i] = acc.m[s];
            s_b[i] = acc.big[s];
            s_l[i] = acc.l[s];
        }
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
        float *dst = sum + (size_t)(tg * R + rg * 16 + g) * S::kPad + 8 * n + 2 * c;
        *reinterpret_cast<float2 *>(dst) = make_float2(acc.o[n][0], acc.o[n][1]);
        *reinterpret_cast<float2 *>(dst + 8 * S::kPad) = make_float2(acc.o[n][2], acc.o[n][3]);
    }
    named_barrier_sync(1, kConsumers * 32);
    const int pieces = pc.last - pc.first + 1;
    const int slot = (int)blockIdx.x * 2 + (pc.first == (int)blockIdx.x);
    constexpr int Q = D / 4;
    for (int i = tid; i < pc.rows * Q; i += kConsumers * 32) {
        const int row = i / Q, d = i % Q * 4;
        float m = -INFINITY, b = -INFINITY;
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            m = fmaxf(m, s_m[t * R + row]);
            b = fmaxf(b, s_b[t * R + row]);
        }
        const float mz = m == -INFINITY ? 0.0f : m, bz = b == -INFINITY ? 0.0f : b;
        float l = 0.0f;
        float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            l += s_l[t * R + row] * ex2(s_m[t * R + row] - mz);
            const float w = ex2(s_b[t * R + row] - bz);
            const float4 v = *reinterpret_cast<const float4 *>(sum + (size_t)(t * R + row) * S::kPad + d);
            o.x += v.x * w;
            o.y += v.y * w;
            o.z += v.z * w;
            o.w += v.w * w;
        }
        // l is NaN where a score was: then so is the row
        const float f = l == 0.0f ? 0.0f : exp2f(bz - mz) / l;
        o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
        const float lse2 = l == 0.0f ? -INFINITY : mz + log2f(l);
        if (pieces == 1) {
            const int r = pc.row0 + row;
            const size_t at = (size_t)(pc.q0 + r / a.group) * p.q_heads + pc.head * a.group + r % a.group;
            store_bf16x4(p.out + at * D + d, o);
            if (d == 0 && p.lse)
                p.lse[at] = lse2 * 0.69314718055994530942f;
        } else {
            __stcg(reinterpret_cast<float4 *>(a.part + ((size_t)slot * kRows + row) * D + d), o);
            if (d == 0)
                __stcg(a.part_lse + slot * kRows + row, lse2);
        }
    }
    if (pieces > 1) {
        __threadfence();
        named_barrier_sync(1, kConsumers * 32);
        if (tid == 0) {
            __threadfence();
            *s_last = atomicAdd(a.tickets + pc.first, 1u) == (uint32_t)(pieces - 1);
            __threadfence();
        }
        named_barrier_sync(1, kConsumers * 32);
        if (*s_last) {
            for (int i = tid; i < pc.rows * Q; i += kConsumers * 32) {
                const int row = i / Q, d = i % Q * 4;
                auto at = [&](int k) { return (size_t)(pc.first + k) * 2 + (k == 0); };
                float m = -INFINITY;
                for (int k = 0; k < pieces; ++k)
                    m = fmaxf(m, __ldcg(a.part_lse + at(k) * kRows + row));
                const float mz = m == -INFINITY ? 0.0f : m;
                float l = 0.0f;
                float4 o = make_float4(0, 0, 0, 0);
#pragma unroll 4
                for (int k = 0; k < pieces; ++k) {
                    const float w = ex2(__ldcg(a.part_lse + at(k) * kRows + row) - mz);
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(a.part + (at(k) * kRows + row) * D + d));
                    l += w;
                    o.x += v.x * w;
                    o.y += v.y * w;
                    o.z += v.z * w;
                    o.w += v.w * w;
                }
                const float f = l == 0.0f ? 0.0f : 1.0f / l;
                const int r = pc.row0 + row;
                const size_t to = (size_t)(pc.q0 + r / a.group) * p.q_heads + pc.head * a.group + r % a.group;
                store_bf16x4(p.out + to * D + d, make_float4(o.x * f, o.y * f, o.z * f, o.w * f));
                if (d == 0 && p.lse)
                    p.lse[to] = l == 0.0f ? -INFINITY : (mz + log2f(l)) * 0.69314718055994530942f;
            }
        }
    }
    named_barrier_sync(1, kConsumers * 32);       // the join buffer is free again
}

template <int D, int RG>
__device__ __forceinline__ void consume_piece(const AttnArgs &a, const Piece &pc, uint8_t *sm, uint64_t *full,
                                              uint64_t *empty, long long &it, bool &dead, int *s_last) {
    Acc<D> acc;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc.o[n][e] = 0.0f;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        acc.m[s] = acc.big[s] = -INFINITY;
        acc.l[s] = 0.0f;
    }
    attend<D, RG>(a, pc, sm, full, empty, it, dead, acc);
    finish<D, RG>(a, pc, sm, acc, s_last);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ AttnArgs a) {
    using S = Smem<D>;
    extern __shared__ __align__(128) uint8_t sm[];
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + S::kBars), *empty = full + S::kStages;
    int *s_last = reinterpret_cast<int *>(empty + S::kStages);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, kConsumers);
        }
        fence_barrier_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x >= kConsumers * 32) {
        produce<D>(a, sm, full, empty);
        return;
    }
    Walk walk(a);
    Piece pc;
    long long it = 0;
    bool dead = false;
    while (walk.next(pc)) {
        if (pc.rows <= 16)
            consume_piece<D, 1>(a, pc, sm, full, empty, it, dead, s_last);
        else if (pc.rows <= 32)
            consume_piece<D, 2>(a, pc, sm, full, empty, it, dead, s_last);
        else
            consume_piece<D, 4>(a, pc, sm, full, empty, it, dead, s_last);
    }
}

constexpr int kMaxCtas = 256;

}  // namespace

AttnLayout AttnLayout::make(int T, int B, int q_heads, int kv_heads, int head_dim) {
    AttnLayout L{};
    const long long group = q_heads / kv_heads;
    const size_t recs = (size_t)((long long)T * group / kRows + B);
    size_t o = kHeaderBytes;
    auto take = [&](size_t bytes) { o = align_up(o, 256); size_t r = o; o += bytes; return r; };
    L.plan = take(sizeof(Plan));
    L.starts = take(kMaxCtas * sizeof(Start));
    L.tickets = take(kMaxCtas * sizeof(uint32_t));
    L.recs = take(recs * sizeof(RowTile));
    L.part = take((size_t)2 * kMaxCtas * kRows * head_dim * sizeof(float));
    L.part_lse = take((size_t)2 * kMaxCtas * kRows * sizeof(float));
    L.total = align_up(o, 256);
    return L;
}

cudaError_t launch_kv_attention(const AttnProblem &p, void *ws, int sms, cudaStream_t stream) {
    const AttnLayout L = AttnLayout::make(p.T, p.B, p.q_heads, p.cache.kv_heads, p.cache.head_dim);
    const int group = p.q_heads / p.cache.kv_heads;
    const int max_recs = (int)((long long)p.T * group / kRows + p.B);
    int shift = 4;
    while ((1 << shift) < p.cache.block_size)
        ++shift;
    AttnArgs a{p, group, shift, p.scale * 1.44269504088896340736f, ws_at<Plan>(ws, L.plan), ws_at<Start>(ws, L.starts),
               ws_at<RowTile>(ws, L.recs), ws_at<uint32_t>(ws, L.tickets), ws_at<float>(ws, L.part),
               ws_at<float>(ws, L.part_lse), ws_at<uint32_t>(ws, 0)};
    const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
    cudaError_t e = launch_pdl(attn_plan_kernel, dim3(1), dim3(kPlanThreads), p.B * sizeof(int), stream, a,
                               ws_at<Plan>(ws, L.plan), ws_at<Start>(ws, L.starts), ws_at<RowTile>(ws, L.recs), ctas, max_recs);
    if (e != cudaSuccess)
        return e;
    auto go = [&](auto kernel, size_t smem) {
        cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        return r != cudaSuccess ? r : launch_pdl(kernel, dim3(ctas), dim3(kThreads), smem, stream, a);
    };
    return p.cache.head_dim == 64 ? go(attn_kernel<64>, Smem<64>::kBytes) : go(attn_kernel<128>, Smem<128>::kBytes);
}

}  // namespace moe
