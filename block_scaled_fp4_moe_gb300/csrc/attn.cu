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
// The weight of d_j is w_ij = 2^(x_ij + b_j - M_i + 15), M_i = max_j (x_ij + b_j): the
// block's exponent is inside the power, so that the f16 rounding of w (2^-12
// of itself, or 2^-40 of the row's largest) is relative to what the row's
// largest contribution can be.  The largest weight is 2^15, f16's last whole binade: a block whose exponent lies far
// above the others' leaves them their bits, in the dims where it has nothing itself, down to 29 binades below it (with a largest
// weight of 1, 14: those dims were off by 5e-3 at 16 binades and 0.67 at 24).
// l is summed from the unrounded fp32 p with its own maximum m.
// The power of p is one FMA, x's product exact; m, rounded, may lie under it by half of its last place.  Where a warp's maxima pass
// kFar (half a place of 2^28 is a factor of 2^16) a loop of its own takes over, in which the products are rounded first, as m was, so that
// no power is above zero, and M is kept as M - m, which has all its bits however large the scores are.
//
// Work.  A unit is (request, up to 64 rows, key/value head), a row being a
// (token, query head of the group) pair, so that a key is read once for the
// whole group.  A plan lists the row tiles with the 128-token tiles of
// cache that each sees; the units' tiles, laid end to end, are cut into
// equal ranges, one for each CTA of a persistent grid (one per SM).  A range that
// cuts a unit writes its part (sum and log-sum) to the workspace, and the last of
// the unit's CTAs to arrive joins the parts in the order of the cache.  Few
// row tiles (a decode step): every CTA makes the plan itself in shared memory; many:
// a kernel before this one makes it in the workspace.
//
// CTA: eight consumer warps, one warp that streams the keys, one that streams the values (a warp issues a
// copy in about 100 cycles, and blocks of 16 tokens need 8 of each for a tile) and two that prepare the queries of the next unit.  The cache comes in tiles (16-token
// sub-blocks, 16 * D consecutive bytes of a block, as bulk copies of all
// that lies together) through a ring of shared-memory stages; block ids and scales are
// loaded two batches of four tiles ahead.  A consumer warp takes 16 rows (units
// of up to 16) or 32, and the warps of the same rows share a tile's sub-blocks.
// A sub-block's 8 x 16 byte operand tiles come by ldmatrix (32 bits = 4 codes
// of a thread's row) and are converted in registers: 16 dims of 8 keys are the
// B operand of one MMA, or of two with 32 rows.  Thread (g, c) of a warp holds codes
// 4c .. 4c+3, as K positions 2c, 2c+1, 2c+8, 2c+9: q's dims (and, for the
// values, the weights' tokens) are taken in that order.
//
// Measured, key/value heads of 128: 64 requests of 31,000 tokens, 8 heads with 8 query heads each, 592 us (6.67 TB/s of the 6.78 of a copy: bound by
// memory); 48 ragged requests of 5,000 in blocks of 16, 102 us (5.2 TB/s: a request's first tiles and last join are a larger part);
// one of 1,000, 9.8 us (launch, plan, block ids, tiles, join: latency).  24 rows a request run at 3.6 TB/s and 32
// at 3.5, bound by the chain of products and powers in eight warps.
#include "attn_plan.cuh"

namespace moe {
namespace {

constexpr int kRows = 64;              // rows of a unit
constexpr int kConsumers = 8;          // consumer warps
constexpr int kThreads = 384;          // three warpgroups: two of consumers, one of producers
constexpr int kQWarps = 2;
constexpr int kSmallRequests = 256;    // most requests and row tiles of a plan in shared memory
constexpr int kSmallTiles = 288;
constexpr float kLift = 15.0f;         // the largest weight's power

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(AttnArgs a) {
    extern __shared__ int s_first[];
    __shared__ long long red[32];
    pdl_wait();
    pdl_trigger();
    make_plan(a, s_first, red, a.recs, a.plan, true);
}

// -------------------------------------------------------------- attention

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

// What the consumers need of a row.
struct RowInfo {
    float f;               // factor of its products
    int lo, hi;            // positions it sees
};

template <int D>
struct Smem {
    static constexpr int kSubBytes = 16 * D;
    static constexpr int kTileBytes = kTile * D;
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kQBytes = kRows * D * 2;                        // queries in operand order: [16 rows][16 dims][lane][16 bytes]
    static constexpr size_t kQ = (size_t)kStages * kStageBytes;          // two units'
    static constexpr size_t kInfo = kQ + 2 * kQBytes;                    // RowInfo [2][kRows]
    static constexpr size_t kPieces = kInfo + 2 * kRows * sizeof(RowInfo);      // Piece [2]
    static constexpr int kPad = D + 8;                                   // floats of a row of the join buffer
    static constexpr size_t kJoin = kPieces + 128;                       // [8 warps][8 rows][kPad]
    static constexpr size_t kStats = kJoin + (size_t)kConsumers * 8 * kPad * 4; // m, M, l [256]
    static constexpr size_t kExps = kStats + 3 * 256 * 4;                // [stage][2][kSubs]
    static constexpr size_t kRecs = kExps + (size_t)kStages * 2 * kSubs * 4;
    static constexpr size_t kBars = kRecs + kSmallTiles * sizeof(RowTile);
    static constexpr size_t kBytes = kBars + (2 * kStages + 4) * 8 + 16;
    static_assert(2 * sizeof(Piece) <= 128 && kInfo % 16 == 0 && kJoin % 16 == 0 && kRecs % 8 == 0 && kBars % 8 == 0 && kBytes <= 227 * 1024, "shared memory");
};

// A barrier that or's a predicate.
__device__ __forceinline__ bool barrier_any(int id, int threads, bool v) {
    uint32_t r;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.cta.red.or.pred q, %2, %3, p;\nselp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}

// Up to four tiles of a piece: a lane for each of their sub-blocks.
struct Batch {
    int tiles;                    // 0: there is none
    int head, page, scale;
    long long tok;                // the lane's first token
    bool live;
};

template <int D>
__device__ __forceinline__ void stream_cache(const AttnArgs &a, const Plan &pl, const RowTile *recs, uint8_t *sm, uint64_t *full,
                                             uint64_t *empty, bool is_v) {
    using S = Smem<D>;
    const AttnProblem &p = a.p;
    const int lane = threadIdx.x & 31, sub = lane & (kSubs - 1);
    const uint64_t policy = l2_evict_first_policy();
    const uint8_t *codes = is_v ? p.cache.v : p.cache.k, *scale = is_v ? p.cache.v_scale : p.cache.k_scale;
    Walk walk(a, pl, recs);
    Piece pc;
    int t = 0, lo = 0, hi = 0;                  // the piece's next tile; the positions that its rows see: from the first row's first
    bool more = true;
    auto next_piece = [&] {
        more = walk.next(pc);
        if (!more)
            return;
        t = pc.t0;
        row_range(p, a.group, pc.kv, pc.n, pc.row0, lo, hi);        // blocks before may be gone from the table
        hi = p.causal ? min(pc.kv, pc.kv - pc.n + (pc.row0 + pc.rows - 1) / a.group + 1) : pc.kv;
    };
    next_piece();
    // the next batch, its block ids asked for
    auto pages = [&](Batch &b) {
        b.tiles = 0;
        while (more && t == pc.t1)
            next_piece();
        if (!more)
            return;
        b.tiles = min(4, pc.t1 - t);
        b.head = pc.head;
        b.tok = (long long)(pc.tile0 + t) * kTile + lane * 16;
        b.live = lane < kSubs * b.tiles && b.tok < hi && b.tok + 16 > lo;
        b.page = b.live ? __ldg(p.table + (size_t)pc.request * p.max_blocks + (b.tok >> a.shift)) : 0;
        t += b.tiles;
    };
    auto scales = [&](Batch &b) {
        if (b.tiles == 0)
            return;
        if (b.page < 0 || b.page >= p.cache.num_blocks) {
            record_status(a.hdr, MOE_ERR_DEVICE_ASSERT);
            b.page = 0;
        }
        const size_t unit = (size_t)b.page * p.cache.kv_heads + b.head;
        b.scale = b.live ? __ldg(scale + unit) : 127;
    };
    long long it = 0;
    bool dead = false;
    Batch b0, b1, b2;
    pages(b0);
    pages(b1);
    scales(b0);
    while (b0.tiles > 0) {
        pages(b2);
        scales(b1);
        // sub-blocks of one block that lie in one tile are one copy, issued by the first one's lane
        const uint32_t live = __ballot_sync(0xffffffffu, b0.live);
        const int in_block = (int)(b0.tok & ((1 << a.shift) - 1)) >> 4, block_subs = 1 << (a.shift - 4);
        const uint32_t here = (live >> (lane & ~(kSubs - 1))) & ((1u << kSubs) - 1);         // one run of the tile's sub-blocks
        const int left = 32 - __clz(here) - sub;
        const bool leads = b0.live && (sub == __ffs(here) - 1 || in_block == 0);
        const uint32_t bytes = (uint32_t)min(block_subs - in_block, left) * S::kSubBytes;
        const size_t src = ((((size_t)b0.page * p.cache.kv_heads + b0.head) << a.shift) + in_block * 16) * D;
        for (int i = 0; i < b0.tiles; ++i, ++it) {
            const int st = (int)(it % S::kStages);
            if (!dead && it >= S::kStages)
                dead = !__all_sync(0xffffffffu, wait_phase(empty + st, (uint32_t)((it / S::kStages - 1) & 1)));
            if (dead) {
                if (lane == 0)
                    record_status(a.hdr, MOE_ERR_DEVICE_TIMEOUT);
                continue;                        // no further copies; the consumers' waits run out
            }
            const bool mine = lane / kSubs == i;
            if (mine) {
                float *ex = reinterpret_cast<float *>(sm + S::kExps) + st * 2 * kSubs + sub;
                if (is_v)
                    ex[kSubs] = (float)(b0.scale - 127);
                else
                    ex[0] = exp2i(min(max(b0.scale, 1), 254) - 127);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive_expect_tx(full + st, S::kSubBytes * __popc((live >> (i * kSubs)) & ((1u << kSubs) - 1)));
            __syncwarp();
            if (mine && leads) {
                const uint32_t dst = smem_u32(sm + (size_t)st * S::kStageBytes + (is_v ? S::kTileBytes : 0) + sub * S::kSubBytes);
                asm volatile(
                    "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, "
                    "[%3], %4;" ::"r"(dst), "l"(codes + src), "r"(bytes), "r"(smem_u32(full + st)), "l"(policy)
                    : "memory");
            }
        }
        b0 = b1;
        b1 = b2;
    }
    // copies still in flight must land before the CTA's shared memory goes away
    for (long long i = it > S::kStages ? it - S::kStages : 0; i < it && !dead; ++i)
        wait_phase(full + i % S::kStages, (uint32_t)((i / S::kStages) & 1));
}

// Queries of one unit after the other: bf16 to scaled f16 in the MMA's A operand order, 16 rows a warp.
template <int D>
__device__ __forceinline__ void load_queries(const AttnArgs &a, const Plan &pl, const RowTile *recs, uint8_t *sm, uint64_t *q_full,
                                             uint64_t *q_empty) {
    using S = Smem<D>;
    const AttnProblem &p = a.p;
    const int warp = (threadIdx.x >> 5) - kConsumers - 2, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    Walk walk(a, pl, recs);
    Piece pc;
    bool dead = false, more = true;
    for (int u = 0; more; ++u) {
        const int buf = u & 1;
        more = walk.next(pc);
        if (!more)
            pc.rows = 0;                        // there is no further piece
        if (!dead && u >= 2)
            dead = !__all_sync(0xffffffffu, wait_phase(q_empty + buf, (uint32_t)((u / 2 - 1) & 1)));
        if (warp == 0 && lane == 0)
            reinterpret_cast<Piece *>(sm + S::kPieces)[buf] = pc;
        RowInfo *info = reinterpret_cast<RowInfo *>(sm + S::kInfo) + buf * kRows;
        // rows up to the next multiple of 32, as the consumers read them
        for (int rg = warp; rg * 16 < (pc.rows <= 16 ? pc.rows : (pc.rows + 31) / 32 * 32); rg += kQWarps) {
            uint32_t *dst = reinterpret_cast<uint32_t *>(sm + S::kQ + (size_t)buf * S::kQBytes + (size_t)rg * 32 * D) + lane * 4;
#pragma unroll 1
            for (int s = 0; s < 2; ++s) {
                const int rr = rg * 16 + g + 8 * s;
                const bool live = rr < pc.rows;
                const int row = pc.row0 + (live ? rr : 0);
                const uint16_t *src =
                    p.q + (int64_t)(pc.q0 + row / a.group) * p.q_st + (int64_t)(pc.head * a.group + row % a.group) * p.q_sh + 4 * c;
                uint2 raw[D / 16];
                float mx = 0.0f;
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    raw[j] = live ? __ldg(reinterpret_cast<const uint2 *>(src + 16 * j)) : make_uint2(0, 0);
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    mx = fmaxf(mx, fmaxf(fmaxf(fabsf(__uint_as_float(raw[j].x << 16)), fabsf(__uint_as_float(raw[j].x & 0xFFFF0000u))),
                                         fmaxf(fabsf(__uint_as_float(raw[j].y << 16)), fabsf(__uint_as_float(raw[j].y & 0xFFFF0000u)))));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const int sh = f16_shift_for_max(mx);
                const float sc = exp2i(sh);
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    const __half2 lo = __floats2half2_rn(__uint_as_float(raw[j].x << 16) * sc, __uint_as_float(raw[j].x & 0xFFFF0000u) * sc);
                    const __half2 hi = __floats2half2_rn(__uint_as_float(raw[j].y << 16) * sc, __uint_as_float(raw[j].y & 0xFFFF0000u) * sc);
                    dst[j * 128 + s] = *reinterpret_cast<const uint32_t *>(&lo);
                    dst[j * 128 + 2 + s] = *reinterpret_cast<const uint32_t *>(&hi);
                }
                if (c == 0) {
                    RowInfo r{a.scale_log2 * exp2i(-sh), 0, pc.kv};
                    row_range(p, a.group, pc.kv, pc.n, row, r.lo, r.hi);
                    if (!live)                  // from the first row's first position, so that nothing unread is looked at for it
                        r.hi = pc.kv;
                    info[rr] = r;
                }
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(q_full + buf);
    }
}

// Rows g and g + 8 times r0 and r1.
template <int N>
__device__ __forceinline__ void scale_rows(float (&o)[N][4], float r0, float r1) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        o[n][0] *= r0;
        o[n][1] *= r0;
        o[n][2] *= r1;
        o[n][3] *= r1;
    }
}

// The state of a warp: MT x 16 rows, rows g and g + 8 of each for thread (g, c).
template <int D, int MT>
struct Acc {
    float o[MT][D / 8][4];
    float m[MT][2], big[MT][2], l[MT][2];       // m_i, M_i (far, and when all tiles are done, M_i - m_i), l_i (l: this thread's columns)
};

// One piece's tiles: RG groups of MT x 16 rows; the warps of a row group form SG sets that take tiles in turn, those of
// a set sharing a tile's sub-blocks.  (SG = 2 where all warps have the same rows: a warp's chain of products, maxima and powers
// is as long for 32 tokens as for 16.  One set: 64 requests of 31,000 tokens and 8 rows take 694 us for 600, 32 of 8,000 tokens
// and 24 rows 120 for 105.)
// Returns the tile after the last one: not FAR stops at the tile where some row's maximum passes kFar, with nothing of it done.
template <int D, int MT, int RG, int SG, bool FAR>
__device__ __forceinline__ int attend_tiles(const Piece &pc, uint8_t *sm, int qbuf, uint64_t *full, uint64_t *empty, uint32_t *hdr,
                                            long long it, int t, bool &dead, Acc<D, MT> &acc) {
    using S = Smem<D>;
    constexpr int TG = kConsumers / RG / SG, NS = kSubs / TG;    // warps of a set, sub-blocks of a warp in a tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int rg = warp % RG, tg = warp / RG % TG;
    const uint4 *q = reinterpret_cast<const uint4 *>(sm + S::kQ + (size_t)qbuf * S::kQBytes + (size_t)rg * MT * 32 * D) + lane;
    const RowInfo *info = reinterpret_cast<const RowInfo *>(sm + S::kInfo) + qbuf * kRows + rg * MT * 16 + g;
    float f[MT][2];
    int min_hi = INT_MAX, max_lo = 0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const RowInfo r = info[mt * 16 + 8 * s];
            f[mt][s] = r.f;
            min_hi = min(min_hi, r.hi);
            max_lo = max(max_lo, r.lo);
        }
    min_hi = __reduce_min_sync(0xffffffffu, min_hi);
    max_lo = __reduce_max_sync(0xffffffffu, max_lo);
    const uint32_t base = smem_u32(sm);
    // ldmatrix rows.  Keys: matrix = (half, chunk of 16 dims); the MMA's column i is token 4 (i / 2) + i % 2, plus 2 in the
    // second half.  Values: matrix = 8 dims, row = dim.
    const int mi = lane >> 3, ri = lane & 7;
    const uint32_t k_off = (uint32_t)((mi >> 1) * 256 + (4 * (ri >> 1) + (ri & 1) + 2 * (mi & 1)) * 16), v_off = (uint32_t)(lane * 16);

    for (; t < pc.t1; t += SG) {
        const uint32_t at = (uint32_t)(it + (t - pc.t0)), st = at % S::kStages;
        if (!dead) {
            dead = !__all_sync(0xffffffffu, wait_phase(full + st, (at / S::kStages) & 1));
            if (dead && lane == 0)
                record_status(hdr, MOE_ERR_DEVICE_TIMEOUT);
        }
        const int tok0 = (pc.tile0 + t) * kTile;
        const uint32_t ks = base + st * S::kStageBytes, vs = ks + S::kTileBytes;
        const float *ex = reinterpret_cast<const float *>(sm + S::kExps) + st * 2 * kSubs;
        const bool edge = tok0 + kTile > min_hi || tok0 < max_lo;
        float x[MT][NS][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < NS; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[mt][i][e >> 2][e & 3] = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 16; j += 2) {
            uint4 qa[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    qa[mt][u] = q[mt * 2 * D + (j + u) * 32];
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                uint32_t w[4];
                ldmatrix4(w, ks + (uint32_t)((i * TG + tg) * S::kSubBytes + j * 256) + k_off);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t b0, b1;
                        codes_to_f16(w[2 * u + h], b0, b1);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            mma_m16n8k16_f16(x[mt][i][h], qa[mt][u].x, qa[mt][u].y, qa[mt][u].z, qa[mt][u].w, b0, b1, x[mt][i][h]);
                    }
            }
        }
        // maxima: m over x, M over x + b (products times fi are x; fi > 0, so that -infinity stays)
        auto factor = [&](int mt, int s, int i) { return fmaxf(f[mt][s] * ex[i * TG + tg], 1.2e-38f); };
        auto hide = [&](int mt) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int lo = info[mt * 16 + 8 * s].lo, hi = info[mt * 16 + 8 * s].hi;
#pragma unroll
                for (int i = 0; i < NS; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int k = tok0 + (i * TG + tg) * 16 + 4 * c + 2 * h + e;
                            if (k < lo || k >= hi)
                                x[mt][i][h][2 * s + e] = -INFINITY;
                        }
            }
        };
        float mz[MT][2], up[MT][2];                           // m to subtract (0 where nothing is seen yet), m - M + 15
        if constexpr (!FAR) {
            float nm[MT][2], nb[MT][2];
            bool grew = false, far = false;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (edge)
                    hide(mt);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    nm[mt][s] = acc.m[mt][s];
                    nb[mt][s] = acc.big[mt][s];
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        const float v = factor(mt, s, i) * fmaxf(fmaxf(x[mt][i][0][2 * s], x[mt][i][0][2 * s + 1]),
                                                                 fmaxf(x[mt][i][1][2 * s], x[mt][i][1][2 * s + 1]));
                        nm[mt][s] = fmaxf(nm[mt][s], v);
                        nb[mt][s] = fmaxf(nb[mt][s], v + ex[kSubs + i * TG + tg]);
                    }
                }
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    nm[mt][s] = fmaxf(nm[mt][s], __shfl_xor_sync(0xffffffffu, nm[mt][s], 1));
                    nb[mt][s] = fmaxf(nb[mt][s], __shfl_xor_sync(0xffffffffu, nb[mt][s], 1));
                    nm[mt][s] = fmaxf(nm[mt][s], __shfl_xor_sync(0xffffffffu, nm[mt][s], 2));
                    nb[mt][s] = fmaxf(nb[mt][s], __shfl_xor_sync(0xffffffffu, nb[mt][s], 2));
                    mz[mt][s] = seen(nm[mt][s]);
                    grew |= nb[mt][s] > acc.big[mt][s];
                    far |= fabsf(mz[mt][s]) > kFar;
                }
            }
            if (__any_sync(0xffffffffu, far))
                break;
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    scale_rows(acc.o[mt], ex2(acc.big[mt][0] - seen(nb[mt][0])), ex2(acc.big[mt][1] - seen(nb[mt][1])));
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    acc.l[mt][s] *= ex2(acc.m[mt][s] - mz[mt][s]);
                    acc.m[mt][s] = nm[mt][s];
                    acc.big[mt][s] = nb[mt][s];
                    up[mt][s] = mz[mt][s] - seen(nb[mt][s]) + kLift;
                }
        } else {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (edge)
                    hide(mt);
                float r[2];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    float v[NS], nm = acc.m[mt][s];
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        v[i] = -INFINITY;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float &y = x[mt][i][e >> 1][2 * s + (e & 1)];
                            y = __fmul_rn(y, factor(mt, s, i));
                            v[i] = fmaxf(v[i], y);
                        }
                        nm = fmaxf(nm, v[i]);
                    }
                    nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, 1));
                    nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, 2));
                    const float z = seen(nm), was = acc.big[mt][s] + (acc.m[mt][s] - z);       // M from the new m
                    float nb = was;
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        nb = fmaxf(nb, (v[i] - z) + ex[kSubs + i * TG + tg]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float &y = x[mt][i][e >> 1][2 * s + (e & 1)];
                            y = __fsub_rn(y, z);
                        }
                    }
                    nb = fmaxf(nb, __shfl_xor_sync(0xffffffffu, nb, 1));
                    nb = fmaxf(nb, __shfl_xor_sync(0xffffffffu, nb, 2));
                    r[s] = was == -INFINITY ? 0.0f : ex2(was - nb);
                    acc.l[mt][s] *= ex2(acc.m[mt][s] - z);
                    acc.m[mt][s] = nm;
                    acc.big[mt][s] = nb;
                    mz[mt][s] = 0.0f;
                    up[mt][s] = kLift - seen(nb);
                }
                scale_rows(acc.o[mt], r[0], r[1]);
            }
        }
        uint32_t pw[MT][NS][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            // weights: p 2^(b + m - M + 15).  The power is at most 2^126: above it (M - m far below b) p is zero.
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const float b = ex[kSubs + i * TG + tg];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const float r = ex2(fminf(b + up[mt][s], 126.0f)), fi = FAR ? 1.0f : factor(mt, s, i);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float p0 = ex2(fmaf(x[mt][i][h][2 * s], fi, -mz[mt][s])), p1 = ex2(fmaf(x[mt][i][h][2 * s + 1], fi, -mz[mt][s]));
                        acc.l[mt][s] += p0 + p1;
                        const __half2 u = __floats2half2_rn(p0 * r, p1 * r);
                        pw[mt][i][2 * h + s] = *reinterpret_cast<const uint32_t *>(&u);
                    }
                }
            }
        }
        uint32_t nan_seen = 0;
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int n = 0; n < D / 8; n += 4) {
                uint32_t vc[4];
                ldmatrix4(vc, vs + (uint32_t)((i * TG + tg) * S::kSubBytes + n * 128) + v_off);
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
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        mma_m16n8k16_f16(acc.o[mt][n + u], pw[mt][i][0], pw[mt][i][1], pw[mt][i][2], pw[mt][i][3], b0, b1, acc.o[mt][n + u]);
                }
            }
        if (edge && __any_sync(0xffffffffu, nan_seen != 0)) {
            // looked at again, without the tokens that no row sees: in unused slots such codes are common
            int some_lo = INT_MAX, some_hi = 0;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    some_lo = min(some_lo, info[mt * 16 + 8 * s].lo);
                    some_hi = max(some_hi, info[mt * 16 + 8 * s].hi);
                }
            some_lo = __reduce_min_sync(0xffffffffu, some_lo);
            some_hi = __reduce_max_sync(0xffffffffu, some_hi);
            nan_seen = 0;
#pragma unroll 1
            for (int i = 0; i < NS; ++i) {
                const int k = tok0 + (i * TG + tg) * 16 + 4 * c, from = min(max(some_lo - k, 0), 4), to = min(max(some_hi - k, 0), 4);
                const uint32_t seen = (uint32_t)((1ull << (8 * to)) - 1) & ~(uint32_t)((1ull << (8 * from)) - 1);
#pragma unroll 1
                for (int n = 0; n < D / 8; n += 4) {
                    uint32_t vc[4];
                    ldmatrix4(vc, vs + (uint32_t)((i * TG + tg) * S::kSubBytes + n * 128) + v_off);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        nan_seen |= __vcmpeq4(vc[u] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) & seen;
                }
            }
        }
        if (edge && __any_sync(0xffffffffu, nan_seen != 0)) {
            const uint8_t *vb = sm + (size_t)st * S::kStageBytes + S::kTileBytes;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const RowInfo r0 = info[mt * 16], r1 = info[mt * 16 + 8];
#pragma unroll 1
                for (int k = 0; k < NS * 16; ++k) {
                    const int at = ((k >> 4) * TG + tg) * S::kSubBytes + (k & 15), j = tok0 + ((k >> 4) * TG + tg) * 16 + (k & 15);
                    const bool see0 = j >= r0.lo && j < r0.hi, see1 = j >= r1.lo && j < r1.hi;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if ((e < 2 ? see0 : see1) && (vb[at + (8 * n + 2 * c + (e & 1)) * 16] & 0x7F) == 0x7F)
                                acc.o[mt][n][e] = __uint_as_float(0x7FFFFFFFu);
                }
            }
        }
        __syncwarp();
        if (lane == 0)                  // for the warps of the other sets too
            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(empty + st)), "r"(SG) : "memory");
    }
    return t;
}

template <int D, int MT, int RG, int SG>
__device__ __forceinline__ void attend(const Piece &pc, uint8_t *sm, int qbuf, uint64_t *full, uint64_t *empty, uint32_t *hdr,
                                       long long &it, bool &dead, Acc<D, MT> &acc) {
    const int sg = (threadIdx.x >> 5) * SG / kConsumers;
    const int t = attend_tiles<D, MT, RG, SG, false>(pc, sm, qbuf, full, empty, hdr, it, pc.t0 + sg, dead, acc);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int s = 0; s < 2; ++s)                          // M from m from here on
            acc.big[mt][s] = acc.m[mt][s] == -INFINITY ? -INFINITY : acc.big[mt][s] - acc.m[mt][s];
    if (__builtin_expect(t < pc.t1, 0))
        attend_tiles<D, MT, RG, SG, true>(pc, sm, qbuf, full, empty, hdr, it, t, dead, acc);
    it += pc.t1 - pc.t0;
}

// Whether a row of the piece sees a position: one that does and has no weights had scores past fp32's range only.
__device__ __forceinline__ bool sees(const AttnArgs &a, const Piece &pc, int row) {
    int lo, hi;
    row_range(a.p, a.group, pc.kv, pc.n, pc.row0 + row, lo, hi);
    return lo < hi;
}

// Joins the token groups of a piece and writes the rows: to the output, or,
// where the unit has other pieces, to the workspace, the last CTA joining those.
// Eight rows of each warp at a time go through shared memory; a thread then adds four dims of a row over the warps.
template <int D, int MT, int RG>
__device__ __forceinline__ void finish(const AttnArgs &a, const Piece &pc, uint8_t *sm, Acc<D, MT> &acc, int *s_last) {
    using S = Smem<D>;
    constexpr int TG = kConsumers / RG, R = RG * MT * 16, Q = D / 4;
    const AttnProblem &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int rg = warp % RG, tg = warp / RG;
    float *s_m = reinterpret_cast<float *>(sm + S::kStats), *s_b = s_m + 256, *s_l = s_b + 256, *join = reinterpret_cast<float *>(sm + S::kJoin);
    const int pieces = pc.last - pc.first + 1;
    const int slot = (int)blockIdx.x * 2 + (pc.first == (int)blockIdx.x);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            acc.l[mt][s] += __shfl_xor_sync(0xffffffffu, acc.l[mt][s], 1);
            acc.l[mt][s] += __shfl_xor_sync(0xffffffffu, acc.l[mt][s], 2);
        }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (mt * 16 + 8 * s >= pc.rows)
                break;
            if (mt > 0 || s > 0)
                named_barrier_sync(1, kConsumers * 32);      // the buffer is free
            if (mt == 0 && s == 0 && c == 0) {
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i) {
                    const int at = tg * R + rg * MT * 16 + 8 * i + g;
                    s_m[at] = acc.m[i >> 1][i & 1];
                    s_b[at] = acc.big[i >> 1][i & 1];
                    s_l[at] = acc.l[i >> 1][i & 1];
                }
            }
            float *to = join + (size_t)(warp * 8 + g) * S::kPad + 2 * c;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2 *>(to + 8 * n) = make_float2(acc.o[mt][n][2 * s], acc.o[mt][n][2 * s + 1]);
            named_barrier_sync(1, kConsumers * 32);
#pragma unroll
            for (int i0 = 0; i0 < RG * 8 * Q; i0 += kConsumers * 32) {
                const int i = i0 + tid, r8 = i / Q % 8, wr = i / (8 * Q), d = i % Q * 4, row = wr * MT * 16 + mt * 16 + 8 * s + r8;
                if (row >= pc.rows || (RG * 8 * Q < kConsumers * 32 && i >= RG * 8 * Q))
                    continue;
                float m = -INFINITY, b = -INFINITY, l = 0.0f;        // b: M from m
#pragma unroll
                for (int t = 0; t < TG; ++t)
                    m = fmaxf(m, s_m[t * R + row]);
                const float mz = seen(m);
#pragma unroll
                for (int t = 0; t < TG; ++t)
                    b = fmaxf(b, s_b[t * R + row] + (s_m[t * R + row] - mz));
                const float bz = seen(b);
                float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int t = 0; t < TG; ++t) {
                    const float up = s_m[t * R + row] - mz;
                    l += s_l[t * R + row] * ex2(up);
                    const float w = ex2(s_b[t * R + row] + up - bz - kLift);
                    const float4 v = *reinterpret_cast<const float4 *>(join + (size_t)((t * RG + wr) * 8 + r8) * S::kPad + d);
                    o.x += v.x * w;
                    o.y += v.y * w;
                    o.z += v.z * w;
                    o.w += v.w * w;
                }
                // l is NaN where a score was, or was infinite: then so is the row
                if (l == 0.0f && pieces == 1 && sees(a, pc, row))
                    l = __uint_as_float(0x7FFFFFFFu);
                const float f = l == 0.0f ? 0.0f : exp2f(bz) / l;
                o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
                if (pieces == 1) {
                    const int r = pc.row0 + row;
                    if (!MOE_DBG_IN_RANGE(pc.q0 + r / a.group, p.T, a.hdr))
                        continue;
                    const size_t at = (size_t)(pc.q0 + r / a.group) * p.q_heads + pc.head * a.group + r % a.group;
                    uint32_t x, y;
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(o.y), "f"(o.x));
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(o.w), "f"(o.z));
                    *reinterpret_cast<uint2 *>(p.out + at * D + d) = make_uint2(x, y);
                    if (d == 0 && p.lse)
                        p.lse[at] = l == 0.0f ? -INFINITY : (mz + log2f(l)) * 0.69314718055994530942f;
                } else if (MOE_DBG_IN_RANGE(slot, 2 * a.ctas, a.hdr) && MOE_DBG_IN_RANGE(row, a.part_rows, a.hdr)) {
                    __stcg(reinterpret_cast<float4 *>(a.part + ((size_t)slot * a.part_rows + row) * D + d), o);
                    if (d == 0)
                        __stcg(a.part_sum + (size_t)slot * a.part_rows + row, make_float2(m, l * 0x1p-31f));   // no number of tokens brings that past 1
                }
            }
        }
    if (pieces > 1) {
        __threadfence();
        named_barrier_sync(1, kConsumers * 32);
        if (tid == 0) {
            __threadfence();
            const bool last = MOE_DBG_IN_RANGE(pc.first, a.ctas, a.hdr) && atomicAdd(a.tickets + pc.first, 1u) == (uint32_t)(pieces - 1);
            if (last)
                a.tickets[pc.first] = 0;              // for the next call
            *s_last = last;
            __threadfence();
        }
        named_barrier_sync(1, kConsumers * 32);
        if (*s_last) {
            constexpr int U = 8;                      // parts' loads in flight
            for (int i = tid; i < pc.rows * Q; i += kConsumers * 32) {
                const int row = i / Q, d = i % Q * 4;
                float m = -INFINITY, l = 0.0f;
                float4 o = make_float4(0, 0, 0, 0);
                for (int k0 = 0; k0 < pieces; k0 += U) {
                    float2 e[U];                  // m, l 2^-31
                    float4 v[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int k = k0 + u;
                        const size_t at = ((size_t)(pc.first + k) * 2 + (k == 0)) * a.part_rows + row;
                        const bool is = k < pieces && MOE_DBG_IN_RANGE(at, 2ll * a.ctas * a.part_rows, a.hdr);
                        e[u] = is ? __ldcg(a.part_sum + at) : make_float2(-INFINITY, 0.0f);
                        v[u] = is ? __ldcg(reinterpret_cast<const float4 *>(a.part + at * D + d)) : make_float4(0, 0, 0, 0);
                    }
                    float nm = m;
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        nm = fmaxf(nm, e[u].x);
                    const float mz = seen(nm), w0 = ex2(m - mz);
                    l *= w0;
                    o = make_float4(o.x * w0, o.y * w0, o.z * w0, o.w * w0);
                    m = nm;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const float w = e[u].y * ex2(e[u].x - mz);
                        l += w;
                        o.x += v[u].x * w;
                        o.y += v[u].y * w;
                        o.z += v[u].z * w;
                        o.w += v[u].w * w;
                    }
                }
                if (l == 0.0f && sees(a, pc, row))
                    l = __uint_as_float(0x7FFFFFFFu);
                const float w = l == 0.0f ? 0.0f : 1.0f / l;
                const int r = pc.row0 + row;
                const size_t to = (size_t)(pc.q0 + r / a.group) * p.q_heads + pc.head * a.group + r % a.group;
                uint32_t lo, hi;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(o.y * w), "f"(o.x * w));
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(o.w * w), "f"(o.z * w));
                *reinterpret_cast<uint2 *>(p.out + to * D + d) = make_uint2(lo, hi);
                if (d == 0 && p.lse)
                    p.lse[to] = l == 0.0f ? -INFINITY : (m + (log2f(l) + 31.0f)) * 0.69314718055994530942f;
            }
        }
    }
}

template <int D, int MT, int RG>
__device__ __forceinline__ void consume_piece(const AttnArgs &a, const Piece &pc, uint8_t *sm, int qbuf, uint64_t *full, uint64_t *empty,
                                              uint64_t *q_empty, long long &it, bool &dead, int *s_last) {
    Acc<D, MT> acc;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc.o[mt][n][e] = 0.0f;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            acc.m[mt][s] = acc.big[mt][s] = -INFINITY;
            acc.l[mt][s] = 0.0f;
        }
    }
    attend<D, MT, RG, RG == 1 ? 2 : 1>(pc, sm, qbuf, full, empty, a.hdr, it, dead, acc);
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(q_empty);
    finish<D, MT, RG>(a, pc, sm, acc, s_last);
}

template <int D, bool SMALL>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ AttnArgs a) {
    using S = Smem<D>;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ long long red[32];
    __shared__ Plan s_plan;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + S::kBars), *empty = full + S::kStages;
    uint64_t *q_full = empty + S::kStages, *q_empty = q_full + 2;
    int *s_last = reinterpret_cast<int *>(q_empty + 2);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full + i, 2);                // keys, values
            mbar_init(empty + i, kConsumers);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + i, kQWarps);
            mbar_init(q_empty + i, kConsumers);
        }
        fence_barrier_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const RowTile *recs = a.recs;
    if (SMALL) {
        RowTile *mine = reinterpret_cast<RowTile *>(sm + S::kRecs);
        make_small_plan(a, red, mine, &s_plan, blockIdx.x == 0);
        recs = mine;
    }
    const Plan pl = SMALL ? s_plan : *a.plan;
    const int warp = threadIdx.x >> 5;
    if (warp >= kConsumers) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp < kConsumers + 2)
            stream_cache<D>(a, pl, recs, sm, full, empty, warp > kConsumers);
        else
            load_queries<D>(a, pl, recs, sm, q_full, q_empty);
        return;
    }
    // 256 threads x 216 + 128 x 72 registers = the 384 x 168 of the launch
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    long long it = 0;
    bool dead = false;
    for (int u = 0;; ++u) {
        const int buf = u & 1;
        if (!dead) {
            dead = !__all_sync(0xffffffffu, wait_phase(q_full + buf, (uint32_t)((u / 2) & 1)));
            if (dead && (threadIdx.x & 31) == 0)
                record_status(a.hdr, MOE_ERR_DEVICE_TIMEOUT);
        }
        // all eight warps leave together, or none; and the last piece's join buffer is free
        const Piece pc = reinterpret_cast<const Piece *>(sm + S::kPieces)[buf];
        if (barrier_any(1, kConsumers * 32, dead || pc.rows == 0))
            break;
        if (pc.rows <= 16)
            consume_piece<D, 1, 1>(a, pc, sm, buf, full, empty, q_empty + buf, it, dead, s_last);
        else if (pc.rows <= 32)
            consume_piece<D, 2, 1>(a, pc, sm, buf, full, empty, q_empty + buf, it, dead, s_last);
        else
            consume_piece<D, 2, 2>(a, pc, sm, buf, full, empty, q_empty + buf, it, dead, s_last);
    }
}

// Rows of a part in the workspace.
int part_rows(int T, int group, int rows) { return (int)((long long)T * group < rows ? (long long)T * group : rows); }

int max_row_tiles(int T, int B, int group, int rows) { return (int)((long long)T * group / rows + B); }

}  // namespace

AttnLayout AttnLayout::make(int T, int B, int q_heads, int kv_heads, int head_dim) {
    AttnLayout L{};
    const int group = q_heads / kv_heads;
    const long long rows = (long long)T * group;
    size_t o = kInitBytes;
    auto take = [&](size_t bytes) { o = align_up(o, 256); size_t r = o; o += bytes; return r; };
    L.plan = take(sizeof(Plan));
    L.recs = take((size_t)max_row_tiles(T, B, group, kRows) * sizeof(RowTile));
    // a CTA has parts of at most two units; in the tensor-memory form of up to two row halves or token halves each
    const size_t cut = part_rows(T, group, kRows), tall = rows <= kAttnTcMinRows ? 0 : part_rows(T, group, 128);
    const size_t parts = (size_t)kMaxAttnCtas * (2 * cut > 4 * tall ? 2 * cut : 4 * tall);
    L.part = take(parts * head_dim * sizeof(float));
    L.part_sum = take(parts * sizeof(float2));
    L.nans = take(tall ? (size_t)kMaxAttnCtas * kAttnNanBytes : 0);
    L.total = align_up(o, 256);
    return L;
}

cudaError_t launch_kv_attention(const AttnProblem &p, void *ws, int sms, cudaStream_t stream) {
    const AttnLayout L = AttnLayout::make(p.T, p.B, p.q_heads, p.cache.kv_heads, p.cache.head_dim);
    const int group = p.q_heads / p.cache.kv_heads;
    int shift = 4;
    while ((1 << shift) < p.cache.block_size)
        ++shift;
    AttnArgs a{p, group, shift, kRows, part_rows(p.T, group, kRows), sms < kMaxAttnCtas ? sms : kMaxAttnCtas, max_row_tiles(p.T, p.B, group, kRows),
               p.scale * 1.44269504088896340736f, ws_at<Plan>(ws, L.plan), ws_at<RowTile>(ws, L.recs),
               ws_at<uint32_t>(ws, kHeaderBytes), ws_at<float>(ws, L.part), ws_at<float2>(ws, L.part_sum),
               ws_at<uint8_t>(ws, L.nans), ws_at<uint32_t>(ws, 0)};
    // The tensor-memory form where requests have more than 24 rows on average (us of it and of this one: 16 requests of
    // 1..4 tokens x 12 heads of a group 144 and 177, 32 of 1..10 x 4 rows 158 and 196; of 1..3 x 8 141 and 97; requests of 32 rows
    // each, 143 and 99, are the price of telling them from ragged ones by the average alone) and there are units enough
    // that its longer way from a unit's start to its end does not show (16 x 8 rows of four requests over 20,000 tokens 106
    // and 110, of two 114 and 74).
    const long long rows = (long long)p.T * group, units = ((rows + kAttnTcRows - 1) / kAttnTcRows + p.B - 1) * p.cache.kv_heads;
    const bool tall = rows > (long long)kAttnTcMinRows * p.B && units >= 32;
    auto go = [&](auto kernel, size_t smem) {
        cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        return r != cudaSuccess ? r : launch_pdl(kernel, dim3(a.ctas), dim3(kThreads), smem, stream, a);
    };
    if (!tall && p.B <= kSmallRequests && a.max_tiles <= kSmallTiles)
        return p.cache.head_dim == 64 ? go(attn_kernel<64, true>, Smem<64>::kBytes) : go(attn_kernel<128, true>, Smem<128>::kBytes);
    if (tall) {
        a.rows = kAttnTcRows;
        a.max_tiles = max_row_tiles(p.T, p.B, group, kAttnTcRows);
    }
    cudaError_t e = launch_pdl(attn_plan_kernel, dim3(1), dim3(kPlanThreads), p.B * sizeof(int), stream, a);
    if (e != cudaSuccess)
        return e;
    if (tall)
        return launch_attn_tc(&a, p.cache.head_dim, a.ctas, stream);
    return p.cache.head_dim == 64 ? go(attn_kernel<64, false>, Smem<64>::kBytes) : go(attn_kernel<128, false>, Smem<128>::kBytes);
}

}  // namespace moe
