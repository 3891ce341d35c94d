// latent.cu -- attention over a cache of one latent vector and one rotary key a token (moe_attn.h, b8).
//
//   s_j = q_latent.c_j + q_rope.r_j,   p_j = 2^((s_j - m) f),  f = softmax_scale log2(e),   out = sum_j p_j c_j / sum_j p_j
//
// All heads of a token read the same cache, so a row (a token's head) costs no bytes of its own: a token of the cache is 2 (L + 64) bytes and
// 2 (2 L + 64) operations a row, 121 operations a byte at 64 rows.  The work is to keep the loads running beside two products.
//
// Both products are made with the cache as the M side, which is never padded however few rows there are:
//   S^T = K Q^T     M = 64 tokens,      N = rows (up to 64), K = L + 64: the tile as it lies in the cache, dims innermost
//   O^T += C^T P^T  M = 128 dims a time, N = rows,           K = 64 tokens: the same bytes, read along the other axis
// A tile of 64 tokens is loaded once, by tensor copies (128-byte swizzle) of 64 dims each: the rotary key's 8 KB, and pairs of 64 dims (16 KB)
// in a ring of their own, which the second product gives back one by one.  O^T (L columns of 32-bit sums for 64 rows: 256
// columns) and two S^T stay in tensor memory.
//
// Softmax.  In S^T a row is a column, spread over 64 lanes, and a maximum over tokens would be a walk through shuffles for each.
// None is needed: any score of a row serves as its reference m as long as the powers stay in range.  The reference is the score of the
// piece's first token; a row's moves (to its maximum, with O and the sums) when a power passes 2^32, which one vote a tile finds out.
// s - m is taken before the factor, so that it is as exact as the scores, of any size.
// The product takes weights in bf16, each within 2^-8 of itself: the operands of an MMA have one type, and the values are bf16.  O is
// divided by the sum of those same rounded weights, so that it is an average of values, and a weight's rounding moves it by the token's
// distance from the average only: a row that one token dominates is that token, whatever its weight's bits.  (Over the sum of the unrounded ones
// it was off by up to 2^-8; mean errors with scores of standard deviation 3 and 6, on the CPU: 0.0021 and 0.0020, and 0.0019 and 0.0017.)  lse is
// of the sum of the unrounded ones.
//
// What a row does not see: its weight is 0, and the values of such tokens must be finite for the product.  In tiles that some row does not see
// in full (the last ones of a request) values past the last row's end become zero; those that some rows see become zero where they
// are not finite, and their weight NaN for the rows that do see them.
//
// Work is cut as in attn.cu (attn_plan.cuh): units of rows, their tiles laid end to end and cut into equal ranges; a range that cuts a
// unit leaves its sums in the workspace, and latent_join_kernel adds them up (one request's parts are many: the last CTA alone would be a
// while at it).  With more than 64 heads and single tokens two CTAs take the halves of a unit's rows, side by side, so that the second reads
// the cache from L2.
//
// Warps: 0..7 softmax (warp % 4 = lane quarter, 16 tokens each; warp / 4 = half of the rows), 8 streams the cache, 9 and 10 issue the products
// (one warp for both was often at the scores' when weights were ready: 64 requests of 16,384 tokens, 64 heads, 292 us for 261).  With 64 rows the
// queries take 72 KB and leave the ring 8 pairs, two tiles; with 16 rows 11.
//
// Measured: 64 requests of up to 49,152 tokens, 64 heads, 387 us (6.0 TB/s, 88 % of a copy's rate; a tile takes 1.76 us, 1.66 at that rate).  The
// way of a tile from its copies to the last pair given back takes 3.7 us, two are under way.  152 requests of 8,192, 16 heads, 222 us (6.5 TB/s).
// Where bytes are shared by more rows, shared memory is next: an MMA of the scores reads 2 KB of the cache and 32 bytes a row in
// 32 cycles, one of the values 4 KB and 32 bytes a row in 48 (both measured back to back; 24 and 39 with 16 rows): with 64 rows and the tile's arrival
// 2,500 cycles a tile, 1.2 us.  48 ragged requests of 96 heads, two CTAs to a unit, run at 1.4 us a tile, prompt chunks with 256 dims at
// 0.74 of 0.69.  One request of 1,000 tokens takes 14.0 us, steps that wait for one another: start and plan, walk and queries, tiles (16 of
// them over seven CTAs, three at most; the first CTA's range is the unit's fixed cost), results, the join's start and work.  Tried: the next tiles asked into L2 by tensor prefetches (no change, 3 % slower with 16 rows).
#define MOE_PLAN_TILE 64
#define MOE_PLAN_UNIT_COST 3
#define MOE_PLAN_MIN_COST 3
#include <type_traits>

#include "attn_plan.cuh"

namespace moe {
namespace {

constexpr int kSoftWarps = 8, kThreads = (kSoftWarps + 3) * 32, kSoft = kSoftWarps * 32;
constexpr int kMaxRows = 64;                 // of a CTA's unit
constexpr int kChunkBytes = kTile * 128;     // 64 dims of a tile
constexpr int kMaxSlots = 12;                // pairs of chunks in the ring
constexpr int kMaxSmem = 227 * 1024;         // of a CTA
constexpr int kRopeSlots = 2;
constexpr int kSCol = 256;                   // tensor memory: O^T at 64 m, S^T from here
constexpr float kMostPower = 32.0f;

constexpr int kSmallUnits = 152, kSmallRequests = 256;       // most of a plan that every CTA makes for itself
constexpr long long kSmallTokens = 1ll << 29;               // and tokens of a request: its work fits an int

// A cut unit that begins in a CTA: where its rows go, its parts.
struct LatentJoin {
    long long row;                           // first of its rows in out
    int rows, first, last;
    int blind;                               // its first rows that see nothing
};

struct LatentArgs {
    AttnArgs a;                              // the plan's view: one key/value head, `heads` query heads
    LatentProblem p;
    int split;                               // CTAs that share a unit's rows: 1 or 2
    int small;                               // whether every CTA makes the plan for itself
    int q_rows;                              // rows of the query buffer
    int slots;                               // pairs in the ring
    int cap;                                 // rows of a part
    float factor;
    LatentJoin *joins;
    float *part;                             // [slot][cap][L]
    float4 *part_sum;                        // [slot][cap]: m, sum, sum of the rounded weights
};

template <int L>
struct LatentSmem {
    static constexpr int kPairs = L / 128;
    static constexpr int kChunks = L / 64 + 1;
    uint8_t *ring, *rope, *p, *q;
    uint64_t *pair_full, *pair_empty, *rope_full, *rope_empty, *s_full, *p_ready, *o_done, *o_free, *q_ready;
    Plan *plan;
    float *ref, *sum;                        // [64] each
    float *red, *fac;                        // [2][4][64] and [64], over the weights while no product reads them
    int *hi;                                 // [64]
    uint32_t *bad;                           // a bit for each token of a tile
    uint32_t *taddr;
    int *before;                             // [kSmallUnits], and which request and row tile of it
    uint16_t *which;
    static constexpr int kBars = 2 * kMaxSlots + 2 * kRopeSlots + 8;
    static constexpr size_t kTail = kBars * 8 + sizeof(Plan) + 3 * 64 * 4 + 16 + kSmallUnits * 6;
    __host__ __device__ static size_t fixed(int q_rows) { return (size_t)kRopeSlots * kChunkBytes + kChunkBytes + (size_t)q_rows * 128 * kChunks + kTail + 1024; }
    __host__ __device__ static size_t bytes(int q_rows, int slots) { return fixed(q_rows) + (size_t)slots * 2 * kChunkBytes; }
    __host__ static int slots_for(int q_rows) {
        const int n = (int)((kMaxSmem - fixed(q_rows)) / (2 * kChunkBytes));
        return n < kMaxSlots ? n : kMaxSlots;
    }
    __device__ LatentSmem(uint8_t *base, int q_rows, int slots) {
        ring = base;
        rope = ring + (size_t)slots * 2 * kChunkBytes;
        p = rope + kRopeSlots * kChunkBytes;
        q = p + kChunkBytes;
        uint64_t *b = reinterpret_cast<uint64_t *>(q + (size_t)q_rows * 128 * kChunks);
        pair_full = b;
        pair_empty = b + kMaxSlots;
        rope_full = b + 2 * kMaxSlots;
        rope_empty = rope_full + kRopeSlots;
        s_full = rope_empty + kRopeSlots;
        p_ready = s_full + 2;
        o_done = p_ready + 2;
        o_free = o_done + 1;
        q_ready = o_free + 1;
        plan = reinterpret_cast<Plan *>(b + kBars);
        ref = reinterpret_cast<float *>(plan + 1);
        sum = ref + 64;
        red = reinterpret_cast<float *>(p);
        fac = red + 512;
        hi = reinterpret_cast<int *>(sum + 64);
        bad = reinterpret_cast<uint32_t *>(hi + 64);
        taddr = bad + 2;
        before = reinterpret_cast<int *>(bad + 4);
        which = reinterpret_cast<uint16_t *>(before + kSmallUnits);
    }
};

// A warp's walk through the range of its CTA (of its CTAs, where they share units), as Walk's; the units are listed in shared memory or
// in the workspace, and the search for the first looks at 32 of them at a time.
template <int L>
struct LatentWalk {
    const LatentArgs &g;
    const LatentSmem<L> &s;
    long long pos, end, base, per;
    int unit, units, cta;
    RowTile r;

    __device__ long long begins(int u) const { return g.small ? s.before[u] : g.a.recs[u].before; }
    __device__ void load() {
        if (!g.small) {
            r = g.a.recs[unit];
            return;
        }
        const int request = s.which[unit] & 255, q0 = __ldg(g.a.p.q_offsets + request);
        r = row_tile(g.a, request, q0, __ldg(g.a.p.q_offsets + request + 1) - q0, __ldg(g.a.p.kv_lens + request), (s.which[unit] >> 8) * g.a.rows);
        r.before = s.before[unit];
    }
    __device__ LatentWalk(const LatentArgs &args, const LatentSmem<L> &smem) : g(args), s(smem), cta((int)blockIdx.x / args.split) {
        const Plan pl = *s.plan;
        units = pl.row_tiles;
        per = pl.per;
        pos = (long long)cta * per;
        end = min(pos + per, pl.work);
        unit = units;
        if (cta >= pl.ctas || pos >= pl.work)
            return;
        int lo = 0, hi = units;                 // the last unit that begins at pos or before
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, i = lo + (int)(threadIdx.x & 31) * step;
            const int n = __popc(__ballot_sync(0xffffffffu, i < hi && begins(i) <= pos));        // the first always does
            hi = min(hi, lo + n * step);
            lo += (n - 1) * step;
        }
        unit = lo;
        load();
        base = r.before;
    }
    // The next piece; false at the end of the range.
    __device__ bool next(Piece &pc) {
        while (unit < units && base < end) {
            const int lo = (int)min(max(pos - base - kUnitCost, 0ll), (long long)r.tiles);
            const int hi = (int)max(min(end - base - kUnitCost, (long long)r.tiles), 0ll);
            const bool mine = r.tiles == 0 ? base >= pos : hi > lo;
            if (mine) {
                pc.request = r.request;
                pc.head = 0;
                pc.row0 = r.row0;
                pc.q0 = r.q0;
                pc.n = r.n;
                pc.kv = r.kv;
                pc.rows = min(g.a.rows, r.n * g.a.group - r.row0);
                pc.tile0 = r.tile0;
                pc.t0 = lo;
                pc.t1 = hi;
                pc.first = pc.last = cta;
                const long long t0 = base + kUnitCost, t1 = t0 + r.tiles - 1;
                if (r.tiles > 0 && (t0 < pos || t1 >= end)) {      // cut
                    pc.first = t0 < pos ? (int)(t0 / per) : cta;
                    pc.last = t1 >= end ? (int)(t1 / per) : cta;
                }
            }
            base += r.tiles + kUnitCost;
            if (++unit < units && base < end)
                load();
            if (mine)
                return true;
        }
        return false;
    }
};

// A CTA's share of a piece: its rows and the tiles that they see.
struct Mine {
    int row0, rows, n_side;                  // rows, and rounded up to the MMA's N
    int tok0, tiles;
    int hi_min, hi_max;                      // positions that the first and the last row see

    __device__ Mine() {}
    __device__ Mine(const LatentArgs &g, const Piece &pc) {
        const int part = g.split == 1 ? 0 : (int)blockIdx.x & 1;
        const int per = g.split == 1 ? pc.rows : ((pc.rows + 1) / 2 + 15) / 16 * 16;
        row0 = pc.row0 + part * per;
        rows = max(0, min(pc.rows - part * per, per));
        n_side = (rows + 15) / 16 * 16;
        tok0 = (pc.tile0 + pc.t0) * kTile;
        tiles = hi_min = hi_max = 0;
        if (rows > 0) {
            int lo;
            row_range(g.a.p, g.a.group, pc.kv, pc.n, row0, lo, hi_min);
            row_range(g.a.p, g.a.group, pc.kv, pc.n, row0 + rows - 1, lo, hi_max);
            const int end = min((pc.tile0 + pc.t1) * kTile, hi_max);
            tiles = end > tok0 ? (end - tok0 + kTile - 1) / kTile : 0;
        }
    }
};

// ------------------------------------------------------------------ tcgen05

// Operand descriptors, rows of 128 bytes in swizzled atoms of 8.  Low word: address, and the distance of 64 further elements along the
// row where the summed axis runs across the rows (a chunk; not used where it runs along).  The high word is the same for all.
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_along(uint32_t addr) { return ((addr & 0x3FFFF) >> 4) | 1u << 16; }
__device__ __forceinline__ uint32_t desc_across(uint32_t addr) { return ((addr & 0x3FFFF) >> 4) | (uint32_t)(kChunkBytes >> 4) << 16; }

// fp32 sums of bf16 products; across: both operands are read across their rows.
__device__ __forceinline__ uint32_t idesc_bf16(int m, int n, bool across) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (across ? (1u << 15) | (1u << 16) : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

// Four products in a row, the operands' addresses STEP 16-byte units apart, issued by one elected lane of a converged warp.
template <int STEP>
__device__ __forceinline__ void mma4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p, q;\n.reg .b64 a, b;\n.reg .b32 x, y;\n"
        "elect.sync _|p, 0xffffffff;\nsetp.ne.b32 q, %4, 0;\n"
        "mov.b64 a, {%1, %5};\nmov.b64 b, {%2, %5};\n"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n"
        "add.u32 x, %1, %6;\nadd.u32 y, %2, %6;\nmov.b64 a, {x, %5};\nmov.b64 b, {y, %5};\n"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, 1;\n"
        "add.u32 x, x, %6;\nadd.u32 y, y, %6;\nmov.b64 a, {x, %5};\nmov.b64 b, {y, %5};\n"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, 1;\n"
        "add.u32 x, x, %6;\nadd.u32 y, y, %6;\nmov.b64 a, {x, %5};\nmov.b64 b, {y, %5};\n"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, 1;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHigh), "n"(STEP)
        : "memory");
}

__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile(
        "{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\n"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16 lanes x 32 columns: v[4 i + 2 k + e] is lane lane / 4 + 8 k, column 8 i + 2 (lane % 4) + e.
__device__ __forceinline__ void tmem_ld_16x32(float (&v)[16], uint32_t addr) {
    uint32_t *u = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]), "=r"(u[9]),
          "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld_32x16(float (&v)[16], uint32_t addr) {
    uint32_t *u = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]), "=r"(u[9]),
          "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_st_32x16(uint32_t addr, const float (&v)[16]) {
    const uint32_t *u = reinterpret_cast<const uint32_t *>(v);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n"
                 "tcgen05.wait::st.sync.aligned;" ::"r"(addr),
                 "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]),
                 "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
                 : "memory");
}

// [1][rows][64 dims] or [2][rows][64 dims] of chunks c.. and rows row.. of the cache, by one elected lane of a converged warp (in a
// branch of one lane a copy takes 60 ns to issue).
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, int row, int c, uint32_t bar) {
    asm volatile(
        "{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\n"
        "@p cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(c), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\n@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(bar), "r"(bytes)
        : "memory");
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// (a0, a1) += (b0, b1), in one instruction.
__device__ __forceinline__ void add2(float &a0, float &a1, float b0, float b1) {
    asm("{\n.reg .b64 a, b;\nmov.b64 a, {%0, %1};\nmov.b64 b, {%2, %3};\nadd.rn.f32x2 a, a, b;\nmov.b64 {%0, %1}, a;\n}\n"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1));
}

// A barrier of the softmax warps, and one that or's a predicate.
__device__ __forceinline__ void soft_sync() { named_barrier_sync(1, kSoft); }
__device__ __forceinline__ bool soft_any(bool v) {
    uint32_t r;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.cta.red.or.pred q, 1, %2, p;\nselp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(kSoft)
        : "memory");
    return r != 0;
}

// Waits of a role's warp; after one that gave up it waits no more.
struct Waiter {
    uint32_t *hdr;
    bool dead;
    __device__ void operator()(uint64_t *bar, uint32_t parity) {
        if (!dead) {
            dead = !__all_sync(0xffffffffu, wait_phase(bar, parity));
            if (dead && (threadIdx.x & 31) == 0)
                record_status(hdr, MOE_ERR_DEVICE_TIMEOUT);
        }
        fence_after();
    }
};

// A place in a ring of slots, and the parity of its full barrier.
struct Place {
    uint32_t slot = 0, parity = 0;
    __device__ void next(uint32_t slots) {
        if (++slot == slots) {
            slot = 0;
            parity ^= 1;
        }
    }
};

// ------------------------------------------------------------ the cache's tiles

template <int L>
__device__ __forceinline__ void latent_stream(const LatentArgs &g, const LatentSmem<L> &s, const CUtensorMap *pair_map,
                                              const CUtensorMap *chunk_map) {
    const AttnProblem &p = g.a.p;
    const int lane = threadIdx.x & 31;
    const int box_shift = min(g.a.shift, 6), subs = kTile >> box_shift;          // a box's rows lie in one block
    bool dead = false;
    LatentWalk<L> walk(g, s);
    Piece pc;
    Place pair, rope;
    uint32_t pairs = 0, ropes = 0;
    while (walk.next(pc)) {
        const Mine m(g, pc);
        const int32_t *row = p.table + (size_t)pc.request * p.max_blocks;
        // the rows of the cache of 32 boxes at a time, a lane each; the next ones' block ids on their way
        auto fetch = [&](int box) {
            const long long tok = (long long)m.tok0 + ((long long)(box + lane) << box_shift);
            return tok < m.hi_max && box + lane < m.tiles * subs ? __ldg(row + (tok >> g.a.shift)) : -1;
        };
        int next = m.tiles > 0 ? fetch(0) : -1, at = 0;
        for (int t = 0; t < m.tiles; ++t) {
            const int box = t * subs;
            if (box % 32 == 0) {
                int page = next;
                const long long tok = (long long)m.tok0 + ((long long)(box + lane) << box_shift);
                const bool used = tok < m.hi_max && box + lane < m.tiles * subs;
                if (used && (page < 0 || page >= p.cache.num_blocks)) {
                    record_status(g.a.hdr, MOE_ERR_DEVICE_ASSERT);
                    page = 0;
                }
                at = used ? (page << g.a.shift) + (int)(tok & ((1 << g.a.shift) - 1)) : -1;
                next = box + 32 < m.tiles * subs ? fetch(box + 32) : -1;
            }
            // boxes of this tile that hold something, and where in the cache
            const int live = min(subs, (m.hi_max - (m.tok0 + t * kTile) + (1 << box_shift) - 1) >> box_shift);
            const uint32_t chunk_bytes = (uint32_t)(live << box_shift) * 128;
            int to[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                to[k] = __shfl_sync(0xffffffffu, at, ((box & 31) + k) & 31);
            // chunks c .. c + n - 1
            auto load = [&](uint32_t dst, uint64_t *full, uint64_t *empty, uint32_t parity, bool used, int c, int n) {
                if (used && !dead) {
                    dead = !__all_sync(0xffffffffu, wait_phase(empty, parity));
                    if (dead && lane == 0)
                        record_status(g.a.hdr, MOE_ERR_DEVICE_TIMEOUT);
                }
                if (dead)
                    return;
                const uint32_t bar = smem_u32(full);
                expect_bytes(bar, chunk_bytes * n);
                if (subs == 1) {
                    copy_box(dst, n == 2 ? pair_map : chunk_map, to[0], c, bar);
                    return;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < live)
                        for (int i = 0; i < n; ++i)
                            copy_box(dst + i * kChunkBytes + (k << box_shift) * 128, chunk_map, to[k], c + i, bar);
            };
            load(smem_u32(s.rope) + rope.slot * kChunkBytes, s.rope_full + rope.slot, s.rope_empty + rope.slot, rope.parity ^ 1, ropes >= kRopeSlots,
                 L / 64, 1);
            rope.next(kRopeSlots);
            ++ropes;
#pragma unroll 1
            for (int i = 0; i < LatentSmem<L>::kPairs; ++i, ++pairs) {
                load(smem_u32(s.ring) + pair.slot * (2 * kChunkBytes), s.pair_full + pair.slot, s.pair_empty + pair.slot, pair.parity ^ 1,
                     pairs >= (uint32_t)g.slots, 2 * i, 2);
                pair.next(g.slots);
            }
        }
    }
    // copies in flight end before the CTA's memory goes away
    Waiter wait{g.a.hdr, dead};
    for (uint32_t i = pairs > (uint32_t)g.slots ? pairs - g.slots : 0; i < pairs && !wait.dead; ++i)
        wait(s.pair_full + i % g.slots, (i / g.slots) & 1);
    for (uint32_t i = ropes > kRopeSlots ? ropes - kRopeSlots : 0; i < ropes && !wait.dead; ++i)
        wait(s.rope_full + i % kRopeSlots, (i / kRopeSlots) & 1);
}

// S^T = K Q^T
template <int L>
__device__ __forceinline__ void latent_scores(const LatentArgs &g, const LatentSmem<L> &s, uint32_t tmem) {
    constexpr int kPairs = LatentSmem<L>::kPairs;
    Waiter wait{g.a.hdr, false};
    LatentWalk<L> walk(g, s);
    Piece pc;
    Place pair, rope;
    uint32_t tiles = 0, units = 0;
    const uint32_t q_chunk = (uint32_t)g.q_rows * 128 / 16, dq = desc_along(smem_u32(s.q));
    while (walk.next(pc)) {
        const Mine m(g, pc);
        if (m.tiles == 0)
            continue;
        const uint32_t is = idesc_bf16(kTile, m.n_side, false);
        wait(s.q_ready, units & 1);
        ++units;
        for (int t = 0; t < m.tiles; ++t, ++tiles) {
            const uint32_t d = tmem + kSCol + 64 * (tiles & 1);
            if (tiles >= 2)                        // the weights of the scores that were here have been made
                wait(s.p_ready + (tiles & 1), ((tiles >> 1) - 1) & 1);
            wait(s.rope_full + rope.slot, rope.parity);
            if (!wait.dead)
                mma4<2>(d, desc_along(smem_u32(s.rope + rope.slot * kChunkBytes)), dq + (L / 64) * q_chunk, is, 0);
            commit(s.rope_empty + rope.slot);
            rope.next(kRopeSlots);
#pragma unroll 1
            for (int i = 0; i < kPairs; ++i) {
                const uint32_t dk = desc_along(smem_u32(s.ring + (size_t)pair.slot * 2 * kChunkBytes));
                wait(s.pair_full + pair.slot, pair.parity);
                if (!wait.dead) {
                    mma4<2>(d, dk, dq + 2 * i * q_chunk, is, 1);
                    mma4<2>(d, dk + (kChunkBytes >> 4), dq + (2 * i + 1) * q_chunk, is, 1);
                }
                pair.next(g.slots);
            }
            commit(s.s_full + (tiles & 1));
        }
    }
    if (tiles > 0)                                 // issued products end before the CTA's memory goes away
        wait(s.s_full + ((tiles - 1) & 1), ((tiles - 1) >> 1) & 1);
}

// O^T += C^T P^T
template <int L>
__device__ __forceinline__ void latent_values(const LatentArgs &g, const LatentSmem<L> &s, uint32_t tmem) {
    Waiter wait{g.a.hdr, false};
    LatentWalk<L> walk(g, s);
    Piece pc;
    Place pair;
    uint32_t tiles = 0, units = 0;
    const uint32_t dp = desc_across(smem_u32(s.p));
    while (walk.next(pc)) {
        const Mine m(g, pc);
        if (m.tiles == 0)
            continue;
        const uint32_t io = idesc_bf16(128, m.n_side, true);
        if (units > 0)
            wait(s.o_free, (units - 1) & 1);
        ++units;
        for (int t = 0; t < m.tiles; ++t, ++tiles) {
            wait(s.p_ready + (tiles & 1), (tiles >> 1) & 1);
#pragma unroll 1
            for (int i = 0; i < LatentSmem<L>::kPairs; ++i) {
                if (!wait.dead)
                    mma4<16 * 128 / 16>(tmem + 64 * i, desc_across(smem_u32(s.ring + (size_t)pair.slot * 2 * kChunkBytes)), dp, io, t > 0);
                commit(s.pair_empty + pair.slot);
                pair.next(g.slots);
            }
            commit(s.o_done);
        }
    }
    if (tiles > 0)
        wait(s.o_done, (tiles - 1) & 1);
}

// ------------------------------------------------------------------ softmax

template <int L>
__device__ __forceinline__ void latent_softmax(const LatentArgs &g, const LatentSmem<L> &s, uint32_t tmem) {
    constexpr int kPairs = LatentSmem<L>::kPairs;
    const LatentProblem &p = g.p;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, tid = threadIdx.x;
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const int part = g.split == 1 ? 0 : (int)blockIdx.x & 1;
    const int col0 = 32 * half + 2 * (lane & 3);            // this thread's columns: col0 + 8 i + e
    const int tok_a = 16 * quarter + (lane >> 2);           // its tokens of a tile: tok_a + 8 k
    const float f = g.factor;
    Waiter wait{g.a.hdr, false};
    LatentWalk<L> walk(g, s);
    Piece pc{};
    Mine m;
    LatentJoin join{0, 0, 0, 0, 0};
    uint32_t tiles = 0;                                      // so far
    auto first_row = [&] { return (long long)pc.q0 * p.heads + m.row0; };
    auto slot_of = [&] { return (walk.cta * 2 + (walk.cta == pc.first)) * g.split + part; };
    // the next piece with something to see; those without have their results at once
    auto advance = [&]() -> bool {
        while (walk.next(pc)) {
            m = Mine(g, pc);
            if (m.rows == 0)
                continue;
            if (pc.first != pc.last && walk.cta == pc.first) {
                // a row sees something unless its token lies before position 0
                const int token = p.causal ? max(0, pc.n - pc.kv) : 0;
                join = LatentJoin{first_row(), m.rows, pc.first, pc.last, (int)max(0ll, min((long long)token * p.heads - m.row0, (long long)m.rows))};
            }
            if (m.tiles > 0)
                return true;
            if (pc.first == pc.last) {
                uint4 *to = reinterpret_cast<uint4 *>(p.out + first_row() * L);
                for (int i = tid; i < m.rows * (L / 8); i += kSoft)
                    to[i] = make_uint4(0, 0, 0, 0);
                if (p.lse && tid < m.rows)
                    p.lse[first_row() + tid] = -INFINITY;
            } else if (tid < m.rows) {
                __stcg(g.part_sum + (size_t)slot_of() * g.cap + tid, make_float4(-INFINITY, 0.0f, 0.0f, 0.0f));
            }
        }
        return false;
    };
    // a piece's queries on their way, zero past the last row: a warp a row, all copies in flight together
    auto load_queries = [&] {
        for (int r = warp; r < m.n_side; r += kSoftWarps) {
            const int64_t t = pc.q0 + (m.row0 + r) / p.heads, h = (m.row0 + r) % p.heads;
            const uint16_t *ql = p.ql + t * p.ql_st + h * p.ql_sh, *qr = p.qr + t * p.qr_st + h * p.qr_sh;
#pragma unroll
            for (int k = 0; k < (L / 8 + 8 + 31) / 32; ++k) {
                const int c = lane + 32 * k;
                uint8_t *to = s.q + (size_t)(c >> 3) * g.q_rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
                if (c < L / 8 + 8) {
                    if (r < m.rows)
                        cp_async16(to, c < L / 8 ? ql + 8 * c : qr + (8 * c - L));
                    else
                        *reinterpret_cast<uint4 *>(to) = make_uint4(0, 0, 0, 0);
                }
            }
        }
        cp_async_commit();
    };
    bool more = advance(), stored = false;
    if (more)
        load_queries();
    while (more) {
        const bool whole = pc.first == pc.last;
        if (tid < kMaxRows) {
            int lo, hi = m.hi_max;
            if (tid < m.rows)
                row_range(g.a.p, g.a.group, pc.kv, pc.n, m.row0 + tid, lo, hi);
            s.hi[tid] = hi;
        }
        cp_async_wait<0>();
        fence_async();
        soft_sync();
        if (tid == 0)
            mbar_arrive(s.q_ready);
        const int groups = max(0, min(4, (m.n_side - 32 * half) / 8));           // columns of this warp, by 8
        float ref[8], sum[8], even[8];                       // even: of the weights as the product takes them
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ref[i] = sum[i] = even[i] = 0.0f;
        for (int t = 0; t < m.tiles; ++t, ++tiles) {
            const int tok = m.tok0 + t * kTile;
            const bool edge = tok + kTile > m.hi_min;        // some row does not see all of the tile
            wait(s.s_full + (tiles & 1), (tiles >> 1) & 1);
            float x[16];
            tmem_ld_16x32(x, lanes + kSCol + 64 * (tiles & 1) + 32 * half);
            if (edge) {
                if (tid < 2)
                    s.bad[tid] = 0;
                soft_sync();
                const int j0 = max(0, m.hi_min - tok), n = (kTile - j0) * (L / 8);
                for (int i = tid; i < n; i += kSoft) {
                    const int j = j0 + i / (L / 8), c = i % (L / 8);
                    const uint32_t ring = (tiles * kPairs + c / 16) % g.slots;
                    uint4 *at = reinterpret_cast<uint4 *>(s.ring + (size_t)ring * 2 * kChunkBytes + (c / 8 & 1) * kChunkBytes + j * 128 +
                                                          (((c & 7) ^ (j & 7)) << 4));
                    if (tok + j >= m.hi_max) {
                        *at = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    const uint4 v = *at;
                    uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    bool odd = false;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t not_finite = __vcmpeq2(w[e] & 0x7F807F80u, 0x7F807F80u);
                        odd |= not_finite != 0;
                        w[e] &= ~not_finite;
                    }
                    if (odd) {
                        atomicOr(s.bad + j / 32, 1u << (j & 31));
                        *at = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                fence_async();
                soft_sync();
            }
            if (t == 0) {
                // the first token's scores are the references; rows that do not see it see nothing here
                if (quarter == 0 && lane < 4)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        s.ref[col0 + 8 * (i >> 1) + (i & 1)] = x[4 * (i >> 1) + (i & 1)];
                soft_sync();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int col = col0 + 8 * (i >> 1) + (i & 1);
                    ref[i] = tok < s.hi[col] ? fmaxf(s.ref[col], -3.4e38f) : 0.0f;         // finite, should that score have left fp32 below
                }
            }
            uint32_t pair[8];                                // the weights, by two columns, and the tile's share of the sums
            float of_sum[8], of_even[8];
            // Weights of the scores, two columns in an instruction; whether one has grown too far.  (Its forms are apart, so that one has no
            // branches: with the edge's tests inside, a tile took 150 ns more.)
            auto weigh_as = [&](auto groups_of, auto edge_of) -> bool {
                constexpr int G = decltype(groups_of)::value;
                constexpr bool EDGE = decltype(edge_of)::value;
                float most = -INFINITY;
#pragma unroll
                for (int i = 0; i < G; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float y0, y1;
                        asm("{\n.reg .b64 a, b;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nadd.rn.f32x2 a, a, b;\nmov.b64 b, {%6, %6};\n"
                            "mul.rn.f32x2 a, a, b;\nmov.b64 {%0, %1}, a;\n}\n"
                            : "=f"(y0), "=f"(y1)
                            : "f"(x[4 * i + 2 * k]), "f"(x[4 * i + 2 * k + 1]), "f"(-ref[2 * i]), "f"(-ref[2 * i + 1]), "f"(f));
                        float v0 = ex2(y0), v1 = ex2(y1);
                        if (EDGE) {
                            const int j = tok_a + 8 * k, c = col0 + 8 * i;
                            const bool sees0 = tok + j < s.hi[c], sees1 = tok + j < s.hi[c + 1];
                            if (s.bad[j / 32] >> (j & 31) & 1)
                                v0 = v1 = __uint_as_float(0x7FFFFFFFu);
                            v0 = sees0 ? v0 : 0.0f;
                            v1 = sees1 ? v1 : 0.0f;
                            y0 = sees0 ? y0 : -INFINITY;
                            y1 = sees1 ? y1 : -INFINITY;
                        }
                        const uint32_t r = bf16_pair(v0, v1);
                        const float r0 = __uint_as_float(r << 16), r1 = __uint_as_float(r & 0xFFFF0000u);
                        pair[2 * i + k] = r;
                        if (k == 0) {
                            of_sum[2 * i] = v0, of_sum[2 * i + 1] = v1;
                            of_even[2 * i] = r0, of_even[2 * i + 1] = r1;
                        } else {
                            add2(of_sum[2 * i], of_sum[2 * i + 1], v0, v1);
                            add2(of_even[2 * i], of_even[2 * i + 1], r0, r1);
                        }
                        most = fmaxf(most, fmaxf(y0, y1));
                    }
                return most > kMostPower;
            };
            auto weigh = [&]() -> bool {
                using std::integral_constant;
                if (groups == 4)
                    return edge ? weigh_as(integral_constant<int, 4>(), std::true_type()) : weigh_as(integral_constant<int, 4>(), std::false_type());
                if (groups == 2)
                    return edge ? weigh_as(integral_constant<int, 2>(), std::true_type()) : weigh_as(integral_constant<int, 2>(), std::false_type());
                return false;
            };
            auto store = [&] {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < groups) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int j = tok_a + 8 * k, c = col0 + 8 * i;       // 8 columns are 16 bytes
                            *reinterpret_cast<uint32_t *>(s.p + j * 128 + (((c >> 3) ^ (j & 7)) << 4) + (c & 7) * 2) = pair[2 * i + k];
                        }
                    }
                fence_async();
            };
            // once, or again from references at the maxima (one copy of the code: a request of few tokens waits for it to arrive)
#pragma unroll 1
            for (int pass = 0;; ++pass) {
                const bool grew = weigh();
                if (pass == 0 && t > 0)                      // the weights before have been read
                    wait(s.o_done, (tiles - 1) & 1);
                store();
                fence_before();
                if (pass == 1) {
                    soft_sync();
                    break;
                }
                if (!soft_any(grew))
                    break;
                // references to the maxima; with them the sums, and O
                float top[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int col = col0 + 8 * (i >> 1) + (i & 1);
                    top[i] = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (!edge || tok + tok_a + 8 * k < s.hi[col])
                            top[i] = fmaxf(top[i], x[4 * (i >> 1) + 2 * k + (i & 1)]);
#pragma unroll
                    for (int d = 4; d < 32; d *= 2)
                        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], d));
                    if (lane < 4)
                        s.red[64 * quarter + col] = top[i];
                }
                soft_sync();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int col = col0 + 8 * (i >> 1) + (i & 1);
                    const float most = fmaxf(fmaxf(s.red[col], s.red[64 + col]), fmaxf(s.red[128 + col], s.red[192 + col]));
                    const bool moves = (most - ref[i]) * f > kMostPower;         // the other rows keep theirs, and their bits
                    const float to = moves ? most : ref[i];
                    const float by = t == 0 ? 0.0f : moves ? ex2((ref[i] - to) * f) : 1.0f;
                    ref[i] = to;
                    sum[i] = t == 0 ? 0.0f : sum[i] * by;
                    even[i] = t == 0 ? 0.0f : even[i] * by;
                    if (quarter == 0 && lane < 4)
                        s.fac[col] = by;
                }
                soft_sync();
                if (t > 0) {
                    fence_after();
#pragma unroll 1
                    for (int i = 0; i < 2 * kPairs; ++i)
                        if (16 * (i & 1) < 8 * groups) {
                            float o[16];
                            const int c = 32 * half + 16 * (i & 1);
                            tmem_ld_32x16(o, lanes + 64 * (i >> 1) + c);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] *= s.fac[c + e];
                            tmem_st_32x16(lanes + 64 * (i >> 1) + c, o);
                        }
                }
                soft_sync();                                 // the factors lie where the weights go
            }
            if (tid == 0)
                mbar_arrive(s.p_ready + (tiles & 1));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < groups) {
                    add2(sum[2 * i], sum[2 * i + 1], of_sum[2 * i], of_sum[2 * i + 1]);
                    add2(even[2 * i], even[2 * i + 1], of_even[2 * i], of_even[2 * i + 1]);
                }
        }
        // the scores are all made: the next piece's queries may come, unless results are put together where they go
        const long long out_row = first_row();
        const int slot = slot_of();
        int rows = m.rows;
        if (!MOE_DBG_IN_RANGE(slot, 2 * kMaxAttnCtas, g.a.hdr) || !MOE_DBG_IN_RANGE(rows - 1, g.cap, g.a.hdr) ||
            !MOE_DBG_IN_RANGE(out_row, (long long)p.T * p.heads - rows + 1, g.a.hdr))
            rows = 0;
        more = advance();
        if (more && !whole)
            load_queries();
        wait(s.o_done, (tiles - 1) & 1);
        // sums of the columns: eight lanes, four warps, in this order; lanes that exchange keep one half of what they have each
        {
            float v[16];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = sum[i], v[8 + i] = even[i];
#pragma unroll
            for (int step = 0; step < 3; ++step)
#pragma unroll
                for (int i = 0; i < 8 >> step; ++i) {
                    const bool up = lane & (4 << step);
                    const float a = v[i], b = v[(8 >> step) + i];
                    v[i] = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 4 << step);
                }
            const int col = col0 + 8 * ((lane >> 2 & 2) + (lane >> 4));            // of sum, or of even
            *reinterpret_cast<float2 *>(s.red + 256 * (lane >> 2 & 1) + 64 * quarter + col) = make_float2(v[0], v[1]);
            if (quarter == 0 && lane < 4)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s.ref[col0 + 8 * (i >> 1) + (i & 1)] = ref[i];
        }
        soft_sync();
        if (tid < rows) {
            float l = (s.red[tid] + s.red[64 + tid]) + (s.red[128 + tid] + s.red[192 + tid]);
            const float by = (s.red[256 + tid] + s.red[320 + tid]) + (s.red[384 + tid] + s.red[448 + tid]);
            const bool out_of_range = whole && l == 0.0f && s.hi[tid] > 0;     // it sees positions, and every score left fp32 below
            if (out_of_range)
                l = __uint_as_float(0x7FFFFFFFu);
            s.sum[tid] = out_of_range ? l : l == 0.0f ? 0.0f : 1.0f / by;
            if (!whole)
                __stcg(g.part_sum + (size_t)slot * g.cap + tid, make_float4(l == 0.0f ? -INFINITY : s.ref[tid], l, by, 0.0f));
            else if (p.lse)
                p.lse[out_row + tid] = l == 0.0f ? -INFINITY : fmaf(s.ref[tid], p.scale, logf(l));
        }
        soft_sync();
        if (!whole) {
#pragma unroll 1
            for (int i = 0; i < 2 * kPairs; ++i) {
                const int c = 32 * half + 16 * (i & 1), n = rows - c;          // rows c .. c + 15 of dims 128 (i / 2) + lane
                if (n <= 0)
                    continue;
                float o[16];
                tmem_ld_32x16(o, lanes + 64 * (i >> 1) + c);
                float *to = g.part + ((size_t)slot * g.cap + c) * L + 128 * (i >> 1) + 32 * quarter + lane;
                if (n >= 16) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        __stcg(to + e * L, o[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 15; ++e)
                        if (e < n)
                            __stcg(to + e * L, o[e]);
                }
            }
        } else {
            // rows of out lie one after the other: they are put together where the queries were, and leave as one copy
#pragma unroll 1
            for (int i = 0; i < 2 * kPairs; ++i) {
                const int c = 32 * half + 16 * (i & 1), n = rows - c;
                if (n <= 0)
                    continue;
                float o[16];
                tmem_ld_32x16(o, lanes + 64 * (i >> 1) + c);
                const int odd = lane & 1;
                uint8_t *to = s.q + (size_t)(c + odd) * (2 * L) + 256 * (i >> 1) + 64 * quarter + 4 * (lane >> 1);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {            // lanes 2 i and 2 i + 1 exchange, so that each has two dims of a row
                    const float a = o[e] * s.sum[c + e], b = o[e + 1] * s.sum[c + e + 1];
                    const float other = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
                    if (e + odd < n)
                        *reinterpret_cast<uint32_t *>(to + e * (2 * L)) = odd ? bf16_pair(other, b) : bf16_pair(a, other);
                }
            }
            fence_async();
            stored = true;
        }
        fence_before();
        soft_sync();                                         // also: s.sum and s.ref have been read
        if (tid == 0) {
            mbar_arrive(s.o_free);
            if (whole && rows > 0)
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\ncp.async.bulk.commit_group;" ::"l"(p.out + out_row * L),
                             "r"(smem_u32(s.q)), "r"((uint32_t)rows * (2 * L))
                             : "memory");
        }
        if (whole && more) {
            if (tid == 0)
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            soft_sync();
            load_queries();
        }
    }
    if (stored && tid == 0)
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (tid == 0)
        g.joins[blockIdx.x] = join;
}

// The plan of up to 32 requests, by one warp (make_small_plan takes a microsecond longer).
template <int L>
__device__ __forceinline__ void few_requests_plan(const LatentArgs &g, const LatentSmem<L> &s) {
    const AttnProblem &p = g.a.p;
    const int lane = threadIdx.x & 31;
    int lo = 0, n = 0, kv = 0;
    bool bad = false;
    if (lane < p.B) {
        const int hi = p.q_offsets[lane + 1];
        lo = p.q_offsets[lane];
        kv = p.kv_lens[lane];
        n = hi - lo;
        bad = lo < 0 || hi < lo || hi > p.T || kv < 0 || kv > ((long long)p.max_blocks << g.a.shift);
    }
    bad = __any_sync(0xffffffffu, bad);
    const int count = bad ? 0 : (int)(((long long)n * g.a.group + g.a.rows - 1) / g.a.rows);
    int cost = 0;                                // small plans' work fits an int
    for (int i = 0; i < count; ++i)
        cost += row_tile(g.a, lane, lo, n, kv, i * g.a.rows).tiles + kUnitCost;
    int units = count, work = cost;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, units, d), w = __shfl_up_sync(0xffffffffu, work, d);
        if (lane >= d) {
            units += u;
            work += w;
        }
    }
    const int total = __shfl_sync(0xffffffffu, units, 31);
    const bool fits = total <= g.a.max_tiles;    // offsets within T leave no other choice
    int before = work - cost;
    for (int i = 0; i < count && fits; ++i) {
        s.before[units - count + i] = before;
        s.which[units - count + i] = (uint16_t)(lane | i << 8);
        before += row_tile(g.a, lane, lo, n, kv, i * g.a.rows).tiles + kUnitCost;
    }
    if (lane == 31) {
        if ((bad || !fits) && blockIdx.x == 0)
            record_status(g.a.hdr, MOE_ERR_DEVICE_ASSERT);
        *s.plan = bad || !fits ? Plan{0, 1, 0, 0} : plan_of(g.a, work, total);
    }
}

template <int L>
__global__ void __launch_bounds__(kThreads, 1) latent_kernel(const __grid_constant__ LatentArgs g, const __grid_constant__ CUtensorMap pair_map,
                                                             const __grid_constant__ CUtensorMap chunk_map) {
    extern __shared__ __align__(1024) uint8_t raw_smem[];
    const LatentSmem<L> s(raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023), g.q_rows, g.slots);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(s.pair_full + i, 1);
            mbar_init(s.pair_empty + i, 1);
        }
        for (int i = 0; i < kRopeSlots; ++i) {
            mbar_init(s.rope_full + i, 1);
            mbar_init(s.rope_empty + i, 1);
        }
        mbar_init(s.s_full, 1);
        mbar_init(s.s_full + 1, 1);
        mbar_init(s.p_ready, 1);
        mbar_init(s.p_ready + 1, 1);
        mbar_init(s.o_done, 1);
        mbar_init(s.o_free, 1);
        mbar_init(s.q_ready, 1);
        fence_barrier_init();
    }
    if (warp == kSoftWarps + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(s.taddr)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *s.taddr;
    pdl_wait();
    pdl_trigger();
    if (g.small && g.a.p.B <= 32) {              // a lane a request
        if (warp == 0)
            few_requests_plan<L>(g, s);
    } else if (g.small) {                        // the plan, made where the cache's tiles go and kept in few words
        RowTile *recs = reinterpret_cast<RowTile *>(s.ring + 1024);
        make_small_plan(g.a, reinterpret_cast<long long *>(s.ring), recs, s.plan, blockIdx.x == 0);
        for (int i = threadIdx.x; i < s.plan->row_tiles; i += kThreads) {
            s.before[i] = (int)recs[i].before;
            s.which[i] = (uint16_t)(recs[i].request | recs[i].row0 / g.a.rows << 8);
        }
        fence_async();
    } else if (threadIdx.x == 0) {
        *s.plan = *g.a.plan;
    }
    __syncthreads();
    if (warp < kSoftWarps)
        latent_softmax<L>(g, s, tmem);
    else if (warp == kSoftWarps)
        latent_stream<L>(g, s, &pair_map, &chunk_map);
    else if (warp == kSoftWarps + 1)
        latent_scores<L>(g, s, tmem);
    else
        latent_values<L>(g, s, tmem);
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kSoftWarps + 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

__global__ void __launch_bounds__(kPlanThreads) latent_plan_kernel(AttnArgs a) {
    extern __shared__ int s_first[];
    __shared__ long long red[32];
    pdl_wait();
    pdl_trigger();
    make_plan(a, s_first, red, a.recs, a.plan, true);
}

// The parts of cut units, in the order of the cache.  A warp takes a row by itself (with a row to a CTA and barriers 9,600 rows of two or
// three parts each took 40 us); where there are fewer, 128 dims of a row, or two, four or eight warps of a CTA take those and share
// the parts (64 rows of 152 parts: 26 us by single warps, 10).
constexpr int kJoinWarps = 8;
template <int L>
__global__ void __launch_bounds__(kJoinWarps * 32, 4) latent_join_kernel(const LatentArgs g, int ctas) {
    constexpr int kCols = L / 128, U = 4, kPer = kMaxAttnCtas / 32;
    __shared__ LatentJoin s_join[kMaxAttnCtas];
    __shared__ int s_end[kMaxAttnCtas];          // rows to join of the CTAs up to this one
    __shared__ float s_w[kJoinWarps][kMaxAttnCtas];
    __shared__ float4 s_o[kJoinWarps][32];
    static_assert(kMaxAttnCtas % 32 == 0 && kMaxAttnCtas <= kJoinWarps * 32, "a thread a CTA");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();                               // the kernel after may be scheduled while this one waits: it waits for this one's end
    pdl_wait();
    LatentJoin mine{0, 0, 0, 0, 0};
    if (tid < ctas)
        mine = g.joins[tid];
    if (tid < kMaxAttnCtas)
        s_join[tid] = mine;
    if (!__syncthreads_or(mine.rows))
        return;
    if (warp == 0) {                             // the sums of rows
        int n[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            sum += n[i] = s_join[kPer * lane + i].rows;
        int ahead = sum;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, ahead, d);
            ahead += lane >= d ? v : 0;
        }
        ahead -= sum;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            s_end[kPer * lane + i] = ahead += n[i];
    }
    __syncthreads();
    const int rows = s_end[kMaxAttnCtas - 1];
    LatentJoin j{0, 0, 0, 0, 0};
    int r = 0, part = 0, parts = 0;
    float m = 0.0f, l = 0.0f, even = 0.0f;       // the row's reference, its sums as in latent_softmax
    auto slot = [&](int k) { return (size_t)(((j.first + k) * 2 + (k == 0)) * g.split + part) * g.cap + r; };
    // row i: where it is, its reference and sum, the weights of its parts; false where the range-checked build finds it out of range
    auto find = [&](int i) -> bool {
        int c = 0;                               // whose row it is: CTAs with no more rows up to them
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            c += __popc(__ballot_sync(0xffffffffu, s_end[32 * k + lane] <= i));
        if (!MOE_DBG_IN_RANGE(c, ctas, g.a.hdr))
            return false;
        j = s_join[c];
        r = i - (c ? s_end[c - 1] : 0);
        part = g.split == 1 ? 0 : c & 1;
        parts = j.last - j.first + 1;
        if (!MOE_DBG_IN_RANGE(r, g.cap, g.a.hdr) || !MOE_DBG_IN_RANGE(parts - 1, kMaxAttnCtas, g.a.hdr) ||
            !MOE_DBG_IN_RANGE(j.row + r, (long long)g.p.T * g.p.heads, g.a.hdr))
            return false;
        float4 e[kPer];
        m = -INFINITY;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const int k = 32 * q + lane;
            e[q] = 32 * q < parts && k < parts ? __ldcg(g.part_sum + slot(k)) : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
            m = fmaxf(m, e[q].x);
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        l = even = 0.0f;
        __syncwarp();
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const float w = ex2((e[q].x - m) * g.factor);
            s_w[warp][32 * q + lane] = e[q].y == 0.0f ? -1.0f : w;             // below zero: it saw nothing, and its sums were not written
            l += e[q].y == 0.0f ? 0.0f : e[q].y * w;
            even += e[q].y == 0.0f ? 0.0f : e[q].z * w;
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2) {
            l += __shfl_xor_sync(0xffffffffu, l, d);
            even += __shfl_xor_sync(0xffffffffu, even, d);
        }
        if (l == 0.0f && r >= j.blind)           // it sees positions, and every score left fp32 below
            l = even = __uint_as_float(0x7FFFFFFFu);
        __syncwarp();
        return true;
    };
    // four dims of parts first, + stride, ...
    auto add = [&](int d, int first, int stride) {
        float4 o = make_float4(0, 0, 0, 0);
        for (int k0 = first; k0 < parts; k0 += U * stride) {
            float4 v[U];
            float w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * stride;
                const bool in = k < parts && !(s_w[warp][k] < 0.0f);
                w[u] = in ? s_w[warp][k] : 0.0f;
                v[u] = in ? __ldcg(reinterpret_cast<const float4 *>(g.part + slot(k) * L) + d) : make_float4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                o.x = fmaf(v[u].x, w[u], o.x);
                o.y = fmaf(v[u].y, w[u], o.y);
                o.z = fmaf(v[u].z, w[u], o.z);
                o.w = fmaf(v[u].w, w[u], o.w);
            }
        }
        return o;
    };
    auto write = [&](int d, float4 o) {
        const float by = l == 0.0f ? 0.0f : 1.0f / even;
        reinterpret_cast<uint2 *>(g.p.out + (j.row + r) * L)[d] = make_uint2(bf16_pair(o.x * by, o.y * by), bf16_pair(o.z * by, o.w * by));
        if (d == 0 && g.p.lse)
            g.p.lse[j.row + r] = l == 0.0f ? -INFINITY : fmaf(m, g.p.scale, logf(l));
    };
    const int jobs = rows * kCols;
    int share = 1;                               // warps of a job of 128 dims; then a CTA has 8 / share of them, once
    while (share < kJoinWarps && jobs <= (int)gridDim.x * kJoinWarps / (2 * share))
        share *= 2;
    if (share == 1) {                            // a row a warp, or 128 dims where that leaves warps without
        const int cols = 2 * rows >= (int)gridDim.x * kJoinWarps ? kCols : 1;
        for (int i = blockIdx.x * kJoinWarps + warp; i < jobs / cols; i += gridDim.x * kJoinWarps)
            if (find(i * cols / kCols))
                for (int col = i * cols % kCols, k = 0; k < cols; ++k, ++col)
                    write(col * 32 + lane, add(col * 32 + lane, 0, 1));
        return;
    }
    const int job = blockIdx.x * (kJoinWarps / share) + warp / share, d = job % kCols * 32 + lane;
    const bool mine_here = job < jobs && find(job / kCols);
    if (mine_here)
        s_o[warp][lane] = add(d, warp % share, share);
    __syncthreads();
    if (mine_here && warp % share == 0) {
        float4 o = s_o[warp][lane];
        for (int w = 1; w < share; ++w) {
            const float4 v = s_o[warp + w][lane];
            o.x += v.x;
            o.y += v.y;
            o.z += v.z;
            o.w += v.w;
        }
        write(d, o);
    }
}

// How rows become units.  Requests of single tokens (T <= B, so that no more is known but that) of more than 64 heads: two CTAs share units
// of up to 128 rows, the heads cut evenly, so that the cache is read from memory once (48 ragged requests of 96 heads 106 us, and 115 with a
// unit a CTA; 64 of 128 heads 236 and 263).  Otherwise units of 64 rows, a CTA each: what several tokens of a request read again comes from L2
// as often as not, and no CTA waits for rows that its unit lacks (16 requests of 1..4 tokens of 32 heads 76 us, and 91 with two CTAs a unit; one
// of 400 tokens of 64 heads 169 and 181).
struct Shape {
    int split, rows, q_rows, cap;
    Shape(int T, int B, int heads) {
        const long long all = (long long)T * heads;
        split = T <= B && heads > kMaxRows ? 2 : 1;
        const int most = split * kMaxRows, units = T <= B ? (heads + most - 1) / most : 1;
        rows = T <= B ? (heads + units - 1) / units : kMaxRows;
        q_rows = split == 1 ? rows : (rows + 1) / 2;
        if (q_rows > all)
            q_rows = (int)all;
        q_rows = (q_rows + 15) / 16 * 16;
        cap = q_rows;
    }
};

// Most units of any lengths: a request with n tokens has ceil(n heads / rows), no more than n ceil(heads / rows).
int max_units(int T, int B, const Shape &s, int heads) {
    const long long a = (long long)T * ((heads + s.rows - 1) / s.rows), b = ((long long)T * heads + (long long)(T < B ? T : B) * (s.rows - 1)) / s.rows;
    return (int)(a < b ? a : b);
}

struct LatentLayout {
    size_t plan, recs, joins, part, part_sum, total;
    LatentLayout(int units, int cap, int L) {
        size_t o = kInitBytes;
        auto take = [&](size_t bytes) { o = align_up(o, 256); size_t r = o; o += bytes; return r; };
        plan = take(sizeof(Plan));
        recs = take((size_t)units * sizeof(RowTile));
        joins = take(kMaxAttnCtas * sizeof(LatentJoin));
        part = take((size_t)2 * kMaxAttnCtas * cap * L * sizeof(float));         // a CTA has parts of at most two units
        part_sum = take((size_t)2 * kMaxAttnCtas * cap * sizeof(float4));
        total = align_up(o, 256);
    }
    LatentLayout(int T, int B, const Shape &s, int heads, int L) : LatentLayout(max_units(T, B, s, heads), s.cap, L) {}
};

template <int L>
cudaError_t launch(const LatentProblem &p, void *ws, int sms, cudaStream_t stream) {
    const Shape shape(p.T, p.B, p.heads);
    const LatentLayout lay(p.T, p.B, shape, p.heads, L);
    int shift = 4;
    while ((1 << shift) < p.cache.block_size)
        ++shift;
    LatentArgs g{};
    AttnProblem &ap = g.a.p;                                 // what the plan looks at
    ap.T = p.T;
    ap.q_heads = p.heads;
    ap.cache.num_blocks = p.cache.num_blocks;
    ap.cache.kv_heads = 1;
    ap.cache.block_size = p.cache.block_size;
    ap.table = p.table;
    ap.max_blocks = p.max_blocks;
    ap.q_offsets = p.q_offsets;
    ap.kv_lens = p.kv_lens;
    ap.B = p.B;
    ap.causal = p.causal;
    const int ctas = (sms < kMaxAttnCtas ? sms : kMaxAttnCtas) / shape.split * shape.split;
    g.a.group = p.heads;
    g.a.shift = shift;
    g.a.rows = shape.rows;
    g.a.ctas = ctas / shape.split;
    g.a.max_tiles = max_units(p.T, p.B, shape, p.heads);
    g.a.plan = ws_at<Plan>(ws, lay.plan);
    g.a.recs = ws_at<RowTile>(ws, lay.recs);
    g.a.hdr = ws_at<uint32_t>(ws, 0);
    g.p = p;
    g.split = shape.split;
    g.small = g.a.max_tiles <= kSmallUnits && p.B <= kSmallRequests && (long long)p.max_blocks * p.cache.block_size <= kSmallTokens;
    g.q_rows = shape.q_rows;
    g.slots = LatentSmem<L>::slots_for(shape.q_rows);
    g.cap = shape.cap;
    const double factor = (double)p.scale * 1.44269504088896340736;
    g.factor = factor < 3.4e38 ? (float)factor : 3.4e38f;
    g.joins = ws_at<LatentJoin>(ws, lay.joins);
    g.part = ws_at<float>(ws, lay.part);
    g.part_sum = ws_at<float4>(ws, lay.part_sum);
    // the cache as [chunk of 64 dims][slot][64 dims]
    const uint64_t dims[3] = {64, (uint64_t)p.cache.num_blocks * p.cache.block_size, L / 64 + 1}, strides[2] = {(L + kRopeDims) * 2, 128};
    uint32_t box[3] = {64, (uint32_t)(p.cache.block_size < kTile ? p.cache.block_size : kTile), 1};
    CUtensorMap chunk_map, pair_map;
    cudaError_t e = encode_tiled(&chunk_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.cache.data, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    box[2] = 2;
    if (e == cudaSuccess)
        e = encode_tiled(&pair_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.cache.data, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    const size_t smem = LatentSmem<L>::bytes(g.q_rows, g.slots);
    if (e == cudaSuccess)                                    // a limit of the whole process: the same one from every thread's call
        e = cudaFuncSetAttribute(latent_kernel<L>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess && !g.small)
        e = launch_pdl(latent_plan_kernel, dim3(1), dim3(kPlanThreads), p.B * sizeof(int), stream, g.a);
    if (e == cudaSuccess)
        e = launch_pdl(latent_kernel<L>, dim3(ctas), dim3(kThreads), smem, stream, g, pair_map, chunk_map);
    return e != cudaSuccess ? e : launch_pdl(latent_join_kernel<L>, dim3(4 * ctas), dim3(kJoinWarps * 32), 0, stream, g, ctas);
}

}  // namespace

size_t latent_attention_need(int T, int B, int heads, int latent_dim) {
    return T == 0 || B == 0 ? align_up(kInitBytes, 256) : LatentLayout(T, B, Shape(T, B, heads), heads, latent_dim).total;
}

// Of any step of up to T tokens of up to B requests.  Steps have units of the one shape or the other as they have more tokens than requests
// or not, and those of a smaller step may be the larger (10 tokens of 4 requests, 16 heads: parts of 64 rows; 64 tokens of 64: 16).  Either
// shape's units and parts grow with T and with B.
size_t latent_attention_workspace(int T, int B, int heads, int latent_dim) {
    if (T == 0 || B == 0)
        return align_up(kInitBytes, 256);
    const int t = T < B ? T : B;                  // most tokens of a step of no more tokens than requests
    const Shape one(t, B, heads);
    int units = max_units(t, B, one, heads), cap = one.cap;
    if (T > 1) {                                  // and a step of more has T - 1 requests at most
        const int b = B < T - 1 ? B : T - 1;
        const Shape more(T, b, heads);
        const int n = max_units(T, b, more, heads);
        units = units > n ? units : n;
        cap = cap > more.cap ? cap : more.cap;
    }
    return LatentLayout(units, cap, latent_dim).total;
}

cudaError_t launch_latent_attention(const LatentProblem &p, void *ws, int sms, cudaStream_t stream) {
    return p.cache.latent_dim == 256 ? launch<256>(p, ws, sms, stream) : launch<512>(p, ws, sms, stream);
}

}  // namespace moe
