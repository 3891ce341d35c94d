// attn_tc.cu -- the attention of attn.cu for many rows to a key/value head
// (prompt chunks, verification of several drafted tokens): both products on
// tcgen05, scores, weights and sums in tensor memory.  Formulas, numbers, units
// and ranges are those of attn.cu.
//
// Why another form.  With more than 16 rows a warp's mma.sync products, the conversion of the
// codes that every warp of a tile repeats and the softmax share the same issue slots: 64 rows ran
// at 29 % of the mma.sync rate.  Here the codes are converted once for up to 256 rows, and the products cost no issue slots.
//
// A unit has up to 256 rows.  Two "halves" each own 128 TMEM lanes = rows: with more than 128 rows
// the halves take rows 0..127 and 128..255 of every tile; with up to 128 they take the same
// rows and every other tile, and their sums are joined like those of two CTAs.  Half h: S_h = Q_h K^T
// (M = 128 rows, N = 128 tokens) in TMEM columns 128 h.., the f16 weights W_h, O_h += W_h V (A in TMEM, N = head
// dim) in columns 256 + D h...  At D = 64 the weights have columns of their own and the next scores are issued before the
// product that they wait for; at D = 128 they lie over the scores just read.  One half's softmax runs
// beside the other half's products.
//
// Warps: 0..7 softmax (warp % 4 = TMEM lane quarter, warp / 4 the half; a thread has a row), 8..13 convert, 14 streams the cache,
// 15 issues the MMAs.  (Two threads to a row, 16 warps of at most 88 registers, took as long: more latency hidden, more moves
// and exchanges.)
//
// Measured: three requests' chunks of 500 tokens over 9,000, 48 query heads of 64, 151 us (548 TFLOP/s): nine instructions a score, all roles together,
// in half of the issue slots (a pass for the maxima before the weights: 165; four such tiles unrolled: 180); the special-function pipe is
// busy a quarter of the time, the tensor pipe too.  Chunks of up to 600 over up to 16,000, 40 heads of 128, 341 us (857 TFLOP/s),
// where shared memory, read and written for codes, operands and products, is busy three quarters of the time; 16 requests of up to 48 rows
// over 10,000 tokens 145 us, bound by a tile's way through conversion, product, softmax and product with few rows.
//
// The operands pass in the order K0, K1, V0, K2, V1, ...: as codes into a ring of raw tiles
// by bulk copies, then as f16 into a ring of operand tiles, rows (tokens of K, dims of V) of 64
// elements in the 128-byte swizzle.  The cache's innermost 16 bytes run along the summed axis for both, so the two
// conversions are the same code.
//
// The running maxima of a row are references that move only where scores have outgrown them (16 weights sum to more than
// f16 holds; its rounding is relative).  A largest weight is 2^6 when they have moved, so that 20 binades below it keep their bits
// (2^8, with less room to grow, takes 161 us for 152 on the first case above; 2^0 to 2^6 the same).  So a score is read once: 32 of a row at a time become weights,
// whose sums say whether they fit.  Where they do not, the references move to the maxima (of the tile, or of the 32 where the
// weights lie over the scores), the half waits for its last product and rescales O, and the tile's weights so far, in TMEM; then
// the weights are made, and not looked at again.  Only a unit's first tile is read for its maxima first.
//
// The reference of the weights is kept relative to that of l (rel = M - m) and moves by whole powers of two: weights stored already
// lose nothing to it but what falls below f16, and it has all its bits however large the scores are.  A weight's power is fma(y, fi, -m), the
// product exact; m, rounded, may lie under it by half of its last place.  Past kFar that would matter (half a place of 2^28 is a
// factor of 2^16).  There, and wherever the references have just moved, the product is rounded as m was before m is
// taken from it, so that no power is above zero, and every tile is read for its maxima first.
#include "attn_plan.cuh"

namespace moe {
namespace {

constexpr int kSoftWarps = 8, kConvWarps = 6;
constexpr int kTcThreads = (kSoftWarps + kConvWarps + 2) * 32;
constexpr int kNanEntries = 2048;
// What 16 weights may sum to before the references move: f16's largest number; 2^-32: with that factor, what 16 terms of l may.  The
// power of a largest weight when they have: 16 of them sum to 2^10, the rest is room to grow.
constexpr float kMostWeight = 65504.0f, kLeastSum = 0x1p-32f, kLift = 6.0f;

// A value's NaN codes in a tile that some rows see in part: the unit, the position, the dims.  A CTA's list of them is
// never written over: past its end values are only counted (and found in the cache, nan_rows).  A unit's are in it before its
// last product ends; those of the next unit may be on their way then, so that an entry counts from its mark on.
struct NanEntry {
    int unit, token;
    uint32_t dims[4];
    int pad[2];
};
static_assert(sizeof(NanEntry) * kNanEntries == kAttnNanBytes, "list");

template <int D>
struct TcSmem {
    static constexpr int kRawBytes = kTile * D;              // one operand's codes
    static constexpr int kOpBytes = 2 * kTile * D;           // in f16
    static constexpr int kRaw = D == 128 ? 4 : 8, kOps = D == 128 ? 3 : 4;
    static constexpr int kQBytes = 128 * D * 2;              // of a half
    // tiles whose exponents are kept: the stream is at most (kRaw + kOps + 1) / 2 + 1 ahead of the softmax
    static constexpr int kMetaTiles = D == 128 ? 8 : 16;
    static constexpr size_t kOffOps = 2 * kQBytes;
    static constexpr size_t kOffRaw = kOffOps + (size_t)kOps * kOpBytes;
    static constexpr size_t kOffMeta = kOffRaw + (size_t)kRaw * kRawBytes;     // float [tile][2][kSubs]
    static constexpr size_t kOffBars = kOffMeta + kMetaTiles * 2 * kSubs * 4;
    static constexpr bool kOwnW = D == 64;                   // weights in columns of their own
    __host__ __device__ static constexpr int w_col(int h, int tok) { return kOwnW ? 384 + 64 * h + tok / 2 : 128 * h + (tok >= 64 ? 64 : 0) + (tok % 64) / 2; }
    static constexpr int kBarCount = 2 * kRaw + 2 * kOps + 8 + 1;
    static constexpr size_t kOffMarks = kOffBars + kBarCount * 8 + 32;         // a bit for each entry of the list of NaN values
    static constexpr size_t kBytes = kOffMarks + kNanEntries / 8 + 1024;       // + alignment to 1024
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

// 64-element f16 rows in 128-byte-swizzled atoms of 8.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// fp32 D, f16 A and B, K-major, M = 128.
__host__ __device__ constexpr uint32_t f16_idesc(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24); }

// Issued by one elected lane of a converged warp.
template <int N>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p, q;\nelect.sync _|p, 0xffffffff;\nsetp.ne.b32 q, %4, 0;\n"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "n"(f16_idesc(N)), "r"(acc)
        : "memory");
}

template <int N>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p, q;\nelect.sync _|p, 0xffffffff;\nsetp.ne.b32 q, %4, 0;\n"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "n"(f16_idesc(N)), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile(
        "{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\n"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
        : "memory");
}

// The load and its wait are one statement: nothing that uses v can come between.
__device__ __forceinline__ void tmem_ld32(float (&v)[32], uint32_t addr) {
    uint32_t *u = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
        "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]), "=r"(u[9]),
          "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]),
          "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]),
          "=r"(u[30]), "=r"(u[31])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(float (&v)[16], uint32_t addr) {
    uint32_t *u = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]), "=r"(u[9]),
          "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(addr)
        : "memory");
}

// Two fp32 values in one instruction each.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const float (&v)[32]) {
    const uint32_t *u = reinterpret_cast<const uint32_t *>(v);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
        "%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]),
        "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]), "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]),
        "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]), "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&u)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr), "r"(u[0]),
                 "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]),
                 "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
                 : "memory");
}

// A piece as the halves see it: pair = the halves have rows of their own.
__device__ __forceinline__ int half_tiles(const Piece &pc, bool pair, int h) {
    const int n = pc.t1 - pc.t0;
    return pair ? n : (n + 1 - h) / 2;
}

// Operands of a piece of n tiles in their order: K0, K1, V0, K2, V1, ... V(n-1).
__device__ __forceinline__ int k_order(int t) { return t == 0 ? 0 : 2 * t - 1; }
__device__ __forceinline__ int v_order(int t, int n) { return t < n - 1 ? 2 * t + 2 : 2 * n - 1; }

struct Bars {
    uint64_t *raw_full, *raw_empty, *op_full, *op_empty, *s_full, *w_ready, *o_done, *q_ready, *spare;
};

// ------------------------------------------------------------ the cache's tiles

template <int D>
__device__ __forceinline__ void tc_stream(const AttnArgs &a, const Plan &pl, uint8_t *sm, const Bars &b) {
    using S = TcSmem<D>;
    const AttnProblem &p = a.p;
    const int lane = threadIdx.x & 31, sub = lane & (kSubs - 1);
    Walk walk(a, pl, a.recs);
    Piece pc;
    uint32_t op = 0, tile = 0;             // operands and tiles so far
    bool dead = false;
    while (walk.next(pc)) {
        const int n = pc.t1 - pc.t0;
        const int hi = p.causal ? min(pc.kv, pc.kv - pc.n + (pc.row0 + pc.rows - 1) / a.group + 1) : pc.kv;
        int lo, unused;                    // the first row sees furthest back: blocks before may be gone from the table
        row_range(p, a.group, pc.kv, pc.n, pc.row0, lo, unused);
        const int32_t *row = p.table + (size_t)pc.request * p.max_blocks;
        // a batch of four tiles' blocks and scales at a time, a lane for each sub-block; the next batch's on their way
        int page, ks, vs;
        auto fetch = [&](int t0, int &pg) {
            const long long tok = (long long)(pc.tile0 + pc.t0 + t0) * kTile + lane * 16;
            pg = t0 < n && tok < hi && tok + 16 > lo && t0 + lane / kSubs < n ? __ldg(row + (tok >> a.shift)) : -1;
        };
        int next;
        fetch(0, next);
        int vpage = 0;                     // the batch before: a tile's values come after the next tile's keys
        uint32_t vlive = 0;
        for (int t0 = 0; t0 < n; t0 += 4) {
            page = next;
            fetch(t0 + 4, next);
            const long long tok = (long long)(pc.tile0 + pc.t0 + t0) * kTile + lane * 16;
            const bool live = t0 + lane / kSubs < n && tok < hi && tok + 16 > lo;
            if (live && (page < 0 || page >= p.cache.num_blocks)) {
                record_status(a.hdr, MOE_ERR_DEVICE_ASSERT);
                page = 0;
            }
            const size_t unit = (size_t)(live ? page : 0) * p.cache.kv_heads + pc.head;
            ks = live ? __ldg(p.cache.k_scale + unit) : 127;
            vs = live ? __ldg(p.cache.v_scale + unit) : 127;
            const uint32_t mask = __ballot_sync(0xffffffffu, live);
            for (int i = 0; i < 4 && t0 + i < n; ++i) {
                const int t = t0 + i;
                // the order is K(t), V(t-1), then V of the last tile
                for (int step = 0; step < (t == n - 1 ? 3 : 2); ++step) {
                    const bool is_v = step > 0;
                    const int vt = step == 1 ? t - 1 : t;          // tile of the values
                    if (is_v && vt < 0)
                        continue;
                    // values of tile t - 1 may belong to the batch before: its lanes' blocks were kept
                    const bool old = is_v && vt < t0;
                    const int pg = old ? vpage : page;
                    const uint32_t lv = old ? vlive : mask;
                    const int at = is_v ? (vt & 3) : i;             // place in its batch
                    const int st = (int)(op % S::kRaw);
                    if (!dead && op >= S::kRaw)
                        dead = !__all_sync(0xffffffffu, wait_phase(b.raw_empty + st, (op / S::kRaw - 1) & 1));
                    if (dead) {
                        if (lane == 0)
                            record_status(a.hdr, MOE_ERR_DEVICE_TIMEOUT);
                        ++op;
                        continue;
                    }
                    const bool mine = lane / kSubs == at;
                    if (!is_v && mine) {
                        float *m = reinterpret_cast<float *>(sm + S::kOffMeta) + ((tile + t) % S::kMetaTiles) * 2 * kSubs + sub;
                        m[0] = exp2i(min(max(ks, 1), 254) - 127);
                        m[kSubs] = (float)(vs - 127);
                    }
                    __syncwarp();
                    const uint32_t here = (lv >> (at * kSubs)) & ((1u << kSubs) - 1);
                    if (lane == 0)
                        mbar_arrive_expect_tx(b.raw_full + st, S::kRawBytes / kSubs * __popc(here));
                    __syncwarp();
                    const long long tk = (long long)(pc.tile0 + pc.t0 + (is_v ? vt : t)) * kTile + sub * 16;
                    const int in_block = (int)(tk & ((1 << a.shift) - 1)) >> 4, block_subs = 1 << (a.shift - 4);
                    if (mine && (here >> sub & 1) && (sub == __ffs(here) - 1 || in_block == 0)) {    // one run of sub-blocks
                        const uint32_t bytes = (uint32_t)min(block_subs - in_block, 32 - __clz(here) - sub) * (16 * D);
                        const size_t src = ((((size_t)pg * p.cache.kv_heads + pc.head) << a.shift) + in_block * 16) * D;
                        asm volatile(
                            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                smem_u32(sm + S::kOffRaw + (size_t)st * S::kRawBytes + sub * 16 * D)),
                            "l"((is_v ? p.cache.v : p.cache.k) + src), "r"(bytes), "r"(smem_u32(b.raw_full + st))
                            : "memory");
                    }
                    ++op;
                }
            }
            vpage = live ? page : 0;
            vlive = mask;
        }
        tile += n;
    }
    for (uint32_t i = op > S::kRaw ? op - S::kRaw : 0; i < op && !dead; ++i)
        wait_phase(b.raw_full + i % S::kRaw, (i / S::kRaw) & 1);
}

// ---------------------------------------------------------- codes to f16

template <int D>
__device__ __forceinline__ void tc_convert(const AttnArgs &a, const Plan &pl, uint8_t *sm, const Bars &b, uint32_t *nan_count) {
    using S = TcSmem<D>;
    const int tid = threadIdx.x - kSoftWarps * 32, lane = tid & 31;
    NanEntry *nans = reinterpret_cast<NanEntry *>(static_cast<uint8_t *>(a.nans) + (size_t)blockIdx.x * kAttnNanBytes);
    uint32_t *marks = reinterpret_cast<uint32_t *>(sm + S::kOffMarks);
    Walk walk(a, pl, a.recs);
    Piece pc;
    uint32_t op = 0;
    bool dead = false;
    for (int unit = 0; walk.next(pc); ++unit) {
        const int n = pc.t1 - pc.t0;
        int lo0, hi0, lo1, hi1;
        row_range(a.p, a.group, pc.kv, pc.n, pc.row0, lo0, hi0);
        row_range(a.p, a.group, pc.kv, pc.n, pc.row0 + pc.rows - 1, lo1, hi1);
        // the order K0, K1, V0, ...: operand j
        for (int j = 0; j < 2 * n; ++j, ++op) {
            const bool is_v = j > 0 && ((j & 1) == 0 || j == 2 * n - 1);
            const int t = !is_v ? (j + 1) / 2 : j == 2 * n - 1 ? n - 1 : j / 2 - 1;
            const int tok0 = (pc.tile0 + pc.t0 + t) * kTile;
            const int rs = (int)(op % S::kRaw), os = (int)(op % S::kOps);
            if (!dead) {
                dead = !__all_sync(0xffffffffu, wait_phase(b.raw_full + rs, (op / S::kRaw) & 1));
                if (!dead && op >= S::kOps)
                    dead = !__all_sync(0xffffffffu, wait_phase(b.op_empty + os, (op / S::kOps - 1) & 1));
                if (dead && lane == 0)
                    record_status(a.hdr, MOE_ERR_DEVICE_TIMEOUT);
            }
            const uint4 *raw = reinterpret_cast<const uint4 *>(sm + S::kOffRaw + (size_t)rs * S::kRawBytes);
            uint8_t *out = sm + S::kOffOps + (size_t)os * S::kOpBytes;
            // rows see this tile in part: values that no row may meet, or not every row, are taken out
            const bool edge = is_v && (tok0 + kTile > hi0 || tok0 < lo1);
            // 16 codes of a row: keys [sub][chunk of dims][token], values [sub][dim]; the row's chunk is 32 bytes of f16
            auto place = [&](int u, int &row, int &chunk) {
                row = is_v ? u % D : u / D * 16 + u % 16;
                chunk = is_v ? u / D : u % D / 16;
            };
            const int atom = (is_v ? D : kTile) * 128;
            auto store = [&](const uint4 &c, int row, int chunk) {
                const uint32_t w[4] = {c.x, c.y, c.z, c.w};
                uint32_t h[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    h[2 * q] = e4m3x2_to_f16x2((uint16_t)w[q]);
                    h[2 * q + 1] = e4m3x2_to_f16x2((uint16_t)(w[q] >> 16));
                }
                uint8_t *at = out + (chunk >> 2) * atom + row * 128;
                const int c0 = (chunk & 3) * 2, x = row & 7;
                *reinterpret_cast<uint4 *>(at + ((c0 ^ x) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4 *>(at + (((c0 + 1) ^ x) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
            };
            constexpr int kUnits = kTile * D / 16, kStep = kConvWarps * 32;
            if (!edge) {
#pragma unroll 1
                for (int u0 = tid; u0 < kUnits; u0 += 3 * kStep) {
                    uint4 c[3];
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        if (u0 + i * kStep < kUnits)
                            c[i] = raw[u0 + i * kStep];
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        if (u0 + i * kStep < kUnits) {
                            int row, chunk;
                            place(u0 + i * kStep, row, chunk);
                            store(c[i], row, chunk);
                        }
                }
            } else {
#pragma unroll 1
                for (int u = tid; u < kUnits; u += kStep) {
                    uint4 c = raw[u];
                    uint32_t *w = reinterpret_cast<uint32_t *>(&c);
                    int row, chunk;
                    place(u, row, chunk);
                    const int left = hi1 - (tok0 + chunk * 16), skip = lo0 - (tok0 + chunk * 16);    // some row sees tokens skip .. left - 1 of the chunk
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int k = left - 4 * q;
                        if (k < 4)
                            w[q] &= k <= 0 ? 0u : (1u << (8 * k)) - 1;
                        if (skip > 4 * q)
                            w[q] &= skip >= 4 * q + 4 ? 0u : 0xFFFFFFFFu << (8 * (skip - 4 * q));
                        uint32_t nan = __vcmpeq4(w[q] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                        w[q] &= ~nan;
#pragma unroll 1
                        while (nan) {
                            const int e = (__ffs(nan) - 1) >> 3;
                            nan &= ~(0xFFu << (8 * e));
                            if (*reinterpret_cast<volatile uint32_t *>(nan_count) > kNanEntries)
                                continue;                    // counted far enough
                            const uint32_t at = atomicAdd(nan_count, 1u);
                            if (at >= kNanEntries)
                                continue;
                            NanEntry x{unit, tok0 + chunk * 16 + 4 * q + e, {0, 0, 0, 0}, {0, 0}};
                            x.dims[row >> 5] = 1u << (row & 31);
                            nans[at] = x;
                            __threadfence();
                            atomicOr(marks + at / 32, 1u << (at & 31));
                        }
                    }
                    store(c, row, chunk);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(b.raw_empty + rs);
                mbar_arrive(b.op_full + os);
            }
        }
    }
}

// --------------------------------------------------------------------- MMAs

template <int D>
__device__ __forceinline__ void tc_issue(const AttnArgs &a, const Plan &pl, uint8_t *sm, const Bars &b, uint32_t tmem) {
    using S = TcSmem<D>;
    const int lane = threadIdx.x & 31;
    Walk walk(a, pl, a.recs);
    Piece pc;
    uint32_t op = 0, units = 0, wn[2] = {0, 0}, qn[2] = {0, 0};    // operands before the piece; weights, queries waited for
    bool dead = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!dead) {
            dead = !__all_sync(0xffffffffu, wait_phase(bar, parity));
            if (dead && lane == 0)
                record_status(a.hdr, MOE_ERR_DEVICE_TIMEOUT);
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    };
    auto operand = [&](uint32_t o) { return smem_u32(sm + S::kOffOps + (size_t)(o % S::kOps) * S::kOpBytes); };
    auto scores = [&](int h, uint32_t o) {
        const uint64_t dq = desc_sw128(smem_u32(sm + (size_t)h * S::kQBytes)), dk = desc_sw128(operand(o));
        if (!dead) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j)           // atoms of 64 dims: 128 rows x 128 bytes
                mma_ss<128>(tmem + 128 * h, dq + (j >> 2) * 1024 + (j & 3) * 2, dk + (j >> 2) * 1024 + (j & 3) * 2, j > 0);
        }
        commit(b.s_full + h);
    };
    auto values = [&](int h, uint32_t o, bool first) {
        const uint64_t dv = desc_sw128(operand(o));
        if (!dead) {
#pragma unroll
            for (int j = 0; j < kTile / 16; ++j)       // atoms of 64 tokens: D rows x 128 bytes
                mma_ts<D>(tmem + 256 + D * h, tmem + S::w_col(h, 16 * j), dv + (j >> 2) * (D * 8) + (j & 3) * 2, !first || j > 0);
        }
        commit(b.o_done + h);
    };
    for (; walk.next(pc); ++units) {
        const int n = pc.t1 - pc.t0;
        const bool pair = pc.rows > 128;
        if (n == 0)
            continue;
        auto acquire = [&](uint32_t o) { wait(b.op_full + o % S::kOps, (o / S::kOps) & 1); };
        auto queries = [&](int h) {
            wait(b.q_ready + h, qn[h] & 1);
            ++qn[h];
        };
        auto weights = [&](int h) {
            wait(b.w_ready + h, wn[h] & 1);
            ++wn[h];
        };
        acquire(op + k_order(0));
        queries(0);
        scores(0, op + k_order(0));
        if (pair) {
            queries(1);
            scores(1, op + k_order(0));
        }
        commit(b.op_empty + (op + k_order(0)) % S::kOps);
        if (!pair && n > 1) {
            acquire(op + k_order(1));
            queries(1);
            scores(1, op + k_order(1));
            commit(b.op_empty + (op + k_order(1)) % S::kOps);
        }
        // weights of a tile are the sign that its scores were read too
        auto half_step = [&](int h, uint32_t ov, bool first, uint32_t ok, bool more) {
            weights(h);
            if (S::kOwnW && more)
                scores(h, ok);
            values(h, ov, first);
            if (!S::kOwnW && more)
                scores(h, ok);
        };
        for (int t = 0; t < n; ++t) {
            const uint32_t ov = op + v_order(t, n);
            const int tk = pair ? t + 1 : t + 2;
            const bool more = tk < n;
            const uint32_t ok = op + k_order(tk);
            if (pair) {
                if (more)
                    acquire(ok);
                acquire(ov);
                half_step(0, ov, t == 0, ok, more);
                half_step(1, ov, t == 0, ok, more);
                commit(b.op_empty + ov % S::kOps);
                if (more)
                    commit(b.op_empty + ok % S::kOps);
            } else {
                acquire(ov);
                if (more && S::kOwnW)
                    acquire(ok);
                weights(t & 1);
                if (S::kOwnW && more) {
                    scores(t & 1, ok);
                    commit(b.op_empty + ok % S::kOps);
                }
                values(t & 1, ov, t < 2);
                commit(b.op_empty + ov % S::kOps);
                if (!S::kOwnW && more) {
                    acquire(ok);
                    scores(t & 1, ok);
                    commit(b.op_empty + ok % S::kOps);
                }
            }
        }
        op += 2 * n;
    }
    commit(b.spare);                               // issued MMAs end before the CTA's memory goes away
    wait_phase(b.spare, 0);
}

// ------------------------------------------------------------------ softmax

// The workers (CTAs, or their halves) of a unit and the place of this one among them.
struct Workers {
    int count, slot, ticket;
};

// Scores of positions outside [lo, hi) to -infinity; x holds those of k .. k + 31.
// The warp-wide step keeps it behind a branch: as predicated instructions it cost every tile 400 issue slots a warp.
__device__ __forceinline__ void hide(float (&x)[32], int k, int lo, int hi) {
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (k + e < lo || k + e >= hi)
            x[e] = -INFINITY;
}

// Where more values were NaN than the list holds: a row looks through the cache itself, at tiles first, first + step .. before
// last that some row of its piece sees in part, and writes NaN over its results' dims d0 .. d1 - 1.  (Not inlined, and by
// value: the softmax's loop is the faster for it.)
template <int D>
__device__ __noinline__ void nan_rows(const AttnArgs &a, int request, int head, int kv, int n, int row0, int rows, int first, int last, int step,
                                      int lo, int hi, int d0, int d1, uint16_t *out, float *part, int cap) {
    int lo0, hi0, lo1, hi1;
    row_range(a.p, a.group, kv, n, row0, lo0, hi0);
    row_range(a.p, a.group, kv, n, row0 + rows - 1, lo1, hi1);
    for (int t = first; t < last; t += step) {
        if ((t + 1) * kTile <= hi0 && t * kTile >= lo1)
            continue;                              // seen by all: the product has them
        for (int j = max(t * kTile, lo); j < min((t + 1) * kTile, hi); ++j) {
            int page = __ldg(a.p.table + (size_t)request * a.p.max_blocks + (j >> a.shift));
            if (page < 0 || page >= a.p.cache.num_blocks)
                page = 0;
            const int off = j & ((1 << a.shift) - 1);
            const uint8_t *v = a.p.cache.v + ((((size_t)page * a.p.cache.kv_heads + head) << a.shift) + (off & ~15)) * D + (off & 15);
            for (int d = d0; d < d1; ++d)
                if ((__ldg(v + 16 * d) & 0x7F) == 0x7F) {
                    if (out)
                        out[d] = 0x7FFF;
                    else
                        __stcg(part + (size_t)(d >> 2) * cap * 4 + (d & 3), __uint_as_float(0x7FFFFFFFu));
                }
        }
    }
}

// A row's references, m and M - m (less kLift), and its l with respect to m.
struct Refs {
    float m, rel, l;
};

// A tile as one row finds it.
struct TileRow {
    uint32_t lanes;          // the warp's rows in tensor memory
    int h;                   // their half
    const float *meta;       // the sub-blocks' exponents
    float f;                 // factor of the row's products
    int lo, hi, tok0;        // positions that it sees, the tile's first
    int edge;                // some row of the warp does not see all of it
    uint64_t *product;       // barrier of the half's last product, if there was one, and its parity
    uint32_t parity;
    uint32_t *hdr;
};

__device__ __forceinline__ float factor(float f, const float *meta, int sub) { return fmaxf(f * meta[sub], 1.2e-38f); }

// The tile's scores 32 c .. 32 c + 31.
__device__ __forceinline__ void row_scores(float (&x)[32], const TileRow &t, int c) {
    tmem_ld32(x, t.lanes + 128 * t.h + 32 * c);
    if (t.edge)
        hide(x, t.tok0 + 32 * c, t.lo, t.hi);
}

// 32 scores (LESS: less their reference already) to weights; their terms of l to sum; whether they outgrew the references.
template <bool LESS>
__device__ __forceinline__ bool weigh(const float (&x)[32], const float *meta, float f, int c, const Refs &refs, uint32_t (&w)[16], float &sum) {
    const float mz = LESS ? 0.0f : seen(refs.m), below = seen(refs.rel);
    const uint64_t minus_m = pack2(-mz, -mz);
    bool grew = false;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const float *y = x + 16 * u;
        const float fi = LESS ? 1.0f : factor(f, meta, 2 * c + u), bb = meta[kSubs + 2 * c + u];
        const float r = ex2(fminf(bb - below, 126.0f));
        const uint64_t fi2 = pack2(fi, fi), r2 = pack2(r, r);
        uint64_t s2[2];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const float2 t2 = unpack2(fma2(pack2(y[e], y[e + 1]), fi2, minus_m));
            const uint64_t p2 = pack2(ex2(t2.x), ex2(t2.y));
            s2[e >> 1 & 1] = e < 4 ? p2 : add2(s2[e >> 1 & 1], p2);
            const float2 w2 = unpack2(mul2(p2, r2));
            const __half2 h2 = __floats2half2_rn(w2.x, w2.y);
            w[8 * u + e / 2] = *reinterpret_cast<const uint32_t *>(&h2);
        }
        const float2 t = unpack2(add2(s2[0], s2[1]));
        const float s16 = t.x + t.y;
        sum += s16;
        grew |= fmaxf(s16 * r, s16 * kLeastSum) > kMostWeight;
    }
    return grew;
}

// The weights of a tile's chunks (of 32 scores) from c on, the references first moved to the maxima where those lie above, of the whole tile
// or, behind weights that are stored already, of a chunk where it outgrows them.  With the references moves what was made with
// them: l, the half's sums, the stored weights.
template <int D>
__device__ __forceinline__ Refs move_and_weigh(Refs r, const TileRow &t, int c) {
    using S = TcSmem<D>;
    int top = c;                                   // the references are no less than the scores of the chunks before
    bool move = true;
#pragma unroll 1
    while (c < 4) {
        if (move) {
            top = c == 0 ? 4 : c + 1;
            float nm = -INFINITY, nrel = -INFINITY;        // largest x, and x + b less that
#pragma unroll 1
            for (int k = c; k < top; ++k) {
                float x[32];
                row_scores(x, t, k);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float *y = x + 16 * u;
                    float v0 = max3(y[0], y[1], y[2]), v1 = max3(y[3], y[4], y[5]), v2 = max3(y[6], y[7], y[8]), v3 = max3(y[9], y[10], y[11]);
                    v0 = max3(v0, y[12], y[13]);
                    v1 = max3(v1, y[14], y[15]);
                    const float v = fmaxf(max3(v0, v1, v2), v3) * factor(t.f, t.meta, 2 * k + u), to = fmaxf(nm, v), z = seen(to);
                    nrel = fmaxf(nrel + (nm - z), (v - z) + t.meta[kSubs + 2 * k + u]);
                    nm = to;
                }
            }
            const float to = fmaxf(nm, r.m), z = seen(to);
            const float was = r.rel + (r.m - z), want = fmaxf(nrel + (nm - z) - kLift, -INFINITY);     // M from the new m, as it is and at least
            // nothing is left of sums 150 binades down: their reference may be far off, and is not added to
            const bool anew = !(want - was < 150.0f);
            const float up = anew ? 0.0f : fmaxf(ceilf(want - was), 0.0f), by = anew ? 0.0f : ex2(-up);
            r.l *= ex2(r.m - z);
            r.m = to;
            r.rel = anew ? want : was + up;
            if (t.product) {
                if (!__all_sync(0xffffffffu, wait_phase(t.product, t.parity)) && (threadIdx.x & 31) == 0)
                    record_status(t.hdr, MOE_ERR_DEVICE_TIMEOUT);
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                    const uint32_t at = t.lanes + 256 + D * t.h + 32 * k;
                    float x[32];
                    tmem_ld32(x, at);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        x[e] *= by;
                    tmem_st32(at, x);
                }
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
#pragma unroll 1
            for (int k = 0; k < c; ++k) {
                uint32_t w[16];
                tmem_ld16(reinterpret_cast<float(&)[16]>(w), t.lanes + S::w_col(t.h, 32 * k));
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 f2 = __half22float2(*reinterpret_cast<const __half2 *>(w + e));      // f16 holds no factor below 2^-24
                    const __half2 v = __floats2half2_rn(f2.x * by, f2.y * by);
                    w[e] = *reinterpret_cast<const uint32_t *>(&v);
                }
                tmem_st16(t.lanes + S::w_col(t.h, 32 * k), w);
            }
        }
        float x[32], sum = 0.0f;
        uint32_t w[16];
        row_scores(x, t, c);                       // no weights lie over these yet
        const float z = seen(r.m);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            x[e] = __fsub_rn(__fmul_rn(x[e], factor(t.f, t.meta, 2 * c + e / 16)), z);
        move = __any_sync(0xffffffffu, weigh<true>(x, t.meta, t.f, c, r, w, sum)) && c >= top;
        if (move)
            continue;
        r.l += sum;
        tmem_st16(t.lanes + S::w_col(t.h, 32 * c), w);
        ++c;
    }
    return r;
}

template <int D>
__device__ __forceinline__ void tc_softmax(const AttnArgs &a, const Plan &pl, uint8_t *sm, const Bars &b, uint32_t tmem,
                                           uint32_t *nan_count, int *s_last) {
    using S = TcSmem<D>;
    const AttnProblem &p = a.p;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int h = warp >> 2, tid = threadIdx.x & 127;                                   // tid = TMEM lane = row
    const uint32_t lanes = tmem + ((uint32_t)(tid & ~31) << 16), s_at = lanes + 128 * h, o_at = lanes + 256 + D * h;
    uint8_t *q_at = sm + (size_t)h * S::kQBytes + tid * 128;
    uint32_t sn = 0, on = 0, tile = 0;             // score tiles and products of this half, tiles of the CTA
    bool dead = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!dead) {
            dead = !__all_sync(0xffffffffu, wait_phase(bar, parity));
            if (dead && lane == 0)
                record_status(a.hdr, MOE_ERR_DEVICE_TIMEOUT);
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    };
    Walk walk(a, pl, a.recs);
    Piece pc;
    for (int unit = 0; walk.next(pc); ++unit) {
        const int n = pc.t1 - pc.t0;
        const bool pair = pc.rows > 128;
        const int mine = half_tiles(pc, pair, h);
        const int rr = pair ? 128 * h + tid : tid;
        const bool live = rr < pc.rows, idle = (rr & ~31) >= pc.rows;
        const int row = pc.row0 + (live ? rr : 0);
        if (mine == 0 && (n > 0 || (h > 0 && !pair))) {     // one tile for two halves, or none: the first half's
            tile += n;
            continue;
        }
        // the row's query, scaled into f16, and its limits
        const uint16_t *src = p.q + (int64_t)(pc.q0 + row / a.group) * p.q_st + (int64_t)(pc.head * a.group + row % a.group) * p.q_sh;
        uint2 raw[D / 4];
        float mx = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 4; ++j)
            raw[j] = live ? __ldg(reinterpret_cast<const uint2 *>(src + 4 * j)) : make_uint2(0, 0);
#pragma unroll
        for (int j = 0; j < D / 4; ++j)
            mx = fmaxf(mx, fmaxf(fmaxf(fabsf(__uint_as_float(raw[j].x << 16)), fabsf(__uint_as_float(raw[j].x & 0xFFFF0000u))),
                                 fmaxf(fabsf(__uint_as_float(raw[j].y << 16)), fabsf(__uint_as_float(raw[j].y & 0xFFFF0000u)))));
        const int sh = f16_shift_for_max(mx);
        const float sc = exp2i(sh), f = a.scale_log2 * exp2i(-sh);
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint2 v = raw[2 * j + e];
                const __half2 x = __floats2half2_rn(__uint_as_float(v.x << 16) * sc, __uint_as_float(v.x & 0xFFFF0000u) * sc);
                const __half2 y = __floats2half2_rn(__uint_as_float(v.y << 16) * sc, __uint_as_float(v.y & 0xFFFF0000u) * sc);
                w[2 * e] = *reinterpret_cast<const uint32_t *>(&x);
                w[2 * e + 1] = *reinterpret_cast<const uint32_t *>(&y);
            }
            *reinterpret_cast<uint4 *>(q_at + (j >> 3) * 16384 + (((j & 7) ^ (tid & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0 && mine > 0)
            mbar_arrive(b.q_ready + h);
        // a lane without a row sees from the first row's first position on: what lies before is not read, and it has a vote in its warp
        int lo, hi;
        row_range(p, a.group, pc.kv, pc.n, row, lo, hi);
        if (!live)
            hi = pc.kv;
        const int min_hi = __reduce_min_sync(0xffffffffu, hi), max_lo = __reduce_max_sync(0xffffffffu, lo);

        Refs refs{-INFINITY, -INFINITY, 0.0f};
        for (int i = 0; i < mine; ++i) {
            const int t = pair ? i : 2 * i + h;
            const int tok0 = (pc.tile0 + pc.t0 + t) * kTile;
            wait(b.s_full + h, sn & 1);
            ++sn;
            if (!idle) {
                const bool edge = tok0 + kTile > min_hi || tok0 < max_lo;
                const float *meta = reinterpret_cast<const float *>(sm + S::kOffMeta) + ((tile + t) % S::kMetaTiles) * 2 * kSubs;
                const TileRow tr{lanes, h, meta, f, lo, hi, tok0, edge, i > 0 && !dead ? b.o_done + h : nullptr, (on - 1) & 1, a.hdr};
                auto scores = [&](float (&x)[32], int c) {
                    tmem_ld32(x, s_at + 32 * c);
                    if (edge)
                        hide(x, tok0 + 32 * c, lo, hi);
                };
                // where weights have columns of their own these scores came before the last product: it must have read its weights
                if (S::kOwnW && i > 0)
                    wait(b.o_done + h, (on - 1) & 1);
                // The loops are rolled: unrolled, their instructions cost more to fetch than the steps they save (9 to 12 % of the kernel).
                int made = 4;                      // chunks of 32 with their weights
                if (__any_sync(0xffffffffu, !(fabsf(refs.m) <= kFar))) {            // no reference yet, or a far one
                    made = 0;
                } else if (S::kOwnW) {
                    // the scores outlive the weights: one vote a tile (four take 159 us for 147)
                    float sum = 0.0f;
                    bool grew = false;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        float x[32];
                        uint32_t w[16];
                        scores(x, c);
                        grew |= weigh<false>(x, meta, f, c, refs, w, sum);
                        tmem_st16(lanes + S::w_col(h, 32 * c), w);
                    }
                    if (__any_sync(0xffffffffu, grew))
                        made = 0;
                    else
                        refs.l += sum;
                } else {
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        float x[32], sum = 0.0f;
                        uint32_t w[16];
                        scores(x, c);
                        if (__any_sync(0xffffffffu, weigh<false>(x, meta, f, c, refs, w, sum))) {
                            made = c;
                            break;
                        }
                        refs.l += sum;
                        tmem_st16(lanes + S::w_col(h, 32 * c), w);
                    }
                }
                if (made < 4)
                    refs = move_and_weigh<D>(refs, tr, made);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                mbar_arrive(b.w_ready + h);
            ++on;
        }
        if (mine > 0)
            wait(b.o_done + h, (on - 1) & 1);
        tile += n;

        // ---- the rows' result: l is NaN where a score was (or was infinite), and then so is the row
        float m = refs.m, l = refs.l, scale = l == 0.0f ? 0.0f : exp2f(refs.rel) / l;
        const int ctas = pc.last - pc.first + 1;
        // Halves that share the rows of an uncut unit join here: through the space of their queries, which nothing reads
        // any more, each learns the other's reference and sum, and makes half of the dims from both products.
        const bool both = !pair && ctas == 1 && n > 1;
        float other_scale = 0.0f;
        if (both) {
            *reinterpret_cast<float4 *>(q_at) = make_float4(scale, m, l, 0.0f);
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            named_barrier_sync(3, 256);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const float4 other = *reinterpret_cast<const float4 *>(sm + (size_t)(1 - h) * S::kQBytes + tid * 128);
            const float rm = fmaxf(m, other.y), z = rm == -INFINITY ? 0.0f : rm;
            const float w0 = l * ex2(m - z), w1 = other.z * ex2(other.y - z), wt = w0 + w1 == 0.0f ? 0.0f : 1.0f / (w0 + w1);
            scale *= w0 * wt;
            other_scale = other.x * w1 * wt;
            m = rm;
            l = w0 + w1;
        }
        // workers of a cut unit: its CTAs, twice those with two tiles or more where the halves share rows
        Workers w{1, 0, 0};
        {
            const int cta = (int)blockIdx.x;
            w.slot = (cta * 2 + (cta == pc.first)) * 2 + h;
            w.ticket = pc.first * 2 + (pair ? h : 0);
            // tiles of the unit in the first and the last of its CTAs; those between have pl.per of them
            w.count = pair || ctas == 1 ? ctas : min(2, pc.first_tiles) + min(2, pc.last_tiles) + (int)min(2ll, pl.per) * (ctas - 2);
        }
        if (w.count == 1 && l == 0.0f && lo < hi)  // it sees positions, and every score overflowed
            scale = other_scale = l = __uint_as_float(0x7FFFFFFFu);
        const int rows_here = pair ? min(128, pc.rows - 128 * h) : pc.rows;
        const int cap = min(128, (int)min((long long)p.T * a.group, 128ll));       // rows of a part in the workspace
        // values so far, this unit's all among them
        const uint32_t nan_seen = *reinterpret_cast<volatile uint32_t *>(nan_count);
        const volatile uint32_t *marks = reinterpret_cast<const volatile uint32_t *>(sm + S::kOffMarks);
        const size_t to = (size_t)(pc.q0 + row / a.group) * p.q_heads + pc.head * a.group + row % a.group;
        const NanEntry *nans = reinterpret_cast<const NanEntry *>(static_cast<const uint8_t *>(a.nans) + (size_t)blockIdx.x * kAttnNanBytes);
#pragma unroll 1
        for (int c = both ? h * (D / 64) : 0; c < (both ? (h + 1) * (D / 64) : D / 32); ++c) {
            float x[32];
            if (mine > 0) {
                tmem_ld32(x, o_at + 32 * c);
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    x[e] = 0.0f;
            }
            uint32_t bad = 0;                      // dims whose values this row saw as NaN
            for (uint32_t k = 0; k < min(nan_seen, (uint32_t)kNanEntries); ++k) {
                if (!(marks[k / 32] >> (k & 31) & 1))
                    continue;
                __threadfence();
                const int nu = __ldcg(&nans[k].unit), nt = __ldcg(&nans[k].token);
                if (nu == unit && nt >= lo && nt < hi && (pair || both || (((nt / kTile - pc.tile0 - pc.t0) & 1) == h)))
                    bad |= __ldcg(&nans[k].dims[c]);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e)
                x[e] *= scale;
            if (both) {
#pragma unroll
                for (int u = 0; u < 32; u += 16) {
                    float y[16];
                    tmem_ld16(y, lanes + 256 + D * (1 - h) + 32 * c + u);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        x[u + e] = fmaf(y[e], other_scale, x[u + e]);
                }
            }
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (bad >> e & 1)
                    x[e] = __uint_as_float(0x7FFFFFFFu);
            if (live && w.count == 1) {
                if (!MOE_DBG_IN_RANGE(pc.q0 + row / a.group, p.T, a.hdr))
                    continue;
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v[q]) : "f"(x[e + 2 * q + 1]), "f"(x[e + 2 * q]));
                    uint2 *dst = reinterpret_cast<uint2 *>(p.out + to * D + 32 * c + e);
                    dst[0] = make_uint2(v[0], v[1]);
                    dst[1] = make_uint2(v[2], v[3]);
                }
            } else if (live && MOE_DBG_IN_RANGE(w.slot, 4 * a.ctas, a.hdr) && MOE_DBG_IN_RANGE(tid, cap, a.hdr)) {
                // [dim / 4][row][4]: a warp's stores lie together
                float4 *dst = reinterpret_cast<float4 *>(a.part + (size_t)w.slot * cap * D) + (size_t)8 * c * cap + tid;
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    __stcg(dst + (size_t)(e / 4) * cap, make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]));
            }
        }
        if (live && nan_seen > (uint32_t)kNanEntries) {
            const int at = pc.tile0 + pc.t0;
            nan_rows<D>(a, pc.request, pc.head, pc.kv, pc.n, pc.row0, pc.rows, at + (pair || both ? 0 : h), at + n, pair || both ? 1 : 2, lo, hi,
                        both ? h * (D / 2) : 0, both ? (h + 1) * (D / 2) : D, w.count == 1 ? p.out + to * D : nullptr,
                        a.part + ((size_t)w.slot * cap * D + 4 * tid), cap);
        }
        __syncwarp();
        if (both) {                                // the products may be made anew
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            named_barrier_sync(3, 256);
        }
        if (live && w.count == 1) {
            if (p.lse && (!both || h == 0))
                p.lse[to] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
        } else if (live && MOE_DBG_IN_RANGE(w.slot, 4 * a.ctas, a.hdr) && MOE_DBG_IN_RANGE(tid, cap, a.hdr)) {
            __stcg(a.part_sum + (size_t)w.slot * cap + tid, make_float2(m, l));
        }
        if (w.count > 1) {
            __threadfence();
            named_barrier_sync(1 + h, 128);
            if (tid == 0) {
                __threadfence();
                const bool last = MOE_DBG_IN_RANGE(w.ticket, 2 * a.ctas, a.hdr) && atomicAdd(a.tickets + w.ticket, 1u) == (uint32_t)(w.count - 1);
                if (last)
                    a.tickets[w.ticket] = 0;       // for the next call
                s_last[h] = last;
                __threadfence();
            }
            named_barrier_sync(1 + h, 128);
            if (s_last[h]) {
                // Parts in the order of the cache's CTAs, a CTA's first half before its second.  A thread has 16 dims of
                // a row at a time: the row's log-sum, then four parts' loads in flight.
                auto has_two = [&](int k) { return !pair && (k == 0 ? pc.first_tiles : k == ctas - 1 ? pc.last_tiles : pl.per) >= 2; };
                const int parts = pair ? ctas : 2 * ctas;
                auto slot_of = [&](int k) {        // -1: the part does not exist
                    const int c = pair ? k : k >> 1, g = pair ? h : k & 1;
                    const int slot = ((pc.first + c) * 2 + (c == 0)) * 2 + g;
                    return k < parts && (pair || g == 0 || has_two(c)) && MOE_DBG_IN_RANGE(slot, 4 * a.ctas, a.hdr) ? slot : -1;
                };
                constexpr int U = 4;
                for (int i = tid; i < rows_here * (D / 16); i += 128) {
                    const int r = i % rows_here, d = i / rows_here * 4;
                    float rm = -INFINITY, rl = 0.0f;
                    for (int k0 = 0; k0 < parts; k0 += 2 * U) {
                        float2 e[2 * U];           // m, l
#pragma unroll
                        for (int u = 0; u < 2 * U; ++u) {
                            const int slot = slot_of(k0 + u);
                            e[u] = slot >= 0 ? __ldcg(a.part_sum + (size_t)slot * cap + r) : make_float2(-INFINITY, 0.0f);
                        }
                        float nm = rm;
#pragma unroll
                        for (int u = 0; u < 2 * U; ++u)
                            nm = fmaxf(nm, e[u].x);
                        const float z = nm == -INFINITY ? 0.0f : nm;
                        rl *= ex2(rm - z);
                        rm = nm;
#pragma unroll
                        for (int u = 0; u < 2 * U; ++u)
                            rl += e[u].y * ex2(e[u].x - z);
                    }
                    const int grow = pc.row0 + (pair ? 128 * h : 0) + r;
                    if (rl == 0.0f) {              // it sees nothing, or every score overflowed
                        int rlo, rhi;
                        row_range(p, a.group, pc.kv, pc.n, grow, rlo, rhi);
                        if (rlo < rhi)
                            rl = __uint_as_float(0x7FFFFFFFu);
                    }
                    const float z = rm == -INFINITY ? 0.0f : rm, wt = rl == 0.0f ? 0.0f : 1.0f / rl;
                    const size_t at = (size_t)(pc.q0 + grow / a.group) * p.q_heads + pc.head * a.group + grow % a.group;
                    float o[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        o[e] = 0.0f;
                    for (int k0 = 0; k0 < parts; k0 += U) {
                        float2 e[U];
                        float4 v[U][4];
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const int slot = slot_of(k0 + u);
                            e[u] = slot >= 0 ? __ldcg(a.part_sum + (size_t)slot * cap + r) : make_float2(-INFINITY, 0.0f);
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                v[u][q] = slot >= 0 ? __ldcg(reinterpret_cast<const float4 *>(a.part + (size_t)slot * cap * D) + (size_t)(d + q) * cap + r)
                                                    : make_float4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const float w = e[u].y * ex2(e[u].x - z) * wt;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                o[4 * q] += v[u][q].x * w;
                                o[4 * q + 1] += v[u][q].y * w;
                                o[4 * q + 2] += v[u][q].z * w;
                                o[4 * q + 3] += v[u][q].w * w;
                            }
                        }
                    }
                    uint2 *dst = reinterpret_cast<uint2 *>(p.out + at * D + d * 4);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t x0, x1;
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x0) : "f"(o[4 * q + 1]), "f"(o[4 * q]));
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x1) : "f"(o[4 * q + 3]), "f"(o[4 * q + 2]));
                        dst[q] = make_uint2(x0, x1);
                    }
                    if (d == 0 && p.lse)
                        p.lse[at] = rl == 0.0f ? -INFINITY : (rm + log2f(rl)) * 0.69314718055994530942f;
                }
            }
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) attn_tc_kernel(const __grid_constant__ AttnArgs a) {
    using S = TcSmem<D>;
    extern __shared__ __align__(1024) uint8_t raw_smem[];
    uint8_t *sm = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + S::kOffBars);
    Bars b;
    b.raw_full = bar;
    b.raw_empty = b.raw_full + S::kRaw;
    b.op_full = b.raw_empty + S::kRaw;
    b.op_empty = b.op_full + S::kOps;
    b.s_full = b.op_empty + S::kOps;
    b.w_ready = b.s_full + 2;
    b.o_done = b.w_ready + 2;
    b.q_ready = b.o_done + 2;
    b.spare = b.q_ready + 2;
    uint32_t *s_taddr = reinterpret_cast<uint32_t *>(bar + S::kBarCount), *nan_count = s_taddr + 1;
    int *s_last = reinterpret_cast<int *>(s_taddr + 3);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kRaw; ++i) {
            mbar_init(b.raw_full + i, 1);
            mbar_init(b.raw_empty + i, kConvWarps);
        }
        for (int i = 0; i < S::kOps; ++i) {
            mbar_init(b.op_full + i, kConvWarps);
            mbar_init(b.op_empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(b.s_full + i, 1);
            mbar_init(b.w_ready + i, 4);
            mbar_init(b.o_done + i, 1);
            mbar_init(b.q_ready + i, 4);
        }
        mbar_init(b.spare, 1);
        *nan_count = 0;
        fence_barrier_init();
    }
    if (threadIdx.x < kNanEntries / 32)
        reinterpret_cast<uint32_t *>(sm + S::kOffMarks)[threadIdx.x] = 0;
    if (warp == kSoftWarps + kConvWarps + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(s_taddr)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *s_taddr;
    pdl_wait();
    pdl_trigger();
    const Plan pl = *a.plan;
    // 256 threads x 176 + 256 x 80 registers = the 512 x 128 of the launch
    if (warp < kSoftWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        tc_softmax<D>(a, pl, sm, b, tmem, nan_count, s_last);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp < kSoftWarps + kConvWarps)
            tc_convert<D>(a, pl, sm, b, nan_count);
        else if (warp == kSoftWarps + kConvWarps)
            tc_stream<D>(a, pl, sm, b);
        else
            tc_issue<D>(a, pl, sm, b, tmem);
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == kSoftWarps + kConvWarps + 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

}  // namespace

cudaError_t launch_attn_tc(const void *args, int head_dim, int ctas, cudaStream_t stream) {
    const AttnArgs a = *static_cast<const AttnArgs *>(args);
    auto go = [&](auto kernel, size_t smem) {
        cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        return r != cudaSuccess ? r : launch_pdl(kernel, dim3(ctas), dim3(kTcThreads), smem, stream, a);
    };
    return head_dim == 64 ? go(attn_tc_kernel<64>, TcSmem<64>::kBytes) : go(attn_tc_kernel<128>, TcSmem<128>::kBytes);
}

}  // namespace moe
