// Attention of drafted tokens over the paged cache and over their own tree:
// the device code.
//
// What it computes: for node i of sequence b (row r) and query head g, with m the
// largest score,
//     out[r, g] = sum_j exp(scale q.k_j - m) v_j / sum_j exp(scale q.k_j - m)
// over the sequence's cached tokens and over the nodes its mask names.
//
// How it runs on B200:
//  * All drafted tokens of a sequence read the same cache, and the G query heads
//    of a kv head read the same keys, so (node, head of the group) pairs are the
//    128 rows of one tcgen05.mma and each K and V byte leaves HBM once for up to
//    128 * STREAMS query rows.
//  * A unit of work is (sequence, kv head, row chunk): its tiles of cached tokens,
//    then those of the drafted rows.  One CTA per slot of the GPU stays for the
//    whole call and takes an equal share of all tiles, in order, so that neither
//    the lengths nor the number of sequences leave SMs idle; a unit that is cut by
//    a border between two CTAs leaves partial states for a second kernel.
//  * Two producer warps walk the units, dereference the block table and stage tiles
//    with TMA, one those of K, one those of V, each into its own ring.  The first
//    also describes each tile (sequence, rows, valid tokens) in a ring of its own.
//  * One thread for each 128 rows issues the products: S = Q K^T (bf16, fp32
//    accumulator in TMEM) and O += P V with P read from TMEM.
//  * Four warps for each 128 rows run the softmax, a row to a thread: no shuffles.
//    P goes back to TMEM as bf16: 8 significant bits for each weight, as many as the
//    values it multiplies have, and as the output keeps; the sum of the weights is
//    fp32 and unrounded.  (pa_decode keeps two parts of a weight and returns fp32;
//    a second part here would need 64 more columns than TMEM has for a CTA.)
//  * A tile is 64 tokens: a thread holds its row's 64 scores in registers, which frees
//    the score buffer for the next tile's product while the exponentials run, and P
//    has two buffers, so that neither product is waited for.  128-token tiles in one
//    buffer need half the mma instructions for the scores (65 cycles each at N = 64 as
//    at N = 128), but scores, softmax and product of a stream then follow one another:
//    133 us against 73 us on 64 sequences of up to 4096 tokens with 32/8 heads.
//  * The running maximum moves only when a score exceeds it by more than 2^8 in
//    weight: O stays in TMEM and is rescaled a few times in a row's life instead of
//    once a tile.  fp32 holds weights up to 2^8 as well as up to 1, and the
//    quotient at the end does not depend on which reference was used.
//  * STREAMS = 1 (up to 128 query rows, bound by HBM): two CTAs on an SM.  STREAMS = 2
//    (more rows, bound by the products and the exponentials): two groups of 128 rows
//    share each K and V tile.
//  * What a row does not see has no part in it.  Scores are replaced, not added
//    to; V rows past the sequence's end are zeroed in shared memory before they meet
//    a weight of zero; non-finite values of drafted V rows (which some rows see and
//    others do not) are taken out of the product and added at the end to the rows
//    that see them.
#pragma once

#include <float.h>

#include "pa_common.cuh"

namespace pa {
namespace {

constexpr float kTreeLog2e = 1.4426950408889634f;
constexpr int kTileM = 128;        // query rows of one stream
constexpr int kTreeBox = 16;        // drafted rows of one TMA box
constexpr float kMaxRise = 8.0f;   // log2 of the largest weight before the reference moves

template <int HEAD_DIM, int STREAMS>
struct TreeCfg {
    static constexpr int kTileN = 64;                          // tokens of one tile
    static constexpr uint32_t kBufs = 2;                       // weight (P) buffers of a stream
    static constexpr int kBoxes = HEAD_DIM / 64;               // 128-byte wide column boxes
    static constexpr int kBoxBytes = kTileN * 128;             // one box of a K or V tile
    static constexpr int kTileBytes = kBoxes * kBoxBytes;
    static constexpr int kQBoxBytes = kTileM * 128;
    static constexpr int kQBytes = kBoxes * kQBoxBytes;        // one stream's queries
    static constexpr uint32_t kSlots = STREAMS * (HEAD_DIM == 64 ? 4 : 2);  // tiles of K, and of V, in shared memory
    static constexpr uint32_t kMetas = 16;                     // tile descriptions
    static constexpr int kCtasPerSm = STREAMS == 1 ? 2 : 1;
    static constexpr int kSoftmaxWarps = 4 * STREAMS;
    static constexpr int kThreads = (kSoftmaxWarps + 2 + STREAMS) * 32;  // + producers of K and of V, product warps
    // TMEM of one stream: the scores, two buffers of weights (bf16: half the columns), O.
    static constexpr int kPCol = kTileN, kOCol = 128;
    static_assert(kPCol + kBufs * kTileN / 2 <= kOCol, "TMEM columns of a stream");
    static constexpr int kStreamCols = 128 + 128;
    static constexpr int kCols = STREAMS * kStreamCols;
    static constexpr uint32_t kBars = 4 * kSlots + 2 * kMetas + STREAMS * (2 * kBufs + 6) + 2 + (STREAMS == 2 ? 8 : 0);
    static constexpr int kDataBytes = STREAMS * kQBytes + 2 * kSlots * kTileBytes;
    // Each softmax warp turns its rows of the output into whole 64-byte pieces here.
    static constexpr int kStageBytes = kSoftmaxWarps * 2048;
    static constexpr int kTailBytes = kStageBytes + kMetas * 48 + kBars * 8 + 32 * 8 + 2 * 16 + 16 + 64 /* TreeSpot */ + 16;
    static constexpr int kSmemBytes = 1024 /* align slack */ + kDataBytes + kTailBytes;
    static_assert(kCtasPerSm * kCols <= 512, "TMEM columns of an SM");
    static_assert(kCtasPerSm * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of an SM");
    // What a unit costs besides its tiles (its output, and tiles that are not whole: 3 to 4 us, a tile 1.1 us), and
    // the shortest pieces worth cutting off, in tiles.  Measured on 64 sequences of up to 4096 tokens with 32/8 heads
    // | 24 of up to 2048 with 32/32, in us: 2 and 2 72.7 | 77.5, 3 and 2 70.2 | 78.4, 4 and 2 70.8 | 79.7, 3 and 1
    // 70.5 | 78.4, 3 and 3 70.2 | 79.7.
    static constexpr int kUnitCost = 3;
    static constexpr int kSnap = 2;
};

// Where a CTA's share begins: tile `tile` of unit `unit` of sequence `b` (b = batch: nowhere), whose rows begin at
// `floor` or later.
struct TreeMark {
    int b, unit, tile, floor;
};

// What the second kernel joins: the unit inside which a CTA begins (0 pieces: it begins with a unit), and the first of
// the CTAs that begin inside it.
struct __align__(16) TreeJoin {
    int pieces, cut0, first, nodes, node0, h, pad[2];
};

struct TreeParams {
    uint16_t *out;             // [T, Hq, d] bf16
    float *part_o;             // [CTAs, 2, rows of a unit, d]: states of units that are cut (NULL: none is)
    float *part_ml;            // [CTAs, 2, rows of a unit, 2]
    TreeJoin *joins;           // [CTAs]
    const uint16_t *v_tree;
    const int32_t *tables, *lens, *cu, *masks;
    int32_t *err_flag;
    int64_t v_stride, num_blocks;
    int num_rows, batch, max_blocks, max_seq_len, max_nodes, words;
    int q_heads, kv_heads, group, group_shift, block_size;
    int min_share;             // tiles that a CTA takes at least
    int pool_rows;             // rows of the pools' tensor maps: a row outside of them reads as zeros
    float scale_log2;
};

// ---- tcgen05 and TMA forms that only this kernel uses ----

__device__ __forceinline__ void tma_load_3d(void *smem_dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// bf16 operands, fp32 accumulator of M = 128 rows and N columns; B transposed: stored [K, N]
__host__ __device__ constexpr uint32_t tree_idesc(int n, bool b_transposed) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_transposed ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kTileM >> 4) << 24);
}

// V as the [K = tokens, N = dims] operand: rows of 128 bytes (64 dims) with the 128-byte swizzle, 8-token
// groups 1024 bytes apart, the next 64 dims `box_bytes` further on.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t saddr, uint32_t box_bytes) {
    return (uint64_t)((saddr & 0x3ffffu) >> 4) | ((uint64_t)(box_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ void umma_bf16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// A from TMEM (two bf16 in each column)
__device__ __forceinline__ void umma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// 32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float *v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}

// The lowest n bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t low_bits(int n) {
    uint32_t x;
    asm("shl.b32 %0, %1, %2;" : "=r"(x) : "r"(0xffffffffu), "r"((uint32_t)max(n, 0)));  // a shift by 32 or more gives 0
    return ~x;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// mbar_wait_bounded without reading the clock when the phase is already there, and with the loop kept in one
// place: the kernel waits in some twenty of them, and its warps run different parts of it at the same time, so
// that instruction fetches are what they stall on most.
__device__ __noinline__ bool tree_wait_long(uint64_t *bar, uint32_t parity, int32_t *flag) {
    return mbar_wait_bounded(bar, parity, flag);
}
__device__ __forceinline__ bool tree_wait(uint64_t *bar, uint32_t parity, int32_t *flag) {
    return mbar_try_wait(bar, parity) || tree_wait_long(bar, parity, flag);
}
// Barriers kept in a ring: use n of it has its place and its parity (ring lengths are powers of two).
template <uint32_t N>
__device__ __forceinline__ bool ring_wait(uint64_t *bars, uint32_t n, int32_t *flag) {
    return tree_wait(bars + (n & (N - 1)), (n / N) & 1, flag);
}

// Whether any bf16 of v is an infinity or NaN (0: none is): an exponent of ones carries into the sign's place.
__device__ __forceinline__ uint32_t not_finite8(const uint4 &v) {
    auto test = [](uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; };
    return (test(v.x) | test(v.y) | test(v.z) | test(v.w)) & 0x80008000u;
}
// w with the halves that are not finite set to zero.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

// m c is rounded, by up to 32 where it is below 2^30; further out that would make all weights of a row infinite or 0.
// A score below the row's largest, m, is below it by m 2^-24 at least, as fp32 has it: out there it has no weight, and
// the scale may as well be another.
__device__ __forceinline__ bool tree_far(float m, float c) { return fabsf(m * c) > 0x1p30f && !isinf(m); }
// The scale in log2 of such a row: the power of two that takes m exactly to between 2^31 and 2^32.
__device__ __forceinline__ float tree_row_scale(float m, float c) {
    return tree_far(m, c) ? __int_as_float(min(254 + 31 - ((__float_as_int(m) >> 23) & 255), 254) << 23) : c;
}
// The reference of a partial state in log2: that of such a row is beyond 2^30 too, and larger where m is by 2^-17 of it
// or more.  (A sum of 64 or 128 products in fp32 is not known any better.)
__device__ __forceinline__ float tree_reference(float m, float c) {
    if (tree_far(m, c)) return copysignf((float)(__float_as_int(m) & 0x7fffffff) * 128.f, m);
    return m == -INFINITY ? m : m * c;
}

// A bound between sequences' rows.
__device__ __forceinline__ int tree_bound(const TreeParams &p, int i) { return min(max(__ldg(p.cu + i), 0), p.num_rows); }

// The sequence of a CTA, as every kernel of one call sees it.  Each row has one owner, whatever the bounds: `floor` is
// the largest of the bounds before b (where no bound is below the one before it, 0 does as well), and a sequence that
// begins below it has no nodes.
struct TreeSeq {
    int first, nodes, len;
    int end;  // the floor of the next sequence
    bool bad;
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams &p, int b, int floor) {
    const int lo = __ldg(p.cu + b), hi = __ldg(p.cu + b + 1), raw = __ldg(p.lens + b);
    TreeSeq s;
    s.first = min(max(lo, 0), p.num_rows);
    s.end = max(min(max(hi, 0), p.num_rows), max(s.first, floor));
    s.nodes = s.first < floor ? 0 : min(s.end - s.first, p.max_nodes);
    s.len = min(max(raw, 0), min(p.max_seq_len, p.max_blocks * p.block_size));
    s.bad = s.first != lo || s.end != hi || s.nodes != s.end - s.first || s.len != raw;
    return s;
}

// Row chunks of a sequence (units of one kv head) and the tiles of each.
struct TreeUnits {
    int chunks, ctx, tiles;
};
template <int HEAD_DIM, int STREAMS>
__device__ __forceinline__ TreeUnits tree_units(const TreeParams &p, const TreeSeq &q) {
    constexpr int N = TreeCfg<HEAD_DIM, STREAMS>::kTileN;
    const int rows = STREAMS * kTileM;
    TreeUnits u;
    u.chunks = ((q.nodes << p.group_shift) + rows - 1) / rows;
    u.ctx = (q.len + N - 1) / N;
    u.tiles = u.ctx + (q.nodes + N - 1) / N;
    return u;
}

// All tiles of the call, plus a fixed cost for each unit, form one line; `count` CTAs cut it into equal
// parts.  A cut near a unit's end moves there (where units may not be cut, every cut does).
struct TreeLine {
    int64_t total, before, mine;  // this thread's sequences [b0, b1) lie at [before, before + mine)
    int b0, b1, count, step, rest;
    int floor;  // of sequence b0
};

template <int HEAD_DIM, int STREAMS, int THREADS>
__device__ __forceinline__ TreeLine tree_line(const TreeParams &p, int ctas, int64_t *scan, bool report) {
    using C = TreeCfg<HEAD_DIM, STREAMS>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = p.batch <= THREADS ? 1 : (p.batch + THREADS - 1) / THREADS;
    TreeLine n;
    n.b0 = min((int)threadIdx.x * per, p.batch);
    n.b1 = min(n.b0 + per, p.batch);
    n.floor = 0;
    int64_t incl;
    for (bool ordered = true;;) {  // once, or a second time where bounds decrease
        bool down = false;
        n.mine = 0;
        for (int b = n.b0, floor = n.floor; b < n.b1; ++b) {
            const TreeSeq seq = tree_seq(p, b, floor);
            if (seq.bad && report) raise_flag(p.err_flag, PA_FLAG_BAD_LEN);
            const TreeUnits u = tree_units<HEAD_DIM, STREAMS>(p, seq);
            n.mine += (int64_t)(u.chunks * p.kv_heads) * (u.tiles + C::kUnitCost);
            down |= tree_bound(p, b + 1) < tree_bound(p, b);
            floor = seq.end;
        }
        incl = n.mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += up;
        }
        if (lane == 31) scan[warp] = incl;
        if (!__syncthreads_or(ordered && down)) break;
        ordered = false;
        for (int b = 0; b < n.b0; ++b) n.floor = max(n.floor, tree_bound(p, b));
    }
    n.before = incl - n.mine;
    n.total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) n.before += scan[w];
        n.total += scan[w];
    }
    // Shares of at least min_share tiles, so that neighbouring cuts never coincide inside a unit.
    if (n.total <= INT32_MAX) {
        n.count = max(1, min(ctas, (int)n.total / p.min_share));
        n.step = (int)n.total / n.count;
        n.rest = (int)n.total - n.step * n.count;
    } else {
        n.count = ctas;
        n.step = -1;
        n.rest = 0;
    }
    return n;
}

// What is left of it for one CTA: where the unit of its first mark begins.
struct TreeSpot {
    int64_t begin;
    TreeLine line;
};

// Where cut i lies on the line.
__device__ __forceinline__ int64_t tree_cut(const TreeLine &n, int i) {
    if (i >= n.count) return n.total;
    return n.step >= 0 ? (int64_t)n.step * i + n.rest * i / n.count : n.total / n.count * i;
}

// The tile at which a cut `at` into a sequence's units falls, as (unit, tile).
template <int HEAD_DIM, int STREAMS>
__device__ __forceinline__ TreeMark tree_mark(const TreeParams &p, const TreeUnits &u, int b, int64_t at) {
    using C = TreeCfg<HEAD_DIM, STREAMS>;
    const int weight = u.tiles + C::kUnitCost;
    TreeMark m{b, at <= INT32_MAX ? (int)at / weight : (int)(at / weight), 0, 0};
    const int tile = (int)(at - (int64_t)m.unit * weight) - C::kUnitCost;
    if (p.part_o ? tile > u.tiles - C::kSnap : 2 * tile >= u.tiles)
        ++m.unit;
    else if (p.part_o && tile >= C::kSnap)
        m.tile = tile;
    return m;
}

// The marks of cuts i and i + 1.  Every CTA computes the same cuts from the lengths alone.
template <int HEAD_DIM, int STREAMS, int THREADS>
__device__ __forceinline__ void tree_marks(const TreeParams &p, int ctas, int i, int64_t *scan, TreeMark *mark,
                                           TreeSpot *spot, bool report) {
    using C = TreeCfg<HEAD_DIM, STREAMS>;
    const TreeLine n = tree_line<HEAD_DIM, STREAMS, THREADS>(p, ctas, scan, report);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        int64_t at = tree_cut(n, i + k);
        if (threadIdx.x == 0 && at >= n.total) mark[k] = TreeMark{p.batch, 0, 0, 0};
        at -= n.before;
        if (at < 0 || at >= n.mine) continue;
        for (int b = n.b0, floor = n.floor; b < n.b1; ++b) {
            const TreeSeq seq = tree_seq(p, b, floor);
            const TreeUnits u = tree_units<HEAD_DIM, STREAMS>(p, seq);
            const int64_t weight = (int64_t)(u.chunks * p.kv_heads) * (u.tiles + C::kUnitCost);
            if (at < weight) {
                mark[k] = tree_mark<HEAD_DIM, STREAMS>(p, u, b, at);
                mark[k].floor = floor;
                if (k == 0) {
                    spot->line = n;
                    spot->begin = tree_cut(n, i) - at + (int64_t)mark[k].unit * (u.tiles + C::kUnitCost);
                }
                break;
            }
            at -= weight;
            floor = seq.end;
        }
    }
    __syncthreads();
}

// One tile, as the producer describes it to the other warps.
enum { kFirst = 1, kLast = 2, kTree = 4, kTwo = 8, kEnd = 16, kPlain = 32 };
struct __align__(16) TileMeta {
    int flags;   // first / last of its piece, drafted rows, both streams have rows, no tile, seen whole by all
                 // rows
    int start;   // first token (or node)
    int valid;   // tokens (or nodes) in it
    int dest;    // -1: the piece is a whole unit; else its partial state's place
    int first, nodes, node0, h;
    uint32_t words[4];  // the tokens that are there: not past the end, not in a bad block
};

template <int HEAD_DIM, int STREAMS>
__global__ void __launch_bounds__(TreeCfg<HEAD_DIM, STREAMS>::kThreads, TreeCfg<HEAD_DIM, STREAMS>::kCtasPerSm)
    tree_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap kt_map,
                const __grid_constant__ CUtensorMap vt_map, const TreeParams p) {
    using C = TreeCfg<HEAD_DIM, STREAMS>;
    constexpr int kTileN = C::kTileN;
    constexpr uint32_t kBufs = C::kBufs, kSlots = C::kSlots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint8_t *ring = smem + STREAMS * C::kQBytes;
    uint8_t *stage = smem + C::kDataBytes;
    TileMeta *meta = reinterpret_cast<TileMeta *>(stage + C::kStageBytes);
    TreeMark *mark = reinterpret_cast<TreeMark *>(meta + C::kMetas);  // [2]
    int64_t *scan = reinterpret_cast<int64_t *>(mark + 2);            // [32]
    uint64_t *full = reinterpret_cast<uint64_t *>(scan + 32);  // K's slots, then V's: the tile is there
    uint64_t *empty = full + 2 * kSlots;          // every stream has used the tile
    uint64_t *meta_full = empty + 2 * kSlots;
    uint64_t *meta_free = meta_full + C::kMetas;  // every softmax warp is done with the description
    uint64_t *s_full = meta_free + C::kMetas;     // [stream]: scores are in TMEM
    uint64_t *q_full = s_full + STREAMS;          // [stream]: the piece's queries are in shared memory
    uint64_t *pv_done = q_full + STREAMS;         // [stream][buffer]: the buffer's tile has been added to O
    uint64_t *o_done = pv_done + kBufs * STREAMS; // [stream]: a piece's last tile has
    uint64_t *p_full = o_done + STREAMS;          // [stream][buffer]: weights are in TMEM
    uint64_t *s_free = p_full + kBufs * STREAMS;  // [stream]: scores have been read
    uint64_t *o_free = s_free + STREAMS;          // [stream]: a piece's O has been read
    uint64_t *cleaned = o_free + STREAMS;         // [streams - 1]: the softmax warps of one / both have cleaned V
    uint64_t *drained = cleaned + 2;              // [stream]: every product has completed
    uint64_t *turn = drained + STREAMS;           // [stream][warp] of two: the stream's warp has had the exponentials
    TreeSpot *spot = reinterpret_cast<TreeSpot *>(turn + (STREAMS == 2 ? 8 : 0));
    static_assert(sizeof(TreeSpot) <= 64, "fits its place");
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(spot + 1);
    volatile uint32_t *found = tmem_slot + 4;     // [streams - 1][2]: the last cleaning that found something

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.group;
    const int tile_nodes = kTileM / G;  // nodes of one stream's rows

    if (warp == C::kSoftmaxWarps && lane == 0) {
        prefetch_tensormap(&k_map);
        prefetch_tensormap(&v_map);
        prefetch_tensormap(&q_map);
        prefetch_tensormap(&kt_map);
        prefetch_tensormap(&vt_map);
    }
    // One barrier for each thread: all are in one row, their counts follow from where they are.
    static_assert(C::kBars <= C::kThreads, "one thread initialises one barrier");
    if (threadIdx.x < C::kBars) {
        uint64_t *bar = full + threadIdx.x;
        mbar_init(bar, bar >= empty && bar < meta_full       ? STREAMS
                       : bar >= meta_free && bar < s_full    ? C::kSoftmaxWarps
                       : bar >= p_full && bar < cleaned      ? 4
                       : bar >= cleaned && bar < drained     ? 4 * (int)(bar - cleaned + 1)
                                                             : 1);
        fence_mbar_init();
    }
    if (threadIdx.x < 4) found[threadIdx.x] = 0;
    if (warp == C::kSoftmaxWarps + 2) {
        tmem_alloc(smem_addr(tmem_slot), C::kCols);
        tmem_relinquish();
        tc_fence_before();
    }
    tree_marks<HEAD_DIM, STREAMS, C::kThreads>(p, gridDim.x, blockIdx.x, scan, mark, spot, blockIdx.x == 0);  // synchronises
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
    // The joining CTAs find room only where CTAs of this grid have ended: this hides their launch, not their wait.
    if (p.part_o) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // The tiles of this CTA are numbered through all its pieces: tile t has slot t of K's ring and of V's.
    if (warp < C::kSoftmaxWarps + 2 && warp >= C::kSoftmaxWarps) {
        // ---------------- producers: units, block-table dereference, TMA ----------------
        // One warp for K, which also describes the tiles, one for V.  A copy costs the warp that issues it some
        // 60 cycles, and a tile of 16-token pages is 16 copies: one warp for both took 2500 cycles a tile.
        const bool is_k = warp == C::kSoftmaxWarps;
        full += is_k ? 0 : kSlots;
        empty += is_k ? 0 : kSlots;
        ring += is_k ? 0 : kSlots * C::kTileBytes;
        const int pages = kTileN / p.block_size;  // of one tile
        const int page = lane / C::kBoxes, box = lane % C::kBoxes;
        const TreeMark end = mark[1];
        // K and V are read once by one row chunk, again soon (from L2) by the others
        const uint64_t policy = p.max_nodes > STREAMS * tile_nodes ? l2_policy_evict_normal() : l2_policy_evict_first();

        // The walk over units and their tiles, from this CTA's mark to the next one's.  What stays the same
        // within a piece is worked out when the piece begins.
        TreeMark cur = mark[0];
        TreeSeq seq{}, ahead{};
        TreeUnits of{};
        if (cur.b < p.batch) {
            seq = tree_seq(p, cur.b, cur.floor);
            of = tree_units<HEAD_DIM, STREAMS>(p, seq);
            if (cur.b + 1 < p.batch) ahead = tree_seq(p, cur.b + 1, seq.end);
        }
        // A tile to be loaded: this lane loads column box `box` of block `id` of it, if it has a page at all.
        struct Tile {
            int flags, start, valid, id;
            bool mine;
            int dest, first, nodes, node0, h;  // the piece's
        };
        Tile piece{};
        int stop = 0;       // the piece's tiles end here
        bool fresh = true;  // a piece begins
        const int32_t *entries = nullptr;  // this lane's page of the sequence's first tile
        auto next_tile = [&]() -> Tile {
            if (fresh) {
                piece.flags = kEnd;
                piece.mine = false;
                for (;;) {
                    const bool more = cur.b != end.b        ? cur.b < end.b
                                      : cur.unit != end.unit ? cur.unit < end.unit
                                                             : cur.tile < end.tile;
                    if (!more) return piece;
                    if (cur.unit < of.chunks * p.kv_heads) break;
                    ++cur.b;  // on to the next sequence
                    cur.unit = cur.tile = of.chunks = 0;
                    seq = ahead;
                    if (cur.b < p.batch) of = tree_units<HEAD_DIM, STREAMS>(p, seq);
                    if (cur.b + 1 < p.batch) ahead = tree_seq(p, cur.b + 1, seq.end);
                }
                piece.h = of.chunks == 1 ? cur.unit : cur.unit / of.chunks;
                piece.node0 = (cur.unit - piece.h * of.chunks) * (STREAMS * tile_nodes);
                stop = cur.b == end.b && cur.unit == end.unit ? end.tile : of.tiles;
                piece.dest = cur.tile == 0 && stop == of.tiles ? -1 : 2 * (int)blockIdx.x + (cur.tile == 0);
                piece.first = seq.first;
                piece.nodes = seq.nodes;
                piece.flags = kFirst | (STREAMS == 2 && piece.node0 + tile_nodes < seq.nodes ? kTwo : 0);
                entries = p.tables + (int64_t)cur.b * p.max_blocks + page;
            }
            Tile t = piece;
            piece.flags &= ~kFirst;
            if (cur.tile < of.ctx) {
                t.start = cur.tile * kTileN;
                t.valid = min(kTileN, seq.len - t.start);
                t.mine = page < pages && t.start + page * p.block_size < seq.len;
                if (t.mine) t.id = __ldg(entries + cur.tile * pages);
                if (t.valid == kTileN) t.flags |= kPlain;
            } else {
                t.flags |= kTree;
                t.start = (cur.tile - of.ctx) * kTileN;
                t.valid = min(kTileN, seq.nodes - t.start);
            }
            fresh = ++cur.tile == stop;
            if (fresh) {
                t.flags |= kLast;
                if (stop == of.tiles) {
                    ++cur.unit;
                    cur.tile = 0;
                }
            }
            return t;
        };
        auto load = [&](const Tile &t, uint32_t slot) {
            uint8_t *dst = ring + slot * C::kTileBytes;
            // V past the end is read from outside of the tensor, which gives zeros: whatever the ring held
            // must not meet a weight of zero.  (The rest of a partly used box is zeroed by the softmax warps.)
            if (t.flags & kTree) {
                if (lane == 0)
                    mbar_arrive_expect_tx(full + slot, is_k ? C::kBoxes * ((t.valid + kTreeBox - 1) / kTreeBox) * kTreeBox * 128
                                                            : C::kTileBytes);
                __syncwarp();
                const int box_row = page * kTreeBox;
                if (box_row < (is_k ? t.valid : kTileN))
                    tma_load_3d(dst + box * C::kBoxBytes + box_row * 128, is_k ? &kt_map : &vt_map, box * 64, t.h,
                                box_row < t.valid ? t.first + t.start + box_row : p.num_rows, full + slot);
                return;
            }
            const bool mine = t.mine || (!is_k && page < pages);
            const int loads = __popc(__ballot_sync(0xffffffffu, mine));
            if (lane == 0) mbar_arrive_expect_tx(full + slot, loads * p.block_size * 128);
            __syncwarp();
            if (mine) {
                // a bad block reads as zeros too
                const bool none = !t.mine || t.id < 0 || t.id >= p.num_blocks;
                const int row = none ? p.pool_rows : (int)(((int64_t)t.id * p.kv_heads + t.h) * p.block_size);
                tma_load_2d(dst + box * C::kBoxBytes + page * p.block_size * 128, is_k ? &k_map : &v_map, box * 64, row,
                            full + slot, policy);
            }
        };
        // A tile is drawn one turn before it is loaded, so that table entries are there when they are needed.
        int landed = -1;  // lane x: the last tile loaded into slot x
        Tile next = next_tile();
#pragma unroll 1
        for (uint32_t t = 0;; ++t) {
            Tile now = next;
            if (!(now.flags & kEnd)) next = next_tile();
            // Everything that does not need the slot comes before the wait for it: in steady state the loads
            // wait for slots, and what lies between a free slot and its copy is lost.
            if (is_k) {
                const uint32_t holes = __ballot_sync(0xffffffffu, now.mine && box == 0 && (now.id < 0 || now.id >= p.num_blocks));
                if (holes) {
                    if (lane == 0) raise_flag(p.err_flag, PA_FLAG_BAD_BLOCK);
                    now.flags &= ~kPlain;
                }
                const uint32_t mt = t & (C::kMetas - 1);
                const bool free = t < C::kMetas || ring_wait<C::kMetas>(meta_free, t - C::kMetas, p.err_flag);
                if (!__all_sync(0xffffffffu, free)) break;
                if (lane == 0) {
                    int4 *d = reinterpret_cast<int4 *>(meta + mt);
                    d[0] = make_int4(now.flags, now.start, now.valid, now.dest);
                    d[1] = make_int4(now.first, now.nodes, now.node0, now.h);
                }
                if (!(now.flags & (kPlain | kEnd)) && lane < 4) {
                    uint32_t bits = low_bits(now.valid - 32 * lane);
                    if (holes)
                        for (int x = 0; x < 32; ++x) {
                            const int at = (32 * lane + x) / p.block_size;
                            if (at < pages && ((holes >> (at * C::kBoxes)) & 1)) bits &= ~(1u << x);
                        }
                    meta[mt].words[lane] = bits;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(meta_full + mt);
            }
            if (now.flags & kEnd) break;
            const bool free = t < kSlots || ring_wait<kSlots>(empty, t - kSlots, p.err_flag);
            if (!__all_sync(0xffffffffu, free)) break;
            if (lane == (int)(t & (kSlots - 1))) landed = (int)t;
            load(now, t & (kSlots - 1));
        }
        // If this CTA begins inside a unit: which others do, that is, how many pieces the unit has.
        if (is_k && p.part_o) {
            TreeJoin j{0, 0, 0, 0, 0, 0, {}};
            const TreeMark at = mark[0];
            if (at.b < p.batch && at.tile != 0) {
                const TreeSeq q = tree_seq(p, at.b, at.floor);
                const TreeUnits u = tree_units<HEAD_DIM, STREAMS>(p, q);
                const TreeLine &line = spot->line;
                auto inside = [&](int i) {  // cut i is one of this unit
                    if (i < 0 || i >= line.count) return false;
                    const int64_t x = tree_cut(line, i) - spot->begin;
                    if (x < 0 || x >= u.tiles + C::kUnitCost) return false;
                    const TreeMark m = tree_mark<HEAD_DIM, STREAMS>(p, u, at.b, x);
                    return m.unit == 0 && m.tile != 0;
                };
                auto run = [&](int from, int by) {  // cuts from, from + by, ... that are
                    int n = 0;
                    for (;;) {
                        const uint32_t is = __ballot_sync(0xffffffffu, inside(from + by * (n + lane)));
                        if (is != 0xffffffffu) return n + __ffs(~is) - 1;
                        n += 32;
                    }
                };
                const int before = run((int)blockIdx.x - 1, -1);
                j.pieces = before + run((int)blockIdx.x + 1, 1) + 2;
                j.cut0 = (int)blockIdx.x - before;
                j.first = q.first;
                j.nodes = q.nodes;
                j.h = at.unit / u.chunks;
                j.node0 = (at.unit - j.h * u.chunks) * (STREAMS * tile_nodes);
            }
            if (lane == 0) p.joins[blockIdx.x] = j;
        }
        // Every copy has landed before the CTA ends (it has, unless a wait ran out).
        if (lane < (int)kSlots && landed >= 0) mbar_wait_bounded(full + lane, ((uint32_t)landed / kSlots) & 1, p.err_flag);
    } else if (warp >= C::kSoftmaxWarps) {
        // ---------------- products, issued by one thread for each stream ----------------
        // S = Q K^T of tile t, then O += P V of tile t - 1.
        if (lane == 0) {
            constexpr uint32_t kQkDesc = tree_idesc(kTileN, false), kPvDesc = tree_idesc(HEAD_DIM, true);
            const int s = warp - (C::kSoftmaxWarps + 2);
            // Descriptors of the queries and of ring slot 0; a step through the operand or to another
            // slot adds to the start address (16-byte units), which never carries out of its field.
            const uint64_t q_desc = umma_desc_k_sw128(smem_addr(smem + s * C::kQBytes));
            const uint64_t k_desc = umma_desc_k_sw128(smem_addr(ring));
            const uint64_t v_desc = umma_desc_mn_sw128(smem_addr(ring + kSlots * C::kTileBytes), C::kBoxBytes);
            const uint32_t base = tmem + s * C::kStreamCols;
            uint32_t scored = 0, added = 0;  // tiles whose scores / products were issued
            uint32_t pieces_q = 0, pieces_o = 0;
            bool ok = true;
            for (uint32_t t = 0, before = 0;; ++t) {
                if (!(ok = ring_wait<C::kMetas>(meta_full, t, p.err_flag))) break;
                const uint32_t f = *const_cast<volatile int *>(&meta[t & (C::kMetas - 1)].flags);
                if (!(f & kEnd)) {
                    const uint32_t slot = t & (kSlots - 1);
                    if (!(ok = ring_wait<kSlots>(full, t, p.err_flag))) break;
                    if (s == 0 || (f & kTwo)) {
                        if ((f & kFirst) && !(ok = tree_wait(q_full + s, pieces_q++ & 1, p.err_flag))) break;
                        const uint32_t g = scored++;
                        // the last scores have to be in registers
                        if (g > 0 && !(ok = tree_wait(s_free + s, (g - 1) & 1, p.err_flag))) break;
                        tc_fence_after();
                        const uint64_t kd = k_desc + slot * (C::kTileBytes / 16);
#pragma unroll
                        for (int i = 0; i < HEAD_DIM / 16; ++i)
                            umma_bf16_ss(base, q_desc + ((i >> 2) * C::kQBoxBytes + (i & 3) * 32) / 16,
                                         kd + ((i >> 2) * C::kBoxBytes + (i & 3) * 32) / 16, kQkDesc, i > 0);
                        umma_commit(s_full + s);
                        umma_commit(empty + slot);
                    } else {
                        mbar_arrive(empty + slot);
                    }
                }
                if (t > 0) {  // `before`: the last tile's flags
                    const uint32_t slot = (t - 1) & (kSlots - 1);
                    if (!(ok = ring_wait<kSlots>(full + kSlots, t - 1, p.err_flag))) break;
                    if (s == 0 || (before & kTwo)) {
                        const uint32_t g = added++, buf = g & (kBufs - 1);
                        if (!(ok = ring_wait<kBufs>(p_full + kBufs * s, g, p.err_flag))) break;
                        // a new piece overwrites O: the last one's has to have been read
                        if ((before & kFirst) && pieces_o++ > 0 && !(ok = tree_wait(o_free + s, pieces_o & 1, p.err_flag))) break;
                        tc_fence_after();
                        const uint64_t vd = v_desc + slot * (C::kTileBytes / 16);
                        const uint32_t a = base + C::kPCol + buf * (kTileN / 2);
#pragma unroll
                        for (int i = 0; i < kTileN / 16; ++i)
                            umma_bf16_ts(base + C::kOCol, a + 8 * i, vd + i * (2048 / 16), kPvDesc, !(before & kFirst) || i > 0);
                        umma_commit(pv_done + kBufs * s + buf);
                        if (before & kLast) umma_commit(o_done + s);
                        umma_commit(empty + kSlots + slot);
                    } else {
                        mbar_arrive(empty + kSlots + slot);
                    }
                }
                if (f & kEnd) break;
                before = f;
            }
            umma_commit(drained + s);
            mbar_wait_bounded(drained + s, 0, p.err_flag);
        }
    } else {
        // ---------------- softmax: one row to a thread ----------------
        const int s = warp >> 2;
        const int r = threadIdx.x & (kTileM - 1);
        const uint32_t base = tmem + s * C::kStreamCols + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t o_addr = base + C::kOCol;
        // A scale of 0 must not meet -inf: the smallest value there is leaves every weight within 2^-20 of 1.
        const float c = fmaxf(p.scale_log2, __int_as_float(1));
        const float rise = fminf(kMaxRise / c, FLT_MAX);  // an infinite one would hide the first maximum (-inf + inf)

        // One thread of each stream loads its queries: the first piece's at once, the next one's when the
        // last scores of a piece are there, while their softmax and the piece's output are still to come.
        uint32_t q_loads = 0;
        auto load_queries = [&](uint32_t t) {
            if (!ring_wait<C::kMetas>(meta_full, t, p.err_flag)) return;
            const volatile TileMeta &m = meta[t & (C::kMetas - 1)];
            const int f = m.flags, row = m.first + m.node0 + s * tile_nodes, head = m.h * G;
            if ((f & kEnd) || (s == 1 && !(f & kTwo))) return;
            mbar_arrive_expect_tx(q_full + s, C::kQBytes);
            for (int x = 0; x < C::kBoxes; ++x)
                tma_load_3d(smem + s * C::kQBytes + x * C::kQBoxBytes, &q_map, x * 64, head, row, q_full + s);
            ++q_loads;
        };
        if ((warp & 3) == 0 && lane == 0) load_queries(0);

        constexpr int kWords = kTileN / 32;
        uint32_t g = 0, pieces = 0;  // tiles and pieces of this stream so far
        int node = 0;                // of this thread's row
        bool live = false, seen = false, dirty = false;
        uint32_t turns = 0;                    // so far
        uint2 cleanings = make_uint2(0u, 0u);  // so far, of one stream and of both
        uint32_t tree_bits[kWords] = {};  // the row's mask of the first drafted tile
        float m = -INFINITY, l = 0.f, row_c = c;
        bool ok = true;
        for (uint32_t t = 0;; ++t) {
            const uint32_t mt = t & (C::kMetas - 1);
            ok = ring_wait<C::kMetas>(meta_full, t, p.err_flag);
            if (!__all_sync(0xffffffffu, ok)) break;
            const int flags = meta[mt].flags;
            if (flags & kEnd) break;
            if (s == 1 && !(flags & kTwo)) {
                if ((flags & kLast) && (warp & 3) == 0 && lane == 0) load_queries(t + 1);
                __syncwarp();
                if (lane == 0) mbar_arrive(meta_free + mt);
                continue;
            }
            if (flags & kFirst) {
                const TileMeta &tile = meta[mt];
                node = tile.node0 + s * tile_nodes + (r >> p.group_shift);
                live = node < tile.nodes;
                seen = dirty = false;
                // Rows past the last node have the queries of whatever follows: no score of theirs may exceed their
                // maximum and move the reference of the warp's other rows, which decides how their weights round.
                m = live ? -INFINITY : INFINITY;
                l = 0.f;
                row_c = c;
                // the nodes of the first drafted tile that the row sees: needed at the end of the piece, fetched now
#pragma unroll
                for (int w = 0; w < kWords; ++w)
                    tree_bits[w] = !live ? 0u
                                   : !p.masks ? low_bits(node + 1 - 32 * w)
                                   : w < p.words ? (uint32_t)__ldg(p.masks + (int64_t)(tile.first + node) * p.words + w)
                                                 : 0u;
            }
            ok = tree_wait(s_full + s, g & 1, p.err_flag);
            if (!__all_sync(0xffffffffu, ok)) break;
            if ((flags & kLast) && (warp & 3) == 0 && lane == 0) load_queries(t + 1);
            // the tokens of the tile that this row sees
            uint32_t see[kWords];
            if (!(flags & kPlain)) {
                const TileMeta &tile = meta[mt];
                if ((flags & kTree) && tile.start > 0) {  // a later tile of a large tree
#pragma unroll
                    for (int w = 0; w < kWords; ++w) {
                        const int word = tile.start / 32 + w;
                        tree_bits[w] = !live ? 0u
                                       : !p.masks ? low_bits(node + 1 - 32 * word)
                                       : word < p.words ? (uint32_t)__ldg(p.masks + (int64_t)(tile.first + node) * p.words + word)
                                                        : 0u;
                    }
                }
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    see[w] = tile.words[w] & (flags & kTree ? tree_bits[w] : 0xffffffffu);
                    seen |= see[w] != 0;
                }
            } else {
                seen = true;
            }
            __syncwarp();
            tc_fence_after();
            float x[kTileN];
#pragma unroll
            for (int q = 0; q < kTileN / 32; ++q) tmem_ld32(base + 32 * q, x + 32 * q);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_free + s);  // the next tile's scores may be made
            if (!(flags & kPlain)) {
#pragma unroll
                for (int i = 0; i < kTileN; ++i) x[i] = (see[i >> 5] >> (i & 31)) & 1u ? x[i] : -INFINITY;
            }
            float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int i = 4; i < kTileN; ++i) top[i & 3] = fmaxf(top[i & 3], x[i]);
            const float tile_max = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            if (__any_sync(0xffffffffu, tile_max > m + rise)) {
                const float next = fmaxf(m, tile_max);
                const float down = next == -INFINITY ? 1.f : fast_exp2((m - next) * c);
                m = next;
                l *= down;
                row_c = tree_row_scale(m, c);
                if (!(flags & kFirst)) {  // O has been written: wait for the last product, then rescale it
                    ok = ring_wait<kBufs>(pv_done + kBufs * s, g - 1, p.err_flag);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int q = 0; q < HEAD_DIM / 16; ++q) {
                        uint32_t w[16];
                        tmem_ld16(o_addr + 16 * q, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * down);
                        tmem_st16(o_addr + 16 * q, w);
                    }
                }
            }
            // the weights take the place of an earlier tile's: its product has to be done
            const uint32_t buf = g & (kBufs - 1);
            ok = g < kBufs || ring_wait<kBufs>(pv_done + kBufs * s, g - kBufs, p.err_flag);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            if constexpr (STREAMS == 2) {
                // A warp of each stream shares a scheduler with one of the other.  Left alone they run in step, and
                // both want the exponentials at the same time and nothing else afterwards (94 against 87 us on 4
                // sequences of 8190 tokens with 512 query rows of each of 8 kv heads).  So they take turns: stream 0
                // waits for the other's turn at the tile before, stream 1 for that at this tile.
                if (flags & kTwo) {
                    const uint32_t n = turns++ - (s == 0);
                    ok = n == UINT32_MAX || tree_wait(turn + 4 * (1 - s) + (warp & 3), n & 1, p.err_flag);
                    if (!__all_sync(0xffffffffu, ok)) break;
                }
            }
            const uint32_t p_addr = base + C::kPCol + buf * (kTileN / 2);
            const float bias = m == -INFINITY ? 0.f : -m * row_c;
            const float2 c2 = make_float2(row_c, row_c), bias2 = make_float2(bias, bias);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int q = 0; q < kTileN / 32; ++q) {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 e = fma2(make_float2(x[32 * q + 2 * i], x[32 * q + 2 * i + 1]), c2, bias2);
                    const float2 pr = make_float2(fast_exp2(e.x), fast_exp2(e.y));
                    sum[i & 1] = add2(sum[i & 1], pr);
                    w[i] = pack_bf16x2(pr.x, pr.y);
                }
                tmem_st16(p_addr + 16 * q, w);
            }
            if constexpr (STREAMS == 2) {
                if ((flags & kTwo) && lane == 0) mbar_arrive(turn + 4 * s + (warp & 3));
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            if (!(flags & kPlain)) {
                // What must not meet a weight of zero: the rows past the end of a partly used box become
                // zeros, and values that are not finite leave drafted rows, which some rows do not see.
                // Both streams share the work, and none of their rows goes on before it is done.  (The
                // product of tile t - 2 is done, so what the slot held before V(t) has landed and the
                // parity of `full` is that of V(t).)
                const int valid = meta[mt].valid, box_rows = flags & kTree ? kTreeBox : p.block_size;
                if ((flags & kTree) || (valid & (box_rows - 1))) {
                    ok = ring_wait<kSlots>(full + kSlots, t, p.err_flag);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    const uint32_t v0 = smem_addr(ring) + (kSlots + (t & (kSlots - 1))) * C::kTileBytes;
                    const int end = (valid + box_rows - 1) & -box_rows;
                    const bool two = STREAMS == 2 && (flags & kTwo);
                    const int at = two ? threadIdx.x : r, rows = two ? 32 : 16;  // a row is eight chunks
                    const uint32_t mine = v0 + (at >> 3) * 128 + (at & 7) * 16;
                    auto put = [](uint32_t addr, const uint4 &v) {
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
                                     "r"(v.w)
                                     : "memory");
                    };
#pragma unroll 1
                    for (int row = valid + (at >> 3); row < end; row += rows)
#pragma unroll
                        for (int x = 0; x < C::kBoxes; ++x)
                            put(mine + (row - (at >> 3)) * 128 + x * C::kBoxBytes, make_uint4(0u, 0u, 0u, 0u));
                    bool odd = false;
                    if (flags & kTree) {
                        // All loads at once, one test for all of them; looked at one by one only if it says so.
                        uint32_t bad = 0;
#pragma unroll
                        for (int k = 0; k < kTileN; k += 16)
                            if (k / 16 * rows + (at >> 3) < valid)
#pragma unroll
                                for (int x = 0; x < C::kBoxes; ++x)
                                    bad |= not_finite8(lds128(mine + k / 16 * rows * 128 + x * C::kBoxBytes));
                        odd = bad != 0;
                        if (odd)
#pragma unroll 1
                            for (int row = at >> 3; row < valid; row += rows)
#pragma unroll 1
                                for (int x = 0; x < C::kBoxes; ++x) {
                                    const uint32_t addr = mine + (row - (at >> 3)) * 128 + x * C::kBoxBytes;
                                    const uint4 v = lds128(addr);
                                    put(addr, make_uint4(finite2(v.x), finite2(v.y), finite2(v.z), finite2(v.w)));
                                }
                    }
                    // A barrier of its own for one and for two streams: the second stream skips tiles without
                    // rows of its own.  Two cleanings of a kind take turns with the word that says what was found.
                    fence_proxy_async_smem();
                    const uint32_t n = two ? cleanings.y++ : cleanings.x++;
                    if (odd) found[2 * two + (n & 1)] = n + 1;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(cleaned + two);
                    ok = tree_wait(cleaned + two, n & 1, p.err_flag);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    dirty |= found[2 * two + (n & 1)] == n + 1;
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(p_full + kBufs * s + buf);
            }
            ++g;
            if (!(flags & kLast)) {
                if (lane == 0) mbar_arrive(meta_free + mt);
                continue;
            }

            // ---- the piece's output ----
            const int first = meta[mt].first, nodes = meta[mt].nodes, dest = meta[mt].dest, h = meta[mt].h;
            const int node_base = meta[mt].node0 + s * tile_nodes;
            __syncwarp();
            if (lane == 0) mbar_arrive(meta_free + mt);
            // Rows leave through shared memory: a lane holds a row, but four lanes store 64 bytes of one,
            // eight rows at a time.  Chunk k of row w is at k ^ (w / 2 % 4): no bank conflicts either way.
            const bool whole = dest < 0;
            const uint32_t mine = smem_addr(stage) + warp * 2048;
            const uint32_t put = mine + lane * 64, put_x = (lane >> 1) & 3;
            const uint32_t get = mine + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
            const int64_t state = (int64_t)dest * (STREAMS * kTileM) + s * kTileM;  // of the stream's row 0
            char *dst[4];  // of the rows this lane stores (NULL: past the last node)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int row = (warp & 3) * 32 + 8 * k + (lane >> 2), n = node_base + (row >> p.group_shift);
                dst[k] = n >= nodes ? nullptr
                         : whole ? reinterpret_cast<char *>(
                                       p.out + ((int64_t)(first + n) * p.q_heads + (h * G + (row & (G - 1)))) * HEAD_DIM)
                                 : reinterpret_cast<char *>(p.part_o + (state + row) * HEAD_DIM);
                if (dst[k]) dst[k] += (lane & 3) * 16;
            }
            auto store64 = [&](int bytes, const uint4 (&v)[4]) {
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(put + ((k ^ put_x) << 4)), "r"(v[k].x),
                                 "r"(v[k].y), "r"(v[k].z), "r"(v[k].w)
                                 : "memory");
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // row 8 k + lane / 4: its swizzle is that of row lane / 4
                    const uint4 x = lds128(get + k * 512);
                    if (dst[k]) *reinterpret_cast<uint4 *>(dst[k] + bytes) = x;
                }
            };
            ok = tree_wait(o_done + s, pieces++ & 1, p.err_flag);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            // The state's two special cases: a NaN or +inf score (l is NaN) gets m = +inf, so that joining
            // pieces keeps it; a row that saw only scores of -inf keeps m = -inf with l = NaN, so that a
            // piece with a finite score outweighs it.  Nothing seen: m = -inf, l = 0.
            if (l != l)
                m = INFINITY;
            else if (m == -INFINITY && seen)
                l = NAN;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            // 32 columns at a time: 128 bytes of a partial state, half of that of a whole unit's bf16 rows
#pragma unroll 1
            for (int q = 0; q < HEAD_DIM / 32; ++q) {
                float o[32];
                __syncwarp();
                tmem_ld32(o_addr + 32 * q, o);
                tmem_wait_ld();
                if (live && dirty) {  // the values that were kept out of the product
#pragma unroll 1
                    for (int k = 0; k < nodes; ++k) {
                        const bool sees = p.masks ? (__ldg(p.masks + (int64_t)(first + node) * p.words + (k >> 5)) >> (k & 31)) & 1
                                                  : k <= node;
                        if (!sees) continue;
                        const uint16_t *src = p.v_tree + (int64_t)(first + k) * p.v_stride + h * HEAD_DIM + 32 * q;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const uint32_t bits = (uint32_t)src[i] << 16;
                            if ((bits & 0x7f800000u) == 0x7f800000u) o[i] += __uint_as_float(bits);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = l == 0.f ? 0.f : o[i] * inv;
                uint4 v[4];
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]), pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                                          pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
                    store64(64 * q, v);
                } else {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] = make_uint4(__float_as_uint(o[16 * x + 4 * i]), __float_as_uint(o[16 * x + 4 * i + 1]),
                                              __float_as_uint(o[16 * x + 4 * i + 2]), __float_as_uint(o[16 * x + 4 * i + 3]));
                        store64(128 * q + 64 * x, v);
                    }
                }
            }
            if (live && !whole)
                *reinterpret_cast<float2 *>(p.part_ml + (state + r) * 2) = make_float2(tree_reference(m, c), l);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free + s);
        }
        if (q_loads > 0) mbar_wait_bounded(q_full + s, (q_loads - 1) & 1, p.err_flag);  // the last copy has landed
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == C::kSoftmaxWarps + 2) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kCols);
    }
}

// Joins the states of the units that were cut:
//   out = sum_p 2^(m_p - M) l_p o_p / sum_p 2^(m_p - M) l_p,  M = max_p m_p.
// CTA (i, y) belongs to the unit inside which cut i + 1 lies.  Where a unit has few pieces the CTAs of its first cut
// join it, 32 rows each, four to a warp.  More pieces have the CTAs of all its cuts, and where that leaves warps over,
// several take the same rows and a part of the pieces each: a sequence alone on the GPU is cut into 40 pieces, and a
// warp that goes through all of them waits for 20 loads in a row (4 sequences of up to 10364 tokens with 8/2 heads of
// 64: 53 us for the whole call, now 31).  The piece before the first cut is the second state of the CTA before, the
// pieces after the cuts are the first states of the CTAs that begin there.
constexpr int kJoinWarps = 8;
constexpr int kJoinRows = 32;
// Pieces that a warp joins alone: where all CTAs of the grid are on the GPU at once, and where they are not and the
// CTAs of the other cuts would only be in the way.  Measured with 2 | 3 | 4 | 8 for the first: 2 sequences of up to
// 13545 tokens with 40/40 heads and 16 rows of each kv head 94.8 | 94.8 | 95.2 | 96.0 us, 16 of up to 4096 with 32/8
// heads 51.8 | 51.7 | 52.2 | 52.0; with 3 | 8 for the second: 4 of up to 8190 with 64/8 heads and 512 rows 88.5 | 87.0.
constexpr int kJoinAlone = 3, kJoinAloneWaves = 8;

template <int HEAD_DIM, int STREAMS>
__global__ void __launch_bounds__(kJoinWarps * 32, 4) tree_join_kernel(const TreeParams p) {
    constexpr int V = HEAD_DIM / 32, R = kJoinRows / kJoinWarps;
    constexpr int kRows = STREAMS * kTileM;
    __shared__ float s_acc[kJoinWarps][R][HEAD_DIM];
    __shared__ float s_state[kJoinWarps][R][3];  // M, den, none
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cut = blockIdx.x + 1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const TreeJoin *unit = p.joins + cut;
    const int pieces = unit->pieces, first = unit->cut0;
    constexpr unsigned kWave = STREAMS == 1 ? 2 : 4;  // rows of this grid that fit the GPU
    const bool shared = pieces > (gridDim.y <= kWave ? kJoinAlone : kJoinAloneWaves);
    if (pieces == 0 || (!shared && cut != first)) return;  // the whole CTA
    const int rows = min((unit->nodes - unit->node0) << p.group_shift, kRows);
    int each = 1;  // warps that share a group of R rows
    int r0 = ((int)blockIdx.y * kJoinWarps + warp) * R;
    if (shared) {
        const int ctas = (pieces - 1) * (int)gridDim.y, groups = (rows + R - 1) / R;
        while (each < kJoinWarps && groups * 2 * each <= ctas * kJoinWarps) each *= 2;
        r0 = (((cut - first) * (int)gridDim.y + (int)blockIdx.y) * kJoinWarps + warp) / each * R;
    }
    if (r0 >= rows && each == 1) return;
    // state of piece k: 2 * first - 1, then 2 * first, 2 * first + 2, ...
    auto state = [&](int k) { return (int64_t)(k == 0 ? 2 * first - 1 : 2 * (first + k - 1)) * kRows + r0; };
    float M[R], den[R], none[R], acc[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        M[r] = -INFINITY;
        den[r] = none[r] = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[r][e] = 0.f;
    }
#pragma unroll 2
    for (int k = r0 < rows ? warp & (each - 1) : pieces; k < pieces; k += each) {
        float2 ml[R];
        float o[R][V];
        // rows past the last node hold whatever the workspace held: they are not stored below
#pragma unroll
        for (int r = 0; r < R; ++r) {
            ml[r] = *(reinterpret_cast<const float2 *>(p.part_ml) + state(k) + r);
            const float *src = p.part_o + (state(k) + r) * HEAD_DIM + lane * V;
            if constexpr (V == 4) {
                const float4 v = *reinterpret_cast<const float4 *>(src);
                o[r][0] = v.x, o[r][1] = v.y, o[r][2] = v.z, o[r][3] = v.w;
            } else {
                const float2 v = *reinterpret_cast<const float2 *>(src);
                o[r][0] = v.x, o[r][1] = v.y;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (ml[r].x == -INFINITY) {  // nothing, or (NaN) only scores of -inf
                none[r] += ml[r].y;
                continue;
            }
            const float top = fmaxf(M[r], ml[r].x);
            const float down = fast_exp2(M[r] - top), w = fast_exp2(ml[r].x - top) * ml[r].y;
            M[r] = top;
            den[r] = den[r] * down + w;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[r][e] = acc[r][e] * down + w * o[r][e];
        }
    }
    if (each > 1) {  // the sums so far are states of their own
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int e = 0; e < V; ++e) s_acc[warp][r][lane * V + e] = acc[r][e];
            if (lane < 3) s_state[warp][r][lane] = lane == 0 ? M[r] : lane == 1 ? den[r] : none[r];
        }
        __syncthreads();
        if ((warp & (each - 1)) != 0 || r0 >= rows) return;
#pragma unroll 1
        for (int w = warp + 1; w < warp + each; ++w)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float m = s_state[w][r][0], top = fmaxf(M[r], m);
                none[r] += s_state[w][r][2];
                if (m == -INFINITY) continue;
                const float down = fast_exp2(M[r] - top), up = fast_exp2(m - top);
                M[r] = top;
                den[r] = den[r] * down + up * s_state[w][r][1];
#pragma unroll
                for (int e = 0; e < V; ++e) acc[r][e] = acc[r][e] * down + up * s_acc[w][r][lane * V + e];
            }
    }
    const int node0 = unit->node0, head0 = unit->h * p.group, row0 = unit->first, nodes = unit->nodes;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = r0 + r, node = node0 + (row >> p.group_shift);
        if (node >= nodes) break;
        uint32_t *dst = reinterpret_cast<uint32_t *>(
            p.out + ((int64_t)(row0 + node) * p.q_heads + head0 + (row & (p.group - 1))) * HEAD_DIM + lane * V);
#pragma unroll
        for (int e = 0; e < V; e += 2)
            dst[e / 2] = M[r] == -INFINITY ? pack_bf16x2(none[r], none[r]) : pack_bf16x2(acc[r][e] / den[r], acc[r][e + 1] / den[r]);
    }
}

}  // namespace
}  // namespace pa
