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
//  * One CTA per (sequence, kv head, row chunk[, partition of the cache]).  A
//    producer warp dereferences the block table and stages 64-token tiles of K
//    and V (and, at the end, of the drafted rows) with TMA into one ring of tiles,
//    in the order in which they are used: K0 K1 V0 K2 V1 ...
//  * One warp issues the products.  S = Q K^T (bf16, fp32 accumulator in TMEM, two
//    buffers, so that the scores of the next tile are ready while this one's
//    softmax runs) and O += P V with P read from TMEM.
//  * Four warps for each 128 rows run the softmax, a row to a thread: no shuffles.
//    P replaces its scores in TMEM as bf16: 8 significant bits for each weight, as
//    many as the values it multiplies have, and as the output keeps; the sum of the
//    weights is fp32 and unrounded.
//  * The running maximum moves only when a score exceeds it by more than 2^8 in
//    weight: O stays in TMEM and is rescaled a few times in a row's life instead of
//    once a tile.  fp32 holds weights up to 2^8 as well as up to 1, and the
//    quotient at the end does not depend on which reference was used.
//  * What a row does not see has no part in it.  Scores are replaced, not added
//    to; V rows past the sequence's end are zeroed in shared memory before they meet
//    a weight of zero; non-finite values of drafted V rows (which some rows see and
//    others do not) are taken out of the product and added at the end to the rows
//    that see them.
#pragma once

#include "pa_common.cuh"

namespace pa {
namespace {

constexpr float kTreeLog2e = 1.4426950408889634f;
constexpr int kTileN = 64;         // tokens of one tile
constexpr int kTileM = 128;        // query rows of one stream
constexpr float kMaxRise = 8.0f;   // log2 of the largest weight before the reference moves

template <int HEAD_DIM, int STREAMS>
struct TreeCfg {
    static constexpr int kBoxes = HEAD_DIM / 64;               // 128-byte wide column boxes
    static constexpr int kBoxBytes = kTileN * 128;             // one box of a K or V tile
    static constexpr int kTileBytes = kBoxes * kBoxBytes;
    static constexpr int kQBoxBytes = kTileM * 128;
    static constexpr int kQBytes = kBoxes * kQBoxBytes;        // one stream's queries
    // Ring depth: two CTAs share an SM with one stream, one CTA has it alone with two.
    static constexpr int kSlots = (STREAMS == 1 ? 4 : 8) * (HEAD_DIM == 64 ? 2 : 1);
    static constexpr int kCtasPerSm = STREAMS == 1 ? 2 : 1;
    static constexpr int kSoftmaxWarps = 4 * STREAMS;
    static constexpr int kThreads = (kSoftmaxWarps + 2) * 32;
    // TMEM of one stream: two score buffers (P in the first half of each), then O.
    static constexpr int kStreamCols = 2 * kTileN + 128;
    static constexpr int kCols = STREAMS * kStreamCols;
    static constexpr int kBars = 2 * kSlots + 1 + STREAMS * 6;
    static constexpr int kDataBytes = STREAMS * kQBytes + kSlots * kTileBytes;
    static constexpr int kSmemBytes = 1024 /* align slack */ + kDataBytes + kBars * 8 + 16;
    static_assert(kCtasPerSm * kCols <= 512, "TMEM columns of an SM");
};

struct TreeParams {
    uint16_t *out;             // [T, Hq, d] bf16
    float *part_o;             // [T, Hq, parts, d]  (split)
    float *part_ml;            // [T, Hq, parts, 2]  (split)
    const uint16_t *v_tree;
    const int32_t *tables, *lens, *cu, *masks;
    int32_t *err_flag;
    int64_t v_stride, num_blocks;
    int num_rows, batch, max_blocks, max_seq_len, max_nodes, words;
    int q_heads, kv_heads, group, block_size;
    int part_tokens, num_parts, chunks;
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
constexpr uint32_t tree_idesc(int n, bool b_transposed) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_transposed ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kTileM >> 4) << 24);
}

// V as the [K = tokens, N = dims] operand: rows of 128 bytes (64 dims) with the 128-byte swizzle, 8-token
// groups 1024 bytes apart, the next 64 dims `box_bytes` further on.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t saddr, uint32_t box_bytes) {
    return (uint64_t)((saddr & 0x3ffffu) >> 4) | ((uint64_t)(box_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
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

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A barrier of the softmax warps of one CTA that also ORs a predicate over them.
template <int THREADS>
__device__ __forceinline__ bool softmax_any(bool mine) {
    uint32_t any;
    __syncwarp();  // an aligned barrier wants whole warps
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.aligned.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)mine), "n"(THREADS)
        : "memory");
    return any != 0;
}

// Whether either bf16 of w is an infinity or NaN.
__device__ __forceinline__ bool not_finite2(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
// w with the halves that are not finite set to zero.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

// The sequence of a CTA, as every kernel of one call sees it.
struct TreeSeq {
    int first, nodes, len;
    bool bad;
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams &p, int b) {
    const int lo = __ldg(p.cu + b), hi = __ldg(p.cu + b + 1), raw = __ldg(p.lens + b);
    TreeSeq s;
    s.first = min(max(lo, 0), p.num_rows);
    const int end = max(min(max(hi, 0), p.num_rows), s.first);
    s.nodes = min(end - s.first, p.max_nodes);
    s.len = min(max(raw, 0), min(p.max_seq_len, p.max_blocks * p.block_size));
    s.bad = s.first != lo || end != hi || s.nodes != end - s.first || s.len != raw;
    return s;
}

template <int HEAD_DIM, int STREAMS>
__global__ void __launch_bounds__(TreeCfg<HEAD_DIM, STREAMS>::kThreads, TreeCfg<HEAD_DIM, STREAMS>::kCtasPerSm)
    tree_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap kt_map,
                const __grid_constant__ CUtensorMap vt_map, const TreeParams p) {
    using C = TreeCfg<HEAD_DIM, STREAMS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint8_t *ring = smem + STREAMS * C::kQBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kDataBytes);
    uint64_t *empty = full + C::kSlots;
    uint64_t *q_full = empty + C::kSlots;
    uint64_t *s_full = q_full + 1;              // [stream][buffer]: scores are in TMEM
    uint64_t *p_full = s_full + 2 * STREAMS;    // [stream][buffer]: weights are in TMEM
    uint64_t *pv_done = p_full + 2 * STREAMS;   // [stream]: a tile has been added to O
    uint64_t *o_done = pv_done + STREAMS;       // [stream]: all of them have
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(o_done + STREAMS);
    volatile int *tree_dirty = reinterpret_cast<volatile int *>(tmem_slot + 1);  // drafted V holds NaN or infinities

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunk = blockIdx.x % p.chunks, part = blockIdx.x / p.chunks;
    const int h = blockIdx.y, b = blockIdx.z;
    const TreeSeq seq = tree_seq(p, b);
    if (seq.bad && threadIdx.x == 0 && blockIdx.x == 0 && h == 0) raise_flag(p.err_flag, PA_FLAG_BAD_LEN);

    // ---- the work: rows [row0, ...) of the sequence, tokens [t0, t1) and (first partition) the tree ----
    const int G = p.group;
    const int tile_nodes = kTileM / G;
    const int node0 = chunk * STREAMS * tile_nodes;
    if (node0 >= seq.nodes) return;
    const int t0 = part * p.part_tokens;
    const int t1 = min(seq.len, t0 + p.part_tokens);
    const int n_ctx = t1 > t0 ? (t1 - t0 + kTileN - 1) / kTileN : 0;
    // a chain's rows see no node after their own
    const int reach = p.masks ? seq.nodes : min(seq.nodes, node0 + STREAMS * tile_nodes);
    const int n_tree = part == 0 ? (reach + kTileN - 1) / kTileN : 0;
    const int n = n_ctx + n_tree;
    if (n == 0) return;
    const int streams = STREAMS == 2 && node0 + tile_nodes < seq.nodes ? 2 : 1;
    const bool whole = seq.len <= p.part_tokens;  // no other partition: the output is written here
    if (p.num_parts > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(q_full, 1);
        for (int s = 0; s < 2 * STREAMS; ++s) {
            mbar_init(s_full + s, 1);
            mbar_init(p_full + s, 4);
        }
        for (int s = 0; s < STREAMS; ++s) {
            mbar_init(pv_done + s, 1);
            mbar_init(o_done + s, 1);
        }
        *tree_dirty = 0;
        fence_mbar_init();
    }
    if (warp == C::kSoftmaxWarps + 1) {
        tmem_alloc(smem_addr(tmem_slot), C::kCols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tmem_slot);

    // Place in the ring of K and V of tile j: K0 K1 V0 K2 V1 ... V(n-2) V(n-1).
    auto k_item = [](int j) { return j + (j > 1 ? j - 1 : 0); };
    auto v_item = [&](int j) { return j + (j + 2 < n ? j + 2 : n); };

    if (warp == C::kSoftmaxWarps) {
        // ---------------- producer: block-table dereference + TMA ----------------
        const int pages = kTileN / p.block_size;          // of one tile
        const int page = lane / C::kBoxes, box = lane % C::kBoxes;
        const int32_t *table = p.tables + (int64_t)b * p.max_blocks;
        const int last = (t1 + p.block_size - 1) / p.block_size;  // blocks of the range end here
        // Block id of this lane's page of tile j: -1 past the range, -2 a bad id.
        auto entry = [&](int j) -> int {
            if (j >= n_ctx || page >= pages) return -1;
            const int at = t0 / p.block_size + j * pages + page;
            if (at >= last) return -1;
            const int id = __ldg(table + at);
            return id < 0 || id >= p.num_blocks ? -2 : id;
        };
        if (lane == 0) {
            mbar_arrive_expect_tx(q_full, streams * C::kQBytes);
            for (int s = 0; s < streams; ++s)
                for (int x = 0; x < C::kBoxes; ++x)
                    tma_load_3d(smem + s * C::kQBytes + x * C::kQBoxBytes, &q_map, x * 64, h * G,
                                seq.first + node0 + s * tile_nodes, q_full);
        }
        const uint64_t policy = l2_policy_evict_first();
        // entries of tiles v, v + 1 (the K beside it), and two more that are on their way
        int e0 = entry(0), e1 = entry(1), e2 = entry(2), e3 = entry(3);
        int v = 0, issued = 0;
        for (int it = 0; it < 2 * n; ++it) {
            const int slot = it % C::kSlots;
            bool ok = true;
            if (it >= C::kSlots) ok = mbar_wait_bounded(empty + slot, (it / C::kSlots - 1) & 1, p.err_flag);
            if (!__all_sync(0xffffffffu, ok)) break;
            const int ahead = (it + 1) >> 1;
            const bool is_k = it == 0 || ((it & 1) && ahead < n);
            const int j = is_k ? ahead : v;
            const int id = is_k && it > 0 ? e1 : e0;
            uint8_t *dst = ring + slot * C::kTileBytes;
            if (j < n_ctx) {
                if (id == -2 && is_k && box == 0) raise_flag(p.err_flag, PA_FLAG_BAD_BLOCK);
                const int loads = __popc(__ballot_sync(0xffffffffu, id != -1));
                if (lane == 0) mbar_arrive_expect_tx(full + slot, loads * p.block_size * 128);
                __syncwarp();
                if (id != -1) {
                    // a bad block reads as zeros (a row outside of the map)
                    const int row = id == -2 ? p.pool_rows : (int)(((int64_t)id * p.kv_heads + h) * p.block_size);
                    tma_load_2d(dst + box * C::kBoxBytes + page * p.block_size * 128, is_k ? &k_map : &v_map, box * 64,
                                row, full + slot, policy);
                }
            } else {
                if (lane == 0) {
                    mbar_arrive_expect_tx(full + slot, C::kTileBytes);
                    for (int x = 0; x < C::kBoxes; ++x)
                        tma_load_3d(dst + x * C::kBoxBytes, is_k ? &kt_map : &vt_map, x * 64, h,
                                    seq.first + (j - n_ctx) * kTileN, full + slot);
                }
            }
            if (!is_k) {
                ++v;
                e0 = e1;
                e1 = e2;
                e2 = e3;
                e3 = entry(v + 3);
            }
            issued = it + 1;
        }
        // Every copy has landed before the CTA ends (they have, unless a wait ran out).
        for (int it = issued > C::kSlots ? issued - C::kSlots : 0; it < issued; ++it)
            if (!mbar_wait_bounded(full + it % C::kSlots, (it / C::kSlots) & 1, p.err_flag)) break;
        mbar_wait_bounded(q_full, 0, p.err_flag);
    } else if (warp == C::kSoftmaxWarps + 1) {
        // ---------------- products ----------------
        const uint32_t q_addr = smem_addr(smem), ring_addr = smem_addr(ring);
        constexpr uint32_t kQkDesc = tree_idesc(kTileN, false), kPvDesc = tree_idesc(HEAD_DIM, true);
        auto all_ok = [&](bool ok) { return __all_sync(0xffffffffu, ok); };
        auto wait_item = [&](int it) {
            return all_ok(mbar_wait_bounded(full + it % C::kSlots, (it / C::kSlots) & 1, p.err_flag));
        };
        // S[stream][j & 1] = Q K_j^T
        auto scores = [&](int j, int s) {
            const uint32_t k0 = ring_addr + (k_item(j) % C::kSlots) * C::kTileBytes;
            const uint32_t d = tmem + s * C::kStreamCols + (j & 1) * kTileN;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < HEAD_DIM / 16; ++i)
                umma_bf16_ss(d, umma_desc_k_sw128(q_addr + s * C::kQBytes + (i >> 2) * C::kQBoxBytes + (i & 3) * 32),
                             umma_desc_k_sw128(k0 + (i >> 2) * C::kBoxBytes + (i & 3) * 32), kQkDesc, i > 0);
            umma_commit(s_full + 2 * s + (j & 1));
        };
        bool ok = all_ok(mbar_wait_bounded(q_full, 0, p.err_flag));
        for (int j = 0; ok && j < min(2, n); ++j) {
            ok = wait_item(k_item(j));
            if (ok && lane == 0) {
                for (int s = 0; s < streams; ++s) scores(j, s);
                umma_commit(empty + k_item(j) % C::kSlots);
            }
            __syncwarp();
        }
        for (int j = 0; ok && j < n; ++j) {
            const int slot = v_item(j) % C::kSlots;
            if (!(ok = wait_item(v_item(j)))) break;
            const uint32_t v0 = ring_addr + slot * C::kTileBytes;
            const int rows = j < n_ctx ? t1 - t0 - j * kTileN : reach - (j - n_ctx) * kTileN;
            if (rows < kTileN) {  // rows past the end: zeros, whatever the ring held
                for (int x = lane; x < (kTileN - rows) * 8 * C::kBoxes; x += 32) {
                    const int bx = x / ((kTileN - rows) * 8), y = x - bx * (kTileN - rows) * 8;
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v0 + bx * C::kBoxBytes +
                                                                                   rows * 128 + y * 16),
                                 "r"(0u)
                                 : "memory");
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            for (int s = 0; ok && s < streams; ++s) {
                ok = all_ok(mbar_wait_bounded(p_full + 2 * s + (j & 1), (j >> 1) & 1, p.err_flag));
                if (!ok) break;
                if (s == 0 && j >= n_ctx && *tree_dirty) {
                    for (int x = lane; x < C::kTileBytes / 16; x += 32) {
                        const uint4 w = lds128(v0 + x * 16);
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(v0 + x * 16), "r"(finite2(w.x)),
                                     "r"(finite2(w.y)), "r"(finite2(w.z)), "r"(finite2(w.w))
                                     : "memory");
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) {
                    tc_fence_after();
                    const uint32_t base = tmem + s * C::kStreamCols;
#pragma unroll
                    for (int i = 0; i < kTileN / 16; ++i)
                        umma_bf16_ts(base + 2 * kTileN, base + (j & 1) * kTileN + 8 * i,
                                     umma_desc_mn_sw128(v0 + i * 2048, C::kBoxBytes), kPvDesc, j > 0 || i > 0);
                    umma_commit(j + 1 < n ? pv_done + s : o_done + s);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (lane == 0) umma_commit(empty + slot);
            if (j + 2 < n) {
                if (!(ok = wait_item(k_item(j + 2)))) break;
                for (int s = 0; s < streams; ++s) {
                    // the new scores take the place of P_j: its product has to be done
                    ok = all_ok(mbar_wait_bounded(pv_done + s, j & 1, p.err_flag));
                    if (!ok) break;
                    if (lane == 0) scores(j + 2, s);
                    __syncwarp();
                }
                if (lane == 0) umma_commit(empty + k_item(j + 2) % C::kSlots);
            }
            __syncwarp();
        }
        // Every product has completed before TMEM is freed.
        for (int s = 0; ok && s < streams; ++s) ok = mbar_wait_bounded(o_done + s, 0, p.err_flag);
    } else if (warp < 4 * streams) {
        // ---------------- softmax: one row to a thread ----------------
        const int s = warp >> 2;
        const int r = threadIdx.x & (kTileM - 1);
        const int node = node0 + s * tile_nodes + r / G;
        const bool live = node < seq.nodes;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t base = tmem + s * C::kStreamCols + lanes;
        const uint32_t o_addr = base + 2 * kTileN;

        // While the first tiles are on their way: do drafted V rows hold values that must not meet a
        // weight of zero, and does the block table name blocks that are not there?
        bool dirty = false, holes = false;
        constexpr int kVecs = HEAD_DIM / 8;
        if (n_tree) {
            for (int x = threadIdx.x; x < reach * kVecs; x += 128 * streams) {
                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p.v_tree + (int64_t)(seq.first + x / kVecs) * p.v_stride +
                                                                      h * HEAD_DIM) + x % kVecs);
                dirty |= not_finite2(w.x) || not_finite2(w.y) || not_finite2(w.z) || not_finite2(w.w);
            }
        }
        const int32_t *table = p.tables + (int64_t)b * p.max_blocks;
        for (int at = t0 / p.block_size + threadIdx.x; at < (t1 + p.block_size - 1) / p.block_size; at += 128 * streams) {
            const int id = __ldg(table + at);
            holes |= id < 0 || id >= p.num_blocks;
        }
        if (streams == STREAMS) {
            dirty = softmax_any<128 * STREAMS>(dirty);
            holes = softmax_any<128 * STREAMS>(holes);
        } else {
            dirty = softmax_any<128>(dirty);
            holes = softmax_any<128>(holes);
        }
        if (dirty && threadIdx.x == 0) *tree_dirty = 1;  // before this thread's first arrival on p_full

        // a negative scale turns the order of the scores around; a scale of 0 must not meet -inf
        const bool flip = p.scale_log2 < 0.f;
        const float c = p.scale_log2 == 0.f ? 1e-30f : fabsf(p.scale_log2);
        const float rise = kMaxRise / c;
        float m = -INFINITY, l = 0.f;
        bool seen = false;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            // the tokens of the tile that this row sees
            uint32_t see[2] = {0xffffffffu, 0xffffffffu};
            if (j < n_ctx) {
                const int left = t1 - t0 - j * kTileN;
                if (left < kTileN) {
                    see[0] = left >= 32 ? 0xffffffffu : (1u << left) - 1;
                    see[1] = left <= 32 ? 0u : (1u << (left - 32)) - 1;
                }
                if (holes) {
                    const int at = (t0 + j * kTileN) / p.block_size;
                    for (int x = 0; x * p.block_size < min(left, kTileN); ++x) {
                        const int id = __ldg(table + at + x);
                        if (id < 0 || id >= p.num_blocks)
                            for (int t = x * p.block_size; t < (x + 1) * p.block_size; ++t) see[t >> 5] &= ~(1u << (t & 31));
                    }
                }
            } else {
                const int at = (j - n_ctx) * kTileN;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int first = at + 32 * w;  // the word's first node
                    uint32_t bits = 0u;
                    if (live && first < seq.nodes) {
                        if (p.masks)
                            bits = (uint32_t)__ldg(p.masks + (int64_t)(seq.first + node) * p.words + (first >> 5));
                        else
                            bits = node < first ? 0u : node - first >= 31 ? 0xffffffffu : (2u << (node - first)) - 1;
                        if (seq.nodes - first < 32) bits &= (1u << (seq.nodes - first)) - 1;
                    }
                    see[w] = bits;
                }
            }
            seen |= (see[0] | see[1]) != 0;

            ok = mbar_wait_bounded(s_full + 2 * s + (j & 1), (j >> 1) & 1, p.err_flag);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            __syncwarp();
            tc_fence_after();
            const uint32_t s_addr = base + (j & 1) * kTileN;
            float x[kTileN];
            tmem_ld32(s_addr, x);
            tmem_ld32(s_addr + 32, x + 32);
            tmem_wait_ld();
            if (flip) {
#pragma unroll
                for (int i = 0; i < kTileN; ++i) x[i] = -x[i];
            }
            if (!__all_sync(0xffffffffu, (see[0] & see[1]) == 0xffffffffu)) {
#pragma unroll
                for (int i = 0; i < kTileN; ++i)
                    x[i] = (see[i >> 5] >> (i & 31)) & 1u ? x[i] : -INFINITY;
            }
            float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int i = 4; i < kTileN; ++i) top[i & 3] = fmaxf(top[i & 3], x[i]);
            const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            if (__any_sync(0xffffffffu, mt > m + rise)) {
                const float next = fmaxf(m, mt);
                const float down = next == -INFINITY ? 1.f : fast_exp2((m - next) * c);
                m = next;
                l *= down;
                if (j > 0) {  // O has been written: wait for the last product, then rescale it
                    ok = mbar_wait_bounded(pv_done + s, (j - 1) & 1, p.err_flag);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int q = 0; q < HEAD_DIM / 32; ++q) {
                        float o[32];
                        tmem_ld32(o_addr + 32 * q, o);
                        tmem_wait_ld();
                        uint32_t w[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i] * down);
                        tmem_st32(o_addr + 32 * q, w);
                    }
                }
            }
            const float bias = m == -INFINITY ? 0.f : -m * c;
            uint32_t w[kTileN / 2];
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kTileN; i += 2) {
                const float p0 = fast_exp2(fmaf(x[i], c, bias)), p1 = fast_exp2(fmaf(x[i + 1], c, bias));
                sum[i & 2] += p0;
                sum[(i & 2) + 1] += p1;
                w[i / 2] = pack_bf16x2(p0, p1);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_st32(s_addr, w);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + 2 * s + (j & 1));
        }
        // A barrier of its own: pv_done may be one or two phases ahead of this thread by now, and a
        // parity tells only neighbouring phases apart.
        if (ok) ok = mbar_wait_bounded(o_done + s, 0, p.err_flag);
        if (__all_sync(0xffffffffu, ok)) {
            tc_fence_after();
            // The state's two special cases: a NaN or +inf score (l is NaN) gets m = +inf, so that joining
            // partitions keeps it; a row that saw only scores of -inf keeps m = -inf with l = NaN, so
            // that a partition with a finite score outweighs it.  Nothing seen: m = -inf, l = 0.
            if (l != l)
                m = INFINITY;
            else if (m == -INFINITY && seen)
                l = NAN;
            const int64_t row = (int64_t)(seq.first + node) * p.q_heads + h * G + r % G;
            const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
            for (int q = 0; q < HEAD_DIM / 32; ++q) {
                float o[32];
                __syncwarp();
                tmem_ld32(o_addr + 32 * q, o);
                tmem_wait_ld();
                if (live && dirty) {  // the values that were kept out of the product
                    for (int k = 0; k < reach; ++k) {
                        const bool sees = p.masks ? (__ldg(p.masks + (int64_t)(seq.first + node) * p.words + (k >> 5)) >> (k & 31)) & 1
                                                  : k <= node;
                        if (!sees) continue;
                        const uint16_t *src = p.v_tree + (int64_t)(seq.first + k) * p.v_stride + h * HEAD_DIM + 32 * q;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const uint32_t bits = (uint32_t)src[i] << 16;
                            if ((bits & 0x7f800000u) == 0x7f800000u) o[i] += __uint_as_float(bits);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = l == 0.f ? 0.f : o[i] * inv;
                if (live && whole) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + row * HEAD_DIM + 32 * q);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dst[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]), pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                                            pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
                } else if (live) {
                    float4 *dst = reinterpret_cast<float4 *>(p.part_o + (row * p.num_parts + part) * HEAD_DIM + 32 * q);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
            }
            if (live && !whole)
                *reinterpret_cast<float2 *>(p.part_ml + (row * p.num_parts + part) * 2) = make_float2(m == -INFINITY ? m : m * c, l);
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == C::kSoftmaxWarps + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kCols);
    }
}

// Joins the partitions of one (row, query head), one to a warp:
//   out = sum_p 2^(m_p - M) l_p o_p / sum_p 2^(m_p - M) l_p,  M = max_p m_p.
constexpr int kTreeReduceWarps = 8;

template <int HEAD_DIM>
__global__ void __launch_bounds__(kTreeReduceWarps * 32) tree_reduce_kernel(const TreeParams p) {
    constexpr int V = HEAD_DIM / 32;
    const int lane = threadIdx.x & 31;
    const int item = blockIdx.x * kTreeReduceWarps + (threadIdx.x >> 5);
    const TreeSeq seq = tree_seq(p, blockIdx.y);
    const int parts = (seq.len + p.part_tokens - 1) / p.part_tokens;
    if (parts <= 1 || item >= seq.nodes * p.q_heads) return;  // written by the attention itself
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = (int64_t)seq.first * p.q_heads + item;
    const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml) + row * p.num_parts;
    const float *po = p.part_o + row * p.num_parts * HEAD_DIM + lane * V;
    float M = -INFINITY, none = 0.f;
    for (int i = lane; i < parts; i += 32) {
        const float2 s = ml[i];
        M = fmaxf(M, s.x);
        none += s.x == -INFINITY ? s.y : 0.f;  // NaN where all scores of a partition were -inf
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        none += __shfl_xor_sync(0xffffffffu, none, off);
    }
    float acc[V], den = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    if (M != -INFINITY) {
#pragma unroll 4
        for (int i = 0; i < parts; ++i) {
            const float2 s = ml[i];
            const float w = s.x == -INFINITY ? 0.f : fast_exp2(s.x - M) * s.y;
            if (s.x != -INFINITY) {
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] += w * po[(int64_t)i * HEAD_DIM + e];
            }
            den += w;
        }
    }
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + row * HEAD_DIM + lane * V);
#pragma unroll
    for (int e = 0; e < V; e += 2)
        dst[e / 2] = M == -INFINITY ? pack_bf16x2(none, none) : pack_bf16x2(acc[e] / den, acc[e + 1] / den);
}

}  // namespace
}  // namespace pa
