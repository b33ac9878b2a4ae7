// Block tables, slot maps and tree masks built on the device.
//
// All of it is integer bookkeeping of a few bytes for each token: bound by
// launch and memory latency, not by bandwidth, so what counts is the number of
// launches and of dependent loads.
#include "pa_common.cuh"

namespace pa {
namespace {

// ---------------------------------------------------------------------------
// Table growth
// ---------------------------------------------------------------------------

// One CTA reads all lengths (they are needed as a whole: block offsets are a
// prefix sum, and nothing may be written before the total is known to fit),
// kPlanThreads sequences at a time.
constexpr int kPlanThreads = 1024;
// Rows that the planning CTA maps itself; more rows go to a second launch over
// the whole GPU.  Measured (64 sequences, calls back to back): 512 rows 6.2 us of
// GPU time here, 8.3 with the second launch; 4096 rows 8.3 and 8.2, of which the
// host's 9.7 and 11.8 hide both; 8192 rows 12.4 and 8.3; 32768 rows 36 and 8.3.
constexpr int kPlanRows = 4 * kPlanThreads;
constexpr int kMapThreads = 256;

struct ExtendParams {
    int32_t *tables;
    const int32_t *lens, *add;
    int32_t *lens_out;
    const int32_t *free_blocks, *cursor;
    int32_t *cursor_out, *slots, *positions, *cu;
    const int32_t *cu_rows, *path;
    int32_t *err_flag;
    int64_t num_blocks;
    int max_blocks, batch, block_size, num_free, num_rows, max_path;
    int map_here;  // the planning CTA maps the rows too
};

// Exclusive prefix sums of (tokens, blocks) over the CTA, and their totals.
__device__ __forceinline__ void scan2(int tokens, int blocks, int64_t &tok_before, int64_t &blk_before,
                                      int64_t &tok_total, int64_t &blk_total) {
    __shared__ int64_t s_tok[kPlanThreads / 32], s_blk[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t t = tokens, b = blocks;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t tu = __shfl_up_sync(0xffffffffu, t, off), bu = __shfl_up_sync(0xffffffffu, b, off);
        if (lane >= off) {
            t += tu;
            b += bu;
        }
    }
    __syncthreads();  // the previous call's totals have been read
    if (lane == 31) {
        s_tok[warp] = t;
        s_blk[warp] = b;
    }
    __syncthreads();
    if (warp == 0) {
        int64_t x = s_tok[lane], y = s_blk[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t xu = __shfl_up_sync(0xffffffffu, x, off), yu = __shfl_up_sync(0xffffffffu, y, off);
            if (lane >= off) {
                x += xu;
                y += yu;
            }
        }
        s_tok[lane] = x;
        s_blk[lane] = y;
    }
    __syncthreads();
    tok_before = t - tokens + (warp ? s_tok[warp - 1] : 0);
    blk_before = b - blocks + (warp ? s_blk[warp - 1] : 0);
    tok_total = s_tok[kPlanThreads / 32 - 1];
    blk_total = s_blk[kPlanThreads / 32 - 1];
}

// The largest i in [0, n) with a[i] <= x (a[0] <= x), a nondecreasing.
template <typename Get>
__device__ __forceinline__ int last_at_most(Get a, int n, int64_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a(mid) <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Slot and position of row r, from the tables, lengths and counts already written.
__device__ __forceinline__ void map_row(const ExtendParams &p, int r) {
    int64_t slot = -1;
    int at = 0;
    int b = -1, k = 0;  // the row holds new token k of sequence b
    if (p.cu_rows == nullptr) {
        if (r < p.cu[p.batch]) {
            b = last_at_most([&](int i) { return p.cu[i]; }, p.batch, r);
            k = r - p.cu[b];
        }
    } else if (r >= __ldg(p.cu_rows) && r < __ldg(p.cu_rows + p.batch)) {
        const int s = last_at_most([&](int i) { return __ldg(p.cu_rows + i); }, p.batch, r);
        const int node = r - __ldg(p.cu_rows + s);
        const int n = p.cu[s + 1] - p.cu[s];
        for (k = 0; k < n; ++k)
            if (__ldg(p.path + (int64_t)s * p.max_path + k) == node) {
                b = s;
                break;
            }
    }
    if (b >= 0) {
        at = p.lens_out[b] - (p.cu[b + 1] - p.cu[b]) + k;
        const int64_t phys = p.tables[(int64_t)b * p.max_blocks + at / p.block_size];
        if (phys < 0 || phys >= p.num_blocks)
            raise_flag(p.err_flag, PA_FLAG_BAD_BLOCK);
        else
            slot = phys * p.block_size + at % p.block_size;
    }
    p.slots[r] = (int32_t)slot;
    if (p.positions) p.positions[r] = at;
}

// 14 us together with the mapping launch for 64 prompts of up to 4096 tokens (131072 rows, 0.2 us of bytes): each
// step of the plan waits for the one before (lengths, sums, list, table, sums, slots).
// Pass 1 adds up the tokens and blocks of all sequences; pass 2 scans them again
// and writes lengths, counts and table entries.  Batches of up to kPlanThreads
// sequences stay in registers between the two.
__global__ void __launch_bounds__(kPlanThreads, 1) extend_plan_kernel(const ExtendParams p) {
    __shared__ int s_blk[kPlanThreads + 1];  // blocks taken before each sequence of this chunk
    __shared__ int s_old[kPlanThreads];      // entries its table had
    const int cursor = *p.cursor;  // may be cursor_out
    const int64_t cap = (int64_t)p.max_blocks * p.block_size;
    int len = 0, add = 0, blocks = 0;
    int unordered = 0;  // bounds of drafted rows that decrease or leave the rows: a token could miss its row
    int64_t tok_before = 0, blk_before = 0, tok_total, blk_total;
    auto read = [&](int b, bool report) {
        len = add = blocks = 0;
        if (b >= p.batch) return;
        len = p.lens[b];  // may be lens_out: read before any write of this sequence
        add = __ldg(p.add + b);
        bool ok = len >= 0 && add >= 0 && (int64_t)len + add <= cap;
        if (p.path && report) {
            const int lo = __ldg(p.cu_rows + b), hi = __ldg(p.cu_rows + b + 1);
            unordered |= lo < 0 || hi < lo || hi > p.num_rows;
        }
        if (p.path && ok) {  // as many tokens as the path has names: one without a row would leave a hole in the cache
            ok = add <= p.max_path;
            int least = 0;  // no early end: the loads do not wait for each other
#pragma unroll 8
            for (int k = 0; k < (ok ? add : 0); ++k) least = min(least, __ldg(p.path + (int64_t)b * p.max_path + k));
            ok &= least >= 0;
        }
        if (!ok) {
            if (report) raise_flag(p.err_flag, PA_FLAG_BAD_LEN);
            add = 0;
        }
        if (add > 0) blocks = (len + add + p.block_size - 1) / p.block_size - (len + p.block_size - 1) / p.block_size;
    };
    const int chunks = (p.batch + kPlanThreads - 1) / kPlanThreads;
    int64_t all_tok = 0, all_blk = 0;
    for (int c = 0; c < chunks; ++c) {
        read(c * kPlanThreads + threadIdx.x, true);
        scan2(add, blocks, tok_before, blk_before, tok_total, blk_total);
        all_tok += tok_total;
        all_blk += blk_total;
    }
    int bad = p.path && __syncthreads_or(unordered) ? PA_FLAG_BAD_LEN : 0;
    if (cursor < 0 || cursor + all_blk > p.num_free) bad |= PA_FLAG_NO_BLOCKS;
    if (all_tok > (p.path ? (int64_t)INT32_MAX : (int64_t)p.num_rows)) bad |= PA_FLAG_BAD_LEN;
    if (bad && threadIdx.x == 0) raise_flag(p.err_flag, bad);

    int64_t tok0 = 0, blk0 = 0;
    for (int c = 0; c < chunks; ++c) {
        const int b = c * kPlanThreads + threadIdx.x;
        if (chunks > 1) {
            read(b, false);
            scan2(add, blocks, tok_before, blk_before, tok_total, blk_total);
        }
        const int kept = bad ? 0 : add;
        if (b < p.batch) {
            p.lens_out[b] = len + kept;
            p.cu[b] = bad ? 0 : (int32_t)(tok0 + tok_before);
            if (b == p.batch - 1) p.cu[p.batch] = bad ? 0 : (int32_t)(tok0 + tok_before + add);
        }
        if (!bad) {
            s_blk[threadIdx.x] = (int)blk_before;
            s_old[threadIdx.x] = (len > 0 ? len + p.block_size - 1 : 0) / p.block_size;
            __syncthreads();
            const int n = min(kPlanThreads, p.batch - c * kPlanThreads);
            for (int e = threadIdx.x; e < (int)blk_total; e += kPlanThreads) {
                const int s = last_at_most([&](int i) { return s_blk[i]; }, n, e);
                const int32_t id = __ldg(p.free_blocks + cursor + blk0 + e);
                if (id < 0 || id >= p.num_blocks) raise_flag(p.err_flag, PA_FLAG_BAD_BLOCK);
                p.tables[(int64_t)(c * kPlanThreads + s) * p.max_blocks + s_old[s] + e - s_blk[s]] = id;
            }
        }
        tok0 += tok_total;
        blk0 += blk_total;
        __syncthreads();
    }
    if (threadIdx.x == 0) *p.cursor_out = cursor + (bad ? 0 : (int)all_blk);
    if (p.map_here)
        for (int r = threadIdx.x; r < p.num_rows; r += kPlanThreads) map_row(p, r);
}

__global__ void __launch_bounds__(kMapThreads) extend_map_kernel(const ExtendParams p) {
    // The plan has been written.  Nothing triggers this launch before the plan's end, so that only its set-up overlaps.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int r = blockIdx.x * kMapThreads + threadIdx.x;
    if (r < p.num_rows) map_row(p, r);
}

// ---------------------------------------------------------------------------
// Tree masks
// ---------------------------------------------------------------------------

constexpr int kMaskThreads = 256;
// CTAs for each SM (two rounds of eight) before one takes several sequences: the bounds before a CTA's sequences are
// read by all of them.  Measured (calls back to back) with one sequence to a CTA | 8 | 16 CTAs: 1200 trees of 100
// 6.5 | 8.1 | 6.5 us, 4096 of 8 10.1 | 8.4 | 9.1, 65536 of 2 462 | 85 | 88.
constexpr int kMaskCtasPerSm = 16;

// 6.2 us for 256 trees of up to 256 nodes alone, 7.0 in a row (0.3 us of bytes; an empty launch of this size takes 4).
// A CTA for each sequence, or for several in turn where there are many: every thread walks the
// ancestors of its nodes, which takes as many steps as the tree is deep, and sets their bits in a mask row of its own.
// Item `batch` clears the rows that belong to no sequence.
__global__ void __launch_bounds__(kMaskThreads) tree_masks_kernel(
    int32_t *__restrict__ masks, int32_t *__restrict__ positions, const int32_t *__restrict__ parents,
    const int32_t *__restrict__ cu, const int32_t *__restrict__ lens, int batch, int num_rows, int max_nodes,
    int words, int per_cta, int32_t *__restrict__ err_flag) {
    extern __shared__ int32_t s_tree[];
    int32_t *s_parent = s_tree;             // [max_nodes]
    int32_t *s_mask = s_tree + max_nodes;   // [max_nodes, words]
    __shared__ int s_floor;
    auto bound = [&](int i) { return min(max(__ldg(cu + i), 0), num_rows); };
    auto clear = [&](int lo, int hi) {
        for (int64_t x = (int64_t)lo * words + threadIdx.x; x < (int64_t)hi * words; x += kMaskThreads) masks[x] = 0;
        if (positions)
            for (int r = lo + threadIdx.x; r < hi; r += kMaskThreads) positions[r] = 0;
    };
    const unsigned b0 = blockIdx.x * per_cta, b1 = min(b0 + per_cta, batch + 1u);
    int top = 0;  // of the earlier bounds, over all threads
    for (unsigned j = threadIdx.x; j < b0; j += kMaskThreads) top = max(top, bound(j));
    for (unsigned x = b0; x < b1; ++x) {
        const int b = (int)x;
        // Each row is written by one CTA, whatever the bounds: the rows of sequence b begin at the largest of bounds
        // 0 .. b.  A sequence that begins below an earlier bound would lose its first nodes there and is left without
        // any.  Its nodes' parents are read before that is known.
        const int lo = bound(b), hi = b < batch ? bound(b + 1) : lo;
        int n = min(max(hi - lo, 0), max_nodes);
        bool late = false;
        for (int i = threadIdx.x; i < n; i += kMaskThreads) {
            int parent = __ldg(parents + lo + i);
            if (parent < -1 || parent >= i) {
                late = true;
                parent = -1;
            }
            s_parent[i] = parent;
        }
        int start = lo;
        if (__syncthreads_or(top > lo)) {
            if (threadIdx.x == 0) s_floor = 0;
            __syncthreads();
            atomicMax(&s_floor, top);
            __syncthreads();
            start = s_floor;
            n = 0;
            late = false;
        }
        top = max(top, lo);
        if (b == batch) {
            clear(0, bound(0));
            clear(start, num_rows);
            return;
        }
        const int end = max(hi, start);
        if (threadIdx.x == 0 && (start != __ldg(cu + b) || end != __ldg(cu + b + 1) || n != end - start))
            raise_flag(err_flag, PA_FLAG_BAD_LEN);
        if (late) raise_flag(err_flag, PA_FLAG_BAD_TREE);
        for (int i = threadIdx.x; i < n; i += kMaskThreads) {
            int32_t *row = s_mask + i * words;
            for (int w = 0; w < words; ++w) row[w] = 0;
            int depth = -1;
            for (int j = i; j >= 0; j = s_parent[j]) {  // parents come first: the walk ends
                row[j >> 5] |= 1u << (j & 31);
                ++depth;
            }
            if (positions) positions[lo + i] = __ldg(lens + b) + depth;
        }
        __syncthreads();
        for (int x = threadIdx.x; x < n * words; x += kMaskThreads) masks[(int64_t)lo * words + x] = s_mask[x];
        clear(start + n, end);
    }
}

}  // namespace
}  // namespace pa

extern "C" {

int pa_extend_tables(int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens,
                     const int32_t *add_lens, int32_t *seq_lens_out, int batch, int block_size,
                     int64_t num_blocks, const int32_t *free_blocks, int num_free, const int32_t *free_cursor,
                     int32_t *free_cursor_out, int32_t *slot_mapping, int32_t *positions, int32_t *cu_tokens,
                     int num_rows, const int32_t *cu_rows, const int32_t *path, int max_path,
                     int32_t *err_flag, void *stream) {
    if (batch < 0 || max_blocks_per_seq < 0 || num_blocks <= 0 || num_free < 0 || num_rows < 0 || max_path < 0)
        return PA_ERR_INVALID_ARG;
    if (!pa::supported_block_size(block_size)) return PA_ERR_UNSUPPORTED;
    if (num_blocks > INT32_MAX / block_size) return PA_ERR_INVALID_ARG;  // a slot is an int32
    // a length is an int32, and so is one rounded up to whole blocks
    if ((int64_t)max_blocks_per_seq * block_size > INT32_MAX - block_size) return PA_ERR_INVALID_ARG;
    if ((cu_rows == nullptr) != (path == nullptr)) return PA_ERR_INVALID_ARG;
    if (batch == 0) return PA_OK;
    if (!seq_lens || !add_lens || !seq_lens_out || !free_cursor || !free_cursor_out || !cu_tokens)
        return PA_ERR_INVALID_ARG;
    if ((max_blocks_per_seq > 0 && !block_tables) || (num_free > 0 && !free_blocks) || (num_rows > 0 && !slot_mapping))
        return PA_ERR_INVALID_ARG;
    pa::ExtendParams p{};
    p.tables = block_tables;
    p.lens = seq_lens;
    p.add = add_lens;
    p.lens_out = seq_lens_out;
    p.free_blocks = free_blocks;
    p.cursor = free_cursor;
    p.cursor_out = free_cursor_out;
    p.slots = slot_mapping;
    p.positions = positions;
    p.cu = cu_tokens;
    p.cu_rows = cu_rows;
    p.path = path;
    p.err_flag = err_flag;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.batch = batch;
    p.block_size = block_size;
    p.num_free = num_free;
    p.num_rows = num_rows;
    p.max_path = max_path;
    p.map_here = num_rows <= pa::kPlanRows;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    pa::extend_plan_kernel<<<1, pa::kPlanThreads, 0, s>>>(p);
    pa::count_launch();
    const int st = pa::launch_status();
    if (st != PA_OK || p.map_here) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((num_rows + pa::kMapThreads - 1) / pa::kMapThreads));
    cfg.blockDim = dim3(pa::kMapThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, pa::extend_map_kernel, p);
    pa::count_launch();
    return e == cudaSuccess ? pa::launch_status() : PA_ERR_CUDA;
}

int pa_tree_masks(int32_t *masks, int32_t *positions, const int32_t *parents, const int32_t *cu_nodes,
                  const int32_t *seq_lens, int batch, int num_rows, int max_nodes, int32_t *err_flag,
                  void *stream) {
    if (batch < 0 || num_rows < 0 || max_nodes < 0) return PA_ERR_INVALID_ARG;
    if (max_nodes > PA_TREE_MAX_NODES) return PA_ERR_UNSUPPORTED;
    if (batch == 0 || num_rows == 0) return PA_OK;
    if (max_nodes == 0 || !masks || !parents || !cu_nodes || !seq_lens) return PA_ERR_INVALID_ARG;
    const int words = (max_nodes + 31) / 32;
    const size_t smem = (size_t)max_nodes * (words + 1) * 4;
    static_assert(PA_TREE_MAX_NODES * (PA_TREE_MAX_NODES / 32 + 1) * 4 <= 48 * 1024, "fits without an opt-in");
    const int per_cta = batch / (pa::kMaskCtasPerSm * pa::device_sm_count()) + 1;
    pa::tree_masks_kernel<<<(unsigned)(batch / per_cta) + 1, pa::kMaskThreads, smem, static_cast<cudaStream_t>(stream)>>>(
        masks, positions, parents, cu_nodes, seq_lens, batch, num_rows, max_nodes, words, per_cta, err_flag);
    pa::count_launch();
    return pa::launch_status();
}

}  // extern "C"
