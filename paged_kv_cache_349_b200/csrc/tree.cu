// Host side of the attention of drafted tokens: tensor maps, the split over the
// cache's length, the workspace and the launches (the device code is in
// tree_kernels.cuh).
#include <mutex>

#include "tree_kernels.cuh"

namespace pa {
namespace {

using EncodeTiledFn = decltype(&cuTensorMapEncodeTiled);

EncodeTiledFn tree_encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

// bf16 tensor of `rank` dimensions, innermost first, read in boxes of 64 values
// with the 128-byte swizzle; strides in bytes from the second dimension on.
bool tree_map(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
              const cuuint32_t *box) {
    EncodeTiledFn enc = tree_encode_fn();
    if (!enc) return false;
    const cuuint32_t step[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows [num_rows, heads, head_dim] at a row stride, read as `box_rows` rows of `box_heads` heads.
bool tree_rows_map(CUtensorMap *map, const void *base, int64_t stride, int num_rows, int heads, int head_dim,
                   int box_heads, int box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)num_rows};
    const cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    return tree_map(map, base, 3, dims, strides, box);
}

bool tree_pool_map(CUtensorMap *map, const void *base, uint64_t rows, int head_dim, int block_size) {
    const cuuint64_t dims[2] = {(cuuint64_t)head_dim, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)head_dim * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)block_size};
    return tree_map(map, base, 2, dims, strides, box);
}

// More than 128 query rows of a kv head: two streams of 128 rows share each K and V tile.
int tree_streams(int max_nodes, int group) { return (int64_t)max_nodes * group > kTileM ? 2 : 1; }

int tree_chunks(int max_nodes, int group) {
    const int nodes = tree_streams(max_nodes, group) * (kTileM / group);
    return (max_nodes + nodes - 1) / nodes;
}

// Tokens of one partition, -1 for no split.  The default weighs whole waves of
// CTAs: each costs its share of the cache plus kFixed tokens' worth of start and end.
int tree_partition(int batch, int num_q_heads, int num_kv_heads, int max_seq_len, int max_nodes, int requested) {
    if (requested < 0) return -1;
    if (requested > 0) return requested >= max_seq_len ? -1 : requested;
    const int group = num_q_heads / num_kv_heads;
    const int64_t units = (int64_t)batch * num_kv_heads * tree_chunks(max_nodes, group);
    const int64_t resident = (int64_t)device_sm_count() * (tree_streams(max_nodes, group) == 1 ? 2 : 1);
    constexpr int64_t kFixed = 256;
    int best = -1;
    int64_t best_cost = 0;
    for (int parts = 1; parts <= 64; ++parts) {
        const int64_t tokens = ((max_seq_len + parts - 1) / parts + 127) / 128 * 128;
        if (parts > 1 && tokens < 256) break;
        const int64_t cost = (units * parts + resident - 1) / resident * (tokens + kFixed);
        if (best < 0 || cost < best_cost) {
            best = (int)tokens;
            best_cost = cost;
        }
    }
    return best >= max_seq_len ? -1 : best;
}

struct TreeLayout {
    size_t ml, total;
};

TreeLayout tree_layout(int num_rows, int num_q_heads, int head_dim, int64_t parts) {
    const int64_t rows = (int64_t)num_rows * num_q_heads * parts;
    TreeLayout l{};
    l.ml = (size_t)((rows * head_dim * 4 + 255) / 256 * 256);
    l.total = l.ml + (size_t)(rows * 2 * 4);
    return l;
}

struct TreeMaps {
    CUtensorMap q, k, v, kt, vt;
};

template <int HEAD_DIM, int STREAMS>
int launch_tree(const TreeMaps &m, const TreeParams &p, cudaStream_t stream) {
    using C = TreeCfg<HEAD_DIM, STREAMS>;
    auto kern = tree_kernel<HEAD_DIM, STREAMS>;
    {
        // The shared-memory opt-in belongs to the kernel as loaded on one device: once per device.
        static std::mutex mu;
        static bool done[64] = {};
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PA_ERR_CUDA;
        std::lock_guard<std::mutex> lock(mu);
        if (!done[dev]) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess)
                return PA_ERR_CUDA;
            done[dev] = true;
        }
    }
    const dim3 grid((unsigned)(p.chunks * p.num_parts), (unsigned)p.kv_heads, (unsigned)p.batch);
    kern<<<grid, C::kThreads, C::kSmemBytes, stream>>>(m.q, m.k, m.v, m.kt, m.vt, p);
    count_launch();
    const int st = launch_status();
    if (st != PA_OK || p.num_parts == 1) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.max_nodes * p.q_heads + kTreeReduceWarps - 1) / kTreeReduceWarps), (unsigned)p.batch);
    cfg.blockDim = dim3(kTreeReduceWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_reduce_kernel<HEAD_DIM>, p);
    count_launch();
    return e == cudaSuccess ? launch_status() : PA_ERR_CUDA;
}

bool bad_rows(const void *p, int64_t stride, int heads, int head_dim) {
    return !p || !aligned16(p) || stride % 8 || stride < (int64_t)heads * head_dim;
}

}  // namespace
}  // namespace pa

extern "C" {

int pa_decode_tree_partition_tokens(int batch, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                    int max_seq_len, int max_nodes, int partition_tokens) {
    if (batch <= 0 || max_seq_len <= 0 || max_nodes <= 0 ||
        !pa::supported_shape(num_q_heads, num_kv_heads, head_dim, block_size))
        return -1;
    return pa::tree_partition(batch, num_q_heads, num_kv_heads, max_seq_len, max_nodes, partition_tokens);
}

size_t pa_decode_tree_workspace_size(int batch, int num_rows, int num_q_heads, int num_kv_heads, int head_dim,
                                     int block_size, int max_seq_len, int max_nodes, int partition_tokens) {
    const int pt = pa_decode_tree_partition_tokens(batch, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len,
                                                   max_nodes, partition_tokens);
    if (pt <= 0 || num_rows <= 0) return 0;
    return pa::tree_layout(num_rows, num_q_heads, head_dim, ((int64_t)max_seq_len + pt - 1) / pt).total;
}

int pa_decode_tree(void *out, const void *q, int64_t q_stride, const void *k_tree, int64_t k_stride,
                   const void *v_tree, int64_t v_stride, int num_rows, const void *k_cache, const void *v_cache,
                   const int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens,
                   const int32_t *cu_nodes, const int32_t *masks, int batch, int max_seq_len, int max_nodes,
                   int num_q_heads, int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                   float scale, int partition_tokens, void *workspace, size_t workspace_bytes,
                   int32_t *err_flag, void *stream) {
    if (batch < 0 || max_seq_len < 0 || max_nodes < 0 || num_rows < 0 || num_blocks <= 0 || max_blocks_per_seq < 0)
        return PA_ERR_INVALID_ARG;
    if (!pa::supported_shape(num_q_heads, num_kv_heads, head_dim, block_size)) return PA_ERR_UNSUPPORTED;
    if (batch == 0 || num_rows == 0) return PA_OK;
    if (max_nodes == 0 || !out || !k_cache || !v_cache || !seq_lens || !cu_nodes) return PA_ERR_INVALID_ARG;
    if (max_blocks_per_seq > 0 && !block_tables) return PA_ERR_INVALID_ARG;
    if (!pa::aligned16(out) || !pa::aligned16(k_cache) || !pa::aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    if (pa::bad_rows(q, q_stride, num_q_heads, head_dim) || pa::bad_rows(k_tree, k_stride, num_kv_heads, head_dim) ||
        pa::bad_rows(v_tree, v_stride, num_kv_heads, head_dim))
        return PA_ERR_INVALID_ARG;
    if (partition_tokens > 0 && partition_tokens % 128) return PA_ERR_INVALID_ARG;
    if (batch > 65535 || num_q_heads > 65535) return PA_ERR_UNSUPPORTED;
    const uint64_t rows = (uint64_t)num_blocks * (uint64_t)num_kv_heads * (uint64_t)block_size;
    if (rows >= (1ull << 31)) return PA_ERR_UNSUPPORTED;  // TMA row coordinate is int32
    pa::TreeParams p{};
    p.out = static_cast<uint16_t *>(out);
    p.v_tree = static_cast<const uint16_t *>(v_tree);
    p.tables = block_tables;
    p.lens = seq_lens;
    p.cu = cu_nodes;
    p.masks = masks;
    p.err_flag = err_flag;
    p.v_stride = v_stride;
    p.num_blocks = num_blocks;
    p.num_rows = num_rows;
    p.max_blocks = max_blocks_per_seq;
    p.max_seq_len = max_seq_len;
    p.max_nodes = max_nodes;
    p.words = (max_nodes + 31) / 32;
    p.batch = batch;
    p.q_heads = num_q_heads;
    p.kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.block_size = block_size;
    p.pool_rows = (int)rows;
    p.scale_log2 = scale * pa::kTreeLog2e;
    p.chunks = pa::tree_chunks(max_nodes, p.group);
    const int pt = max_seq_len > 0 ? pa::tree_partition(batch, num_q_heads, num_kv_heads, max_seq_len, max_nodes,
                                                        partition_tokens)
                                   : -1;
    p.part_tokens = pt > 0 ? pt : (max_seq_len > 0 ? max_seq_len : 1);
    p.num_parts = pt > 0 ? (max_seq_len + pt - 1) / pt : 1;
    if (pt > 0) {
        const pa::TreeLayout l = pa::tree_layout(num_rows, num_q_heads, head_dim, p.num_parts);
        if (!workspace || workspace_bytes < l.total || !pa::aligned16(workspace)) return PA_ERR_INVALID_ARG;
        p.part_o = static_cast<float *>(workspace);
        p.part_ml = reinterpret_cast<float *>(static_cast<char *>(workspace) + l.ml);
    }
    if ((int64_t)p.chunks * p.num_parts > INT32_MAX || (int64_t)max_nodes * num_q_heads > INT32_MAX) return PA_ERR_UNSUPPORTED;
    pa::TreeMaps m;
    if (!pa::tree_rows_map(&m.q, q, q_stride, num_rows, num_q_heads, head_dim, p.group, pa::kTileM / p.group) ||
        !pa::tree_rows_map(&m.kt, k_tree, k_stride, num_rows, num_kv_heads, head_dim, 1, pa::kTileN) ||
        !pa::tree_rows_map(&m.vt, v_tree, v_stride, num_rows, num_kv_heads, head_dim, 1, pa::kTileN) ||
        !pa::tree_pool_map(&m.k, k_cache, rows, head_dim, block_size) ||
        !pa::tree_pool_map(&m.v, v_cache, rows, head_dim, block_size))
        return PA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (pa::tree_streams(max_nodes, p.group) == 2)
        return head_dim == 128 ? pa::launch_tree<128, 2>(m, p, s) : pa::launch_tree<64, 2>(m, p, s);
    return head_dim == 128 ? pa::launch_tree<128, 1>(m, p, s) : pa::launch_tree<64, 1>(m, p, s);
}

}  // extern "C"
