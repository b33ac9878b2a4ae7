// Host side of the attention of drafted tokens: tensor maps, the choice of
// variant, the workspace and the launches (the device code is in
// tree_kernels.cuh).
#include <math.h>

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

// More than 128 query rows of a kv head: two streams of 128 rows share each K and V tile, so that half as much is read.
// Up to 128 rows one stream: two CTAs on an SM hide each other's waits.  Measured with one | two streams: 4 sequences
// of up to 8190 tokens with 512 rows of each kv head 100 | 91 us; with 128 rows, 64 of up to 4096 70 | 99 us, 8 of
// 32768 190 | 264 us.
int tree_streams(int max_nodes, int group) { return (int64_t)max_nodes * group > kTileM ? 2 : 1; }

int tree_tile(int max_nodes, int group) { return tree_streams(max_nodes, group) == 2 ? TreeCfg<128, 2>::kTileN : TreeCfg<128, 1>::kTileN; }

// CTAs that the device holds at once: the grid, whatever the batch.
int tree_ctas(int max_nodes, int group) {
    return device_sm_count() *
           (tree_streams(max_nodes, group) == 2 ? TreeCfg<128, 2>::kCtasPerSm : TreeCfg<128, 1>::kCtasPerSm);
}

// Tokens that a piece of a cut unit has at least, or -1 when no unit is cut.  Caches that fit a few tiles
// are left whole by default: the second launch (6 to 8 us) would cost more than the balance gains.  Measured on 64
// sequences of up to 4096 tokens with 32/8 heads, uncut | pieces of 256 | 512 | 1024: 91 | 70 | 70 | 70 us; on 24 of
// up to 2048 with 32/32 heads 95 | 77 | 77 | 95 (1024 leaves them uncut).
constexpr int kTreeShare = 256;
int tree_share(int max_seq_len, int requested) {
    if (requested < 0) return -1;
    const int share = requested > 0 ? requested : kTreeShare;
    return max_seq_len <= 2 * share ? -1 : share;
}

// Workspace: two states for each CTA, of a unit that began before it and of one that ends after it,
// then what there is to join.
struct TreeLayout {
    size_t ml, joins, total;
};

TreeLayout tree_layout(int ctas, int streams, int head_dim) {
    const size_t rows = (size_t)ctas * 2 * streams * kTileM;
    TreeLayout l{};
    l.ml = rows * head_dim * 4;
    l.joins = l.ml + rows * 8;
    l.total = l.joins + (size_t)ctas * sizeof(TreeJoin);
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
    const int ctas = tree_ctas(p.max_nodes, p.group);
    kern<<<ctas, C::kThreads, C::kSmemBytes, stream>>>(m.q, m.k, m.v, m.kt, m.vt, p);
    count_launch();
    const int st = launch_status();
    if (st != PA_OK || !p.part_o) return st;
    cudaLaunchConfig_t cfg = {};
    const int rows = min(STREAMS * kTileM, p.max_nodes * p.group);  // of a unit, at most
    cfg.gridDim = dim3((unsigned)(ctas - 1), (unsigned)((rows + kJoinRows - 1) / kJoinRows));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_join_kernel<HEAD_DIM, STREAMS>, p);
    count_launch();
    return e == cudaSuccess ? launch_status() : PA_ERR_CUDA;
}

bool bad_rows(const void *p, int64_t stride, int heads, int head_dim) {
    return !p || !aligned16(p) || stride % 8 || stride < (int64_t)heads * head_dim;
}

}  // namespace
}  // namespace pa

extern "C" {

size_t pa_decode_tree_workspace_size(int batch, int num_rows, int num_q_heads, int num_kv_heads, int head_dim,
                                     int block_size, int max_seq_len, int max_nodes, int partition_tokens) {
    if (batch <= 0 || num_rows <= 0 || max_seq_len <= 0 || max_nodes <= 0 ||
        !pa::supported_shape(num_q_heads, num_kv_heads, head_dim, block_size) ||
        pa::tree_share(max_seq_len, partition_tokens) < 0)
        return 0;
    const int group = num_q_heads / num_kv_heads;
    return pa::tree_layout(pa::tree_ctas(max_nodes, group), pa::tree_streams(max_nodes, group), head_dim).total;
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
    if (!(scale >= 0.f && scale * pa::kTreeLog2e < HUGE_VALF)) return PA_ERR_INVALID_ARG;
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
    p.group_shift = p.group == 8 ? 3 : p.group >> 1;
    p.block_size = block_size;
    p.pool_rows = (int)rows;
    p.scale_log2 = scale * pa::kTreeLog2e;
    const int streams = pa::tree_streams(max_nodes, p.group), tile = pa::tree_tile(max_nodes, p.group);
    const int share = pa::tree_share(max_seq_len, partition_tokens);
    p.min_share = share > tile ? share / tile : 1;
    if (share > 0) {
        const pa::TreeLayout l = pa::tree_layout(pa::tree_ctas(max_nodes, p.group), streams, head_dim);
        if (!workspace || workspace_bytes < l.total || !pa::aligned16(workspace)) return PA_ERR_INVALID_ARG;
        p.part_o = static_cast<float *>(workspace);
        p.part_ml = reinterpret_cast<float *>(static_cast<char *>(workspace) + l.ml);
        p.joins = reinterpret_cast<pa::TreeJoin *>(static_cast<char *>(workspace) + l.joins);
    }
    // row numbers and places of a unit are int32
    if ((int64_t)max_nodes * num_q_heads > INT32_MAX / 2 || (int64_t)max_blocks_per_seq * block_size > INT32_MAX / 2)
        return PA_ERR_UNSUPPORTED;
    pa::TreeMaps m;
    if (!pa::tree_rows_map(&m.q, q, q_stride, num_rows, num_q_heads, head_dim, p.group, pa::kTileM / p.group) ||
        !pa::tree_rows_map(&m.kt, k_tree, k_stride, num_rows, num_kv_heads, head_dim, 1, pa::kTreeBox) ||
        !pa::tree_rows_map(&m.vt, v_tree, v_stride, num_rows, num_kv_heads, head_dim, 1, pa::kTreeBox) ||
        !pa::tree_pool_map(&m.k, k_cache, rows, head_dim, block_size) ||
        !pa::tree_pool_map(&m.v, v_cache, rows, head_dim, block_size))
        return PA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (streams == 2)
        return head_dim == 128 ? pa::launch_tree<128, 2>(m, p, s) : pa::launch_tree<64, 2>(m, p, s);
    return head_dim == 128 ? pa::launch_tree<128, 1>(m, p, s) : pa::launch_tree<64, 1>(m, p, s);
}

}  // extern "C"
