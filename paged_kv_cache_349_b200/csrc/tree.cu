// Attention of drafted tokens over the paged cache and over their own tree.
//
// Row r (node i of sequence b) and query head g:
//   out = sum_j exp(scale q.k_j - m) v_j / sum_j exp(scale q.k_j - m)
// over the sequence's cached tokens and the nodes its mask names.
//
// One warp computes one (row, query head): the lanes share the head dimension,
// a running maximum and sum carry the softmax over the tokens.
#include "pa_common.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTreeWarps = 8;

struct TreeParams {
    uint16_t *out;
    const uint16_t *q, *k_tree, *v_tree, *k_pool, *v_pool;
    const int32_t *tables, *lens, *cu, *masks;
    int32_t *err_flag;
    int64_t q_stride, k_stride, v_stride, num_blocks;
    int num_rows, batch, max_blocks, max_seq_len, max_nodes, words;
    int q_heads, kv_heads, group, block_size;
    float scale_log2;
};

template <int HEAD_DIM>
__global__ void __launch_bounds__(kTreeWarps * 32) tree_kernel(const TreeParams p) {
    constexpr int V = HEAD_DIM / 32;  // values of one lane
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.z, g = blockIdx.y, h = g / p.group;
    const int i = blockIdx.x * kTreeWarps + (threadIdx.x >> 5);
    const int lo = min(max(__ldg(p.cu + b), 0), p.num_rows);
    const int hi = max(min(max(__ldg(p.cu + b + 1), 0), p.num_rows), lo);
    const int nodes = min(hi - lo, p.max_nodes);
    const int raw = __ldg(p.lens + b);
    const int L = min(max(raw, 0), min(p.max_seq_len, p.max_blocks * p.block_size));
    if (g == 0 && blockIdx.x == 0 && threadIdx.x == 0 &&
        (raw != L || lo != __ldg(p.cu + b) || hi != __ldg(p.cu + b + 1) || nodes != hi - lo))
        raise_flag(p.err_flag, PA_FLAG_BAD_LEN);
    if (i >= nodes) return;
    const int64_t r = lo + i;

    auto load = [&](const uint16_t *src, float (&x)[V]) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(src + lane * V + e));
            x[e] = bf16_lo_to_float(w);
            x[e + 1] = bf16_hi_to_float(w);
        }
    };
    float q[V], o[V], m = -INFINITY, l = 0.f;
    bool any = false;  // the row sees something
    load(p.q + r * p.q_stride + g * HEAD_DIM, q);
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
    auto take = [&](const uint16_t *k_row, const uint16_t *v_row) {
        float k[V], v[V], s = 0.f;
        load(k_row, k);
        load(v_row, v);
#pragma unroll
        for (int e = 0; e < V; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
        for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= p.scale_log2;
        any = true;
        const float top = fmaxf(m, s);
        const float ref = top == -INFINITY ? 0.f : top;  // nothing seen yet: weights 0, a NaN score stays NaN
        const float down = exp2f(m - ref), w = exp2f(s - ref);
        m = top;
        l = l * down + w;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = o[e] * down + w * v[e];
    };
    for (int t = 0; t < L; ++t) {
        const int64_t phys = __ldg(p.tables + (int64_t)b * p.max_blocks + t / p.block_size);
        if (phys < 0 || phys >= p.num_blocks) {
            if (lane == 0) raise_flag(p.err_flag, PA_FLAG_BAD_BLOCK);
            continue;
        }
        const int64_t row = ((phys * p.kv_heads + h) * p.block_size + t % p.block_size) * HEAD_DIM;
        take(p.k_pool + row, p.v_pool + row);
    }
    for (int j = 0; j < nodes; ++j) {
        const bool seen = p.masks ? (__ldg(p.masks + r * p.words + (j >> 5)) >> (j & 31)) & 1 : j <= i;
        if (seen)
            take(p.k_tree + (int64_t)(lo + j) * p.k_stride + h * HEAD_DIM,
                 p.v_tree + (int64_t)(lo + j) * p.v_stride + h * HEAD_DIM);
    }
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + (r * p.q_heads + g) * HEAD_DIM + lane * V);
#pragma unroll
    for (int e = 0; e < V; e += 2)
        // nothing seen: zeros; all scores -inf: 0 / 0
        dst[e / 2] = !any ? 0u : pack_bf16x2(o[e] / l, o[e + 1] / l);
}

bool bad_rows(const void *p, int64_t stride, int heads, int head_dim) {
    return !p || !aligned16(p) || stride % 8 || stride < (int64_t)heads * head_dim;
}

}  // namespace
}  // namespace pa

extern "C" {

int pa_decode_tree_partition_tokens(int batch, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                    int max_seq_len, int max_nodes, int partition_tokens) {
    (void)batch, (void)num_q_heads, (void)num_kv_heads, (void)head_dim, (void)block_size, (void)max_seq_len;
    (void)max_nodes, (void)partition_tokens;
    return -1;
}

size_t pa_decode_tree_workspace_size(int batch, int num_rows, int num_q_heads, int num_kv_heads, int head_dim,
                                     int block_size, int max_seq_len, int max_nodes, int partition_tokens) {
    (void)batch, (void)num_rows, (void)num_q_heads, (void)num_kv_heads, (void)head_dim, (void)block_size;
    (void)max_seq_len, (void)max_nodes, (void)partition_tokens;
    return 0;
}

int pa_decode_tree(void *out, const void *q, int64_t q_stride, const void *k_tree, int64_t k_stride,
                   const void *v_tree, int64_t v_stride, int num_rows, const void *k_cache, const void *v_cache,
                   const int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens,
                   const int32_t *cu_nodes, const int32_t *masks, int batch, int max_seq_len, int max_nodes,
                   int num_q_heads, int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                   float scale, int partition_tokens, void *workspace, size_t workspace_bytes,
                   int32_t *err_flag, void *stream) {
    (void)workspace, (void)workspace_bytes;
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
    p.q = static_cast<const uint16_t *>(q);
    p.k_tree = static_cast<const uint16_t *>(k_tree);
    p.v_tree = static_cast<const uint16_t *>(v_tree);
    p.k_pool = static_cast<const uint16_t *>(k_cache);
    p.v_pool = static_cast<const uint16_t *>(v_cache);
    p.tables = block_tables;
    p.lens = seq_lens;
    p.cu = cu_nodes;
    p.masks = masks;
    p.err_flag = err_flag;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.num_blocks = num_blocks;
    p.num_rows = num_rows;
    p.batch = batch;
    p.max_blocks = max_blocks_per_seq;
    p.max_seq_len = max_seq_len;
    p.max_nodes = max_nodes;
    p.words = (max_nodes + 31) / 32;
    p.q_heads = num_q_heads;
    p.kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.block_size = block_size;
    p.scale_log2 = scale * pa::kLog2e;
    const dim3 grid((unsigned)((max_nodes + pa::kTreeWarps - 1) / pa::kTreeWarps), (unsigned)num_q_heads, (unsigned)batch);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (head_dim == 128)
        pa::tree_kernel<128><<<grid, pa::kTreeWarps * 32, 0, s>>>(p);
    else
        pa::tree_kernel<64><<<grid, pa::kTreeWarps * 32, 0, s>>>(p);
    pa::count_launch();
    return pa::launch_status();
}

}  // extern "C"
