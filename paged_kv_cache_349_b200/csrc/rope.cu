// Rotary positions on q and k, alone or together with the cache write.
//
// Mathematics: pair i of a head at position p is turned by the angle
// 2 pi p turns[i].  p * turns[i] is formed in fp64 and only its fraction of a
// turn goes on to fp32 (sincospif): at position 10^6 an fp32 product of
// radians is already off by up to 0.03.  The rotation itself is fp32,
// rounded once, to bf16 or to E4M3.
//
// Bound: HBM.  Every q, k and v value is read once and written once; the angles
// are computed once for each token and shared by all heads through shared
// memory.  A thread keeps one place in the row (a head, and 16 values of it)
// for all tokens of its CTA, so that the loop over tokens has no index
// arithmetic; the loads of all its tokens are issued before the angles are
// computed.  8192 tokens of 32 + 8 heads take 35 us, 5.7 TB/s (a division for each
// 16 values: 55 us).
#include <math.h>

#include "pa_common.cuh"

namespace pa {
namespace {

// Threads of a CTA at most, and its tokens where there are enough to fill the GPU with such CTAs.  Measured
// (8192 tokens of 32 + 8 heads, bf16 pools | 3001 tokens of 40 + 40 heads, fp8 pools): 35.1 | 28.2 us;
// with 512 threads and 4 tokens 53.2 | 38.8, with 256 and 4 35.3 | 29.7, with 128 and 5 38.0 | 29.4.
constexpr int kRopeThreads = 128;
constexpr int kRopeTokens = 3;

struct RopeParams {
    const uint16_t *q, *k, *v;
    uint16_t *q_out, *k_out;  // k_out: pa_rope only
    void *k_cache, *v_cache;
    const int32_t *slots, *positions;
    const double *turns;
    int32_t *err_flag;
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride, num_slots;
    int num_tokens, q_heads, kv_heads, rotary, block_size;
    float gain, k_inv_scale, v_inv_scale;
};

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16_lo_to_float(w[e]);
        x[2 * e + 1] = bf16_hi_to_float(w[e]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float inv_scale) {
    uint32_t out[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 pair = make_float2(__fmul_rn(x[2 * e], inv_scale), __fmul_rn(x[2 * e + 1], inv_scale));
        out[e >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(pair, __NV_SATFINITE, __NV_E4M3) << ((e & 1) * 16);
    }
    return make_uint2(out[0], out[1]);
}

// A place is 16 values of one head in two vectors of 8: for a rotated one the pairs 8i .. 8i+7 (values 8i.. and
// rotary / 2 + 8i.. of the head, or 16i.. and 16i + 8.. where pairs are interleaved), else 16 that pass through.
// CACHE: k and v go to the pools (FP8: as E4M3 codes); else the rotated k goes to k_out.
template <int HEAD_DIM, bool INTERLEAVED, bool CACHE, bool FP8, int TOKENS>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
    constexpr int kPlaces = HEAD_DIM / 16;  // of one head
    // cos and sin of pairs 8i + 2s, 8i + 2s + 1 of token t at [t][s][i]: the places of a head read
    // neighbouring 16-byte words
    __shared__ float4 s_cs[TOKENS * 4 * kPlaces];
    __shared__ int64_t s_row[TOKENS];  // pool offset of the token's row of head 0, or -1
    const int t0 = blockIdx.x * TOKENS;
    const int tokens = min(TOKENS, p.num_tokens - t0);
    const int places = (p.q_heads + p.kv_heads * (CACHE ? 2 : 1)) * kPlaces;

    for (int x0 = 0; x0 < places; x0 += blockDim.x) {
        const int x = x0 + threadIdx.x;
        const int i = x % kPlaces, head = x / kPlaces;
        const bool is_q = head < p.q_heads, is_v = CACHE && head >= p.q_heads + p.kv_heads;
        const int h = is_q ? head : head - p.q_heads - (is_v ? p.kv_heads : 0);
        const bool turn = !is_v && 16 * i < p.rotary;
        const int a = turn && !INTERLEAVED ? 8 * i : 16 * i;
        const int b = turn && !INTERLEAVED ? p.rotary / 2 + 8 * i : 16 * i + 8;
        uint4 lo[TOKENS], hi[TOKENS];
        if (x < places) {
            const int64_t stride = is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride;
            const uint16_t *src = (is_q ? p.q : is_v ? p.v : p.k) + t0 * stride + h * HEAD_DIM;
#pragma unroll
            for (int u = 0; u < TOKENS; ++u)
                if (u < tokens) {
                    lo[u] = *reinterpret_cast<const uint4 *>(src + u * stride + a);
                    hi[u] = *reinterpret_cast<const uint4 *>(src + u * stride + b);
                }
        }
        if (x0 == 0) {
            const int pairs = p.rotary / 2;
            for (int y = threadIdx.x; y < tokens * pairs; y += blockDim.x) {
                const int u = y / pairs, j = y - u * pairs;
                const double at = (double)__ldg(p.positions + t0 + u) * __ldg(p.turns + j);
                float c, s;
                sincospif((float)(2.0 * (at - rint(at))), &s, &c);
                // pair j is half (j & 1) of word (j / 2) % 4 of place j / 8
                float2 *dst = reinterpret_cast<float2 *>(s_cs + (u * 4 + ((j >> 1) & 3)) * kPlaces + (j >> 3)) + (j & 1);
                *dst = make_float2(c * p.gain, s * p.gain);
            }
            if (CACHE && threadIdx.x < tokens) {
                const int64_t slot = __ldg(p.slots + t0 + threadIdx.x);
                int64_t row = -1;
                if (slot >= 0 && slot < p.num_slots) {
                    const int64_t blk = slot / p.block_size;
                    row = (blk * p.kv_heads * p.block_size + (slot - blk * p.block_size)) * HEAD_DIM;
                } else if (slot != -1) {
                    raise_flag(p.err_flag, PA_FLAG_BAD_SLOT);
                }
                s_row[threadIdx.x] = row;
            }
            __syncthreads();
        }
        if (x >= places) continue;
#pragma unroll
        for (int u = 0; u < TOKENS; ++u) {
            if (u >= tokens) break;
            float v[8], w[8];
            unpack8(lo[u], v);
            unpack8(hi[u], w);
            if (turn) {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float4 cs = s_cs[(u * 4 + s) * kPlaces + i];
                    if (INTERLEAVED) {  // pairs (2e, 2e + 1): 0..3 in v, 4..7 in w
                        float(&z)[8] = s < 2 ? v : w;
                        const int e = 4 * (s & 1);
                        const float a0 = z[e], b0 = z[e + 1], a1 = z[e + 2], b1 = z[e + 3];
                        z[e] = a0 * cs.x - b0 * cs.y;
                        z[e + 1] = b0 * cs.x + a0 * cs.y;
                        z[e + 2] = a1 * cs.z - b1 * cs.w;
                        z[e + 3] = b1 * cs.z + a1 * cs.w;
                    } else {
                        const int e = 2 * s;
                        const float a0 = v[e], b0 = w[e], a1 = v[e + 1], b1 = w[e + 1];
                        v[e] = a0 * cs.x - b0 * cs.y;
                        w[e] = b0 * cs.x + a0 * cs.y;
                        v[e + 1] = a1 * cs.z - b1 * cs.w;
                        w[e + 1] = b1 * cs.z + a1 * cs.w;
                    }
                }
            }
            if (CACHE && !is_q) {
                int64_t row = s_row[u];
                if (row < 0) continue;
                row += (int64_t)h * p.block_size * HEAD_DIM;
                if (FP8) {
                    uint8_t *dst = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) + row;
                    const float inv = is_v ? p.v_inv_scale : p.k_inv_scale;
                    *reinterpret_cast<uint2 *>(dst + a) = quantise8(v, inv);
                    *reinterpret_cast<uint2 *>(dst + b) = quantise8(w, inv);
                    continue;
                }
                uint16_t *dst = static_cast<uint16_t *>(is_v ? p.v_cache : p.k_cache) + row;
                *reinterpret_cast<uint4 *>(dst + a) = turn ? pack8(v) : lo[u];
                *reinterpret_cast<uint4 *>(dst + b) = turn ? pack8(w) : hi[u];
                continue;
            }
            // what passes through keeps its bits
            uint16_t *dst = (is_q ? p.q_out + (t0 + u) * p.q_out_stride : p.k_out + (t0 + u) * p.k_out_stride) + h * HEAD_DIM;
            *reinterpret_cast<uint4 *>(dst + a) = turn ? pack8(v) : lo[u];
            *reinterpret_cast<uint4 *>(dst + b) = turn ? pack8(w) : hi[u];
        }
    }
}

template <int HEAD_DIM, bool INTERLEAVED, int TOKENS>
void launch_rope_n(const RopeParams &p, bool cache, bool fp8, cudaStream_t s) {
    // As few passes over the places of a row as kRopeThreads allow, of equal size.
    const int places = (p.q_heads + p.kv_heads * (cache ? 2 : 1)) * (HEAD_DIM / 16);
    const int passes = (places + kRopeThreads - 1) / kRopeThreads;
    const int threads = ((places + passes - 1) / passes + 31) / 32 * 32;
    const unsigned grid = (unsigned)((p.num_tokens + TOKENS - 1) / TOKENS);
    if (!cache)
        rope_kernel<HEAD_DIM, INTERLEAVED, false, false, TOKENS><<<grid, threads, 0, s>>>(p);
    else if (fp8)
        rope_kernel<HEAD_DIM, INTERLEAVED, true, true, TOKENS><<<grid, threads, 0, s>>>(p);
    else
        rope_kernel<HEAD_DIM, INTERLEAVED, true, false, TOKENS><<<grid, threads, 0, s>>>(p);
}

template <int HEAD_DIM, bool INTERLEAVED>
void launch_rope(const RopeParams &p, bool cache, bool fp8, cudaStream_t s) {
    // Measured with one | three tokens to a CTA (32 + 8 heads, bf16 pools; 40 + 40, fp8 pools): 1200 tokens 8.2 | 8.2 and
    // 16.5 | 18.7 us, 1500 12.3 | 12.1 and 22.7 | 20.5, 1776 (the border here) 14.1 | 12.3 and 25.0 | 22.4, 2400
    // 16.2 | 14.5 and 28.5 | 24.8: a border at 1400 would do as well or better.
    if (p.num_tokens >= 4 * kRopeTokens * device_sm_count())
        launch_rope_n<HEAD_DIM, INTERLEAVED, kRopeTokens>(p, cache, fp8, s);
    else
        launch_rope_n<HEAD_DIM, INTERLEAVED, 1>(p, cache, fp8, s);
}

bool bad_rows(const void *p, int64_t stride, int heads, int head_dim) {
    return !p || !aligned16(p) || stride % 8 || stride < (int64_t)heads * head_dim;
}

// Shared body: the row arguments of q and k are checked here, those of the destination by the callers.
int rope_impl(RopeParams p, int head_dim, int interleaved, bool cache, bool fp8, void *stream) {
    if (p.num_tokens < 0 || p.q_heads < 0 || p.kv_heads < 0) return PA_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (p.rotary < 16 || p.rotary > head_dim || p.rotary % 16) return PA_ERR_UNSUPPORTED;
    if (p.q_heads > 65535 || p.kv_heads > 65535) return PA_ERR_UNSUPPORTED;
    const int heads = p.q_heads + p.kv_heads * (cache ? 2 : 1);
    if (heads == 0) return PA_ERR_INVALID_ARG;
    if (p.num_tokens == 0) return PA_OK;
    if (!p.positions || !p.turns) return PA_ERR_INVALID_ARG;
    if (p.q_heads && (bad_rows(p.q, p.q_stride, p.q_heads, head_dim) ||
                      bad_rows(p.q_out, p.q_out_stride, p.q_heads, head_dim)))
        return PA_ERR_INVALID_ARG;
    if (p.kv_heads && bad_rows(p.k, p.k_stride, p.kv_heads, head_dim)) return PA_ERR_INVALID_ARG;
    // in place at another stride, rows would be written that others have still to read
    if (p.num_tokens > 1 && ((p.q_heads && p.q == p.q_out && p.q_stride != p.q_out_stride) ||
                             (p.kv_heads && p.k == p.k_out && p.k_stride != p.k_out_stride)))
        return PA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (head_dim == 128)
        interleaved ? launch_rope<128, true>(p, cache, fp8, s) : launch_rope<128, false>(p, cache, fp8, s);
    else
        interleaved ? launch_rope<64, true>(p, cache, fp8, s) : launch_rope<64, false>(p, cache, fp8, s);
    count_launch();
    return launch_status();
}

int rope_and_cache_impl(const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride, int num_q_heads,
                        const void *k, int64_t k_stride, const void *v, int64_t v_stride, int num_kv_heads,
                        void *k_cache, void *v_cache, const int32_t *slot_mapping, int64_t num_blocks,
                        int block_size, const int32_t *positions, const double *turns, int rotary_dim,
                        int interleaved, float gain, int num_tokens, int head_dim, bool fp8, float k_scale,
                        float v_scale, int32_t *err_flag, void *stream) {
    if (num_tokens < 0 || num_blocks <= 0 || num_kv_heads <= 0) return PA_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (!supported_block_size(block_size)) return PA_ERR_UNSUPPORTED;
    if (fp8 && !(k_scale > 0.f && v_scale > 0.f && k_scale < 3.0e38f && v_scale < 3.0e38f)) return PA_ERR_INVALID_ARG;
    if (num_tokens > 0) {
        if (!slot_mapping || !k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
        if (bad_rows(v, v_stride, num_kv_heads, head_dim)) return PA_ERR_INVALID_ARG;
    }
    RopeParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.slots = slot_mapping;
    p.positions = positions;
    p.turns = turns;
    p.err_flag = err_flag;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out_stride = q_out_stride;
    p.num_slots = num_blocks * block_size;
    p.num_tokens = num_tokens;
    p.q_heads = num_q_heads;
    p.kv_heads = num_kv_heads;
    p.rotary = rotary_dim;
    p.block_size = block_size;
    p.gain = gain;
    p.k_inv_scale = fp8 ? 1.0f / k_scale : 1.f;
    p.v_inv_scale = fp8 ? 1.0f / v_scale : 1.f;
    return rope_impl(p, head_dim, interleaved, true, fp8, stream);
}

}  // namespace
}  // namespace pa

extern "C" {

int pa_rope(const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride, int num_q_heads, const void *k,
            int64_t k_stride, void *k_out, int64_t k_out_stride, int num_kv_heads, const int32_t *positions,
            const double *turns, int rotary_dim, int interleaved, float gain, int num_tokens, int head_dim,
            void *stream) {
    pa::RopeParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_out = static_cast<uint16_t *>(k_out);
    p.positions = positions;
    p.turns = turns;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.num_tokens = num_tokens;
    p.q_heads = num_q_heads;
    p.kv_heads = num_kv_heads;
    p.rotary = rotary_dim;
    p.gain = gain;
    if ((head_dim == 64 || head_dim == 128) && num_tokens > 0 && num_kv_heads > 0 &&
        pa::bad_rows(k_out, k_out_stride, num_kv_heads, head_dim))
        return PA_ERR_INVALID_ARG;
    return pa::rope_impl(p, head_dim, interleaved, false, false, stream);
}

int pa_rope_and_cache(const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride, int num_q_heads,
                      const void *k, int64_t k_stride, const void *v, int64_t v_stride, int num_kv_heads,
                      void *k_cache, void *v_cache, const int32_t *slot_mapping, int64_t num_blocks,
                      int block_size, const int32_t *positions, const double *turns, int rotary_dim,
                      int interleaved, float gain, int num_tokens, int head_dim, int32_t *err_flag, void *stream) {
    return pa::rope_and_cache_impl(q, q_stride, q_out, q_out_stride, num_q_heads, k, k_stride, v, v_stride,
                                   num_kv_heads, k_cache, v_cache, slot_mapping, num_blocks, block_size, positions,
                                   turns, rotary_dim, interleaved, gain, num_tokens, head_dim, false, 1.f, 1.f,
                                   err_flag, stream);
}

int pa_rope_and_cache_fp8(const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride, int num_q_heads,
                          const void *k, int64_t k_stride, const void *v, int64_t v_stride, int num_kv_heads,
                          void *k_cache, void *v_cache, const int32_t *slot_mapping, int64_t num_blocks,
                          int block_size, const int32_t *positions, const double *turns, int rotary_dim,
                          int interleaved, float gain, int num_tokens, int head_dim, float k_scale,
                          float v_scale, int32_t *err_flag, void *stream) {
    return pa::rope_and_cache_impl(q, q_stride, q_out, q_out_stride, num_q_heads, k, k_stride, v, v_stride,
                                   num_kv_heads, k_cache, v_cache, slot_mapping, num_blocks, block_size, positions,
                                   turns, rotary_dim, interleaved, gain, num_tokens, head_dim, true, k_scale, v_scale,
                                   err_flag, stream);
}

int pa_rope_frequencies(double *turns, float *gain, int rotary_dim, double base, int scaling, double factor,
                        double original_len, double low, double high) {
    if (scaling < PA_ROPE_NONE || scaling > PA_ROPE_BY_WAVELENGTH) return PA_ERR_UNSUPPORTED;
    if (!turns || !gain || rotary_dim <= 0 || rotary_dim % 2 || !(base > 1.0 && base < HUGE_VAL)) return PA_ERR_INVALID_ARG;
    if (scaling != PA_ROPE_NONE && !(factor >= 1.0 && factor < HUGE_VAL)) return PA_ERR_INVALID_ARG;
    if (scaling == PA_ROPE_NTK && rotary_dim <= 2) return PA_ERR_INVALID_ARG;
    const bool ramped = scaling == PA_ROPE_BY_PARTS || scaling == PA_ROPE_BY_WAVELENGTH;
    if (ramped && !(original_len > 0.0 && original_len < HUGE_VAL && low > 0.0 && low < high && high < HUGE_VAL))
        return PA_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925;
    const double dim = rotary_dim;
    if (scaling == PA_ROPE_NTK) base *= pow(factor, dim / (dim - 2.0));
    *gain = scaling == PA_ROPE_BY_PARTS ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    // BY_PARTS: the pair numbers that turn `high` and `low` times within original_len,
    // taken to whole pairs inside the head
    double first = 0.0, last = 0.0;
    if (scaling == PA_ROPE_BY_PARTS) {
        first = fmax(floor(dim * log(original_len / (high * two_pi)) / (2.0 * log(base))), 0.0);
        last = fmin(ceil(dim * log(original_len / (low * two_pi)) / (2.0 * log(base))), dim - 1.0);
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / dim);
        double slow = 0.0;  // how far the pair is slowed down by `factor`
        if (scaling == PA_ROPE_LINEAR)
            slow = 1.0;
        else if (scaling == PA_ROPE_BY_PARTS)
            slow = fmin(fmax((i - first) / fmax(last - first, 0.001), 0.0), 1.0);
        else if (scaling == PA_ROPE_BY_WAVELENGTH)
            slow = 1.0 - fmin(fmax((original_len * f / two_pi - low) / (high - low), 0.0), 1.0);
        if (slow > 0.0) f = f / factor * slow + f * (1.0 - slow);
        turns[i] = f / two_pi;
    }
    return PA_OK;
}

}  // extern "C"
