// Device side shared by the prompt attention kernels (pa_prefill,
// pa_prefill_paged; include/pa.h): parameters, the rows of a sequence and the
// plain row-at-a-time form.
#pragma once

#include "pa_common.cuh"

namespace pa {

struct PrefillParams {
    void *out;
    const void *q;
    const void *k, *v;  // packed rows, or the pools
    const int32_t *cu_seqlens;
    const int32_t *block_tables, *context_lens;  // paged only
    int num_seqs, num_tokens, num_heads, num_kv_heads;
    int block_size, max_blocks_per_seq, num_blocks, ctx_limit;  // paged only
    long long q_stride, k_stride, v_stride;                     // elements from token to token
    float scale_log2;                                           // |scale| * log2(e), above 0
    unsigned int *errors;
};

// Query rows [row0, row0 + n) of sequence s and the keys it has; row i of them
// sees the first keys - n + i + 1.
struct SeqRange {
    int row0, n, keys;
};

template <bool PAGED>
__device__ __forceinline__ SeqRange seq_range(const PrefillParams &p, int s, unsigned &bad) {
    int a = p.cu_seqlens[s], b = p.cu_seqlens[s + 1];
    if (a < 0 || b < a || b > p.num_tokens) bad |= PA_DEVERR_TOKENS;
    a = min(max(a, 0), p.num_tokens);
    b = min(max(b, a), p.num_tokens);
    SeqRange r{a, b - a, b - a};
    if constexpr (PAGED) {
        const int c = p.context_lens[s];
        if (c < 0 || c > p.ctx_limit) bad |= PA_DEVERR_CONTEXT;
        r.keys = min(max(c, 0), p.ctx_limit);
    }
    return r;
}

// One row by one warp: keys a lane each for the scores, head elements a lane
// each for the values, the running maximum and sum of the softmax in 32 bits.
// Reads the visible keys and values only. q_smem: D floats of this warp; negate:
// the scale is -scale_log2.
template <int D, typename T, bool PAGED>
__device__ __noinline__ void attend_row(const PrefillParams &p, int s, int row, int h, int visible, float *q_smem,
                           bool negate, unsigned &bad) {
    constexpr int E = D / 32;  // output elements of a lane
    const int lane = threadIdx.x & 31;
    const int kvh = h / (p.num_heads / p.num_kv_heads);
    const int row0 = PAGED ? 0 : p.cu_seqlens[s];
    auto base = [&](const void *x, long long stride, int j) {
        if constexpr (PAGED) {
            int id = p.block_tables[(size_t)s * p.max_blocks_per_seq + j / p.block_size];
            if ((unsigned)id >= (unsigned)p.num_blocks) {
                bad |= PA_DEVERR_BLOCK_ID;
                id = 0;
            }
            return static_cast<const T *>(x) +
                   (((size_t)id * p.num_kv_heads + kvh) * p.block_size + j % p.block_size) * D;
        } else {
            return static_cast<const T *>(x) + (size_t)(row0 + j) * stride + (size_t)kvh * D;
        }
    };
    const T *qp = static_cast<const T *>(p.q) + (size_t)row * p.q_stride + (size_t)h * D;
    __syncwarp();
    for (int i = lane; i < D / 2; i += 32) {
        const float2 x = Elem<T>::pair(reinterpret_cast<const uint32_t *>(qp)[i]);
        q_smem[2 * i] = x.x;
        q_smem[2 * i + 1] = x.y;
    }
    __syncwarp();
    float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int j0 = 0; j0 < visible; j0 += 32) {
        const int count = min(32, visible - j0);
        float z = -INFINITY;
        if (lane < count) {
            const uint4 *kp = reinterpret_cast<const uint4 *>(base(p.k, p.k_stride, j0 + lane));
            float dot = 0.f;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                float x[8];
                unpack8<T>(kp[c], x);
#pragma unroll
                for (int i = 0; i < 8; ++i) dot = fmaf(x[i], q_smem[8 * c + i], dot);
            }
            z = (negate ? -dot : dot) * p.scale_log2;
        }
        float mt = z;
#pragma unroll
        for (int o = 16; o; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(FULL_MASK, mt, o));
        const float m_new = fmaxf(m, mt);
        const float ref = m_new == -INFINITY ? 0.f : m_new;  // nothing above -inf yet
        const float f = exp2f(m - ref);
        const float w = lane < count ? exp2f(z - ref) : 0.f;
        m = m_new;
        float sum = w;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
        l = l * f + sum;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= f;
        for (int c = 0; c < count; ++c) {
            const float wc = __shfl_sync(FULL_MASK, w, c);
            const uint32_t *vp = reinterpret_cast<const uint32_t *>(base(p.v, p.v_stride, j0 + c)) + lane * (E / 2);
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                const float2 x = Elem<T>::pair(vp[e]);
                acc[2 * e] = fmaf(wc, x.x, acc[2 * e]);
                acc[2 * e + 1] = fmaf(wc, x.y, acc[2 * e + 1]);
            }
        }
    }
    // A row that sees nothing is zero; one whose scores are all -inf is 0 / 0.
    const float inv = visible > 0 ? 1.f / l : 0.f;
    uint32_t *op = reinterpret_cast<uint32_t *>(static_cast<T *>(p.out) + ((size_t)row * p.num_heads + h) * D) +
                   lane * (E / 2);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) op[e] = Elem<T>::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
}

}  // namespace pa
