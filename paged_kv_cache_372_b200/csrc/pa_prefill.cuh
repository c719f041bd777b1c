// Device side of the prompt attention (pa_prefill, pa_prefill_paged;
// include/pa.h): the row-at-a-time form, for rows of very large scores, and
// values that are not finite.
#pragma once

#include "pa_prefill_plan.cuh"

namespace pa {

// Row j of sequence s in the keys or values x.
template <int D, typename T, bool PAGED>
__device__ __forceinline__ const T *kv_row(const PrefillParams &p, const void *x, long long stride, int s, int row0,
                                           int kvh, int j) {
    if constexpr (PAGED) {
        int id = p.block_tables[(size_t)s * p.max_blocks_per_seq + j / p.block_size];
        if ((unsigned)id >= (unsigned)p.num_blocks) id = 0;  // flagged where the tile was loaded
        return static_cast<const T *>(x) + (((size_t)id * p.num_kv_heads + kvh) * p.block_size + j % p.block_size) * D;
    } else {
        return static_cast<const T *>(x) + (size_t)(row0 + j) * stride + (size_t)kvh * D;
    }
}

// What a row has from a range of keys: weighted values relative to the maximum
// m (log2 units) and the sum of the weights; D / 32 elements a lane.
template <int D>
struct RowPart {
    float acc[D / 32], m, l;
};

// One row over the keys [lo, hi), all visible to it, by one warp: a key a lane
// for the scores, D / 32 elements a lane for the values, the running maximum
// and sum of the softmax in 32 bits. Reads no other key or value.
template <int D, typename T, bool PAGED>
__device__ __noinline__ RowPart<D> attend_row(const PrefillParams &p, int s, int row0, int row, int h, int lo, int hi) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int kvh = h / (p.num_heads / p.num_kv_heads);
    auto base = [&](const void *x, long long stride, int j) {
        return kv_row<D, T, PAGED>(p, x, stride, s, row0, kvh, j);
    };
    const uint32_t *qp =
        reinterpret_cast<const uint32_t *>(static_cast<const T *>(p.q) + (size_t)row * p.q_stride + (size_t)h * D);
    float q[E];  // elements lane * E ..
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
        const float2 x = Elem<T>::pair(qp[lane * (E / 2) + e]);
        q[2 * e] = p.negate ? -x.x : x.x;
        q[2 * e + 1] = p.negate ? -x.y : x.y;
    }
    RowPart<D> r;
    r.m = -INFINITY;
    r.l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) r.acc[e] = 0.f;
    for (int j0 = lo; j0 < hi; j0 += 32) {
        const int count = min(32, hi - j0);
        const uint4 *kp = reinterpret_cast<const uint4 *>(base(p.k, p.k_stride, j0 + min(lane, count - 1)));
        float dot = 0.f;
        for (int c = 0; c < D / 8; ++c) {
            float x[8];
            unpack8<T>(kp[c], x);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot = fmaf(x[i], __shfl_sync(FULL_MASK, q[i % E], c * 8 / E + i / E), dot);
        }
        const float z = lane < count ? dot * p.scale_log2 : -INFINITY;
        float mt = z;
#pragma unroll
        for (int o = 16; o; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(FULL_MASK, mt, o));
        const float m_new = fmaxf(r.m, mt);
        const float ref = m_new == -INFINITY ? 0.f : m_new;  // nothing above -inf yet
        const float f = exp2f(r.m - ref);
        const float w = lane < count ? exp2f(z - ref) : 0.f;
        r.m = m_new;
        float sum = w;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
        r.l = r.l * f + sum;
#pragma unroll
        for (int e = 0; e < E; ++e) r.acc[e] *= f;
        for (int c = 0; c < count; ++c) {
            const float wc = __shfl_sync(FULL_MASK, w, c);
            const uint32_t *vp = reinterpret_cast<const uint32_t *>(base(p.v, p.v_stride, j0 + c)) + lane * (E / 2);
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                const float2 x = Elem<T>::pair(vp[e]);
                r.acc[2 * e] = fmaf(wc, x.x, r.acc[2 * e]);
                r.acc[2 * e + 1] = fmaf(wc, x.y, r.acc[2 * e + 1]);
            }
        }
    }
    return r;
}

// Puts back the values that are not finite among the keys [from, to) of a KV head, which the products took as 0: the sum
// of those that a row sees is added to its stored result (PART: part, else output), a lane a row of the warp (seen: its
// visible keys, at most to; at: its row in the results). What a weight above 0 makes of an infinity or a NaN does not
// depend on the weight; where the key is not finite either, the weight may be 0 and the result is NaN.
template <int D, typename T, bool PAGED, bool PART>
__device__ __noinline__ void add_bad_values(const PrefillParams &p, int s, int row0, int kvh, int from, int to, int seen,
                                            size_t at) {
    constexpr int E = D / 32, AHEAD = 8;  // keys loaded at a time
    const int lane = threadIdx.x & 31;
    auto words = [&](const void *x, long long stride, int j) {  // this lane's elements of row j
        return reinterpret_cast<const uint32_t *>(kv_row<D, T, PAGED>(p, x, stride, s, row0, kvh, j)) + lane * (E / 2);
    };
    auto fine = [](float x) { return fabsf(x) < INFINITY; };
    float sum[E] = {};
    for (int j0 = from; j0 < to; j0 += AHEAD) {
        uint32_t v[AHEAD][E / 2];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int e = 0; e < E / 2; ++e) v[i][e] = words(p.v, p.v_stride, min(j0 + i, to - 1))[e];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int j = j0 + i;
            if (j >= to) break;
            bool bad = false;
            float add[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float2 x = Elem<T>::pair(v[i][e / 2]);
                add[e] = e % 2 ? x.y : x.x;
                bad = bad || !fine(add[e]);
            }
            if (__any_sync(FULL_MASK, bad)) {
                bool bad_key = false;
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    const float2 x = Elem<T>::pair(words(p.k, p.k_stride, j)[e]);
                    bad_key = bad_key || !fine(x.x) || !fine(x.y);
                }
                bad_key = __any_sync(FULL_MASK, bad_key);
#pragma unroll
                for (int e = 0; e < E; ++e) sum[e] += fine(add[e]) ? 0.f : bad_key ? NAN : add[e];
            }
            bool any = false;
#pragma unroll
            for (int e = 0; e < E; ++e) any = any || !fine(sum[e]);
            if (!__any_sync(FULL_MASK, any)) continue;
            for (unsigned rows = __ballot_sync(FULL_MASK, seen == j + 1); rows; rows &= rows - 1) {
                const size_t row = __shfl_sync(FULL_MASK, at, __ffs(rows) - 1);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (fine(sum[e])) continue;
                    if constexpr (PART) {
                        p.part_acc[row * D + lane * E + e] += sum[e];
                    } else {
                        T &o = static_cast<T *>(p.out)[row * D + lane * E + e];
                        o = T((float)o + sum[e]);
                    }
                }
            }
        }
    }
    __syncwarp();
}

// Stores a part of a split context as row `at` of the parts.
template <int D>
__device__ __forceinline__ void store_part(const PrefillParams &p, size_t at, const RowPart<D> &r) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < E; ++e) p.part_acc[at * D + lane * E + e] = r.acc[e];
    if (lane == 0) p.part_ml[at] = make_float2(r.m, r.l);
}

// Stores a row's output.
template <int D, typename T>
__device__ __forceinline__ void store_row(const PrefillParams &p, int row, int h, const RowPart<D> &r) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const size_t at = (size_t)row * p.num_heads + h;
    const float inv = 1.f / r.l;  // scores that are all -inf give 0 / 0
    uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<T *>(p.out) + at * D) + lane * (E / 2);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) out[e] = Elem<T>::pack(r.acc[2 * e] * inv, r.acc[2 * e + 1] * inv);
}

}  // namespace pa
