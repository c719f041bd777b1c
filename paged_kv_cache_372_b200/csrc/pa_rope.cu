// pa_rope_and_cache: rotary positions of q and k, and the write of the rotated
// k and of v into the paged cache (include/pa.h).
//
// One pass over the rows: every element is read once and written once (k twice
// where k_out is wanted too), so the copy bandwidth bounds it (8192 tokens of 96
// heads of 128: 80 us, 5.9 TB/s). A thread handles
// two 16-byte vectors at a time whose elements pair up under the rotation: in
// the half layout the vectors at 8u and rot_dim/2 + 8u, interleaved the two
// neighbours at 16u; both use frequencies 8u .. 8u+7. The angles belong to the
// token and are shared by all its heads: a CTA computes the cosines and sines
// of its tokens once, into shared memory.
//
// The angle p * inv_freq is reduced in 64 bits: in turns, t = p * (inv_freq /
// 2 pi), a - 2 pi rint(t) has |t - rint(t)| <= 1/2, and only that remainder is
// rounded to 32 bits (2^-25 turns), so a position of 2^20 is as good as 0.
#define PA_ERROR_WORD_ELSEWHERE
#include "pa_common.cuh"
#include "pa_host.h"

namespace {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_W = 3;            // units a thread has in flight
constexpr int ROPE_MAX_TOKENS = 16;  // tokens of a CTA

struct RopeParams {
    void *q_out, *k_out;
    const void *q, *k, *v;
    void *k_pool, *v_pool;
    const int32_t *positions;
    const int64_t *slot_mapping;
    const double *inv_freq;
    int num_tokens, num_heads, num_kv_heads, head_dim, rot_dim, block_size;
    long long num_slots;
    int q_stride, k_stride, v_stride;
    float mscale;
    int lanes_log2, tokens_per_cta;  // threads of a token, tokens of a CTA
    unsigned int *errors;
};

// Rotates the 8 pairs of two vectors; cs holds (cos, sin) of their frequencies.
template <typename T, bool INTERLEAVED>
__device__ __forceinline__ void rotate(uint4 &a, uint4 &b, const float2 *cs) {
    float x[8], y[8];
    pa::unpack8<T>(a, x);
    pa::unpack8<T>(b, y);
    if constexpr (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 c = cs[i], d = cs[i + 4];
            const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
            x[2 * i] = x0 * c.x - x1 * c.y;
            x[2 * i + 1] = x1 * c.x + x0 * c.y;
            y[2 * i] = y0 * d.x - y1 * d.y;
            y[2 * i + 1] = y1 * d.x + y0 * d.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 c = cs[i];
            const float x0 = x[i], y0 = y[i];
            x[i] = x0 * c.x - y0 * c.y;
            y[i] = y0 * c.x + x0 * c.y;
        }
    }
    using E = pa::Elem<T>;
    a = make_uint4(E::pack(x[0], x[1]), E::pack(x[2], x[3]), E::pack(x[4], x[5]), E::pack(x[6], x[7]));
    b = make_uint4(E::pack(y[0], y[1]), E::pack(y[2], y[3]), E::pack(y[4], y[5]), E::pack(y[6], y[7]));
}

// D: head size, W: units (pairs of vectors) a thread has in flight.
template <typename T, bool INTERLEAVED, int D, int W>
__global__ void __launch_bounds__(ROPE_THREADS) pa_rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float2 cs[ROPE_MAX_TOKENS][64];
    constexpr int UNITS = D / 16;  // units of a head
    const int rot = p.rot_dim, half = rot / 2;
    const int H = p.num_heads, Hkv = p.num_kv_heads;
    const int t0 = blockIdx.x * p.tokens_per_cta;
    const int nt = min(p.tokens_per_cta, p.num_tokens - t0);
    for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
        const int t = i / half, f = i - t * half;
        const double turns = (double)p.positions[t0 + t] * (p.inv_freq[f] * 0.15915494309189533577);
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        cs[t][f] = make_float2(c * p.mscale, s * p.mscale);
    }
    __syncthreads();
    const int per_token = (H + (p.v_pool ? 2 : 1) * Hkv) * UNITS;
    const int lanes = 1 << p.lanes_log2, lane = threadIdx.x & (lanes - 1);
    for (int tl = threadIdx.x >> p.lanes_log2; tl < nt; tl += blockDim.x >> p.lanes_log2) {
        const int t = t0 + tl;
        if (p.positions[t] < 0) continue;
        int64_t at = -1;  // first element of the token's slot in head 0
        if (p.k_pool) {
            const int64_t slot = p.slot_mapping[t];
            if (slot >= p.num_slots) {
                if (lane == 0) atomicOr(p.errors, PA_DEVERR_SLOT);
            } else if (slot >= 0) {
                const int64_t blk = slot / p.block_size;
                at = (blk * Hkv * p.block_size + (slot - blk * p.block_size)) * D;
            }
        }
        const T *q = static_cast<const T *>(p.q) + (size_t)t * p.q_stride;
        const T *k = static_cast<const T *>(p.k) + (size_t)t * p.k_stride;
        const T *v = static_cast<const T *>(p.v) + (size_t)t * p.v_stride;
        for (int r0 = lane; r0 < per_token; r0 += lanes * W) {
            uint4 a[W], b[W];
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const int r = r0 + w * lanes, head = r / UNITS, u = r % UNITS;
                if (r >= per_token) break;
                const bool is_v = head >= H + Hkv, turn = !is_v && 16 * u < rot;
                const T *src = head < H ? q + (size_t)head * D : is_v ? v + (size_t)(head - H - Hkv) * D : k + (size_t)(head - H) * D;
                a[w] = *reinterpret_cast<const uint4 *>(src + (turn && !INTERLEAVED ? 8 * u : 16 * u));
                b[w] = *reinterpret_cast<const uint4 *>(src + (turn && !INTERLEAVED ? half + 8 * u : 16 * u + 8));
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const int r = r0 + w * lanes, head = r / UNITS, u = r % UNITS;
                if (r >= per_token) break;
                const bool is_q = head < H, is_v = head >= H + Hkv, turn = !is_v && 16 * u < rot;
                const int e0 = turn && !INTERLEAVED ? 8 * u : 16 * u;
                const int e1 = turn && !INTERLEAVED ? half + 8 * u : 16 * u + 8;
                if (turn) rotate<T, INTERLEAVED>(a[w], b[w], &cs[tl][8 * u]);
                if (is_q) {
                    T *dst = static_cast<T *>(p.q_out) + ((size_t)t * H + head) * D;
                    *reinterpret_cast<uint4 *>(dst + e0) = a[w];
                    *reinterpret_cast<uint4 *>(dst + e1) = b[w];
                    continue;
                }
                const int h = is_v ? head - H - Hkv : head - H;
                if (!is_v && p.k_out) {
                    T *dst = static_cast<T *>(p.k_out) + ((size_t)t * Hkv + h) * D;
                    *reinterpret_cast<uint4 *>(dst + e0) = a[w];
                    *reinterpret_cast<uint4 *>(dst + e1) = b[w];
                }
                if (at >= 0) {
                    T *dst = static_cast<T *>(is_v ? p.v_pool : p.k_pool) + at + (int64_t)h * p.block_size * D;
                    *reinterpret_cast<uint4 *>(dst + e0) = a[w];
                    *reinterpret_cast<uint4 *>(dst + e1) = b[w];
                }
            }
        }
    }
}

template <typename T, bool INTERLEAVED>
void launch(const RopeParams &p, unsigned grid, unsigned threads, cudaStream_t s) {
    if (p.head_dim == 128)
        pa_rope_kernel<T, INTERLEAVED, 128, ROPE_W><<<grid, threads, 0, s>>>(p);
    else
        pa_rope_kernel<T, INTERLEAVED, 64, ROPE_W><<<grid, threads, 0, s>>>(p);
}

}  // namespace

extern "C" pa_status pa_rope_and_cache(void *q_out, void *k_out, const void *q, const void *k, const void *v,
                                       void *k_pool, void *v_pool, const int32_t *positions,
                                       const int64_t *slot_mapping, const void *inv_freq, int num_tokens,
                                       int num_heads, int num_kv_heads, int head_dim, int rot_dim, int interleaved,
                                       int block_size, int num_blocks, int q_stride, int k_stride, int v_stride,
                                       float mscale, int dtype, pa_stream_t stream) {
    using namespace pa_host;
    pa_internal_set_last_error("");
    const bool cache = k_pool || v_pool;
    if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || (cache && num_blocks <= 0))
        return fail(PA_ERR_INVALID, "negative or zero size argument");
    if (dtype != PA_F16 && dtype != PA_BF16) return fail(PA_ERR_INVALID, "dtype %d", dtype);
    if (head_dim != 64 && head_dim != 128) return fail(PA_ERR_UNSUPPORTED, "head_dim %d", head_dim);
    if (rot_dim <= 0 || rot_dim % 16 || rot_dim > head_dim)
        return fail(PA_ERR_UNSUPPORTED, "rot_dim %d (a multiple of 16 in [16, head_dim])", rot_dim);
    if (cache && !block_size_supported(block_size)) return fail(PA_ERR_UNSUPPORTED, "block_size %d", block_size);
    if (num_heads > 65536 || num_kv_heads > 65536) return fail(PA_ERR_UNSUPPORTED, "more than 65536 heads");
    if (!(mscale - mscale == 0.f)) return fail(PA_ERR_INVALID, "mscale must be finite");
    if (num_tokens == 0) return PA_OK;
    if (!q_out || !q || !k || !positions || !inv_freq) return fail(PA_ERR_INVALID, "null pointer");
    if (cache && (!k_pool || !v_pool || !v || !slot_mapping))
        return fail(PA_ERR_INVALID, "k_pool, v_pool, v and slot_mapping go together");
    if (!cache && !k_out) return fail(PA_ERR_INVALID, "neither k_out nor pools to take the rotated keys");
    if (!aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(positions, 4) || !aligned(slot_mapping, 8) ||
        !aligned(inv_freq, 8))
        return fail(PA_ERR_INVALID, "misaligned pointer (16 B tensors, 8 B inv_freq and slot_mapping, 4 B positions)");
    const long long q_row = (long long)num_heads * head_dim, kv_row = (long long)num_kv_heads * head_dim;
    if (q_stride % 8 || k_stride % 8 || q_stride < q_row || k_stride < kv_row ||
        (cache && (v_stride % 8 || v_stride < kv_row)))
        return fail(PA_ERR_INVALID, "token strides must be multiples of 8 and hold a token's heads");
    if ((q_out == q && q_stride != q_row) || (k_out == k && k_stride != kv_row))
        return fail(PA_ERR_INVALID, "in place needs a contiguous input");
    RopeParams p{q_out, k_out, q, k, v, k_pool, v_pool, positions, slot_mapping, static_cast<const double *>(inv_freq),
                 num_tokens, num_heads, num_kv_heads, head_dim, rot_dim, cache ? block_size : 16,
                 cache ? (long long)num_blocks * block_size : 0, q_stride, k_stride, v_stride, mscale, 5, 1, nullptr};
    int dev, sms;
    pa_status st = pa_internal_device(&dev, &sms);
    if (st != PA_OK) return st;
    if ((st = pa_internal_error_word(&p.errors)) != PA_OK) return st;
    // A token has the threads that its units fill with ROPE_W each in flight, a CTA as
    // many tokens at a time as fit, two times where the tokens are many; fewer where the
    // SMs would not have two CTAs each. (2049 tokens of 24 heads of 64: 5.9 us, 11.8 with a
    // whole CTA a token; 8192 tokens of 96 heads of 128: 80 us with two tokens a CTA, 83 with
    // one or four.)
    const int units = (num_heads + (cache ? 2 : 1) * num_kv_heads) * (head_dim / 16);
    p.lanes_log2 = 5;
    while ((1 << p.lanes_log2) < ROPE_THREADS && (ROPE_W << p.lanes_log2) < units) ++p.lanes_log2;
    int at_once = ROPE_THREADS >> p.lanes_log2;
    while (at_once > 1 && num_tokens / at_once < 2 * sms) at_once /= 2;
    const unsigned threads = (unsigned)at_once << p.lanes_log2;
    p.tokens_per_cta = num_tokens / (2 * at_once) < 8 * sms ? at_once : 2 * at_once;
    const unsigned grid = (unsigned)((num_tokens + (long long)p.tokens_per_cta - 1) / p.tokens_per_cta);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == PA_F16)
        interleaved ? launch<__half, true>(p, grid, threads, s) : launch<__half, false>(p, grid, threads, s);
    else
        interleaved ? launch<__nv_bfloat16, true>(p, grid, threads, s) : launch<__nv_bfloat16, false>(p, grid, threads, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "pa_rope_and_cache launch");
    pa_internal_count_launch();
    return PA_OK;
}
