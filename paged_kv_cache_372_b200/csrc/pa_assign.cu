// pa_assign_slots: block tables, slots and positions of a step's tokens from
// request lengths (include/pa.h).
//
// Every quantity is a prefix sum over the requests: new tokens (the packed
// boundaries), blocks taken and blocks given back (places on the free stack).
// The requests are few (thousands) and the outputs may be many (a slot and a
// position for each new token), so every CTA sums over all the requests by
// itself, and the CTAs share the outputs; an output finds its request by a
// binary search in the sums, held in shared memory.
//
// The free stack after the ended requests' pushes is free_blocks[0 .. nf)
// followed by the released ids, so it is never materialised: the i-th block
// taken is entry top - 1 - i, read from the free list or straight from the
// ended request's table row. Only entries of the new stack at nf or above are
// written. No entry that is read is written (released and tail entries lie
// below a request's block count, new ones at or above it; the free list is
// read below nf and written from nf on), except where the caller passes the
// lengths in place: a single CTA writes those behind a barrier after its last
// read; where there are more, a second launch of one CTA sums again and writes
// them.
//
// Latency bounds it: a decode step's 256 tokens are one CTA and one launch
// (3.7 us in a graph, most of it the launch); 150,000 slots of 192 prompts took
// 31 us on a cluster of 8 CTAs, whose barrier let it write the lengths too, and
// take 9.5 with a CTA an SM and the second launch.
#include <atomic>

#define PA_ERROR_WORD_ELSEWHERE
#include "pa_common.cuh"
#include "pa_host.h"

namespace {

constexpr int ASSIGN_MAX_SEQS = 8192;

// What a launch writes: the outputs, the lengths and the size of the free list.
constexpr int ASSIGN_OUTPUTS = 1, ASSIGN_LENGTHS = 2;
constexpr int SUM_CAP = (1 << 30) - 1;  // prefix sums saturate here: above every valid total, and two of them fit an int

struct AssignParams {
    int32_t *block_tables, *free_blocks, *context_lens_out, *num_free_out, *positions, *cu_seqlens;
    int64_t *slot_mapping;
    const int32_t *context_lens, *num_free, *new_lens;
    int num_seqs, width, block_size, num_blocks, max_tokens, writes;
    unsigned int *errors;
};

__device__ __forceinline__ int sat_add(int a, int b) { return min(a + b, SUM_CAP); }

// The request s in [0, n) with off[s] <= x < off[s + 1] (x below off[n]).
__device__ __forceinline__ int find_seq(const int *off, int n, int x) {
    int lo = 0, hi = n;  // off[lo] <= x < off[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

template <int ASSIGN_THREADS>
__global__ void __launch_bounds__(ASSIGN_THREADS) pa_assign_kernel(const __grid_constant__ AssignParams p) {
    extern __shared__ int smem[];
    const int B = p.num_seqs, bs = p.block_size;
    int *tok = smem, *take = tok + B + 1, *back = take + B + 1, *ctx = back + B + 1;
    constexpr int NW = ASSIGN_THREADS / 32;
    __shared__ int warp_sum[3][NW];
    __shared__ int carry[3];
    __shared__ unsigned bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < 3) carry[tid] = 0;
    if (tid == 0) bad = 0u;
    const int nf = *p.num_free;
    __syncthreads();

    // Exclusive prefix sums of new tokens, blocks taken and blocks given back.
    const long long row_tokens = (long long)p.width * bs;
    for (int base = 0; base < B; base += ASSIGN_THREADS) {
        const int s = base + tid;
        int v[3] = {0, 0, 0};
        if (s < B) {
            int c = p.context_lens[s];
            int n = p.new_lens[s];
            if (c < 0 || c > row_tokens || (n > 0 && (long long)c + n > row_tokens)) {
                atomicOr(&bad, PA_DEVERR_CONTEXT);
                c = 0;
                n = 0;
            }
            const int held = (c + bs - 1) / bs;
            if (n < 0) {
                v[2] = held;
            } else {
                v[0] = min(n, SUM_CAP);
                v[1] = (c + n + bs - 1) / bs - held;
            }
            ctx[s] = c;
        }
        int mine[3] = {v[0], v[1], v[2]};
#pragma unroll
        for (int off = 1; off < 32; off <<= 1)
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const int up = __shfl_up_sync(pa::FULL_MASK, v[k], off);
                if (lane >= off) v[k] = sat_add(v[k], up);
            }
        if (lane == 31)
#pragma unroll
            for (int k = 0; k < 3; ++k) warp_sum[k][warp] = v[k];
        __syncthreads();
        if (warp < 3) {
            int w = lane < NW ? warp_sum[warp][lane] : 0;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int up = __shfl_up_sync(pa::FULL_MASK, w, off);
                if (lane >= off) w = sat_add(w, up);
            }
            if (lane < NW) warp_sum[warp][lane] = w;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int before = sat_add(carry[k], warp ? warp_sum[k][warp - 1] : 0);
            v[k] = sat_add(before, v[k]);  // inclusive
        }
        if (s < B) {
            // Exclusive values; a saturated sum is refused below.
            tok[s] = v[0] - mine[0];
            take[s] = v[1] - mine[1];
            back[s] = v[2] - mine[2];
        }
        __syncthreads();
        if (tid < 3) carry[tid] = sat_add(carry[tid], warp_sum[tid][NW - 1]);
        __syncthreads();
    }
    const int new_tokens = carry[0], taken = carry[1], given = carry[2];
    if (tid == 0) {
        tok[B] = new_tokens;
        take[B] = taken;
        back[B] = given;
        unsigned why = bad;
        if (new_tokens > p.max_tokens) why |= PA_DEVERR_TOKENS;
        if (nf < 0 || nf > p.num_blocks || given > p.num_blocks - nf || taken > nf + given) why |= PA_DEVERR_BLOCKS;
        bad = why;
        if (why && blockIdx.x == 0) atomicOr(p.errors, why);
    }
    __syncthreads();
    const bool ok = bad == 0u;
    const int worker = (int)blockIdx.x * ASSIGN_THREADS + tid;
    const int workers = (int)gridDim.x * ASSIGN_THREADS;
    bool bad_id = false;

    // Entry i of the stack of free blocks: the free list, then the released blocks.
    auto stack_at = [&](int i) {
        int id;
        if (i < nf) {
            id = p.free_blocks[i];
        } else {
            const int s = find_seq(back, B, i - nf);
            id = p.block_tables[(size_t)s * p.width + (i - nf - back[s])];
        }
        bad_id |= (unsigned)id >= (unsigned)p.num_blocks;
        return id;
    };
    if (ok && (p.writes & ASSIGN_OUTPUTS)) {
        const int top = nf + given, left = top - taken;
        for (int i = worker; i < taken; i += workers) {
            const int s = find_seq(take, B, i);
            const int held = (ctx[s] + bs - 1) / bs;
            p.block_tables[(size_t)s * p.width + held + (i - take[s])] = stack_at(top - 1 - i);
        }
        for (int i = nf + worker; i < left; i += workers) p.free_blocks[i] = stack_at(i);
        for (int t = worker; t < p.max_tokens; t += workers) {
            int pos = -1;
            int64_t slot = -1;
            if (t < new_tokens) {
                const int s = find_seq(tok, B, t);
                const int c = ctx[s];
                pos = c + (t - tok[s]);
                const int held = (c + bs - 1) / bs, j = pos / bs;
                int id;
                if (j < held) {
                    id = p.block_tables[(size_t)s * p.width + j];
                    bad_id |= (unsigned)id >= (unsigned)p.num_blocks;
                } else {
                    id = stack_at(top - 1 - (take[s] + j - held));
                }
                slot = (int64_t)id * bs + (pos - j * bs);
            }
            p.positions[t] = pos;
            p.slot_mapping[t] = slot;
        }
    } else if (p.writes & ASSIGN_OUTPUTS) {
        for (int t = worker; t < p.max_tokens; t += workers) {
            p.positions[t] = -1;
            p.slot_mapping[t] = -1;
        }
    }
    if (bad_id) atomicOr(p.errors, PA_DEVERR_BLOCK_ID);
    if (p.writes & ASSIGN_OUTPUTS)
        for (int s = worker; s <= B; s += workers) p.cu_seqlens[s] = ok ? tok[s] : 0;
    if (p.writes & ASSIGN_LENGTHS) {  // one CTA: it has read the lengths, they may now be replaced in place
        __syncthreads();
        for (int s = tid; s < B; s += ASSIGN_THREADS) {
            const int n = p.new_lens[s];
            p.context_lens_out[s] = !ok ? p.context_lens[s] : n < 0 ? 0 : ctx[s] + n;
        }
        if (tid == 0) *p.num_free_out = ok ? nf + given - taken : nf;
    }
}

template <int THREADS>
pa_status launch(const AssignParams &p, int ctas, cudaStream_t stream) {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> done[kMaxDevices];
    int dev, sms;
    const pa_status st = pa_internal_device(&dev, &sms);
    if (st != PA_OK) return st;
    if (!done[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(pa_assign_kernel<THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (4 * ASSIGN_MAX_SEQS + 3) * (int)sizeof(int));
        if (e != cudaSuccess) return pa_host::cuda_fail(e, "cudaFuncSetAttribute");
        done[dev].store(true, std::memory_order_release);
    }
    if (ctas > sms) ctas = sms;
    pa_assign_kernel<THREADS><<<ctas, THREADS, (4 * p.num_seqs + 3) * sizeof(int), stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return pa_host::cuda_fail(e, "pa_assign_slots launch");
    pa_internal_count_launch();
    return PA_OK;
}

}  // namespace

extern "C" pa_status pa_assign_slots(int32_t *block_tables, int32_t *free_blocks, int32_t *context_lens_out,
                                     int32_t *num_free_out, int64_t *slot_mapping, int32_t *positions,
                                     int32_t *cu_seqlens, const int32_t *context_lens, const int32_t *num_free,
                                     const int32_t *new_lens, int num_seqs, int max_blocks_per_seq, int block_size,
                                     int num_blocks, int max_tokens, pa_stream_t stream) {
    using namespace pa_host;
    pa_internal_set_last_error("");
    if (num_seqs < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || max_tokens < 0)
        return fail(PA_ERR_INVALID, "negative or zero size argument");
    if (!block_size_supported(block_size)) return fail(PA_ERR_UNSUPPORTED, "block_size %d", block_size);
    if (num_seqs > ASSIGN_MAX_SEQS) return fail(PA_ERR_UNSUPPORTED, "%d sequences (at most %d)", num_seqs, ASSIGN_MAX_SEQS);
    if (max_tokens >= SUM_CAP || num_blocks >= SUM_CAP || (long long)max_blocks_per_seq * block_size >= SUM_CAP)
        return fail(PA_ERR_UNSUPPORTED, "max_tokens, num_blocks and the tokens of a table row must be below 2^30 - 1");
    if (!free_blocks || !num_free_out || !cu_seqlens || !num_free ||
        (num_seqs > 0 && (!block_tables || !context_lens_out || !context_lens || !new_lens)) ||
        (max_tokens > 0 && (!slot_mapping || !positions)))
        return fail(PA_ERR_INVALID, "null pointer");
    if (!aligned(block_tables, 4) || !aligned(free_blocks, 4) || !aligned(context_lens_out, 4) ||
        !aligned(num_free_out, 4) || !aligned(slot_mapping, 8) || !aligned(positions, 4) || !aligned(cu_seqlens, 4) ||
        !aligned(context_lens, 4) || !aligned(num_free, 4) || !aligned(new_lens, 4))
        return fail(PA_ERR_INVALID, "misaligned pointer (4 B int32 arrays, 8 B slot_mapping)");
    AssignParams p{block_tables, free_blocks,  context_lens_out, num_free_out, positions,
                   cu_seqlens,   slot_mapping, context_lens,     num_free,     new_lens,
                   num_seqs,     max_blocks_per_seq, block_size, num_blocks,   max_tokens,
                   ASSIGN_OUTPUTS | ASSIGN_LENGTHS, nullptr};
    const pa_status st = pa_internal_error_word(&p.errors);
    if (st != PA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // One CTA where the outputs are few, a small one where the requests are too (us in a
    // graph, 256 threads / 1024 threads / a CTA an SM and the second launch: 256 requests of
    // one token 3.7 / 4.2 / 6.6; 64 of 16 6.2 / 4.8 / 7.4; 64 of 64 14.2 / 7.9 / 7.6; 64 of 256
    // 49.9 / 19.2 / 7.6; 8192 of one 66 / 27 / 29).
    if (max_tokens <= 512 && num_seqs <= 256) return launch<256>(p, 1, s);
    if (max_tokens <= 4096 || max_tokens <= num_seqs) return launch<1024>(p, 1, s);
    p.writes = ASSIGN_OUTPUTS;
    const pa_status out = launch<1024>(p, (max_tokens + 1023) / 1024, s);
    if (out != PA_OK) return out;
    p.writes = ASSIGN_LENGTHS;
    return launch<1024>(p, 1, s);
}
