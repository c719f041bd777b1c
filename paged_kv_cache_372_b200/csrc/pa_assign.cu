// pa_assign_slots: block tables, slots and positions of a step's tokens from
// request lengths (include/pa.h).
//
// Every quantity is a prefix sum over the requests: new tokens (the packed
// boundaries), blocks taken and blocks given back (places on the free stack).
// The requests are few (thousands) and the outputs may be many (a slot and a
// position for each new token), so each CTA of one cluster sums over all the
// requests by itself, and the CTAs share the output rows; an output finds its
// request by a binary search in the sums, held in shared memory.
//
// The free stack after the ended requests' pushes is free_blocks[0 .. nf)
// followed by the released ids, so it is never materialised: the i-th block
// taken is entry top - 1 - i, read from the free list or straight from the
// ended request's table row. Only entries of the new stack at nf or above are
// written. No entry that is read is written (released and tail entries lie
// below a request's block count, new ones at or above it; the free list is
// read below nf and written from nf on), except where the caller passes the
// lengths in place: those are written after a cluster barrier behind the
// last read.
#include <cooperative_groups.h>

#define PA_ERROR_WORD_ELSEWHERE
#include "pa_common.cuh"
#include "pa_host.h"

namespace {

namespace cg = cooperative_groups;

constexpr int ASSIGN_THREADS = 1024;
constexpr int ASSIGN_MAX_SEQS = 8192;
constexpr int ASSIGN_MAX_CLUSTER = 8;
constexpr int SUM_CAP = (1 << 30) - 1;  // prefix sums saturate here: above every valid total, and two of them fit an int

struct AssignParams {
    int32_t *block_tables, *free_blocks, *context_lens_out, *num_free_out, *positions, *cu_seqlens;
    int64_t *slot_mapping;
    const int32_t *context_lens, *num_free, *new_lens;
    int num_seqs, width, block_size, num_blocks, max_tokens;
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

__global__ void __launch_bounds__(ASSIGN_THREADS) pa_assign_kernel(AssignParams p) {
    extern __shared__ int smem[];
    const int B = p.num_seqs, bs = p.block_size;
    int *tok = smem, *take = tok + B + 1, *back = take + B + 1, *ctx = back + B + 1;
    __shared__ int warp_sum[3][32];
    __shared__ int carry[3];
    __shared__ unsigned bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cg::cluster_group cluster = cg::this_cluster();
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
            int w = warp_sum[warp][lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int up = __shfl_up_sync(pa::FULL_MASK, w, off);
                if (lane >= off) w = sat_add(w, up);
            }
            warp_sum[warp][lane] = w;
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
        if (tid < 3) carry[tid] = sat_add(carry[tid], warp_sum[tid][31]);
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
        if (why && cluster.block_rank() == 0) atomicOr(p.errors, why);
    }
    __syncthreads();
    const bool ok = bad == 0u;
    const int worker = (int)cluster.block_rank() * ASSIGN_THREADS + tid;
    const int workers = (int)cluster.num_blocks() * ASSIGN_THREADS;
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
    if (ok) {
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
    } else {
        for (int t = worker; t < p.max_tokens; t += workers) {
            p.positions[t] = -1;
            p.slot_mapping[t] = -1;
        }
    }
    if (bad_id) atomicOr(p.errors, PA_DEVERR_BLOCK_ID);
    for (int s = worker; s <= B; s += workers) p.cu_seqlens[s] = ok ? tok[s] : 0;
    // Every CTA has read the lengths: they may now be replaced in place.
    cluster.sync();
    for (int s = worker; s < B; s += workers) {
        const int n = p.new_lens[s];
        p.context_lens_out[s] = !ok ? p.context_lens[s] : n < 0 ? 0 : ctx[s] + n;
    }
    if (worker == 0) *p.num_free_out = ok ? nf + given - taken : nf;
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
                   num_seqs,     max_blocks_per_seq, block_size, num_blocks,   max_tokens, nullptr};
    pa_status st = pa_internal_error_word(&p.errors);
    if (st != PA_OK) return st;
    const int smem = (4 * num_seqs + 3) * (int)sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(pa_assign_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (4 * ASSIGN_MAX_SEQS + 3) * (int)sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    int ctas = 1;
    while (ctas < ASSIGN_MAX_CLUSTER && ctas * ASSIGN_THREADS * 4 < max_tokens) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(ASSIGN_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, pa_assign_kernel, p);
    if (e != cudaSuccess) return cuda_fail(e, "pa_assign_slots launch");
    pa_internal_count_launch();
    return PA_OK;
}
