// Host side of pa_prefill and pa_prefill_paged (include/pa.h).
#define PA_ERROR_WORD_ELSEWHERE
#include <cudaTypedefs.h>
#include <float.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "pa_host.h"
#include "pa_prefill_mma.cuh"

namespace {

using namespace pa_host;

// Rows [tokens][heads][D] with the given token stride, in boxes of 64 elements x
// box_heads x box_tokens, 128-byte swizzle.
pa_status encode_rows(PFN_cuTensorMapEncodeTiled enc, CUtensorMap *map, CUtensorMapDataType type, const void *x, int D,
                      int heads, int tokens, long long stride, int box_heads, int box_tokens) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens}, step[3] = {1, 1, 1};
    const CUresult r = enc(map, type, 3, const_cast<void *>(x), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PA_OK : fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

// A pool's (block, KV head) chunks, each one box: groups of 8 rows, and in a
// group one 64-element column of all 8 rows after the other.
pa_status encode_pool(PFN_cuTensorMapEncodeTiled enc, CUtensorMap *map, CUtensorMapDataType type, const void *x, int D,
                      int block_size, long long chunks) {
    const cuuint64_t dims[5] = {64, 8, (cuuint64_t)D / 64, (cuuint64_t)block_size / 8, (cuuint64_t)chunks};
    const cuuint64_t strides[4] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 16, (cuuint64_t)D * 2 * block_size};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)D / 64, (cuuint32_t)block_size / 8, 1}, step[5] = {1, 1, 1, 1, 1};
    const CUresult r = enc(map, type, 5, const_cast<void *>(x), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PA_OK : fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

constexpr int kMaxDevices = 64;

// Contexts of at least kSplitLeast key tiles are split below kSplitItems items an SM,
// where the longest item may be more than an SM's share, if the rows (token, query
// head) are few: each row's parts are written, read and joined, 3 ns a row, and a key
// tile is 1.4 us of one SM's time, so a third of a row a key tile is 10% more time. Where
// half of the SMs would have no item, up to kSplitRows rows a key of the longest.
// Split / not split in us, 32/8 heads of 128, tokens each (items an SM):
//   contexts of equal length
//   1 x 32768: 8 tokens (0.05) 37 / 267, 512 (0.43) 257 / 370, 1024 (0.86) 509 / 409 *
//   1 x 4096: 8 (0.05) 17 / 38, 128 (0.11) 35 / 55, 256 (0.22) 57 / 55, 512 (0.43) 87 / 57 *
//   16 x 32768 (0.86): 8 343 / 342, 32 404 / 336 *; whole prompt of 2048 (1.7) 212 / 53 *
//   contexts of 4096-32768
//   8 (0.43): 8 82 / 210; 16 (0.86): 8 199 / 263; 36 (1.95): 8 421 / 464; 48 (2.6): 8 571 / 565 *
//   contexts of 512-4096
//   8 (0.43): 8 27 / 35; 16 (0.86): 1 39 / 42, 16 60 / 43 *
// (*: the rule does not split). The device deals the key tiles to the SMs in equal
// shares. It counts those that a mask hides, so a prompt's first chunk is dealt unevenly.
constexpr int kSplitLeast = 16, kSplitRows = 2, kSplitItems = 2;

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Tokens of the two tiles of rows of an item.
int item_tokens(int num_heads, int num_kv_heads) { return pa::PF_NQ * pa::PF_BM / (num_heads / num_kv_heads); }

// Items of the packed tokens of num_seqs sequences, at most: each sequence has at most one that is not full.
long long max_items(int num_seqs, int num_tokens, int num_heads, int num_kv_heads) {
    return (num_tokens / item_tokens(num_heads, num_kv_heads) + (long long)std::min(num_seqs, num_tokens)) *
           num_kv_heads;
}

template <int D, typename T, bool PAGED>
pa_status launch(pa::PrefillParams &p, cudaStream_t stream) {
    int dev, sms;
    pa_status st = pa_internal_device(&dev, &sms);
    if (st != PA_OK) return st;
    void *fn;
    if ((st = pa_internal_tensor_map_encoder(&fn)) != PA_OK) return st;
    const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled>(fn);
    const auto type = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int group = p.num_heads / p.num_kv_heads;
    pa::PrefillMaps maps;
    if ((st = encode_rows(enc, &maps.q, type, p.q, D, p.num_heads, p.num_tokens, p.q_stride, group,
                          pa::PF_BM / group)) != PA_OK)
        return st;
    if (PAGED) {
        const long long chunks = (long long)p.num_blocks * p.num_kv_heads;
        if ((st = encode_pool(enc, &maps.k, type, p.k, D, p.block_size, chunks)) != PA_OK) return st;
        if ((st = encode_pool(enc, &maps.v, type, p.v, D, p.block_size, chunks)) != PA_OK) return st;
    } else {
        if ((st = encode_rows(enc, &maps.k, type, p.k, D, p.num_kv_heads, p.num_tokens, p.k_stride, 1, pa::PF_BN)) !=
            PA_OK)
            return st;
        if ((st = encode_rows(enc, &maps.v, type, p.v, D, p.num_kv_heads, p.num_tokens, p.v_stride, 1, pa::PF_BN)) !=
            PA_OK)
            return st;
    }
    using SH = pa::PrefillShape<D>;
    auto kernel = pa::pa_prefill_mma_kernel<D, T, PAGED>;
    static std::atomic<bool> done[kMaxDevices];
    if (!done[dev].load(std::memory_order_acquire)) {
        cudaFuncAttributes attr;
        cudaError_t e = cudaFuncGetAttributes(&attr, kernel);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes");
        if (attr.numRegs < SH::REGS_LAUNCH)  // the warps' shares come out of these
            return fail(PA_ERR_CUDA, "the kernel was built with %d registers a thread, %d needed", attr.numRegs,
                        SH::REGS_LAUNCH);
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SH::BYTES);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
        done[dev].store(true, std::memory_order_release);
    }
    const long long grid =
        p.deal ? p.deal_ctas : max_items(p.num_seqs, p.num_tokens, p.num_heads, p.num_kv_heads);
    if (grid >= (1ll << 31)) return fail(PA_ERR_UNSUPPORTED, "too many tiles");
    kernel<<<(unsigned)grid, SH::THREADS, SH::BYTES, stream>>>(p, maps);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, PAGED ? "pa_prefill_paged launch" : "pa_prefill launch");
    pa_internal_count_launch();
    if (PAGED && p.deal) {
        // Started early, it waits for the attention launch behind its own look-ups.
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(p.num_tokens * p.num_heads));
        cfg.blockDim = dim3(128);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, pa::pa_prefill_join_kernel<D, T>, p);
        if (e != cudaSuccess) return cuda_fail(e, "pa_prefill_paged launch");
        pa_internal_count_launch();
    }
    return PA_OK;
}

template <bool PAGED>
pa_status dispatch(pa::PrefillParams &p, int head_dim, int dtype, cudaStream_t s) {
    if (head_dim == 128)
        return dtype == PA_F16 ? launch<128, __half, PAGED>(p, s) : launch<128, __nv_bfloat16, PAGED>(p, s);
    return dtype == PA_F16 ? launch<64, __half, PAGED>(p, s) : launch<64, __nv_bfloat16, PAGED>(p, s);
}

// Whether a paged call's contexts are split.
bool splits(int num_seqs, int num_tokens, int num_heads, int num_kv_heads, int max_keys, int sms) {
    const long long items = std::max<long long>(std::min(num_seqs, num_tokens),
                                                ceil_div(num_tokens, item_tokens(num_heads, num_kv_heads))) *
                            num_kv_heads;
    const long long tiles = ceil_div(max_keys, pa::PF_BN), rows = (long long)num_tokens * num_heads;
    if (items >= kSplitItems * sms || tiles < kSplitLeast) return false;
    return 3 * rows <= items * tiles || (2 * items <= sms && rows <= (long long)kSplitRows * max_keys);
}

// Places for the parts of a split call: struct Deal. Each has room for an item's rows.
long long part_slots(int num_seqs, int num_tokens, int num_heads, int num_kv_heads, int sms) {
    return max_items(num_seqs, num_tokens, num_heads, num_kv_heads) + sms;
}

constexpr size_t kPartRows = pa::PF_NQ * pa::PF_BM;

size_t parts_bytes(long long slots, int head_dim) {
    return (size_t)slots * kPartRows * (sizeof(float2) + head_dim * sizeof(float));
}

// The limit of a wait: 4 s, and for each key that a row may see the time that the
// 32 rows of a warp take for it one after the other in the row form (100 ns each
// with the keys in L2, three times that allowed), since the other warps wait
// meanwhile for this item's end.
unsigned long long wait_limit_ns(int max_keys) { return 4000000000ull + 10000ull * max_keys; }

template <bool PAGED>
pa_status run(pa::PrefillParams &p, int head_dim, float scale, int dtype, cudaStream_t s) {
    // A negative scale is a positive one of the negated queries (the matrix
    // instruction negates them); 0 stands for the least positive one, so that
    // a masked score of -inf stays -inf.
    const float a = fabsf(scale) * 1.4426950408889634f;
    p.scale_log2 = a < FLT_MIN ? FLT_MIN : a;
    p.negate = scale < 0.f;
    p.wait_ns = wait_limit_ns(PAGED ? p.ctx_limit : p.num_tokens);
    return dispatch<PAGED>(p, head_dim, dtype, s);
}

bool heads_supported(int num_heads, int num_kv_heads) {
    if (num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads) return false;
    const int g = num_heads / num_kv_heads;
    return g == 1 || g == 2 || g == 4 || g == 8;
}

// What both entry points check before anything else.
pa_status check_common(int num_seqs, int num_tokens, int num_heads, int num_kv_heads, int head_dim, float scale,
                       int dtype) {
    if (num_seqs < 0 || num_tokens < 0) return fail(PA_ERR_INVALID, "negative size argument");
    if (dtype != PA_F16 && dtype != PA_BF16) return fail(PA_ERR_INVALID, "dtype %d", dtype);
    if (!heads_supported(num_heads, num_kv_heads))
        return fail(PA_ERR_UNSUPPORTED, "heads %d/%d (1, 2, 4 or 8 query heads per KV head)", num_heads, num_kv_heads);
    if (num_heads > 65535) return fail(PA_ERR_UNSUPPORTED, "more than 65535 heads");
    if (head_dim != 64 && head_dim != 128) return fail(PA_ERR_UNSUPPORTED, "head_dim %d", head_dim);
    if (num_tokens >= (1 << 27)) return fail(PA_ERR_UNSUPPORTED, "num_tokens must be below 2^27");
    if (!(scale - scale == 0.f) || fabsf(scale) > FLT_MAX / 2)
        return fail(PA_ERR_INVALID, "scale must be finite and at most 2^127 in magnitude");
    return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_prefill(void *out, const void *q, const void *k, const void *v, const int32_t *cu_seqlens, int num_seqs,
                     int num_tokens, int num_heads, int num_kv_heads, int head_dim, int q_stride, int k_stride,
                     int v_stride, float scale, int dtype, pa_stream_t stream) {
    pa_internal_set_last_error("");
    pa_status st = check_common(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, scale, dtype);
    if (st != PA_OK) return st;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!out || !q || !k || !v || !cu_seqlens) return fail(PA_ERR_INVALID, "null pointer");
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(cu_seqlens, 4))
        return fail(PA_ERR_INVALID, "misaligned pointer (16 B tensors, 4 B cu_seqlens)");
    const long long q_row = (long long)num_heads * head_dim, kv_row = (long long)num_kv_heads * head_dim;
    if (q_stride % 8 || k_stride % 8 || v_stride % 8 || q_stride < q_row || k_stride < kv_row || v_stride < kv_row)
        return fail(PA_ERR_INVALID, "token strides must be multiples of 8 and hold a token's heads");
    pa::PrefillParams p{};
    p.out = out;
    p.q = q;
    p.k = k;
    p.v = v;
    p.cu_seqlens = cu_seqlens;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    if ((st = pa_internal_error_word(&p.errors)) != PA_OK) return st;
    return run<false>(p, head_dim, scale, dtype, static_cast<cudaStream_t>(stream));
}

size_t pa_prefill_paged_workspace_size(int num_seqs, int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                       int block_size, int max_context_len) {
    if (num_seqs < 0 || num_tokens < 0 || max_context_len < 0 || !heads_supported(num_heads, num_kv_heads) ||
        num_heads > 65535 || (head_dim != 64 && head_dim != 128) || !block_size_supported(block_size) ||
        num_tokens >= (1 << 27) || max_context_len >= (1 << 30))
        return 0;
    if (num_seqs == 0 || num_tokens == 0) return 256;
    int dev, sms;
    if (pa_internal_device(&dev, &sms) != PA_OK) return 0;
    // Enough for every call that is no larger: one that splits has fewer than kSplitItems
    // full items an SM, and as many that are not full.
    if (ceil_div(max_context_len, pa::PF_BN) < kSplitLeast) return 256;
    const long long most = (2 * kSplitItems + 1) * sms;
    return parts_bytes(std::min(part_slots(num_seqs, num_tokens, num_heads, num_kv_heads, sms), most), head_dim);
}

pa_status pa_prefill_paged(void *out, const void *q, const void *k_pool, const void *v_pool,
                           const int32_t *block_tables, const int32_t *context_lens, const int32_t *cu_seqlens,
                           int num_seqs, int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                           int block_size, int max_blocks_per_seq, int num_blocks, int max_context_len, int q_stride,
                           float scale, int dtype, void *workspace, size_t workspace_bytes, pa_stream_t stream) {
    pa_internal_set_last_error("");
    if (max_blocks_per_seq <= 0 || num_blocks <= 0 || max_context_len < 0)
        return fail(PA_ERR_INVALID, "negative or zero size argument");
    pa_status st = check_common(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, scale, dtype);
    if (st != PA_OK) return st;
    if (!block_size_supported(block_size)) return fail(PA_ERR_UNSUPPORTED, "block_size %d", block_size);
    if (max_context_len >= (1 << 30) || (long long)num_blocks * num_kv_heads >= (1ll << 31))
        return fail(PA_ERR_UNSUPPORTED, "max_context_len must be below 2^30, num_blocks * num_kv_heads below 2^31");
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !context_lens || !cu_seqlens || !workspace)
        return fail(PA_ERR_INVALID, "null pointer");
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(cu_seqlens, 4) || !aligned(workspace, 256))
        return fail(PA_ERR_INVALID, "misaligned pointer (16 B tensors, 4 B int arrays, 256 B workspace)");
    if (q_stride % 8 || q_stride < (long long)num_heads * head_dim)
        return fail(PA_ERR_INVALID, "the token stride must be a multiple of 8 and hold a token's heads");
    if (workspace_bytes < 256) return fail(PA_ERR_INVALID, "workspace %zu bytes < 256", workspace_bytes);
    int dev, sms;
    if ((st = pa_internal_device(&dev, &sms)) != PA_OK) return st;
    const bool deal = splits(num_seqs, num_tokens, num_heads, num_kv_heads, max_context_len, sms);
    const long long slots = deal ? part_slots(num_seqs, num_tokens, num_heads, num_kv_heads, sms) : 0;
    const size_t need = deal ? parts_bytes(slots, head_dim) : 256;
    if (workspace_bytes < need)
        return fail(PA_ERR_INVALID, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    pa::PrefillParams p{};
    p.out = out;
    p.q = q;
    p.k = k_pool;
    p.v = v_pool;
    p.cu_seqlens = cu_seqlens;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    const long long table_tokens = (long long)max_blocks_per_seq * block_size;
    p.ctx_limit = (int)(table_tokens < max_context_len ? table_tokens : max_context_len);
    p.q_stride = q_stride;
    if ((st = pa_internal_error_word(&p.errors)) != PA_OK) return st;
    p.deal = deal;
    p.deal_ctas = sms;  // a CTA an SM
    p.part_slots = (int)slots;
    p.part_ml = static_cast<float2 *>(workspace);
    p.part_acc = reinterpret_cast<float *>(p.part_ml + slots * kPartRows);
    return run<true>(p, head_dim, scale, dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
