// Tensor-core kernel of pa_prefill and pa_prefill_paged (include/pa.h).
//
// A work item is two tiles of 128 query rows of one (sequence, KV head), walked
// over the keys they see in tiles of 128. The rows are (token, query head) pairs
// of the group, head fastest: all query heads of a KV head share its key and value
// tiles, and a tile spans few tokens, so little of it is masked. For each tile
//   S = Q K^T      tcgen05.mma, both operands in shared memory, S in TMEM
//   P = exp2(S * scale_log2 - m + lift)   a thread for each row, in registers; P
//                  rounded to the input type goes back to TMEM over S
//   O += P V       tcgen05.mma, P from TMEM, V from shared memory, O in TMEM
// m is a running maximum of the row and l the running sum, both 32 bits; O and
// l are rescaled only when the maximum has grown by more than 2^8 (P 2^-lift then
// stays below 2^8), which after the first tiles is rare. P is rounded since the
// products take one type; the sum l is of the weights before that rounding.
//
// Warps: four softmax warps for each tile of rows, one that issues the copies
// (TMA), one for each tile of rows that issues its matrix instructions, and one
// that finds the next work item. While the softmax of one tile of rows runs, the
// other's products do: at head size 128 a tile needs 128 x 128 exponentials at
// 16 a clock and 4 x 128^3 product operations at 8192 a clock, 1024 clocks
// either way, so 4 or 5 of 16 exponentials go to the FMA units (ex2_fma).
//
// CTAs are persistent: a CTA that works on an item takes over the launch of the
// next one that has not started (clusterlaunchcontrol) and its copies and first
// product run ahead of the item's end; with a CTA for each item its set-up and end
// cost 16,000 clocks, as much as five key tiles. Items come longest first.
//
// Measured (head size 128): a key tile of both tiles of rows takes about 2,700
// clocks, 2,048 of them products: the chain of a tile of rows (scores 512, to
// registers 150, maximum 300, exponentials 1,200, hand-over twice 200, last
// quarter of the product 128) is what remains, and two chains are all that the
// 512 columns of TMEM hold. 16384 tokens, 32/8 heads, bf16: 1.53 ms after a pause
// (1,437 TFLOP/s at 1.8 GHz), 1.78 ms back to back, where 1,000 W hold the clock
// at 1.45 GHz. The tensor pipe is active 73% of the time. 5-8 tokens of 8 requests
// over 4096-32768 tokens: 92 us, 5.3 TB/s of the cache.
//
// Masked places: S is replaced by -inf there (a selection, so NaN and
// infinities in masked keys do not spread) and P is 0. Value rows that no row of an
// item sees are made 0. A NaN or infinity in another masked value row still comes
// through 0 x V. So an item with a row that is not finite is walked again: this time
// the copying warp looks through the value rows that are hidden from some row (at
// most 256, at the diagonal) when they have landed, and makes what is not finite 0
// there (clear_bad); at the item's end it is added to the results of the rows that
// see it (add_bad_values). Looked through in every item, by whichever warps, they
// cost 2 to 6% of a call. A row whose scores are NaN or infinite is NaN as it is.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "pa_prefill.cuh"

namespace pa {

// Of 16 pairs of exponentials, those on the FMA units. 8192 tokens, 32/8 heads of
// 64, us at 0 / 2 / 4 / 6 / 8 pairs: bf16 350 / 385 / 340 / 345 / 367, fp16 352 / 374 /
// 340 / 345 / 381; 16384 tokens, heads of 128, bf16, at 3 / 4 / 5 / 6: 1585 / 1510 / 1495 / 1493,
// LLaMA-7B-shaped prompts, fp16, 199 / 192 / 190 / 195.
template <int D>
constexpr int PF_POLY = D == 64 ? 4 : 5;
// What the weights are relative to, m * scale_log2, is rounded to 32 bits: a row's weights all carry a factor, up
// to 2^(1/4) at the size below, which cancels. It grows with the scores (2^32 at 2^30), until the weights leave fp16's
// range or ex2_fma's. Rows whose maximum has been past this size are computed again by the row form, which
// subtracts the maximum from the scaled scores.
constexpr float PF_COARSE = 4194304.f;  // 2^22
// What an item's warps say of it: a row is not finite, it has to be walked again; values were made 0.
constexpr uint32_t PF_AGAIN = 1, PF_CLEARED = 2;
// Sums of weights are below this: 2^30 keys of 2^15. From here on one of them was NaN.
constexpr float PF_SOUND = 1152921504606846976.f;  // 2^60
// Weights are lifted to where the type has room. fp16: by 2^7, so that the largest
// (2^15 and the factor above) is just below 65504 and rounding is to 2^-32 of the
// largest, not 2^-25: long contexts of small weights add up. bf16, whose range has
// room below: by 2^-8, so that none is above 1 and sums of values overflow no sooner.
template <typename T>
constexpr float PF_LIFT = std::is_same<T, __half>::value ? 7.f : -8.f;

template <int D>
struct PrefillShape {
    static constexpr int HALVES = D / 64;     // 128-byte columns of a row
    static constexpr int TILE = 128 * D * 2;  // bytes of a tile of rows (queries, keys or values)
    static constexpr int SOFTMAX_WARPS = PF_NQ * 4;
    static constexpr int COPY_WARP = SOFTMAX_WARPS, MMA_WARP = COPY_WARP + 1, PLAN_WARP = COPY_WARP + 3;
    static constexpr int THREADS = SOFTMAX_WARPS * 32 + 128;
    static constexpr int STAGES = D == 128 ? 5 : 8;
    // Registers move from the other warps to the softmax warps: 384 threads x 168 = 256 x 216 + 128 x 72.
    static constexpr int REGS_LAUNCH = 168, REGS_SOFTMAX = 216, REGS_OTHER = 72;
    static_assert(SOFTMAX_WARPS * 32 * REGS_SOFTMAX + 128 * REGS_OTHER <= THREADS * REGS_LAUNCH,
                  "more registers than launched");
    static constexpr int TMEM_COLS = 512;
    static constexpr int S_COL = 0, O_COL = PF_NQ * 128;
    static constexpr int OFF_KV = PF_NQ * TILE;
    static constexpr int OFF_NEXT = OFF_KV + STAGES * TILE;  // 16 bytes: the launch taken over
    static constexpr int OFF_ITEM = OFF_NEXT + 16;           // the work item, 11 integers
    static constexpr int OFF_TMEM = OFF_ITEM + 48;           // TMEM address
    static constexpr int OFF_NOTE = OFF_TMEM + 4;            // of an item and the next: PF_AGAIN, PF_CLEARED
    static constexpr int OFF_BAR = OFF_TMEM + 16;
    static constexpr int NUM_BARS = 2 * STAGES + 6 + 6 * PF_NQ;
    static constexpr int OFF_SWAP = OFF_BAR + (NUM_BARS + 1) / 2 * 16;  // the second tile's maxima and sums
    static constexpr int BYTES = OFF_SWAP + PF_BM * 8 + 1024;           // and slack for the alignment to 1024
};

// ---- tcgen05 ------------------------------------------------------------------------------------------
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The matrix instructions and their commits are issued by the one thread whose
// `one` is set; the whole warp runs the code around them, so that descriptors
// and addresses stay in uniform registers. (Issued under a branch of one lane,
// 8 instructions took 650 to 970 clocks to issue, more than they run.)
// A value that all lanes have, as a uniform register (a warp reduction leaves it in one).
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(FULL_MASK, x); }

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one;
}

__device__ __forceinline__ void tc_commit(uint32_t bar, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(one)
        : "memory");
}

// Shared-memory matrix descriptor with the 128-byte swizzle: start address and
// leading byte offset in the low word, stride byte offset, version 1 (bit 46)
// and swizzle (bit 61) in the high word, all in units of 16 bytes.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return addr >> 4 | (lbo >> 4) << 16; }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo) { return sbo >> 4 | 1u << 14 | 2u << 29; }

__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t add, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %6, 0;\n\tsetp.ne.u32 e, %7, 0;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(add), "r"(one)
        : "memory");
}

// A from TMEM.
__device__ __forceinline__ void tc_mma_ta(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                          uint32_t add, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 e, %6, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(add), "r"(one)
        : "memory");
}

// 32 columns of this thread's lane; there after tc_landed.
__device__ __forceinline__ void tc_ld32(uint32_t addr, float *x) {
    uint32_t *r = reinterpret_cast<uint32_t *>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}

// Ties loaded registers to the wait before: nothing that uses them moves above it.
template <int N>
__device__ __forceinline__ void tc_pin(float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(x[i]));
}

// Waits for the loads issued before, x among them.
template <int N>
__device__ __forceinline__ void tc_landed(float (&x)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    tc_pin(x);
}

__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ uint32_t load_shared(uint32_t at) {
    uint32_t x;
    asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
    return x;
}

// A set bit 15 or 31 for each half that is NaN or infinite: a full exponent carries into the sign's place.
template <typename T>
__device__ __forceinline__ uint32_t bad_halves(uint32_t x) {
    constexpr uint32_t MASK = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
    constexpr uint32_t ONE = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
    return (x & MASK) + ONE & 0x80008000u;
}

__device__ __forceinline__ uint4 load_shared_16(uint32_t at) {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
    return x;
}

// Makes what is NaN or infinite 0 in the value rows [from, to) of a stage, by one warp, and says so before in the word
// at `note`. GROUP, HALF: bytes from 8 rows to the next 8, and from one 64-element column to the next.
template <int D, typename T, uint32_t GROUP, uint32_t HALF>
__device__ __forceinline__ void clear_bad(uint32_t stage, int from, int to, uint32_t note) {
    constexpr int VECTORS = D / 8;  // of a row
    for (int i = from * VECTORS + (threadIdx.x & 31); i < to * VECTORS; i += 32) {
        const int row = i / VECTORS, col = i % VECTORS;
        const uint32_t at = stage + (row >> 3) * GROUP + (col >> 3) * HALF + (row & 7) * 128 + (col & 7) * 16;
        const uint4 x = load_shared_16(at);
        const uint32_t bx = bad_halves<T>(x.x), by = bad_halves<T>(x.y), bz = bad_halves<T>(x.z), bw = bad_halves<T>(x.w);
        if (bx | by | bz | bw) {
            auto good = [](uint32_t x, uint32_t bad) { return x & ~((bad >> 15) * 0xffffu); };
            asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(note), "r"(PF_CLEARED) : "memory");
            asm volatile("st.volatile.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(good(x.x, bx)),
                         "r"(good(x.y, by)), "r"(good(x.z, bz)), "r"(good(x.w, bw))
                         : "memory");
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// ---- tensor-map copies --------------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// The whole chunk `row` of a pool: (block, KV head) rows in groups of 8, 128-byte columns.
__device__ __forceinline__ void tma_load_chunk(uint32_t dst, const CUtensorMap *map, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %2, %2, %2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(bar)
        : "memory");
}

// 32 bytes at once: a whole sector of a row, where each lane has a row.
__device__ __forceinline__ void store_32b(void *at, const uint32_t *x) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                 "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)),
          "l"(*reinterpret_cast<uint64_t *>(&c)));
    return *reinterpret_cast<float2 *>(&r);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// 2^x without the special-function unit: x = n + f with n the nearest integer
// (adding 1.5 x 2^23 leaves it in the low bits), 2^f by a polynomial and n added
// to the exponent. The coefficients minimise the largest relative error on
// [-1/2, 1/2] with the constant term 1 (a linear programme over 4001 points):
// 1.0e-4 of degree 3 for bf16, whose weights are rounded to 2^-9, 2.9e-6 of degree
// 4 for fp16. x below -127 counts as -127, whose f is 0 and whose result is 0.
// x up to 16; a NaN gives a weight near 2^128, past any that a sum of others reaches (PF_SOUND).
template <typename T>
__device__ __forceinline__ float2 ex2_fma(float2 x) {
    x.x = max_nan(x.x, -127.f);
    x.y = max_nan(x.y, -127.f);
    const float2 big = make_float2(12582912.f, 12582912.f), less = make_float2(-12582912.f, -12582912.f);
    const float2 r = add2(x, big);
    const float2 f = fma2(add2(r, less), make_float2(-1.f, -1.f), x);
    float2 y;
    auto c = [](float v) { return make_float2(v, v); };
    if constexpr (std::is_same<T, __half>::value) {
        y = fma2(f, c(0.009582576f), c(0.055906828f));
        y = fma2(f, y, c(0.24024107f));
        y = fma2(f, y, c(0.6931241f));
    } else {
        y = fma2(f, c(0.05500906f), c(0.24221097f));
        y = fma2(f, y, c(0.6932829f));
    }
    y = fma2(f, y, c(1.f));
    y.x = __int_as_float(__float_as_int(y.x) + (__float_as_int(r.x) << 23));
    y.y = __int_as_float(__float_as_int(y.y) + (__float_as_int(r.y) << 23));
    return y;
}

struct PrefillMaps {
    CUtensorMap q, k, v;
};

template <int D, typename T, bool PAGED>
__global__ void __launch_bounds__(PrefillShape<D>::THREADS, 1)
    pa_prefill_mma_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ PrefillMaps maps) {
    using SH = PrefillShape<D>;
    constexpr int HALVES = SH::HALVES, NS = SH::STAGES, NQ = PF_NQ;
    // Keys and values: rows of 128 bytes in groups of 8 (1024 bytes), for the
    // packed form column after column, for the pools' chunks row group after row group.
    constexpr uint32_t KV_GROUP = PAGED ? HALVES * 1024 : 1024, KV_HALF = PAGED ? 1024 : 16384;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    const uint32_t base = smem_u32(smem);
    const uint32_t bars = base + SH::OFF_BAR;
    auto kv_full = [&](int i) { return bars + 8 * i; };
    auto kv_empty = [&](int i) { return bars + 8 * (NS + i); };
    const uint32_t item_full = bars + 8 * (2 * NS), item_empty = item_full + 8, next_full = item_full + 16,
                   pair_full = item_full + 24, pair_empty = item_full + 32, look_full = item_full + 40;
    auto stream_bar = [&](int k, int t) { return bars + 8 * (2 * NS + 6 + k * NQ + t); };
    auto q_full = [&](int t) { return stream_bar(0, t); };
    auto q_empty = [&](int t) { return stream_bar(1, t); };
    auto s_full = [&](int t) { return stream_bar(2, t); };
    auto p_most = [&](int t) { return stream_bar(3, t); };
    auto p_full = [&](int t) { return stream_bar(4, t); };
    auto o_full = [&](int t) { return stream_bar(5, t); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + SH::OFF_TMEM);

    const int warp = __shfl_sync(FULL_MASK, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int group = p.num_heads / p.num_kv_heads;
    const int tm = PF_BM / group;  // tokens of a tile of rows

    if (warp == SH::COPY_WARP) {
        if (lane == 0) {
            for (int i = 0; i < NS; ++i) {
                mbar_init(kv_full(i), 1);
                mbar_init(kv_empty(i), NQ);
            }
            mbar_init(item_full, 1);
            mbar_init(item_empty, SH::SOFTMAX_WARPS + 1 + NQ);
            mbar_init(next_full, 1);
            mbar_init(pair_full, 4);
            mbar_init(pair_empty, 4);
            mbar_init(look_full, 1);
            for (int t = 0; t < NQ; ++t) {
                mbar_init(q_full(t), 1);
                mbar_init(q_empty(t), 1);
                mbar_init(s_full(t), 1);
                mbar_init(p_most(t), 4);
                mbar_init(p_full(t), 4);
                mbar_init(o_full(t), 1);
            }
            fence_barrier_init();
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.q)) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k)) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.v)) : "memory");
        }
        __syncwarp();
    } else if (warp == SH::MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "n"(SH::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(FULL_MASK, *tmem_slot, 0);

    // A wait that runs out ends this warp's work: the error bit is set, later
    // waits and work are skipped, and the CTA still frees its TMEM. The limit is
    // longer than an item can last (wait_limit_ns).
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (alive && !__all_sync(FULL_MASK, mbar_wait_bounded(bar, parity, p.wait_ns))) {
            alive = false;
            if (lane == 0) atomicOr(p.errors, PA_DEVERR_TIMEOUT);
        }
        return alive;
    };
    // The nth item, for every warp but the one that finds them.
    auto next_item = [&](int nth, Item &it) {
        if (!wait(item_full, nth & 1)) return false;
        const int *at = reinterpret_cast<const int *>(smem + SH::OFF_ITEM);
        it.s = __shfl_sync(FULL_MASK, at[0], 0);
        it.tok0 = __shfl_sync(FULL_MASK, at[1], 0);
        it.row0 = __shfl_sync(FULL_MASK, at[2], 0);
        it.n = __shfl_sync(FULL_MASK, at[3], 0);
        it.keys = __shfl_sync(FULL_MASK, at[4], 0);
        it.slot = __shfl_sync(FULL_MASK, at[5], 0);
        it.parts = __shfl_sync(FULL_MASK, at[6], 0);
        it.kvh = __shfl_sync(FULL_MASK, at[7], 0);
        it.j0 = __shfl_sync(FULL_MASK, at[8], 0);
        it.j1 = __shfl_sync(FULL_MASK, at[9], 0);
        it.look = __shfl_sync(FULL_MASK, at[10], 0);
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty);
        return it.s >= 0;
    };

    if (warp >= SH::SOFTMAX_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SH::REGS_OTHER));
        if (warp == SH::PLAN_WARP) {
            // ---- finds the work items ----
            Finder<PAGED> finder;
            const bool deal = PAGED && p.deal;
            unsigned bad = 0;
            int launches = 0;   // asked for
            bool more = true;   // there may be further items
            auto find_next = [&](Item &it) {
                if (deal) return finder.next_piece(p, NQ * tm, it, bad);
                int index = blockIdx.x;
                if (launches > 0) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(next_full, 16);
                        asm volatile(
                            "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                            ::"r"(base + SH::OFF_NEXT), "r"(next_full)
                            : "memory");
                    }
                    __syncwarp();
                    if (!wait(next_full, (launches - 1) & 1)) return false;
                    uint32_t taken, x;
                    asm volatile(
                        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
                        "ld.shared.b128 r, [%2];\n\t"
                        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
                        "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
                        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
                        : "=r"(taken), "=r"(x)
                        : "r"(base + SH::OFF_NEXT)
                        : "memory");
                    fence_proxy_async_smem();  // read before it is written again
                    index = __shfl_sync(FULL_MASK, taken ? (int)x : -1, 0);
                }
                ++launches;
                return index >= 0 && finder.find(p, index, NQ * tm, it, bad);
            };
            // Items go out one ahead of the softmax warps. When all warps have one, the softmax warps are done with
            // the one before, and what they say of it holds: it goes out again, or the next one does. Behind the last
            // an empty item (no rows) waits for what they say of that.
            Item last{}, before{};
            for (int nth = 0;; ++nth) {
                Item it{};
                it.parts = 1;
                const uint32_t note = base + SH::OFF_NOTE + (nth & 1) * 4;
                if (nth >= 2 && __shfl_sync(FULL_MASK, load_shared(note), 0) == PF_AGAIN) {
                    it = before;
                    it.look = 1;
                } else if (more && (more = find_next(it))) {
                    it.look = 0;
                } else if (nth == 0 || last.n == 0 || last.look) {
                    it.s = -1;
                }
                if (nth == 0 && __any_sync(FULL_MASK, bad != 0) && bad) atomicOr(p.errors, bad);
                __syncwarp();
                if (lane == 0) {
                    tmem_slot[1 + (nth & 1)] = 0;
                    int *at = reinterpret_cast<int *>(smem + SH::OFF_ITEM);
                    at[0] = it.s;
                    at[1] = it.tok0;
                    at[2] = it.row0;
                    at[3] = it.n;
                    at[4] = it.keys;
                    at[5] = it.slot;
                    at[6] = it.parts;
                    at[7] = it.kvh;
                    at[8] = it.j0;
                    at[9] = it.j1;
                    at[10] = it.look;
                    mbar_arrive(item_full);
                }
                __syncwarp();
                if (it.s < 0 || !wait(item_empty, nth & 1)) break;
                before = last;
                last = it;
            }
        } else if (warp == SH::COPY_WARP) {
            // ---- copies ----
            Item it;
            int c = 0, uses[NQ] = {}, looks = 0;  // chunks (key or value tiles) issued; query tiles; chunks looked through
            for (int nth = 0; alive && next_item(nth, it); ++nth) {
                const Walk w = walk_of(it, tm, PAGED);
                auto queries = [&](int t) {
                    if (w.count[t] == 0 || (uses[t] > 0 && !wait(q_empty(t), (uses[t] - 1) & 1))) return;
                    ++uses[t];
                    if (lane == 0) {
                        mbar_arrive_expect_tx(q_full(t), SH::TILE);
                        for (int h = 0; h < HALVES; ++h)
                            tma_load_3d(base + t * SH::TILE + h * 16384, &maps.q, h * 64, it.kvh * group,
                                        it.row0 + it.tok0 + (w.halves ? 0 : t * tm), q_full(t));
                    }
                    __syncwarp();
                };
                queries(0);
                const int per_tile = PAGED ? PF_BN / p.block_size : 0;
                auto block_of = [&](int j) {  // this lane's block of key tile j
                    const int b = j * per_tile + lane;
                    int id = 0;
                    if (lane < per_tile && b * p.block_size < w.kv_end) {
                        id = p.block_tables[(size_t)it.s * p.max_blocks_per_seq + b];
                        if ((unsigned)id >= (unsigned)p.num_blocks) {
                            atomicOr(p.errors, PA_DEVERR_BLOCK_ID);
                            id = 0;
                        }
                    }
                    return id;
                };
                const int hidden = w.first + it.tok0 + 1;  // keys from here on are hidden from some row
                // Two forms of the loop: the tests for the rare one in the other's code cost 2 to 5% of a call.
                auto copy_tiles = [&](auto looking) {
                    constexpr bool LOOK = decltype(looking)::value;
                    int id_next = 0;
                    if constexpr (PAGED) id_next = block_of(w.j0);
                    for (int j = w.j0; j < w.j1 && alive; ++j) {
                        [[maybe_unused]] const int id = id_next;
                        if constexpr (PAGED) {
                            if (j + 1 < w.j1) id_next = block_of(j + 1);
                        }
#pragma unroll
                        for (int kv = 0; kv < 2; ++kv) {
                            const int stage = c % NS;
                            if (c >= NS && !wait(kv_empty(stage), (c / NS - 1) & 1)) break;
                            const CUtensorMap *map = kv ? &maps.v : &maps.k;
                            const uint32_t dst = base + SH::OFF_KV + stage * SH::TILE;
                            const bool look = LOOK && kv && (j + 1) * PF_BN > hidden;
                            const uint32_t full = look ? look_full : kv_full(stage);
                            if constexpr (PAGED) {
                                const int chunk = p.block_size * D * 2;
                                const int blocks = min(per_tile, (w.kv_end - j * PF_BN + p.block_size - 1) / p.block_size);
                                if (lane == 0) mbar_arrive_expect_tx(full, blocks * chunk);
                                __syncwarp();
                                if (lane < blocks)
                                    tma_load_chunk(dst + lane * chunk, map, id * p.num_kv_heads + it.kvh, full);
                            } else if (lane == 0) {
                                mbar_arrive_expect_tx(full, SH::TILE);
                                for (int h = 0; h < HALVES; ++h)
                                    tma_load_3d(dst + h * 16384, map, h * 64, it.kvh, it.row0 + j * PF_BN, full);
                            }
                            if constexpr (LOOK) {
                                if (look) {
                                    ++looks;
                                    if (!wait(look_full, (looks - 1) & 1)) break;
                                    clear_bad<D, T, KV_GROUP, KV_HALF>(dst, max(hidden - j * PF_BN, 0),
                                                                       min(w.kv_end - j * PF_BN, PF_BN),
                                                                       base + SH::OFF_NOTE + (nth & 1) * 4);
                                    if (lane == 0) mbar_arrive(kv_full(stage));
                                }
                            }
                            __syncwarp();
                            ++c;
                            // The second tile of rows still multiplies the last item's keys: its
                            // queries come behind the first keys.
                            if (kv == 0 && j == w.j0) queries(1);
                        }
                    }
                };
                if (it.look)
                    copy_tiles(std::true_type());
                else
                    copy_tiles(std::false_type());
            }
            if (!alive) {  // copies in flight land before the CTA leaves
                for (int i = max(0, c - NS); i < c; ++i) mbar_wait_bounded(kv_full(i % NS), (i / NS) & 1, p.wait_ns);
                if (looks > 0) mbar_wait_bounded(look_full, (looks - 1) & 1, p.wait_ns);
                for (int t = 0; t < NQ; ++t)
                    if (uses[t] > 0) mbar_wait_bounded(q_full(t), (uses[t] - 1) & 1, p.wait_ns);
            }
        } else if (warp < SH::MMA_WARP + NQ) {
            // ---- matrix instructions: a warp for each tile of rows ----
            // Instruction descriptor: 32-bit accumulator, both operands of the input
            // type (0 fp16, 1 bf16), N / 8 at bit 17, M / 16 at bit 24; bit 13 negates
            // A, bit 16 takes B with its columns contiguous.
            constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
            constexpr uint32_t common = 1u << 4 | type << 7 | type << 10 | (uint32_t)(PF_BM >> 4) << 24;
            const uint32_t idesc_qk = common | (p.negate ? 1u << 13 : 0u);  // and N
            constexpr uint32_t idesc_pv = common | (uint32_t)(D >> 3) << 17 | 1u << 16;
            const uint32_t one = elect_one();
            const int t = warp - SH::MMA_WARP;
            const uint32_t s_at = uniform(tmem + SH::S_COL + t * 128), o_at = uniform(tmem + SH::O_COL + t * D);
            auto qk = [&](int stage, int cols) {  // cols: keys, a multiple of 16
                const uint32_t idesc = idesc_qk | (uint32_t)(cols >> 3) << 17;
                const uint32_t q = desc_lo(base + t * SH::TILE, 16), k = desc_lo(base + SH::OFF_KV + stage * SH::TILE, 16);
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    tc_mma(s_at, q + ((i >> 2) * 16384 + (i & 3) * 32) / 16, desc_hi(1024),
                           k + ((i >> 2) * KV_HALF + (i & 3) * 32) / 16, desc_hi(KV_GROUP), idesc, i > 0, one);
                tc_commit(s_full(t), one);
            };
            int weights = 0;  // tiles of weights taken
            // The product with the values in a stage; there: keys of the tile below kv_end, cols: those multiplied.
            auto pv = [&](int stage, int there, int cols, bool add) {
                const uint32_t v = base + SH::OFF_KV + stage * SH::TILE, vd = desc_lo(v, KV_HALF);
                if (there < cols) {
                    // Value rows behind all that is seen (slots behind the context, the next sequence's
                    // rows) hold anything: their weights are 0, their values made 0.
                    for (int i = there * HALVES * 8 + lane; i < cols * HALVES * 8; i += 32) {
                        const int row = i / (HALVES * 8), col = i % (HALVES * 8);
                        const uint32_t at = v + (row >> 3) * KV_GROUP + (col >> 3) * KV_HALF + (row & 7) * 128 + (col & 7) * 16;
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                auto step = [&](int i) {  // keys 16 i to 16 i + 15
                    tc_mma_ta(o_at, s_at + i * 8, vd + i * 2 * KV_GROUP / 16, desc_hi(KV_GROUP), idesc_pv, add || i > 0,
                              one);
                };
                const int steps = cols / 16;
                // The product starts on the first three quarters of the weights.
                if (!wait(p_most(t), weights & 1)) return;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < 6; ++i)
                    if (i < steps) step(i);
                if (!wait(p_full(t), weights & 1)) return;
                tc_fence_after();
                if (steps > 6) step(6);
                if (steps > 7) step(7);
                ++weights;
            };
            Item it;
            int c = 0, uses = 0;  // chunks taken, query tiles
            for (int nth = 0; alive && next_item(nth, it); ++nth) {
                const Walk w = walk_of(it, tm, PAGED);
                const int tiles = w.j1 - w.j0, mine = t == 0 ? w.count[0] : w.count[1];
                if (tiles == 0) continue;
                // Keys of tile j that any row of this one sees, in the steps of 16 of the products.
                const int end = t == 0 ? w.end[0] : w.end[1];
                auto cols = [&](int j) { return min((end - (w.j0 + j) * PF_BN + 15) & ~15, PF_BN); };
                auto there = [&](int j) { return w.kv_end - (w.j0 + j) * PF_BN; };
                if (mine > 0) {
                    if (!wait(q_full(t), uses & 1)) break;
                    ++uses;
                }
                if (PAGED && w.halves) {
                    // Every other key tile, chunks in their order.
                    for (int j = 0; j < tiles; ++j, c += 2) {
                        const bool own = (j & 1) == t;
                        const int sk = c % NS, sv = (c + 1) % NS;
                        if (!wait(kv_full(sk), (c / NS) & 1)) break;
                        if (own) {
                            qk(sk, cols(j));
                            if (j + 2 >= tiles) tc_commit(q_empty(t), one);
                        }
                        tc_commit(kv_empty(sk), one);
                        if (!wait(kv_full(sv), ((c + 1) / NS) & 1)) break;
                        if (own) {
                            pv(sv, there(j), cols(j), j > 1);
                            if (!alive) break;
                            if (j + 2 >= tiles) tc_commit(o_full(t), one);
                        }
                        tc_commit(kv_empty(sv), one);
                    }
                    continue;
                }
                if (!wait(kv_full(c % NS), (c / NS) & 1)) break;
                if (mine > 0) {
                    qk(c % NS, cols(0));
                    if (mine == 1) tc_commit(q_empty(t), one);
                }
                tc_commit(kv_empty(c % NS), one);
                ++c;
                for (int j = 0; j < tiles; ++j) {
                    const int sv = c % NS, sk = (c + 1) % NS;
                    if (!wait(kv_full(sv), (c / NS) & 1)) break;
                    const bool more = j + 1 < tiles;
                    if (more && !wait(kv_full(sk), ((c + 1) / NS) & 1)) break;
                    if (j < mine) {
                        pv(sv, there(j), cols(j), j > 0);
                        if (!alive) break;
                        // The next scores follow in the same pipe: they replace weights that are read by then.
                        if (j + 1 < mine) {
                            qk(sk, cols(j + 1));
                            if (j + 2 == mine) tc_commit(q_empty(t), one);
                        } else {
                            tc_commit(o_full(t), one);
                        }
                    }
                    tc_commit(kv_empty(sv), one);
                    ++c;
                    if (more) {
                        tc_commit(kv_empty(sk), one);
                        ++c;
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SH::REGS_SOFTMAX));
        // ---- softmax: a thread for each row ----
        const int t = warp >> 2, quarter = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_addr = lanes + SH::S_COL + t * 128, o_addr = lanes + SH::O_COL + t * D;
        const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
        const bool wide = reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
        Item it;
        int scores = 0, results0 = 0, results1 = 0, pairs = 0;  // tiles of scores taken, accumulators, items in halves
        for (int nth = 0; alive && next_item(nth, it); ++nth) {
            const Walk w = walk_of(it, tm, PAGED);
            const int mine = t == 0 ? w.count[0] : w.count[1];
            const int r = quarter * 32 + lane, tok0 = it.tok0 + (w.halves ? 0 : t * tm);  // row of the tile
            const int tok = tok0 + r / group, head = it.kvh * group + r % group;
            const bool valid = tok < it.n;
            const int visible = valid ? max(w.first + tok + 1, 0) : 0;
            // Keys that all of the warp's rows see.
            const int clear = max(w.first + tok0 + (r - lane) / group + 1, 0);
            float m = -INFINITY, l = 0.f;  // m: what the weights are relative to, unscaled
            bool coarse = false;           // m has been past PF_COARSE
            for (int j = 0; j < mine; ++j) {
                if (!wait(s_full(t), scores & 1)) break;
                ++scores;
                tc_fence_after();
                float x[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tc_ld32(s_addr + c * 32, x[c]);
                tc_landed(x[0]);
#pragma unroll
                for (int c = 1; c < 4; ++c) tc_pin(x[c]);
                const int key0 = (w.j0 + (w.halves ? 2 * j + t : j)) * PF_BN;
                if (key0 + PF_BN > clear) {
                    const int left = visible - key0;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        {
                        const int rest = left - c * 32;
                        const uint32_t seen_bits = rest >= 32 ? ~0u : rest <= 0 ? 0u : (1u << rest) - 1u;
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[c][i] = (seen_bits >> i) & 1u ? x[c][i] : -INFINITY;
                    }
                }
                float mx[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; i += 2) mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], x[c][i], x[c][i + 1]);
                const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                const bool grow = (top - m) * p.scale_log2 > 8.f;
                if (__any_sync(FULL_MASK, grow)) {
                    const float f = grow ? ex2((m - top) * p.scale_log2) : 1.f;
                    m = grow ? top : m;
                    coarse = coarse || (fabsf(m) * p.scale_log2 >= PF_COARSE && fabsf(m) < INFINITY);
                    l = l < PF_SOUND ? l * f : NAN;
                    if (j > 0) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            tc_ld32(o_addr + c, o);
                            tc_landed(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= f;
                            tc_st32(o_addr + c, reinterpret_cast<uint32_t *>(o));
                        }
                    }
                }
                // nothing above -inf yet: weights 0
                const float ref = m == -INFINITY ? 0.f : fmaf(-m, p.scale_log2, PF_LIFT<T>);
                const float2 ref2 = make_float2(ref, ref);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                auto weigh = [&](int c) {
                    uint32_t y16[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 y = fma2(make_float2(x[c][2 * i], x[c][2 * i + 1]), scale2, ref2);
                        if (i * PF_POLY<D> % 16 < PF_POLY<D>)
                            y = ex2_fma<T>(y);
                        else
                            y = make_float2(ex2(y.x), ex2(y.y));
                        sum[i & 1] = add2(sum[i & 1], y);
                        y16[i] = Elem<T>::pack(y.x, y.y);
                    }
                    tc_st16(s_addr + c * 16, y16);
                };
                auto ready = [&](uint32_t bar) {
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar);
                };
                // One form for all tiles: a second one for masked tiles, which skips what none of the
                // warp's rows sees, made the loop longer and every call 3 to 6% slower.
                weigh(0);
                weigh(1);
                weigh(2);
                ready(p_most(t));
                weigh(3);
                ready(p_full(t));
                const float2 both = add2(sum[0], sum[1]);
                l += both.x + both.y;
            }
            // ---- the item's rows ----
            const int lo = w.j0 * PF_BN, hi = min(visible, w.j1 * PF_BN);  // keys the row has seen here
            const bool some = hi > lo;
            float f0 = 1.f, f1 = 0.f;  // what the two tiles' results are multiplied by
            if (w.halves) {
                float2 *swap = reinterpret_cast<float2 *>(smem + SH::OFF_SWAP) + r;
                if (t == 1) {
                    *swap = make_float2(m, coarse ? -1.f : l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pair_full);
                    if (!wait(pair_empty, pairs & 1)) break;
                    ++pairs;
                    ++results0;
                    ++results1;
                    continue;
                }
                if (!wait(pair_full, pairs & 1) || !wait(o_full(1), results1 & 1)) break;
                ++pairs;
                const float2 other = *swap;
                coarse = coarse || other.y < 0.f;
                const float top = fmaxf(m, other.x);
                f0 = m == -INFINITY ? 0.f : ex2((m - top) * p.scale_log2);
                f1 = other.x == -INFINITY ? 0.f : ex2((other.x - top) * p.scale_log2);
                l = (l < PF_SOUND ? l : NAN) * f0 + (other.y < PF_SOUND ? other.y : NAN) * f1;
                m = top;
            }
            // Else a score is NaN or +inf, or none is above -inf: the row is NaN.
            const bool sound = l > 0.f && l < PF_SOUND;
            if (it.parts == 1) {
                const float inv = sound ? 1.f / l : NAN;
                f0 *= inv;
                f1 *= inv;
            } else if (!(l < PF_SOUND)) {
                l = NAN;
            }
            if (mine > 0) {
                if (!wait(o_full(t), (t == 0 ? results0 : results1) & 1)) break;
                tc_fence_after();
            }
            results0 += w.count[0] > 0;
            results1 += w.count[1] > 0;
            const size_t at = (size_t)(it.row0 + tok) * p.num_heads + head;
            const size_t part_at = (size_t)it.slot * (NQ * PF_BM) + (tok0 - it.tok0) * group + r;
            float2 nan[4] = {};  // 0 as long as all that goes in is finite
            const uint32_t other_addr = w.halves ? o_addr + D : o_addr;  // not in halves: f1 is 0
#pragma unroll 1
            for (int c = 0; c < D && mine > 0; c += 32) {
                float o[32];
                tc_ld32(o_addr + c, o);
                if constexpr (PAGED) {
                    float other[32];
                    tc_ld32(other_addr + c, other);
                    tc_landed(o);
                    tc_pin(other);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = fmaf(other[i], f1, o[i] * f0);
                } else {
                    tc_landed(o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] *= f0;
                }
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float2 &at = nan[(i >> 1) & 3];
                    at = fma2(make_float2(o[i], o[i + 1]), make_float2(0.f, 0.f), at);
                }
                __syncwarp();
                if (!valid) {
                    // rows of no token: nothing to store
                } else if (PAGED && it.parts > 1) {
                    uint32_t *out = reinterpret_cast<uint32_t *>(p.part_acc + part_at * D + c);
#pragma unroll
                    for (int i = 0; i < 32; i += 8) store_32b(out + i, reinterpret_cast<uint32_t *>(o) + i);
                } else {
                    uint32_t y[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[i] = Elem<T>::pack(o[2 * i], o[2 * i + 1]);
                    T *out = static_cast<T *>(p.out) + at * D + c;
                    if (wide) {
                        store_32b(out, y);
                        store_32b(out + 16, y + 8);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            reinterpret_cast<uint4 *>(out)[i] =
                                make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                    }
                }
                __syncwarp();
            }
            if (PAGED && it.parts > 1 && valid)
                p.part_ml[part_at] =
                    make_float2(some ? -fmaf(-m, p.scale_log2, PF_LIFT<T>) : -INFINITY, some ? l : 0.f);
            if (valid && !some) {  // a row that sees nothing here: zeros, over what is in its place
                const uint32_t none[8] = {};
                if (PAGED && it.parts > 1) {
                    for (int c = 0; c < D; c += 8) store_32b(p.part_acc + part_at * D + c, none);
                } else {
                    uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + at * D);
                    for (int i = 0; i < D / 8; ++i) out[i] = make_uint4(0, 0, 0, 0);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (w.halves && lane == 0) mbar_arrive(pair_empty);
            const float2 any = add2(add2(nan[0], nan[1]), add2(nan[2], nan[3]));
            const uint32_t note = base + SH::OFF_NOTE + (nth & 1) * 4;
            // Not finite, though the weights are (in a part they may all be 0).
            const bool unsure = some && !coarse && !(any.x + any.y == 0.f) && (it.parts == 1 ? sound : l < PF_SOUND);
            if (!it.look) {
                if (__any_sync(FULL_MASK, unsure) && lane == 0)
                    asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(note), "r"(PF_AGAIN) : "memory");
            } else if (__any_sync(FULL_MASK, load_shared(note) == PF_CLEARED)) {
                const int from = max(w.first + it.tok0 + 1, lo), to = min(w.kv_end, w.j1 * PF_BN);
                if (PAGED && it.parts > 1)
                    add_bad_values<D, T, PAGED, true>(p, it.s, it.row0, it.kvh, from, to, hi, part_at);
                else
                    add_bad_values<D, T, PAGED, false>(p, it.s, it.row0, it.kvh, from, to, hi, at);
            }
            for (unsigned rows = __ballot_sync(FULL_MASK, some && coarse); rows; rows &= rows - 1) {
                const int src = __ffs(rows) - 1;
                const int row = it.row0 + __shfl_sync(FULL_MASK, tok, src), h = __shfl_sync(FULL_MASK, head, src);
                const RowPart<D> part =
                    attend_row<D, T, PAGED>(p, it.s, it.row0, row, h, lo, __shfl_sync(FULL_MASK, hi, src));
                if (PAGED && it.parts > 1)
                    store_part<D>(p, __shfl_sync(FULL_MASK, part_at, src), part);
                else
                    store_row<D, T>(p, row, h, part);
            }
        }
    }
    __syncthreads();
    if (warp == SH::MMA_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(SH::TMEM_COLS));
    }
}

// Joins the parts of split contexts: four warps for each (token, head) row, a
// quarter of the parts each.
//   out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i,  M = max_i m_i
template <int D, typename T>
__global__ void __launch_bounds__(128) pa_prefill_join_kernel(const __grid_constant__ PrefillParams p) {
    constexpr int E = D / 32;
    __shared__ float acc_of[4][D];
    __shared__ float2 ml_of[4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int item = blockIdx.x, row = item / p.num_heads;
    // The last sequence that starts at or before the row.
    int lo = 0, hi = p.num_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_seqlens[mid] <= row)
            lo = mid;
        else
            hi = mid;
    }
    // The parts of its chain, from all sequences' chains.
    __shared__ long long sums[4][3];
    __shared__ int most[4];
    unsigned bad = 0;
    const int TM = PF_NQ * PF_BM / (p.num_heads / p.num_kv_heads);
    long long sum = 0, before = 0, chains_before = 0;
    int longest = 1;
    for (int s = threadIdx.x; s < p.num_seqs; s += 128) {
        const Deal d = Deal::of(seq_range<true>(p, s, bad), TM);
        sum += d.all(p);
        before += s < lo ? d.all(p) : 0;
        chains_before += s < lo ? (long long)d.chains * p.num_kv_heads : 0;
        if (d.chains > 0) longest = max(longest, d.tiles);
    }
    sum = warp_sum(sum);
    before = warp_sum(before);
    chains_before = warp_sum(chains_before);
    longest = __reduce_max_sync(FULL_MASK, longest);
    if (lane == 0) sums[warp][0] = sum, sums[warp][1] = before, sums[warp][2] = chains_before, most[warp] = longest;
    __syncthreads();
    sum = sums[0][0] + sums[1][0] + sums[2][0] + sums[3][0];
    before = sums[0][1] + sums[1][1] + sums[2][1] + sums[3][1];
    chains_before = sums[0][2] + sums[1][2] + sums[2][2] + sums[3][2];
    longest = max(max(most[0], most[1]), max(most[2], most[3]));
    const SeqRange r = seq_range<true>(p, lo, bad);
    const bool inside = row >= r.row0 && row < r.row0 + r.n;
    const RowParts w = parts_of_row(p, r, inside ? row - r.row0 : 0, item % p.num_heads, TM,
                                    Deal::share_of(sum, longest, p.deal_ctas), before, chains_before);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the attention launch before this one is done
    if (!inside || w.parts == 1) return;
    float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int i = warp; i < w.parts; i += 4) {
        const size_t at = (size_t)min(w.slot + i, p.part_slots - 1) * (PF_NQ * PF_BM) + w.row;
        const float2 ml = p.part_ml[at];
        const float *a = p.part_acc + at * D + lane * E;
        float x[E];
        if constexpr (E == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(a);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2 *>(a);
            x[0] = v.x, x[1] = v.y;
        }
        const float top = fmaxf(m, ml.x), ref = top == -INFINITY ? 0.f : top;
        const float f0 = exp2f(m - ref), f1 = exp2f(ml.x - ref);
        m = top;
        l = l * f0 + ml.y * f1;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * f0 + x[e] * f1;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc_of[warp][lane * E + e] = acc[e];
    if (lane == 0) ml_of[warp] = make_float2(m, l);
    __syncthreads();
    if (warp) return;
    const float top = fmaxf(fmaxf(ml_of[0].x, ml_of[1].x), fmaxf(ml_of[2].x, ml_of[3].x));
    const float ref = top == -INFINITY ? 0.f : top;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float f = exp2f(ml_of[i].x - ref);
        l = fmaf(ml_of[i].y, f, l);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(acc_of[i][lane * E + e], f, acc[e]);
    }
    const bool some = r.keys - r.n + (row - r.row0) + 1 > 0;
    const float inv = some ? 1.f / l : 0.f;
    uint32_t *op = reinterpret_cast<uint32_t *>(static_cast<T *>(p.out) + (size_t)item * D) + lane * (E / 2);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) op[e] = Elem<T>::pack(some ? acc[2 * e] * inv : 0.f, some ? acc[2 * e + 1] * inv : 0.f);
}

}  // namespace pa
