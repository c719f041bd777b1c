// Tensor-core kernel of pa_prefill and pa_prefill_paged (include/pa.h).
//
// A CTA takes NQ tiles of 128 query rows of one (sequence, KV head) and walks
// the keys they see in tiles of 128. The rows are (token, query head) pairs of
// the group, head fastest: all query heads of a KV head share its key and value
// tiles, and a tile spans few tokens, so little of it is masked. For each tile
//   S = Q K^T      tcgen05.mma, both operands in shared memory, S in TMEM
//   P = exp2(S * scale_log2 - m)   a thread for each row, registers; P rounded
//                  to the input type goes back to TMEM over S
//   O += P V       tcgen05.mma, P from TMEM, V from shared memory, O in TMEM
// m is a running maximum of the row and l the running sum, both 32 bits; O and
// l are rescaled only when the maximum has grown by more than 2^8 (P then stays
// below 2^8, far inside fp16's range), which after the first tiles is rare.
//
// Warps: four softmax warps for each tile of rows, one that issues the copies
// (TMA) and one that issues the matrix instructions. While the softmax of one
// tile of rows runs, the other tile's products do. A tile of rows is bound by
// two things at once at head size 128: 128 x 128 exponentials at 16 a clock and
// 4 x 128^3 product operations at 8192 a clock, 1024 clocks either way.
//
// Masked places: S is replaced by -inf there (a selection, so NaN and
// infinities in masked keys do not spread) and P is 0. A NaN or infinity in a
// masked value row would still come through 0 x V: such a row of O is NaN, is
// seen at the end, and is computed again by the row form (attend_row), which
// reads the visible rows only.
#pragma once

#include <cuda.h>

#include "pa_prefill.cuh"

namespace pa {

constexpr int PF_BM = 128;  // rows of a tile
constexpr int PF_BN = 128;  // keys of a tile
constexpr uint64_t PF_WAIT_NS = 1000000000ull;

template <int D, int NQ>
struct PrefillShape {
    static constexpr int HALVES = D / 64;            // 128-byte columns of a row
    static constexpr int TILE = 128 * D * 2;         // bytes of a tile of rows (queries, keys or values)
    static constexpr int THREADS = NQ * 128 + 128;
    // NQ = 2: one CTA an SM; NQ = 1: two.
    static constexpr int STAGES = NQ == 2 ? (D == 128 ? 5 : 8) : (D == 128 ? 2 : 5);
    static constexpr int TMEM_COLS = NQ == 2 ? 512 : 256;
    static constexpr int S_COL = 0, O_COL = NQ * 128;
    static constexpr int OFF_KV = NQ * TILE;
    static constexpr int OFF_BAR = OFF_KV + STAGES * TILE;
    static constexpr int NUM_BARS = 2 * STAGES + 1 + 3 * NQ;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;        // TMEM address, scratch of locate_tile
    static constexpr int BYTES = OFF_MISC + 8 + 2 * 16 * 4 + 8 * 4 + 1024;  // and slack for the 1024-byte alignment
};

// ---- tcgen05 ------------------------------------------------------------------------------------------
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

// A from TMEM.
__device__ __forceinline__ void tc_mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
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

// Waits for the loads issued before and ties their registers to the wait, so
// that nothing that uses them is moved above it.
template <int N>
__device__ __forceinline__ void tc_landed(float (&x)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(x[i]));
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

// Shared-memory matrix descriptor with the 128-byte swizzle: start address,
// leading and stride byte offsets in 16-byte units, version 1 (bit 46).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr >> 4) & 0x3fff) | (uint64_t)((lbo >> 4) & 0x3fff) << 16 |
           (uint64_t)((sbo >> 4) & 0x3fff) << 32 | 1ull << 46 | 2ull << 61;
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

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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

// ---- which tile a CTA takes ---------------------------------------------------------------------------
// Tiles are handed out from the longest to the shortest: a tile's level is its
// position in the context in units of TM tokens, C(d) = number of tiles at
// level d or above, and tile k has the level d with C(d + 1) <= k < C(d). Every
// thread of the CTA takes part.
struct TileAt {
    int s, tok0;  // sequence, first token of the tile among its rows
    SeqRange r;
};

template <bool PAGED, int NT>
__device__ bool locate_tile(const PrefillParams &p, int k, int TM, int *scratch, int *found, TileAt &tile,
                            unsigned &bad) {
    constexpr int NW = NT / 32;
    const int tid = threadIdx.x, warp = tid >> 5, B = p.num_seqs;
    auto level = [&](int s, int &base, int &count) {
        const SeqRange r = seq_range<PAGED>(p, s, bad);
        count = (r.n + TM - 1) / TM;
        base = max(r.keys - r.n, 0) / TM;
    };
    int base0 = 0, count0 = 0;
    if (tid < B) level(tid, base0, count0);
    int turn = 0;
    auto above = [&](int d) {  // C(d)
        int c = max(0, min(count0, base0 + count0 - d));
        for (int s = tid + NT; s < B; s += NT) {
            int b, n;
            level(s, b, n);
            c += max(0, min(n, b + n - d));
        }
        c = __reduce_add_sync(FULL_MASK, c);
        int *w = scratch + (turn++ & 1) * 16;  // two buffers: one barrier a sum
        if ((tid & 31) == 0) w[warp] = c;
        __syncthreads();
        int sum = 0;
#pragma unroll
        for (int i = 0; i < NW; ++i) sum += w[i];
        return sum;
    };
    if (k >= above(0)) return false;
    int top = base0 + count0;
    for (int s = tid + NT; s < B; s += NT) {
        int b, n;
        level(s, b, n);
        top = max(top, b + n);
    }
    top = __reduce_max_sync(FULL_MASK, top);
    {
        int *w = scratch + (turn++ & 1) * 16;
        if ((tid & 31) == 0) w[warp] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NW; ++i) top = max(top, w[i]);
    }
    int lo = 0, hi = top, before = 0;  // C(lo) > k >= C(hi) = before
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        const int c = above(mid);
        if (c > k) {
            lo = mid;
        } else {
            hi = mid;
            before = c;
        }
    }
    int rank = k - before;  // among the sequences with a tile at level lo, in order
    for (int s0 = 0; s0 < B; s0 += NT) {
        const int s = s0 + tid;
        int b = base0, n = count0;
        if (s0 && s < B) level(s, b, n);
        const bool has = s < B && b <= lo && lo < b + n;
        const unsigned m = __ballot_sync(FULL_MASK, has);
        int *w = scratch + (turn++ & 1) * 16;
        if ((tid & 31) == 0) w[warp] = __popc(m);
        __syncthreads();
        int prev = 0, all = 0;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            prev += i < warp ? w[i] : 0;
            all += w[i];
        }
        if (has && prev + __popc(m & ((1u << (tid & 31)) - 1)) == rank) {
            found[0] = s;
            found[1] = (lo - b) * TM;
        }
        if (rank < all) break;
        rank -= all;
    }
    __syncthreads();
    tile.s = found[0];
    tile.tok0 = found[1];
    tile.r = seq_range<PAGED>(p, tile.s, bad);
    return true;
}

struct PrefillMaps {
    CUtensorMap q, k, v;
};

template <int D, typename T, bool PAGED, int NQ>
__global__ void __launch_bounds__(PrefillShape<D, NQ>::THREADS, NQ == 2 ? 1 : 2)
    pa_prefill_mma_kernel(const PrefillParams p, const __grid_constant__ PrefillMaps maps, bool negate) {
    using SH = PrefillShape<D, NQ>;
    constexpr int HALVES = SH::HALVES, NS = SH::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    const uint32_t base = smem_u32(smem);
    const uint32_t bars = base + SH::OFF_BAR;
    auto kv_full = [&](int i) { return bars + 8 * i; };
    auto kv_empty = [&](int i) { return bars + 8 * (NS + i); };
    const uint32_t q_full = bars + 8 * (2 * NS);
    auto s_full = [&](int t) { return bars + 8 * (2 * NS + 1 + t); };
    auto p_full = [&](int t) { return bars + 8 * (2 * NS + 1 + NQ + t); };
    auto o_full = [&](int t) { return bars + 8 * (2 * NS + 1 + 2 * NQ + t); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + SH::OFF_MISC);
    int *scratch = reinterpret_cast<int *>(smem + SH::OFF_MISC + 8);
    int *found = scratch + 32;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = p.num_heads / p.num_kv_heads;
    const int tm = PF_BM / group;  // tokens of a tile of rows
    const int kvh = blockIdx.x % p.num_kv_heads;
    unsigned bad = 0;
    TileAt tile;
    const bool work =
        locate_tile<PAGED, SH::THREADS>(p, blockIdx.x / p.num_kv_heads, NQ * tm, scratch, found, tile, bad);
    if (bad) atomicOr(p.errors, bad);
    bad = 0;
    if (!work) return;

    // Row i of the sequence's n sees the keys below first + i + 1.
    const int first = tile.r.keys - tile.r.n;
    int tiles[NQ], kv_end = 0, num_tiles = 0;
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
        const int a = tile.tok0 + t * tm, b = min(tile.r.n, a + tm);
        const int end = a < b ? max(first + b, 0) : 0;
        tiles[t] = (end + PF_BN - 1) / PF_BN;
        kv_end = max(kv_end, end);
        num_tiles = max(num_tiles, tiles[t]);
    }

    if (warp == NQ * 4) {
        if (lane == 0) {
            for (int i = 0; i < NS; ++i) {
                mbar_init(kv_full(i), 1);
                mbar_init(kv_empty(i), 1);
            }
            mbar_init(q_full, 1);
            for (int t = 0; t < NQ; ++t) {
                mbar_init(s_full(t), 1);
                mbar_init(p_full(t), 4);
                mbar_init(o_full(t), 1);
            }
            fence_barrier_init();
        }
        __syncwarp();
    } else if (warp == NQ * 4 + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "n"(SH::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // A wait that runs out ends this warp's work: the error bit is set, later
    // waits and work are skipped, and the CTA still frees its TMEM.
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (alive && !__all_sync(FULL_MASK, mbar_wait_bounded(bar, parity, PF_WAIT_NS))) {
            alive = false;
            if (lane == 0) atomicOr(p.errors, PA_DEVERR_TIMEOUT);
        }
        return alive;
    };

    if (warp == NQ * 4) {
        // ---- copies ----
        if (num_tiles > 0) {
            if (lane == 0) {
                uint32_t bytes = 0;
                for (int t = 0; t < NQ; ++t) bytes += tiles[t] > 0 ? SH::TILE : 0;
                mbar_arrive_expect_tx(q_full, bytes);
                for (int t = 0; t < NQ; ++t)
                    if (tiles[t] > 0)
                        for (int h = 0; h < HALVES; ++h)
                            tma_load_3d(base + t * SH::TILE + h * 16384, &maps.q, h * 64, kvh * group,
                                        tile.r.row0 + tile.tok0 + t * tm, q_full);
            }
            __syncwarp();
            int issued = 0;
            const int per_tile = PAGED ? PF_BN / p.block_size : 0;
            auto block_of = [&](int j) {  // this lane's block of key tile j
                const int b = j * per_tile + lane;
                int id = 0;
                if (lane < per_tile && b * p.block_size < kv_end) {
                    id = p.block_tables[(size_t)tile.s * p.max_blocks_per_seq + b];
                    if ((unsigned)id >= (unsigned)p.num_blocks) {
                        atomicOr(p.errors, PA_DEVERR_BLOCK_ID);
                        id = 0;
                    }
                }
                return id;
            };
            int id = 0, id_next = 0;
            if constexpr (PAGED) id_next = block_of(0);
            for (int c = 0; c < 2 * num_tiles; ++c) {
                const int j = c >> 1, stage = c % NS;
                if constexpr (PAGED) {
                    if (!(c & 1)) {
                        id = id_next;
                        if (j + 1 < num_tiles) id_next = block_of(j + 1);
                    }
                }
                if (c >= NS && !wait(kv_empty(stage), (c / NS - 1) & 1)) break;
                const CUtensorMap *map = c & 1 ? &maps.v : &maps.k;
                const uint32_t dst = base + SH::OFF_KV + stage * SH::TILE;
                if constexpr (PAGED) {
                    const int chunk = p.block_size * D * 2;
                    const int blocks = min(per_tile, (kv_end - j * PF_BN + p.block_size - 1) / p.block_size);
                    if (lane == 0) mbar_arrive_expect_tx(kv_full(stage), blocks * chunk);
                    __syncwarp();
                    if (lane < blocks)
                        tma_load_chunk(dst + lane * chunk, map, id * p.num_kv_heads + kvh, kv_full(stage));
                } else if (lane == 0) {
                    mbar_arrive_expect_tx(kv_full(stage), SH::TILE);
                    for (int h = 0; h < HALVES; ++h)
                        tma_load_3d(dst + h * 16384, map, h * 64, kvh, tile.r.row0 + j * PF_BN, kv_full(stage));
                }
                __syncwarp();
                ++issued;
            }
            if (!alive)  // copies in flight land before the CTA leaves
                for (int c = max(0, issued - NS); c < issued; ++c)
                    mbar_wait_bounded(kv_full(c % NS), (c / NS) & 1, PF_WAIT_NS);
        }
    } else if (warp == NQ * 4 + 1) {
        // ---- matrix instructions ----
        // Instruction descriptor: 32-bit accumulator, both operands of the input
        // type (0 fp16, 1 bf16), N / 8 at bit 17, M / 16 at bit 24; bit 13 negates
        // A, bit 16 takes B with its columns contiguous.
        constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
        constexpr uint32_t common = 1u << 4 | type << 7 | type << 10 | (uint32_t)(PF_BM >> 4) << 24;
        const uint32_t idesc_qk = common | (uint32_t)(PF_BN >> 3) << 17 | (negate ? 1u << 13 : 0u);
        constexpr uint32_t idesc_pv = common | (uint32_t)(D >> 3) << 17 | 1u << 16;
        // Keys and values: rows of 128 bytes in groups of 8 (1024 bytes), for the
        // packed form column after column, for the pools' chunks row group after row group.
        constexpr uint32_t KV_GROUP = PAGED ? HALVES * 1024 : 1024, KV_HALF = PAGED ? 1024 : 16384;
        auto qk = [&](int t, int stage) {
            if (lane == 0) {
                const uint32_t q = base + t * SH::TILE, k = base + SH::OFF_KV + stage * SH::TILE;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    tc_mma(tmem + SH::S_COL + t * 128, smem_desc(q + (i >> 2) * 16384 + (i & 3) * 32, 16, 1024),
                           smem_desc(k + (i >> 2) * KV_HALF + (i & 3) * 32, 16, KV_GROUP), idesc_qk, i > 0);
                tc_commit(s_full(t));
            }
            __syncwarp();
        };
        if (num_tiles > 0 && wait(q_full, 0) && wait(kv_full(0), 0)) {
            tc_fence_after();
            for (int t = 0; t < NQ; ++t)
                if (tiles[t] > 0) qk(t, 0);
            if (lane == 0) tc_commit(kv_empty(0));
            for (int j = 0; j < num_tiles && alive; ++j) {
                const int cv = 2 * j + 1, sv = cv % NS, ck = cv + 1, sk = ck % NS;
                if (!wait(kv_full(sv), (cv / NS) & 1)) break;
                const uint32_t v = base + SH::OFF_KV + sv * SH::TILE;
                if (PAGED && kv_end < (j + 1) * PF_BN) {
                    // Slots behind the context hold anything: their weights are 0, their values made 0.
                    for (int i = (kv_end - j * PF_BN) * HALVES * 8 + lane; i < PF_BN * HALVES * 8; i += 32) {
                        const int row = i / (HALVES * 8), c = i % (HALVES * 8);
                        const uint32_t at = v + (row >> 3) * KV_GROUP + (c >> 3) * KV_HALF + (row & 7) * 128 + (c & 7) * 16;
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                const bool more = j + 1 < num_tiles;
                if (more && !wait(kv_full(sk), (ck / NS) & 1)) break;
                for (int t = 0; t < NQ; ++t) {
                    if (j >= tiles[t]) continue;
                    if (!wait(p_full(t), j & 1)) break;
                    tc_fence_after();
                    if (lane == 0) {
#pragma unroll
                        for (int i = 0; i < PF_BN / 16; ++i)
                            tc_mma_ta(tmem + SH::O_COL + t * D, tmem + SH::S_COL + t * 128 + i * 8,
                                      smem_desc(v + i * 2 * KV_GROUP, KV_HALF, KV_GROUP), idesc_pv, j > 0 || i > 0);
                        if (j + 1 == tiles[t]) tc_commit(o_full(t));
                    }
                    __syncwarp();
                    if (j + 1 < tiles[t]) qk(t, sk);
                }
                if (lane == 0 && alive) {
                    tc_commit(kv_empty(sv));
                    if (more) tc_commit(kv_empty(sk));
                }
                __syncwarp();
            }
        }
    } else if (warp < NQ * 4) {
        // ---- softmax: a thread for each row ----
        const int t = warp >> 2, quarter = warp & 3;
        const int r = t * PF_BM + quarter * 32 + lane;  // row of the CTA
        const int tok = tile.tok0 + r / group, head = kvh * group + r % group;
        const bool valid = tok < tile.r.n;
        const int visible = valid ? max(first + tok + 1, 0) : 0;
        const int clear = max(first + tile.tok0 + (t * PF_BM + quarter * 32) / group + 1, 0);  // seen by all the warp's rows
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_addr = lanes + SH::S_COL + t * 128, o_addr = lanes + SH::O_COL + t * D;
        const int n_tiles = t == 0 ? tiles[0] : tiles[NQ - 1];
        const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
        float m = -INFINITY, l = 0.f;  // m: what the weights are relative to, unscaled
        for (int j = 0; j < n_tiles; ++j) {
            if (!wait(s_full(t), j & 1)) break;
            tc_fence_after();
            float x[PF_BN];
#pragma unroll
            for (int c = 0; c < PF_BN; c += 32) tc_ld32(s_addr + c, x + c);
            tc_landed(x);
            if ((j + 1) * PF_BN > clear) {
                const int left = visible - j * PF_BN;
#pragma unroll
                for (int c = 0; c < PF_BN; ++c) x[c] = c < left ? x[c] : -INFINITY;
            }
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int c = 4; c < PF_BN; c += 4)
#pragma unroll
                for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], x[c + i]);
            const float top = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
            const bool grow = (top - m) * p.scale_log2 > 8.f;
            if (__any_sync(FULL_MASK, grow)) {
                const float f = grow ? ex2((m - top) * p.scale_log2) : 1.f;
                m = grow ? top : m;
                l *= f;
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
            const float ref = m == -INFINITY ? 0.f : -m * p.scale_log2;  // nothing above -inf yet: weights 0
            const float2 ref2 = make_float2(ref, ref);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < PF_BN; c += 64) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float2 y = fma2(make_float2(x[c + 2 * i], x[c + 2 * i + 1]), scale2, ref2);
                    y.x = ex2(y.x);
                    y.y = ex2(y.y);
                    sum[i & 1] = add2(sum[i & 1], y);
                    w[i] = Elem<T>::pack(y.x, y.y);
                }
                tc_st32(s_addr + c / 2, w);
            }
            const float2 both = add2(sum[0], sum[1]);
            l += both.x + both.y;
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(t));
        }
        // ---- epilogue ----
        const float inv = 1.f / l;
        bool again = visible > 0 && !(l > 0.f && l < INFINITY);
        if (n_tiles > 0) wait(o_full(t), 0);
        tc_fence_after();
        T *out = static_cast<T *>(p.out) + ((size_t)(tile.r.row0 + tok) * p.num_heads + head) * D;
        if (alive) {
            float nan = 0.f;
            uint32_t w[D / 2];
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                float o[32];
                if (n_tiles > 0) {
                    tc_ld32(o_addr + c, o);
                    tc_landed(o);
                }
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float a = visible > 0 ? o[i] * inv : 0.f, b = visible > 0 ? o[i + 1] * inv : 0.f;
                    nan = fmaf(a, 0.f, fmaf(b, 0.f, nan));
                    w[(c + i) / 2] = Elem<T>::pack(a, b);
                }
            }
            again = again || (visible > 0 && !(nan == 0.f));
            if (valid && !again) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    reinterpret_cast<uint4 *>(out)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            }
            // A row of floats for each warp, in the tile of queries: its products are done.
            float *q_row = reinterpret_cast<float *>(smem + t * SH::TILE) + quarter * D;
            for (unsigned m_again = __ballot_sync(FULL_MASK, again); m_again; m_again &= m_again - 1) {
                const int from = __ffs(m_again) - 1;
                attend_row<D, T, PAGED>(p, tile.s, tile.r.row0 + __shfl_sync(FULL_MASK, tok, from),
                                        __shfl_sync(FULL_MASK, head, from), __shfl_sync(FULL_MASK, visible, from), q_row,
                                        negate, bad);
            }
            if (bad) atomicOr(p.errors, bad);
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == NQ * 4 + 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(SH::TMEM_COLS));
    }
}

}  // namespace pa
