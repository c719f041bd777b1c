// The prompt attention's work plan (pa_prefill, pa_prefill_paged; include/pa.h):
// parameters, the rows of a sequence, and which work items there are, in which
// order. Integer arithmetic and warp votes only.
#pragma once

#include "pa_common.cuh"

namespace pa {

constexpr int PF_NQ = 2;    // tiles of rows of an item
constexpr int PF_BM = 128;  // rows of a tile
constexpr int PF_BN = 128;  // keys of a tile

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
    bool negate;                                                // the scale is -scale_log2
    bool deal;         // whether contexts are split (paged; struct Deal)
    int deal_ctas;     // CTAs that share the key tiles then
    int part_slots;    // places for parts of a chain
    float *part_acc;   // [slot][row of the chain][head_dim]: weighted values of the parts
    float2 *part_ml;   // [slot][row of the chain]: what they are relative to (log2), sum of the weights
    unsigned long long wait_ns;  // after which a wait gives up
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

struct Item {
    int s, tok0;           // sequence, first token of the tile among its rows
    int row0, n, keys;     // as SeqRange
    int slot, parts, kvh;  // the part's place, how many parts the chain has, KV head
    int j0, j1;            // key tiles of the part, where there are more than one
    int look;              // whether hidden values are looked through
};

// Key tiles an item walks, [j0, j1), and how its two tiles of rows share them:
// each walks all that its rows see. Where the second has no rows (the last rows of
// a prompt, few rows over a long context) both take the first one's rows, one the
// even and one the odd key tiles, and their results are joined at the end: one
// tile of rows alone would wait for its softmax half of the time.
struct Walk {
    int first;           // row i of the sequence sees the keys below first + i + 1
    int j0, j1, kv_end;  // kv_end: the keys that any of the rows sees
    bool halves;
    int count[PF_NQ], end[PF_NQ];  // key tiles of a tile of rows, the keys that any of its rows sees
};

// halves: whether items may be walked in halves (few rows over a paged context).
__device__ __forceinline__ Walk walk_of(const Item &it, int tm, bool halves) {
    Walk w;
    w.first = it.keys - it.n;
    w.kv_end = 0;
    int tiles[PF_NQ];
#pragma unroll
    for (int t = 0; t < PF_NQ; ++t) {
        const int a = it.tok0 + t * tm, b = min(it.n, a + tm);
        w.end[t] = a < b ? max(w.first + b, 0) : 0;
        tiles[t] = (w.end[t] + PF_BN - 1) / PF_BN;
        w.kv_end = max(w.kv_end, w.end[t]);
    }
    const int all = (w.kv_end + PF_BN - 1) / PF_BN;
    w.j0 = it.parts > 1 ? min(it.j0, all) : 0;
    w.j1 = it.parts > 1 ? min(it.j1, all) : all;
#pragma unroll
    for (int t = 0; t < PF_NQ; ++t) w.count[t] = max(min(tiles[t], w.j1) - w.j0, 0);
    w.halves = halves && it.tok0 + tm >= it.n && w.count[0] > 1;
    if (w.halves) {
        w.count[1] = w.count[0] / 2;
        w.count[0] -= w.count[1];
        w.end[1] = w.end[0];
    }
    return w;
}

// Few rows over long contexts: the key tiles of all (sequence, KV head, tile of
// rows), a chain each and the chains one after the other, are dealt to the CTAs
// in equal shares, cut where a share ends. A chain's parts are the shares it
// touches. The part of the chain with index c that CTA b walks has the place c + b:
// of two parts that follow one another the later has the next chain, the next CTA
// or both, so no place is used twice and all lie below chains + CTAs.
struct Deal {
    int chains, tiles;  // of a sequence: chains of a KV head, key tiles of a chain

    __device__ __forceinline__ static Deal of(const SeqRange &r, int TM) {
        return Deal{(r.n + TM - 1) / TM, max((r.keys + PF_BN - 1) / PF_BN, 1)};
    }
    // Key tiles of a sequence's chains.
    __device__ __forceinline__ long long all(const PrefillParams &p) const {
        return (long long)chains * tiles * p.num_kv_heads;
    }
    // An equal share, but no chain in parts of less than 4. sum: all key tiles, longest: of a chain.
    __device__ __forceinline__ static long long share_of(long long sum, int longest, int ctas) {
        return max((sum + ctas - 1) / ctas, (long long)min(longest, 4));
    }
    // Parts of a chain whose first key tile is number `start` of all.
    __device__ __forceinline__ int parts(long long start, long long share) const {
        return (int)((start + tiles - 1) / share - start / share) + 1;
    }
    // Place of a part; boundaries that overlap (flagged) can make more chains than there is room for.
    __device__ __forceinline__ static int slot(const PrefillParams &p, long long chain, long long cta) {
        return (int)min(chain + cta, (long long)p.part_slots - 1);
    }
};

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(FULL_MASK, x, o);
    return x;
}

// Items are handed out from the longest to the shortest, roughly: a tile's
// position in its context counts in units of TM tokens, positions 0 to 7 are
// levels of their own and then 8 of them make one, and the items of a level
// come sequence by sequence and head by head, so that the tiles that walk the
// same keys run at the same time and share them in L2. (Heads first: a piece of
// 512 tokens over 32768 read its keys from memory 3 times.) With C(d) the
// number of tiles of level d or above, item k has the level d with
// C(d + 1) <= k / heads < C(d). One warp. The search starts from the last item's
// level, since the launches that a CTA takes over mostly come with growing k; no
// order of them is promised, so for a smaller k it starts from the highest again.
template <bool PAGED>
struct Finder {
    int level = -1, above = 0, all = 0;  // C(level) = above <= the last k / heads; C(0) = all
    int top = 0;                         // C(top) = 0
    int2 mine;                  // this lane's sequence among the first 32: base, count
    long long share = 0, at = 0, end = 0;  // this CTA's share of a deal

    __device__ __forceinline__ static int start(int d) { return d < 8 ? d : 8 * (d - 7); }
    __device__ __forceinline__ static int level_of(int position) { return position < 8 ? position : 7 + position / 8; }

    __device__ __forceinline__ static void tiles(const PrefillParams &p, int s, int TM, int &base, int &count,
                                                 unsigned &bad) {
        const SeqRange r = seq_range<PAGED>(p, s, bad);
        count = (r.n + TM - 1) / TM;
        base = max(r.keys - r.n, 0) / TM;
    }

    __device__ __forceinline__ static void take(const PrefillParams &p, int s, Item &it, unsigned &bad) {
        const SeqRange r = seq_range<PAGED>(p, s, bad);
        it.s = s;
        it.row0 = r.row0;
        it.n = r.n;
        it.keys = r.keys;
    }

    // The next piece of this CTA's share of a deal.
    __device__ bool next_piece(const PrefillParams &p, int TM, Item &it, unsigned &bad) {
        const int lane = threadIdx.x & 31, B = p.num_seqs;
        if (share == 0) {
            long long sum = 0;
            int longest = 1;
            for (int s = lane; s < B; s += 32) {
                const Deal d = Deal::of(seq_range<PAGED>(p, s, bad), TM);
                sum += d.all(p);
                if (d.chains > 0) longest = max(longest, d.tiles);
            }
            sum = warp_sum(sum);
            share = Deal::share_of(sum, __reduce_max_sync(FULL_MASK, longest), p.deal_ctas);
            at = min(share * blockIdx.x, sum);
            end = min(at + share, sum);
        }
        if (at >= end) return false;
        long long before = 0, chains_before = 0;
        for (int s0 = 0; s0 < B; s0 += 32) {
            Deal d{0, 1};
            if (s0 + lane < B) d = Deal::of(seq_range<PAGED>(p, s0 + lane, bad), TM);
            long long sum = d.all(p), chains_sum = (long long)d.chains * p.num_kv_heads;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(FULL_MASK, sum, o);
                const long long chains_up = __shfl_up_sync(FULL_MASK, chains_sum, o);
                if (lane >= o) {
                    sum += up;
                    chains_sum += chains_up;
                }
            }
            const unsigned m = __ballot_sync(FULL_MASK, before + sum > at);
            if (m) {
                const int src = __ffs(m) - 1;
                d.chains = __shfl_sync(FULL_MASK, d.chains, src);
                d.tiles = __shfl_sync(FULL_MASK, d.tiles, src);
                const long long in = at - before - (__shfl_sync(FULL_MASK, sum, src) - d.all(p));
                const int chain = (int)(in / d.tiles);
                it.j0 = (int)(in % d.tiles);
                const long long first_chain =
                    chains_before + __shfl_sync(FULL_MASK, chains_sum, src) - (long long)d.chains * p.num_kv_heads;
                it.slot = Deal::slot(p, first_chain + chain, blockIdx.x);
                it.parts = d.parts(at - it.j0, share);
                it.j1 = (int)min((long long)d.tiles, it.j0 + (end - at));
                it.kvh = chain / d.chains;
                it.tok0 = chain % d.chains * TM;
                take(p, s0 + src, it, bad);
                at += it.j1 - it.j0;
                return true;
            }
            before += __shfl_sync(FULL_MASK, sum, 31);
            chains_before += __shfl_sync(FULL_MASK, chains_sum, 31);
        }
        return false;
    }

    // The kth item.
    __device__ bool find(const PrefillParams &p, int k, int TM, Item &it, unsigned &bad) {
        const int lane = threadIdx.x & 31, B = p.num_seqs, heads = p.num_kv_heads;
        auto count_above = [&](int d, int *top) {  // C(d), and the highest level + 1
            int c = 0, last = 0;
            const int from = start(d);
            for (int s = lane; s < B; s += 32) {
                int b = mine.x, n = mine.y;
                if (s >= 32) tiles(p, s, TM, b, n, bad);
                c += max(0, min(n, b + n - from));
                if (n > 0) last = max(last, level_of(b + n - 1) + 1);
            }
            if (top) *top = __reduce_max_sync(FULL_MASK, last);
            return (int)__reduce_add_sync(FULL_MASK, c);
        };
        if (level < 0) {
            mine = make_int2(0, 0);
            if (lane < B) tiles(p, lane, TM, mine.x, mine.y, bad);
            all = count_above(0, &top);
            level = top;
        }
        if (k >= all * heads) return false;
        if (k < above * heads) {
            level = top;
            above = 0;
        }
        int lo = 0, hi = level, before = above;  // C(lo) > k / heads >= C(hi) = before
        for (int step = 1; hi - lo > 1;) {
            const int mid = step < 4 ? max(hi - step, 1) : (lo + hi) >> 1;  // most often one of the next levels
            step *= 2;
            const int c = count_above(mid, nullptr);
            if (c * heads > k) {
                lo = mid;
                step = 4;
            } else {
                hi = mid;
                before = c;
            }
        }
        level = hi;
        above = before;
        int rank = k - before * heads;  // within level lo
        const int from = start(lo), to = start(lo + 1);
        for (int s0 = 0; s0 < B; s0 += 32) {
            const int s = s0 + lane;
            int b = 0, n = 0, first = 0, last = 0;  // the sequence's tiles in this level
            if (s < B) {
                b = mine.x, n = mine.y;
                if (s >= 32) tiles(p, s, TM, b, n, bad);
                first = max(from - b, 0);
                last = min(n, to - b);
            }
            const int here = max(last - first, 0) * heads;
            int sum = here;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(FULL_MASK, sum, o);
                if (lane >= o) sum += up;
            }
            const unsigned m = __ballot_sync(FULL_MASK, sum > rank);
            if (m) {
                const int src = __ffs(m) - 1;
                const int in = rank - __shfl_sync(FULL_MASK, sum - here, src);
                first = __shfl_sync(FULL_MASK, first, src);
                last = __shfl_sync(FULL_MASK, last, src);
                it.kvh = in / (last - first);
                it.tok0 = (last - 1 - in % (last - first)) * TM;
                it.slot = it.j0 = it.j1 = 0;
                it.parts = 1;
                take(p, s0 + src, it, bad);
                return true;
            }
            rank -= __shfl_sync(FULL_MASK, sum, 31);
        }
        return false;
    }
};

// Where a row's parts lie: places slot .. slot + parts - 1, the row's number in each.
struct RowParts {
    int slot, parts, row;
};

// Of row `token` (from the sequence's first) of head h in sequence s. before,
// chains_before: key tiles and chains of the sequences before s.
__device__ __forceinline__ RowParts parts_of_row(const PrefillParams &p, const SeqRange &r, int token, int h, int TM,
                                                 long long share, long long before, long long chains_before) {
    const int group = p.num_heads / p.num_kv_heads;
    const Deal d = Deal::of(r, TM);
    const int chain = h / group * d.chains + token / TM;
    const long long start = before + (long long)chain * d.tiles;
    return RowParts{Deal::slot(p, chains_before + chain, start / share), d.parts(start, share),
                    token % TM * group + h % group};
}

}  // namespace pa
