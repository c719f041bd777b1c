// Runs the prompt attention's work plan (csrc/pa_prefill_plan.cuh) on the CPU: a
// warp is 32 fibers that meet at each vote or shuffle. Reads calls from standard
// input and prints the items found. Built by tests/test_prompt_plan.py beside a
// copy of the header; the few device names it uses are defined here.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <ucontext.h>

#include <algorithm>
#include <functional>
#include <vector>

#define __device__
#define __forceinline__ inline
using std::max;
using std::min;
struct int2 {
    int x, y;
};
struct float2 {
    float x, y;
};
static int2 make_int2(int x, int y) { return int2{x, y}; }

namespace emu {

struct Index {
    int x;
};
static ucontext_t scheduler, lanes[32];
static std::vector<char> stacks[32];
static bool done[32];
static unsigned turns[32];
static long long slots[2][32];
static int lane_now;
static std::function<void()> body;

static void entry() {
    body();
    done[lane_now] = true;
    swapcontext(&lanes[lane_now], &scheduler);
}

// Runs f on the 32 lanes of a warp; every lane has to meet the others at each collective.
static void run_warp(const std::function<void()> &f);

static const long long *meet(long long v) {
    const int l = lane_now;
    const int at = turns[l]++ & 1;
    slots[at][l] = v;
    swapcontext(&lanes[l], &scheduler);
    return slots[at];
}

}  // namespace emu

static emu::Index threadIdx, blockIdx;

static void emu::run_warp(const std::function<void()> &f) {
    body = f;
    for (int l = 0; l < 32; ++l) {
        done[l] = false;
        turns[l] = 0;
        stacks[l].resize(1 << 16);
        getcontext(&lanes[l]);
        lanes[l].uc_stack.ss_sp = stacks[l].data();
        lanes[l].uc_stack.ss_size = stacks[l].size();
        lanes[l].uc_link = &scheduler;
        makecontext(&lanes[l], entry, 0);
    }
    for (bool any = true; any;) {
        any = false;
        for (int l = 0; l < 32; ++l) {
            if (done[l]) continue;
            lane_now = threadIdx.x = l;
            swapcontext(&scheduler, &lanes[l]);
            any = any || !done[l];
        }
    }
    for (int l = 1; l < 32; ++l)
        if (turns[l] != turns[0]) {
            fprintf(stderr, "lane %d met %u times, lane 0 %u\n", l, turns[l], turns[0]);
            exit(3);
        }
}

template <typename T>
static T __shfl_sync(unsigned, T v, int src) {
    return (T)emu::meet((long long)v)[src & 31];
}
template <typename T>
static T __shfl_up_sync(unsigned, T v, int by) {
    const int l = threadIdx.x;
    const long long *all = emu::meet((long long)v);
    return (T)(l >= by ? all[l - by] : all[l]);
}
template <typename T>
static T __shfl_xor_sync(unsigned, T v, int with) {
    const int l = threadIdx.x;
    return (T)emu::meet((long long)v)[l ^ with];
}
static unsigned __ballot_sync(unsigned, bool v) {
    const long long *all = emu::meet(v);
    unsigned m = 0;
    for (int l = 0; l < 32; ++l) m |= (unsigned)(all[l] != 0) << l;
    return m;
}
static int __reduce_max_sync(unsigned, int v) {
    const long long *all = emu::meet(v);
    return (int)*std::max_element(all, all + 32);
}
static int __reduce_add_sync(unsigned, int v) {
    const long long *all = emu::meet(v);
    long long s = 0;
    for (int l = 0; l < 32; ++l) s += all[l];
    return (int)s;
}
static int __ffs(unsigned m) { return __builtin_ffs((int)m); }

#include "pa_prefill_plan.cuh"

static std::vector<int> numbers(int n) {
    std::vector<int> x(n);
    for (int &v : x)
        if (scanf("%d", &v) != 1) exit(4);
    return x;
}

static pa::PrefillParams params;
static int TM;

// The items of the indices in `order`, asked of one warp one after the other.
template <bool PAGED>
static void find_items(const std::vector<int> &order) {
    std::vector<pa::Item> items(order.size());
    std::vector<char> found(order.size());
    unsigned bads[32] = {};
    emu::run_warp([&] {
        pa::Finder<PAGED> finder;
        const int lane = threadIdx.x;
        for (size_t i = 0; i < order.size(); ++i) {
            pa::Item it = {};
            const bool ok = finder.find(params, order[i], TM, it, bads[lane]);
            if (lane == 0) items[i] = it, found[i] = ok;
        }
    });
    for (size_t i = 0; i < order.size(); ++i)
        printf("%d %d %d %d %d %d %d %d\n", order[i], (int)found[i], items[i].s, items[i].tok0, items[i].kvh,
               items[i].row0, items[i].n, items[i].keys);
}

// The pieces that each CTA walks where contexts are split, and where the rows' parts lie.
static void deal() {
    for (int cta = 0; cta < params.deal_ctas; ++cta) {
        std::vector<pa::Item> items;
        unsigned bads[32] = {};
        blockIdx.x = cta;
        emu::run_warp([&] {
            pa::Finder<true> finder;
            const int lane = threadIdx.x;
            pa::Item it = {};
            while (finder.next_piece(params, TM, it, bads[lane]))
                if (lane == 0) items.push_back(it);
        });
        for (const pa::Item &it : items)
            printf("1 %d %d %d %d %d %d %d %d\n", cta, it.s, it.tok0, it.kvh, it.j0, it.j1, it.slot, it.parts);
    }
    unsigned bad = 0;
    long long sum = 0, before = 0, chains_before = 0;
    int longest = 1;
    std::vector<pa::SeqRange> rows;
    for (int s = 0; s < params.num_seqs; ++s) {
        rows.push_back(pa::seq_range<true>(params, s, bad));
        const pa::Deal d = pa::Deal::of(rows[s], TM);
        sum += d.all(params);
        if (d.chains > 0) longest = max(longest, d.tiles);
    }
    const long long share = pa::Deal::share_of(sum, longest, params.deal_ctas);
    for (int s = 0; s < params.num_seqs; ++s) {
        for (int i = 0; i < rows[s].n; ++i)
            for (int h = 0; h < params.num_heads; ++h) {
                const pa::RowParts r = pa::parts_of_row(params, rows[s], i, h, TM, share, before, chains_before);
                printf("2 %d %d %d %d %d %d\n", s, i, h, r.slot, r.parts, r.row);
            }
        const pa::Deal d = pa::Deal::of(rows[s], TM);
        before += d.all(params);
        chains_before += (long long)d.chains * params.num_kv_heads;
    }
}

int main() {
    char what[16];
    while (scanf("%15s", what) == 1) {
        // paged, sequences, tokens, heads, KV heads, limit of a context, CTAs and slots of a deal, count of indices
        const std::vector<int> a = numbers(9);
        const std::vector<int> cu = numbers(a[1] + 1), ctx = numbers(a[1]), order = numbers(a[8]);
        params = pa::PrefillParams{};
        params.num_seqs = a[1];
        params.num_tokens = a[2];
        params.num_heads = a[3];
        params.num_kv_heads = a[4];
        params.ctx_limit = a[5];
        params.deal_ctas = a[6];
        params.part_slots = a[7];
        params.cu_seqlens = cu.data();
        params.context_lens = ctx.data();
        TM = pa::PF_NQ * pa::PF_BM / (a[3] / a[4]);
        if (what[0] == 'd')
            deal();
        else
            a[0] ? find_items<true>(order) : find_items<false>(order);
        printf("end\n");
        fflush(stdout);
    }
    return 0;
}
