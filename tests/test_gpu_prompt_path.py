"""The prompt's way into the cache on the GPU: pa_assign_slots against the host
block manager, pa_rope_and_cache, pa_prefill and pa_prefill_paged against their
64-bit forms, and a run of them together with pa_decode."""
import math

import pytest
import torch

import paged_kv_cache_372_b200 as pa
from paged_kv_cache_372_b200.block_manager import BlockManager
from tests import prompt_reference as ref

pytestmark = pytest.mark.gpu

I32, I64 = torch.int32, torch.int64


def ints(x, dtype=I32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def bits(t):
    return t.contiguous().view(torch.int16)


def check(out, want, bound):
    err = (out.double() - want).abs()
    worst = (err - bound).nan_to_num(nan=1e9).max().item() if err.numel() else 0.0
    assert worst <= 0, f"error exceeds its bound by {worst:.3e} (largest error {err.max().item():.3e})"


# ---- pa_assign_slots ----------------------------------------------------------------------------------

class Slots:
    """A batch on the device beside a host block manager that holds the same requests."""

    def __init__(self, B, W, NB, bs, seed):
        order = torch.randperm(NB, generator=torch.Generator().manual_seed(seed)).tolist()
        self.B, self.W, self.NB, self.bs = B, W, NB, bs
        self.bm = BlockManager(NB, bs, order)
        self.table = torch.full((B, W), -1, dtype=I32, device="cuda")
        self.free, self.ctx, self.nf = ints(order), ints([0] * B), ints([NB])
        self.live = {}
        self.next = 0

    def step(self, new, rows, in_place=True):
        # Host: ended requests first, then tokens one by one in request order.
        for s, n in enumerate(new):
            if n < 0 and s in self.live:
                self.bm.free_seq(self.live.pop(s))
        slots, positions, cu = [], [], [0]
        for s, n in enumerate(new):
            if n > 0 and s not in self.live:
                self.live[s] = self.next
                self.next += 1
                self.bm.allocate(self.live[s], 0)
            for _ in range(max(n, 0)):
                positions.append(self.bm.lens[self.live[s]])
                slots.append(self.bm.append_slot(self.live[s]).slot)
            cu.append(len(slots))
        got_slots = torch.full((rows,), 77, dtype=I64, device="cuda")
        got_pos = torch.full((rows,), 77, dtype=I32, device="cuda")
        got_cu = torch.full((self.B + 1,), 77, dtype=I32, device="cuda")
        if in_place:
            pa.pa_assign_slots(self.table, self.free, self.ctx, self.nf, ints(new), self.bs, got_slots, got_pos, got_cu)
        else:
            ctx, nf = torch.full_like(self.ctx, 5), torch.full_like(self.nf, 5)
            for _ in range(2):  # a repeated call on the same inputs gives the same result
                pa.pa_assign_slots(self.table, self.free, self.ctx, self.nf, ints(new), self.bs, got_slots, got_pos,
                                   got_cu, ctx, nf)
            self.ctx, self.nf = ctx, nf
        assert pa.pa_device_errors() == 0
        pad = rows - len(slots)
        assert got_slots.tolist() == slots + [-1] * pad
        assert got_pos.tolist() == positions + [-1] * pad
        assert got_cu.tolist() == cu
        lens = [self.bm.lens[self.live[s]] if s in self.live else 0 for s in range(self.B)]
        assert self.ctx.tolist() == lens
        assert self.nf.item() == len(self.bm.free)
        assert self.free[:self.nf.item()].tolist() == self.bm.free
        for s, n in enumerate(lens):
            w = -(-n // self.bs)
            assert self.table[s, :w].tolist() == (self.bm.tables[self.live[s]][:w] if s in self.live else [])


@pytest.mark.parametrize("B,bs", [(1, 16), (3, 32), (37, 16), (300, 64), (1500, 16)])
@pytest.mark.parametrize("in_place", [True, False])
def test_assign_follows_the_block_manager(B, bs, in_place):
    g = torch.Generator().manual_seed(B + bs)
    top = 40 if B > 100 else 300
    st = Slots(B, 64, B * 20 + 8, bs, B)
    for step in range(8):
        r = torch.randint(0, 10, (B,), generator=g).tolist()
        n = torch.randint(1, top, (B,), generator=g).tolist()
        held = st.ctx.tolist()
        new = [-1 if x == 0 else 0 if x == 1 else 1 if x < 6 else n[s] for s, x in enumerate(r)]
        # keep within the table row and the pool: at most 20 blocks a request
        new = [0 if x > 0 and held[s] + x > 20 * bs else x for s, x in enumerate(new)]
        T = sum(max(x, 0) for x in new)
        st.step(new, T + (0, 1, 63)[step % 3], in_place)


def test_assign_of_no_requests_and_no_tokens():
    st = Slots(4, 4, 8, 16, 0)
    st.step([0, 0, 0, 0], 3)
    st.step([0, -1, 0, 0], 0)
    nf, cu = ints([8]), ints([9])
    empty = torch.empty((0,), dtype=I32, device="cuda")
    slots, pos = torch.full((2,), 9, dtype=I64, device="cuda"), ints([9, 9])
    pa.pa_assign_slots(torch.empty((0, 4), dtype=I32, device="cuda"), ints(range(8)), empty, nf, empty, 16, slots, pos, cu)
    assert pa.pa_device_errors() == 0
    assert (cu.tolist(), nf.tolist(), slots.tolist(), pos.tolist()) == ([0], [8], [-1, -1], [-1, -1])


@pytest.mark.parametrize("what,flag", [("blocks", pa.DEVERR_BLOCKS), ("tokens", pa.DEVERR_TOKENS),
                                       ("width", pa.DEVERR_CONTEXT), ("negative", pa.DEVERR_CONTEXT),
                                       ("huge", pa.DEVERR_CONTEXT), ("free", pa.DEVERR_BLOCKS)])
def test_assign_refuses_a_batch_whole(what, flag):
    ctx, new, nf, rows = [17, 5, 0], [3, -1, 20], 4, 64
    if what == "blocks":
        nf = 1
        new[1] = 0
    elif what == "tokens":
        rows = 22
    elif what == "width":
        new[2] = 65
    elif what == "negative":
        ctx[0] = -3
    elif what == "huge":
        new[2] = 2 ** 31 - 1
    else:
        nf = 9
    table = ints([[3, 4, -1, -1], [5, -1, -1, -1], [-1] * 4])
    free, dctx, dnf = ints([0, 1, 2, 6, 7, 7, 7, 7]), ints(ctx), ints([nf])
    before = [table.clone(), free.clone(), dctx.clone(), dnf.clone()]
    slots, pos = torch.full((rows,), 9, dtype=I64, device="cuda"), torch.full((rows,), 9, dtype=I32, device="cuda")
    cu = ints([9] * 4)
    pa.pa_assign_slots(table, free, dctx, dnf, ints(new), 16, slots, pos, cu)
    assert pa.pa_device_errors() == flag
    for a, b in zip(before, [table, free, dctx, dnf]):
        assert torch.equal(a, b)
    assert (slots == -1).all() and (pos == -1).all() and (cu == 0).all()


def test_assign_flags_a_block_id_out_of_range():
    table = ints([[99, -1]])
    slots, pos, cu = torch.empty((1,), dtype=I64, device="cuda"), ints([0]), ints([0, 0])
    pa.pa_assign_slots(table, ints([0, 1, 2, 3]), ints([5]), ints([4]), ints([1]), 16, slots, pos, cu)
    assert pa.pa_device_errors() == pa.DEVERR_BLOCK_ID


# ---- pa_rope_and_cache --------------------------------------------------------------------------------

def rope_case(T, H, Hkv, D, rot, interleaved, dtype, bs, max_pos, mscale, fused, k_out, seed=0):
    g = gen(seed)
    if fused:
        x = normal((T, H + 2 * Hkv, D), dtype, g)
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    else:
        q, k, v = (normal((T, h, D), dtype, g) for h in (H, Hkv, Hkv))
    nb = -(-T // bs) + 3
    kp, vp = normal((nb, Hkv, bs, D), dtype, g), normal((nb, Hkv, bs, D), dtype, g)
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:T].contiguous()
    pos = torch.randint(0, max_pos, (T,), generator=g, device="cuda", dtype=I32)
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / (rot // 2))
    return q, k, v, kp, vp, slots, pos, inv


def rope_bound(x, want, inv, mscale, dtype):
    # one rounding to the type; two 32-bit products and their sum of 32-bit cosines and sines (4 roundings,
    # and 2^-22 for the angle and the function) over the two elements, |x| + |y| <= 2 max
    u = ref.U[dtype]
    return u * want.abs() + 2.0 ** -21 * mscale * 2 * x.double().abs().amax(-1, keepdim=True) + 2.0 ** -25


@pytest.mark.parametrize("T,H,Hkv,D,rot,bs", [(1, 1, 1, 64, 16, 16), (5, 2, 2, 64, 64, 16), (33, 8, 1, 128, 48, 32),
                                              (257, 32, 8, 128, 128, 16), (640, 3, 5, 128, 64, 64),
                                              (2501, 16, 4, 64, 32, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fused,k_out", [(True, False), (False, True)])
def test_rope_and_cache(T, H, Hkv, D, rot, bs, interleaved, dtype, fused, k_out):
    mscale = 1.125 if k_out else 1.0
    q, k, v, kp, vp, slots, pos, inv = rope_case(T, H, Hkv, D, rot, interleaved, dtype, bs, 1 << 20, mscale, fused, k_out)
    if T > 4:
        slots[1] = -1         # no cache write
        pos[3] = -1           # skipped altogether
    kp0, vp0 = kp.clone(), vp.clone()
    qo = torch.full((T, H, D), float("nan"), dtype=dtype, device="cuda")
    ko = torch.full((T, Hkv, D), float("nan"), dtype=dtype, device="cuda") if k_out else None
    pa.pa_rope_and_cache(qo, q, k, v, kp, vp, pos, slots, inv, mscale=mscale, interleaved=interleaved, k_out=ko)
    assert pa.pa_device_errors() == 0
    live = pos >= 0
    assert torch.isnan(qo[~live]).all()
    wq, wk = ref.rope(q, pos, inv, mscale, interleaved), ref.rope(k, pos, inv, mscale, interleaved)
    check(qo[live], wq[live], rope_bound(q, wq, inv, mscale, dtype)[live])
    assert torch.equal(bits(qo[live][..., rot:]), bits(q[live][..., rot:]))
    if k_out:
        check(ko[live], wk[live], rope_bound(k, wk, inv, mscale, dtype)[live])
        assert torch.isnan(ko[~live]).all()
    w = live & (slots >= 0)
    blk, off = slots[w] // bs, slots[w] % bs
    assert torch.equal(bits(vp[blk, :, off]), bits(v[w]))
    check(kp[blk, :, off], wk[w], rope_bound(k, wk, inv, mscale, dtype)[w])
    kp[blk, :, off] = kp0[blk, :, off]
    vp[blk, :, off] = vp0[blk, :, off]
    assert torch.equal(bits(kp), bits(kp0)) and torch.equal(bits(vp), bits(vp0))


def test_rope_in_place_and_without_a_cache():
    q, k, v, kp, vp, slots, pos, inv = rope_case(70, 8, 2, 128, 64, False, torch.bfloat16, 16, 4096, 1.0, False, True)
    want = torch.empty_like(q), torch.empty_like(k)
    pa.pa_rope_and_cache(want[0], q, k, v, kp, vp, pos, slots, inv, k_out=want[1])
    q2, k2 = q.clone(), k.clone()
    pa.pa_rope_and_cache(q2, q2, k2, None, None, None, pos, None, inv, k_out=k2)
    assert torch.equal(bits(q2), bits(want[0])) and torch.equal(bits(k2), bits(want[1]))
    # the slots of the write are pa_reshape_and_cache's
    kp2, vp2 = torch.zeros_like(kp), torch.zeros_like(vp)
    pa.pa_reshape_and_cache(want[1], v, kp2, vp2, slots)
    blk, off = slots // 16, slots % 16
    assert torch.equal(bits(kp[blk, :, off]), bits(kp2[blk, :, off]))


def test_rope_far_positions_and_slot_past_the_pool():
    T = 40
    q, k, v, kp, vp, slots, pos, inv = rope_case(T, 4, 4, 64, 64, True, torch.float16, 16, 64, 1.0, False, False)
    pos[:] = 2 ** 31 - 1 - torch.arange(T, device="cuda", dtype=I32)
    slots[7] = kp.shape[0] * 16
    vp0 = vp.clone()
    qo = torch.empty_like(q)
    pa.pa_rope_and_cache(qo, q, k, v, kp, vp, pos, slots, inv, interleaved=True)
    assert pa.pa_device_errors() == pa.DEVERR_SLOT
    want = ref.rope(q, pos, inv, 1.0, True)
    check(qo, want, rope_bound(q, want, inv, 1.0, torch.float16))
    ok = torch.arange(T, device="cuda") != 7
    blk, off = slots[ok] // 16, slots[ok] % 16
    vp0[blk, :, off] = v[ok]
    assert torch.equal(bits(vp), bits(vp0))


# ---- pa_prefill ---------------------------------------------------------------------------------------

def packed(lens, H, Hkv, D, dtype, fused, seed, tail=3, head=0):
    g = gen(seed)
    T = head + sum(lens) + tail
    if fused:
        x = normal((T, H + 2 * Hkv, D), dtype, g)
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    else:
        q, k, v = (normal((T, h, D), dtype, g) for h in (H, Hkv, Hkv))
    cu = [head]
    for n in lens:
        cu.append(cu[-1] + n)
    return q, k, v, cu


def run_packed(q, k, v, cu, scale, compare=True):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    assert pa.pa_prefill(out, q, k, v, ints(cu), scale) is out
    assert pa.pa_device_errors() == 0
    assert (out[:cu[0]] == 7.0).all() and (out[cu[-1]:] == 7.0).all()
    if compare:
        for a, b in zip(cu, cu[1:]):
            if b > a:
                check(out[a:b], *ref.attention(q[a:b], k[a:b], v[a:b], scale, 0))
    return out


LENS = [[1], [1, 7, 16, 33], [0, 31, 0, 0, 32, 65, 0], [127, 128, 129], [300, 5, 511], [1025]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("H,Hkv,D", [(2, 2, 64), (4, 4, 128), (4, 2, 64), (4, 1, 128), (16, 2, 128), (8, 1, 64)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_prefill(lens, H, Hkv, D, dtype):
    q, k, v, cu = packed(lens, H, Hkv, D, dtype, H != Hkv, sum(lens) + H + D, head=2 * (len(lens) % 2))
    run_packed(q, k, v, cu, 1 / math.sqrt(D))


@pytest.mark.parametrize("H,Hkv", [(8, 8), (8, 2), (8, 1)])
def test_prefill_many_ragged(H, Hkv):
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 200, (90,), generator=g).tolist() + [700, 1, 0]
    q, k, v, cu = packed(lens, H, Hkv, 128, torch.bfloat16, True, 9)
    run_packed(q, k, v, cu, 1 / math.sqrt(128))


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0])
def test_prefill_scales(scale):
    # scores of up to about 60 at scale 1: one key takes nearly all the weight, the sums' error grows with them
    q, k, v, cu = packed([200, 77], 4, 2, 64, torch.float16, False, 3)
    q = q * 0.5
    run_packed(q, k, v, cu, scale)


def test_prefill_rising_scores():
    # each key's score above the last one's by more than the running maximum may lag
    n, D = 700, 128
    q = torch.zeros((n, 2, D), dtype=torch.float16, device="cuda")
    k = torch.zeros((n, 1, D), dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    k[:, 0, 0] = torch.arange(n, device="cuda") * 3.0
    v = normal((n, 1, D), torch.float16, gen(4))
    run_packed(q, k, v, [0, n], 1.0)
    run_packed(q, k, v, [0, n], -1.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), "lowest"])
@pytest.mark.parametrize("Hkv", [1, 4])
def test_prefill_bad_values_reach_only_rows_that_see_them(bad, Hkv):
    dtype = torch.bfloat16
    bad = torch.finfo(dtype).min if bad == "lowest" else bad
    lens, at = [150, 260, 40], 150 + 201
    q, k, v, cu = packed(lens, 4, Hkv, 128, dtype, False, 12, tail=30)
    clean = run_packed(q, k, v, cu, 0.088)
    for what in ("k", "v", "both"):
        k2, v2 = k.clone(), v.clone()
        if what != "v":
            k2[at, :, 5] = bad
        if what != "k":
            v2[at, :, 9] = bad
        v2[cu[-1]:] = bad
        k2[cu[-1]:] = bad
        out = run_packed(q, k2, v2, cu, 0.088, compare=False)
        same = torch.ones(q.shape[0], dtype=torch.bool)
        same[at:cu[2]] = False
        assert torch.isfinite(out[same.cuda()].float()).all()
        err = (out[same.cuda()].float() - clean[same.cuda()].float()).abs().max().item()
        assert err <= 2 * 2.0 ** -8 * v.abs().max().item()
        # the rows from `at` on all see it: what the formula gives there
        a, b = cu[1], cu[2]
        want, bound = ref.attention(q[at:b], k2[a:b], v2[a:b], 0.088, at - a)
        got = out[at:b].double()
        fin = torch.isfinite(want)
        if bad != bad or abs(bad) == float("inf"):
            assert torch.equal(torch.isfinite(got), fin)
            assert ((got - want).abs() <= bound)[fin].all()


def test_prefill_masked_scores_of_minus_infinity():
    # every score of the first rows is -inf: 0 / 0, and later keys of finite score are found all the same
    n, D = 140, 64
    q = torch.ones((n, 1, D), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    k[:70] = -float("inf")
    v = normal((n, 1, D), torch.bfloat16, gen(1))
    out = run_packed(q, k, v, [0, n], 0.1, compare=False)
    assert torch.isnan(out[:70]).all()
    want, bound = ref.attention(q[70:], k[70:], v[70:], 0.1, 0)
    check(out[70:], want, bound)


@pytest.mark.parametrize("cu", [[0, 50, 40, 64], [-3, 20, 64], [0, 30, 65], [70, 80]])
def test_prefill_flags_bad_boundaries(cu):
    q, k, v, _ = packed([61], 2, 1, 64, torch.float16, False, 2)
    out = torch.zeros_like(q)
    pa.pa_prefill(out, q, k, v, ints(cu), 0.1)
    assert pa.pa_device_errors() == pa.DEVERR_TOKENS


def test_prefill_same_bits_each_time_and_on_another_stream():
    q, k, v, cu = packed([513, 70, 129], 8, 2, 128, torch.bfloat16, True, 6)
    first = run_packed(q, k, v, cu, 0.09)
    side = torch.cuda.Stream()
    outs = [torch.full_like(first, 7.0) for _ in range(3)]
    cu_d = ints(cu)
    torch.cuda.synchronize()
    for o in outs[:2]:
        pa.pa_prefill(o, q, k, v, cu_d, 0.09, stream=side)
    pa.pa_prefill(outs[2], q, k, v, cu_d, 0.09)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(bits(o), bits(first))


# ---- pa_prefill_paged ---------------------------------------------------------------------------------

def pooled(ctx, new, H, Hkv, D, bs, dtype, seed, extra=5, stale=None, shared=0):
    g = gen(seed)
    width = max(-(-c // bs) for c in ctx) + 2
    nb = sum(-(-c // bs) for c in ctx) + extra
    kp, vp = normal((nb, Hkv, bs, D), dtype, g), normal((nb, Hkv, bs, D), dtype, g)
    ids = torch.randperm(nb, generator=g, device="cuda").tolist()
    rows, at = [], 0
    for s, c in enumerate(ctx):
        w = -(-c // bs)
        row = ids[at:at + w]
        if s and shared:
            row[:min(w, shared)] = rows[0][:min(w, shared)]
        at += w
        rows.append(row + [-7] * (width - w))
        if stale is not None and c % bs:
            kp[row[-1], :, c % bs:] = stale
            vp[row[-1], :, c % bs:] = stale
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = normal((cu[-1] + 2, H, D), dtype, g)
    return q, kp, vp, ints(rows), cu


def run_paged(q, kp, vp, table, ctx, cu, scale, max_ctx=None, workspace=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    pa.pa_prefill_paged(out, q, kp, vp, table, ints(ctx), ints(cu), scale, max_ctx or max(ctx), workspace)
    assert pa.pa_device_errors() == 0
    assert (out[cu[-1]:] == 7.0).all()
    for s, c in enumerate(ctx):
        a, b = cu[s], cu[s + 1]
        if b > a:
            k, v = ref.gather(kp, table[s], c), ref.gather(vp, table[s], c)
            check(out[a:b], *ref.attention(q[a:b], k, v, scale, c - (b - a)))
    return out


PAGED = [([5], [5]), ([1, 7, 16, 33], [1, 7, 16, 33]), ([40, 64, 65, 300], [1, 1, 5, 8]),
         ([700, 129, 128, 0, 50], [300, 128, 1, 0, 0]), ([1500, 20], [3, 7]), ([3000], [130])]


@pytest.mark.parametrize("ctx,new", PAGED, ids=str)
@pytest.mark.parametrize("H,Hkv,D,bs", [(2, 2, 64, 16), (4, 4, 128, 32), (8, 2, 128, 16), (4, 2, 64, 64), (8, 1, 128, 64)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_prefill_paged(ctx, new, H, Hkv, D, bs, dtype):
    q, kp, vp, table, cu = pooled(ctx, new, H, Hkv, D, bs, dtype, sum(ctx) + D + bs)
    run_paged(q, kp, vp, table, ctx, cu, 1 / math.sqrt(D))


@pytest.mark.parametrize("stale", [float("nan"), float("inf")])
def test_prefill_paged_stale_slots(stale):
    ctx, new = [33, 130, 260, 17, 1000], [33, 9, 200, 1, 4]
    q, kp, vp, table, cu = pooled(ctx, new, 8, 2, 128, 16, torch.float16, 8, stale=stale)
    run_paged(q, kp, vp, table, ctx, cu, 0.1)


def test_prefill_paged_rows_that_see_nothing_and_limits():
    # more new tokens than context: the first rows see nothing and are zero
    ctx, new = [3, 0, 20], [9, 4, 20]
    q, kp, vp, table, cu = pooled(ctx, new, 4, 1, 64, 16, torch.bfloat16, 3)
    out = run_paged(q, kp, vp, table, ctx, cu, 0.1)
    assert (out[:6] == 0).all() and (out[9:13] == 0).all()
    # a context above the limit is clamped and flagged
    pa.pa_prefill_paged(out, q, kp, vp, table, ints(ctx), ints(cu), 0.1, 16)
    assert pa.pa_device_errors() == pa.DEVERR_CONTEXT
    # a block id out of range is flagged
    table[2, 0] = kp.shape[0]
    pa.pa_prefill_paged(out, q, kp, vp, table, ints(ctx), ints(cu), 0.1, 32)
    assert pa.pa_device_errors() == pa.DEVERR_BLOCK_ID


def test_prefill_paged_many_sequences_shared_prefix():
    g = torch.Generator().manual_seed(2)
    new = torch.randint(1, 40, (70,), generator=g).tolist()
    ctx = [512 + n for n in new]
    q, kp, vp, table, cu = pooled(ctx, new, 8, 2, 128, 16, torch.bfloat16, 4, shared=32)
    run_paged(q, kp, vp, table, ctx, cu, 0.09)


def test_prefill_paged_long_context_few_rows():
    ctx, new = [20000, 777, 9001], [5, 2, 17]
    q, kp, vp, table, cu = pooled(ctx, new, 8, 2, 128, 64, torch.bfloat16, 14)
    first = run_paged(q, kp, vp, table, ctx, cu, 0.09)
    ws = pa.alloc_prefill_workspace(3, q.shape[0], 8, 2, 128, 64, 32768)
    ws.fill_(255)
    again = run_paged(q, kp, vp, table, ctx, cu, 0.09, 32768, ws)
    err = (first.double() - again.double()).abs().max().item()
    assert err <= 2.0 ** -8 * 2


def test_prefill_paged_captured_and_replayed():
    ctx, new = [600, 3000, 40], [90, 3, 40]
    q, kp, vp, table, cu = pooled(ctx, new, 8, 2, 128, 16, torch.float16, 21)
    want = run_paged(q, kp, vp, table, ctx, cu, 0.1)
    out = torch.full_like(want, 7.0)
    ws = pa.alloc_prefill_workspace(3, q.shape[0], 8, 2, 128, 16, 3000)
    ctx_d, cu_d = ints(ctx), ints(cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_prefill_paged(out, q, kp, vp, table, ctx_d, cu_d, 0.1, 3000, ws)
    for _ in range(3):
        out.fill_(7.0)
        ws.fill_(255)
        graph.replay()
        assert torch.equal(bits(out), bits(want))
    # other lengths through the same graph
    ctx2, new2 = [33, 2999, 600], [33, 90, 10]
    q2, kp2, vp2, table2, cu2 = pooled(ctx2, new2, 8, 2, 128, 16, torch.float16, 22)
    assert q2.shape == q.shape and kp2.shape[0] <= kp.shape[0]
    q.copy_(q2)
    kp[:kp2.shape[0]] = kp2
    vp[:vp2.shape[0]] = vp2
    table[:, :table2.shape[1]] = table2[:, :table.shape[1]]
    ctx_d.copy_(ints(ctx2))
    cu_d.copy_(ints(cu2))
    graph.replay()
    assert pa.pa_device_errors() == 0
    for s, c in enumerate(ctx2):
        a, b = cu2[s], cu2[s + 1]
        check(out[a:b], *ref.attention(q[a:b], ref.gather(kp, table[s], c), ref.gather(vp, table[s], c), 0.1, c - (b - a)))


# ---- the operators together ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_prompts_then_chunks_then_decode(dtype):
    """Three requests: prompts through assign, rope and packed attention; a further chunk of two of them through
    assign, rope and paged attention; then a token of each through assign, rope and pa_decode."""
    H, Hkv, D, bs, NB, B, W = 8, 2, 128, 16, 64, 3, 32
    g = gen(31)
    inv = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
    kp = torch.full((NB, Hkv, bs, D), float("nan"), dtype=dtype, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    table = torch.full((B, W), -1, dtype=I32, device="cuda")
    free, nf, ctx = torch.arange(NB, dtype=I32, device="cuda"), ints([NB]), ints([0] * B)
    keys, vals = [[] for _ in range(B)], [[] for _ in range(B)]
    scale = 1 / math.sqrt(D)
    for step, new in enumerate([[50, 7, 130], [33, 0, 5], [1, 1, 1]]):
        T, rows = sum(new), 192
        x = normal((rows, H + 2 * Hkv, D), dtype, g)
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        slots = torch.empty(rows, dtype=I64, device="cuda")
        pos = torch.empty(rows, dtype=I32, device="cuda")
        cu = torch.empty(B + 1, dtype=I32, device="cuda")
        pa.pa_assign_slots(table, free, ctx, nf, ints(new), bs, slots, pos, cu)
        qr = torch.full((rows, H, D), float("nan"), dtype=dtype, device="cuda")
        kr = torch.full((rows, Hkv, D), float("nan"), dtype=dtype, device="cuda")
        pa.pa_rope_and_cache(qr, q, k, v, kp, vp, pos, slots, inv, k_out=kr)
        out = torch.full((rows, H, D), 7.0, dtype=dtype, device="cuda")
        if step == 0:
            pa.pa_prefill(out, qr, kr, v, cu, scale)
            out2 = torch.full_like(out, 7.0)
            pa.pa_prefill_paged(out2, qr, kp, vp, table, ctx, cu, scale, W * bs)
            assert (out2[T:] == 7.0).all()
        elif step == 1:
            pa.pa_prefill_paged(out, qr, kp, vp, table, ctx, cu, scale, W * bs)
        else:
            pa.pa_decode(out[:B], qr[:B], kp, vp, table, ctx, scale, W * bs)
        assert pa.pa_device_errors() == 0
        assert (out[T:] == 7.0).all()
        ends = cu.tolist()
        assert ends[-1] == T
        for s in range(B):
            a, b = ends[s], ends[s + 1]
            keys[s].append(kr[a:b])
            vals[s].append(v[a:b])
            if b > a:
                kk, vv = torch.cat(keys[s]), torch.cat(vals[s])
                want, bound = ref.attention(qr[a:b], kk, vv, scale, kk.shape[0] - (b - a))
                check(out[a:b], want, bound)
                if step == 0:
                    check(out2[a:b], want, bound)
    assert nf.item() == NB - sum(-(-n // bs) for n in ctx.tolist())
