"""Calls of the prompt path that its documentation allows and ordinary use rarely makes: split contexts with
bad values, unaligned outputs, thousands of sequences, caches behind 2^31 elements, calls at once on two streams,
captured calls, every position of a bad key."""
import math

import pytest
import torch

import paged_kv_cache_372_b200 as pa
from tests import prompt_reference as ref
from tests.test_gpu_prompt_path import bits, check, gen, ints, normal, packed, pooled, run_packed, run_paged

pytestmark = pytest.mark.gpu

I32, I64 = torch.int32, torch.int64


def test_prefill_nonfinite_key_at_every_place_of_a_chunk():
    # a key of NaN or infinity among the first 16: the rows before it are as without it, those from it on are not finite
    n, D = 130, 128
    q, k, v, cu = packed([n], 4, 4, D, torch.float16, False, 40, tail=0)
    clean = run_packed(q, k, v, cu, 0.09)
    for at in range(0, 34):
        for bad in (float("nan"), float("inf")):
            k2 = k.clone()
            k2[at, :, 3] = bad
            out = run_packed(q, k2, v, cu, 0.09, compare=False)
            assert torch.equal(bits(out[:at]), bits(clean[:at]))
            want, _ = ref.attention(q[at:], k2, v, 0.09, at)
            assert torch.equal(torch.isfinite(out[at:]), torch.isfinite(want))


@pytest.mark.parametrize("offset", [8, 16])
def test_prefill_output_at_16_bytes(offset):
    q, k, v, cu = packed([200, 33], 4, 2, 64, torch.bfloat16, False, 41, tail=0)
    want = run_packed(q, k, v, cu, 0.1)
    buf = torch.full((q.numel() + 64,), 7.0, dtype=q.dtype, device="cuda")
    out = buf[offset:offset + q.numel()].view(q.shape)
    pa.pa_prefill(out, q, k, v, ints(cu), 0.1)
    assert pa.pa_device_errors() == 0
    assert torch.equal(bits(out), bits(want))
    assert (buf[:offset] == 7.0).all() and (buf[offset + q.numel():] == 7.0).all()


@pytest.mark.parametrize("paged", [False, True])
def test_two_thousand_short_sequences(paged):
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(0, 5, (2000,), generator=g).tolist()
    if paged:
        ctx = [n + (i % 40) for i, n in enumerate(lens)]
        q, kp, vp, table, cu = pooled(ctx, lens, 4, 1, 64, 16, torch.float16, 42)
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        pa.pa_prefill_paged(out, q, kp, vp, table, ints(ctx), ints(cu), 0.1, max(ctx))
    else:
        q, k, v, cu = packed(lens, 4, 1, 64, torch.float16, True, 43)
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        pa.pa_prefill(out, q, k, v, ints(cu), 0.1)
    assert pa.pa_device_errors() == 0
    assert (out[cu[-1]:] == 7.0).all() and not (out[:cu[-1]] == 7.0).all(-1).any()
    for s in range(0, 2000, 13):
        a, b = cu[s], cu[s + 1]
        if b > a:
            if paged:
                kk, vv = ref.gather(kp, table[s], ctx[s]), ref.gather(vp, table[s], ctx[s])
                check(out[a:b], *ref.attention(q[a:b], kk, vv, 0.1, ctx[s] - (b - a)))
            else:
                check(out[a:b], *ref.attention(q[a:b], k[a:b], v[a:b], 0.1, 0))


@pytest.mark.parametrize("H,Hkv,D,bs", [(8, 2, 128, 16), (4, 4, 64, 64), (8, 1, 64, 32)])
@pytest.mark.parametrize("scale", [0.09, -0.09])
def test_split_contexts(H, Hkv, D, bs, scale):
    """Few rows over long contexts (parts, walked in halves), with rows that see nothing, one key, or end inside a part."""
    ctx, new = [2000, 3, 0, 517, 4096, 129], [7, 9, 4, 1, 40, 129]
    q, kp, vp, table, cu = pooled(ctx, new, H, Hkv, D, bs, torch.bfloat16, 44, stale=float("nan"))
    assert pa.pa_prefill_paged_workspace_size(6, q.shape[0], H, Hkv, D, bs, 4096) > 256
    out = run_paged(q, kp, vp, table, ctx, cu, scale)
    assert (out[cu[1]:cu[1] + 6] == 0).all() and (out[cu[2]:cu[3]] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_split_contexts_with_a_bad_value_row(bad):
    ctx, new = [3000], [20]
    q, kp, vp, table, cu = pooled(ctx, new, 4, 1, 128, 16, torch.float16, 45)
    clean = run_paged(q, kp, vp, table, ctx, cu, 0.1, 4096)
    at = 2990  # among the new tokens: 10 rows before it, 10 from it on
    vp[table[0, at // 16].long(), :, at % 16, 5] = bad
    out = torch.empty_like(clean)
    pa.pa_prefill_paged(out, q, kp, vp, table, ints(ctx), ints(cu), 0.1, 4096)
    assert pa.pa_device_errors() == 0
    assert torch.isfinite(out[:10]).all()
    want, bound = ref.attention(q[:10], ref.gather(kp, table[0], 2990), ref.gather(vp, table[0], 2990), 0.1, 2980)
    check(out[:10], want, bound)
    assert not torch.isfinite(out[10:20, :, 5]).any()
    assert torch.isfinite(out[10:20, :, 6:]).all()


def test_caches_behind_two_to_the_31_elements():
    bs, Hkv, D, NB = 64, 8, 128, 33200            # 65536 elements a block: 2.18e9 elements a pool
    kp = torch.empty((NB, Hkv, bs, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    g = gen(46)
    ids = list(range(NB - 8, NB))
    T = 400
    slots = torch.tensor([ids[t // bs] * bs + t % bs for t in range(T)], dtype=I64, device="cuda")
    q, k, v = normal((T, 8, D), torch.bfloat16, g), normal((T, Hkv, D), torch.bfloat16, g), normal((T, Hkv, D), torch.bfloat16, g)
    pos = torch.arange(T, dtype=I32, device="cuda")
    inv = 10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pa.pa_rope_and_cache(qo, q, k, v, kp, vp, pos, slots, inv, k_out=ko)
    table = ints([ids])
    out = torch.empty_like(q)
    pa.pa_prefill_paged(out, qo, kp, vp, table, ints([T]), ints([0, T]), 0.088, T)
    assert pa.pa_device_errors() == 0
    assert torch.equal(bits(ref.gather(kp, table[0], T)), bits(ko))
    check(out, *ref.attention(qo, ko, v, 0.088, 0))


def test_two_calls_at_once_on_two_streams():
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    ctx, new = [3000, 40, 700], [30, 40, 9]
    q, kp, vp, table, cu = pooled(ctx, new, 8, 2, 128, 16, torch.bfloat16, 47)
    want = run_paged(q, kp, vp, table, ctx, cu, 0.1)
    q2, k2, v2, cu2 = packed([600, 31, 200], 8, 2, 128, torch.bfloat16, False, 48)
    want2 = run_packed(q2, k2, v2, cu2, 0.1)
    ctx_d, cu_d, cu2_d = ints(ctx), ints(cu), ints(cu2)
    outs = [[torch.full_like(want, 7.0), torch.full_like(want2, 7.0)] for _ in range(6)]
    torch.cuda.synchronize()
    for i, (x, y) in enumerate(outs):
        s, t = (a, b) if i % 2 else (b, a)
        # no workspace given: each call has its own
        pa.pa_prefill_paged(x, q, kp, vp, table, ctx_d, cu_d, 0.1, max(ctx), stream=s)
        pa.pa_prefill(y, q2, k2, v2, cu2_d, 0.1, stream=t)
    torch.cuda.synchronize()
    assert pa.pa_device_errors() == 0
    for x, y in outs:
        assert torch.equal(bits(x), bits(want)) and torch.equal(bits(y), bits(want2))


def test_a_step_captured_and_replayed():
    """Slots, rotation, cache write and attention of a step in one graph, replayed: each replay is the next step."""
    H, Hkv, D, bs, NB, B, W = 4, 2, 64, 16, 40, 2, 16
    g = gen(49)
    kp, vp = torch.zeros((NB, Hkv, bs, D), dtype=torch.float16, device="cuda"), torch.zeros((NB, Hkv, bs, D),
                                                                                         dtype=torch.float16, device="cuda")
    table, free = torch.full((B, W), -1, dtype=I32, device="cuda"), torch.arange(NB, dtype=I32, device="cuda")
    ctx, nf, new = ints([0, 0]), ints([NB]), ints([5, 3])
    slots, pos, cu = torch.empty(10, dtype=I64, device="cuda"), ints([0] * 10), ints([0] * 3)
    inv = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
    q, k, v = (normal((10, h, D), torch.float16, g) for h in (H, Hkv, Hkv))
    qo, ko, out = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(q)
    ws = pa.alloc_prefill_workspace(B, 10, H, Hkv, D, bs, W * bs)

    def step():
        pa.pa_assign_slots(table, free, ctx, nf, new, bs, slots, pos, cu)
        pa.pa_rope_and_cache(qo, q, k, v, kp, vp, pos, slots, inv, k_out=ko)
        pa.pa_prefill_paged(out, qo, kp, vp, table, ctx, cu, 0.125, W * bs, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    keys, vals = [[], []], [[], []]
    for i in range(12):
        q.copy_(normal(q.shape, q.dtype, g))
        k.copy_(normal(k.shape, k.dtype, g))
        v.copy_(normal(v.shape, v.dtype, g))
        graph.replay()
        assert pa.pa_device_errors() == 0
        assert ctx.tolist() == [5 * (i + 1), 3 * (i + 1)]
        for s, (a, b) in enumerate([(0, 5), (5, 8)]):
            keys[s].append(ko[a:b].clone())
            vals[s].append(v[a:b].clone())
            kk, vv = torch.cat(keys[s]), torch.cat(vals[s])
            check(out[a:b], *ref.attention(qo[a:b], kk, vv, 0.125, kk.shape[0] - (b - a)))


def test_assign_larger_than_one_cta_refuses_whole_and_in_place():
    # past the size of one CTA's launch: refused whole, then served in place
    B, W, NB, bs = 64, 32, 4096, 16
    table, free = torch.full((B, W), -1, dtype=I32, device="cuda"), torch.arange(NB, dtype=I32, device="cuda")
    ctx, nf = ints([0] * B), ints([NB])
    T = B * 200
    slots, pos, cu = torch.empty(T, dtype=I64, device="cuda"), torch.empty(T, dtype=I32, device="cuda"), ints([0] * (B + 1))
    pa.pa_assign_slots(table, free, ctx, nf, ints([201] * B), bs, slots, pos, cu)
    assert pa.pa_device_errors() == pa.DEVERR_TOKENS
    assert (table == -1).all() and (ctx == 0).all() and nf.item() == NB and (slots == -1).all() and (pos == -1).all()
    pa.pa_assign_slots(table, free, ctx, nf, ints([200] * B), bs, slots, pos, cu)
    assert pa.pa_device_errors() == 0
    assert (ctx == 200).all() and nf.item() == NB - B * 13
    assert pos.view(B, 200).eq(torch.arange(200, device="cuda", dtype=I32)).all()
    blk = table.long()[:, :13].repeat_interleave(bs, dim=1)[:, :200]
    assert torch.equal(slots.view(B, 200), blk * bs + torch.arange(200, device="cuda") % bs)
    pa.pa_assign_slots(table, free, ctx, nf, ints([-1] * B), bs, slots, pos, cu)
    assert pa.pa_device_errors() == 0
    assert (ctx == 0).all() and nf.item() == NB and sorted(free.tolist()) == list(range(NB))


def test_rope_of_one_head_and_many_heads():
    for H, Hkv, T in [(1, 1, 3), (640, 1, 2), (100, 60, 700)]:
        g = gen(H)
        q, k, v = normal((T, H, 64), torch.float16, g), normal((T, Hkv, 64), torch.float16, g), None
        pos = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=I32)
        inv = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        pa.pa_rope_and_cache(qo, q, k, v, None, None, pos, None, inv, k_out=ko)
        want = ref.rope(q, pos, inv, 1.0, False)
        bound = 2.0 ** -11 * want.abs() + 2.0 ** -20 * q.double().abs().amax(-1, keepdim=True) + 2.0 ** -25
        check(qo, want, bound)


def test_prefill_far_from_the_diagonal_is_split_over_the_running_maximum():
    # the maximum grows by a little less, then a little more, than the lag the weights may have
    n, D = 600, 64
    for step in (7.9, 8.1, 40.0):
        q = torch.zeros((n, 4, D), dtype=torch.bfloat16, device="cuda")
        k = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
        q[..., 0] = 1.0
        k[:, 0, 0] = (torch.arange(n, device="cuda") // 128) * step * math.log(2.0)
        v = normal((n, 1, D), torch.bfloat16, gen(50))
        run_packed(q, k, v, [0, n], 1.0)


@pytest.mark.parametrize("seed", range(12))
def test_dealt_key_tiles(seed):
    """Few rows over contexts of any lengths, more than 32 sequences among them, limits far above the contexts."""
    g = torch.Generator().manual_seed(100 + seed)

    def pick(*x):
        return x[int(torch.randint(0, len(x), (1,), generator=g))]

    B = pick(1, 2, 5, 33, 70)
    Hkv = pick(1, 2)
    H = Hkv * pick(1, 2, 4, 8)
    D, bs, dtype = pick(64, 128), pick(16, 32, 64), pick(torch.float16, torch.bfloat16)
    top = pick(3, 200, 1500) if B > 5 else pick(40, 3000, 9000)
    ctx = torch.randint(0, top + 1, (B,), generator=g).tolist()
    new = [int(torch.randint(0, 12, (1,), generator=g)) if torch.rand(1, generator=g) < 0.8 else 0 for _ in ctx]
    if sum(new) == 0:
        new[0] = 1
    if max(ctx) == 0:
        ctx[0] = top
    limit = pick(max(ctx), 9216, 65536)
    q, kp, vp, table, cu = pooled(ctx, new, H, Hkv, D, bs, dtype, seed, stale=float("nan") if seed % 2 else None)
    wide = torch.full((B, -(-max(limit, 1) // bs)), -1, dtype=I32, device="cuda")
    wide[:, :min(table.shape[1], wide.shape[1])] = table[:, :wide.shape[1]]
    first = run_paged(q, kp, vp, wide, ctx, cu, 0.08, limit)
    ws = pa.alloc_prefill_workspace(B, q.shape[0], H, Hkv, D, bs, limit)
    ws.fill_(255)
    again = run_paged(q, kp, vp, wide, ctx, cu, 0.08, limit, ws)
    assert torch.equal(bits(first), bits(again))
