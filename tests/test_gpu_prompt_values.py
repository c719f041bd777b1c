"""Prompt attention on scores and values far from the ordinary: scores that 32 bits hold to whole numbers only, weights
far below the largest, values near the type's largest, infinities and NaN."""
import pytest
import torch

import paged_kv_cache_372_b200 as pa
from tests import prompt_reference as ref
from tests.test_gpu_prompt_path import bits, check, gen, ints, normal, run_packed, run_paged

pytestmark = pytest.mark.gpu

U = ref.U


def one_pool(k, v, bs):
    """k, v [m][Hkv][D] as the blocks of one sequence, in order."""
    m, Hkv, D = k.shape
    nb = -(-m // bs)
    kp, vp = (torch.zeros((nb * bs, Hkv, D), dtype=k.dtype, device="cuda") for _ in range(2))
    kp[:m], vp[:m] = k, v
    kp, vp = (x.view(nb, bs, Hkv, D).transpose(1, 2).contiguous() for x in (kp, vp))
    return kp, vp, ints([list(range(nb))])


def equal_scores(n, rows, H, Hkv, D, dtype, a, seed):
    """Every score of the last rows is the same: a^2 D scale, exactly; the weights are equal."""
    q = torch.full((rows, H, D), a, dtype=dtype, device="cuda")
    k = torch.full((n, Hkv, D), a, dtype=dtype, device="cuda")
    return q, k, normal((n, Hkv, D), dtype, gen(seed))


# Powers of two, so that every product and sum of the scores is exact; the scaled score has 2^20 to 2^61.
SIZES = [(torch.float16, 2.0 ** 9), (torch.float16, 2.0 ** 11), (torch.float16, 2.0 ** 13), (torch.float16, 2.0 ** 14.5 // 1),
         (torch.bfloat16, 2.0 ** 13), (torch.bfloat16, 2.0 ** 16), (torch.bfloat16, 2.0 ** 28)]


@pytest.mark.parametrize("dtype,a", SIZES, ids=lambda x: str(x))
@pytest.mark.parametrize("H,Hkv,D", [(2, 2, 64), (4, 1, 128)])
@pytest.mark.parametrize("scale", [0.0912, -0.0912])
def test_equal_scores_of_any_size_weigh_equally(dtype, a, H, Hkv, D, scale):
    n = 300
    q, k, v = equal_scores(n, n, H, Hkv, D, dtype, a, 80)
    out = run_packed(q, k, v, [0, n], scale, compare=False)
    rows = torch.arange(1, n + 1, device="cuda", dtype=torch.float64)[:, None, None]
    mean = (v.double().cumsum(0) / rows).repeat_interleave(H // Hkv, 1)
    size = (v.double().abs().cumsum(0) / rows).repeat_interleave(H // Hkv, 1)
    # its rounding, the weights' rounding to the type, 32-bit sums of n products
    bound = U[dtype] * mean.abs() + (U[dtype] + 2 * n * 2.0 ** -24) * size + 2.0 ** -25
    check(out, mean, bound)


@pytest.mark.parametrize("dtype,a", SIZES, ids=lambda x: str(x))
@pytest.mark.parametrize("n,rows", [(2500, 3), (700, 300)])
def test_one_score_above_many_equal_ones_of_any_size(dtype, a, n, rows):
    # the largest key's score is a quarter above the others': it takes all of the weight
    q, k, v = equal_scores(n, rows, 4, 2, 128, dtype, a, 81)
    at = n - rows // 2 - 1
    k[at] *= 1.25
    kp, vp, table = one_pool(k, v, 16)
    out = torch.full_like(q, 7.0)
    pa.pa_prefill_paged(out, q, kp, vp, table, ints([n]), ints([0, rows]), 0.0912, n)
    assert pa.pa_device_errors() == 0
    sees = n - rows + torch.arange(rows, device="cuda") >= at
    assert torch.equal(bits(out[sees]), bits(v[at].repeat_interleave(2, 0).expand(int(sees.sum()), 4, 128)))
    i = torch.arange(n, device="cuda")[None, :, None, None]
    seen = (i <= n - rows + torch.arange(rows, device="cuda")[:, None, None, None])[~sees]
    count = seen.sum(1)
    mean = (seen * v.double()[None]).sum(1) / count
    size = (seen * v.double().abs()[None]).sum(1) / count
    bound = U[dtype] * mean.abs() + (U[dtype] + 2 * n * 2.0 ** -24) * size + 2.0 ** -25
    check(out[~sees], mean.repeat_interleave(2, 1), bound.repeat_interleave(2, 1))


@pytest.mark.parametrize("n,rows", [(40000, 2), (9000, 300)])
def test_many_weights_far_below_the_largest_add_up_in_fp16(n, rows):
    # the first key takes nearly all of the weight and has the value 0; each other one has e^-18, below 2^-25
    q = torch.zeros((rows, 2, 64), dtype=torch.float16, device="cuda")
    k = torch.zeros((n, 1, 64), dtype=torch.float16, device="cuda")
    v = torch.ones((n, 1, 64), dtype=torch.float16, device="cuda")
    q[..., 0], k[0, :, 0], v[0] = 1.0, 18.0, 0.0
    kp, vp, table = one_pool(k, v, 64)
    out = torch.full_like(q, 7.0)
    pa.pa_prefill_paged(out, q, kp, vp, table, ints([n]), ints([0, rows]), 1.0, n)
    assert pa.pa_device_errors() == 0
    rest = (n - rows + torch.arange(rows, device="cuda", dtype=torch.float64)) * torch.exp(torch.tensor(-18.0).double())
    want = (rest / (1 + rest))[:, None, None].expand(out.shape)
    # its rounding; each weight is off by 2^-25 of 2^7 times the largest; 32-bit sums and exponentials (2^-17)
    check(out, want, 2.0 ** -11 * want + n * 2.0 ** -32 + 2.0 ** -17 * want)


@pytest.mark.parametrize("n,rows", [(300, 300), (1500, 4)])
def test_sums_of_values_near_the_largest_of_bf16(n, rows):
    q = torch.zeros((rows, 4, 128), dtype=torch.bfloat16, device="cuda")
    k = normal((n, 2, 128), torch.bfloat16, gen(82))
    v = torch.full((n, 2, 128), 2.0 ** 120, dtype=torch.bfloat16, device="cuda")
    kp, vp, table = one_pool(k, v, 32)
    out = torch.full_like(q, 7.0)
    pa.pa_prefill_paged(out, q, kp, vp, table, ints([n]), ints([0, rows]), 0.1, n)
    assert pa.pa_device_errors() == 0
    assert (out == 2.0 ** 120).all()
    if n == rows:
        assert (run_packed(q, k, v, [0, n], 0.1, compare=False) == 2.0 ** 120).all()


def long_row(n):
    """Seconds and the result of one row over n keys in the row form, a warp's work, while the 8 warps' next work item
    waits: the last of 56 sequences is long, and one of its 8 heads has scores of 2^30."""
    H, D, bs, B = 8, 64, 64, 56
    width = -(-n // bs)
    q, kp, vp = (normal(s, torch.float16, gen(83)) for s in ((B, H, D), (3, H, bs, D), (3, H, bs, D)))
    q[-1, 0] = 8192.0
    kp[:2, 0] = 8192.0
    kp[1, 0, 0] *= 1.25  # the key that takes all of the weight
    table = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    table[:-1, 0] = 2
    table[-1, width // 2] = 1
    out = torch.full_like(q, 7.0)
    args = (out, q, kp, vp, table, ints([1] * (B - 1) + [n]), ints(list(range(B + 1))), 0.125, n)
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ends[0].record()
    pa.pa_prefill_paged(*args)
    ends[1].record()
    assert pa.pa_device_errors() == 0
    assert torch.equal(bits(out[-1, 0]), bits(vp[1, 0, 0]))
    assert torch.equal(bits(out[:-1]), bits(vp[2, :, 0].expand(B - 1, H, D)))
    return ends[0].elapsed_time(ends[1]) / 1e3


def test_an_item_may_last_longer_than_a_wait():
    # a wait of 4 seconds would have run out
    assert long_row(50_000_000) > 4.2


def milliseconds(call):
    for _ in range(2):
        call()
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ends[0].record()
    call()
    ends[1].record()
    torch.cuda.synchronize()
    assert pa.pa_device_errors() == 0
    return ends[0].elapsed_time(ends[1])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["first key", "first value", "all values", "behind the last"])
def test_one_bad_row_does_not_slow_the_others(bad, where):
    # a row alone, key by key, takes 100 ns a key: 8190 rows of 8 heads in that form took 400 times the whole call
    n, tail = 8190, 50
    q, k, v = (normal((n + tail, h, 128), torch.bfloat16, gen(84)) for h in (8, 2, 2))
    out, cu = torch.empty_like(q), ints([0, n])
    clean = milliseconds(lambda: pa.pa_prefill(out, q, k, v, cu, 0.088))
    want = out.clone()
    if where == "first key":
        k[0, :, 5] = bad
    elif where == "first value":
        v[0, :, 5] = bad
    elif where == "all values":
        v[:, :, 5] = float("nan")
    else:
        k[n:], v[n:], q[n:] = bad, bad, bad
    took = milliseconds(lambda: pa.pa_prefill(out, q, k, v, cu, 0.088))
    assert took < 5 * clean + 0.5, f"{took:.2f} ms against {clean:.2f}"
    if where == "behind the last":
        assert torch.equal(bits(out[:n]), bits(want[:n]))
    elif where == "first key":
        assert torch.isnan(out[:n]).all() if bad != bad else True
    else:
        assert not torch.isfinite(out[:n, :, 5]).any()
        others = torch.arange(128, device="cuda") != 5
        assert torch.equal(bits(out[:n, :, others]), bits(want[:n, :, others]))


def formula(q, k, v, scale, first):
    """ref.attention where values that are not finite count for the rows that see them only."""
    want, bound = ref.attention(q, k, v.where(torch.isfinite(v), 0.0), scale, first)
    n, H, D = q.shape
    for j, h, d in (~torch.isfinite(v)).nonzero().tolist():
        heads = slice(h * H // v.shape[1], (h + 1) * H // v.shape[1])
        z = torch.einsum("ngd,d->ng", q[max(j - first, 0):, heads].double(), k[j, h].double()) * scale
        # weight 0 (a score of -inf) times infinity is NaN
        want[max(j - first, 0):, heads, d] += torch.where(z == -float("inf"), float("nan"), v[j, h, d].double())
    return want, bound


@pytest.mark.parametrize("seed", range(16))
def test_bad_values_anywhere(seed):
    """NaN, infinities and values half of the type's largest at random places of keys and values: what the formula gives, row by row."""
    g = torch.Generator().manual_seed(300 + seed)

    def pick(*x):
        return x[int(torch.randint(0, len(x), (1,), generator=g))]

    Hkv, group, D, bs = pick(1, 2), pick(1, 2, 4, 8), pick(64, 128), pick(16, 64)
    dtype = pick(torch.float16, torch.bfloat16)
    H, n = Hkv * group, pick(150, 700, 1500)
    rows = n if seed % 2 else pick(3, 40)
    q, k, v = (normal((n, h, D), dtype, gen(300 + seed)) for h in (H, Hkv, Hkv))
    for x, kinds in ((k, [float("nan"), float("inf"), -float("inf")]),
                     (v, [float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).max / 2])):
        for _ in range(pick(0, 1, 3, 20)):
            j = int(torch.randint(0, n, (1,), generator=g)) if pick(0, 1) else n - 1 - int(torch.randint(0, 140, (1,), generator=g))
            x[j, pick(*range(Hkv)), int(torch.randint(0, D, (1,), generator=g))] = pick(*kinds)
    want, bound = formula(q[n - rows:], k, v, 0.09, n - rows)
    outs = []
    if rows == n:
        outs.append(run_packed(q, k, v, [0, n], 0.09, compare=False))
    kp, vp, table = one_pool(k, v, bs)
    out = torch.full((rows, H, D), 7.0, dtype=dtype, device="cuda")
    pa.pa_prefill_paged(out, q[n - rows:], kp, vp, table, ints([n]), ints([0, rows]), 0.09, n)
    assert pa.pa_device_errors() == 0
    for out in outs + [out]:
        fine = torch.isfinite(want)
        assert torch.isnan(out[torch.isnan(want)]).all()
        assert not torch.isfinite(out[~fine]).any()
        err = (out.double() - want).abs()
        assert (err <= bound)[fine].all()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("Hkv,group,D,dtype", [(2, 1, 128, torch.float16), (1, 4, 128, torch.bfloat16),
                                               (2, 8, 64, torch.bfloat16)])
def test_bad_values_in_some_of_many_sequences(paged, Hkv, group, D, dtype):
    """Several work items for each SM, some walked twice: the other sequences' rows keep their bits."""
    g = torch.Generator().manual_seed(Hkv + group)
    lens = torch.randint(0, 500, (150,), generator=g).tolist() + [2500, 1, 0, 900]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T, H = cu[-1], Hkv * group
    q, k, v = (normal((T + 9, h, D), dtype, gen(310)) for h in (H, Hkv, Hkv))
    v[T:] = float("nan")
    if paged:
        bs = 32
        width = -(-max(lens) // bs)
        used = [-(-n // bs) for n in lens]
        table = torch.full((len(lens), width), -3, dtype=torch.int32)
        first = 0
        for s, w in enumerate(used):
            table[s, :w] = torch.arange(first, first + w)
            first += w
        table = table.cuda()

    def run(v):
        out = torch.full_like(q, 7.0)
        if not paged:
            pa.pa_prefill(out, q, k, v, ints(cu), 0.09)
        else:
            pools = []
            for x in (k, v):
                rows = torch.full((first * bs, Hkv, D), float("nan"), dtype=dtype, device="cuda")
                at = 0
                for s, w in enumerate(used):
                    rows[at:at + lens[s]] = x[cu[s]:cu[s + 1]]
                    at += w * bs
                pools.append(rows.view(first, bs, Hkv, D).transpose(1, 2).contiguous())
            pa.pa_prefill_paged(out, q, *pools, table, ints(lens), ints(cu), 0.09, max(lens))
        assert pa.pa_device_errors() == 0
        assert (out[T:] == 7.0).all()
        return out

    clean = run(v)
    bad = v.clone()
    hurt = [s for s in range(0, len(lens), 7) if lens[s]] + [150, 153]
    for s in hurt:
        for kind in (float("nan"), float("inf"), -float("inf")):
            j = cu[s] + int(torch.randint(0, lens[s], (1,), generator=g))
            bad[j, int(torch.randint(0, Hkv, (1,), generator=g)), int(torch.randint(0, D, (1,), generator=g))] = kind
    out = run(bad)
    for s in range(len(lens)):
        a, b = cu[s], cu[s + 1]
        if s not in hurt:
            assert torch.equal(bits(out[a:b]), bits(clean[a:b]))
        elif b > a:
            want, bound = formula(q[a:b], k[a:b], bad[a:b], 0.09, 0)
            fine = torch.isfinite(want)
            assert torch.isnan(out[a:b][torch.isnan(want)]).all()
            assert not torch.isfinite(out[a:b][~fine]).any()
            assert torch.equal(out[a:b][fine], clean[a:b][fine])


@pytest.mark.parametrize("rows", [1, 3, 40, 100])
@pytest.mark.parametrize("Hkv,group,D,bs,dtype", [(1, 1, 64, 16, torch.float16), (2, 4, 128, 32, torch.bfloat16),
                                                  (1, 8, 128, 64, torch.float16)])
def test_bad_values_in_split_contexts(rows, Hkv, group, D, bs, dtype):
    """Parts of a chain, walked in halves where the rows are few: bad rows at the diagonal, in other parts, at a part's edge."""
    n, H = 5000, Hkv * group
    g = torch.Generator().manual_seed(rows + group)
    q, k, v = (normal((m, h, D), dtype, gen(320 + rows)) for m, h in ((rows, H), (n, Hkv), (n, Hkv)))
    assert pa.pa_prefill_paged_workspace_size(1, rows, H, Hkv, D, bs, n) > 256
    places = [0, 127, 128, 2559, 2560, n - 1, n - rows, n - 1 - rows // 2, n - 1 - rows // 3]
    for i, j in enumerate(places):
        kind = (float("nan"), float("inf"), -float("inf"))[i % 3]
        d = int(torch.randint(0, D, (1,), generator=g))
        v[j, i % Hkv, d] = kind
        if i % 4 == 3:
            k[j, i % Hkv, (d + 1) % D] = -float("inf")
    kp, vp, table = one_pool(k, v, bs)
    out = torch.full((rows, H, D), 7.0, dtype=dtype, device="cuda")
    pa.pa_prefill_paged(out, q, kp, vp, table, ints([n]), ints([0, rows]), 0.09, n)
    assert pa.pa_device_errors() == 0
    want, bound = formula(q, k, v, 0.09, n - rows)
    fine = torch.isfinite(want)
    assert torch.isnan(out[torch.isnan(want)]).all()
    assert not torch.isfinite(out[~fine]).any()
    assert ((out.double() - want).abs() <= bound)[fine].all()
