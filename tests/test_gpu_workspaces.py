"""Workspaces on the GPU: a call without one, on the current stream, directly followed by one on another stream."""
import pytest
import torch

import paged_kv_cache_372_b200 as pa
from tests.test_gpu_prompt_path import bits, ints, pooled, run_paged

pytestmark = pytest.mark.gpu


def test_split_calls_without_a_workspace_on_the_current_and_on_another_stream():
    side = torch.cuda.Stream()
    calls = []
    for seed in (60, 61):
        ctx, new = [9000, 40, 5000], [30, 40, 9]
        q, kp, vp, table, cu = pooled(ctx, new, 8, 2, 128, 16, torch.bfloat16, seed)
        calls.append((q, kp, vp, table, ints(ctx), ints(cu), run_paged(q, kp, vp, table, ctx, cu, 0.1)))
    torch.cuda.synchronize()
    for _ in range(20):
        outs = [torch.full_like(calls[i % 2][-1], 7.0) for i in range(4)]
        torch.cuda.synchronize()
        for i, out in enumerate(outs):
            q, kp, vp, table, ctx, cu, want = calls[i % 2]
            pa.pa_prefill_paged(out, q, kp, vp, table, ctx, cu, 0.1, 9000, stream=side if i % 2 else None)
        torch.cuda.synchronize()
        assert pa.pa_device_errors() == 0
        for i, out in enumerate(outs):
            assert torch.equal(bits(out), bits(calls[i % 2][-1]))


@pytest.mark.parametrize("call", [pa.pa_decode, pa.pa_decode_shared], ids=lambda f: f.__name__)
def test_decodes_without_a_workspace_on_the_current_and_on_another_stream(call):
    side = torch.cuda.Stream()
    calls = []
    for seed in (62, 63):
        ctx = [9000, 40, 5000, 1]
        q, kp, vp, table, _ = pooled(ctx, [1] * 4, 8, 2, 128, 16, torch.bfloat16, seed)
        q = q[:4].contiguous()
        args = (q, kp, vp, table, ints(ctx), 0.1, 9000)
        calls.append((args, call(torch.full_like(q, 7.0), *args)))
    torch.cuda.synchronize()
    assert pa.pa_device_errors() == 0
    for _ in range(20):
        outs = [torch.full_like(calls[i % 2][1], 7.0) for i in range(4)]
        torch.cuda.synchronize()
        for i, out in enumerate(outs):
            call(out, *calls[i % 2][0], stream=side if i % 2 else None)
        torch.cuda.synchronize()
        assert pa.pa_device_errors() == 0
        for i, out in enumerate(outs):
            # partitions may merge in any order: 32-bit sums, one rounding to the type
            want = calls[i % 2][1].float()
            assert ((out.float() - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -18).all()


@pytest.mark.parametrize("H,Hkv,D", [(32, 8, 128), (8, 1, 64), (4, 4, 128)])
def test_prefill_workspace_size_grows_with_every_size(H, Hkv, D):
    def size(b, t, c):
        return pa.pa_prefill_paged_workspace_size(b, t, H, Hkv, D, 16, c)

    seqs, tokens, limits = (1, 2, 8, 16, 64, 400), (1, 3, 16, 64, 500, 2048, 4096, 9000), (40, 1000, 1024, 2944, 32768)
    for b in seqs:
        for t in tokens:
            for c in limits:
                n = size(b, t, c)
                assert 256 <= n <= 138 << 20
                assert all(size(*x) <= n for x in ((b - 1, t, c), (b, t - 1, c), (b, t, c - 1), (1, t, c), (b, 1, c)))


def test_a_workspace_for_the_largest_sizes_serves_smaller_calls():
    H, Hkv, D, bs, most = 8, 2, 128, 16, (64, 9000, 8192)
    ws = pa.alloc_prefill_workspace(most[0], most[1], H, Hkv, D, bs, most[2])
    for ctx, new in [([8000], [1]), ([40], [40]), ([3000, 5, 8192], [8, 5, 700]), ([1100] * 64, [3] * 64),
                     ([8192, 808], [8192, 808])]:
        q, kp, vp, table, cu = pooled(ctx, new, H, Hkv, D, bs, torch.bfloat16, 70)
        ws.fill_(255)
        for limit in (max(ctx), most[2]):
            run_paged(q, kp, vp, table, ctx, cu, 0.1, limit, ws)


def test_a_workspace_too_small_for_its_call_is_refused():
    ctx, new = [3000], [8]
    q, kp, vp, table, cu = pooled(ctx, new, 8, 2, 128, 16, torch.bfloat16, 71)
    out = torch.full_like(q, 7.0)
    n = pa.pa_prefill_paged_workspace_size(1, q.shape[0], 8, 2, 128, 16, 3000)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    with pytest.raises(pa.PagedAttentionError) as e:
        pa.pa_prefill_paged(out, q, kp, vp, table, ints(ctx), ints(cu), 0.1, 3000, ws[:n - 256])
    assert e.value.status == pa.PA_ERR_INVALID and (out == 7.0).all()


def microseconds(call):
    for _ in range(3):
        call()
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ends[0].record()
    for _ in range(20):
        call()
    ends[1].record()
    torch.cuda.synchronize()
    return ends[0].elapsed_time(ends[1]) * 50


@pytest.mark.parametrize("n,limit", [(2048, 2048), (3500, 3500), (2048, 32768)])
def test_a_whole_prompt_over_the_cache_takes_about_the_packed_call(n, limit):
    # split among the SMs it took four times as long
    H, Hkv, D, bs = 32, 8, 128, 16
    q, kp, vp, table, cu = pooled([n], [n], H, Hkv, D, bs, torch.bfloat16, 72)
    wide = torch.zeros((1, limit // bs + 1), dtype=torch.int32, device="cuda")
    wide[:, :min(table.shape[1], wide.shape[1])] = table[:, :wide.shape[1]]
    ctx, cu = ints([n]), ints(cu)
    out, ws = torch.empty_like(q), pa.alloc_prefill_workspace(1, q.shape[0], H, Hkv, D, bs, limit)
    k, v = torch.randn((2, q.shape[0], Hkv, D), device="cuda").to(q.dtype)
    paged = microseconds(lambda: pa.pa_prefill_paged(out, q, kp, vp, wide, ctx, cu, 0.09, limit, ws))
    whole = microseconds(lambda: pa.pa_prefill(out, q, k, v, cu, 0.09))
    assert pa.pa_device_errors() == 0
    assert paged < 2 * whole, f"{paged:.0f} us against {whole:.0f}"


def test_a_few_tokens_over_unequal_contexts_take_no_longer_than_their_cache():
    # 16 requests over 4096 to 32768 tokens: whole, the longest of them took the SMs that have it 263 us; split 199
    H, Hkv, D, bs, B, n = 32, 8, 128, 64, 16, 8
    ctx = [4096 + 28672 * i // (B - 1) for i in range(B)]
    q, kp, vp, table, cu = pooled(ctx, [n] * B, H, Hkv, D, bs, torch.bfloat16, 73)
    ctx_d, cu = ints(ctx), ints(cu)
    out, ws = torch.empty_like(q), pa.alloc_prefill_workspace(B, q.shape[0], H, Hkv, D, bs, max(ctx))
    took = microseconds(lambda: pa.pa_prefill_paged(out, q, kp, vp, table, ctx_d, cu, 0.09, max(ctx), ws))
    assert pa.pa_device_errors() == 0
    bytes_read = 2 * 2 * D * Hkv * sum(ctx)
    assert took < 1.2 * bytes_read / 6.0e6 + 20, f"{took:.0f} us for {bytes_read / 1e6:.0f} MB"
