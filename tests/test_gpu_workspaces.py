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
