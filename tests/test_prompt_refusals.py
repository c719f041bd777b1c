"""What the prompt path's entry points refuse, at the C ABI and in the binding,
before anything reaches a device (CPU only)."""
import ctypes

import pytest
import torch

import paged_kv_cache_372_b200 as pa

P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(258)
F = ctypes.c_float


def assign(**kw):
    a = dict(tables=P, free=P, ctx_out=P, nf_out=P, slots=P, positions=P, cu=P, ctx=P, nf=P, new=P, seqs=4, width=8,
             bs=16, blocks=32, tokens=64)
    a.update(kw)
    return pa.lib().pa_assign_slots(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(seqs=-1), pa.PA_ERR_INVALID), (dict(width=0), pa.PA_ERR_INVALID), (dict(blocks=0), pa.PA_ERR_INVALID),
    (dict(tokens=-1), pa.PA_ERR_INVALID), (dict(bs=24), pa.PA_ERR_UNSUPPORTED), (dict(seqs=8193), pa.PA_ERR_UNSUPPORTED),
    (dict(tokens=(1 << 30) - 1), pa.PA_ERR_UNSUPPORTED), (dict(blocks=(1 << 30) - 1), pa.PA_ERR_UNSUPPORTED),
    (dict(width=1 << 26), pa.PA_ERR_UNSUPPORTED), (dict(tables=None), pa.PA_ERR_INVALID),
    (dict(slots=None), pa.PA_ERR_INVALID), (dict(nf=None), pa.PA_ERR_INVALID), (dict(cu=ODD), pa.PA_ERR_INVALID),
    (dict(slots=ctypes.c_void_p(260)), pa.PA_ERR_INVALID)])
def test_assign_slots_refuses(kw, status):
    assert assign(**kw) == status
    assert pa.lib().pa_last_error() != b""


def rope(**kw):
    a = dict(q_out=P, k_out=P, q=P, k=P, v=P, kp=P, vp=P, positions=P, slots=P, inv=P, tokens=4, heads=8, kv=2, D=128,
             rot=64, interleaved=0, bs=16, blocks=8, qs=1024, ks=256, vs=256, mscale=F(1.0), dtype=0)
    a.update(kw)
    return pa.lib().pa_rope_and_cache(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), pa.PA_ERR_INVALID), (dict(heads=0), pa.PA_ERR_INVALID), (dict(blocks=0), pa.PA_ERR_INVALID),
    (dict(dtype=2), pa.PA_ERR_INVALID), (dict(D=96), pa.PA_ERR_UNSUPPORTED), (dict(rot=0), pa.PA_ERR_UNSUPPORTED),
    (dict(rot=24), pa.PA_ERR_UNSUPPORTED), (dict(rot=144), pa.PA_ERR_UNSUPPORTED), (dict(bs=8), pa.PA_ERR_UNSUPPORTED),
    (dict(heads=65537), pa.PA_ERR_UNSUPPORTED), (dict(mscale=F(float("inf"))), pa.PA_ERR_INVALID),
    (dict(mscale=F(float("nan"))), pa.PA_ERR_INVALID), (dict(q=None), pa.PA_ERR_INVALID),
    (dict(vp=None), pa.PA_ERR_INVALID), (dict(slots=None), pa.PA_ERR_INVALID), (dict(v=None), pa.PA_ERR_INVALID),
    (dict(k_out=None, v=None, kp=None, vp=None, slots=None), pa.PA_ERR_INVALID), (dict(q=ODD), pa.PA_ERR_INVALID),
    (dict(inv=ctypes.c_void_p(260)), pa.PA_ERR_INVALID), (dict(qs=1028), pa.PA_ERR_INVALID),
    (dict(qs=1016), pa.PA_ERR_INVALID), (dict(ks=248), pa.PA_ERR_INVALID), (dict(vs=260), pa.PA_ERR_INVALID),
    (dict(qs=2048), pa.PA_ERR_INVALID)])  # the last: q_out is q, which is not contiguous
def test_rope_and_cache_refuses(kw, status):
    assert rope(**kw) == status
    assert pa.lib().pa_last_error() != b""


def test_rope_and_cache_of_nothing_is_fine():
    assert rope(tokens=0, q=None) == pa.PA_OK


def prefill(**kw):
    a = dict(out=P, q=P, k=P, v=P, cu=P, seqs=2, tokens=64, heads=8, kv=2, D=128, qs=1024, ks=256, vs=256,
             scale=F(0.1), dtype=0)
    a.update(kw)
    return pa.lib().pa_prefill(*a.values(), None)


def paged(**kw):
    a = dict(out=P, q=P, kp=P, vp=P, tables=P, ctx=P, cu=P, seqs=2, tokens=64, heads=8, kv=2, D=128, bs=16, width=8,
             blocks=32, max_ctx=128, qs=1024, scale=F(0.1), dtype=0, ws=P, bytes=1 << 40)
    a.update(kw)
    return pa.lib().pa_prefill_paged(*a.values(), None)


COMMON = [
    (dict(seqs=-1), pa.PA_ERR_INVALID), (dict(tokens=-1), pa.PA_ERR_INVALID), (dict(dtype=2), pa.PA_ERR_INVALID),
    (dict(heads=0), pa.PA_ERR_UNSUPPORTED), (dict(heads=6), pa.PA_ERR_UNSUPPORTED),
    (dict(heads=7), pa.PA_ERR_UNSUPPORTED), (dict(heads=32), pa.PA_ERR_UNSUPPORTED), (dict(D=96), pa.PA_ERR_UNSUPPORTED),
    (dict(tokens=1 << 27), pa.PA_ERR_UNSUPPORTED), (dict(scale=F(float("nan"))), pa.PA_ERR_INVALID),
    (dict(scale=F(float("inf"))), pa.PA_ERR_INVALID), (dict(out=None), pa.PA_ERR_INVALID),
    (dict(cu=None), pa.PA_ERR_INVALID), (dict(q=ODD), pa.PA_ERR_INVALID), (dict(cu=ODD), pa.PA_ERR_INVALID),
    (dict(qs=1020), pa.PA_ERR_INVALID), (dict(qs=1016), pa.PA_ERR_INVALID)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(k=None), pa.PA_ERR_INVALID), (dict(ks=248), pa.PA_ERR_INVALID), (dict(vs=257), pa.PA_ERR_INVALID)])
def test_prefill_refuses(kw, status):
    assert prefill(**kw) == status
    assert pa.lib().pa_last_error() != b""


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(bs=48), pa.PA_ERR_UNSUPPORTED), (dict(width=0), pa.PA_ERR_INVALID), (dict(blocks=0), pa.PA_ERR_INVALID),
    (dict(max_ctx=-1), pa.PA_ERR_INVALID), (dict(kp=None), pa.PA_ERR_INVALID), (dict(ws=None), pa.PA_ERR_INVALID),
    (dict(tables=ODD), pa.PA_ERR_INVALID), (dict(ws=ctypes.c_void_p(128)), pa.PA_ERR_INVALID),
    (dict(bytes=0), pa.PA_ERR_INVALID)])
def test_prefill_paged_refuses(kw, status):
    assert paged(**kw) == status
    assert pa.lib().pa_last_error() != b""


def test_empty_calls_are_fine():
    assert prefill(seqs=0, q=None) == pa.PA_OK
    assert prefill(tokens=0, q=None) == pa.PA_OK
    assert paged(seqs=0, q=None) == pa.PA_OK
    assert paged(tokens=0, q=None) == pa.PA_OK


def test_workspace_size():
    assert pa.lib().pa_prefill_paged_workspace_size(4, 64, 8, 2, 96, 16, 128) == 0
    assert pa.lib().pa_prefill_paged_workspace_size(4, 64, 6, 2, 128, 16, 128) == 0
    assert pa.lib().pa_prefill_paged_workspace_size(-1, 64, 8, 2, 128, 16, 128) == 0
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_prefill_paged_workspace_size(4, 64, 8, 2, 128, 24, 128)


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    i32, i64, f16 = torch.int32, torch.int64, torch.float16
    q, k = torch.zeros(4, 8, 64, dtype=f16), torch.zeros(4, 2, 64, dtype=f16)
    pool = torch.zeros(3, 2, 16, 64, dtype=f16)
    cu, ctx, tab = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 4, dtype=i32)
    with pytest.raises(ValueError):
        pa.pa_prefill(torch.empty_like(q), q, k, k, cu, 0.1)
    with pytest.raises(ValueError):
        pa.pa_prefill_paged(torch.empty_like(q), q, pool, pool, tab, ctx, cu, 0.1, 64)
    with pytest.raises(ValueError):
        pa.pa_rope_and_cache(torch.empty_like(q), q, k, k, pool, pool, torch.zeros(4, dtype=i32),
                             torch.zeros(4, dtype=i64), torch.ones(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        pa.pa_rope_and_cache(torch.empty_like(q), q, k, None, pool, pool, torch.zeros(4, dtype=i32),
                             torch.zeros(4, dtype=i64), torch.ones(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        pa.pa_assign_slots(tab, torch.zeros(3, dtype=i32), ctx, torch.zeros(1, dtype=i32), ctx, 16,
                           torch.zeros(4, dtype=i64), torch.zeros(4, dtype=i32), cu)


def test_binding_refuses_numbers_past_32_bits():
    # a view of every second token of a very wide buffer: no memory behind it here
    def rows(step):
        x = torch.empty_strided((2, 8, 64), (step, 64, 1), dtype=torch.float16, device="meta")
        return pa._rows(x, "q", x.shape, torch.float16, x.get_device())

    assert rows((1 << 31) - 8) == (1 << 31) - 8
    for step in (1 << 31, (1 << 32) + 512):
        with pytest.raises(ValueError, match="apart"):
            rows(step)
    with pytest.raises(ValueError, match="max_context_len"):
        pa.pa_prefill_paged_workspace_size(4, 64, 8, 2, 128, 16, (1 << 32) + 128)
    for n in (1 << 30, (1 << 31) - 1):
        assert paged(max_ctx=n) == pa.PA_ERR_UNSUPPORTED
