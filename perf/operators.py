"""What is measured of the prompt path: the operators a serving step runs before and around paged decode.

  assign   pa_assign_slots     block tables, slots and positions of a batch from request lengths
  rope     pa_rope_and_cache   rotary positions of q and k, rotated k and v written to the paged cache
  prefill  pa_prefill          causal attention over whole prompts, packed one after another
  paged    pa_prefill_paged    the same for the last tokens of each context over the paged cache

Each has its plain form (elementary torch operations in 32 bits, 64 for the
angles) and the library's call, chosen by the module's name ``own``.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---- cases ------------------------------------------------------------------------------------------

def listed():
    return [
        # One token appended to each of 256 running requests: what every decode step of the
        # Llama-3-8B-shaped batch does before its attention. The smallest call, latency only.
        dict(name="assign_decode_256", op="assign", seqs=256, block_size=16, lo=16, hi=8192, dist="lognormal",
             new="one", release=0, lens_seed=11),
        # 192 prompts arrive while 64 requests end: the largest map, hundreds of thousands of slots.
        dict(name="assign_prompts_256", op="assign", seqs=256, block_size=16, lo=16, hi=8192, dist="lognormal",
             new="prompt", release=64, lens_seed=12),
        # The rotation and cache write of a decode step: 256 tokens, grouped heads, far positions,
        # q, k and v as views of one fused projection.
        dict(name="rope_decode_256", op="rope", tokens=256, heads=32, kv_heads=8, head_dim=128, rot_dim=128,
             interleaved=False, block_size=16, dtype="bf16", fused=True, max_pos=1 << 20, mscale=1.0, k_out=False),
        # A step of prompts: 8192 tokens, one query head per KV head, half of each head rotated,
        # adjacent pairs, and an attention factor as long-context scalings have it.
        dict(name="rope_prompt_8192", op="rope", tokens=8192, heads=32, kv_heads=32, head_dim=128, rot_dim=64,
             interleaved=True, block_size=16, dtype="f16", fused=False, max_pos=8192, mscale=1.125, k_out=True),
        # An odd number of tokens at head size 64, as a ragged prompt step gives it.
        dict(name="rope_prompt_2049_d64", op="rope", tokens=2049, heads=16, kv_heads=4, head_dim=64, rot_dim=64,
             interleaved=False, block_size=32, dtype="bf16", fused=True, max_pos=32768, mscale=1.0, k_out=True),
        # The four short prompts of the tiny batch: contexts 1, 7, 16 and 33.
        dict(name="prefill_tiny", op="prefill", lens="1,7,16,33", heads=2, kv_heads=2, head_dim=64, dtype="f16",
             fused=False),
        # Prompts of the LLaMA-7B-shaped batch: one query head per KV head, 128 to 2048 tokens.
        dict(name="prefill_llama7b", op="prefill", seqs=12, lo=128, hi=2048, dist="uniform", lens_seed=21, heads=32,
             kv_heads=32, head_dim=128, dtype="f16", fused=False),
        # Prompts of the Llama-3-8B-shaped batch: ragged, mostly short, a few long, four heads a group.
        dict(name="prefill_llama3_8b", op="prefill", seqs=32, lo=16, hi=8192, dist="lognormal", lens_seed=22,
             heads=32, kv_heads=8, head_dim=128, dtype="bf16", fused=True),
        # One long document, the largest call.
        dict(name="prefill_one_16384", op="prefill", lens="16384", heads=32, kv_heads=8, head_dim=128, dtype="bf16",
             fused=False),
        # Five to eight tokens a request checked at once over long contexts: few rows, much cache.
        dict(name="paged_verify_8", op="paged", seqs=8, lo=4096, hi=32768, dist="uniform", lens_seed=31,
             chunk_lo=5, chunk_hi=8, shared=0, heads=32, kv_heads=8, head_dim=128, block_size=16, dtype="bf16"),
        # Requests that share a 1024-token prefix, each with its own suffix to compute (the beam batch's sizes).
        dict(name="paged_suffix_64", op="paged", seqs=64, lo=16, hi=512, dist="uniform", lens_seed=32,
             chunk_lo=0, chunk_hi=0, shared=1024, heads=32, kv_heads=8, head_dim=128, block_size=16, dtype="bf16"),
        # 512-token pieces of eight 32768-token prompts: the 4096 prompt tokens of the long32k step, computed.
        dict(name="paged_chunk_long32k", op="paged", seqs=8, lo=32768, hi=32768, dist="uniform", lens_seed=33,
             chunk_lo=512, chunk_hi=512, shared=0, heads=32, kv_heads=8, head_dim=128, block_size=64, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["assign", "rope", "prefill", "prefill", "paged", "paged"])
    heads, kv_heads = rng.choice([(2, 2), (8, 1), (16, 2), (32, 4), (32, 8), (32, 16), (32, 32)])
    head_dim = rng.choice([64, 128])
    dtype = rng.choice(["f16", "bf16"])
    block_size = rng.choice([16, 32, 64])
    seed = rng.randrange(1 << 30)
    if op == "assign":
        seqs = _spread(rng, 1, 1024)
        return dict(op=op, seqs=seqs, block_size=block_size, lo=1, hi=_spread(rng, 16, 8192), dist="lognormal",
                    new=rng.choice(["one", "prompt"]), release=rng.randint(0, seqs // 2), lens_seed=seed)
    if op == "rope":
        return dict(op=op, tokens=_spread(rng, 1, 8192), heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                    rot_dim=rng.choice([x for x in (16, 32, 48, 64, 96, 128) if x <= head_dim]),
                    interleaved=rng.random() < 0.5, block_size=block_size, dtype=dtype, fused=rng.random() < 0.5,
                    max_pos=_spread(rng, 64, 1 << 20), mscale=rng.choice([1.0, 1.125]), k_out=rng.random() < 0.5)
    if op == "prefill":
        seqs = _spread(rng, 1, 48)
        hi = _spread(rng, 1, 16384 if seqs <= 2 else 8192 if seqs <= 6 else 2048)
        return dict(op=op, seqs=seqs, lo=1, hi=hi, dist="uniform", lens_seed=seed, heads=heads, kv_heads=kv_heads,
                    head_dim=head_dim, dtype=dtype, fused=rng.random() < 0.5)
    seqs = _spread(rng, 1, 32)
    hi = _spread(rng, 16, 32768 if seqs <= 8 else 4096)
    return dict(op=op, seqs=seqs, lo=1, hi=hi, dist="uniform", lens_seed=seed, chunk_lo=1,
                chunk_hi=_spread(rng, 1, 512), shared=0, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                block_size=block_size, dtype=dtype)


def _lens(case):
    """The request lengths a case names (the same for every seed)."""
    if case.get("lens"):
        return [int(x) for x in case["lens"].split(",")]
    rng = random.Random(case["lens_seed"])
    lo, hi, n = case["lo"], case["hi"], case["seqs"]
    if case["dist"] == "uniform":
        return [rng.randint(lo, hi) for _ in range(n)]
    return [max(lo, min(hi, round(math.exp(rng.gauss(math.log(512.0), 1.0))))) for _ in range(n)]


def _paged_lens(case):
    """(context lengths, new tokens of each) of a paged case."""
    lens = _lens(case)
    if case["shared"]:
        return [case["shared"] + n for n in lens], lens
    rng = random.Random(case["lens_seed"] + 1)
    return lens, [min(n, rng.randint(case["chunk_lo"], case["chunk_hi"])) for n in lens]


def _assign_lens(case):
    """(context lengths, new lengths: -1 releases the request)."""
    lens = _lens(case)
    rng = random.Random(case["lens_seed"] + 1)
    gone = set(rng.sample(range(len(lens)), case["release"]))
    if case["new"] == "one":
        return lens, [-1 if s in gone else 1 for s in range(len(lens))]
    # Prompts come to empty rows; the requests that end hold a context.
    ctx = [n if s in gone else 0 for s, n in enumerate(lens)]
    return ctx, [-1 if s in gone else n for s, n in enumerate(lens)]


# ---- inputs -----------------------------------------------------------------------------------------

def _normal(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _qkv(tokens, heads, kv_heads, head_dim, dtype, fused, gen):
    """q, k, v: tensors of their own, or views of one fused projection's output."""
    if not fused:
        return tuple(_normal((tokens, h, head_dim), dtype, gen) for h in (heads, kv_heads, kv_heads))
    x = _normal((tokens, heads + 2 * kv_heads, head_dim), dtype, gen)
    return x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]


def _int(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _cdiv(a, b):
    return -(-a // b)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op == "assign":
        return _prepare_assign(case, gen)
    dtype, D, H, Hkv = DTYPES[case["dtype"]], case["head_dim"], case["heads"], case["kv_heads"]
    if op == "rope":
        T, bs = case["tokens"], case["block_size"]
        q, k, v = _qkv(T, H, Hkv, D, dtype, case["fused"], gen)
        nb = _cdiv(T, bs) + 4
        slots = torch.randperm(nb * bs, generator=gen, device="cuda")[:T].contiguous()
        half = case["rot_dim"] // 2
        inv_freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        st = dict(case=case, q=q, k=k, v=v, slots=slots, inv_freq=inv_freq,
                  positions=torch.randint(0, case["max_pos"], (T,), generator=gen, device="cuda", dtype=torch.int32),
                  k_pool=_normal((nb, Hkv, bs, D), dtype, gen), v_pool=_normal((nb, Hkv, bs, D), dtype, gen),
                  q_out=torch.empty((T, H, D), dtype=dtype, device="cuda"),
                  k_out=torch.empty((T, Hkv, D), dtype=dtype, device="cuda") if case["k_out"] else None)
        return st
    scale = 1.0 / math.sqrt(D)
    if op == "prefill":
        lens = _lens(case)
        T = sum(lens)
        q, k, v = _qkv(T, H, Hkv, D, dtype, case["fused"], gen)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        return dict(case=case, q=q, k=k, v=v, cu=_int(cu), lens=lens, scale=scale,
                    out=torch.empty((T, H, D), dtype=dtype, device="cuda"))
    ctx, new = _paged_lens(case)
    bs = case["block_size"]
    pre = case["shared"] // bs
    need = pre + sum(_cdiv(n, bs) - pre for n in ctx)
    nb = need + need // 4 + 1
    ids = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(ctx), max(_cdiv(n, bs) for n in ctx)), -1, dtype=torch.int32, device="cuda")
    at = pre
    for s, n in enumerate(ctx):
        w = _cdiv(n, bs)
        table[s, :pre] = ids[:pre]
        table[s, pre:w] = ids[at:at + w - pre]
        at += w - pre
    T = sum(new)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st = dict(case=case, q=_normal((T, H, D), dtype, gen), k_pool=_normal((nb, Hkv, bs, D), dtype, gen),
              v_pool=_normal((nb, Hkv, bs, D), dtype, gen), table=table, ctx=_int(ctx), cu=_int(cu), ctx_list=ctx,
              new_list=new, scale=scale, out=torch.empty((T, H, D), dtype=dtype, device="cuda"))
    if own:
        import paged_kv_cache_372_b200 as pa
        st["workspace"] = pa.alloc_prefill_workspace(len(ctx), T, H, Hkv, D, bs, max(ctx))
    return st


def _prepare_assign(case, gen):
    ctx, new = _assign_lens(case)
    bs = case["block_size"]
    held = [_cdiv(n, bs) for n in ctx]
    after = [_cdiv(c + max(n, 0), bs) for c, n in zip(ctx, new)]
    nb = sum(held) + sum(a - h for a, h in zip(after, held)) + 64
    width = max(max(after), 1)
    ids = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(ctx), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(held):
        table[s, :n] = ids[at:at + n]
        at += n
    free = torch.full((nb,), -1, dtype=torch.int32, device="cuda")
    free[:nb - at] = ids[at:]
    T = sum(max(n, 0) for n in new)
    # A padded batch: a few rows more than the tokens it holds.
    rows = max(_cdiv(T, 64) * 64, 64)
    dev = dict(device="cuda")
    return dict(case=case, table=table, free=free, ctx=_int(ctx), new=_int(new), num_free=_int([nb - at]),
                ctx_out=torch.empty(len(ctx), dtype=torch.int32, **dev),
                num_free_out=torch.empty(1, dtype=torch.int32, **dev),
                slots=torch.empty(rows, dtype=torch.int64, **dev),
                positions=torch.empty(rows, dtype=torch.int32, **dev),
                cu=torch.empty(len(ctx) + 1, dtype=torch.int32, **dev))


# ---- one pass ---------------------------------------------------------------------------------------

def run(state):
    return {"assign": _run_assign, "rope": _run_rope, "prefill": _run_prefill,
            "paged": _run_paged}[state["case"]["op"]](state)


def _run_assign(st):
    bs = st["case"]["block_size"]
    if own:
        import paged_kv_cache_372_b200 as pa
        pa.pa_assign_slots(st["table"], st["free"], st["ctx"], st["num_free"], st["new"], bs, st["slots"],
                           st["positions"], st["cu"], st["ctx_out"], st["num_free_out"])
        return [st["table"], st["free"], st["ctx_out"], st["num_free_out"], st["slots"], st["positions"], st["cu"]]
    table, free, ctx, new = st["table"], st["free"], st["ctx"].long(), st["new"].long()
    B, W = table.shape
    rows = st["slots"].numel()
    gone = new < 0
    add = torch.where(gone, 0, new)
    held = (ctx + bs - 1) // bs
    cols = torch.arange(W, device=table.device)
    nf = st["num_free"].long()
    # Released blocks go on top of the free list, in request and then table order.
    back = table[(gone[:, None] & (cols < held[:, None]))].int()
    at = torch.arange(free.numel(), device=table.device)
    top = nf + back.numel()
    stack = torch.where((at >= nf) & (at < top), torch.cat([back, back.new_zeros(1)])[(at - nf).clamp(0, back.numel())],
                        free)
    # New blocks come off its end, in request and then table order.
    need = torch.where(gone, 0, (ctx + add + bs - 1) // bs - held)
    fresh = (~gone[:, None]) & (cols >= held[:, None]) & (cols < (held + need)[:, None])
    taken = int(need.sum())
    table[fresh] = stack[top - 1 - torch.arange(taken, device=table.device)]
    left = top - taken
    free.copy_(torch.where((at >= nf) & (at < left), stack, free))
    cu = torch.cat([add.new_zeros(1), torch.cumsum(add, 0)])
    tok = torch.arange(rows, device=table.device)
    live = tok < cu[-1]
    seq = (torch.searchsorted(cu, tok, right=True) - 1).clamp(0, B - 1)
    pos = torch.where(live, ctx[seq] + tok - cu[seq], 0)
    slot = table[seq, pos // bs].long() * bs + pos % bs
    return [table, free, torch.where(gone, 0, ctx + add).int(), left.int(), torch.where(live, slot, -1),
            torch.where(live, pos, -1).int(), cu.int()]


def _rotate(x, cos, sin, rot, interleaved):
    """x [T][h][D] in 32 bits, its first rot elements of each head turned by the token's angles."""
    a, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        e, o = a[..., 0::2], a[..., 1::2]
        turned = torch.stack([e * cos - o * sin, o * cos + e * sin], dim=-1).flatten(-2)
    else:
        e, o = a[..., :rot // 2], a[..., rot // 2:]
        turned = torch.cat([e * cos - o * sin, o * cos + e * sin], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _run_rope(st):
    case = st["case"]
    if own:
        import paged_kv_cache_372_b200 as pa
        pa.pa_rope_and_cache(st["q_out"], st["q"], st["k"], st["v"], st["k_pool"], st["v_pool"], st["positions"],
                             st["slots"], st["inv_freq"], mscale=case["mscale"], interleaved=case["interleaved"],
                             k_out=st["k_out"])
        return [st["q_out"], st["k_pool"], st["v_pool"]] + ([st["k_out"]] if case["k_out"] else [])
    rot, bs, dtype = case["rot_dim"], case["block_size"], st["q"].dtype
    angle = st["positions"].double()[:, None] * st["inv_freq"]
    cos = (torch.cos(angle) * case["mscale"]).float()[:, None, :]
    sin = (torch.sin(angle) * case["mscale"]).float()[:, None, :]
    q = _rotate(st["q"].float(), cos, sin, rot, case["interleaved"]).to(dtype)
    k = _rotate(st["k"].float(), cos, sin, rot, case["interleaved"]).to(dtype)
    blk, off = st["slots"] // bs, st["slots"] % bs
    st["k_pool"][blk, :, off] = k
    st["v_pool"][blk, :, off] = st["v"]
    return [q, st["k_pool"], st["v_pool"]] + ([k] if case["k_out"] else [])


def _attend(q, k, v, scale, first):
    """q [n][H][D], k and v [m][Hkv][D]; row i sees the keys up to first + i. In 32 bits, by groups of heads and rows
    that keep the scores at a few GB."""
    n, H, D = q.shape
    m, Hkv, _ = k.shape
    group = H // Hkv
    out = torch.empty_like(q)
    kv_step = max(1, min(Hkv, (1 << 28) // max(1, group * n * m)))
    row_step = max(1, min(n, (1 << 28) // max(1, group * m * kv_step)))
    for h in range(0, Hkv, kv_step):
        e = min(h + kv_step, Hkv)
        kk = k[:, h:e].float().permute(1, 2, 0)                     # [heads][D][m]
        vv = v[:, h:e].float().permute(1, 0, 2)                     # [heads][m][D]
        for r in range(0, n, row_step):
            t = min(r + row_step, n)
            seen = min(m, first + t)
            qq = q[r:t, h * group:e * group].float().permute(1, 0, 2).reshape(e - h, group * (t - r), D)
            s = (qq @ kk[:, :, :seen] * scale).view(e - h, group, t - r, seen)
            hidden = torch.arange(seen, device=q.device) > first + torch.arange(r, t, device=q.device)[:, None]
            s = s.masked_fill(hidden, float("-inf"))
            p = torch.exp(s - s.max(dim=-1, keepdim=True).values)
            p = (p / p.sum(dim=-1, keepdim=True)).view(e - h, group * (t - r), seen)
            o = (p @ vv[:, :seen]).view(e - h, group, t - r, D).permute(2, 0, 1, 3)
            out[r:t, h * group:e * group] = o.reshape(t - r, (e - h) * group, D).to(q.dtype)
    return out


def _run_prefill(st):
    if own:
        import paged_kv_cache_372_b200 as pa
        return pa.pa_prefill(st["out"], st["q"], st["k"], st["v"], st["cu"], st["scale"])
    at = 0
    for n in st["lens"]:
        rows = slice(at, at + n)
        st["out"][rows] = _attend(st["q"][rows], st["k"][rows], st["v"][rows], st["scale"], 0)
        at += n
    return st["out"]


def _run_paged(st):
    if own:
        import paged_kv_cache_372_b200 as pa
        return pa.pa_prefill_paged(st["out"], st["q"], st["k_pool"], st["v_pool"], st["table"], st["ctx"], st["cu"],
                                   st["scale"], max(st["ctx_list"]), workspace=st["workspace"])
    at, bs = 0, st["case"]["block_size"]
    for s, (c, n) in enumerate(zip(st["ctx_list"], st["new_list"])):
        ids = st["table"][s, :_cdiv(c, bs)].long()
        k = st["k_pool"][ids].transpose(1, 2).flatten(0, 1)[:c]
        v = st["v_pool"][ids].transpose(1, 2).flatten(0, 1)[:c]
        st["out"][at:at + n] = _attend(st["q"][at:at + n], k, v, st["scale"], c - n)
        at += n
    return st["out"]


# ---- the work a pass cannot do without --------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "assign":
        ctx, new = _assign_lens(case)
        bs = case["block_size"]
        T = sum(max(n, 0) for n in new)
        fresh = sum(_cdiv(c + n, bs) - _cdiv(c, bs) for c, n in zip(ctx, new) if n > 0)
        tails = sum(1 for c, n in zip(ctx, new) if n > 0 and c % bs)
        back = sum(_cdiv(c, bs) for c, n in zip(ctx, new) if n < 0)
        rows = max(_cdiv(T, 64) * 64, 64)
        B = len(ctx)
        # lengths in and out, boundaries, slots and positions, blocks taken (read, written) and given back
        return {"bytes": 16 * B + 12 + 12 * rows + 8 * fresh + 4 * tails + 8 * max(back - fresh, 0), "flops": 0}
    D, H, Hkv = case["head_dim"], case["heads"], case["kv_heads"]
    if op == "rope":
        T = case["tokens"]
        rows = T * (H + 2 * Hkv) * D * 2
        k_out = T * Hkv * D * 2 if case["k_out"] else 0
        return {"bytes": 2 * rows + k_out + 12 * T + 4 * case["rot_dim"],
                "flops": 3 * T * (H + Hkv) * case["rot_dim"]}
    if op == "prefill":
        lens = _lens(case)
        T = sum(lens)
        return {"bytes": 2 * D * T * (2 * H + 2 * Hkv) + 4 * (len(lens) + 1),
                "flops": 4 * D * H * sum(n * (n + 1) // 2 for n in lens)}
    ctx, new = _paged_lens(case)
    bs, T = case["block_size"], sum(new)
    pre = case["shared"] // bs * bs
    keys = pre + sum(c - pre for c in ctx)
    tables = sum(_cdiv(c, bs) for c in ctx)
    return {"bytes": 2 * D * (2 * H * T + 2 * Hkv * keys) + 4 * tables + 8 * len(ctx) + 4,
            "flops": 4 * D * H * sum(n * (c - n) + n * (n + 1) // 2 for c, n in zip(ctx, new))}


# ---- the definition in 64 bits ----------------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "assign":
        return None                      # whole numbers, equal or wrong
    st = prepare(case, seed)
    if op == "rope":
        return _exact_rope(case, st)
    H, Hkv, D = case["heads"], case["kv_heads"], case["head_dim"]
    out = torch.empty((st["q"].shape[0], H, D), dtype=torch.float64, device="cuda")
    ends = st["cu"].tolist()
    for s in range(len(ends) - 1):
        lo, hi = ends[s], ends[s + 1]
        if op == "prefill":
            total = hi - lo
        else:
            total, bs = case_ctx(st, s), case["block_size"]
            where = torch.arange(total, device="cuda")
            blk = st["table"][s].long()[where // bs]
        for g in range(Hkv):
            if op == "prefill":
                keys, vals = st["k"][lo:hi, g].double(), st["v"][lo:hi, g].double()
            else:
                keys = st["k_pool"][blk, g, where % bs].double()
                vals = st["v_pool"][blk, g, where % bs].double()
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                for a in range(lo, hi, 4096):
                    b = min(a + 4096, hi)
                    last = torch.arange(a, b, device="cuda") - hi + total     # position of each query
                    z = torch.einsum("id,jd->ij", st["q"][a:b, h].double(), keys).mul_(st["scale"])
                    z[torch.arange(total, device="cuda")[None, :] > last[:, None]] = -math.inf
                    z.sub_(z.amax(1, keepdim=True)).exp_()
                    out[a:b, h] = torch.einsum("ij,jd->id", z, vals) / z.sum(1, keepdim=True)
    return out


def case_ctx(st, s):
    return st["ctx_list"][s]


def _exact_rope(case, st):
    rot, bs, m = case["rot_dim"], case["block_size"], case["mscale"]
    half = rot // 2
    # Pair i turns elements (2i, 2i + 1) or (i, i + rot / 2) as one complex number.
    i = torch.arange(half, device="cuda")
    a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    phase = torch.polar(torch.full((st["q"].shape[0], 1, half), float(m), dtype=torch.float64, device="cuda"),
                        (st["positions"].double()[:, None] * st["inv_freq"][None, :])[:, None, :])

    def turn(x):
        y = x.double().clone()
        z = torch.complex(y[..., a], y[..., b]) * phase
        y[..., a], y[..., b] = z.real, z.imag
        return y

    q, k = turn(st["q"]), turn(st["k"])
    k_pool, v_pool = st["k_pool"].double(), st["v_pool"].double()
    for pool, x in ((k_pool, k), (v_pool, st["v"].double())):
        rows = pool.transpose(1, 2)                                   # [block][offset][head][D]
        rows[st["slots"].div(bs, rounding_mode="floor"), st["slots"].remainder(bs)] = x
    return [q, k_pool, v_pool] + ([k] if case["k_out"] else [])
