"""The serving step of a model that mixes gated delta-rule layers with softmax layers: what one
step of a batch of requests runs through, as cases that can be timed and checked.

Operators (``op`` of a case):
  plan    block tables, slot maps and packed offsets of a batch, from the requests' lengths
  append  new K and V rows written into a paged cache of 8-bit values (e4m3), one power-of-two
          scale for each block of tokens and head
  attn    softmax attention of each request's newest tokens over that cache
  slots   the gated delta rule's recurrence over a pool of states, one slot per request

``run`` computes a case in its plain form (elementary torch operations), or, where ``own`` is
true, through this package's entry points.
"""
import math
import random

import torch

own = False
DEV = "cuda"
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
SCALE_EXP_MIN = -100      # exponent of the smallest scale of a block


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's plan: 256 requests, most bring one token, some wait, some have finished
        dict(name="plan_decode_N256", op="plan", N=256, kind="decode", lo=1, hi=16384, bs=64, T=256),
        # the plan of a mixed step: 24 prompts share a budget of 32768 tokens
        dict(name="plan_prefill_N24_T32768", op="plan", N=24, kind="prefill", lo=64, hi=4096, bs=16, T=32768),
        # a decode step's new rows: 256 requests, 8 KV heads, blocks of 64 tokens
        dict(name="append_decode_N256_d128", op="append", N=256, Hkv=8, d=128, bs=64, ctx_hi=2048, new_lo=1, new_hi=1,
             dtype="bf16"),
        # prompts of 24 requests written at once, one layer of 16 KV heads
        dict(name="append_prefill_N24_d128", op="append", N=24, Hkv=16, d=128, bs=64, ctx_hi=500, new_lo=157,
             new_hi=4096, dtype="bf16"),
        # ragged chunks on small blocks, fp32 rows, head size 64
        dict(name="append_ragged_f32_d64", op="append", N=9, Hkv=2, d=64, bs=16, ctx_hi=300, new_lo=1, new_hi=301,
             dtype="f32"),
        # one request early in its answer: latency
        dict(name="attn_one_L700_d64", op="attn", N=1, Hq=8, Hkv=2, d=64, bs=16, kv_lo=700, kv_hi=700, q_lo=1, q_hi=1,
             window=0, dtype="bf16", out="bf16"),
        # an ordinary decode batch of ragged contexts, four query heads to a KV head
        dict(name="attn_decode_N64_d128", op="attn", N=64, Hq=32, Hkv=8, d=128, bs=64, kv_lo=128, kv_hi=16384, q_lo=1,
             q_hi=1, window=0, dtype="bf16", out="bf16"),
        # few requests with long contexts, eight query heads to a KV head, fp32 answers
        dict(name="attn_long_N4_L65536_d128", op="attn", N=4, Hq=32, Hkv=4, d=128, bs=64, kv_lo=65530, kv_hi=65536,
             q_lo=1, q_hi=1, window=0, dtype="bf16", out="f32"),
        # a few drafted tokens to check for each request, within a window, all in fp32
        dict(name="attn_draft_window_f32_d64", op="attn", N=32, Hq=16, Hkv=4, d=64, bs=32, kv_lo=1, kv_hi=8192, q_lo=1,
             q_hi=5, window=4096, dtype="f32", out="f32"),
        # a chunk of each prompt over what the cache holds already
        dict(name="attn_prefill_N4_d128", op="attn", N=4, Hq=32, Hkv=8, d=128, bs=64, kv_lo=2048, kv_hi=6000, q_lo=1000,
             q_hi=2048, window=0, dtype="bf16", out="bf16"),
        # the delta-rule layer of the decode step: 256 requests, 32 heads
        dict(name="slots_decode_N256_H32_d128", op="slots", N=256, Hk=32, Hv=32, dk=128, dv=128, q_lo=1, q_hi=1,
             dtype="bf16", out="f32"),
        # drafted tokens through the same states; two value heads share a key head, some rows are padding
        dict(name="slots_draft_N48_Hk8_Hv16_d64", op="slots", N=48, Hk=8, Hv=16, dk=64, dv=128, q_lo=0, q_hi=6,
             dtype="f32", out="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attn", "attn", "attn", "slots", "slots"])
    if op == "plan":
        kind = rng.choice(["decode", "prefill"])
        n = _log_int(rng, 1, 512) if kind == "decode" else _log_int(rng, 1, 40)
        hi = _log_int(rng, 2, 16384) if kind == "decode" else _log_int(rng, 64, 4096)
        case = dict(op=op, N=n, kind=kind, lo=1, hi=hi, bs=rng.choice([16, 32, 64, 128]))
        case["T"] = _plan_tokens(case) + rng.choice([0, 1, 37])
        return case
    if op == "append":
        dtype = rng.choice(["bf16", "f32"])
        if rng.random() < 0.5:
            n, nlo, nhi = _log_int(rng, 1, 256), 1, rng.choice([1, 1, 2, 7])
        else:
            n, nhi = _log_int(rng, 1, 20), _log_int(rng, 8, 2500)
            nlo = _log_int(rng, 1, nhi)
        return dict(op=op, N=n, Hkv=rng.choice([1, 2, 4, 8, 16]), d=rng.choice([64, 128]),
                    bs=rng.choice([16, 32, 64, 128]), ctx_hi=_log_int(rng, 1, 2000), new_lo=nlo, new_hi=nhi, dtype=dtype)
    if op == "attn":
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 2, 3, 4, 7, 8, 16])
        if rng.random() < 0.7:      # decode or drafted tokens
            n = _log_int(rng, 1, 128)
            hi = _log_int(rng, 1, max(1, min(32768, 700000 // (n * hkv))))
            qlo, qhi = 1, rng.choice([1, 1, 1, 2, 6])
            lo = _log_int(rng, 1, hi)
        else:                       # a chunk of a prompt
            n, g = rng.choice([1, 2, 3]), rng.choice([1, 2, 4])
            hi = _log_int(rng, 40, 5000)
            qhi = _log_int(rng, 17, min(hi, 1500))
            qlo, lo = _log_int(rng, 1, qhi), qhi
        lo = max(lo, min(hi, qhi))
        hi = max(hi, lo)
        return dict(op=op, N=n, Hq=hkv * g, Hkv=hkv, d=rng.choice([64, 128]), bs=rng.choice([16, 32, 64, 128]), kv_lo=lo,
                    kv_hi=hi, q_lo=qlo, q_hi=min(qhi, lo), window=rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
    hk = rng.choice([1, 2, 4, 8, 16])
    hv = hk * rng.choice([1, 2, 3])
    return dict(op=op, N=_log_int(rng, 1, min(200, 8000 // hv)), Hk=hk, Hv=hv, dk=rng.choice([64, 128]),
                dv=rng.choice([64, 128]), q_lo=rng.choice([0, 1]), q_hi=rng.choice([1, 1, 2, 5, 8]),
                dtype=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]))


# ---------------------------------------------------------------- lengths (of the case alone)
def _spread(n, lo, hi, salt):
    """n lengths spread log-uniformly over lo .. hi, both ends among them."""
    r = random.Random(salt * 7919 + n)
    a = max(lo, 1)
    xs = [lo if lo == 0 and r.random() < 0.25 else _log_int(r, a, max(a, hi)) for _ in range(n)]
    if n > 1:
        xs[0] = lo
    xs[-1] = hi
    return xs


def _plan_lens(case):
    """(cached, new) tokens of each request; new = -1: the request has finished."""
    n, r = case["N"], random.Random(case["N"] + 31)
    if case["kind"] == "decode":
        ctx = _spread(n, case["lo"], case["hi"], 1)
        new = [(-1 if i % 17 == 5 else 0 if i % 11 == 7 else 1) for i in range(n)]
    else:
        ctx = [0 if r.random() < 0.6 else r.randint(1, case["hi"]) for _ in range(n)]
        new = _spread(n, case["lo"], case["hi"], 2)
    return ctx, new


def _plan_tokens(case):
    return sum(max(x, 0) for x in _plan_lens(case)[1])


def _append_lens(case):
    return _spread(case["N"], 0, case["ctx_hi"], 3), _spread(case["N"], case["new_lo"], case["new_hi"], 4)


def _attn_lens(case):
    kv = _spread(case["N"], case["kv_lo"], case["kv_hi"], 5)
    q = _spread(case["N"], case["q_lo"], case["q_hi"], 6)
    return kv, [min(a, b) for a, b in zip(q, kv)]


def _slot_lens(case):
    q = _spread(case["N"], case["q_lo"], case["q_hi"], 8)
    return q


def _gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _mixed(lists, seed):
    """The same requests in another order."""
    order = list(range(len(lists[0])))
    random.Random(seed).shuffle(order)
    return [[x[i] for i in order] for x in lists]


def _offsets(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return out


def _tables(lens, bs, gen, spare=8):
    """Block table (N, M) of requests of these lengths, blocks scattered over the pool; -1 elsewhere."""
    need = [-(-x // bs) for x in lens]
    total = sum(need)
    nb = total + spare
    perm = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32)
    m = max(1, max(need))
    cols = torch.arange(m, device=DEV)[None]
    n_t, o_t = torch.tensor(need, device=DEV)[:, None], torch.tensor(_offsets(need)[:-1], device=DEV)[:, None]
    table = torch.where(cols < n_t, perm[(o_t + cols).clamp(max=nb - 1)], torch.tensor(-1, dtype=torch.int32, device=DEV))
    return table.contiguous(), nb, perm[total:].contiguous()


def _rows(shape, gen, dtype, spread=1.0):
    """Activations with a per-(row, head) size that varies, as keys and values do."""
    x = torch.randn(*shape, generator=gen, device=DEV)
    size = torch.exp(spread * torch.randn(shape[0], shape[1], 1, generator=gen, device=DEV))
    return (x * size).to(dtype)


def _filled_cache(nb, hkv, bs, d, gen):
    """A cache in use: e4m3 values that fill their range, scales within a few powers of two."""
    def half():
        c = (torch.randn(nb, hkv, bs, d, generator=gen, device=DEV) * 100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3)
        s = torch.exp2(torch.randint(-9, -5, (nb, hkv), generator=gen, device=DEV).float())
        return c, s
    k, ks = half()
    v, vs = half()
    return k, v, ks, vs


# ---------------------------------------------------------------- prepare
def prepare(case, seed):
    from types import SimpleNamespace
    s = SimpleNamespace(case=case, op=case["op"])
    gen = _gen(seed)
    if s.op == "plan":
        s.ctx_list, s.new_list = _mixed(_plan_lens(case), seed)
        s.bs, s.T = case["bs"], case["T"]
        s.ctx, s.new = _ints(s.ctx_list), _ints(s.new_list)
        table, nb, _ = _tables(s.ctx_list, s.bs, gen, spare=0)
        more = sum(-(-(c + max(n, 0)) // s.bs) + (-c // s.bs) for c, n in zip(s.ctx_list, s.new_list))
        m = max(-(-(c + max(n, 0)) // s.bs) for c, n in zip(s.ctx_list, s.new_list)) + 3
        s.num_blocks = nb + more + 5
        s.table = torch.full((case["N"], m), -1, dtype=torch.int32, device=DEV)
        s.table[:, :table.shape[1]] = table[:, :m]
        fresh = torch.randperm(more + 5, generator=gen, device=DEV).to(torch.int32) + nb
        s.free_list = torch.full((s.num_blocks,), -1, dtype=torch.int32, device=DEV)
        s.free_list[:fresh.numel()] = fresh
        s.free_count = _ints([fresh.numel()])
    elif s.op == "append":
        ctx, new = _mixed(_append_lens(case), seed)
        s.bs, hkv, d = case["bs"], case["Hkv"], case["d"]
        table, nb, _ = _tables([a + b for a, b in zip(ctx, new)], s.bs, gen)
        s.k_cache, s.v_cache, s.k_scale, s.v_scale = _filled_cache(nb, hkv, s.bs, d, gen)
        cu, t = _offsets(new), sum(new)
        seq = torch.repeat_interleave(torch.arange(len(new), device=DEV), torch.tensor(new, device=DEV), output_size=t)
        pos = torch.tensor(ctx, device=DEV)[seq] + torch.arange(t, device=DEV) - torch.tensor(cu[:-1], device=DEV)[seq]
        s.slot_map = (table[seq, pos // s.bs].long() * s.bs + pos % s.bs).to(torch.int32)
        s.touched = sum((a + b - 1) // s.bs - a // s.bs + 1 for a, b in zip(ctx, new))
        s.k = _rows((t, hkv, d), gen, _dtype(case["dtype"]))
        s.v = _rows((t, hkv, d), gen, _dtype(case["dtype"]))
    elif s.op == "attn":
        s.kv_list, s.q_list = _mixed(_attn_lens(case), seed)
        s.bs, s.window, d = case["bs"], case["window"], case["d"]
        s.table, nb, _ = _tables(s.kv_list, s.bs, gen)
        s.k_cache, s.v_cache, s.k_scale, s.v_scale = _filled_cache(nb, case["Hkv"], s.bs, d, gen)
        t = sum(s.q_list)
        s.cu = _ints(_offsets(s.q_list))
        s.kv_lens = _ints(s.kv_list)
        s.max_q = max(s.q_list)
        s.q = torch.randn(t, case["Hq"], d, generator=gen, device=DEV).to(_dtype(case["dtype"]))
        s.scale = 1.0 / math.sqrt(d)
        s.out = _dtype(case["out"])
    else:
        s.q_list, = _mixed([_slot_lens(case)], seed)
        n, hk, hv, dk, dv = case["N"], case["Hk"], case["Hv"], case["dk"], case["dv"]
        t, dt = sum(s.q_list), _dtype(case["dtype"])
        s.cu = _ints(_offsets(s.q_list))
        s.max_q = max(s.q_list)

        def unit(*shape):
            x = torch.randn(*shape, generator=gen, device=DEV)
            return (x / x.norm(dim=-1, keepdim=True)).to(dt)
        s.q, s.k = unit(t, hk, dk), unit(t, hk, dk)
        s.v = torch.randn(t, hv, dv, generator=gen, device=DEV).to(dt)
        s.beta = torch.sigmoid(torch.randn(t, hv, generator=gen, device=DEV))
        s.g = -0.05 * torch.rand(t, hv, generator=gen, device=DEV)
        pool = n + n // 4 + 1
        s.slots = torch.randperm(pool, generator=gen, device=DEV)[:n].to(torch.int32)
        s.state = torch.randn(pool, hv, dk, dv, generator=gen, device=DEV) * 0.1
        s.scale = 1.0 / math.sqrt(dk)
        s.out = _dtype(case["out"])
    _handles(s)
    return s


def _handles(s):
    """What a program keeps from step to step: the cache's handle and the plan's buffers."""
    s.cache = s.plan = None


# ---------------------------------------------------------------- the framework's calls
def _run_own(s):
    import gated_deltanet_sequence_b200 as gdn
    if s.op == "plan":
        if s.plan is None:
            s.plan = gdn.BatchPlan.empty(s.case["N"], s.T, DEV)
        p = gdn.gdn_plan_batch(s.ctx, s.new, s.table, s.free_list, s.free_count, s.bs, s.plan)
        return dict(cu_seqlens=p.cu_seqlens, kv_lens=p.kv_lens, positions=p.positions, seq_ids=p.seq_ids,
                    slot_map=p.slot_map, info=p.info, table=s.table, free_list=s.free_list, free_count=s.free_count)
    if s.op == "slots":
        o = gdn.gdn_decode_slots(s.q, s.k, s.v, s.beta, s.g, s.state, s.slots, s.cu, scale=s.scale, out_dtype=s.out)
        return dict(o=o, state=s.state)
    if s.cache is None:
        s.cache = gdn.KvCache(s.k_cache, s.v_cache, s.k_scale, s.v_scale)
    if s.op == "append":
        gdn.gdn_kv_append(s.cache, s.k, s.v, s.slot_map)
        return dict(k=s.k_cache, v=s.v_cache, k_scale=s.k_scale, v_scale=s.v_scale)
    o, lse = gdn.gdn_kv_attn(s.cache, s.q, s.table, s.cu, s.kv_lens, max_q_len=s.max_q, window=s.window, scale=s.scale,
                             out_dtype=s.out, lse=True)
    return dict(o=o, lse=lse)


# ---------------------------------------------------------------- plain forms
def _plan_plain(s):
    ctx, new, bs = s.ctx.long(), s.new.long(), s.bs
    n, m = s.table.shape
    gone = new < 0
    add = new.clamp(min=0)
    table = s.table.long()
    # blocks of finished requests go on top of the free list, in (request, block) order
    give = (gone[:, None] & (table >= 0)).reshape(-1)
    rank = torch.cumsum(give, 0) - 1
    cap = s.free_list.numel()
    count = s.free_count.long()
    listed_ = torch.cat([s.free_list.long(), torch.zeros(1, dtype=torch.long, device=DEV)])
    listed_.scatter_(0, torch.where(give, (count + rank).clamp(max=cap), cap), table.reshape(-1))
    listed_ = listed_[:cap]
    count = count + give.sum()
    table = torch.where(gone[:, None], -1, table)
    # new blocks come off its top, in (request, block) order; all of them or none
    cols = torch.arange(m, device=DEV)[None]
    have, need = (ctx + bs - 1) // bs, (ctx + add + bs - 1) // bs
    want = ((cols >= have[:, None]) & (cols < need[:, None]) & (table < 0) & ~gone[:, None]).reshape(-1)
    rank = torch.cumsum(want, 0) - 1
    total = want.sum()
    fits = total <= count
    fresh = listed_[(count - 1 - rank).clamp(0, cap - 1)]
    table = torch.where((want & fits).view(n, m), fresh.view(n, m), table)
    short = torch.where(fits, 0, total - count)
    count = count - torch.where(fits, total, 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(add, 0)])
    t = torch.arange(s.T, device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=n - 1)
    live = t < cu[-1]
    pos = ctx[seq] + t - cu[seq]
    block = table[seq, (pos // bs).clamp(0, m - 1)]
    kv = torch.where(gone, 0, ctx + add)
    slot = torch.where(live & (block >= 0), block * bs + pos % bs, -1)
    s.table.copy_(table)
    s.free_list.copy_(listed_)
    s.free_count.copy_(count)
    info = torch.cat([cu[-1:], kv.max().reshape(1), short.reshape(1), count])
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return dict(cu_seqlens=i32(cu), kv_lens=i32(kv), positions=i32(torch.where(live, pos, -1)),
                seq_ids=i32(torch.where(live, seq, -1)), slot_map=i32(slot), info=i32(info), table=s.table,
                free_list=s.free_list, free_count=s.free_count)


def _scale_for(amax):
    """The smallest power of two 2^e, e >= SCALE_EXP_MIN, with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, SCALE_EXP_MIN).clamp(min=SCALE_EXP_MIN)
    return torch.ldexp(torch.ones_like(amax), e)


def _append_plain_one(x, slot_map, cache, scale, touched):
    nb, hkv, bs, d = cache.shape
    t = x.shape[0]
    x = x.float()
    slot = slot_map.long()
    block, off = slot // bs, slot % bs
    first = torch.ones(t, dtype=torch.bool, device=DEV)
    first[1:] = block[1:] != block[:-1]
    run_ = torch.cumsum(first, 0) - 1
    blocks = torch.zeros(touched, dtype=torch.long, device=DEV).scatter_(0, run_, block)
    start = torch.full((touched,), bs, dtype=torch.long, device=DEV).scatter_reduce_(0, run_, off, "amin")
    finite = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)                       # (t, hkv)
    amax = torch.zeros(touched, hkv, device=DEV).scatter_reduce_(0, run_[:, None].expand(t, hkv), finite, "amax")
    old_scale = scale[blocks]
    kept = start > 0
    new_scale = _scale_for(amax)
    new_scale = torch.where(kept[:, None], torch.maximum(old_scale, new_scale), new_scale)
    old = cache[blocks]
    again = (old.float() * (old_scale / new_scale)[:, :, None, None]).to(E4M3)
    rows = torch.arange(bs, device=DEV)
    before = (rows[None] < start[:, None])[:, None, :, None]
    merged = torch.where(before, again.view(torch.uint8), old.view(torch.uint8))
    codes = (x / new_scale[run_][:, :, None]).to(E4M3).view(torch.uint8)
    merged[run_, :, off] = codes
    cache.view(torch.uint8)[blocks] = merged
    scale[blocks] = new_scale


def _append_plain(s):
    _append_plain_one(s.k, s.slot_map, s.k_cache, s.k_scale, s.touched)
    _append_plain_one(s.v, s.slot_map, s.v_cache, s.v_scale, s.touched)
    return dict(k=s.k_cache, v=s.v_cache, k_scale=s.k_scale, v_scale=s.v_scale)


def _attn_plain(s):
    n, hq, hkv, d, bs = s.case["N"], s.case["Hq"], s.case["Hkv"], s.case["d"], s.bs
    g, mq, t = hq // hkv, s.max_q, s.q.shape[0]
    blocks = s.table.long().clamp(min=0)
    lkv = blocks.shape[1] * bs

    def whole(cache, scale):
        x = cache[blocks].float() * scale[blocks][..., None, None]                       # (n, m, hkv, bs, d)
        return x.permute(0, 2, 1, 3, 4).reshape(n, hkv, lkv, d)
    cu, kv = s.cu.long(), s.kv_lens.long()
    ql = cu[1:] - cu[:-1]
    j = torch.arange(mq, device=DEV)
    rows = (cu[:-1, None] + j[None]).clamp(max=t - 1)                                    # (n, mq)
    q = s.q[rows].float().view(n, mq, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * mq, d)
    at = kv[:, None] - ql[:, None] + j[None]                                             # position of each query
    pos = torch.arange(lkv, device=DEV)
    see = (pos[None, None] <= at[..., None]) & (pos[None, None] < kv[:, None, None])
    if s.window > 0:
        see &= pos[None, None] > at[..., None] - s.window
    see = see[:, None, None]                                                             # (n, 1, 1, mq, lkv)
    w = torch.matmul(q, whole(s.k_cache, s.k_scale).transpose(-1, -2)).view(n, hkv, g, mq, lkv)
    w = (w * s.scale).masked_fill_(~see, -math.inf)
    top = w.amax(-1, keepdim=True)
    w = torch.exp_(w.sub_(top.clamp(min=-1e30)))
    total = w.sum(-1, keepdim=True)
    v = whole(s.v_cache, s.v_scale)
    v = torch.where((pos[None] < kv[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(w.view(n, hkv, g * mq, lkv), v).view(n, hkv, g, mq, d) / total.clamp(min=1e-37)
    lse = (top + torch.log(total))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(n * mq, hq, d)
    lse = lse.permute(0, 3, 1, 2).reshape(n * mq, hq)
    tok = torch.arange(t, device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    src = seq * mq + tok - cu[seq]
    return dict(o=o[src].to(s.out), lse=lse[src])


def _slots_plain(s):
    hk, hv = s.case["Hk"], s.case["Hv"]
    cu, t = s.cu.long(), s.q.shape[0]
    ql = cu[1:] - cu[:-1]
    slots = s.slots.long()
    st = s.state[slots]
    o = torch.zeros(t + 1, hv, s.v.shape[-1], device=DEV)
    heads = torch.arange(hv, device=DEV) // (hv // hk)
    for i in range(s.max_q):       # the recurrence: token by token
        live = i < ql
        row = torch.where(live, cu[:-1] + i, 0).clamp(max=max(t - 1, 0))
        q, k, v = s.q[row].float()[:, heads] * s.scale, s.k[row].float()[:, heads], s.v[row].float()
        dec = st * torch.exp(s.g[row])[..., None, None]
        u = s.beta[row][..., None] * (v - (dec * k[..., None]).sum(-2))
        nxt = dec + k[..., None] * u[..., None, :]
        o[torch.where(live, row, t)] = (nxt * q[..., None]).sum(-2)
        st = torch.where(live[:, None, None, None], nxt, st)
    s.state[slots] = st
    return dict(o=o[:t].to(s.out), state=s.state)


def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plan_plain, "append": _append_plain, "attn": _attn_plain, "slots": _slots_plain}[state.op](state)


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "plan":
        ctx, new = _plan_lens(case)
        entries = sum(-(-(c + max(n, 0)) // case["bs"]) - c // case["bs"] for c, n in zip(ctx, new) if n > 0)
        return {"bytes": 4.0 * (2 * case["N"] + 3 * case["T"] + 2 * case["N"] + 2 * entries + 6), "flops": 0.0}
    if op == "append":
        ctx, new = _append_lens(case)
        b = 2 if case["dtype"] == "bf16" else 4
        t = sum(new)
        blocks = sum((a + n - 1) // case["bs"] - a // case["bs"] + 1 for a, n in zip(ctx, new))
        rows = 2.0 * t * case["Hkv"] * case["d"]
        return {"bytes": rows * (b + 1) + 4.0 * t + 16.0 * blocks * case["Hkv"], "flops": 2 * rows}
    if op == "attn":
        kv, ql = _attn_lens(case)
        w, hq, hkv, d = case["window"], case["Hq"], case["Hkv"], case["d"]
        b, ob = (2 if case[x] == "bf16" else 4 for x in ("dtype", "out"))
        read, pairs = 0, 0
        for a, n in zip(kv, ql):
            if n == 0:
                continue
            first = a - n
            read += a - (max(0, first - w + 1) if w else 0)
            if w:
                pairs += sum(min(first + j + 1, w) for j in range(n))
            else:
                pairs += n * first + n * (n + 1) // 2
        t = sum(ql)
        return {"bytes": 2.0 * read * hkv * d + 8.0 * hkv * read / case["bs"] + t * hq * (d * (b + ob) + 4.0),
                "flops": 4.0 * pairs * hq * d}
    ql = _slot_lens(case)
    t, live = sum(ql), sum(x > 0 for x in ql)
    b, ob = (2 if case[x] == "bf16" else 4 for x in ("dtype", "out"))
    hk, hv, dk, dv = (case[x] for x in ("Hk", "Hv", "dk", "dv"))
    return {"bytes": 8.0 * live * hv * dk * dv + t * (2.0 * hk * dk * b + hv * dv * (b + ob) + 8.0 * hv) + 8.0 * case["N"],
            "flops": 7.0 * t * hv * dk * dv}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    """Request by request, from the definitions."""
    op = case["op"]
    if op == "plan":
        return None
    s = prepare(case, seed)
    if op == "append":
        out = {}
        slots = s.slot_map.tolist()
        starts = [i for i in range(len(slots)) if i == 0 or slots[i] // s.bs != slots[i - 1] // s.bs] + [len(slots)]
        for name, x, cache, scale in (("k", s.k, s.k_cache, s.k_scale), ("v", s.v, s.v_cache, s.v_scale)):
            held, unit = cache.double(), scale.double()          # what the codes would be without rounding
            for a, b in zip(starts, starts[1:]):
                block, off = divmod(slots[a], s.bs)
                rows = x[a:b].double().transpose(0, 1)
                m, e = torch.frexp(rows.abs().amax((1, 2)) / E4M3_MAX)             # 2^(e-1) <= it < 2^e
                fit = torch.ldexp(torch.ones_like(m), e - (m == 0.5).int()).clamp(min=2.0 ** SCALE_EXP_MIN)
                if off:
                    fit = torch.maximum(fit, unit[block])
                held[block, :, :off] *= (unit[block] / fit)[:, None, None]
                held[block, :, off:off + b - a] = rows / fit[:, None, None]
                unit[block] = fit
            out[name], out[name + "_scale"] = held, unit
        return out
    if op == "attn":
        hq, hkv, d, bs = case["Hq"], case["Hkv"], case["d"], case["bs"]
        g = hq // hkv
        os_, ls_ = [], []
        at = 0
        for n, (a, m) in enumerate(zip(s.kv_list, s.q_list)):
            ids = s.table[n, : -(-a // bs)].long()
            k, v = ((c[ids].double() * sc[ids].double()[:, :, None, None]).transpose(0, 1).reshape(hkv, -1, d)[:, :a]
                    for c, sc in ((s.k_cache, s.k_scale), (s.v_cache, s.v_scale)))
            q = s.q[at:at + m].double()
            place = torch.arange(a - m, a, device=DEV)[:, None]
            keys = torch.arange(a, device=DEV)[None]
            hide = keys > place
            if case["window"]:
                hide |= keys <= place - case["window"]
            o, l = [], []
            for h in range(hq):
                z = (q[:, h] @ k[h // g].T) * s.scale
                z = z.masked_fill(hide, -math.inf)
                l.append(torch.logsumexp(z, -1))
                o.append(torch.exp(z - l[-1][:, None]) @ v[h // g])
            os_.append(torch.stack(o, 1))
            ls_.append(torch.stack(l, 1))
            at += m
        return dict(o=torch.cat(os_), lse=torch.cat(ls_))
    hk, hv = case["Hk"], case["Hv"]
    state = s.state.double()
    o = torch.zeros(s.q.shape[0], hv, case["dv"], dtype=torch.float64, device=DEV)
    beta, decay = s.beta.double(), torch.exp(s.g.double())
    cu, slots, ql = s.cu.long(), s.slots.long(), torch.tensor(s.q_list, device=DEV)
    for i in range(s.max_q):
        who = torch.nonzero(ql > i)[:, 0]
        row, sl = cu[who] + i, slots[who]
        k, q = (x[row].double().repeat_interleave(hv // hk, 1) for x in (s.k, s.q))
        old = state[sl] * decay[row][:, :, None, None]
        err = s.v[row].double() - torch.einsum("nhij,nhi->nhj", old, k)
        new = old + torch.einsum("nhi,nhj->nhij", k, err * beta[row][:, :, None])
        o[row] = torch.einsum("nhij,nhi->nhj", new, q) * s.scale
        state[sl] = new
    return dict(o=o, state=state)
