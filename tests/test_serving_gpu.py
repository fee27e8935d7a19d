"""GPU parity of the serving calls against plain implementations in 64 bits (or in exact integers).

gdn_plan_batch against a loop over requests, gdn_kv_append bit for bit against numpy, gdn_kv_attn and
gdn_decode_slots against fp64; the sizes, masks and inputs where each can go wrong; a run of all of them together.

Tolerances of gdn_kv_attn, for a row with weights w_p = exp(s_p - max s), A = sum w |v| / sum w:
  scores     each is a sum of d products in fp32 (tensor-core accumulation truncates: 2^-23 of the running sum of
             magnitudes a step), with fp32 queries cut to 22 bits: ds <= scale * sum |q k| * (d + 4) * 2^-23. A weight
             moves by e^ds, numerator and denominator alike: 2 ds A (ds < 0.1). With bf16 queries and a bf16 output the
             queries are two e4m3 parts, scaled so that the row's largest is above 224: exact, but for a half step
             of the smallest part, 2^-10, so at most 2^-10 / 224 of the row's largest: ds grows by
             scale * 2^-10 / 224 * max |q| * sum |k|.
  weights    ex2 and the scale product: 2^-21 A; as one fp16 part 2^-11 A, and below 2^-14 an absolute 2^-25 each
             (n 2^-25 max|v|); as two parts 2^-22 A.
  sums       of n terms in fp32, at most n 2^-24 each way but at most 2^-11 A for the sizes here.
  output     2^-8 |o| as bf16, 2^-24 |o| as fp32.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def S():
    from gated_deltanet_sequence_b200 import serving
    return serving


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_sequence_b200 import _lib
    return _lib


def _gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- plan
def plan_ref(ctx, new, table, free, count, bs, T):
    """gdn_plan_batch by its description, request by request; lists in, lists out."""
    table, free = [list(r) for r in table], list(free)
    n, mb, nb = len(ctx), len(table[0]), len(free)
    bad = False
    c, a = list(ctx), list(new)
    for r in range(n):
        if a[r] == -1:
            continue
        if a[r] < -1 or c[r] < 0 or c[r] + a[r] > mb * bs:
            bad, c[r], a[r] = True, 0, 0
    if sum(max(x, 0) for x in a) > T:
        bad = True
        a = [x if x == -1 else 0 for x in a]
    for r in range(n):
        if a[r] == -1:
            for j in range(mb):
                if table[r][j] >= 0:
                    free[count] = table[r][j]
                    count += 1
                table[r][j] = -1
    want = []
    for r in range(n):
        if a[r] > 0:
            want += [(r, j) for j in range(-(-c[r] // bs), -(-(c[r] + a[r]) // bs)) if table[r][j] < 0]
    short = max(0, len(want) - count)
    if not short:
        for r, j in want:
            count -= 1
            table[r][j] = free[count]
    cu, pos, seq, slot = [0], [-1] * T, [-1] * T, [-1] * T
    for r in range(n):
        for i in range(max(a[r], 0)):
            t = cu[-1] + i
            p = c[r] + i
            b = table[r][p // bs]
            pos[t], seq[t], slot[t] = p, r, (b * bs + p % bs if b >= 0 else -1)
        cu.append(cu[-1] + max(a[r], 0))
    kv = [0 if a[r] == -1 else c[r] + a[r] for r in range(n)]
    return dict(cu_seqlens=cu, kv_lens=kv, positions=pos, seq_ids=seq, slot_map=slot,
                info=[cu[-1], max(kv), short, count], table=table, free=free), bad


def plan_run(S, lib, ctx, new, table, free, count, bs, T):
    p = S.BatchPlan.empty(len(ctx), T, DEV)
    t, f, c = i32(table), i32(free), i32([count])
    S.gdn_plan_batch(i32(ctx), i32(new), t, f, c, bs, p)
    st = lib.gdn_sync_status()
    got = {k: getattr(p, k).tolist() for k in ("cu_seqlens", "kv_lens", "positions", "seq_ids", "slot_map", "info")}
    got.update(table=t.tolist(), free=f.tolist())
    assert c.item() == got["info"][3]
    return got, st


def _plan_state(rng, ctx, bs, mb, spare):
    nb = sum(-(-c // bs) for c in ctx) + spare
    ids = list(rng.permutation(nb))
    table = [[int(ids.pop()) for _ in range(-(-c // bs))] + [-1] * (mb - -(-c // bs)) for c in ctx]
    free = [int(x) for x in ids] + [-7] * (nb - len(ids))
    return table, free, len(ids)


@pytest.mark.parametrize("n,hi,newhi,bs,spare,T_more", [
    (1, 40, 1, 16, 4, 0), (1, 0, 700, 16, 60, 3), (7, 100, 30, 32, 40, 5), (256, 300, 1, 64, 300, 0),
    (300, 5, 90, 16, 2500, 0), (1500, 20, 3, 16, 3000, 1), (8192, 3, 1, 16, 9000, 2), (40, 100, 400, 128, 300, 77), (33, 2000, 2, 16, 3, 0),
])
def test_plan_matches_the_loop(S, lib, n, hi, newhi, bs, spare, T_more):
    rng = np.random.default_rng(n + bs)
    ctx = [int(x) for x in rng.integers(0, hi + 1, n)]
    new = [int(x) for x in rng.integers(0, newhi + 1, n)]
    for r in range(n):
        if n > 4 and rng.random() < 0.1:
            new[r] = -1
    mb = max(-(-(c + max(a, 0)) // bs) for c, a in zip(ctx, new)) + 2
    table, free, count = _plan_state(rng, ctx, bs, mb, spare)
    T = sum(max(a, 0) for a in new) + T_more
    want, bad = plan_ref(ctx, new, table, free, count, bs, T)
    got, st = plan_run(S, lib, ctx, new, table, free, count, bs, T)
    assert not bad and st == 0
    for k in want:
        assert got[k] == want[k], k
    # the same call again: the blocks are there already, nothing more is taken or freed
    again, st = plan_run(S, lib, ctx, new, got["table"], got["free"], got["info"][3], bs, T)
    assert st == 0
    if not want["info"][2]:
        assert again["table"] == got["table"] and again["info"][3] == got["info"][3]
        assert again["slot_map"] == got["slot_map"]


def test_plan_short_of_blocks_takes_none_and_recovers(S, lib):
    bs, mb, T = 16, 8, 200
    ctx, new = [10, 0, 40], [100, 60, 1]                     # needs 6 + 4 + 0 blocks
    table = [[3] + [-1] * 7, [-1] * 8, [0, 1, 2] + [-1] * 5]
    free = [4, 5, 6] + [-1] * 20
    want, _ = plan_ref(ctx, new, table, free, 3, bs, T)
    got, st = plan_run(S, lib, ctx, new, table, free, 3, bs, T)
    assert st == 0 and got == want and got["info"][2] == 7 and got["slot_map"][0] == 3 * 16 + 10 and got["slot_map"][6] == -1
    more = got["free"][:3] + list(range(7, 17)) + [-1] * 10
    got2, st = plan_run(S, lib, ctx, new, got["table"], more, 13, bs, T)
    assert st == 0 and got2 == plan_ref(ctx, new, got["table"], more, 13, bs, T)[0]
    assert got2["info"][2] == 0 and min(got2["slot_map"][:161]) >= 0 and got2["slot_map"][161:] == [-1] * 39


@pytest.mark.parametrize("ctx,new,T", [([5, 3], [4, 9], 12), ([-1, 3], [4, 9], 20), ([5, 60], [1, 5], 20), ([5, 3], [-2, 2], 20)])
def test_plan_reports_bad_lengths(S, lib, ctx, new, T):
    table = [[0] + [-1] * 3, [1] + [-1] * 3]
    free = [2, 3, 4, 5, 6, 7, -1, -1]
    want, bad = plan_ref(ctx, new, table, free, 6, 16, T)
    got, st = plan_run(S, lib, ctx, new, table, free, 6, 16, T)
    assert bad and st == lib.GDN_ERR_INVALID_ARG and got == want
    assert lib.gdn_sync_status() == 0


def test_plan_without_rows_and_with_a_bad_table(S, lib):
    p = S.BatchPlan.empty(2, 0, DEV)
    S.gdn_plan_batch(i32([3, 0]), i32([0, 0]), i32([[0], [-1]]), i32([1, -1]), i32([1]), 16, p)
    assert lib.gdn_sync_status() == 0 and p.cu_seqlens.tolist() == [0, 0, 0] and p.kv_lens.tolist() == [3, 0]
    # a cached token's block is missing, another's number is out of range: their new tokens get no slot
    got, st = plan_run(S, lib, [3, 5], [1, 1], [[-1], [9]], [0, -1], 1, 16, 2)
    assert st == lib.GDN_ERR_INVALID_ARG and got["slot_map"] == [-1, -1]
    # an impossible free count
    got, st = plan_run(S, lib, [0], [1], [[-1]], [0, 1], 5, 16, 1)
    assert st == lib.GDN_ERR_INVALID_ARG and got["info"][2] == 1
    # a finished request's row holds a number out of range: it is dropped
    got, st = plan_run(S, lib, [20], [-1], [[7, 1]], [0, -1, -1], 1, 16, 1)
    assert st == lib.GDN_ERR_INVALID_ARG and got["free"][:2] == [0, 1] and got["info"][3] == 2 and got["table"] == [[-1, -1]]


# ---------------------------------------------------------------- append
def scale_ref(amax):
    """Smallest power of two 2^e, e >= -100, with amax <= 448 * 2^e (float64, exact)."""
    m, e = np.frexp(np.asarray(amax, np.float64) / 448.0)
    e = np.where(m == 0.5, e - 1, e)
    return np.where(amax > 0, np.ldexp(1.0, np.maximum(e, -100)), 2.0 ** -100)


def codes_ref(x):
    """float64 -> e4m3 codes, nearest even (torch's conversion from fp32: x here is exact in fp32)."""
    return torch.from_numpy(x.astype(np.float32)).to(E4M3).view(torch.uint8).numpy()


def append_ref(codes, scale, x, slots, bs):
    """x (T, H, d) float64 into codes (nb, H, bs, d) uint8, scale (nb, H), run by run."""
    codes, scale = codes.copy(), scale.copy()
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        b, off = divmod(slots[t], bs)
        n = 1
        while t + n < len(slots) and slots[t + n] == slots[t] + n and off + n < bs:
            n += 1
        rows = x[t:t + n].transpose(1, 0, 2)
        fin = np.where(np.isfinite(rows), np.abs(rows), 0.0)
        fit = scale_ref(fin.max(axis=(1, 2)))
        if off:
            fit = np.maximum(fit, scale[b])
            grown = fit > scale[b]
            old = torch.from_numpy(codes[b][:, :off]).view(E4M3).float().numpy().astype(np.float64)
            again = codes_ref(old * (scale[b] / fit)[:, None, None])
            codes[b][:, :off] = np.where(grown[:, None, None], again, codes[b][:, :off])
        y = np.where(np.isinf(rows), np.nan, rows / fit[:, None, None])
        codes[b][:, off:off + n] = codes_ref(y)
        scale[b] = fit
        t += n
    return codes, scale


def same_codes(a, b):
    """Equal bytes; NaN codes of either sign are one value."""
    nan = lambda c: (c & 0x7f) == 0x7f  # noqa: E731
    return np.array_equal(np.where(nan(a), 0x7f, a), np.where(nan(b), 0x7f, b))


def make_cache(S, nb, H, bs, d, seed, fill=None):
    g = _gen(seed)
    def half():
        c = (torch.randn(nb, H, bs, d, generator=g, device=DEV) * 100).clamp_(-448, 448).to(E4M3)
        s = torch.exp2(torch.randint(-9, -5, (nb, H), generator=g, device=DEV).float())
        return c, s
    k, ks = half()
    v, vs = half()
    if fill is not None:
        k.view(torch.uint8).fill_(fill)
        v.view(torch.uint8).fill_(fill)
    return S.KvCache(k, v, ks, vs)


def slots_for(ctx, new, bs, seed):
    """Slot map of requests over scattered blocks, the table and the number of blocks."""
    rng = np.random.default_rng(seed)
    need = [-(-(c + a) // bs) for c, a in zip(ctx, new)]
    nb = sum(need) + 2
    ids = list(rng.permutation(nb))
    table = [[int(ids.pop()) for _ in range(k)] for k in need]
    slots = [table[r][p // bs] * bs + p % bs for r in range(len(ctx)) for p in range(ctx[r], ctx[r] + new[r])]
    return slots, table, nb


APPEND = [([0], [1]), ([5], [1]), ([0, 15, 16, 17, 31], [1, 1, 1, 1, 1]), ([0, 3], [130, 61]), ([0], [5000]),
          ([7] * 40, [1, 2, 3, 4, 5, 6, 7, 8, 9, 10] * 4), ([120, 0, 64], [9, 128, 64])]


@pytest.mark.parametrize("case", range(len(APPEND)))
@pytest.mark.parametrize("H,d,bs,dtype", [(1, 64, 16, torch.float32), (3, 128, 64, torch.bfloat16), (2, 64, 128, torch.bfloat16),
                                          (2, 128, 32, torch.float32), (1, 128, 128, torch.float32)])
def test_append_is_exact(S, lib, case, H, d, bs, dtype):
    ctx, new = APPEND[case]
    slots, _, nb = slots_for(ctx, new, bs, seed=case)
    T = len(slots)
    cache = make_cache(S, nb, H, bs, d, seed=case)
    size = torch.exp(2.0 * torch.randn(T, H, 1, generator=_gen(case + 50), device=DEV))
    k, v = ((torch.randn(T, H, d, generator=_gen(case + 60 + i), device=DEV) * size).to(dtype) for i in range(2))
    want = [append_ref(c.view(torch.uint8).cpu().numpy(), s.cpu().numpy().astype(np.float64), x.double().cpu().numpy(), slots, bs)
            for c, s, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v))]
    S.gdn_kv_append(cache, k, v, i32(slots))
    assert lib.gdn_sync_status() == 0
    for (codes, scale), c, s in zip(want, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        assert np.array_equal(s.cpu().numpy(), scale.astype(np.float32))
        assert same_codes(c.view(torch.uint8).cpu().numpy(), codes)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_special_values_skipped_rows_and_strides(S, lib, dtype):
    H, d, bs, nb = 2, 64, 16, 6
    x = torch.randn(40, 2 * H * d + 32, generator=_gen(3), device=DEV).to(dtype)      # one fused projection
    x[2, 5], x[3, 6], x[4, H * d + 7], x[20, 1] = float("nan"), float("inf"), float("-inf"), 448.0
    x[6:9] = 0.0
    x[30, :H * d] = 3e38                                                               # the largest scales
    x[31, :H * d] = 1e-38                                                              # below the smallest
    slots = [-1, 0, 1, 2, 3, 4, 16, 17, 18, -1, 60, 61, 62, 63] + [-1] * 6 + list(range(32, 42)) + [64, 80] + [-1] * 8
    k, v = x[:, :H * d].view(40, H, d), x[:, H * d:2 * H * d].view(40, H, d)
    assert not k.is_contiguous()
    cache = make_cache(S, nb, H, bs, d, seed=9)
    want = [append_ref(c.view(torch.uint8).cpu().numpy(), s.cpu().numpy().astype(np.float64), y.double().cpu().numpy(), slots, bs)
            for c, s, y in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v))]
    S.gdn_kv_append(cache, k, v, i32(slots))
    assert lib.gdn_sync_status() == 0
    for (codes, scale), c, s in zip(want, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        assert np.array_equal(s.cpu().numpy(), scale.astype(np.float32))
        assert same_codes(c.view(torch.uint8).cpu().numpy(), codes)


def test_append_piece_by_piece_gives_the_same_scales_and_values(S):
    """Scales are powers of two: a prompt appended token by token ends with the scales of one call, and with its codes
    but for values that fell below the smallest normal (2^-6 scale) before the scale grew, off by at most one step
    (2^-9 scale) more."""
    H, d, bs, T = 2, 64, 32, 90
    slots, _, nb = slots_for([0], [T], bs, seed=4)
    x = torch.randn(T, H, d, generator=_gen(5), device=DEV) * torch.exp(torch.linspace(-3, 3, T, device=DEV))[:, None, None]
    a, b = make_cache(S, nb, H, bs, d, 6), make_cache(S, nb, H, bs, d, 6)
    S.gdn_kv_append(a, x, x, i32(slots))
    for t in range(T):
        S.gdn_kv_append(b, x[t:t + 1], x[t:t + 1], i32(slots[t:t + 1]))
    assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)
    ka, kb = a.k.float(), b.k.float()
    assert (ka - kb).abs().max().item() <= 2.0 ** -9
    assert torch.equal(ka[ka.abs() > 2.0 ** -5], kb[ka.abs() > 2.0 ** -5])


def test_append_reports_slots_out_of_range(S, lib):
    cache = make_cache(S, 4, 2, 16, 64, 7)
    before = [c.view(torch.uint8).clone() for c in (cache.k, cache.v)]
    k = torch.randn(3, 2, 64, device=DEV)
    S.gdn_kv_append(cache, k, k, i32([64, -2, 2 ** 31 - 1]))
    assert lib.gdn_sync_status() == lib.GDN_ERR_INVALID_ARG
    assert torch.equal(cache.k.view(torch.uint8), before[0]) and torch.equal(cache.v.view(torch.uint8), before[1])
    S.gdn_kv_append(cache, k[:0], k[:0], i32([]))
    assert lib.gdn_sync_status() == 0


# ---------------------------------------------------------------- attention
def attn_ref(cache, q, table, cu, kv, window, scale, parts=False):
    """fp64 on the CPU: o, lse, and the tolerance's pieces A = sum w|v| / sum w, ds and max|v| of each row."""
    q = q.double().cpu()
    k, v = ((c.cpu().float().double() * s.cpu().double()[:, :, None, None]) for c, s in
            ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    T, Hq, d = q.shape
    g = Hq // cache.heads
    o, A, ds, vm = torch.zeros(T, Hq, d).double(), torch.zeros(T, Hq, d).double(), torch.zeros(T, Hq).double(), torch.zeros(T, Hq).double()
    lse = torch.full((T, Hq), -math.inf).double()
    for n in range(len(kv)):
        a, m = kv[n], cu[n + 1] - cu[n]
        if a == 0 or m == 0:
            continue
        ids = torch.tensor(table[n][: -(-a // cache.block_size)])
        kk, vv = (x[ids].transpose(0, 1).reshape(cache.heads, -1, d)[:, :a] for x in (k, v))
        for i in range(m):
            p = a - m + i
            lo = max(0, p - window + 1) if window else 0
            if p < 0:
                continue
            for h in range(Hq):
                ks, vs, qq = kk[h // g][lo:p + 1], vv[h // g][lo:p + 1], q[cu[n] + i, h]
                s = scale * (ks @ qq)
                t, r = cu[n] + i, torch.logsumexp(s, 0)
                w = torch.exp(s - r)
                lse[t, h], o[t, h], A[t, h] = r, w @ vs, w @ vs.abs()
                ds[t, h] = abs(scale) * (ks.abs() @ qq.abs()).max() * (d + 4) * 2.0 ** -23
                if parts:
                    ds[t, h] += abs(scale) * 2.0 ** -10 / 224 * qq.abs().max() * ks.abs().sum(-1).max()
                vm[t, h] = vs.abs().max()
    return o, lse, A, ds, vm


def attn_case(S, kv, ql, Hkv, G, d, bs, dtype, seed, fill=None, spare=2):
    slots, table, nb = slots_for([0] * len(kv), kv, bs, seed)
    cache = make_cache(S, nb + spare, Hkv, bs, d, seed, fill)
    if fill is not None:      # only the rows of the requests hold values; the rest is `fill`
        used = torch.tensor(slots, dtype=torch.long, device=DEV)
        src = make_cache(S, nb + spare, Hkv, bs, d, seed)
        for c, x in ((cache.k, src.k), (cache.v, src.v)):
            c.view(torch.uint8)[used // bs, :, used % bs] = x.view(torch.uint8)[used // bs, :, used % bs]
    mb = max([1] + [len(r) for r in table]) + 1
    tab = i32([r + [-1] * (mb - len(r)) for r in table])
    cu = [0]
    for x in ql:
        cu.append(cu[-1] + x)
    q = torch.randn(cu[-1], Hkv * G, d, generator=_gen(seed + 1), device=DEV).to(dtype)
    return cache, q, table, tab, cu


def behind(q, rows, value=float("nan")):
    """q and rows that belong to nobody behind it."""
    return torch.cat([q, torch.full((rows, *q.shape[1:]), value, dtype=q.dtype, device=DEV)])


def attn_check(S, lib, cache, q, table, tab, cu, kv, window, scale, out, max_q=None, pad=3):
    T = q.shape[0]
    o = torch.full((T + pad, q.shape[1], q.shape[2]), 7.0, dtype=out, device=DEV)
    lse = torch.full((T + pad, q.shape[1]), 7.0, device=DEV)
    qq = behind(q, pad)
    mq = max_q or max([1] + [b - a for a, b in zip(cu, cu[1:])])
    S.gdn_kv_attn(cache, qq, tab, i32(cu), i32(kv), max_q_len=mq, window=window, scale=scale, o=o, lse=lse)
    assert lib.gdn_sync_status() == 0
    assert (o[T:] == 7).all() and (lse[T:] == 7).all()
    ro, rl, A, ds, vm = attn_ref(cache, q, table, cu, kv, window, scale, q.dtype == out == torch.bfloat16)
    o, lse = o[:T].double().cpu(), lse[:T].double().cpu()
    n = max([1] + list(kv))
    sums = min(n * 2.0 ** -23, 2.0 ** -11)
    if out == torch.bfloat16:
        tol = 2.0 ** -8 * ro.abs() + A * (2 * ds[..., None] + 2.0 ** -21 + 2.0 ** -11 + sums) + n * 2.0 ** -25 * vm[..., None]
    else:
        tol = 2.0 ** -24 * ro.abs() + A * (2 * ds[..., None] + 2.0 ** -21 + 2.0 ** -22 + sums) + 1e-30
    bad = ((o - ro).abs() > tol) | torch.isnan(o)
    assert not bad.any(), ((o - ro).abs() / tol).max()
    fin = torch.isfinite(rl)
    assert torch.equal(fin, torch.isfinite(lse)) and (lse[~fin] == -math.inf).all() and (o[~fin] == 0).all()
    # lse: the largest score's error, the sum's, and its own rounding
    lt = ds + 2.0 ** -20 + sums + 2.0 ** -22 * rl.abs()
    assert ((lse - rl).abs()[fin] <= lt[fin]).all()


ATTN = {  # kv lengths, query rows
    "one": ([1], [1]),
    "ragged": ([1, 15, 16, 17, 31, 32, 33, 64, 127, 128, 129, 300], [1] * 12),
    "long": ([5000, 3, 1999], [1, 1, 1]),
    "drafted": ([4, 40, 131, 700], [4, 3, 5, 2]),
    "empty rows": ([0, 3, 0, 50], [1, 5, 0, 0]),
    "prompt": ([150, 37], [70, 37]),
}


@pytest.mark.parametrize("case", list(ATTN))
@pytest.mark.parametrize("Hkv,G,d,bs,dtype,out,window", [
    (2, 4, 128, 64, torch.bfloat16, torch.bfloat16, 0), (1, 1, 64, 16, torch.bfloat16, torch.float32, 0),
    (2, 3, 64, 32, torch.float32, torch.float32, 33), (1, 16, 128, 16, torch.float32, torch.bfloat16, 0),
    (1, 20, 128, 128, torch.bfloat16, torch.float32, 100), (3, 2, 64, 128, torch.bfloat16, torch.bfloat16, 1),
    (1, 7, 128, 32, torch.float32, torch.float32, 0),
])
def test_attn_matches_fp64(S, lib, case, Hkv, G, d, bs, dtype, out, window):
    kv, ql = ATTN[case]
    # what nobody may see is NaN: unused rows of the blocks in use, and whole blocks
    args = attn_case(S, kv, ql, Hkv, G, d, bs, dtype, seed=len(case) + d + bs, fill=0x7f)
    attn_check(S, lib, *args, kv, window, 1.0 / math.sqrt(d), out)


@pytest.mark.parametrize("d,dtype,out", [(128, torch.bfloat16, torch.float32), (64, torch.float32, torch.float32)])
def test_attn_scales_far_apart(S, lib, d, dtype, out):
    """Blocks whose V scales differ by 2^40, those of the heavy tokens smallest, and queries from 1e-20 to 1e10."""
    kv, ql = [200, 90], [2, 1]
    cache, q, table, tab, cu = attn_case(S, kv, ql, 2, 2, d, 16, dtype, seed=31)
    cache.v_scale.copy_(torch.exp2(torch.randint(-30, 10, cache.v_scale.shape, generator=_gen(1), device=DEV).float()))
    cache.k_scale.copy_(torch.exp2(torch.randint(-12, -7, cache.k_scale.shape, generator=_gen(2), device=DEV).float()))
    attn_check(S, lib, cache, q, table, tab, cu, kv, 0, 0.5, out)
    small = (q.float() * 1e-20).to(dtype)
    attn_check(S, lib, cache, small, table, tab, cu, kv, 0, 1e20, out)
    big = (q.float() * 1e10).to(dtype)
    attn_check(S, lib, cache, big, table, tab, cu, kv, 0, 1e-10, out)


@pytest.mark.parametrize("ql", [[5, 1], [40, 3]])
@pytest.mark.parametrize("where", ["k", "v"])
def test_attn_nan_reaches_the_rows_that_see_it(S, lib, where, ql):
    """A NaN at a position (stored by append from a NaN or an infinity) reaches every query that sees the position and
    no other."""
    kv, Hkv, G, d, bs, window = [70, 40], 2, 2, 64, 16, 20
    for win in (0, window):
        cache, q, table, tab, cu = attn_case(S, kv, ql, Hkv, G, d, bs, torch.bfloat16, seed=77)
        at = kv[0] - 3
        hole = cache.k if where == "k" else cache.v
        hole.view(torch.uint8)[table[0][at // bs], 1, at % bs, 9] = 0xff
        at2 = 4                                             # request 1, far back: outside the window
        hole.view(torch.uint8)[table[1][at2 // bs], 0, at2 % bs, 5] = 0x7f
        o, _ = S.gdn_kv_attn(cache, q, tab, i32(cu), i32(kv), max_q_len=max(ql), window=win, scale=0.125)
        lib.gdn_sync_status()
        bad = torch.isnan(o).cpu()
        for n, (p, head) in enumerate(((at, 1), (at2, 0))):
            for i in range(ql[n]):
                pos = kv[n] - ql[n] + i
                sees = pos >= p and (win == 0 or pos - win < p)
                for h in range(Hkv * G):
                    hit = sees and h // G == head
                    col = 9 if n == 0 else 5
                    row = bad[cu[n] + i, h]
                    assert bool(row[col]) == hit, (win, n, i, h)
                    assert bool(row.any()) == hit
                    if where == "v":
                        assert int(row.sum()) == int(hit)


def test_attn_reports_bad_batches(S, lib):
    kv, ql = [40, 50, 60], [1, 1, 1]
    cache, q, table, tab, cu = attn_case(S, kv, ql, 2, 2, 64, 16, torch.bfloat16, seed=12)
    good, _ = S.gdn_kv_attn(cache, q, tab, i32(cu), i32(kv), scale=0.125)
    assert lib.gdn_sync_status() == 0

    def run(tab=tab, cu=cu, kv=kv, max_q_len=1):
        o = torch.full_like(good, 7.0)
        S.gdn_kv_attn(cache, q, tab, i32(cu), i32(kv), max_q_len=max_q_len, scale=0.125, o=o)
        st = lib.gdn_sync_status()
        assert lib.gdn_sync_status() == 0
        return o, st
    mb = tab.shape[1]
    for kw, untouched in ((dict(cu=[0, 1, 0, 3]), [1]), (dict(cu=[0, 1, 2, 4]), [2]), (dict(cu=[-1, 1, 2, 3]), [0]),
                          (dict(kv=[40, -1, 60]), [1]), (dict(kv=[40, mb * 16 + 1, 60]), [1])):
        o, st = run(**kw)
        assert st == lib.GDN_ERR_INVALID_ARG, kw
        for r in untouched:
            assert (o[r] == 7).all(), kw
    o, st = run(cu=[0, 2, 3, 3])                              # two rows where max_q_len says one
    assert st == lib.GDN_ERR_INVALID_ARG and (o[:2] == 7).all()
    for b in (-1, cache.num_blocks, 2 ** 31 - 1):             # a page that does not exist: its positions are left out
        t2 = tab.clone()
        t2[1, 1] = b
        o, st = run(tab=t2)
        assert st == lib.GDN_ERR_INVALID_ARG
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2]) and torch.isfinite(o[1]).all()


def test_attn_takes_strided_queries_and_the_last_block_of_a_large_cache(S, lib):
    d, bs, Hkv, nb = 128, 128, 8, 33000                       # 4.3e9 bytes in each of K and V
    k = torch.zeros(nb, Hkv, bs, d, dtype=torch.uint8, device=DEV).view(E4M3)
    v = torch.zeros(nb, Hkv, bs, d, dtype=torch.uint8, device=DEV).view(E4M3)
    cache = S.KvCache(k, v, torch.ones(nb, Hkv, device=DEV), torch.ones(nb, Hkv, device=DEV))
    n = 100
    x = torch.randn(n, 3 * Hkv * d, generator=_gen(8), device=DEV).bfloat16()
    q, kk, vv = (x[:, i * Hkv * d:(i + 1) * Hkv * d].view(n, Hkv, d) for i in range(3))
    slots = [(nb - 1) * bs + i for i in range(n)]
    S.gdn_kv_append(cache, kk, vv, i32(slots))
    o, lse = S.gdn_kv_attn(cache, q[-1:], i32([[nb - 1]]), i32([0, 1]), i32([n]), scale=d ** -0.5, lse=True)
    o2, _ = S.gdn_kv_attn(cache, q, i32([[nb - 1]]), i32([0, n]), i32([n]), max_q_len=n, scale=d ** -0.5)
    assert lib.gdn_sync_status() == 0
    small = S.KvCache(k[-1:].clone(), v[-1:].clone(), cache.k_scale[-1:].clone(), cache.v_scale[-1:].clone())
    del k, v, cache
    assert small.k.float().abs().sum() > 0
    ro, rl, A, ds, _ = attn_ref(small, q, [[0]], [0, n], [n], 0, d ** -0.5)
    for got, ref, a, e in ((o.double().cpu()[0], ro[-1], A[-1], ds[-1]), (o2.double().cpu(), ro, A, ds)):
        assert ((got - ref).abs() <= 2.0 ** -24 * ref.abs() + a * (2 * e[..., None] + 2.0 ** -19)).all()


@pytest.mark.parametrize("window", [0, 2 ** 31 - 1])
def test_attn_bounds_far_above_the_batch(S, lib, window):
    """max_q_len and the window are bounds: one row under a bound of thousands, a window that nothing outgrows."""
    kv, ql = [30, 5], [1, 3]
    cache, q, table, tab, cu = attn_case(S, kv, ql, 2, 2, 64, 16, torch.bfloat16, seed=17)
    attn_check(S, lib, cache, q, table, tab, cu, kv, 0, 0.125, torch.bfloat16)
    a, l = S.gdn_kv_attn(cache, q, tab, i32(cu), i32(kv), scale=0.125, max_q_len=3, out_dtype=torch.bfloat16, lse=True)
    b, none = S.gdn_kv_attn(cache, q, tab, i32(cu), i32(kv), scale=0.125, max_q_len=2 ** 31 - 1, window=window,
                            out_dtype=torch.bfloat16, lse=False)
    assert lib.gdn_sync_status() == 0 and torch.equal(a, b) and none is None
    one, _ = S.gdn_kv_attn(cache, q[:1], tab[:1], i32([0, 1]), i32(kv[:1]), scale=0.125, max_q_len=4096, window=window,
                           out_dtype=torch.bfloat16)
    assert lib.gdn_sync_status() == 0 and torch.equal(one, a[:1])


def test_attn_streams_graphs_and_two_calls_at_once(S, lib):
    kv, ql = [700, 33, 1200], [1, 2, 1]
    cache, q, table, tab, cu = attn_case(S, kv, ql, 2, 4, 128, 64, torch.bfloat16, seed=5)
    cu_t, kv_t = i32(cu), i32(kv)
    ref, _ = S.gdn_kv_attn(cache, q, tab, cu_t, kv_t, max_q_len=2, scale=0.1)
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(ref) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, o in zip(side, outs):                        # each call has its own workspace
            S.gdn_kv_attn(cache, q, tab, cu_t, kv_t, max_q_len=2, scale=0.1, o=o, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
    # captured once, replayed with other lengths and queries
    o = torch.zeros_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.gdn_kv_attn(cache, q, tab, cu_t, kv_t, max_q_len=2, scale=0.1, o=o)
    kv_t.copy_(i32([650, 20, 1199]))
    q.copy_(q.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    want, _ = S.gdn_kv_attn(cache, q, tab, cu_t, kv_t, max_q_len=2, scale=0.1)
    assert torch.equal(o, want) and not torch.equal(o, ref) and lib.gdn_sync_status() == 0


def test_attn_gives_up_on_a_wait_and_reports_it(S, lib):
    kv, ql = [20000] * 8, [1] * 8             # 330 MB of codes: more than L2, so that the waits have something to wait for
    cache, q, table, tab, cu = attn_case(S, kv, ql, 8, 4, 128, 64, torch.bfloat16, seed=6)
    ref, _ = S.gdn_kv_attn(cache, q, tab, i32(cu), i32(kv), scale=0.1)
    assert lib.gdn_sync_status() == 0
    lib.gdn_set_wait_limit_for_testing(1)
    try:
        S.gdn_kv_attn(cache, q, tab, i32(cu), i32(kv), scale=0.1)
        assert lib.gdn_sync_status() == lib.GDN_ERR_TIMEOUT
    finally:
        lib.gdn_set_wait_limit_for_testing(0)
    o, _ = S.gdn_kv_attn(cache, q, tab, i32(cu), i32(kv), scale=0.1)
    assert lib.gdn_sync_status() == 0 and torch.equal(o, ref)


# A batch for thousands of rows gives its requests of more than 64 rows (tokens x heads of a KV head) to the many-rows
# kernel, whether its rows are used or lie behind the last request: MANY rows behind make small batches take it.
MANY = 9000
PROMPT = {  # kv lengths, query rows
    "just over": ([65], [65]),
    "one tile": ([128], [128]),
    "ragged": ([300, 5, 131, 257], [300, 1, 67, 129]),
    "over a context": ([700, 600], [200, 33]),
    "more rows than tokens": ([100, 0, 20], [130, 80, 1]),
    "long": ([1500], [310]),
}


@pytest.mark.parametrize("case", list(PROMPT))
@pytest.mark.parametrize("Hkv,G,d,bs,window,scale", [
    (1, 1, 128, 64, 0, 0.09), (2, 4, 128, 16, 0, 0.09), (1, 3, 64, 32, 0, 0.125), (2, 1, 64, 128, 100, 0.125),
    (1, 2, 128, 128, 1, -0.09), (1, 8, 64, 16, 300, 0.125), (1, 1, 128, 32, 64, 0.0),
])
@pytest.mark.parametrize("pad", [3, MANY])
def test_attn_prompts_match_fp64(S, lib, case, Hkv, G, d, bs, window, scale, pad):
    kv, ql = PROMPT[case]
    args = attn_case(S, kv, ql, Hkv, G, d, bs, torch.bfloat16, seed=len(case) + d + bs, fill=0x7f)
    attn_check(S, lib, *args, kv, window, scale, torch.bfloat16, pad=pad)


def test_attn_prompts_of_thousands_of_rows(S, lib):
    """No rows behind: 9600 rows, then around the 5920 (40 for each of 148 SMs) that the many-rows kernel begins at."""
    kv, ql = [420, 60], [290, 10]
    args = attn_case(S, kv, ql, 8, 4, 128, 64, torch.bfloat16, seed=3)
    attn_check(S, lib, *args, kv, 0, 0.09, torch.bfloat16, pad=0)
    for m in (184, 185, 186):
        args = attn_case(S, [m], [m], 8, 4, 128, 64, torch.bfloat16, seed=m)
        attn_check(S, lib, *args, [m], 0, 0.09, torch.bfloat16, pad=0)


@pytest.mark.parametrize("pad", [3, MANY])
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 64)])
def test_attn_prompt_scales_far_apart(S, lib, d, bs, pad):
    """V scales of neighbouring blocks 2^40 apart (fp16 cannot hold them together), blocks of zeros, queries of 1e-20."""
    kv, ql = [300, 90], [150, 80]
    cache, q, table, tab, cu = attn_case(S, kv, ql, 2, 2, d, bs, torch.bfloat16, seed=31)
    zero = table[0][1]
    for c, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c.view(torch.uint8)[zero] = 0
        sc[zero] = 2.0 ** -100
    attn_check(S, lib, cache, (q.float() * 1e-20).bfloat16(), table, tab, cu, kv, 0, 1e19, torch.bfloat16, pad=pad)
    attn_check(S, lib, cache, q, table, tab, cu, kv, 0, 0.1, torch.bfloat16, pad=pad)
    cache.v_scale.copy_(torch.exp2(torch.randint(-30, 10, cache.v_scale.shape, generator=_gen(1), device=DEV).float()))
    attn_check(S, lib, cache, q, table, tab, cu, kv, 0, 0.5, torch.bfloat16, pad=pad)


@pytest.mark.parametrize("pad", [0, MANY])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("window", [0, 50])
def test_attn_prompt_nan_reaches_the_rows_that_see_it(S, lib, where, window, pad):
    kv, ql, Hkv, G, d, bs = [200, 150], [120, 150], 2, 1, 64, 16
    cache, q, table, tab, cu = attn_case(S, kv, ql, Hkv, G, d, bs, torch.bfloat16, seed=78)
    q = behind(q, pad)
    at = 133
    hole = cache.k if where == "k" else cache.v
    hole.view(torch.uint8)[table[0][at // bs], 1, at % bs, 9] = 0xff
    o, _ = S.gdn_kv_attn(cache, q, tab, i32(cu), i32(kv), max_q_len=150, window=window, scale=0.125, out_dtype=torch.bfloat16)
    assert lib.gdn_sync_status() == 0
    bad = torch.isnan(o).cpu()
    for i in range(ql[0]):
        pos = kv[0] - ql[0] + i
        hit = pos >= at and (window == 0 or pos - window < at)
        assert not bad[i, 0].any() and bool(bad[i, 1, 9]) == hit and bool(bad[i, 1].any()) == hit, i
        if where == "v":
            assert int(bad[i, 1].sum()) == int(hit)
    assert not bad[cu[1]:cu[2]].any()


def test_attn_prompt_bad_pages_graphs_and_waits(S, lib):
    kv, ql = [400, 30, 300], [400, 1, 90]
    cache, q, table, tab, cu = attn_case(S, kv, ql, 2, 2, 128, 64, torch.bfloat16, seed=14)
    q = behind(q, MANY, 0.0)
    cu_t, kv_t, n = i32(cu), i32(kv), cu[-1]
    kw = dict(max_q_len=400, scale=0.09, out_dtype=torch.bfloat16)
    good, _ = S.gdn_kv_attn(cache, q, tab, cu_t, kv_t, **kw)
    assert lib.gdn_sync_status() == 0
    for b in (-1, cache.num_blocks, 2 ** 31 - 1):             # a page that does not exist: its positions are left out
        t2 = tab.clone()
        t2[0, 2] = b
        o, _ = S.gdn_kv_attn(cache, q, t2, cu_t, kv_t, **kw)
        assert lib.gdn_sync_status() == lib.GDN_ERR_INVALID_ARG and lib.gdn_sync_status() == 0
        assert torch.equal(o[:128], good[:128]) and torch.equal(o[400:n], good[400:n]) and torch.isfinite(o[:n]).all()
        assert not torch.equal(o[128:400], good[128:400])
    # a request with more rows than max_q_len says is left out, by both kernels
    o = torch.full_like(good, 7.0)
    S.gdn_kv_attn(cache, q, tab, cu_t, kv_t, max_q_len=100, scale=0.09, o=o)
    assert lib.gdn_sync_status() == lib.GDN_ERR_INVALID_ARG
    assert (o[:400] == 7).all() and torch.equal(o[400:n], good[400:n]) and (o[n:] == 7).all()
    # captured and replayed with other lengths; two streams at once
    o = torch.zeros_like(good)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.gdn_kv_attn(cache, q, tab, cu_t, kv_t, o=o, **{k: v for k, v in kw.items() if k != "out_dtype"})
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [S.gdn_kv_attn(cache, q, tab, cu_t, kv_t, stream=st, **kw)[0] for st in side for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(x[:n], good[:n]) for x in outs)
    kv_t.copy_(i32([390, 30, 299]))
    graph.replay()
    torch.cuda.synchronize()
    want, _ = S.gdn_kv_attn(cache, q, tab, cu_t, kv_t, **kw)
    assert torch.equal(o[:n], want[:n]) and not torch.equal(o[:n], good[:n]) and lib.gdn_sync_status() == 0
    lib.gdn_set_wait_limit_for_testing(1)
    try:
        S.gdn_kv_attn(cache, q, tab, cu_t, kv_t, **kw)
        assert lib.gdn_sync_status() == lib.GDN_ERR_TIMEOUT
        while lib.gdn_sync_status() != 0:
            pass
    finally:
        lib.gdn_set_wait_limit_for_testing(0)
    o, _ = S.gdn_kv_attn(cache, q, tab, cu_t, kv_t, **kw)
    assert torch.equal(o[:n], want[:n]) and lib.gdn_sync_status() == 0


# ---------------------------------------------------------------- recurrence over slots
def slots_ref(q, k, v, beta, g, state, slots, cu, scale, d_skip=None, xnorm=None, xw=None, eps=1e-6):
    q, k, v, state = (x.double().cpu() for x in (q, k, v, state))
    T, Hv, dv = v.shape
    rep = Hv // q.shape[1]
    q, k = q.repeat_interleave(rep, 1) * scale, k.repeat_interleave(rep, 1)
    o = torch.full((T, Hv, dv), math.nan).double()
    for n, s in enumerate(slots):
        if s < 0:
            continue
        for t in range(cu[n], cu[n + 1]):
            S = state[s]
            if g is not None:
                a = torch.exp(g[t].double().cpu())
                S = S * (a[:, :, None] if a.dim() == 2 else a[:, None, None])
            u = v[t]
            if beta is not None:
                u = beta[t].double().cpu()[:, None] * (u - torch.einsum("hij,hi->hj", S, k[t]))
            S = S + k[t][:, :, None] * u[:, None, :]
            state[s] = S
            x = torch.einsum("hij,hi->hj", S, q[t])
            if d_skip is not None:
                x = x + d_skip.double().cpu() * v[t]
            if xnorm is not None:
                if xnorm == "layer":
                    x = x - x.mean(-1, keepdim=True)
                x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
                if xw is not None:
                    x = x * xw.double().cpu()
            o[t] = x
    return o, state


def slots_inputs(T, Hk, Hv, dk, dv, pool, dtype, seed, vec=False):
    g = _gen(seed)
    def unit(*shape):
        x = torch.randn(*shape, generator=g, device=DEV)
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype)
    q, k = unit(T, Hk, dk), unit(T, Hk, dk)
    v = torch.randn(T, Hv, dv, generator=g, device=DEV).to(dtype)
    beta = torch.sigmoid(torch.randn(T, Hv, generator=g, device=DEV))
    gate = -0.05 * torch.rand(*((T, Hv, dk) if vec else (T, Hv)), generator=g, device=DEV)
    state = 0.1 * torch.randn(pool, Hv, dk, dv, generator=g, device=DEV)
    return q, k, v, beta, gate, state


def close(a, ref, tokens, bf16=False):
    """Each token's step adds rounding of sums of dk + a few fp32 terms of the state's and the output's own size:
    (128 + 8) 2^-24 = 8.1e-6 of the largest value a token at the worst, and it is carried, not amplified
    (|alpha (I - beta k k^T)| <= 1)."""
    ref = ref.double()
    err = (a.double().cpu() - ref).abs()
    tol = 8.2e-6 * (1 + tokens) * ref.abs().max() + (2.0 ** -8 * ref.abs() if bf16 else 0.0)
    return bool((err <= tol).all())


@pytest.mark.parametrize("mode", ["gdn", "delta", "gated", "plain", "vector"])
@pytest.mark.parametrize("Hk,Hv,dk,dv,dtype", [(2, 4, 128, 128, torch.bfloat16), (1, 3, 64, 128, torch.float32),
                                               (2, 2, 128, 64, torch.float32), (1, 1, 64, 64, torch.bfloat16)])
def test_slots_match_fp64(S, lib, mode, Hk, Hv, dk, dv, dtype):
    ql = [1, 0, 3, 1, 7, 2, 1]
    slots = [4, 2, 8, -1, 0, 6, 3]
    cu = [2]                                                 # rows 0 and 1 are nobody's
    for x in ql:
        cu.append(cu[-1] + x)
    T = cu[-1] + 2
    q, k, v, beta, g, state = slots_inputs(T, Hk, Hv, dk, dv, 9, dtype, seed=dk + Hv, vec=mode == "vector")
    beta = None if mode in ("gated", "plain") else beta
    g = None if mode in ("delta", "plain") else g
    ro, rs = slots_ref(q, k, v, beta, g, state, slots, cu, 0.3)
    o = torch.full((T, Hv, dv), 7.0, device=DEV)
    st = state.clone()
    S.gdn_decode_slots(q, k, v, beta, g, st, i32(slots), i32(cu), o=o, scale=0.3)
    assert lib.gdn_sync_status() == 0
    rows = torch.isfinite(ro[:, 0, 0])
    assert close(o[rows.to(DEV)], ro[rows], 7) and close(st, rs, 7)
    assert (o[~rows.to(DEV)] == 7).all()
    idle = [s for s in range(9) if s not in (4, 8, 0, 6, 3)]
    assert torch.equal(st[idle], state[idle])


@pytest.mark.parametrize("xnorm", [None, "rms", "layer"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dv", [64, 128])
def test_slots_options(S, lib, xnorm, out, dv):
    Hk, Hv, dk = 1, 2, 128
    slots, cu = [1, 0, 2], [0, 2, 3, 7]
    q, k, v, beta, g, state = slots_inputs(7, Hk, Hv, dk, dv, 3, torch.bfloat16, seed=3)
    D, w = (torch.randn(Hv, dv, generator=_gen(i), device=DEV) for i in (1, 2))
    xw = None if xnorm is None else w
    ro, rs = slots_ref(q, k, v, beta, g, state, slots, cu, 1.0, D, xnorm, xw)
    o = S.gdn_decode_slots(q, k, v, beta, g, state, i32(slots), i32(cu), out_dtype=out, d_skip=D, xnorm=xnorm,
                           xnorm_weight=xw)
    assert lib.gdn_sync_status() == 0 and o.dtype == out
    assert close(o, ro, 4, out == torch.bfloat16) and close(state, rs, 4)


def test_slots_single_token_equals_the_decode_step(S, lib):
    N, H, d = 6, 4, 128
    q, k, v, beta, g, state = slots_inputs(N, H, H, d, d, 11, torch.bfloat16, seed=21)
    slots = [7, 0, 3, 10, 5, 2]
    dense = state[slots].clone().contiguous()
    want = lib.gdn_decode_step(q, k, v, beta, g, dense, scale=0.2)
    got = S.gdn_decode_slots(q, k, v, beta, g, state, i32(slots), scale=0.2)
    assert lib.gdn_sync_status() == 0
    assert close(got, want.cpu(), 1) and close(state[slots], dense.cpu(), 1)


def test_slots_report_bad_slots_and_strided_rows(S, lib):
    N, H, d = 5, 2, 64
    x = torch.randn(N, 3 * H * d + 1, generator=_gen(4), device=DEV)      # odd row stride: rows of any alignment
    q, k, v = (x[:, 1 + i * H * d:1 + (i + 1) * H * d].view(N, H, d) for i in range(3))
    with pytest.raises(lib.GdnError):                                      # the first row is not 16-byte aligned
        S.gdn_decode_slots(q, k, v, None, None, torch.zeros(6, H, d, d, device=DEV), i32([0, 1, 2, 3, 4]))
    q, k, v = (x[:, i * H * d:(i + 1) * H * d].view(N, H, d) for i in range(3))
    state = torch.zeros(6, H, d, d, device=DEV)
    o = torch.full((N, H, d), 7.0, device=DEV)
    slots = [2, 6, 2, -1, -5]                                              # beyond the pool, named twice, skipped, below -1
    ro, rs = slots_ref(q, k, v, None, None, state, [2, -1, -1, -1, -1], list(range(N + 1)), 1.0)
    S.gdn_decode_slots(q, k, v, None, None, state, i32(slots), o=o)
    assert lib.gdn_sync_status() == lib.GDN_ERR_INVALID_ARG and lib.gdn_sync_status() == 0
    assert close(o[:1], ro[:1], 1) and (o[1:] == 7).all() and close(state, rs, 1)
    S.gdn_decode_slots(q, k, v, None, None, state, i32([0, 1]), i32([0, 3, 2]), o=o)     # offsets that go back
    assert lib.gdn_sync_status() == lib.GDN_ERR_INVALID_ARG
    assert (state[1] == 0).all()


# ---------------------------------------------------------------- together
def test_serving_steps_together(S, lib):
    """A prompt step and eight decode steps of four requests through one softmax layer and one delta-rule layer, the
    decode step captured once and replayed; one request finishes and its blocks serve another. Outputs against fp64 on
    what the cache holds, and against the recurrence over every token since the start."""
    N, Hq, Hkv, d, bs, mb, T = 4, 8, 2, 64, 16, 8, 64
    Hk, Hv = 2, 4
    nb = 14
    cache = S.KvCache.empty(nb, Hkv, bs, d, DEV)
    table = torch.full((N, mb), -1, dtype=torch.int32, device=DEV)
    free, count = i32(list(range(nb))), i32([nb])
    ctx, new = i32([0] * N), i32([20, 1, 33, 0])
    plan = S.BatchPlan.empty(N, T, DEV)
    slots = i32([2, 0, 3, 1])
    state = torch.zeros(N, Hv, d, d, device=DEV)
    log = [[] for _ in range(N)]                             # each request's rows since its start

    q = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device=DEV)
    kv_rows = torch.zeros(T, 2, Hkv, d, dtype=torch.bfloat16, device=DEV)
    gq, gk = (torch.zeros(T, Hk, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    gv = torch.zeros(T, Hv, d, dtype=torch.bfloat16, device=DEV)
    beta, g = torch.zeros(T, Hv, device=DEV), torch.zeros(T, Hv, device=DEV)
    o, og = torch.zeros(T, Hq, d, device=DEV), torch.zeros(T, Hv, d, device=DEV)

    def draw(seed):
        a = slots_inputs(T, Hk, Hv, d, d, 1, torch.bfloat16, seed)
        for dst, src in zip((gq, gk, gv, beta, g), a):
            dst.copy_(src)
        q.copy_(torch.randn(T, Hq, d, generator=_gen(seed + 1), device=DEV))
        kv_rows.copy_(torch.randn(T, 2, Hkv, d, generator=_gen(seed + 2), device=DEV))

    def step(max_q):
        S.gdn_plan_batch(ctx, new, table, free, count, bs, plan)
        S.gdn_kv_append(cache, kv_rows[:, 0], kv_rows[:, 1], plan.slot_map)
        S.gdn_kv_attn(cache, q, table, plan.cu_seqlens, plan.kv_lens, max_q_len=max_q, scale=0.125, o=o)
        S.gdn_decode_slots(gq, gk, gv, beta, g, state, slots, plan.cu_seqlens, o=og, scale=0.125)
        ctx.copy_(plan.kv_lens)

    def check():
        assert lib.gdn_sync_status() == 0
        cu, kv = plan.cu_seqlens.tolist(), plan.kv_lens.tolist()
        t = cu[-1]
        assert plan.info[2].item() == 0 and (plan.slot_map[t:] == -1).all()
        ro, _, A, ds, _ = attn_ref(cache, q[:t], table.tolist(), cu, kv, 0, 0.125)
        assert ((o[:t].double().cpu() - ro).abs() <= 2.0 ** -24 * ro.abs() + A * (2 * ds[..., None] + 2.0 ** -18)).all()
        for n in range(N):
            log[n] += [tuple(x[r].clone() for x in (gq, gk, gv, beta, g)) for r in range(cu[n], cu[n + 1])]
            if cu[n + 1] > cu[n]:
                cols = [torch.stack(c) for c in zip(*log[n])]
                r, rs = slots_ref(*cols, torch.zeros(1, Hv, d, d), [0], [0, len(log[n])], 0.125)
                m = cu[n + 1] - cu[n]
                assert close(og[cu[n]:cu[n + 1]], r[-m:], len(log[n]))
                assert close(state[slots[n]][None], rs, len(log[n]))

    draw(100)
    step(33)
    check()
    # the delta-rule layer's prompt rows through the packed prefill, with the plan's offsets: the same states
    cu = plan.cu_seqlens
    t = cu[-1].item()
    hq, hk, hv = (x[:t].transpose(0, 1).repeat_interleave(r, 0).contiguous() for x, r in ((gq, 2), (gk, 2), (gv, 1)))
    sf = torch.zeros(N, Hv, d, d, device=DEV)
    lib.gdn_chunk_fwd_varlen(hq.float(), hk.float(), hv.float(), beta[:t].T.contiguous(), cu, g[:t].T.contiguous(), s_final=sf,
                             scale=0.125)
    assert lib.gdn_sync_status() == 0
    assert (sf - state[slots.long()]).abs().max() <= 1e-4 * sf.abs().max()
    new.copy_(i32([1, 2, 1, 1]))
    draw(200)
    step(2)
    check()
    graph = torch.cuda.CUDAGraph()
    saved = [x.clone() for x in (state, ctx, table, free, count, cache.k.view(torch.uint8), cache.v.view(torch.uint8),
                                 cache.k_scale, cache.v_scale)]
    with torch.cuda.graph(graph):
        step(2)
    for x, y in zip((state, ctx, table, free, count, cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale,
                     cache.v_scale), saved):
        assert torch.equal(x, y)                             # capture runs nothing
    for i in range(8):
        draw(300 + 10 * i)
        if i == 4:                                           # request 2 finishes
            new.copy_(i32([1, 1, -1, 2]))
            before = count.item()
            log[2] = []
        elif i == 5:                                         # and another takes its place
            state[3].zero_()
            new.copy_(i32([2, 1, 2, 1]))
        graph.replay()
        check()
        if i == 4:
            assert count.item() >= before + 1 and table[2].tolist() == [-1] * mb
