"""The serving calls at the ends of their range: buffers of calls on several streams, blocks and weights whose sizes lie
far apart, values that are not finite, tensors that a step hands to the next one. References and the reasons for their
tolerances are those of test_serving_gpu.py, with what a test adds written beside it."""
import math

import pytest
import torch

from test_serving_gpu import (DEV, S, _gen, attn_case, attn_check, attn_ref, behind, close, i32, lib, make_cache,  # noqa: F401
                              plan_ref, slots_inputs, slots_ref)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- streams
def test_attn_buffers_of_a_passed_stream_are_that_streams_own(S, lib):
    """A long call on the current stream, whose workspace is returned to torch's pool while it still runs, and calls on
    side streams at once, nothing waited for: each makes its own workspace, o and lse."""
    kv, ql = [60000, 50000, 40000, 30000], [1] * 4
    cache, q, table, tab, cu = attn_case(S, kv, ql, 4, 8, 128, 64, torch.bfloat16, seed=15)
    cu_t, kv_t = i32(cu), i32(kv)
    other = i32([x // 3 for x in kv])
    kw = dict(scale=0.09, lse=True)
    want = [S.gdn_kv_attn(cache, q, tab, cu_t, k, **kw) for k in (kv_t, other)]
    side = [torch.cuda.Stream() for _ in range(2)]
    handles = [side[0], side[1].cuda_stream, None]
    torch.cuda.synchronize()
    for turn in range(6):
        outs = []
        for i in range(6):
            st = handles[(i + turn) % 3]
            k = i & 1
            outs.append((k, S.gdn_kv_attn(cache, q, tab, cu_t, (kv_t, other)[k], stream=st, **kw)))
        torch.cuda.synchronize()
        for k, (o, lse) in outs:
            assert torch.equal(o, want[k][0]) and torch.equal(lse, want[k][1]), turn
    assert lib.gdn_sync_status() == 0


def test_results_of_a_passed_stream_outlast_their_reader(S, lib):
    """A result made on a side stream, read by queued work of the current one and dropped: its memory is not given to the
    side stream's next call before that work is through."""
    N, H, d = 64, 8, 128
    q, k, v, beta, g, state = slots_inputs(N, H, H, d, d, N, torch.bfloat16, seed=2)
    slots = i32(list(range(N)))
    states = [state.clone() for _ in range(3)]
    want = S.gdn_decode_slots(q, k, v, beta, g, states[0], slots)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o = S.gdn_decode_slots(q, k, v, beta, g, states[1], slots, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20_000_000)                       # about 10 ms before the copy
    got = torch.empty_like(o)
    got.copy_(o)
    del o
    for _ in range(3):
        S.gdn_decode_slots(q, k, v, None, None, states[2], slots, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and lib.gdn_sync_status() == 0


def test_the_default_stream_by_its_handle(S, lib):
    kv, ql = [300, 40], [1, 1]
    cache, q, table, tab, cu = attn_case(S, kv, ql, 2, 2, 64, 16, torch.bfloat16, seed=16)
    a = S.gdn_kv_attn(cache, q, tab, i32(cu), i32(kv), scale=0.125, lse=True)
    b = S.gdn_kv_attn(cache, q, tab, i32(cu), i32(kv), scale=0.125, lse=True, stream=0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and lib.gdn_sync_status() == 0


def test_calls_on_a_forked_stream_are_captured(S, lib):
    """A graph whose capture forks: attention and recurrence side by side on two streams, results and workspaces made in
    the calls, replayed with other inputs."""
    kv, ql = [900, 70, 2000], [1, 2, 1]
    cache, q, table, tab, cu = attn_case(S, kv, ql, 2, 4, 128, 64, torch.bfloat16, seed=18)
    cu_t, kv_t = i32(cu), i32(kv)
    gq, gk, gv, beta, g, state = slots_inputs(4, 2, 4, 64, 64, 3, torch.bfloat16, seed=19)
    slots, start = i32([2, 0, 1]), state.clone()

    def both(side):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        o, lse = S.gdn_kv_attn(cache, q, tab, cu_t, kv_t, max_q_len=2, scale=0.09, lse=True, stream=side)
        r = S.gdn_decode_slots(gq, gk, gv, beta, g, state, slots, cu_t)
        p, _ = S.gdn_kv_attn(cache, q, tab, cu_t, kv_t, max_q_len=2, scale=0.05)
        here.wait_stream(side)
        return o, lse, r, p

    side = torch.cuda.Stream()
    both(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(side)
    for turn in range(3):
        q.copy_(torch.randn(q.shape, generator=_gen(turn), device=DEV))
        state.copy_(start)
        for x in got:
            x.fill_(5.0)
        graph.replay()
        after = state.clone()
        state.copy_(start)
        want = both(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(after, state), turn
    assert lib.gdn_sync_status() == 0


# ---------------------------------------------------------------- V's block scales
def unit_case(S, scales, n, Hkv, G, d, bs, dtype, seed, positive=True, ql=1):
    """One request of n tokens whose blocks' V scales go through `scales` in turn (a block of zeros where that is None),
    V of one sign, so that sums grow with the tokens."""
    cache, q, table, tab, cu = attn_case(S, [n], [ql], Hkv, G, d, bs, dtype, seed)
    v = cache.v.float()
    if positive:
        cache.v.copy_(v.abs().clamp(min=1.0).to(cache.v.dtype))
    for i, b in enumerate(table[0]):
        e = scales[i % len(scales)]
        if e is None:
            cache.v.view(torch.uint8)[b] = 0
        cache.v_scale[b] = 2.0 ** (-100 if e is None else e)
    return cache, q, table, tab, cu


UNITS = {  # exponents of V's block scales; None: a block of zeros
    "zeros behind 2^20": [20, None, None],
    "zeros behind 2^40": [40, None, None],
    "zeros first": [None, None, 30, None, -20],
    "falling": [90, 60, 30, 0, -30, -60, -90],
    "rising": [-90, -30, 30, 90],
    "both ends": [100, -100, 20, -100],
}


@pytest.mark.parametrize("case", list(UNITS))
@pytest.mark.parametrize("n,bs,d,dtype,out", [
    (4000, 64, 128, torch.bfloat16, torch.bfloat16), (4000, 16, 128, torch.bfloat16, torch.float32),
    (700, 16, 64, torch.float32, torch.float32), (3000, 32, 64, torch.float32, torch.bfloat16),
    (200, 16, 64, torch.bfloat16, torch.bfloat16), (2500, 128, 128, torch.float32, torch.float32)])
def test_attn_v_scales_of_the_whole_range(S, lib, case, n, bs, d, dtype, out):
    """gdn_kv_append makes scales of 2^-100 (a block of zeros) to 2^120: sums in units of one block's scale must neither
    overflow nor be lost when the next block's lies far below or above."""
    cache, q, table, tab, cu = unit_case(S, UNITS[case], n, 2, 4, d, bs, dtype, seed=40)
    attn_check(S, lib, cache, q, table, tab, cu, [n], 0, 0.02, out)


@pytest.mark.parametrize("case", list(UNITS))
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 64)])
def test_attn_prompt_v_scales_of_the_whole_range(S, lib, case, d, bs):
    """The same where the many-rows kernel looks at the request first and leaves it."""
    cache, q, table, tab, cu = unit_case(S, UNITS[case], 500, 2, 2, d, bs, torch.bfloat16, seed=41, ql=120)
    attn_check(S, lib, cache, q, table, tab, cu, [500], 0, 0.02, torch.bfloat16, pad=9000)


@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                       (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("far", [40, 64, 80])
def test_attn_small_values_beside_large_ones_without_weight(S, lib, far, dtype, out):
    """Every other block holds values 2^far larger whose weights vanish (200 nats below): the result is the small
    values' alone. Beyond 2^64 the small blocks' weights take the rest of the power of two, 2^-16 here: as fp16 they
    are then within 2^-25 / 2^-16 = 2^-9 each of the largest weight, as two parts within 2^-21."""
    n, bs, d = 1600, 16, 64
    cache, q, table, tab, cu = unit_case(S, [far - 40, -40], n, 1, 4, d, bs, dtype, seed=42)
    q.copy_(torch.where(q > 0, 1.0, -1.0))
    q[:, 1:] = q[:, :1]                                       # one sign pattern: a key along it scores far below
    big = torch.tensor(table[0][0::2], device=DEV)
    k = cache.k.float()
    k[big] = -448.0 * q[0, 0].float()
    cache.k.copy_(k.to(cache.k.dtype))
    cache.k_scale.fill_(2.0 ** -7)                            # scale 0.9: 0.9 * 64 * 3.5 = 201 below
    scale = 0.9
    cache.k_scale[torch.tensor(table[0][1::2], device=DEV)] = 2.0 ** -12
    q0 = q.clone()
    o, lse = S.gdn_kv_attn(cache, q0, tab, i32(cu), i32([n]), scale=scale, out_dtype=out, lse=True)
    assert lib.gdn_sync_status() == 0
    ro, rl, A, ds, vm = attn_ref(cache, q0, table, cu, [n], 0, scale, dtype == out == torch.bfloat16)
    assert ro.abs().max() < 448 * 2.0 ** -40
    rel = 2.0 ** -8 if out == torch.bfloat16 else 2.0 ** -24
    part = (2.0 ** -11 if out == torch.bfloat16 else 2.0 ** -22) + 2.0 ** -20
    if far > 64:
        part += 2.0 ** -9 if out == torch.bfloat16 else 2.0 ** -21
    tol = rel * ro.abs() + A * (2 * ds[..., None] + part + n * 2.0 ** -23)
    assert ((o.double().cpu() - ro).abs() <= tol).all()
    assert ((lse.double().cpu() - rl).abs() <= ds + 2.0 ** -20 + n * 2.0 ** -23 + 2.0 ** -22 * rl.abs()).all()


# ---------------------------------------------------------------- plan
def plan_call(S, lib, ctx, new, table, free, count, bs, T, ctx_of=None):
    """gdn_plan_batch on lists; ctx_of: makes the cached lengths' tensor from the plan (the plan's own kv_lens)."""
    p = S.BatchPlan.empty(len(ctx), T, DEV)
    c = i32(ctx) if ctx_of is None else ctx_of(p).copy_(i32(ctx))
    t, f, n = i32(table), i32(free), i32([count])
    S.gdn_plan_batch(c, i32(new), t, f, n, bs, p)
    st = lib.gdn_sync_status()
    got = {k: getattr(p, k).tolist() for k in ("cu_seqlens", "kv_lens", "positions", "seq_ids", "slot_map", "info")}
    got.update(table=t.tolist(), free=f.tolist())
    assert n.item() == got["info"][3]
    return got, st


def plan_state(ctx, bs, mb, spare):
    """Tables with the cached tokens' blocks, numbered in order, and a free list of the others."""
    table, at = [], 0
    for c in ctx:
        k = -(-c // bs)
        table.append(list(range(at, at + k)) + [-1] * (mb - k))
        at += k
    return table, list(range(at, at + spare)) + [-1] * at, spare


@pytest.mark.parametrize("N", [33, 700, 3000])
def test_plan_of_a_refused_step_has_its_lengths(S, lib, N):
    """More tokens than the grid has rows: info[1] is the longest cached length, with nothing of the refused tokens in it,
    whichever warp comes last (the long request is each warp's in turn)."""
    bs, mb = 16, 20
    for at in (0, 31, N // 2, N - 1):
        ctx = [(7 * i) % 50 for i in range(N)]
        new = [3] * N
        ctx[at], new[at] = 10, 300
        table, free, count = plan_state(ctx, bs, mb, 4)
        want, bad = plan_ref(ctx, new, table, free, count, bs, 3 * N)
        for _ in range(5):
            got, st = plan_call(S, lib, ctx, new, table, free, count, bs, 3 * N)
            assert bad and st == lib.GDN_ERR_INVALID_ARG and got == want and got["info"][1] == 49


def test_plan_refuses_a_step_with_bad_lengths_too(S, lib):
    """More tokens than rows, and among the requests some whose own lengths are out of range and a finished one."""
    ctx, new = [5, 20, 70, -3, 9, 0], [30, -2, 5, 1, -1, 0]
    table, free, count = plan_state([5, 20, 0, 0, 9, 0], 16, 4, 6)
    want, bad = plan_ref(ctx, new, table, free, count, 16, 8)
    got, st = plan_call(S, lib, ctx, new, table, free, count, 16, 8)
    assert bad and st == lib.GDN_ERR_INVALID_ARG and got == want and got["kv_lens"] == [5, 0, 0, 0, 0, 0]


@pytest.mark.parametrize("N,top,bs", [(5, 3, 16), (300, 2, 32), (40, 400, 64), (2000, 9, 16)])
def test_plan_takes_its_own_kv_lens_as_cached_lengths(S, lib, N, top, bs):
    """A program that hands the plan's kv_lens on as the next step's cached lengths: the same tensor read and written."""
    g = torch.Generator().manual_seed(N)
    mb = -(-(40 + 8 * top) // bs) + 1
    ctx = torch.randint(0, 41, (N,), generator=g).tolist()
    table, free, count = plan_state(ctx, bs, mb, N * mb)
    rows = N * top + 5                                       # N = 40: the tokens' own kernel; the others one block
    p = S.BatchPlan.empty(N, rows, DEV)
    p.kv_lens.copy_(i32(ctx))
    t, f, c = i32(table), i32(free), i32([count])
    for step in range(6):
        new = torch.randint(0, top + 1, (N,), generator=g)
        if step == 3:
            new[torch.rand(N, generator=g) < 0.2] = -1
        new = new.tolist()
        want, bad = plan_ref(ctx, new, table, free, count, bs, rows)
        S.gdn_plan_batch(p.kv_lens, i32(new), t, f, c, bs, p)
        assert not bad and lib.gdn_sync_status() == 0
        for k in ("cu_seqlens", "kv_lens", "positions", "seq_ids", "slot_map", "info"):
            assert getattr(p, k).tolist() == want[k], (step, k)
        assert t.tolist() == want["table"] and f.tolist() == want["free"]
        ctx, table, free, count = want["kv_lens"], want["table"], want["free"], want["info"][3]
    S.gdn_plan_batch(p.kv_lens, i32([top + 2] * N), t, f, c, bs, p)      # more tokens than rows: the lengths stay
    assert lib.gdn_sync_status() == lib.GDN_ERR_INVALID_ARG
    assert p.kv_lens.tolist() == ctx and t.tolist() == table and p.info.tolist() == [0, max(ctx), 0, count]


# ---------------------------------------------------------------- queries that are not finite
@pytest.mark.parametrize("dtype,out,pad", [(torch.bfloat16, torch.bfloat16, 0), (torch.bfloat16, torch.float32, 0),
                                           (torch.float32, torch.float32, 0), (torch.float32, torch.bfloat16, 0),
                                           (torch.bfloat16, torch.bfloat16, 9000)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_attn_of_a_query_that_is_not_finite_is_nan(S, lib, dtype, out, pad, sign, value):
    """Whatever the signs of the codes it meets: with codes of one sign all scores are the same infinity, and a row whose
    scores are all -inf must not pass for one that sees nothing. Rows that do see nothing stay 0."""
    kv, ql, d = [150, 90, 2], [70, 1, 5], 64
    cache, q, table, tab, cu = attn_case(S, kv, ql, 2, 2, d, 16, dtype, seed=50)
    k = cache.k.float()
    k[..., 7] = sign * k[..., 7].abs().clamp(min=1.0)
    cache.k.copy_(k.to(cache.k.dtype))
    q[3, 1, 7] = q[70, 3, 7] = q[71, 0, 7] = q[74, 2, 7] = value       # (row 71 is before position 0)
    want = torch.zeros(q.shape[:2], dtype=torch.bool)
    want[3, 1] = want[70, 3] = want[74, 2] = True
    n = q.shape[0]
    o, lse = S.gdn_kv_attn(cache, behind(q, pad), tab, i32(cu), i32(kv), max_q_len=70, scale=0.125, out_dtype=out, lse=True)
    assert lib.gdn_sync_status() == 0
    assert torch.equal(torch.isnan(o[:n]).all(-1).cpu(), want) and torch.equal(torch.isnan(o[:n]).any(-1).cpu(), want)
    assert torch.equal(torch.isnan(lse[:n]).cpu(), want)
    assert (o[71:74] == 0).all() and (lse[71:74] == -math.inf).all()


# ---------------------------------------------------------------- weights far below the largest
@pytest.mark.parametrize("nats", [10, 20, 25])
@pytest.mark.parametrize("d,bs,dtype", [(128, 64, torch.bfloat16), (64, 16, torch.float32), (64, 32, torch.bfloat16)])
@pytest.mark.parametrize("n", [600, 6000])
def test_attn_fp32_output_keeps_small_weights(S, lib, n, d, bs, dtype, nats):
    """One token `nats` above thousands of others, itself with a V of zeros: the others' weights, down to 2^-36 of
    the largest, carry the whole result. Two fp16 parts, the second 2^12 larger, of weights that start at 2^7: the
    smallest half step is 2^-25 2^-12 2^-7 = 2^-44 of the largest weight for each token, beside the tolerance of
    the other fp32 outputs."""
    cache, q, table, tab, cu = attn_case(S, [n], [1], 2, 4, d, bs, dtype, seed=60)
    g = _gen(61)
    q.copy_(torch.where(torch.randn(1, 2, 1, d, generator=g, device=DEV) > 0, 1.0, -1.0).expand(1, 2, 4, d).reshape(1, 8, d))
    k = torch.randn(cache.k.shape, generator=g, device=DEV)
    at = 37                                               # the token above the others: its key lies along the queries
    b, r = table[0][at // bs], at % bs
    k[b, :, r] = 16.0 * q[0, ::4].float()
    cache.k.copy_(k.to(cache.k.dtype))
    cache.k_scale.fill_(1.0)
    v = cache.v.float().abs().clamp(min=1.0)
    v[b, :, r] = 0.0
    cache.v.copy_(v.to(cache.v.dtype))
    cache.v_scale.fill_(2.0 ** -8)
    scale = nats / (16.0 * d)
    o, lse = S.gdn_kv_attn(cache, q, tab, i32(cu), i32([n]), scale=scale, lse=True)
    assert lib.gdn_sync_status() == 0
    ro, rl, A, ds, vm = attn_ref(cache, q, table, cu, [n], 0, scale)
    tol = 2.0 ** -24 * ro.abs() + A * (2 * ds[..., None] + 2.0 ** -21 + 2.0 ** -22 + min(n * 2.0 ** -23, 2.0 ** -11))
    tol = tol + n * 2.0 ** -44 * vm[..., None]
    err = (o.double().cpu() - ro).abs()
    assert (err <= tol).all(), (err / tol).max()
    assert ((lse.double().cpu() - rl).abs() <= ds + 2.0 ** -20 + n * 2.0 ** -23 + 2.0 ** -22 * rl.abs()).all()


# ---------------------------------------------------------------- positions at the ends of their range
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_attn_windows_near_2_to_31(S, lib, out):
    """The widest window that a table still outgrows, and 70000 rows of which all but three lie before position 0."""
    n, kv, d, bs = 70000, 3, 64, 16
    cache, q, table, tab, cu = attn_case(S, [kv], [n], 1, 1, d, bs, torch.bfloat16, seed=70)
    wide = torch.full((1, (2 ** 31 - 2 ** 16) // bs), -1, dtype=torch.int32, device=DEV)
    wide[:, :tab.shape[1]] = tab
    kw = dict(max_q_len=n, scale=0.125, out_dtype=out, lse=True)
    want = S.gdn_kv_attn(cache, q, wide, i32(cu), i32([kv]), **kw)
    got = S.gdn_kv_attn(cache, q, wide, i32(cu), i32([kv]), window=2 ** 31 - 2 ** 16 - 1, **kw)
    assert lib.gdn_sync_status() == 0
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    o, lse = got
    assert (o[:-kv] == 0).all() and (lse[:-kv] == -math.inf).all() and torch.isfinite(lse[-kv:]).all()
    one = S.gdn_kv_attn(cache, q[-kv:], tab, i32([0, kv]), i32([kv]), max_q_len=kv, scale=0.125, lse=True)
    assert (o[-kv:].float() - one[0]).abs().max() <= 2.0 ** -7 * one[0].abs().max()
    assert (lse[-kv:] - one[1]).abs().max() <= 2.0 ** -18


def test_attn_over_the_longest_context(S, lib):
    """2^31 - 2^16 tokens, one block of 128 named throughout: the result of that block alone, its lse with log n more.
    Each of a warp's 57000 steps adds a rounding of 2^-24 to sums that it carries: 2^-8 at the worst."""
    n, d, bs = 2 ** 31 - 2 ** 16, 64, 128
    cache, q, table, tab, cu = attn_case(S, [bs], [1], 1, 8, d, bs, torch.bfloat16, seed=71)
    long = torch.full((1, n // bs), table[0][0], dtype=torch.int32, device=DEV)
    one = S.gdn_kv_attn(cache, q, tab, i32(cu), i32([bs]), scale=0.125, lse=True)
    for window in (0, n - 1):
        o, lse = S.gdn_kv_attn(cache, q, long, i32(cu), i32([n]), scale=0.125, window=window, lse=True)
        assert lib.gdn_sync_status() == 0
        assert (o - one[0]).abs().max() <= 2.0 ** -7 * one[0].abs().max()
        assert (lse - one[1] - math.log(n // bs)).abs().max() <= 2.0 ** -7


@pytest.mark.parametrize("bs,d,dtype,out", [(16, 64, torch.float32, torch.float32), (16, 128, torch.bfloat16, torch.bfloat16),
                                            (64, 128, torch.bfloat16, torch.float32), (32, 64, torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("window", [1, 9, 40, 200])
def test_attn_blocks_before_the_window_do_not_set_the_unit(S, lib, bs, d, dtype, out, window):
    """Blocks that no row sees hold values 2^150 larger than those in the window, in every place that a window's start
    can have in a step: the result is as exact as without them."""
    for n in (431, 432, 440, 448, 449, 463, 511, 512):
        cache, q, table, tab, cu = unit_case(S, [-70], n, 1, 4, d, bs, dtype, seed=n)
        first = max(0, n - window) // bs
        for i, b in enumerate(table[0]):
            if i < first:
                cache.v_scale[b] = 2.0 ** 80
        attn_check(S, lib, cache, q, table, tab, cu, [n], window, 0.02, out)


@pytest.mark.parametrize("pad", [0, 9000])
@pytest.mark.parametrize("big,codes", [(-60, True), (-84, True), (-90, True), (-60, False)])
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 64)])
def test_attn_prompt_values_at_the_smallest_scale(S, lib, d, bs, big, codes, pad):
    """Blocks of append's smallest scale, 2^-100, that are not zeros, beside blocks of larger values: rows that see them
    alone have them in full. (Blocks of zeros there do not matter.)"""
    n = 300
    cache, q, table, tab, cu = unit_case(S, [big], n, 2, 2, d, bs, torch.bfloat16, seed=43, ql=n)
    for b in table[0][:64 // bs]:                        # the first 64 tokens: half of a unit of the many-rows kernel
        cache.v_scale[b] = 2.0 ** -100
        if not codes:
            cache.v.view(torch.uint8)[b] = 0
    attn_check(S, lib, cache, q, table, tab, cu, [n], 0, 0.02, torch.bfloat16, pad=pad)
