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
