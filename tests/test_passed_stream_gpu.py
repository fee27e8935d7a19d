"""Calls on a passed stream make their results on it: nothing that the current stream has queued (a fill of the result,
work that still uses memory which torch hands out again) reaches them. The current stream is kept busy meanwhile, and
nothing is waited for in between."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from gated_deltanet_sequence_b200 import _lib, workloads
    return _lib, workloads


@pytest.fixture(scope="module")
def calls(api):
    gdn, W = api
    p = W.make_prefill_inputs(2, 4, 200, 128, 128, mode="gdn", in_dtype=torch.bfloat16, s0=True, seed=1, device="cuda")
    v = W.make_varlen_inputs([70, 1, 130], 4, 128, 128, mode="gdn", in_dtype=torch.bfloat16, s0=True, seed=2, device="cuda")
    d = W.make_decode_inputs(8, 4, 128, 128, 1, seed=3, device="cuda")
    b = W.make_prefill_inputs(1, 2, 130, 64, 64, mode="gdn", in_dtype=torch.float32, s0=True, seed=4, device="cuda")
    d_o = torch.randn(1, 2, 130, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    states = [d["state"].clone() for _ in range(8)]
    return {
        "gdn_chunk_fwd": lambda **k: gdn.gdn_chunk_fwd(p["q"], p["k"], p["v"], p["beta"], p["g"], s0=p["s0"], **k)[0],
        "lin_attn_chunk_fwd": lambda **k: gdn.lin_attn_chunk_fwd(p["q"], p["k"], p["v"], p["g"], s0=p["s0"], **k)[0],
        "gdn_chunk_fwd_varlen": lambda **k: gdn.gdn_chunk_fwd_varlen(v["q"], v["k"], v["v"], v["beta"], v["cu_seqlens"], v["g"],
                                                                     s0=v["s0"], **k)[0],
        "lin_attn_chunk_fwd_varlen": lambda **k: gdn.lin_attn_chunk_fwd_varlen(v["q"], v["k"], v["v"], v["cu_seqlens"], v["g"],
                                                                               s0=v["s0"], **k)[0],
        "gdn_decode_step": lambda **k: gdn.gdn_decode_step(d["q"][0], d["k"][0], d["v"][0], d["beta"][0], d["g"][0],
                                                           states.pop(), **k),
        "gdn_chunk_bwd": lambda **k: torch.cat([x.reshape(-1) for x in gdn.gdn_chunk_bwd(
            b["q"], b["k"], b["v"], b["beta"], b["g"], d_o, s0=b["s0"], **k).values()]) if not k else gdn.gdn_chunk_bwd(
                b["q"], b["k"], b["v"], b["beta"], b["g"], d_o, s0=b["s0"], **k),
    }


@pytest.mark.parametrize("name", ["gdn_chunk_fwd", "lin_attn_chunk_fwd", "gdn_chunk_fwd_varlen", "lin_attn_chunk_fwd_varlen",
                                  "gdn_decode_step", "gdn_chunk_bwd"])
@pytest.mark.parametrize("handle", [False, True])
def test_results_are_made_on_the_passed_stream(api, calls, name, handle):
    gdn, _ = api
    f = calls[name]
    want = f()
    side = torch.cuda.Stream()
    f(stream=side)                                     # memory for the side stream and code are loaded before: both
    with torch.cuda.stream(side):                      # would wait for the device
        want.clone(), want.clone()
    junk = [torch.full_like(want, 2.0) for _ in range(4)]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                     # about 100 ms on the current stream ...
    for j in junk:
        j.fill_(3.0)                                   # ... before it writes memory that is torch's again
    del j, junk
    got = f(stream=side.cuda_stream if handle else side)
    side.synchronize()
    with torch.cuda.stream(side):
        early = {k: x.clone() for k, x in got.items()} if isinstance(got, dict) else got.clone()
    torch.cuda.synchronize()
    for r in (early, got):
        flat = torch.cat([x.reshape(-1) for x in r.values()]) if isinstance(r, dict) else r
        assert torch.equal(flat, want)
    assert gdn.gdn_sync_status() == 0
