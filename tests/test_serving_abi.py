"""Argument checks of the serving calls: what the C ABI and the binding refuse, on the host (no GPU: every call
here returns before any CUDA work)."""
import ctypes

import pytest
import torch

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_sequence_b200 import build
    build.build()
    from gated_deltanet_sequence_b200 import _lib
    return _lib


def _plan(lib, **kw):
    a = dict(ctx=FAKE, new=FAKE, N=2, table=FAKE, mb=4, free=FAKE, count=FAKE, nb=8, bs=16, T=4, cu=FAKE, kv=FAKE,
             pos=FAKE, seq=FAKE, slot=FAKE, info=FAKE)
    a.update(kw)
    return lib.lib.gdn_plan_batch(P(a["ctx"]), P(a["new"]), a["N"], P(a["table"]), a["mb"], P(a["free"]), P(a["count"]),
                                  a["nb"], a["bs"], a["T"], P(a["cu"]), P(a["kv"]), P(a["pos"]), P(a["seq"]), P(a["slot"]),
                                  P(a["info"]), None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=0), 1), (dict(T=-1), 1), (dict(mb=0), 1), (dict(nb=0), 1), (dict(ctx=None), 1), (dict(new=FAKE + 2), 1),
    (dict(table=None), 1), (dict(free=None), 1), (dict(count=FAKE + 1), 1), (dict(cu=None), 1), (dict(kv=None), 1),
    (dict(slot=None), 1), (dict(info=None), 1), (dict(bs=48), 2), (dict(bs=8), 2), (dict(N=8193), 2),
    (dict(T=(1 << 30) + 1), 2), (dict(nb=1 << 27, bs=16), 1), (dict(mb=1 << 27, bs=16), 1),
])
def test_plan_rejects_bad_arguments(lib, kw, want):
    assert _plan(lib, **kw) == want


def _append(lib, **kw):
    a = dict(k=FAKE, v=FAKE, ks=256, vs=256, slot=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, T=4, H=2, d=128, nb=8, bs=16,
             dt=1)
    a.update(kw)
    return lib.lib.gdn_kv_append(P(a["k"]), P(a["v"]), a["ks"], a["vs"], P(a["slot"]), P(a["kc"]), P(a["vc"]), P(a["ksc"]),
                                 P(a["vsc"]), a["T"], a["H"], a["d"], a["nb"], a["bs"], a["dt"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(nb=0), 1), (dict(dt=4), 1), (dict(k=None), 1), (dict(v=FAKE + 8), 1),
    (dict(slot=FAKE + 2), 1), (dict(kc=FAKE + 4), 1), (dict(vsc=None), 1), (dict(ks=255), 1), (dict(vs=260), 1),
    (dict(vs=258, dt=0), 1), (dict(d=96), 2), (dict(bs=256), 2), (dict(H=65536), 2), (dict(nb=1 << 27), 1), (dict(T=0), 0),
])
def test_append_rejects_bad_arguments(lib, kw, want):
    assert _append(lib, **kw) == want


def _attn(lib, **kw):
    a = dict(q=FAKE, qs=512, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, table=FAKE, cu=FAKE, kv=FAKE, o=FAKE, lse=None, ws=FAKE,
             wsb=1 << 40, N=2, T=4, Hq=4, Hkv=2, d=128, nb=8, bs=16, mb=4, mq=2, window=0, scale=1.0, dt=1, odt=0)
    a.update(kw)
    return lib.lib.gdn_kv_attn(P(a["q"]), a["qs"], P(a["kc"]), P(a["vc"]), P(a["ksc"]), P(a["vsc"]), P(a["table"]),
                               P(a["cu"]), P(a["kv"]), P(a["o"]), P(a["lse"]), P(a["ws"]), a["wsb"], a["N"], a["T"],
                               a["Hq"], a["Hkv"], a["d"], a["nb"], a["bs"], a["mb"], a["mq"], a["window"], a["scale"],
                               a["dt"], a["odt"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=0), 1), (dict(T=-1), 1), (dict(Hkv=0), 1), (dict(Hq=1), 1), (dict(Hq=5), 1), (dict(mq=0), 1), (dict(mb=0), 1),
    (dict(window=-1), 1), (dict(scale=float("inf")), 1), (dict(dt=2), 1), (dict(odt=3), 1), (dict(q=None), 1),
    (dict(o=FAKE + 8), 1), (dict(qs=508), 1), (dict(qs=513), 1), (dict(lse=FAKE + 2), 1), (dict(ws=None), 1),
    (dict(wsb=16), 1), (dict(kc=FAKE + 8), 1), (dict(table=FAKE + 1), 1), (dict(d=256), 2), (dict(bs=24), 2),
    (dict(Hq=65536, Hkv=2, qs=65536 * 128), 2), (dict(nb=1 << 26), 1), (dict(mb=1 << 27), 1), (dict(T=0), 0),
])
def test_attn_rejects_bad_arguments(lib, kw, want):
    assert _attn(lib, **kw) == want


def test_attn_rejects_tables_whose_positions_pass_32_bits(lib):
    """The kernels look a few thousand positions past a context's end: max_blocks * block_size <= 2^31 - 2^16."""
    for bs in (16, 128):
        most = (2 ** 31 - 2 ** 16) // bs
        assert _attn(lib, mb=most, bs=bs, T=0) == 0 and _attn(lib, mb=most + 1, bs=bs, T=0) == 1


def test_attn_workspace_size(lib):
    size = lib.lib.gdn_kv_attn_workspace_bytes
    assert size(1, 1, 8, 2, 128, 1) > 0 and size(1, 1, 8, 2, 128, 1) % 16 == 0
    assert size(0, 1, 8, 2, 128, 1) == size(1, 1, 7, 2, 128, 1) == size(1, 1, 8, 2, 96, 1) == size(1, 1, 8, 2, 64, 0) == 0


def _slots(lib, opts=None, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=256, ks=256, vs=512, beta=None, g=None, state=FAKE, slots=FAKE, cu=None, o=FAKE,
             N=4, T=4, Hk=2, Hv=4, ns=8, dk=128, dv=128, scale=1.0, dt=1)
    a.update(kw)
    return lib.lib.gdn_decode_slots(P(a["q"]), P(a["k"]), P(a["v"]), a["qs"], a["ks"], a["vs"], P(a["beta"]), P(a["g"]),
                                    P(a["state"]), P(a["slots"]), P(a["cu"]), P(a["o"]), a["N"], a["T"], a["Hk"], a["Hv"],
                                    a["ns"], a["dk"], a["dv"], a["scale"], a["dt"],
                                    None if opts is None else ctypes.byref(opts), None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=0), 1), (dict(T=-1, cu=FAKE), 1), (dict(T=5), 1), (dict(Hk=0), 1), (dict(Hv=3), 1), (dict(Hv=1), 1),
    (dict(ns=0), 1), (dict(scale=float("nan")), 1), (dict(dt=2), 1), (dict(q=None), 1), (dict(state=FAKE + 4), 1),
    (dict(slots=None), 1), (dict(cu=FAKE + 2), 1), (dict(beta=FAKE + 1), 1), (dict(qs=255), 1), (dict(vs=511), 1),
    (dict(o=FAKE + 8), 1), (dict(dk=96), 2), (dict(dv=32), 2), (dict(Hv=131072, vs=131072 * 128), 2),
    (dict(T=0, cu=FAKE), 0),
])
def test_slots_rejects_bad_arguments(lib, kw, want):
    assert _slots(lib, **kw) == want


def test_slots_rejects_bad_options(lib):
    assert _slots(lib, lib.FwdOpts(5)) == 1
    assert _slots(lib, lib.FwdOpts(0, FAKE + 2)) == 1
    assert _slots(lib, lib.FwdOpts(0, None, 2)) == 1
    assert _slots(lib, lib.FwdOpts(0, None, 0, 1, None, 0.0)) == 1       # eps 0


def test_binding_refuses():
    from gated_deltanet_sequence_b200 import serving as S
    f8 = torch.zeros(3, 2, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc = torch.ones(3, 2)
    with pytest.raises(TypeError):                   # not e4m3
        S.KvCache(torch.zeros(3, 2, 16, 64), f8, sc, sc)
    with pytest.raises(ValueError):                  # block size
        S.KvCache(f8[:, :, :8], f8, sc, sc)
    with pytest.raises(ValueError):                  # scales are (num_blocks, Hkv)
        S.KvCache(f8, f8, sc, sc[:2])
    with pytest.raises(ValueError):                  # not contiguous
        S.KvCache(f8, f8, sc, torch.ones(2, 3).T)
    cache = S.KvCache(f8, f8, sc, sc)
    k = torch.zeros(5, 2, 64)
    slot = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError):                  # shapes differ
        S.gdn_kv_append(cache, k, k[:4], slot)
    with pytest.raises(TypeError):                   # types differ
        S.gdn_kv_append(cache, k, k.bfloat16(), slot)
    with pytest.raises(TypeError):
        S.gdn_kv_append(cache, k, k, slot.long())
    with pytest.raises(TypeError):                   # neither bf16 nor fp32: checked before any launch
        S.gdn_kv_append(cache, k.half(), k.half(), slot)
    with pytest.raises(ValueError):                  # heads of a row are not contiguous
        S.gdn_kv_append(cache, torch.zeros(5, 64, 2).transpose(1, 2), k, slot)
    with pytest.raises(ValueError):                  # rows overlap
        S.gdn_kv_append(cache, torch.zeros(1, 2, 64).expand(5, 2, 64), k, slot)
    with pytest.raises(ValueError):                  # CPU tensors
        S.gdn_kv_append(cache, k, k, slot)
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):                  # head size of the cache
        S.gdn_kv_attn(cache, torch.zeros(5, 4, 128), i(2, 3), i(3), i(2))
    with pytest.raises(ValueError):                  # 3 query heads over 2 KV heads
        S.gdn_kv_attn(cache, torch.zeros(5, 3, 64), i(2, 3), i(3), i(2))
    with pytest.raises(ValueError):
        S.gdn_kv_attn(cache, torch.zeros(5, 4, 64), i(2, 3), i(4), i(2))
    with pytest.raises(TypeError):
        S.gdn_kv_attn(cache, torch.zeros(5, 4, 64), i(2, 3), i(3), i(2), out_dtype=torch.float16)
    p = S.BatchPlan.empty(2, 5, "cpu")
    with pytest.raises(ValueError):
        S.gdn_plan_batch(i(3), i(2), i(2, 3), i(6), i(1), 16, p)
    with pytest.raises(TypeError):
        S.gdn_plan_batch(i(2), i(2).long(), i(2, 3), i(6), i(1), 16, p)
    st = torch.zeros(4, 2, 64, 64)
    with pytest.raises(ValueError):                  # rows without offsets
        S.gdn_decode_slots(k, k, k, None, None, st, i(4))
    with pytest.raises(ValueError):                  # value heads over key heads
        S.gdn_decode_slots(k, k, torch.zeros(5, 3, 64), None, None, torch.zeros(4, 3, 64, 64), i(5))
    with pytest.raises(ValueError):                  # state of other sizes
        S.gdn_decode_slots(k, k, k, None, None, torch.zeros(4, 2, 64, 128), i(5))


def test_workspace_size_is_each_device_s_own(monkeypatch):
    """The size goes by the SMs of the device that the call runs on, so one device's is not another's."""
    from gated_deltanet_sequence_b200 import serving as S
    now = [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.back, now[0] = now[0], self.index

        def __exit__(self, *a):
            now[0] = self.back

    class Lib:
        calls = 0

        @staticmethod
        def gdn_kv_attn_workspace_bytes(N, T, Hq, Hkv, d, max_q_len):
            Lib.calls += 1
            return 1000 * (1 + now[0]) + N

    monkeypatch.setattr(S, "lib", Lib)
    monkeypatch.setattr(S, "_device_now", lambda: now[0])
    monkeypatch.setattr(S.torch.cuda, "device", Device)
    monkeypatch.setattr(S.torch.cuda, "is_available", lambda: True)
    S._workspace_bytes.cache_clear()
    try:
        size = S.gdn_kv_attn_workspace_bytes
        for _ in range(2):
            assert size(3, 3, 8, 2, 128) == 1003 and size(3, 3, 8, 2, 128, device="cuda:1") == 2003
            assert size(3, 3, 8, 2, 128, device="cuda") == 1003 and now == [0]
            now[0] = 2
            assert size(3, 3, 8, 2, 128) == 3003 and size(3, 3, 8, 2, 128, device=torch.device("cuda", 0)) == 1003
            assert now == [2]
            now[0] = 0
        assert Lib.calls == 3
    finally:
        S._workspace_bytes.cache_clear()
