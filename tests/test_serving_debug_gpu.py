"""The serving calls on the bounds-checked debug build (libgdn_debug.so): the batch plan in both its forms, appends of
single rows, prompts and growing scales, attention in every form (cut, whole, cluster, many rows, windows, an fp32
output), the recurrence over slots. On valid calls it reports nothing and gives the release build's bits."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import sys, torch
sys.path.insert(0, sys.argv[1])
from gated_deltanet_sequence_b200 import _lib as gdn, serving as S
D = "cuda"
g = torch.Generator(D).manual_seed(5)
rand = lambda *s: torch.randn(*s, generator=g, device=D)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=D)
out, status = {}, {}

def steps(name, Hkv, G, d, bs, dtype, odt, news, window=0, mb=None, pad=3):
    """Steps of a batch through plan, append and attention; news: each step's new tokens."""
    N = len(news[0])
    total = [sum(max(n[r], 0) for n in news) for r in range(N)]
    mb = mb or max(-(-t // bs) for t in total) + 1
    nb = sum(-(-t // bs) for t in total) + N
    cache = S.KvCache.empty(nb, Hkv, bs, d, D)
    table = torch.full((N, mb), -1, dtype=torch.int32, device=D)
    free, count, ctx = i32(list(range(nb))), i32([nb]), i32([0] * N)
    for k, new in enumerate(news):
        T = sum(max(x, 0) for x in new) + pad
        plan = S.BatchPlan.empty(N, T, D)
        S.gdn_plan_batch(ctx, i32(new), table, free, count, bs, plan)
        x = rand(T, 3 * max(G, 1) * Hkv * d).to(dtype) * (1.0 + k)
        kk, vv = (x[:, j * Hkv * d:(j + 1) * Hkv * d].view(T, Hkv, d) for j in range(2))
        S.gdn_kv_append(cache, kk, vv, plan.slot_map)
        q = x[:, 2 * G * Hkv * d:].view(T, G * Hkv, d)
        o = torch.zeros(T, G * Hkv, d, dtype=odt, device=D)
        lse = torch.zeros(T, G * Hkv, device=D)
        S.gdn_kv_attn(cache, q, table, plan.cu_seqlens, plan.kv_lens, max_q_len=max(max(new), 1), window=window,
                      scale=d ** -0.5, o=o, lse=lse)
        ctx = plan.kv_lens.clone()
        out[f"{name} {k}"] = [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in (
            plan.cu_seqlens, plan.kv_lens, plan.positions, plan.seq_ids, plan.slot_map, plan.info, table.clone(),
            free.clone(), cache.k.clone(), cache.v.clone(), cache.k_scale.clone(), cache.v_scale.clone(), o, lse)]
    status[name] = gdn.gdn_sync_status()

bf, f32 = torch.bfloat16, torch.float32
steps("ragged", 2, 4, 128, 64, bf, bf, [[130, 1, 700, 64], [1, 1, 1, 1], [3, -1, 0, 2]])
steps("fp32", 2, 3, 64, 16, f32, f32, [[33, 5, 0, 900], [1, 2, 7, 1]], window=100)
steps("fp32 output", 1, 8, 128, 128, bf, f32, [[1200, 3], [1, 1]])
steps("one", 2, 4, 64, 16, bf, bf, [[700], [1]])
steps("one of few", 2, 4, 64, 32, bf, bf, [[90], [1]])
steps("many rows", 8, 4, 128, 16, bf, bf, [[420, 30, 0], [200, 1, 90], [1, 1, 1]])
steps("many rows 64", 4, 4, 64, 128, bf, bf, [[900, 300]], window=200)
steps("tokens of their own kernel", 1, 1, 64, 32, bf, f32, [[3000, 2000, 100], [1, -1, 5]])
for dk, dv, Hk, Hv, dt in ((128, 128, 2, 4, bf), (64, 128, 1, 3, f32), (128, 64, 2, 2, f32), (64, 64, 1, 1, bf)):
    T = 12
    q, k = ((lambda x: x / x.norm(dim=-1, keepdim=True))(rand(T, Hk, dk)).to(dt) for _ in range(2))
    state = rand(6, Hv, dk, dv)
    o = S.gdn_decode_slots(q, k, rand(T, Hv, dv).to(dt), torch.sigmoid(rand(T, Hv)), -rand(T, Hv).abs(), state,
                           i32([3, 5, -1, 0]), i32([0, 4, 5, 7, 12]), o=torch.zeros(T, Hv, dv, device=D))
    out[f"slots {dk} {dv}"] = [o, state]
status["slots"] = gdn.gdn_sync_status()
torch.save({"status": status, "lib": gdn.LIB_PATH, "out": {k: [t.cpu() for t in v] for k, v in out.items()}}, sys.argv[2])
'''


def _run(tmp_path, debug):
    env = dict(os.environ)
    env.pop("GDN_LIBRARY", None)
    if debug:
        env["GDN_LIBRARY"] = "debug"
    path = str(tmp_path / ("debug.pt" if debug else "release.pt"))
    subprocess.run([sys.executable, "-c", CHILD, ROOT, path], env=env, check=True, timeout=600)
    return torch.load(path)


def test_serving_calls_on_the_debug_build(tmp_path):
    dbg, rel = _run(tmp_path, True), _run(tmp_path, False)
    assert dbg["lib"].endswith("libgdn_debug.so") and rel["lib"].endswith("libgdn.so")
    assert set(dbg["status"].values()) == {0} and set(rel["status"].values()) == {0}, (dbg["status"], rel["status"])
    assert dbg["out"].keys() == rel["out"].keys() and len(rel["out"]) == 21
    for k in rel["out"]:
        for i, (a, b) in enumerate(zip(dbg["out"][k], rel["out"][k])):
            assert torch.equal(a, b), f"{k}, output {i}: debug and release builds differ"
