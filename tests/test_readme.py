"""README's step over an 8-bit cache with eviction, run as it stands there."""
import os
import re

import numpy as np
import pytest
import torch

import fp8_util as f8
import workloads as w
from gpu_util import dev, host_f64
from libbuild import ROOT, build_and_import

pkv = build_and_import()
D = 128


def step_source():
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    (code,) = [b for b in blocks if "kv_evict" in b]
    return code


def test_the_step_is_python():
    compile(step_source(), "README.md", "exec")


@pytest.mark.gpu
def test_steps_before_and_after_an_eviction():
    """Four steps, an eviction after the second and the third: every output is attention over the rows
    that the tables hold by then, and the weights of new tokens start from nothing."""
    g = w.rng(1000)
    hq, hkv, bs, budget, capacity = 8, 2, 256, 64, 400
    lens = [300, 90, 20]
    B = len(lens)
    bm = pkv.BlockManager(16, bs)
    tables = np.full((B, 2), -1, np.int32)
    for t, n in zip(tables, lens):
        need = -(-(n + 4) // bs)
        t[:need] = bm.take(need)
    kc, ks = f8.device_cache(*f8.random_cache(16, bs, hkv, g))
    vc, vs = f8.device_cache(*f8.random_cache(16, bs, hkv, g))
    names = dict(pkv=pkv, torch=torch, bm=bm, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs,
                 scale=D ** -0.5, budget=budget, recent=8, cu_seqlens=None, blocks_needed=B,
                 tables=dev(tables), acc=torch.zeros((B, hkv, capacity), device="cuda"),
                 context_lens=dev(np.array(lens, np.int32) + 1), max_context_len=max(lens) + 1)
    code = compile(step_source(), "README.md", "exec")
    for step in range(4):
        names["over_budget"] = step in (1, 2)
        for n, heads in (("q", hq), ("k", hkv), ("v", hkv)):
            names[n] = dev(w.host_bf16_normal(g, (B, heads, D)))
        if names["over_budget"]:     # (a table as wide as the sequences will need)
            fresh = np.full((B, 2), -1, np.int32)
            fresh[:, 0] = bm.take(B)
            names["fresh_tables"] = dev(fresh)
        before = names["acc"].clone()
        had, at = names["context_lens"].tolist(), names["tables"].cpu().numpy()
        exec(code, names)
        out, acc = host_f64(names["out"]), names["acc"]
        q = host_f64(names["q"])
        total = np.zeros((B, hkv))
        for b, n in enumerate(had):
            K, V = (f8.rows(f8.host_codes(c), s.cpu().numpy().astype(np.float64), at[b], n)
                    for c, s in ((kc, ks), (vc, vs)))
            for h in range(hq):
                x = D ** -0.5 * K[:, h // 4] @ q[b, h]
                p = np.exp(x - x.max())
                p /= p.sum()
                ref, size = p @ V[:, h // 4], p @ np.abs(V[:, h // 4])
                # the output's rounding, the weights' parts and the scores' fp32 sums
                assert (np.abs(out[b, h] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * size).all()
            total[b] = before[b, :, :n].double().sum(-1).cpu().numpy() + 4
        now = names["context_lens"].tolist()
        assert now == [min(n, budget) if names["over_budget"] else n for n in had]
        assert names["max_context_len"] == max(now)
        for b, n in enumerate(now):
            assert (acc[b, :, n:] == 0).all()               # the next tokens' columns
            kept = acc[b, :, :n].double().sum(-1).cpu().numpy()
            # (a step's fp32 weights add up to their 4 heads within 1e-5; what is dropped is the
            # smallest, which may be less than that)
            if names["over_budget"] and had[b] > budget:
                assert (kept <= total[b] * (1 + 1e-5)).all()
            else:
                assert np.allclose(kept, total[b], rtol=1e-5)
        names["context_lens"] += 1                          # the next token
        names["max_context_len"] += 1
    assert pkv.get_device_errors() == 0
