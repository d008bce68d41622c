"""Decode attention where a cache holds values that are not finite."""
import numpy as np
import pytest
import torch

import workloads as w
from libbuild import build_and_import
from test_decode_fp8 import Case

pkv = build_and_import()
D = 128


def _positions(c):
    """Places in the V rows of c's contexts: (sequence, position, KV head, dimension)."""
    g = w.rng(11)
    for b, n in enumerate(c.ctx):
        for _ in range(3 if n else 0):
            yield b, int(g.integers(n)), int(g.integers(c.hkv)), int(g.integers(D))


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(4, 4), (4, 2), (6, 2), (8, 2), (10, 2)])
@pytest.mark.parametrize("many", [False, True])
def test_infinite_values_on_the_bf16_cache_with_weights(hq, hkv, many):
    """An infinite V makes its dimension infinite, or NaN where the other infinity is there too, as
    in paged_decode_attn; every other output and every weight is as without it."""
    ctx = [1, 2, 65, 200, 0, 300, 64, 513]
    c = Case(ctx * 40 if many else ctx, hq, hkv, 256, 600 + hq, fp8=False)
    args = c.device()
    flat = args[2].view(-1, hkv, D)
    want = np.zeros((len(c.ctx), hkv, D))          # 0: finite
    rows = []
    for i, (b, pos, h, d) in enumerate(_positions(c)):
        row = int(c.tables[b, pos // 256]) * 256 + pos % 256
        if (row, h, d) in rows:
            continue
        rows.append((row, h, d))
        sign = 1.0 if i % 4 else -1.0
        d2 = d if i % 5 else 17                      # (some meet in one dimension)
        if (row, h, d2) in rows[:-1]:
            continue
        rows[-1] = (row, h, d2)
        flat[row, h, d2] = sign * float("inf")
        if want[b, h, d2] not in (0.0, sign):
            sign = 2.0                               # NaN
        want[b, h, d2] = sign
    want = torch.from_numpy(np.repeat(want, hq // hkv, axis=1)).cuda()
    assert (want == 1).any() and (want == -1).any()
    finite = list(args)
    finite[2] = torch.where(args[2].isinf(), 1.0, args[2])
    longest = int(max(c.ctx))
    for splits in (0, 1, 3, 9):
        w0, w1 = (torch.zeros((len(c.ctx), hkv, longest), device="cuda") for _ in range(2))
        out = c.run(args, num_splits=splits, weights_out=w0)
        ref = c.run(finite, num_splits=splits, weights_out=w1)
        assert torch.equal(w0, w1)
        assert torch.equal(out[want == 0], ref[want == 0])
        assert (out[want == 1] == float("inf")).all()
        assert (out[want == -1] == -float("inf")).all()
        assert out[want == 2].isnan().all()
        plain = pkv.paged_decode_attn(*args, num_splits=splits)
        assert torch.equal(plain.isinf(), out.isinf()) and torch.equal(plain.isnan(), out.isnan())
    assert pkv.get_device_errors() == 0
