"""The 8-bit cache with scales that are no powers of two, as another program may have written them:
decode attention in every launch form with its weights, the gather, the store after such rows and the
eviction."""
import numpy as np
import pytest
import torch

import fp8_util as f8
import workloads as w
from gpu_util import dev, host_f64
from libbuild import build_and_import
from test_decode_fp8 import Case, check_out, check_weights

pkv = build_and_import()
D = 128


@pytest.fixture
def any_scales(monkeypatch):
    """Random caches whose scales are any float32."""
    powers = f8.random_cache

    def cache(nb, bs, hkv, g, spread=2.0):
        codes, scale = powers(nb, bs, hkv, g, spread)
        scale = scale * g.uniform(0.5, 2.0, scale.shape)
        return codes, scale.astype(np.float32).astype(np.float64)

    monkeypatch.setattr(f8, "random_cache", cache)


def rounds_to(got, x, scale, what):
    """The codes `got` are e4m3 of x / scale but for a quotient computed in fp32 (2^-22 of it)."""
    y = np.clip(x / scale, -448, 448)
    best = np.abs(f8.VALUES[f8.encode(y)] - y)
    off = np.abs(f8.VALUES[got] - y)
    assert (off <= best + 2.0 ** -21 * np.abs(y)).all(), what


# (a score's own error, 140 U A in the log2 domain with A > 1 for these inputs, covers the
# logarithm and the reciprocal of a scale, 2^-20)
@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(16, 8), (8, 2), (16, 2)])
def test_decode(any_scales, hq, hkv):
    c = Case([1, 2, 63, 64, 65, 130, 0, 257, 700, 1025], hq, hkv, 256, 1100 + hq)
    ref, tol, ws, wtol = c.reference()
    for splits in (0, 1, 3, 9):
        check_out(c.run(num_splits=splits), ref, tol, f"splits {splits}")
        weights = torch.zeros((10, hkv, 1025), device="cuda")
        check_out(c.run(num_splits=splits, weights=weights), ref, tol, f"splits {splits}, weights")
        check_weights(weights, torch.zeros_like(weights), ws, wtol, c.ctx)
    assert pkv.get_device_errors() == 0


@pytest.mark.gpu
def test_gather(any_scales):
    """code * scale, rounded to bf16 (from its rounding to fp32)."""
    g = w.rng(1110)
    lens = [300, 1, 64, 700]
    tables, nb = f8.tables_for(lens, 256, g)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    codes, scale = f8.random_cache(nb, 256, 3, g)
    kc, ks = f8.device_cache(codes, scale)
    out, _ = pkv.kv_gather_fp8(kc, kc, ks, ks, dev(tables), dev(cu), int(cu[-1]))
    want = np.concatenate([f8.rows(codes, scale, t, n) for t, n in zip(tables, lens)])
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -126))) - 8)
    off = np.abs(host_f64(out) - want) > step + 2.0 ** -24 * np.abs(want)
    assert not (off & ~np.isnan(want)).any()


@pytest.mark.gpu
@pytest.mark.parametrize("decode", [True, False])
def test_store_after_such_rows(any_scales, decode):
    """Appending to a group of any scale: the larger of it and the new rows' power of two."""
    g = w.rng(1120)
    hkv, bs, start = 2, 256, np.array([10, 64, 100, 255, 300])
    B = len(start)
    tables, nb = f8.tables_for(start + 1, bs, g)
    codes, scale = f8.random_cache(nb, bs, hkv, g)
    kc, ks = f8.device_cache(codes, scale)
    vc, vs = f8.device_cache(codes, scale)
    x = w.f32_to_bf16_bits((np.exp(3 * g.standard_normal((B, 1, 1))) *
                            g.standard_normal((B, hkv, D))).astype(np.float32))
    cu = None if decode else dev(np.arange(B + 1, dtype=np.int32))
    pkv.kv_store_fp8(dev(x), dev(x), dev((start + 1).astype(np.int32)), dev(tables), kc, vc, ks, vs,
                     cu_seqlens=cu)
    x = w.bf16_bits_to_f32(x).astype(np.float64)
    kc, ks = f8.host_codes(kc), ks.cpu().numpy().astype(np.float64)
    grown = 0
    for b, p in enumerate(start):
        blk, off, grp = int(tables[b, p // bs]), p % bs, p % bs // 64
        for h in range(hkv):
            old, new = scale[blk, h, grp], f8.scale_of(x[b:b + 1, h])
            s = max(old, new) if off % 64 else new
            assert ks[blk, h, grp] == s
            rounds_to(kc[blk, off, h], x[b, h], s, (b, h))
            before = slice(off - off % 64, off)
            rounds_to(kc[blk, before, h], f8.VALUES[codes[blk, before, h]] * old, s, (b, h, "before"))
            grown += s > old and off % 64 > 0
    assert grown                                          # (some scales had to grow)
    assert np.array_equal(f8.host_codes(vc), kc)


@pytest.mark.gpu
def test_evict(any_scales):
    g = w.rng(1130)
    hkv, bs, n, budget = 2, 256, 500, 150
    tables, nb = f8.tables_for([n, budget], bs, g)
    pools = [f8.random_cache(nb, bs, hkv, g) for _ in range(2)]
    (kc, ks), (vc, vs) = (f8.device_cache(*p) for p in pools)
    kept, _, _ = pkv.kv_evict(torch.rand((1, hkv, n), device="cuda"),
                              torch.tensor([n], dtype=torch.int32, device="cuda"), n,
                              dev(np.ascontiguousarray(tables[:1])),
                              dev(np.ascontiguousarray(tables[1:])), budget, 30, kc, vc, ks, vs)
    kept = kept.cpu().numpy()[0]
    dst = int(tables[1, 0])
    for (codes, scale), c, s in zip(pools, (kc, vc), (ks, vs)):
        c, s = f8.host_codes(c), s.cpu().numpy().astype(np.float64)
        for h in range(hkv):
            blk, off = tables[0, kept[h] // bs], kept[h] % bs
            mine = scale[blk, h, off // 64]
            for j in range(0, budget, 64):
                top = mine[j:j + 64].max()
                assert s[dst, h, j // 64] == top
                at = slice(j, min(j + 64, budget))
                rounds_to(c[dst, at, h], f8.VALUES[codes[blk[at], off[at], h]] * mine[at][:, None],
                          top, (h, j))
