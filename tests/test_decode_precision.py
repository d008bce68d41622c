"""How exactly the 8-bit decode holds a softmax weight, apart from what scores and outputs round.

The weight w <= 256 of a token is a sum of e4m3 parts, t1 + t2 / 32 + t3 / 32^2 + t4 / 32^3, each
the rounding of 32 times what the ones before left. A rounding is off by at most 2^-4 of its binade's
lower end, so 2^-4 of w after the first part and 2^-5 of that after each further one: 2^-19 w. Below
e4m3's normal range it is off by 2^-10, so 2^-10 / 32^3 = 2^-25 at most, and the reference's own
weight is 2^5.

The GPU tests choose q with one dimension that is not zero, so that a score is one product, and
compare with the output rounded once: |got - ref| <= half a step of bf16 at ref + what the weights
may be off.
"""
import numpy as np
import pytest
import torch

import fp8_util as f8
import workloads as w
from gpu_util import dev, host_f64
from libbuild import build_and_import

pkv = build_and_import()
D = 128
U = 2.0 ** -24


def parts(x, n):
    """The sum of n e4m3 parts of x (float64), and x's distance from it."""
    rest, total = x, np.zeros_like(x)
    for i in range(n):
        t = f8.VALUES[f8.encode(rest)]
        total = total + t * 32.0 ** -i
        rest = 32.0 * (rest - t)
    return total, np.abs(x - total)


def test_four_parts_hold_a_weight():
    g = w.rng(1)
    x = np.concatenate([np.linspace(0, 256, 300001), 2.0 ** g.uniform(-40, 8, 300000),
                        2.0 ** np.arange(-30, 9), 33.033 * 2.0 ** np.arange(-8, 3)])
    x = x.astype(np.float32).astype(np.float64)
    _, off = parts(x, 4)
    assert (off <= np.maximum(2.0 ** -19 * x, 2.0 ** -25)).all()
    # three are off by more than 2^-15 here and there, which four never are
    _, off = parts(x, 3)
    assert (off > np.maximum(2.0 ** -15 * x, 2.0 ** -20)).any()


def half_step(x):
    """Half a step of bf16 at x."""
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 8)


def _one_dim_case(ctx, hq, hkv, seed, pow2):
    """Contexts whose scores are single products: q = +-1.5, 1, .. in dimension h of its head."""
    g = w.rng(seed)
    bs = 256
    tables, nb = f8.tables_for(ctx, bs, g)
    codes, scales = [], []
    for _ in range(2):
        c, s = f8.random_cache(nb, bs, hkv, g)
        if not pow2:
            s = (s * g.uniform(0.5, 2.0, s.shape)).astype(np.float32).astype(np.float64)
        codes.append(c)
        scales.append(s)
    q = np.zeros((len(ctx), hq, D))
    for b in range(len(ctx)):
        for h in range(hq):
            q[b, h, (7 * b + 5 * h) % D] = g.choice([-1.5, -1.0, -0.75, 0.5, 1.0, 1.25])
    return tables, codes, scales, q


def _reference(ctx, tables, codes, scales, q, scale, hkv, tiles):
    """Output in 64 bits, and by how much it may be off before its rounding."""
    B, hq, _ = q.shape
    out, pre = np.zeros((B, hq, D)), np.zeros((B, hq, D))
    ones = np.full_like(codes[1], 0x38)
    c = np.float64(np.float32(scale)) * np.log2(np.e)
    for b, n in enumerate(ctx):
        k, v = (f8.rows(codes[i], scales[i], tables[b], n) for i in range(2))
        vs_all = f8.rows(ones, scales[1], tables[b], n)[:, :, 0]
        for j in range(hq):
            h = j * hkv // hq
            x = c * (k[:, h] @ q[b, j])
            vs = vs_all[:, h]
            y = x + np.log2(vs)
            p = np.exp2(x - x.max())
            p /= p.sum()
            # the score: softmax scale x log2(e), its product with q's power of two and with K's
            # scale, and the last product round (4 U |x|); log2 of V's scale and its sum with the
            # score, the reference and its difference (4 roundings at the largest of them); exp2,
            # log2 and the reciprocal are within 2^-22 each
            ds = 5 * U * np.abs(x).max() + 4 * U * np.abs(y).max() + 2.0 ** -22
            e = 2 * np.log(2) * ds + 4 * 2.0 ** -22
            # every sum of weights and of their products with V in fp32: a unit's tiles
            e += 2 * (tiles + 8) * U + tiles * 4 * 2.0 ** -23
            out[b, j] = p @ v[:, h]
            pre[b, j] = (2.0 ** -19 + e) * (p @ np.abs(v[:, h])) + \
                2.0 ** -30 * (p * vs).max() * (np.abs(v[:, h]) / vs[:, None]).sum(0)
    return out, pre


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(16, 8), (8, 2), (16, 2)])
@pytest.mark.parametrize("pow2", [True, False])
def test_outputs_are_rounded_once(hq, hkv, pow2):
    """Short contexts, where the weights' roundings do not average out; scales that the store
    writes, and others."""
    ctx = [1, 2, 3, 4, 5, 6, 7, 9, 12, 17, 33, 64, 65, 130] * 3
    scale = 0.05
    tables, codes, scales, q = _one_dim_case(ctx, hq, hkv, 40 + hq + pow2, pow2)
    (kc, ks), (vc, vs) = (f8.device_cache(*p) for p in zip(codes, scales))
    out = pkv.paged_decode_attn_fp8(dev(w.f32_to_bf16_bits(q.astype(np.float32))), kc, vc, ks, vs,
                                    dev(tables), dev(np.array(ctx, np.int32)), max(ctx), scale,
                                    num_splits=1)
    ref, pre = _reference(ctx, tables, codes, scales, q, scale, hkv, tiles=2)
    bad = np.abs(host_f64(out) - ref) > half_step(ref) + pre
    assert not bad.any(), f"{bad.sum()} of {bad.size} outputs are not the rounded ones"


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 1), (8, 1)])
def test_a_long_tail_of_small_weights(hq, hkv):
    """One token without a value takes nearly all of the weight, as the first token of a text does;
    131071 others of 2^-24.5 each make the output, in one split. The weights' absolute error adds up
    over them: it has to stay what it is said to be."""
    n, bs = 131072, 256
    nb = n // bs
    codes = np.zeros((2, nb, bs, hkv, D), np.uint8)
    codes[0, ..., 0] = f8.encode(np.array(-12.0))      # K: a score of -12.28 but for the first token
    codes[0, 0, 0, :, 0] = f8.encode(np.array(12.0))
    codes[1] = f8.encode(np.array(448.0))
    codes[1, 0, 0] = 0
    q = np.zeros((1, hq, D))
    q[..., 0] = 1.0234375                             # (8 bits: 131 / 128)
    scales = np.ones((2, nb, hkv, bs // 64))
    tables = np.arange(nb, dtype=np.int32)[None]
    scale = float(np.float32(np.log(2.0)))
    (kc, ks), (vc, vs) = (f8.device_cache(*p) for p in zip(codes, scales))
    out = pkv.paged_decode_attn_fp8(dev(w.f32_to_bf16_bits(q.astype(np.float32))), kc, vc, ks, vs,
                                    dev(tables), dev(np.array([n], np.int32)), n, scale,
                                    num_splits=1)
    d = 24.0 * 1.0234375 * np.float64(np.float32(scale)) * np.log2(np.e)
    p = np.exp2(-d)
    ref = 448.0 * (n - 1) * p / (1 + (n - 1) * p)
    # the sums of 1024 tiles in fp32 (U a tile, 2^-23 a product of 32 tokens) and the score's roundings
    e = 2 * 1032 * U + 4096 * 2.0 ** -23 + 2 * np.log(2) * 9 * U * d + 2.0 ** -19
    tol = half_step(ref) + e * ref + 2.0 ** -30 / (1 + (n - 1) * p) * 448.0 * (n - 1)
    assert np.abs(host_f64(out) - ref).max() <= tol, (host_f64(out)[0, :, 0], ref, tol)
