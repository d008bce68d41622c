"""Decode attention where a cache holds values that are not finite, a table names blocks that do not
exist, or contexts are longer than the call says."""
import numpy as np
import pytest
import torch

import workloads as w
from libbuild import build_and_import
from test_decode_fp8 import Case, check_out, check_weights

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


def _bad_blocks(c, k_scale, v_scale):
    """Block ids outside the pool in c's tables, whose rows count as zeros, and a block 0 that no
    table names, with NaN codes and these scales."""
    g = w.rng(21)
    nb = c.tables.max() + 4
    c.tables = np.where(c.tables >= 0, c.tables + 1, -1).astype(np.int32)
    for i, pool in enumerate(c.pools):
        if c.fp8:
            codes, scale = pool
            nan, one = np.full_like(codes[:1], 0x7F), np.full_like(scale[:1], [k_scale, v_scale][i])
            c.pools[i] = np.concatenate([nan, codes]), np.concatenate([one, scale])
        else:
            c.pools[i] = np.concatenate([np.full_like(pool[:1], w.BF16_NAN_CANARY), pool])
    for b, n in enumerate(c.ctx):
        blocks = -(-int(n) // c.bs)
        for j in range(blocks):
            if b % 7 == 2 or g.random() < 0.4:       # (some sequences have no good block)
                c.tables[b, j] = [-1, 1 << 20, -(1 << 31), nb + 900][g.integers(4)]
                at = slice(j * c.bs, (j + 1) * c.bs)
                for i in range(2):
                    c.values[i][b][at] = 0.0
                if c.v_scale:
                    c.v_scale[b][at] = 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,fp8", [(16, 8, True), (8, 2, True), (16, 2, True), (8, 2, False)])
@pytest.mark.parametrize("k_scale,v_scale,many", [
    (np.nan, np.inf, False), (1.0, 2.0 ** 60, False), (np.inf, np.nan, False),
    (np.nan, np.inf, True)])
def test_bad_block_ids_are_zero_rows(hq, hkv, fp8, k_scale, v_scale, many):
    """Whatever block 0 holds: the rows of a bad id are zeros, with a score of zero and no value."""
    ctx = [700, 300, 300, 1, 257, 0, 513, 900, 65, 513]
    times = 1 + 320 // (10 * hkv) if many else 1    # (many: more units than CTAs)
    c = Case(ctx * times, hq, hkv, 256, 700 + hq, fp8=fp8)
    _bad_blocks(c, k_scale, v_scale)
    ref, tol, ws, wtol = c.reference()
    for splits in (0, 1) if many else (0, 1, 3, 9):
        weights = torch.zeros((len(c.ctx), hkv, 900), device="cuda")
        check_out(c.run(num_splits=splits, weights=weights), ref, tol, f"splits {splits}")
        check_weights(weights, torch.zeros_like(weights), ws, wtol, c.ctx)
        if fp8:
            check_out(c.run(num_splits=splits), ref, tol, f"splits {splits}, no weights")
        assert pkv.get_device_errors() == pkv.DEVERR_BLOCK_RANGE


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,fp8", [(16, 8, True), (16, 2, True), (4, 4, False), (8, 2, False)])
@pytest.mark.parametrize("longest,many", [(0, False), (1, False), (130, False), (500, False),
                                          (130, True)])
def test_contexts_above_the_longest(hq, hkv, fp8, longest, many):
    """A context above max_context_len is reported and counts as that many tokens, whatever its split
    would hold; weights past them are left alone."""
    times = 1 + 320 // (6 * hkv) if many else 1     # (many: more units than CTAs)
    c = Case([150, 3, 700, 130, 1, 0] * times, hq, hkv, 256, 800 + hq, fp8=fp8)
    args = c.device()
    at, cut = (6, 7) if fp8 else (4, 5)
    assert torch.equal(args[at].cpu(), torch.from_numpy(c.ctx).int())
    args[cut] = longest
    short = list(args)
    short[at] = args[at].clamp(max=longest)
    for splits in (0, 1) if many else (0, 1, 2, 9):
        w0, w1 = (torch.full((len(c.ctx), hkv, 800), 7.0, device="cuda") for _ in range(2))
        out = c.run(args, num_splits=splits, weights_out=w0)
        assert pkv.get_device_errors() == pkv.DEVERR_CONTEXT_RANGE
        ref = c.run(short, num_splits=splits, weights_out=w1)
        assert torch.equal(out, ref) and torch.equal(w0, w1)
        assert (w0[:, :, longest:] == 7).all()
        if fp8:
            out = c.run(args, num_splits=splits)
            assert pkv.get_device_errors() == pkv.DEVERR_CONTEXT_RANGE
            assert torch.equal(out, c.run(short, num_splits=splits))
        assert pkv.get_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("longest", [2 ** 31 - 1, 2 ** 31 - 128, 2 ** 31 - 129])
def test_no_bound_on_the_longest_context(fp8, longest):
    """max_context_len as large as an int: one split of that many tokens is not a multiple of a tile
    that an int holds."""
    c = Case([150, 3, 700, 0], 8, 2, 256, 900, fp8=fp8)
    args = c.device()
    args[7 if fp8 else 5] = longest
    out = c.run(args, num_splits=1) if fp8 else pkv.paged_decode_attn(*args, num_splits=1)
    ref, tol, _, _ = c.reference()
    # (the bf16 kernel rounds its weights to bf16, as it does their sum)
    more = 0 if fp8 else np.stack([
        np.abs(np.repeat(v, 4, axis=1)).max(axis=0, initial=0) for v in c.values[1]]) * 2.0 ** -8
    check_out(out, ref, tol + more)
    assert pkv.get_device_errors() == 0
