"""Attention of drafted tokens over the paged cache (bf16 and 8-bit) against 64 bits."""
import numpy as np
import pytest
import torch

from libbuild import build_and_import
from tree_util import Case, D, NAN8, assert_close, bf16_weights, ints, rows_of

pkv = build_and_import()
pytestmark = pytest.mark.gpu
BOTH = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])


def check(c, **kw):
    pkv.get_device_errors(reset=True)
    out = c.attend(pkv, **kw)
    ref, size = c.reference()
    n = sum(c.nodes)
    assert_close(out[:n], ref[:n], size[:n], c.fp8, bf16_weights(c.most, c.hq // c.hkv))
    assert pkv.get_device_errors(reset=True) == 0
    return out


@BOTH
@pytest.mark.parametrize("kind", ["chain", "tree", "random", "all"])
def test_small_batch(kind, fp8):
    check(Case([1, 5, 64, 100, 256, 300], [1, 5, 3, 8, 7, 1], 16, 8, kind=kind, fp8=fp8, seed=1))


@BOTH
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (6, 2), (4, 1), (5, 1), (6, 1), (14, 2), (16, 2),
                                    (16, 1), (20, 1), (33, 1), (32, 32)])
def test_head_groups(hq, hkv, fp8):
    check(Case([70, 333], [9, 21], hq, hkv, fp8=fp8, seed=2))


@BOTH
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257,
                               511, 513, 767, 1025])
def test_lengths(L, fp8):
    n = min(L, 6)
    check(Case([L, L + 3, L], [n, min(L + 3, 9), 1], 8, 4, fp8=fp8, seed=L))


@BOTH
@pytest.mark.parametrize("n,hq,hkv", [(16, 16, 2), (17, 16, 2), (33, 8, 2), (63, 4, 2), (64, 16, 2),
                                      (65, 8, 2), (100, 6, 2), (130, 8, 1), (200, 16, 1), (300, 3, 1)])
def test_many_nodes(n, hq, hkv, fp8):
    check(Case([n, n + 40, n + 700], [n, n - 1, n], hq, hkv, kind="tree", fp8=fp8, seed=n))


@BOTH
def test_many_nodes_of_one_sequence_only(fp8):
    check(Case([900, 1300, 40, 700], [2, 64, 1, 9], 16, 2, fp8=fp8, seed=7))


@BOTH
def test_blocks_of_512(fp8):
    check(Case([600, 1200], [10, 3], 8, 4, bs=512, fp8=fp8, seed=8))


@BOTH
def test_long_contexts(fp8):
    check(Case([9000, 20011], [13, 30], 8, 2, fp8=fp8, seed=9))


@BOTH
def test_one_long_context_with_one_node(fp8):
    check(Case([17188], [1], 2, 1, fp8=fp8, seed=10))


@BOTH
def test_ragged_batch(fp8):
    rng = np.random.default_rng(5)
    nodes = [int(x) for x in rng.integers(0, 9, 200)]
    ctx = [n + int(x) for n, x in zip(nodes, rng.integers(0, 700, 200))]
    check(Case(ctx, nodes, 16, 8, fp8=fp8, seed=11))


@BOTH
def test_many_sequences(fp8):
    rng = np.random.default_rng(6)
    nodes = [int(x) for x in rng.integers(0, 4, 1500)]
    ctx = [n + int(x) for n, x in zip(nodes, rng.integers(0, 60, 1500))]
    check(Case(ctx, nodes, 4, 2, fp8=fp8, seed=12))


@BOTH
def test_empty_rows_and_empty_contexts(fp8):
    c = Case([4, 0, 9], [4, 0, 9], 4, 2, kind="random", fp8=fp8, seed=13)
    out = check(c)
    blind = torch.from_numpy(np.concatenate([~m.any(axis=1) for m in c.masks])).cuda()
    assert blind.any() and (out[blind] == 0).all()


@BOTH
def test_strided_q_and_rows_behind_the_last_sequence(fp8):
    c = Case([130, 300], [6, 11], 6, 2, fp8=fp8, seed=14, stride_pad=2 * 2 * D, tail=5)
    out = torch.full((22, 6, D), 7.0, dtype=torch.bfloat16, device="cuda")
    check(c, out=out)
    assert (out[17:] == 7).all()


@BOTH
def test_large_scores(fp8):
    """Scores of some hundreds: one weight of nearly 1, maxima that move from tile to tile."""
    c = Case([700, 5000], [5, 12], 8, 2, fp8=fp8, seed=15, mag=1.0)
    c.q = (c.q.float() * 12).to(torch.bfloat16)
    pkv.get_device_errors(reset=True)
    out = c.attend(pkv)
    ref, size = c.reference()
    # scores twelve times as large: errors of a weight too
    bound = 2.0 ** -8 * ref.abs() + 2.0 ** -6 * size
    assert ((out.double() - ref).abs() <= bound).all()


@BOTH
def test_rising_scores(fp8):
    """The largest scores come last, so that every tile moves the running maximum."""
    c = Case([1500], [8], 4, 2, kind="chain", fp8=fp8, seed=16)
    L = 1500
    ramp = torch.linspace(0.05, 1.5, L, device="cuda")
    flat = torch.from_numpy(rows_of(c.table_host[0], L, 256)).cuda()
    direction = torch.ones((D,), device="cuda")
    rows = (ramp[:, None, None] * direction).expand(L, 2, D)
    if fp8:
        c.k.view(torch.uint8).view(-1, 2, D)[flat] = (rows * 100).to(torch.float8_e4m3fn).view(torch.uint8)
        c.scales[0].copy_(torch.where(torch.isnan(c.scales[0]), c.scales[0], 2.0 ** -7))
    else:
        c.k.view(-1, 2, D)[flat] = rows.to(torch.bfloat16)
    c.q = (c.q.float().abs()).to(torch.bfloat16)
    check(c)


@BOTH
def test_shared_prefix_blocks(fp8):
    c = Case([600, 600, 600], [5, 7, 2], 8, 4, fp8=fp8, seed=17)
    t = c.table_host
    t[1, :2] = t[2, :2] = t[0, :2]
    c.tables = torch.from_numpy(t).cuda()
    check(c)


@BOTH
def test_not_finite_values_of_nodes_reach_those_that_see_them_only(fp8):
    c = Case([80, 200, 20], [6, 40, 20], 4, 2, kind="tree", fp8=fp8, seed=18)
    # siblings of every tree that some nodes see and others do not
    marks = [(0, 3), (1, 17), (1, 30), (2, 19)]
    for b, node in marks:
        pos = c.ctx[b] - c.nodes[b] + node
        blk, off = int(c.table_host[b, pos // 256]), pos % 256
        for name in ("k", "v"):
            pool = getattr(c, name)
            if fp8:
                pool.view(torch.uint8)[blk, off, :, 5::40] = NAN8
            else:
                pool[blk, off, :, 5::40] = float("nan") if node % 2 else float("inf")
    pkv.get_device_errors(reset=True)
    out = c.attend(pkv)
    t = 0
    clean = Case([80, 200, 20], [6, 40, 20], 4, 2, kind="tree", fp8=fp8, seed=18)
    ref, size = clean.reference()
    for b, n in enumerate(c.nodes):
        hit = np.zeros(n, bool)
        for bb, node in marks:
            if bb == b:
                hit |= c.masks[b][:, node]
        assert hit.any() and not hit.all()
        free = torch.from_numpy(~hit).cuda()
        assert_close(out[t:t + n][free], ref[t:t + n][free], size[t:t + n][free], fp8)
        assert torch.isnan(out[t:t + n][~free]).all()  # (K is not finite either)
        t += n
    # V alone: only its dims are hit
    c.k = clean.k
    out = c.attend(pkv)
    t = 0
    for b, n in enumerate(c.nodes):
        hit = np.zeros(n, bool)
        for bb, node in marks:
            if bb == b:
                hit |= c.masks[b][:, node]
        bad = torch.zeros((n, 4, D), dtype=torch.bool, device="cuda")
        bad[torch.from_numpy(hit).cuda(), :, 5::40] = True
        assert (~torch.isfinite(out[t:t + n]) == bad).all()
        assert_close(out[t:t + n][~bad], ref[t:t + n][~bad], size[t:t + n][~bad], fp8)
        t += n
    assert pkv.get_device_errors(reset=True) == 0


@BOTH
def test_a_nan_in_the_context_reaches_every_node(fp8):
    c = Case([300, 90], [4, 3], 4, 2, fp8=fp8, seed=19)
    blk, off = int(c.table_host[0, 0]), 37
    if fp8:
        c.v.view(torch.uint8)[blk, off, 1, 11] = NAN8
    else:
        c.v[blk, off, 1, 11] = float("nan")
    out = c.attend(pkv)
    bad = torch.isnan(out)
    want = torch.zeros_like(bad)
    want[:4, 2:, 11] = True
    assert (bad == want).all()


@BOTH
def test_bad_lengths_and_blocks(fp8):
    c = Case([300, 200, 520, 100, 80], [4, 3, 5, 6, 2], 4, 2, fp8=fp8, seed=20)
    ref, size = c.reference()
    # a context shorter than its tree, and one longer than the table
    c.lens = ints([300, 2, 520, 5000, 80])
    pkv.get_device_errors(reset=True)
    out = torch.full((20, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    c.attend(pkv, out=out)
    assert pkv.get_device_errors(reset=True) == pkv.DEVERR_CONTEXT_RANGE
    assert (out[4:7] == 0).all() and (out[12:18] == 0).all()
    keep = [*range(4), *range(7, 12), 18, 19]
    assert_close(out[keep], ref[keep], size[keep], fp8)
    # a bad block in the middle counts as zeros; the others do not notice
    c.lens = ints(c.ctx)
    was = c.table_host[2, 1]
    for bad in (-1, c.nb):
        c.tables[2, 1] = bad
        out = c.attend(pkv)
        assert pkv.get_device_errors(reset=True) == pkv.DEVERR_BLOCK_RANGE
        assert torch.isfinite(out).all()
        keep = [*range(7), *range(12, 20)]
        assert_close(out[keep], ref[keep], size[keep], fp8)
    c.tables[2, 1] = int(was)
    # a cu_seqlens entry past the rows, one that decreases, more nodes than max_seqlen_q
    for cu, keep in (([0, 4, 7, 12, 18, 25], range(18)), ([0, 4, 2, 12, 18, 20], [*range(4), 18, 19])):
        c.cu = ints(cu)
        out.fill_(7.0)
        c.attend(pkv, out=out)
        assert pkv.get_device_errors(reset=True) & pkv.DEVERR_SEQLEN_RANGE
        keep = list(keep)
        assert_close(out[keep], ref[keep], size[keep], fp8)
    c.cu = ints([0, 4, 7, 12, 18, 20])
    c.most = 5
    out.fill_(7.0)
    c.attend(pkv, out=out)
    assert pkv.get_device_errors(reset=True) == pkv.DEVERR_SEQLEN_RANGE
    assert (out[12:18] == 7).all()


@BOTH
def test_other_stream_and_given_outputs(fp8):
    c = Case([500, 90], [4, 9], 8, 2, fp8=fp8, seed=21)
    ref, size = c.reference()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = pkv.tree_workspace(2, c.most, 8, 2, D, 500, stream=s)
    ws.fill_(255)
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty((13, 8, D), dtype=torch.bfloat16, device="cuda")
    got = c.attend(pkv, out=out, workspace=ws, stream=s)
    assert got is out
    s.synchronize()
    assert_close(out, ref, size, fp8)


@BOTH
def test_same_bits_again_and_in_a_graph(fp8):
    c = Case([5000, 90, 1200], [14, 9, 3], 16, 2, fp8=fp8, seed=22)
    first = c.attend(pkv)
    for _ in range(3):
        assert torch.equal(c.attend(pkv), first)
    out = torch.empty_like(first)
    ws = pkv.tree_workspace(3, c.most, 16, 2, D, 5000)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attend(pkv, out=out, workspace=ws)
        second = c.attend(pkv)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(second, first)
    # other lengths on the same graph
    lens = [4000, 70, 30]
    c.lens.copy_(ints(lens))
    graph.replay()
    torch.cuda.synchronize()
    c.ctx = lens
    ref, size = c.reference()
    assert_close(out, ref, size, fp8)


@BOTH
def test_placement_of_blocks_does_not_count(fp8):
    c = Case([700, 300], [6, 8], 8, 4, fp8=fp8, seed=23)
    first = c.attend(pkv)
    perm = torch.randperm(c.nb, device="cuda")
    inv = torch.argsort(perm)
    if fp8:
        c.k = c.k.view(torch.uint8)[perm].view(torch.float8_e4m3fn)
        c.v = c.v.view(torch.uint8)[perm].view(torch.float8_e4m3fn)
        c.scales = tuple(s[perm].contiguous() for s in c.scales)
    else:
        c.k, c.v = c.k[perm].contiguous(), c.v[perm].contiguous()
    c.tables = torch.where(c.tables >= 0, inv[c.tables.clamp(min=0).long()].int(), c.tables)
    assert torch.equal(c.attend(pkv), first)


@BOTH
def test_offsets_past_32_bits(fp8):
    """Blocks whose values lie past 2^32 bytes of the pools."""
    hkv, bs = 8, 256
    nb = (1 << 32) // (bs * hkv * D * (1 if fp8 else 2)) + 40
    small = Case([300, 600], [5, 9], 16, hkv, fp8=fp8, seed=24)
    dtype = torch.uint8 if fp8 else torch.bfloat16
    pools = []
    for p in (small.k, small.v):
        big = torch.empty((nb, bs, hkv, D), dtype=dtype, device="cuda")
        big[nb - small.nb:] = p.view(dtype) if fp8 else p
        pools.append(big.view(p.dtype))
    if fp8:
        scales = []
        for s in small.scales:
            big = torch.empty((nb, hkv, bs // 64), device="cuda")
            big[nb - small.nb:] = s
            scales.append(big)
        small.scales = tuple(scales)
    ref, size = Case([300, 600], [5, 9], 16, hkv, fp8=fp8, seed=24).reference()
    small.k, small.v = pools
    small.tables = torch.where(small.tables >= 0, small.tables + (nb - small.nb), small.tables)
    out = small.attend(pkv)
    assert_close(out, ref, size, fp8)


def test_a_chain_of_one_is_decode():
    c = Case([300, 77, 1030], [1, 1, 1], 16, 8, kind="chain", seed=25)
    want = pkv.paged_decode_attn(c.q.contiguous(), c.k, c.v, c.tables, c.lens, 1030, c.scale)
    got = c.attend(pkv)
    ref, size = c.reference()
    # (decode rounds its softmax weights to bf16)
    assert ((got.double() - want.double()).abs() <= 2.0 ** -7 * ref.abs() + 2.0 ** -7 * size).all()


def test_refusals():
    c = Case([70], [3], 4, 2, seed=26)
    with pytest.raises(ValueError):
        c.attend(pkv, tree_mask=torch.zeros((2, 1), dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        c.attend(pkv, tree_mask=torch.zeros((3, 1), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        c.attend(pkv, tree_mask=torch.zeros((3, 0), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        c.attend(pkv, tree_mask=torch.zeros((3, 1), dtype=torch.int64))
    with pytest.raises(pkv.PkvError) as e:
        c.attend(pkv, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert e.value.status == pkv.ERR_WORKSPACE
    c.q = c.q.transpose(1, 2).contiguous().transpose(1, 2)
    with pytest.raises(ValueError):
        c.attend(pkv)
