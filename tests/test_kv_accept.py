"""kv_accept: the accepted rows of a tree, bit for bit."""
import numpy as np
import pytest
import torch

from libbuild import build_and_import
from tree_util import D, GROUP, ints, parents_of, tables_of

pkv = build_and_import()
pytestmark = pytest.mark.gpu
BOTH = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])


class Accept:
    def __init__(self, ctx, nodes, hkv=8, bs=256, fp8=False, seed=0, paths=None, width=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator()
        g.manual_seed(seed)
        self.ctx, self.nodes, self.hkv, self.bs, self.fp8 = ctx, nodes, hkv, bs, fp8
        self.table, self.nb = tables_of(rng, ctx, bs)
        if paths is None:
            paths = []
            for n in nodes:
                path, at = [], int(rng.integers(0, n)) if n else -1
                parents = parents_of(rng, n) if n else []
                while at >= 0:
                    path.append(at)
                    at = parents[at]
                paths.append(path[::-1])
        self.paths = paths
        width = max([len(p) for p in paths] + [1]) if width is None else width
        self.accepted = np.full((len(ctx), width), -1, np.int32)
        for i, p in enumerate(paths):
            self.accepted[i, :len(p)] = p
        self.num = [len(p) for p in paths]
        shape = (self.nb, bs, hkv, D)
        if fp8:
            self.pools = [torch.randint(0, 256, shape, generator=g, dtype=torch.uint8) for _ in "kv"]
            self.scales = [torch.exp2(torch.randint(-9, -3, (self.nb, hkv, bs // GROUP),
                                                    generator=g).float()) for _ in "kv"]
        else:
            self.pools = [torch.randint(-32768, 32768, shape, generator=g, dtype=torch.int16) for _ in "kv"]
            self.scales = None

    def run(self, **kw):
        """(pools, scales, lengths) after the call, on the host."""
        typed = torch.float8_e4m3fn if self.fp8 else torch.bfloat16
        pools = [p.cuda().view(typed) for p in self.pools]
        scales = [s.cuda() for s in self.scales] if self.fp8 else [None, None]
        cu = ints([0] + list(np.cumsum(self.nodes)))
        new = pkv.kv_accept(torch.from_numpy(self.accepted).cuda(), ints(self.num), cu, ints(self.ctx),
                            torch.from_numpy(self.table).cuda(), *pools, *scales, **kw)
        return ([p.view(q.dtype).cpu() for p, q in zip(pools, self.pools)],
                [s.cpu() for s in scales] if self.fp8 else None, new.cpu().tolist())

    def reference(self):
        pools = [p.clone() for p in self.pools]
        scales = [s.clone() for s in self.scales] if self.fp8 else None

        def at(b, pos):
            return int(self.table[b, pos // self.bs]), pos % self.bs

        def rerounded(codes, ratio):  # [hkv, D] codes, a ratio per head
            x = codes.view(torch.float8_e4m3fn).float() * ratio[:, None]
            y = x.to(torch.float8_e4m3fn).view(torch.uint8)
            return torch.where((ratio == 1)[:, None], codes, y)

        for i, (src, dst) in enumerate(zip(self.pools, pools)):
            for b, path in enumerate(self.paths):
                start = self.ctx[b] - self.nodes[b]
                if not self.fp8:
                    for j, node in enumerate(path):
                        dst[at(b, start + j)] = src[at(b, start + node)]
                    continue
                old = self.scales[i]
                moved = [(start + j, start + node) for j, node in enumerate(path)]
                for g in sorted({p // GROUP for p, _ in moved}):
                    here = [(p, f) for p, f in moved if p // GROUP == g]
                    blk, off = at(b, g * GROUP)
                    s0 = old[blk, :, off // GROUP]
                    s = s0.clone()
                    for _, f in here:
                        fb, fo = at(b, f)
                        s = torch.maximum(s, old[fb, :, fo // GROUP])
                    scales[i][blk, :, off // GROUP] = s
                    for pos in range(g * GROUP, start):
                        dst[at(b, pos)] = rerounded(src[at(b, pos)], s0 / s)
                    for p, f in here:
                        fb, fo = at(b, f)
                        dst[at(b, p)] = rerounded(src[fb, fo], old[fb, :, fo // GROUP] / s)
        return pools, scales, [c - n + len(p) for c, n, p in zip(self.ctx, self.nodes, self.paths)]


def same(a, got):
    """The pools' bits, NaN codes as one."""
    want = a.reference()
    assert got[2] == want[2]
    for x, y in zip(got[0], want[0]):
        if a.fp8:
            nan = (y & 0x7F) == 0x7F
            assert ((x & 0x7F) == 0x7F)[nan].all()
            x, y = x.masked_fill(nan, 0), y.masked_fill(nan, 0)
        assert torch.equal(x, y)
    if a.fp8:
        for x, y in zip(got[1], want[1]):
            assert torch.equal(x, y)


def check(a, **kw):
    pkv.get_device_errors(reset=True)
    same(a, a.run(**kw))
    assert pkv.get_device_errors(reset=True) == 0


@BOTH
@pytest.mark.parametrize("hkv", [1, 2, 3, 8, 12])
def test_small_batch(hkv, fp8):
    check(Accept([9, 70, 256, 300, 515], [9, 8, 5, 30, 6], hkv=hkv, fp8=fp8, seed=1))


@BOTH
@pytest.mark.parametrize("start", [0, 1, 40, 63, 64, 100, 190, 250, 255, 256])
def test_places_of_the_tree(start, fp8):
    """Paths that cross groups and blocks."""
    path = [0, 2, 3, 7, *range(20, 100, 3)]
    check(Accept([start + 100, start + 100], [100, 100], hkv=4, fp8=fp8, seed=start + 2,
                 paths=[path, list(range(50))]))


@BOTH
def test_long_paths(fp8):
    check(Accept([600, 400], [400, 300], hkv=2, fp8=fp8, seed=3,
                 paths=[[0, *range(2, 400, 2)], [*range(10), *range(20, 300)]]))


@BOTH
def test_nothing_accepted_and_empty_sequences(fp8):
    check(Accept([50, 20, 0, 64], [10, 0, 0, 64], fp8=fp8, seed=4, paths=[[], [], [], [5]]))


@BOTH
def test_everything_accepted_moves_nothing(fp8):
    a = Accept([50, 300], [10, 64], fp8=fp8, seed=5, paths=[list(range(10)), list(range(64))])
    check(a)


@BOTH
def test_wide_list_and_blocks_of_512(fp8):
    check(Accept([700, 90], [20, 8], bs=512, fp8=fp8, seed=6, width=33))


@BOTH
def test_large_batch(fp8):
    rng = np.random.default_rng(7)
    nodes = [int(x) for x in rng.integers(1, 65, 300)]
    ctx = [n + int(x) for n, x in zip(nodes, rng.integers(0, 300, 300))]
    check(Accept(ctx, nodes, hkv=2, fp8=fp8, seed=7))


def test_blocks_of_64():
    check(Accept([200, 65], [30, 8], bs=64, seed=8))


@BOTH
def test_bad_paths_end_where_they_are_bad(fp8):
    a = Accept([100, 100, 100, 100, 100], [20] * 5, hkv=2, fp8=fp8, seed=9,
               paths=[[0, 3, 3, 5], [0, 2, 20], [-1, 2], [0, 4, 9], [1, 5]])
    a.num[3] = 21
    a.num[4] = -1
    pkv.get_device_errors(reset=True)
    got = a.run()
    assert pkv.get_device_errors(reset=True) == pkv.DEVERR_NODE_RANGE
    a.paths = [[0, 3], [0, 2], [], [], []]
    same(a, got)


@BOTH
def test_bad_lengths_and_blocks(fp8):
    a = Accept([300, 90, 100, 120], [40, 20, 10, 12], hkv=2, fp8=fp8, seed=10)
    a.ctx[1], a.ctx[2] = 5, 4000
    pkv.get_device_errors(reset=True)
    got = a.run()
    assert pkv.get_device_errors(reset=True) == pkv.DEVERR_CONTEXT_RANGE
    assert got[2][1:3] == [0, 0]
    a.paths[1] = a.paths[2] = []
    a.ctx[1], a.ctx[2] = 20, 10  # (the reference's length of an emptied sequence)
    same(a, got)
    # the block of the first rows is bad: nothing is written there; rows that come from it are zeros
    for bad in (-3, a.nb):
        b = Accept([300], [100], hkv=2, fp8=fp8, seed=11, paths=[[0, 5, 60, 70]])
        b.table[0, 0] = bad
        got = b.run()
        assert pkv.get_device_errors(reset=True) == pkv.DEVERR_BLOCK_RANGE
        assert all(torch.equal(x, y) for x, y in zip(got[0], b.pools)) and got[2] == [204]


@BOTH
def test_stream_output_and_graph(fp8):
    a = Accept([300, 90], [40, 20], fp8=fp8, seed=12)
    s = torch.cuda.Stream()
    out = torch.zeros(2, dtype=torch.int32, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        check(a, new_context_lens=out)
    typed = torch.float8_e4m3fn if fp8 else torch.bfloat16
    pools = [p.cuda().view(typed) for p in a.pools]
    scales = [x.cuda() for x in a.scales] if fp8 else [None, None]
    args = (torch.from_numpy(a.accepted).cuda(), ints(a.num), ints([0, 40, 60]), ints(a.ctx),
            torch.from_numpy(a.table).cuda())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new = pkv.kv_accept(*args, *pools, *scales)
    graph.replay()
    torch.cuda.synchronize()
    same(a, ([p.view(q.dtype).cpu() for p, q in zip(pools, a.pools)],
             [x.cpu() for x in scales] if fp8 else None, new.cpu().tolist()))


def test_refusals():
    a = Accept([300, 90], [40, 20], seed=13)
    pool = [p.cuda().view(torch.bfloat16) for p in a.pools]
    lens, cu, table = ints(a.ctx), ints([0, 40, 60]), torch.from_numpy(a.table).cuda()
    acc, num = torch.from_numpy(a.accepted).cuda(), ints(a.num)
    with pytest.raises(pkv.PkvError):  # the other layers still need the old lengths
        pkv.kv_accept(acc, num, cu, lens, table, *pool, new_context_lens=lens)
    with pytest.raises(TypeError):
        pkv.kv_accept(acc.long(), num, cu, lens, table, *pool)
    with pytest.raises(ValueError):
        pkv.kv_accept(acc, num[:1], cu, lens, table, *pool)
    with pytest.raises(ValueError):
        pkv.kv_accept(acc, num, cu[:2], lens, table, *pool)
    with pytest.raises(ValueError):
        pkv.kv_accept(acc.cpu(), num, cu, lens, table, *pool)
    with pytest.raises(ValueError):
        pkv.kv_accept(acc, num, cu, lens, table, *pool, k_scale=torch.ones(1, device="cuda"))
