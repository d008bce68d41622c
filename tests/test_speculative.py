"""The calls of a speculative step together: drafted tokens appended, attended, accepted, and the
next step on what is left."""
import numpy as np
import pytest
import torch

from libbuild import build_and_import
from tree_util import Case, D, assert_close, cdiv, ints, parents_of, rows_of, words_of

pkv = build_and_import()
pytestmark = pytest.mark.gpu


class Model:
    """One layer's projections of tokens: a row of qkv for every (sequence, token)."""

    def __init__(self, hq, hkv, seed):
        self.hq, self.hkv = hq, hkv
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        turn = torch.arange(2048, device="cuda").double()[:, None] * \
            1e6 ** (-torch.arange(64, device="cuda").double() / 64)
        self.cos_sin = torch.cat((turn.cos(), turn.sin()), 1).float()
        self.w = torch.exp(0.2 * torch.randn((2, D), generator=self.g, device="cuda")).to(torch.bfloat16)

    def project(self, n):
        return torch.randn((n, (self.hq + 2 * self.hkv) * D), generator=self.g, device="cuda").to(
            torch.bfloat16)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_steps_of_a_conversation(fp8):
    hq, hkv, bs, B = 8, 2, 256, 3
    rng = np.random.default_rng(3)
    m = Model(hq, hkv, 3)
    bm = pkv.BlockManager(16, bs)
    tables_host = [bm.take(4) for _ in range(B)]
    tables = ints(tables_host)
    shape = (16, bs, hkv, D)
    kept = [[] for _ in range(B)]     # the accepted tokens' projection rows, in order
    if fp8:
        pools = [torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"]
        scales = [torch.ones((16, hkv, bs // 64), device="cuda") for _ in "kv"]
    else:
        pools = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        scales = []

    def append(x, cu, lens, positions, places):
        if fp8:
            return pkv.qk_norm_rope_store_fp8(x, ints(positions, torch.int64), m.cos_sin, ints(lens),
                                              tables, *pools, *scales, hq, m.w[0], m.w[1],
                                              cu_seqlens=ints(cu))
        slots = [tables_host[b][p // bs] * bs + p % bs for b, p in places]
        return pkv.qk_norm_rope_store(x, ints(positions, torch.int64), m.w[0], m.w[1], 1e-6, m.cos_sin,
                                      ints(slots, torch.int64), *pools, hq, hkv)

    prompts = [250, 61, 7]
    lens = list(prompts)
    x = m.project(sum(prompts))
    append(x, [0] + list(np.cumsum(prompts)), lens, [p for n in prompts for p in range(n)],
           [(b, p) for b, n in enumerate(prompts) for p in range(n)])
    t = 0
    for b, n in enumerate(prompts):
        kept[b] += list(x[t:t + n])
        t += n
    pkv.get_device_errors(reset=True)
    for step in range(6):
        nodes = [int(n) for n in rng.integers(1, 30, B)]
        trees = [parents_of(rng, n) for n in nodes]
        masks, depths = [], []
        for parents in trees:
            sees, depth = np.eye(len(parents), dtype=bool), [0] * len(parents)
            for i, p in enumerate(parents):
                if p >= 0:
                    sees[i] |= sees[p]
                    depth[i] = depth[p] + 1
            masks.append(sees)
            depths.append(depth)
        with_drafts = [n + k for n, k in zip(lens, nodes)]
        cu = [0] + list(np.cumsum(nodes))
        x = m.project(sum(nodes))
        q = append(x, cu, with_drafts, [lens[b] + d for b in range(B) for d in depths[b]],
                   [(b, lens[b] + i) for b in range(B) for i in range(nodes[b])])
        mask = words_of(masks, 1)
        args = (tables, ints(with_drafts), max(with_drafts), ints(cu), max(nodes), D ** -0.5, mask)
        out = pkv.paged_tree_attn_fp8(q, *pools, *scales, *args) if fp8 else \
            pkv.paged_tree_attn(q, *pools, *args)
        # against 64 bits on what the cache holds
        c = Case.__new__(Case)
        c.ctx, c.nodes, c.hq, c.hkv, c.bs, c.fp8, c.masks = with_drafts, nodes, hq, hkv, bs, fp8, masks
        c.table_host, c.q, c.scale = np.array(tables_host), q, D ** -0.5
        (c.k, c.v), c.scales = pools, scales or (None, None)
        ref, size = c.reference()
        assert_close(out, ref, size, fp8)
        # keep a path
        paths = []
        for b, parents in enumerate(trees):
            path, at = [], int(rng.integers(0, nodes[b]))
            while at >= 0:
                path.append(at)
                at = parents[at]
            paths.append(path[::-1])
            kept[b] += [x[cu[b] + i] for i in paths[b]]
        width = max(len(p) for p in paths)
        new = pkv.kv_accept(ints([p + [-1] * (width - len(p)) for p in paths]),
                            ints([len(p) for p in paths]), ints(cu), ints(with_drafts), tables, *pools,
                            *scales)
        lens = new.tolist()
        assert lens == [len(k) for k in kept]
    # the cache holds what appending the accepted tokens alone would have put there
    final = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    rows = torch.stack([r for k in kept for r in k])
    where = [(b, p) for b, n in enumerate(lens) for p in range(n)]
    slots = ints([tables_host[b][p // bs] * bs + p % bs for b, p in where], torch.int64)
    pkv.qk_norm_rope_store(rows, ints([p for _, p in where], torch.int64), m.w[0], m.w[1], 1e-6,
                           m.cos_sin, slots, *final, hq, hkv)
    for i in range(2):
        want = final[i].view(-1, hkv, D)[slots]
        if not fp8:
            assert torch.equal(pools[i].view(-1, hkv, D)[slots], want)
            continue
        sc = scales[i].transpose(1, 2).reshape(-1, hkv)[slots // 64][..., None].double()
        got = pools[i].view(torch.uint8).view(-1, hkv, D)[slots].view(torch.float8_e4m3fn).double() * sc
        # a value was rounded to e4m3 once and re-rounded at most twice as its group's scale grew;
        # the bf16 cache's rows are bf16 roundings of n and of y
        bound = 3 * 2.0 ** -4 * want.abs() + 3 * 2.0 ** -10 * sc + 2.0 ** -6 * want.abs().amax(-1, keepdim=True)
        assert ((got - want.double()).abs() <= bound).all()
    assert pkv.get_device_errors(reset=True) == 0
    for t in tables_host:
        bm.deallocate(t)
    assert bm.num_free == 16
