"""Trees of drafted tokens over a paged cache, and their attention in 64 bits."""
import numpy as np
import torch

D = 128
GROUP = 64
NAN8 = 0x7F  # an e4m3 NaN


def cdiv(a, b):
    return -(-a // b)


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def tables_of(rng, lens, bs, spare=2):
    """Block tables [B, W] of shuffled blocks, and the number of blocks."""
    counts = [cdiv(n, bs) for n in lens]
    nb = sum(counts) + spare
    ids = rng.permutation(nb)
    t = np.full((len(lens), max(counts + [1])), -1, np.int32)
    at = 0
    for i, n in enumerate(counts):
        t[i, :n] = ids[at:at + n]
        at += n
    return t, nb


def rows_of(table, n, bs):
    """Pool rows of positions 0 .. n - 1 (host)."""
    pos = np.arange(n)
    return table[pos // bs].astype(np.int64) * bs + pos % bs


def parents_of(rng, n, reach=4):
    return [-1] + [int(rng.integers(max(0, i - reach), i)) for i in range(1, n)]


def masks_of(rng, kind, n):
    """A [n, n] bool mask: 'chain', 'tree', 'random' (rows that see nothing among them), 'all'."""
    if kind == "chain":
        return np.tril(np.ones((n, n), bool))
    if kind == "all":
        return np.ones((n, n), bool)
    if kind == "random":
        m = rng.random((n, n)) < 0.4
        m[:: 3] = False
        return m
    m = np.eye(n, dtype=bool)
    for i, p in enumerate(parents_of(rng, n)):
        if p >= 0:
            m[i] |= m[p]
    return m


def words_of(masks, width):
    rows = []
    for m in masks:
        n = m.shape[0]
        for row in m:
            bits = np.zeros(64 * width, bool)
            bits[:n] = row
            rows.append(np.packbits(bits, bitorder="little").view(np.int64))
    return torch.from_numpy(np.array(rows, np.int64).reshape(-1, width)).cuda()


class Case:
    """A batch of contexts with a tree each. Whatever no position owns is NaN."""

    def __init__(self, ctx, nodes, hq, hkv, bs=256, kind="tree", fp8=False, seed=0, stride_pad=0,
                 tail=0, mag=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.ctx, self.nodes, self.hq, self.hkv, self.bs, self.fp8 = ctx, nodes, hq, hkv, bs, fp8
        self.table_host, self.nb = tables_of(rng, ctx, bs)
        self.masks = [masks_of(rng, kind, n) for n in nodes]
        self.most = max(nodes + [0])
        T = sum(nodes) + tail
        row = hq * D + stride_pad
        self.q = (1.5 * torch.randn((T, row), generator=g, device="cuda")).to(torch.bfloat16)
        self.q = self.q.as_strided((T, hq, D), (row, D, 1))
        self.mask = None if kind == "chain" else words_of(
            self.masks + [np.zeros((tail, 1), bool)] * (tail > 0), max(1, cdiv(self.most, 64)))
        owned = np.concatenate([rows_of(t, n, bs) for t, n in zip(self.table_host, ctx)] or [[]])
        owned = torch.from_numpy(owned.astype(np.int64)).cuda()
        self.scales = (None, None)
        if fp8:
            pools, scales = [], []
            for m in (mag, 0.3):
                codes = torch.full((self.nb * bs, hkv, D), NAN8, dtype=torch.uint8, device="cuda")
                x = (60 * m * torch.randn((len(owned), hkv, D), generator=g, device="cuda"))
                codes[owned] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                pools.append(codes.view(torch.float8_e4m3fn).view(self.nb, bs, hkv, D))
                sc = torch.full((self.nb * bs // GROUP, hkv), float("nan"), device="cuda")
                e = torch.randint(-8, -4, sc.shape, generator=g, device="cuda").float()
                used = torch.unique(owned // GROUP)
                sc[used] = torch.exp2(e)[used]
                scales.append(sc.view(self.nb, bs // GROUP, hkv).transpose(1, 2).contiguous())
            (self.k, self.v), self.scales = pools, tuple(scales)
        else:
            pools = []
            for m in (mag, 0.3):
                p = torch.full((self.nb * bs, hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                p[owned] = (m * torch.randn((len(owned), hkv, D), generator=g, device="cuda")).to(
                    torch.bfloat16)
                pools.append(p.view(self.nb, bs, hkv, D))
            self.k, self.v = pools
        self.tables = torch.from_numpy(self.table_host).cuda()
        self.lens = ints(ctx)
        self.cu = ints([0] + list(np.cumsum(nodes)))
        self.scale = D ** -0.5

    def values(self, name, b):
        """float64 rows of sequence b: [L, hkv, D]."""
        pool = getattr(self, name)
        r = torch.from_numpy(rows_of(self.table_host[b], self.ctx[b], self.bs)).cuda()
        if not self.fp8:
            return pool.view(-1, self.hkv, D)[r].double()
        x = pool.view(torch.uint8).view(-1, self.hkv, D)[r].view(torch.float8_e4m3fn).double()
        sc = self.scales[0 if name == "k" else 1].transpose(1, 2).reshape(-1, self.hkv)
        return x * sc[r // GROUP].double()[..., None]

    def reference(self):
        """(out, size): the attention in 64 bits, and the same over |v| (what errors scale with)."""
        T = self.q.shape[0]
        out = torch.zeros((T, self.hq, D), dtype=torch.float64, device="cuda")
        size = torch.zeros_like(out)
        t = 0
        for b, (L, n) in enumerate(zip(self.ctx, self.nodes)):
            sees = torch.ones((n, L), dtype=torch.bool)
            sees[:, L - n:] = torch.from_numpy(self.masks[b])
            sees = sees.cuda()[:, None, None, :]
            q = self.q[t:t + n].double().view(n, self.hkv, self.hq // self.hkv, D)
            k, v = self.values("k", b), self.values("v", b)
            x = torch.einsum("nhgd,lhd->nhgl", q, k) * self.scale
            x = x.masked_fill(~sees, float("-inf"))
            p = torch.softmax(x, dim=-1).masked_fill(~sees, 0.0)  # (a row of -inf: NaN, then 0)
            out[t:t + n] = torch.einsum("nhgl,lhd->nhgd", p, v).reshape(n, self.hq, D)
            size[t:t + n] = torch.einsum("nhgl,lhd->nhgd", p, v.abs()).reshape(n, self.hq, D)
            t += n
        return out, size

    def attend(self, pkv, **kw):
        a = dict(tree_mask=self.mask)
        a.update(kw)
        args = (self.tables, self.lens, max(self.ctx + [0]), self.cu, self.most, self.scale)
        if self.fp8:
            return pkv.paged_tree_attn_fp8(self.q, self.k, self.v, *self.scales, *args, **a)
        return pkv.paged_tree_attn(self.q, self.k, self.v, *args, **a)


def bf16_weights(nodes, group):
    """Whether a call with trees of up to so many nodes rounds its weights to bf16 (bf16 cache): the
    rows of a KV head, in chunks of 16, are more than a tile of 8 chunks."""
    heads = min(group, 16)
    return cdiv(nodes, 16 // heads) * cdiv(group, 16) > 8


def assert_close(got, ref, size, fp8, bf16=False):
    """bf16 rounding is off by 2^-8 of the value at most. A weight is off by 2^-12 of itself from its
    score (128 products in fp32, |score| up to a few tens) and by 2^-16 (8-bit cache: 2^-11, where
    weights are rounded to bf16: 2^-8) from its rounding. The sum and the normaliser each take the
    first of these errors of sum w |v|, the sum alone the rounding's."""
    weights = 2.0 ** -9 if fp8 else 2.0 ** -10 + (2.0 ** -8 if bf16 else 0)
    bound = 2.0 ** -8 * ref.abs() + weights * size + 1e-30
    off = (got.double() - ref).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (int(bad.sum()), float((off / bound)[bad].max()) if bad.any() else 0,
                           torch.nonzero(bad)[:5].tolist())
