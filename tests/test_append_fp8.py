"""qk_norm_rope_store_fp8: norms and rotation on the way into the 8-bit cache, against 64 bits."""
import numpy as np
import pytest
import torch

from libbuild import build_and_import
from tree_util import D, GROUP, ints, rows_of, tables_of

pkv = build_and_import()
pytestmark = pytest.mark.gpu
EPS = 1e-6


class Append:
    """`new` last tokens of each context; the positions before them are in the cache."""

    def __init__(self, ctx, new, hq=4, hkv=2, bs=256, norm=True, seed=0, step=False, stride_pad=0,
                 tail=0, positions=None, mag=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.ctx, self.new, self.hq, self.hkv, self.bs, self.step = ctx, new, hq, hkv, bs, step
        self.table, self.nb = tables_of(rng, ctx, bs)
        T = (len(ctx) if step else sum(new)) + tail
        width = (hq + 2 * hkv) * D
        x = mag * torch.randn((T, width + stride_pad), generator=g, device="cuda")
        x *= torch.exp(torch.randn((T, 1), generator=g, device="cuda"))
        self.qkv = x.to(torch.bfloat16)[:, :width]
        if positions is None:
            positions = np.concatenate([np.arange(c - n, c) for c, n in zip(ctx, new)] + [np.zeros(tail)])
            if step:
                positions = np.maximum(np.array(ctx) - 1, 0)
        self.positions = ints([int(p) for p in positions], torch.int64)
        most = max(1, max(ctx + [1]))
        turn = torch.arange(most, device="cuda").double()[:, None] * \
            1e6 ** (-torch.arange(64, device="cuda").double() / 64)
        self.cos_sin = torch.cat((turn.cos(), turn.sin()), 1).float()
        self.w = [None, None]
        if norm:
            self.w = list(torch.exp(0.3 * torch.randn((2, D), generator=g, device="cuda")).to(torch.bfloat16))
        shape = (self.nb, bs, hkv, D)
        self.pools = [(100 * torch.randn(shape, generator=g, device="cuda")).clamp(-448, 448).to(
            torch.float8_e4m3fn) for _ in "kv"]
        self.scales = [torch.exp2(torch.randint(-9, -3, (self.nb, hkv, bs // GROUP), generator=g,
                                                device="cuda").float()) for _ in "kv"]
        self.cu = None if step else ints([0] + list(np.cumsum(new)))

    def tables(self):
        return torch.from_numpy(self.table).cuda()

    def run(self, **kw):
        pools = [p.view(torch.uint8).clone().view(p.dtype) for p in self.pools]
        scales = [s.clone() for s in self.scales]
        q = pkv.qk_norm_rope_store_fp8(self.qkv, self.positions, self.cos_sin, ints(self.ctx),
                                       self.tables(), *pools, *scales, self.hq,
                                       q_norm_weight=self.w[0], k_norm_weight=self.w[1], eps=EPS,
                                       cu_seqlens=self.cu, **kw)
        return q, pools, scales

    def rotated(self):
        """y of the query and key heads in 64 bits, and what its errors scale with."""
        T = self.qkv.shape[0]
        x = self.qkv.double().reshape(T, -1, D)
        out = []
        for heads, w in ((x[:, :self.hq], self.w[0]), (x[:, self.hq:self.hq + self.hkv], self.w[1])):
            if w is not None:
                heads = heads * torch.rsqrt((heads * heads).mean(-1, keepdim=True) + EPS) * w.double()
            cs = self.cos_sin.double()[self.positions.clamp(0, len(self.cos_sin) - 1)][:, None]
            c, s = cs[..., :64], cs[..., 64:]
            a, b = heads[..., :64], heads[..., 64:]
            y = torch.cat((a * c - b * s, b * c + a * s), -1)
            size = torch.cat((a.abs() * c.abs() + b.abs() * s.abs(),
                              b.abs() * c.abs() + a.abs() * s.abs()), -1)
            out.append((y, size))
        return out


# fp32: a sum of 128 squares, rsqrt, three products and a sum, each within 2^-22 of its terms
FP32 = 2.0 ** -19


def scale_of(top):
    """The smallest power of two s >= 2^-90 with top <= 448 s."""
    m, e = np.frexp(top)
    return 2.0 ** max(-90, (e - 9 if m <= 0.875 else e - 8)) if top > 0 else 2.0 ** -90


def check(a, skip=(), **kw):
    pkv.get_device_errors(reset=True)
    q, pools, scales = a.run(**kw)
    errors = pkv.get_device_errors(reset=True)
    (yq, sq), (yk, sk) = a.rotated()
    rows = [i for i in range(yq.shape[0]) if i not in skip]
    rows = rows[:len(rows) if a.step else sum(a.new)]
    off = (q.double() - yq).abs()[rows]
    assert (off <= (2.0 ** -8 * yq.abs() + FP32 * sq + 1e-37)[rows]).all()
    # V: kv_store_fp8's bits
    T = a.qkv.shape[0]
    k = a.qkv.reshape(T, -1, D)[:, a.hq:a.hq + a.hkv] if T else a.qkv.reshape(0, a.hkv, D)
    v = a.qkv.reshape(T, -1, D)[:, a.hq + a.hkv:] if T else k
    ref = [p.view(torch.uint8).clone().view(p.dtype) for p in a.pools]
    ref_scales = [s.clone() for s in a.scales]
    pkv.kv_store_fp8(k.contiguous(), v.contiguous(), ints(a.ctx), a.tables(), *ref, *ref_scales,
                     cu_seqlens=a.cu)
    pkv.get_device_errors(reset=True)
    assert torch.equal(pools[1].view(torch.uint8), ref[1].view(torch.uint8))
    assert torch.equal(scales[1], ref_scales[1])
    # K: the group's scale, the codes of the new rows, the rows from before
    was, got = a.pools[0].view(torch.uint8).cpu(), pools[0].view(torch.uint8).cpu()
    was_scale, got_scale = a.scales[0].cpu(), scales[0].cpu()
    yk, sk = yk.cpu(), sk.cpu()
    touched = torch.zeros(was.shape[:2], dtype=torch.bool)
    groups = torch.zeros((a.nb, a.bs // GROUP), dtype=torch.bool)
    t = 0
    for b, (c, n) in enumerate(zip(a.ctx, a.new)):
        start = c - n
        for gr in range(start // GROUP, -(-c // GROUP)):
            pos = [p for p in range(max(start, gr * GROUP), min(c, (gr + 1) * GROUP))]
            tok = [(b if a.step else t + p - start) for p in pos]
            pos, tok = zip(*[(p, i) for p, i in zip(pos, tok) if i not in skip]) if any(
                i not in skip for i in tok) else ((), ())
            if not pos:
                continue
            blk, off = int(a.table[b, pos[0] // a.bs]), pos[0] % a.bs
            g, first = off // GROUP, gr * GROUP
            groups[blk, g] = True
            for h in range(a.hkv):
                y = yk[list(tok), h]
                s = scale_of(float(y[torch.isfinite(y)].abs().max()))
                s0 = float(was_scale[blk, h, g]) if start > first else 0.0
                s = max(s, s0)
                assert float(got_scale[blk, h, g]) == s, (b, gr, h)
                code = got[blk, [p % a.bs for p in pos], h].view(torch.float8_e4m3fn).double()
                bound = 2.0 ** -4 * y.abs() + 2.0 ** -10 * s + FP32 * sk[list(tok), h]
                assert ((code * s - y).abs() <= bound).all(), (b, gr, h)
                old = was[blk, first % a.bs:first % a.bs + max(0, start - first), h]
                new = old if s == s0 else (old.view(torch.float8_e4m3fn).float() * (s0 / s)).to(
                    torch.float8_e4m3fn).view(torch.uint8)
                assert torch.equal(got[blk, first % a.bs:first % a.bs + max(0, start - first), h], new)
            touched[blk, first % a.bs:first % a.bs + max(0, start - first)] = True
            touched[blk, [p % a.bs for p in pos]] = True
        t += n
    # nothing else has changed
    assert torch.equal(got[~touched], was[~touched])
    keep = ~groups[:, None, :].expand_as(was_scale)
    assert torch.equal(got_scale[keep], was_scale[keep])
    return q, pools, scales, errors


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (16, 8), (3, 1), (5, 5), (14, 2)])
def test_prompts_and_chunks(hq, hkv, norm):
    assert check(Append([1, 64, 65, 300, 200, 130], [1, 64, 65, 300, 70, 3], hq, hkv, norm=norm,
                        seed=1))[3] == 0


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (16, 8), (3, 1), (6, 2)])
def test_a_step_of_one_token(hq, hkv, norm):
    ctx = [1, 2, 64, 65, 66, 256, 257, 700]
    assert check(Append(ctx, [1] * 8, hq, hkv, norm=norm, seed=2, step=True))[3] == 0


@pytest.mark.parametrize("start", [0, 1, 63, 64, 100, 250, 255, 256])
def test_places_of_drafted_tokens(start):
    positions = start + np.array([0, 1, 1, 2, 2, 3, 4, 4, 5] * 2) % 6
    assert check(Append([start + 9] * 2, [9] * 2, seed=start + 3, positions=np.minimum(positions, start + 8))
                 )[3] == 0


def test_blocks_of_512_and_strided_rows():
    assert check(Append([600, 90], [500, 90], bs=512, seed=4, stride_pad=24))[3] == 0


def test_large_batch():
    rng = np.random.default_rng(5)
    new = [int(x) for x in rng.integers(0, 150, 120)]
    ctx = [n + int(x) for n, x in zip(new, rng.integers(0, 300, 120))]
    assert check(Append(ctx, new, 16, 8, seed=5))[3] == 0


def test_keys_where_nothing_turns_are_stored_as_they_are():
    """Position 0 and no norm: kv_store_fp8's bits."""
    a = Append([70, 9], [70, 9], norm=False, seed=6, positions=np.zeros(79))
    q, pools, scales = a.run()
    assert torch.equal(q, a.qkv.view(79, -1, D)[:, :4])
    ref = [p.view(torch.uint8).clone().view(p.dtype) for p in a.pools]
    ref_scales = [s.clone() for s in a.scales]
    x = a.qkv.reshape(79, -1, D)
    pkv.kv_store_fp8(x[:, 4:6].contiguous(), x[:, 6:].contiguous(), ints(a.ctx), a.tables(), *ref,
                     *ref_scales, cu_seqlens=a.cu)
    for got, want in zip(pools + scales, ref + ref_scales):
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


def test_tokens_of_no_sequence_and_padding_rows():
    a = Append([30, 20], [10, 20], seed=7, tail=6)
    out = torch.full((36, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    check(a, q_out=out)
    assert (out[30:] == 7).all()
    a = Append([30, 0, 9], [1, 0, 1], seed=8, step=True)  # (a padding row's q is computed)
    assert check(a)[3] == 0


@pytest.mark.parametrize("step", [False, True])
def test_bad_positions(step):
    n = [1, 1, 1] if step else [5, 3, 70]
    a = Append([40, 70, 300], n, seed=9, step=step)
    bad = [1] if step else [2, 8, 20]
    for i in bad:
        a.positions[i] = -1 if i % 2 else len(a.cos_sin)
    out = torch.full((len(a.positions), 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    assert check(a, skip=bad, q_out=out)[3] == pkv.DEVERR_POSITION_RANGE
    assert (out[bad] == 7).all()


def test_values_that_are_not_finite():
    a = Append([90, 30], [90, 30], norm=False, seed=10)
    x = a.qkv.view(120, -1, D)
    x[5, 4, 3], x[7, 5, 90], x[9, 6, 1], x[11, 7, 2] = float("nan"), float("inf"), float("nan"), float("-inf")
    q, pools, scales = a.run()
    assert all(torch.isfinite(s).all() for s in scales)
    rows = rows_of(a.table[0], 90, 256)
    k = pools[0].view(torch.uint8).view(-1, 2, D)[torch.from_numpy(rows).cuda()].cpu()
    nan = (k & 0x7F) == 0x7F
    assert nan[5, 0, 3] and nan[5, 0, 67] and nan[5].sum() == 2 and not nan[20:].any()


def test_bad_lengths_and_blocks():
    a = Append([100, 90, 80, 60], [30, 20, 10, 5], seed=11)
    clean = a.run()
    a.ctx[1], a.ctx[2] = 10, 9000
    pkv.get_device_errors(reset=True)
    out = torch.full((65, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    q, pools, scales = a.run(q_out=out)
    assert pkv.get_device_errors(reset=True) == pkv.DEVERR_SEQLEN_RANGE | pkv.DEVERR_CONTEXT_RANGE
    assert (q[30:60] == 7).all() and torch.equal(q[:30], clean[0][:30]) and torch.equal(q[60:], clean[0][60:])
    for b, same in ((0, True), (1, False), (2, False), (3, True)):
        blk = int(a.table[b, 0])
        for got, new, was in zip(pools, clean[1], a.pools):
            want = new if same else was
            assert torch.equal(got[blk].view(torch.uint8), want[blk].view(torch.uint8))
    for step in (False, True):
        a = Append([100, 90], [1, 1], seed=12, step=step)
        a.table[1, 0] = a.nb
        pkv.get_device_errors(reset=True)
        q, pools, scales = a.run()
        assert pkv.get_device_errors(reset=True) == pkv.DEVERR_BLOCK_RANGE
        assert torch.isfinite(q).all()


def test_stream_and_graph():
    a = Append([100, 90], [30, 20], seed=13)
    want = a.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pools = [p.view(torch.uint8).clone().view(p.dtype) for p in a.pools]
    scales = [x.clone() for x in a.scales]
    lens, tables = ints(a.ctx), a.tables()
    torch.cuda.synchronize()
    args = (a.qkv, a.positions, a.cos_sin, lens, tables, *pools, *scales, 4, *a.w, EPS, a.cu)
    q = pkv.qk_norm_rope_store_fp8(*args, stream=s)
    s.synchronize()
    for got, ref in zip([q, *pools, *scales], [want[0], *want[1], *want[2]]):
        assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))
    for p, was in zip(pools + scales, a.pools + a.scales):
        p.view(torch.uint8).copy_(was.view(torch.uint8))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = pkv.qk_norm_rope_store_fp8(*args)
    graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip([q, *pools, *scales], [want[0], *want[1], *want[2]]):
        assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))


def test_refusals():
    a = Append([100, 90], [30, 20], seed=14)
    good = dict(qkv=a.qkv, positions=a.positions, cos_sin_cache=a.cos_sin, context_lens=ints(a.ctx),
                block_tables=a.tables(), k_cache=a.pools[0], v_cache=a.pools[1],
                k_scale=a.scales[0], v_scale=a.scales[1], num_q_heads=4, q_norm_weight=a.w[0],
                k_norm_weight=a.w[1], cu_seqlens=a.cu)
    for kw in (dict(num_q_heads=3), dict(num_q_heads=0), dict(k_norm_weight=None),
               dict(positions=a.positions[:3]), dict(cos_sin_cache=a.cos_sin[:, :64]),
               dict(qkv=a.qkv.cpu()), dict(q_norm_weight=a.w[0][:64]),
               dict(q_out=torch.empty((50, 5, D), dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            pkv.qk_norm_rope_store_fp8(**{**good, **kw})
    for kw in (dict(positions=a.positions.int()), dict(cos_sin_cache=a.cos_sin.double()),
               dict(qkv=a.qkv.float()), dict(num_q_heads=4.5), dict(eps="x")):
        with pytest.raises(TypeError):
            pkv.qk_norm_rope_store_fp8(**{**good, **kw})
    with pytest.raises(pkv.PkvError):
        pkv.qk_norm_rope_store_fp8(**{**good, "eps": -1.0})
