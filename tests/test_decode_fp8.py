"""Decode attention over the 8-bit cache, and decode attention with weights on either cache,
against softmax attention in 64 bits over the cache's own values.

Tolerances, from the arithmetic (ub = 2^-8 is a half step of bf16, u = 2^-24 of fp32):
  scores   products are exact, the sum of 128 and the scaling round in fp32: |ds| <= 140 u A with
           A = scale log2(e) sum |q_d k_d| in the log2 domain; q's form in two e4m3 parts is off by
           at most 2^-22 max|q| per dimension (8 bits of q' in [128, 256): the low part, scaled
           by 32, has a spacing of 2^-9, so q' is off by 2^-10 / 32 = 2^-15)
  weights  relative 2 ln2 max|ds| + rounding of the log-sum-exp and of the approximate exp2 and
           log2 (2^-22 each, |lse| u): e_w
  output   ub |ref| + (2^-15 + e_w) sum p |v| for the bf16 kernel with weights (it splits each
           weight in two bf16: 2^-17) and for the 8-bit kernel, whose three e4m3 parts of a weight
           w <= 256 hold it within 2^-15 w or 2^-20, the reference's own weight being 2^5:
           2^-25 max_i(p_i scale_i) sum_i |v_i| / scale_i besides
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
SCALE = D ** -0.5
U = 2.0 ** -24
# exp2 flushes results below fp32's smallest normal number to zero, so a weight smaller than it
# is off by up to itself: at most 2^-126 per query head (4.3e-39 is the first one that these
# inputs have)
TINY = 2.0 ** -126


class Case:
    """A cache (bf16 or 8-bit) with NaN everywhere that no context reaches, and its answer."""

    def __init__(self, ctx, hq, hkv, bs, seed, fp8=True, width=None, q_size=1.5, vspread=1.0):
        g = w.rng(seed)
        self.ctx, self.hq, self.hkv, self.bs, self.fp8 = np.asarray(ctx), hq, hkv, bs, fp8
        B = len(ctx)
        self.tables, nb = f8.tables_for(ctx, bs, g, width=width)
        self.q_bits = w.f32_to_bf16_bits((q_size * g.standard_normal((B, hq, D))).astype(np.float32))
        self.q = w.bf16_bits_to_f32(self.q_bits).astype(np.float64)
        live = np.zeros((nb, bs), bool)
        for b, n in enumerate(ctx):
            for j in range(-(-int(n) // bs)):
                live[self.tables[b, j], :min(bs, n - j * bs)] = True
        self.pools, self.values, self.v_scale = [], [], None
        for i in range(2):
            if fp8:
                codes, scale = f8.random_cache(nb, bs, hkv, g)
                if i:   # V's groups differ in size
                    scale = scale * np.exp2(np.round(vspread * 3 * g.standard_normal(scale.shape)))
                used = live.reshape(nb, bs // 64, 64).any(-1)
                codes[~live] = 0x7F
                scale = np.where(used[:, None], scale, [np.nan, np.inf][i])
                self.pools.append((codes, scale))
                self.values.append([f8.rows(codes, scale, self.tables[b], int(n))
                                    for b, n in enumerate(ctx)])
                ones = np.full_like(codes, 0x38)        # 1.0
                self.v_scale = [f8.rows(ones, scale, self.tables[b], int(n))[:, :, 0]
                                for b, n in enumerate(ctx)]
            else:
                bits = w.host_bf16_normal(g, (nb, bs, hkv, D))
                bits[~live] = w.BF16_NAN_CANARY
                self.pools.append(bits)
                flat = w.bf16_bits_to_f32(bits.reshape(nb * bs, hkv, D)).astype(np.float64)
                self.values.append([
                    flat[self.tables[b, np.arange(n) // bs].astype(np.int64) * bs + np.arange(n) % bs]
                    for b, n in enumerate(ctx)])

    def device(self):
        tail = [dev(self.tables), dev(self.ctx.astype(np.int32)), int(max(self.ctx)), SCALE]
        if not self.fp8:
            return [dev(self.q_bits), *map(dev, self.pools), *tail]
        (kc, ks), (vc, vs) = (f8.device_cache(*p) for p in self.pools)
        return [dev(self.q_bits), kc, vc, ks, vs, *tail]

    def reference(self):
        """out, its tolerance [B, Hq, D]; weights and their tolerance [B][Hkv, L]."""
        G = self.hq // self.hkv
        out, tol = np.zeros_like(self.q), np.zeros_like(self.q)
        ws, wtol = [], []
        for b, n in enumerate(self.ctx):
            k, v = self.values[0][b], self.values[1][b]
            wb, tb = np.zeros((self.hkv, n)), np.zeros((self.hkv, n))
            for hq in range(self.hq if n else 0):
                h = hq // G
                c = SCALE * np.log2(np.e)
                x = c * (k[:, h] @ self.q[b, hq])
                A = c * np.abs(k[:, h]) @ np.abs(self.q[b, hq])
                ds = 140 * U * A.max() + 2.0 ** -22 * c * np.abs(self.q[b, hq]).max() * \
                    np.abs(k[:, h]).sum(1).max()
                top = x.max()
                p = np.exp2(x - top)
                lse = top + np.log2(p.sum())
                p /= p.sum()
                e = 2 * np.log(2) * ds + 2.0 ** -20 + 8 * U * (abs(lse) + abs(top))
                out[b, hq] = p @ v[:, h]
                tol[b, hq] = 2.0 ** -8 * np.abs(out[b, hq]) + (2.0 ** -15 + e) * (p @ np.abs(v[:, h]))
                if self.v_scale:
                    vs = self.v_scale[b][:, h]
                    tol[b, hq] += 2.0 ** -25 * (p * vs).max() * (np.abs(v[:, h]) / vs[:, None]).sum(0)
                wb[h] += p
                tb[h] += p * e + TINY
            ws.append(wb)
            wtol.append(tb + 4 * U * wb)
        return out, tol, ws, wtol

    def run(self, args=None, **kw):
        args = args or self.device()
        if self.fp8:
            return pkv.paged_decode_attn_fp8(*args, **kw)
        return pkv.paged_decode_attn_weights(*args, **kw)


def check_out(got, ref, tol, what=""):
    g = host_f64(got)
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    bad = np.abs(g - ref) > tol
    assert not bad.any(), (f"{what}: {bad.sum()} values off, first {np.argwhere(bad)[0]}; worst "
                           f"{(np.abs(g - ref) / np.maximum(tol, 1e-300)).max()} of the tolerance")


def check_weights(got, start, ws, wtol, ctx, what=""):
    g, s = got.cpu().numpy().astype(np.float64), start.cpu().numpy().astype(np.float64)
    for b, n in enumerate(ctx):
        want = s[b, :, :n] + ws[b]
        tol = wtol[b] + 2 * U * np.abs(want)
        bad = np.abs(g[b, :, :n] - want) > tol
        assert not bad.any(), f"{what}: sequence {b}: {bad.sum()} weights off at {np.argwhere(bad)[0]}"


RAGGED = [1, 2, 17, 63, 64, 65, 127, 128, 129, 0, 255, 256, 257, 400, 511, 700]


@pytest.mark.gpu
@pytest.mark.parametrize("num_splits", [0, 1, 2, 3, 5, 8, 9])
def test_fp8_ragged_contexts(num_splits):
    c = Case(RAGGED, 16, 8, 256, 200)
    ref, tol, _, _ = c.reference()
    check_out(c.run(num_splits=num_splits), ref, tol, f"splits {num_splits}")
    assert pkv.get_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (4, 1), (5, 1), (6, 2), (7, 1), (8, 1),
                                    (9, 1), (12, 1), (16, 2), (16, 16), (24, 8), (64, 4)])
@pytest.mark.parametrize("num_splits", [0, 3, 6])
def test_fp8_head_groupings(hq, hkv, num_splits):
    c = Case([5, 300, 1, 129, 0, 777], hq, hkv, 512, 300 + hq + hkv)
    ref, tol, ws, wtol = c.reference()
    check_out(c.run(num_splits=num_splits), ref, tol, f"{hq}/{hkv}")
    start = torch.rand((6, hkv, 777), device="cuda")
    got = start.clone()
    check_out(c.run(num_splits=num_splits, weights=got), ref, tol, f"{hq}/{hkv} with weights")
    check_weights(got, start, ws, wtol, c.ctx)
    assert pkv.get_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(16, 8), (8, 1), (4, 4)])
def test_fp8_work_queue(hq, hkv):
    """More units than CTAs: the persistent grid draws from the queue; splits merge through
    global memory, short contexts are written by their one unit."""
    g = w.rng(310)
    B = 640 // hkv
    ctx = g.integers(0, 900, B)
    ctx[:3] = 2000, 899, 1
    c = Case(ctx, hq, hkv, 256, 311)
    ref, tol, ws, wtol = c.reference()
    args = c.device()
    for splits in (0, 1, 2, 12):
        weights = torch.zeros((B, hkv, 2001), device="cuda")
        ws_t = pkv.decode_fp8_workspace(B, hq, hkv, D, 2000, splits, weights=True)
        for _ in range(2):   # the second call finds the counter as the first left it
            check_out(c.run(args, num_splits=splits, workspace=ws_t, weights_out=weights), ref, tol,
                      f"splits {splits}")
            check_weights(weights, torch.zeros_like(weights), ws, wtol, ctx)
    assert pkv.get_device_errors() == 0


@pytest.mark.gpu
def test_fp8_one_long_context_and_long_tables():
    c = Case([20011], 8, 2, 256, 320, width=200)
    ref, tol, ws, wtol = c.reference()
    for splits in (0, 40):
        weights = torch.zeros((1, 2, 20011), device="cuda")
        check_out(c.run(num_splits=splits, weights=weights), ref, tol, "long")
        check_weights(weights, torch.zeros_like(weights), ws, wtol, c.ctx)


@pytest.mark.gpu
def test_fp8_groups_of_very_different_sizes():
    """V's scales span 2^-40 .. 2^40 and q is large or tiny: the running reference follows the
    largest weight times scale, and the sums lose nothing that shows in the output."""
    for q_size, vspread in ((1.5, 6.0), (40.0, 2.0), (1e-6, 1.0), (1e4, 1.0)):
        c = Case([300, 64, 511, 1030], 4, 2, 256, 330, q_size=q_size, vspread=vspread)
        ref, tol, _, _ = c.reference()
        for splits in (1, 3):
            check_out(c.run(num_splits=splits), ref, tol, f"{q_size} {vspread}")


@pytest.mark.gpu
@pytest.mark.parametrize("num_splits", [0, 1, 2, 5, 9])
@pytest.mark.parametrize("hq,hkv", [(16, 8), (3, 3), (12, 4), (16, 2)])
def test_bf16_weights(hq, hkv, num_splits):
    c = Case(RAGGED, hq, hkv, 256, 340 + hq, fp8=False)
    ref, tol, ws, wtol = c.reference()
    start = torch.rand((len(RAGGED), hkv, 704), device="cuda")
    got = start.clone()
    check_out(c.run(num_splits=num_splits, weights=got), ref, tol)
    check_weights(got, start, ws, wtol, c.ctx)
    for b, n in enumerate(c.ctx):      # entries past the context are left alone
        assert torch.equal(got[b, :, n:], start[b, :, n:])
    # a step's weights add up to one for every query head
    alone = torch.full((len(RAGGED), hkv, 700), 5.0, device="cuda")
    c.run(num_splits=num_splits, weights_out=alone)
    for b, n in enumerate(c.ctx):
        assert torch.equal(alone[b, :, n:], torch.full_like(alone[b, :, n:], 5.0))
        if n:
            s = alone[b, :, :n].double().sum(-1)
            assert torch.allclose(s, torch.full_like(s, hq // hkv), rtol=1e-4)
    assert pkv.get_device_errors() == 0


@pytest.mark.gpu
def test_bf16_weights_work_queue():
    g = w.rng(350)
    ctx = g.integers(0, 700, 100)
    c = Case(ctx, 8, 4, 256, 351, fp8=False)
    ref, tol, ws, wtol = c.reference()
    for splits in (0, 1, 4):
        out = torch.zeros((100, 4, 700), device="cuda")
        check_out(c.run(num_splits=splits, weights_out=out), ref, tol)
        check_weights(out, torch.zeros_like(out), ws, wtol, ctx)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [True, False])
def test_weights_strided_and_out_of_place(fp8):
    c = Case([70, 300, 9], 4, 2, 256, 360, fp8=fp8)
    ref, tol, ws, wtol = c.reference()
    base = torch.rand((3, 2, 1000), device="cuda")
    src = base[:, :, 100:500]                         # rows 1000 apart
    dst = torch.full((3, 2, 301), -1.0, device="cuda")
    keep = base.clone()
    check_out(c.run(weights=src, weights_out=dst), ref, tol)
    check_weights(dst, src, ws, wtol, c.ctx)
    assert torch.equal(base, keep)
    assert (dst[0, :, 70:] == -1).all() and (dst[2, :, 9:] == -1).all()
    c.run(weights=src)                                # in place, through the view
    assert torch.equal(src[1, :, :300], dst[1, :, :300])
    assert torch.equal(base[:, :, :100], keep[:, :, :100]) and torch.equal(base[:, :, 500:], keep[:, :, 500:])


@pytest.mark.gpu
def test_fp8_same_bits_for_any_placement_and_repeat():
    c = Case([700, 90, 1025, 256], 16, 8, 256, 370)
    args = c.device()
    base, again = c.run(args), c.run(args)
    assert torch.equal(base.view(torch.int16), again.view(torch.int16))
    g = w.rng(371)
    nb = c.pools[0][0].shape[0]
    perm = g.permutation(nb)
    moved = Case.__new__(Case)
    moved.__dict__.update(c.__dict__)
    moved.pools = []
    for codes, scale in c.pools:
        c2, s2 = np.empty_like(codes), np.empty_like(scale)
        c2[perm], s2[perm] = codes, scale
        moved.pools.append((c2, s2))
    moved.tables = np.where(c.tables >= 0, perm[np.maximum(c.tables, 0)], -1).astype(np.int32)
    assert torch.equal(moved.run().view(torch.int16), base.view(torch.int16))


@pytest.mark.gpu
def test_fp8_one_token_is_its_value():
    """A context of one token returns the cached value, rounded once to bf16 (exactly: four
    significant bits)."""
    c = Case([1, 1, 1], 16, 8, 256, 380)
    want = np.stack([np.repeat(v[0], 2, axis=0) for v in c.values[1]])
    assert np.array_equal(host_f64(c.run()), want)


@pytest.mark.gpu
def test_fp8_bad_data_is_reported():
    c = Case([300, 40], 4, 2, 256, 390)
    args = c.device()
    good = c.run(args).clone()
    bad = list(args)
    bad[5] = args[5].clone()
    bad[5][0, 1] = 99                                  # a block id past the pool: zeros there
    out = c.run(bad)
    assert pkv.get_device_errors() == pkv.DEVERR_BLOCK_RANGE
    assert torch.equal(out[1], good[1]) and torch.isfinite(out.float()).all()
    bad[5] = args[5]
    bad[6] = torch.tensor([-5, 40], dtype=torch.int32, device="cuda")
    out = c.run(bad)
    assert pkv.get_device_errors() == pkv.DEVERR_CONTEXT_RANGE
    assert (out[0] == 0).all() and torch.equal(out[1], good[1])


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [True, False])
def test_graph_capture_and_side_stream(fp8):
    c = Case([300, 1000, 5], 8, 2, 256, 400, fp8=fp8)
    ref, tol, ws, wtol = c.reference()
    args = c.device()
    make = pkv.decode_fp8_workspace if fp8 else pkv.decode_weights_workspace
    kw = dict(weights=True) if fp8 else {}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    space = make(3, 8, 2, D, 1000, stream=side, **kw)
    weights = torch.zeros((3, 2, 1000), device="cuda")
    out = torch.empty((3, 8, D), dtype=torch.bfloat16, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    c.run(args, workspace=space, weights=weights, out=out, stream=side)
    side.synchronize()
    check_out(out, ref, tol, "side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(args, workspace=space, weights=weights, out=out)
    weights.zero_()
    out.fill_(3.0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    check_out(out, ref, tol, "replayed")
    check_weights(weights, torch.zeros_like(weights), [3 * x for x in ws],
                  [3 * t + 8 * U * x for t, x in zip(wtol, ws)], c.ctx)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [True, False])
def test_abort_bit_stops_the_calls(fp8):
    c = Case([300, 1000, 5], 8, 2, 256, 410, fp8=fp8)
    ref, tol, ws, wtol = c.reference()
    args = c.device()
    weights = torch.full((3, 2, 1000), 9.0, device="cuda")
    for splits in (0, 1, 9):
        out = torch.full((3, 8, D), 3.0, dtype=torch.bfloat16, device="cuda")
        pkv.raise_device_errors(pkv.DEVERR_TIMEOUT)
        try:
            c.run(args, num_splits=splits, weights_out=weights, out=out)
            torch.cuda.synchronize()
            assert (out == 3).all() and (weights == 9).all()
        finally:
            assert pkv.get_device_errors() == pkv.DEVERR_TIMEOUT
        c.run(args, num_splits=splits, weights_out=weights, out=out)
        check_out(out, ref, tol)
        check_weights(weights, torch.zeros_like(weights), ws, wtol, c.ctx)
        weights.fill_(9.0)


@pytest.mark.gpu
def test_refusals():
    c = Case([5, 6], 4, 2, 256, 420)
    q, kc, vc, ks, vs, bt, cl, mx, sc = c.device()
    names = ["q", "k_cache", "v_cache", "k_scale", "v_scale", "block_tables", "context_lens",
             "max_context_len", "scale"]
    ok = dict(zip(names, [q, kc, vc, ks, vs, bt, cl, mx, sc]))
    f = torch.zeros((2, 2, 6), device="cuda")
    for kw in (dict(q=q.float()), dict(q=q[:, :, :64]), dict(q=q.cpu()), dict(k_scale=ks[:1]),
               dict(context_lens=cl[:1]), dict(block_tables=bt.long()), dict(out=q[:1]),
               dict(weights=f[:, :, :5]), dict(weights=f.double()), dict(weights_out=f[:1]),
               dict(weights=f.transpose(0, 1)[:, :, ::2]), dict(v_cache=vc[:, :128])):
        with pytest.raises((TypeError, ValueError)):
            pkv.paged_decode_attn_fp8(**{**ok, **kw})
    tiny = torch.zeros(8, dtype=torch.uint8, device="cuda")
    for kw, status in ((dict(workspace=tiny), pkv.ERR_WORKSPACE),
                       (dict(scale=float("nan")), pkv.ERR_INVALID_ARG),
                       (dict(num_splits=-1), pkv.ERR_INVALID_ARG),
                       (dict(weights=f, workspace=pkv.decode_fp8_workspace(2, 4, 2, D, mx)),
                        pkv.ERR_WORKSPACE)):
        with pytest.raises(pkv.PkvError) as e:
            pkv.paged_decode_attn_fp8(**{**ok, **kw})
        assert e.value.status == status, kw
    with pytest.raises(ValueError):
        b = Case([5, 6], 4, 2, 256, 421, fp8=False)
        pkv.paged_decode_attn_weights(*b.device())
    assert pkv.get_device_errors() == 0


@pytest.mark.gpu
def test_empty_batch():
    c = Case([5], 4, 2, 256, 430)
    q, kc, vc, ks, vs, bt, cl, mx, sc = c.device()
    out = pkv.paged_decode_attn_fp8(q[:0], kc, vc, ks, vs, bt[:0], cl[:0], mx, sc)
    assert out.shape == (0, 4, D)


@pytest.mark.gpu
def test_zero_contexts_give_zeros():
    c = Case([0, 0, 0], 8, 2, 256, 440, width=1)
    for splits in (0, 2):
        out = c.run(num_splits=splits, weights_out=torch.zeros((3, 2, 1), device="cuda"))
        assert (out == 0).all()


@pytest.mark.gpu
def test_nan_stays_where_it_is():
    """A NaN key makes its KV head's outputs of that sequence NaN and nothing else; a NaN value
    code its dimension; an infinite or NaN query its own head."""
    c = Case([300, 200, 129], 8, 2, 256, 450)
    args = c.device()
    good = c.run(args)
    codes = f8.host_codes(args[1]).copy()
    codes[c.tables[1, 0], 77, 1, 5] = 0x7F
    bad = list(args)
    bad[1] = torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn)
    for splits in (0, 1, 3):
        out, ref = c.run(bad, num_splits=splits), c.run(args, num_splits=splits)
        assert out[1, 4:].isnan().all()
        assert torch.equal(out[1, :4], ref[1, :4]) and torch.equal(out[::2], ref[::2])
    codes = f8.host_codes(args[2]).copy()
    codes[c.tables[2, 0], 3, 0, 9] = 0xFF
    bad = list(args)
    bad[2] = torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn)
    out = c.run(bad)
    assert out[2, :4, 9].isnan().all()
    out[2, :4, 9] = good[2, :4, 9]
    assert torch.equal(out, good)
    for value in (float("inf"), float("nan")):
        bad = list(args)
        bad[0] = args[0].clone()
        bad[0][0, 3, 17] = value
        out = c.run(bad)
        assert out[0, 3].isnan().all()
        out[0, 3] = good[0, 3]
        assert torch.equal(out, good)


@pytest.mark.gpu
def test_nan_on_the_bf16_cache_with_weights():
    c = Case([300, 1, 129], 8, 2, 256, 455, fp8=False)
    args = c.device()
    for seq, pos in ((0, 77), (1, 0)):      # among others, and as the only key
        bad = list(args)
        bad[1] = args[1].clone()
        bad[1][c.tables[seq, 0], pos, 1, 5] = float("nan")
        for splits in (0, 1, 3, 9):
            w0, w1 = (torch.zeros((3, 2, 300), device="cuda") for _ in range(2))
            out = c.run(bad, num_splits=splits, weights_out=w0)
            ref = c.run(args, num_splits=splits, weights_out=w1)
            n = int(c.ctx[seq])
            assert out[seq, 4:].isnan().all() and w0[seq, 1, :n].isnan().all()
            out[seq, 4:], w0[seq, 1] = ref[seq, 4:], w1[seq, 1]
            assert torch.equal(out, ref) and torch.equal(w0, w1)


@pytest.mark.gpu
def test_two_streams_at_once():
    """Two calls that overlap, with a workspace each, give what they give alone."""
    cases = [Case([700, 30, 1500], 16, 8, 256, 460 + i) for i in range(2)]
    alone = [c.run(num_splits=12) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    args = [c.device() for c in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            outs[i].append(cases[i].run(args[i], num_splits=12, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, alone[i])


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [True, False])
def test_offsets_past_32_bits(fp8):
    """A pool of more than 2^32 bytes, used at its far end by every call."""
    hkv, bs = 8, 256
    nb = 17000 if fp8 else 9000                       # 4.46 and 4.72 GB a pool
    far = [nb - 1, nb - 2, 3]
    g = w.rng(470)
    lens = [300, 100]
    tables = np.array([[far[0], far[1]], [far[2], -1]], np.int32)
    rows = [dev(w.host_bf16_normal(g, (400, hkv, D))) for _ in range(2)]
    cl, bt = dev(np.array(lens, np.int32)), dev(tables)
    if fp8:
        kc, vc = (torch.empty((nb, bs, hkv, D), dtype=torch.uint8, device="cuda").view(
            torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.empty((nb, hkv, bs // 64), device="cuda") for _ in range(2))
        cu = dev(np.array([0, 300, 400], np.int32))
        pkv.kv_store_fp8(*rows, cl, bt, kc, vc, ks, vs, cu_seqlens=cu)
        k, v = pkv.kv_gather_fp8(kc, vc, ks, vs, bt, cu, 400)
        codes, scale = np.zeros((4, bs, hkv, D), np.uint8), np.ones((4, hkv, bs // 64))
        f8.append(host_f64(rows[0])[:300], codes, scale, [0, 1], 0)
        assert np.array_equal(host_f64(k)[:300], f8.rows(codes, scale, [0, 1], 300))
        scales = dict(k_scale=ks, v_scale=vs)
    else:
        kc, vc = (torch.empty((nb, bs, hkv, D), dtype=torch.bfloat16, device="cuda")
                  for _ in range(2))
        k, v = rows
        slots = np.concatenate([tables[b, np.arange(n) // bs].astype(np.int64) * bs + np.arange(n) % bs
                                for b, n in enumerate(lens)])
        pkv.kv_store(k, v, dev(slots), kc, vc)
        scales = {}
    q = dev(w.host_bf16_normal(g, (2, 16, D)))
    weights = torch.zeros((2, hkv, 300), device="cuda")
    if fp8:
        out = pkv.paged_decode_attn_fp8(q, kc, vc, ks, vs, bt, cl, 300, SCALE, weights=weights)
    else:
        out = pkv.paged_decode_attn_weights(q, kc, vc, bt, cl, 300, SCALE, weights)
    K, V, Q = host_f64(k), host_f64(v), host_f64(q)
    for b, (a, e) in enumerate(((0, 300), (300, 400))):
        for h in range(16):
            x = SCALE * K[a:e, h // 2] @ Q[b, h]
            p = np.exp(x - x.max())
            p /= p.sum()
            ref = p @ V[a:e, h // 2]
            err = np.abs(host_f64(out)[b, h] - ref)
            assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -12 * (p @ np.abs(V[a:e, h // 2]))).all()
    dst = dev(np.array([[nb - 5], [nb - 6]], np.int32))
    kept, _, n2 = pkv.kv_evict(weights, cl, 300, bt, dst, 64, 8, kc, vc, **scales)
    assert n2.tolist() == [64, 64] and pkv.get_device_errors() == 0
    if not fp8:
        at = kept[0, 2].long().cpu().numpy()
        assert np.array_equal(host_f64(kc[nb - 5, :64, 2]), K[:300][at, 2])


@pytest.mark.gpu
@pytest.mark.parametrize("num_splits", [0, 1, 3, 4, 6])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (10, 2), (7, 1)])
def test_bf16_weights_of_larger_groups(hq, hkv, num_splits):
    """Four query heads to a unit, a whole group or the last unit with fewer."""
    c = Case(RAGGED, hq, hkv, 256, 230 + hq, fp8=False)
    ref, tol, ws, wtol = c.reference()
    start = torch.rand((len(RAGGED), hkv, max(RAGGED)), device="cuda")
    weights = start.clone()
    out = c.run(weights=weights, num_splits=num_splits)
    check_out(out, ref, tol)
    check_weights(weights, start, ws, wtol, c.ctx)
    assert pkv.get_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(16, 4), (40, 8)])
def test_bf16_weights_of_larger_groups_work_queue(hq, hkv):
    g = w.rng(250 + hq)
    ctx = g.integers(0, 300, 120)
    ctx[:3] = 700, 1, 0
    c = Case(ctx, hq, hkv, 256, 251, fp8=False)
    ref, tol, ws, wtol = c.reference()
    for num_splits in (0, 2):
        weights = torch.zeros((len(ctx), hkv, int(ctx.max())), device="cuda")
        out = c.run(weights=weights, num_splits=num_splits)
        check_out(out, ref, tol, str(num_splits))
        check_weights(weights, torch.zeros_like(weights), ws, wtol, ctx, str(num_splits))
    assert pkv.get_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(2, 1), (8, 2), (8, 1)])
def test_fp8_few_long_contexts(hq, hkv):
    """More splits than a cluster holds, chosen by the call, next to empty and short contexts; with
    weights the splits of a cluster, whose eight heads leave the weights to a kernel of their own."""
    c = Case([13700, 0, 12400, 1], hq, hkv, 256, 480 + hq)
    ref, tol, ws, wtol = c.reference()
    check_out(c.run(), ref, tol)
    weights = torch.zeros((4, hkv, 13700), device="cuda")
    check_out(c.run(weights=weights), ref, tol, "with weights")
    check_weights(weights, torch.zeros_like(weights), ws, wtol, c.ctx)
    assert pkv.get_device_errors() == 0
