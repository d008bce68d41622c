"""Eviction by accumulated attention weight: the kept positions, their weights and the compacted
rows against a plain selection, exactly (copies; ties go to the lower position), and the path a
server takes: prefill, store, decode with weights, evict, go on decoding."""
import numpy as np
import pytest
import torch

import fp8_util as f8
import workloads as w
from gpu_util import dev, host_bits, host_f64
from libbuild import build_and_import
from test_decode_fp8 import SCALE, U, check_out

pkv = build_and_import()
D = 128


def select(wts, L, budget, recent):
    """Kept positions of one head: weights [>= L] float64."""
    if L <= budget:
        return np.arange(L)
    last = L - recent
    key = np.where(np.isnan(wts[:last]), -np.inf, wts[:last] + 0.0)
    nan = np.isnan(wts[:last])
    order = sorted(range(last), key=lambda i: (nan[i], -key[i], i))[:budget - recent]
    return np.sort(np.concatenate([np.array(order, np.int64), np.arange(last, L)]))


def _weights(g, B, hkv, S, kind):
    x = np.exp(2 * g.standard_normal((B, hkv, S))).astype(np.float32)
    if kind == "ties":                   # few distinct values
        x = np.round(x)
    elif kind == "equal":
        x[:] = 0.25
    elif kind == "special":
        x[g.random(x.shape) < 0.1] = np.nan
        x[g.random(x.shape) < 0.1] = np.inf
        x[g.random(x.shape) < 0.1] = -np.inf
        x[g.random(x.shape) < 0.1] = -0.0
        x[g.random(x.shape) < 0.1] = 0.0
        x[g.random(x.shape) < 0.1] *= -1
        x[g.random(x.shape) < 0.05] = 1e-42      # subnormal
    return x


def _case(ctx, hkv, bs, budget, recent, seed, fp8, kind="normal", weights_stride=0):
    g = w.rng(seed)
    ctx = np.asarray(ctx, np.int32)
    B = len(ctx)
    n = np.minimum(ctx, budget)
    both, nb = f8.tables_for(np.concatenate([ctx, n]), bs, g)
    src, dst = both[:B], both[B:]
    S = int(max(ctx.max(), 1)) + weights_stride
    wts = _weights(g, B, hkv, S, kind)
    if fp8:
        pools = [f8.random_cache(nb, bs, hkv, g) for _ in range(2)]
        (kc, ks), (vc, vs) = (f8.device_cache(*p) for p in pools)
        scales = dict(k_scale=ks, v_scale=vs)
    else:
        pools = [w.host_bf16_normal(g, (nb, bs, hkv, D)) for _ in range(2)]
        kc, vc = map(dev, pools)
        scales = {}
    got = pkv.kv_evict(dev(wts), dev(ctx), int(ctx.max()), dev(np.ascontiguousarray(src)),
                       dev(np.ascontiguousarray(dst)), budget, recent, kc, vc, **scales)
    kept, w_out, lens = (t.cpu().numpy() for t in got)
    assert np.array_equal(lens, n)
    for b in range(B):
        m = int(n[b])
        for h in range(hkv):
            at = select(wts[b, h].astype(np.float64), int(ctx[b]), budget, recent)
            assert np.array_equal(kept[b, h, :m], at), (b, h)
            assert (kept[b, h, m:] == -1).all() and (w_out[b, h, m:] == 0).all()
            assert np.array_equal(w_out[b, h, :m], wts[b, h, at], equal_nan=True)
            # the rows, written into the model's pools
            from_row = src[b, at // bs].astype(np.int64) * bs + at % bs
            j = np.arange(m)
            to_row = dst[b, j // bs].astype(np.int64) * bs + j % bs
            for p in pools:
                if not fp8:
                    flat = p.reshape(nb * bs, hkv, D)
                    flat[to_row, h] = flat[from_row, h]
                    continue
                codes, scale = p
                flat = codes.reshape(nb * bs, hkv, D)
                mine = scale[from_row // bs, h, from_row % bs // 64]
                for j0 in range(0, m, 64):
                    s = mine[j0:j0 + 64].max()
                    x = f8.VALUES[flat[from_row[j0:j0 + 64], h]] * (mine[j0:j0 + 64] / s)[:, None]
                    flat[to_row[j0:j0 + 64], h] = f8.encode(x)
                    scale[to_row[j0] // bs, h, to_row[j0] % bs // 64] = s
    for p, t, s in zip(pools, (kc, vc), ("k_scale", "v_scale")):
        if fp8:
            assert f8.same_codes(f8.host_codes(t), p[0]).all(), s
            assert np.array_equal(scales[s].cpu().numpy().astype(np.float64), p[1]), s
        else:
            assert np.array_equal(host_bits(t), p)
    assert pkv.get_device_errors() == 0


def test_selection_model():
    """The model itself: recent ones first, ties to the lower position, NaN last."""
    x = np.array([3.0, 1.0, 3.0, np.nan, 2.0, 0.0, 9.0])
    assert select(x, 7, 3, 1).tolist() == [0, 2, 6]
    assert select(x, 7, 5, 2).tolist() == [0, 2, 4, 5, 6]
    assert select(np.array([np.nan, np.nan, 1.0, 0.0]), 4, 3, 1).tolist() == [0, 2, 3]
    assert select(x, 7, 2, 2).tolist() == [5, 6]
    assert select(x, 4, 9, 2).tolist() == [0, 1, 2, 3]


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("kind", ["normal", "ties", "equal", "special"])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (64, 10), (100, 0), (257, 256), (130, 130)])
def test_evict(fp8, kind, budget, recent):
    _case([700, 0, 1, 64, 65, 129, 258, 1000, 257], 3, 256, budget, recent, 500, fp8, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [True, False])
def test_evict_long_rows_and_block_sizes(fp8):
    _case([9000, 4096, 4097], 2, 512, 1500, 100, 510, fp8, "normal", weights_stride=7)
    _case([20000], 1, 256, 5000, 33, 511, fp8, "ties")
    _case([5], 1, 256, 400, 3, 512, fp8)
    if not fp8:
        _case([300, 70], 5, 64, 100, 9, 513, fp8)


@pytest.mark.gpu
def test_evict_given_outputs_and_strided_weights():
    g = w.rng(520)
    hkv, bs, budget = 2, 256, 90
    ctx = dev(np.array([200, 50], np.int32))
    both, nb = f8.tables_for([200, 50, 90, 50], bs, g)
    kc, vc = (dev(w.host_bf16_normal(g, (nb, bs, hkv, D))) for _ in range(2))
    base = torch.rand((2, hkv, 512), device="cuda")
    out = torch.full((2, hkv, 300), 4.0, device="cuda")
    kept = torch.empty((2, hkv, budget), dtype=torch.int32, device="cuda")
    lens = torch.empty(2, dtype=torch.int32, device="cuda")
    src, dst = dev(both[:2].copy()), dev(both[2:].copy())
    got = pkv.kv_evict(base[:, :, 7:207], ctx, 200, src, dst, budget, 10, kc, vc, kept=kept,
                       weights_out=out, new_context_lens=lens)
    assert got[0] is kept and got[1] is out and got[2] is lens
    assert (out[:, :, budget:] == 4).all() and (out[1, :, 50:budget] == 0).all()
    x = base[:, :, 7:207].cpu().numpy().astype(np.float64)
    for b, L in enumerate((200, 50)):
        for h in range(hkv):
            at = select(x[b, h], L, budget, 10)
            assert np.array_equal(kept[b, h, :len(at)].cpu().numpy(), at)
            assert np.array_equal(out[b, h, :len(at)].cpu().numpy(), x[b, h, at].astype(np.float32))


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [True, False])
def test_evict_bad_data(fp8):
    """Bad lengths leave an empty sequence, bad source blocks zero rows, bad destination blocks
    nothing; the other sequences are as they should be."""
    g = w.rng(530)
    hkv, bs, budget = 2, 256, 100
    nb = 8
    src = np.array([[0, 1], [0, 1], [0, 50], [2, -1], [3, -1]], np.int32)
    dst = np.array([[4], [4], [5], [77], [6]], np.int32)
    ctx = np.array([-4, 600, 300, 90, 80], np.int32)     # < 0, past max and table, .., .., good
    wts = torch.rand((5, hkv, 512), device="cuda")
    if fp8:
        pools = [f8.random_cache(nb, bs, hkv, g) for _ in range(2)]
        (kc, ks), (vc, vs) = (f8.device_cache(*p) for p in pools)
        kw, codes = dict(k_scale=ks, v_scale=vs), pools[0][0]
        now = lambda: f8.host_codes(kc)  # noqa: E731
    else:
        pools = [w.host_bf16_normal(g, (nb, bs, hkv, D)) for _ in range(2)]
        kc, vc = map(dev, pools)
        kw, codes = {}, pools[0]
        now = lambda: host_bits(kc)  # noqa: E731
    kept, w_out, lens = pkv.kv_evict(wts, dev(ctx), 512, dev(src), dev(dst), budget, 100, kc, vc,
                                     **kw)
    assert pkv.get_device_errors() == pkv.DEVERR_CONTEXT_RANGE | pkv.DEVERR_BLOCK_RANGE
    assert lens.tolist() == [0, 0, 100, 90, 80]
    assert (kept[:2] == -1).all() and (w_out[:2] == 0).all()
    k = now()
    assert (k[4] == codes[4]).all() and (k[:4] == codes[:4]).all() and (k[7] == codes[7]).all()
    # sequence 2 keeps positions 200 .. 299: 56 from block 0, then the bad block's zeros
    assert (k[5, 56:100] == 0).all() and (k[5, 100:] == codes[5, 100:]).all()
    assert (k[6, 80:] == codes[6, 80:]).all()
    if not fp8:
        assert (k[5, :56] == codes[0, 200:]).all() and (k[6, :80] == codes[3, :80]).all()


@pytest.mark.gpu
def test_refusals():
    kc = torch.zeros((3, 256, 2, D), dtype=torch.bfloat16, device="cuda")
    i = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    cl = torch.ones(1, dtype=torch.int32, device="cuda")
    f = torch.zeros((1, 2, 8), device="cuda")
    ok = dict(weights=f, context_lens=cl, max_context_len=8, block_tables=i,
              dst_block_tables=i + 1, budget=4, recent=1, k_cache=kc, v_cache=kc.clone())
    for kw in (dict(budget=0), dict(recent=5), dict(recent=-1), dict(max_context_len=9),
               dict(weights=f.double()), dict(k_cache=kc.float()), dict(block_tables=i[0]),
               dict(k_scale=f), dict(v_cache=kc[:2]), dict(kept=i), dict(context_lens=cl.cpu()),
               dict(weights_out=f[:, :, :3])):
        with pytest.raises((TypeError, ValueError)):
            pkv.kv_evict(**{**ok, **kw})
    for kw in (dict(dst_block_tables=i), dict(new_context_lens=cl), dict(weights_out=f)):
        with pytest.raises(pkv.PkvError) as e:     # outputs that are inputs
            pkv.kv_evict(**{**ok, "block_tables": i, **kw})
        assert e.value.status == pkv.ERR_INVALID_ARG
    got = pkv.kv_evict(**{**ok, "weights": f[:0], "context_lens": cl[:0], "block_tables": i[:0],
                          "dst_block_tables": (i + 1)[:0]})
    assert got[0].shape == (0, 2, 4)
    assert pkv.get_device_errors() == 0


@pytest.mark.gpu
def test_abort_bit_stops_the_call():
    kc = torch.full((3, 256, 2, D), 2.0, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    cl = torch.full((1,), 8, dtype=torch.int32, device="cuda")
    kept = torch.full((1, 2, 4), 77, dtype=torch.int32, device="cuda")
    lens = torch.full((1,), 4, dtype=torch.int32, device="cuda")
    f8c = torch.zeros((3, 256, 2, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sc = torch.full((3, 2, 4), 0.5, device="cuda")
    row = torch.ones((1, 2, D), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    pkv.raise_device_errors(pkv.DEVERR_TIMEOUT)
    try:
        pkv.kv_evict(torch.rand((1, 2, 8), device="cuda"), cl, 8, i, i + 1, 4, 1, kc, kc,
                     kept=kept, new_context_lens=lens)
        for c in (None, cu):
            pkv.kv_store_fp8(row, row, cl, i, f8c, f8c, sc, sc, cu_seqlens=c)
        out = torch.full((8, 2, D), 5.0, dtype=torch.bfloat16, device="cuda")
        pkv.kv_gather_fp8(f8c, f8c, sc, sc, i, cu * 8, 8, k_out=out, v_out=out)
        torch.cuda.synchronize()
        assert (kept == 77).all() and (kc == 2).all() and (out == 5).all()
        assert (f8c.view(torch.uint8) == 0).all() and (sc == 0.5).all()
    finally:
        assert pkv.get_device_errors() == pkv.DEVERR_TIMEOUT


# ------------------------------------------------------------------- together, as a server runs
@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [True, False])
def test_serving_path(fp8):
    """Two conversations, one sharing the other's first block: prompts attended and stored,
    decode steps that accumulate weights, an eviction into fresh blocks, further steps on the
    shortened contexts. Every decode output is checked against softmax attention in 64 bits over
    the rows each head should hold by then."""
    g = w.rng(540)
    hq, hkv, bs, budget, recent = 4, 2, 256, 128, 32
    bm = pkv.BlockManager(16, bs)
    prompts = [list(range(400)), list(range(256)) + [9] * 44]
    tables, cached = zip(*(bm.allocate(p) for p in prompts))
    assert cached == (0, 256) and tables[0][0] == tables[1][0]
    lens = [400, 300]
    nb = 16
    if fp8:
        kc, vc = (torch.zeros((nb, bs, hkv, D), dtype=torch.uint8, device="cuda").view(
            torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.ones((nb, hkv, bs // 64), device="cuda") for _ in range(2))
    else:
        kc, vc = (torch.zeros((nb, bs, hkv, D), dtype=torch.bfloat16, device="cuda")
                  for _ in range(2))

    def rows_of(pool, scale, table, n):
        if fp8:
            return f8.rows(f8.host_codes(pool), scale.cpu().numpy().astype(np.float64), table, n)
        flat = host_f64(pool).reshape(nb * bs, hkv, D)
        return flat[np.asarray(table)[np.arange(n) // bs] * bs + np.arange(n) % bs]

    def table_tensor(ts, width=4):
        t = np.full((2, width), -1, np.int32)
        for r, x in zip(t, ts):
            r[:len(x)] = x
        return dev(t)

    def store(k, v, ctx, ts, new):
        bt = table_tensor(ts)
        if fp8:
            cu = None if new is None else dev(np.cumsum([0] + new).astype(np.int32))
            pkv.kv_store_fp8(k, v, dev(np.array(ctx, np.int32)), bt, kc, vc, ks, vs, cu_seqlens=cu)
        else:
            new = new or [1, 1]
            pos = [np.arange(c - m, c) for c, m in zip(ctx, new)]
            slots = np.concatenate([np.asarray(t)[p // bs] * bs + p % bs for t, p in zip(ts, pos)])
            pkv.kv_store(k, v, dev(slots.astype(np.int64)), kc, vc)

    def rand_rows(n):
        return dev(w.host_bf16_normal(g, (n, hkv, D)))

    # the prompts: the first whole, the second from its cached prefix on
    new = [400, 44]
    store(rand_rows(444), rand_rows(444), lens, list(tables), new)
    q = dev(w.host_bf16_normal(g, (444, hq, D)))
    bt, cu_q = table_tensor(tables), dev(np.array([0, 400, 444], np.int32))
    cu_k = dev(np.array([0, 400, 700], np.int32))
    if fp8:
        k, v = pkv.kv_gather_fp8(kc, vc, ks, vs, bt, cu_k, 700)
        out = pkv.varlen_prefill_attn(q, k, v, cu_q, cu_k, 400, 400, SCALE)
    else:
        out = pkv.varlen_prefill_attn(q, kc, vc, cu_q, cu_k, 400, 400, SCALE, block_table=bt)
    scales = (ks, vs) if fp8 else (None, None)
    for b, first in ((0, 0), (1, 400)):      # each prompt's last query sees all its keys
        K, V = (rows_of(p, s, tables[b], lens[b]) for p, s in ((kc, scales[0]), (vc, scales[1])))
        qq = host_f64(q[first + new[b] - 1])
        for h in range(hq):
            x = SCALE * K[:, h // 2] @ qq[h]
            p = np.exp(x - x.max())
            p /= p.sum()
            ref = p @ V[:, h // 2]
            err = np.abs(host_f64(out[first + new[b] - 1])[h] - ref)
            # output 2^-8, P in bf16 2^-8 (it also enters the sum)
            assert (err <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2.0 ** -16) * (p @ np.abs(V[:, h // 2]))).all()

    weights = torch.zeros((2, hkv, 512), device="cuda")

    def step(ctx, ts, acc):
        store(rand_rows(2), rand_rows(2), ctx, ts, None)
        q = dev(w.host_bf16_normal(g, (2, hq, D)))
        args = (table_tensor(ts), dev(np.array(ctx, np.int32)), max(ctx), SCALE)
        if fp8:
            out = pkv.paged_decode_attn_fp8(q, kc, vc, ks, vs, *args, weights=acc)
        else:
            out = pkv.paged_decode_attn_weights(q, kc, vc, *args, acc)
        qs = host_f64(q)
        ref, tol = np.zeros_like(qs), np.zeros_like(qs)
        probs = []
        for b, n in enumerate(ctx):
            K, V = (rows_of(p, s, ts[b], n) for p, s in ((kc, scales[0]), (vc, scales[1])))
            pb = np.zeros((hkv, n))
            for h in range(hq):
                x = SCALE * K[:, h // 2] @ qs[b, h]
                p = np.exp(x - x.max())
                p /= p.sum()
                pb[h // 2] += p
                ref[b, h] = p @ V[:, h // 2]
                tol[b, h] = 2.0 ** -8 * np.abs(ref[b, h]) + (2.0 ** -11 + 2.0 ** -12) * (p @ np.abs(V[:, h // 2]))
            probs.append(pb)
        check_out(out, ref, tol, f"step at {ctx}")
        return probs

    total = [np.zeros((hkv, 512)) for _ in range(2)]
    ts = [list(t) for t in tables]
    for _ in range(3):
        lens = [n + 1 for n in lens]
        for b, pb in enumerate(step(lens, ts, weights)):
            total[b][:, :lens[b]] += pb
    got = weights.cpu().numpy()
    for b in range(2):
        assert np.allclose(got[b], total[b], rtol=1e-3, atol=2.0 ** -30)

    # evict into fresh blocks; the shared, registered block keeps its contents
    before = kc.view(torch.uint8)[tables[0][0]].clone()
    fresh = [bm.take(1), bm.take(1)]
    assert not set(fresh[0] + fresh[1]) & set(ts[0] + ts[1])
    kept, w2, n2 = pkv.kv_evict(weights, dev(np.array(lens, np.int32)), max(lens),
                                table_tensor(ts), table_tensor(fresh), budget, recent, kc, vc,
                                k_scale=scales[0], v_scale=scales[1])
    assert n2.tolist() == [128, 128]
    assert torch.equal(kc.view(torch.uint8)[tables[0][0]], before)
    kept_h = kept.cpu().numpy()
    for b in range(2):
        K = rows_of(kc, scales[0], ts[b], lens[b])
        K2 = rows_of(kc, scales[0], fresh[b], 128)
        for h in range(hkv):
            at = select(got[b, h].astype(np.float64), lens[b], budget, recent)
            assert np.array_equal(kept_h[b, h], at)
            # the same rows (8-bit: re-rounded to the group's scale, half a step of e4m3)
            tol = 2.0 ** -4 * np.abs(K[at, h]) + (2.0 ** -10 * scales[0][fresh[b][0], h].repeat_interleave(
                64)[:128].cpu().numpy()[:, None] if fp8 else 0) if fp8 else 0.0
            assert (np.abs(K2[:, h] - K[at, h]) <= tol).all()
    for t in ts:
        bm.deallocate(t)
    assert bm.block_hash(tables[0][0]) is not None        # still there to be hit

    # go on: positions 128, 129, .. of the compacted sequences
    weights2 = torch.zeros((2, hkv, 256), device="cuda")
    weights2[:, :, :budget] = w2
    lens = [128, 128]
    for _ in range(130):
        lens = [n + 1 for n in lens]
        if lens[0] % bs == 1:
            for t in fresh:
                t += bm.take(1)
        if lens[0] > 256:
            break
        if lens[0] in (129, 130, 200, 256):
            step(lens, fresh, weights2)
        else:
            store(rand_rows(2), rand_rows(2), lens, fresh, None)
    assert all(len(t) == 2 for t in fresh)
    assert pkv.get_device_errors() == 0


# --------------------------------------------------------------------- the block manager (CPU)
def test_take_hands_out_fresh_blocks():
    bm = pkv.BlockManager(6, 4)
    table, _ = bm.allocate(list(range(8)))
    assert table == [0, 1]
    assert bm.take(2) == [2, 3] and bm.num_free == 2
    assert bm.ref_count(2) == 1 and bm.block_hash(2) is None
    with pytest.raises(pkv.PkvError) as e:
        bm.take(3)
    assert e.value.status == pkv.ERR_NO_BLOCKS and bm.num_free == 2
    assert bm.take(0) == []
    with pytest.raises((pkv.PkvError, ValueError)):
        bm.take(-1)
    bm.deallocate([2, 3])
    bm.deallocate(table)                     # freed, still a possible hit
    assert bm.take(2) == [4, 5]
    again, cached = bm.allocate(list(range(8)))
    assert again == [0, 1] and cached == 8
    bm.deallocate(again)
    assert bm.take(4) == [3, 2, 1, 0]        # oldest freed first (a table: last block first)
    assert bm.block_hash(0) is None
    with pytest.raises(pkv.PkvError):
        bm.allocate([1])
