"""The 8-bit cache: the appending store and the gather against a 64-bit model, code for code.

The store's scales are powers of two, so x / scale is exact and both sides round the same
number once: codes and scales must be equal, not close. The gather's products are exact.
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


# ------------------------------------------------------------------ the model itself (CPU)
def test_model_matches_torch_e4m3():
    x = np.concatenate([f8.VALUES[~np.isnan(f8.VALUES)], np.linspace(-460, 460, 40001),
                        2.0 ** np.arange(-14, 9), 1.5 * 2.0 ** np.arange(-12, 8)])
    x = x[np.abs(x) <= 448]
    t = torch.from_numpy(x).float().to(torch.float8_e4m3fn)
    ok = torch.from_numpy(x).float().double().numpy() == x      # values that float32 holds
    assert np.array_equal(t.view(torch.uint8).numpy()[ok], f8.encode(x)[ok])
    back = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(back, f8.VALUES, equal_nan=True)


@pytest.mark.parametrize("top,e", [(448.0, 0), (449.0, 1), (896.0, 1), (0.0, -90), (1e-40, -90),
                                   (448.0 * 2.0 ** -7, -7), (450.0 * 2.0 ** -7, -6)])
def test_model_scale_rule(top, e):
    assert f8.scale_of(np.array([[top, 0.0, -top]])) == 2.0 ** e


# ------------------------------------------------------------------------------- the store
def _check(got_codes, got_scale, codes, scale, what):
    c = f8.host_codes(got_codes)
    bad = ~f8.same_codes(c, codes)
    assert not bad.any(), f"{what}: {bad.sum()} codes differ, first at {np.argwhere(bad)[0]}"
    assert np.array_equal(got_scale.cpu().numpy().astype(np.float64), scale), f"{what}: scales"


def _bf16(x):
    """float64 array -> (bf16 tensor on the device, the float64 values it holds)."""
    bits = w.f32_to_bf16_bits(x.astype(np.float32))
    return dev(bits), w.bf16_bits_to_f32(bits).astype(np.float64)


def _store_case(ctx, new, hkv, bs, seed, decode, fused=True):
    """One store of `new` rows per sequence ending at `ctx`, against the model."""
    g = w.rng(seed)
    ctx, new = np.asarray(ctx), np.asarray(new)
    tables, nb = f8.tables_for(ctx, bs, g)
    T = len(ctx) if decode else int(new.sum())
    x = g.standard_normal((T, 2, hkv, D)) * np.exp(g.standard_normal((T, 1, 1, 1)))
    qkv = np.concatenate([g.standard_normal((T, 3, hkv * D)), x.reshape(T, 2, hkv * D)], axis=1)
    t, vals = _bf16(qkv)
    if fused:   # views into a fused projection
        k, v = t[:, 3].view(T, hkv, D), t[:, 4].view(T, hkv, D)
    else:
        k, v = (t[:, i].reshape(T, hkv, D).contiguous() for i in (3, 4))
    cu = np.concatenate([[0], np.cumsum(new)])
    got, want = [], []
    for i in range(2):
        codes, scale = f8.random_cache(nb, bs, hkv, g)
        got += list(f8.device_cache(codes, scale))
        xs = vals[:, 3 + i].reshape(T, hkv, D)
        for b in range(len(ctx)):
            rows = xs[b:b + new[b]] if decode else xs[cu[b]:cu[b + 1]]
            f8.append(rows, codes, scale, tables[b], int(ctx[b] - new[b]))
        want += [codes, scale]
    pkv.kv_store_fp8(k, v, dev(ctx.astype(np.int32)), dev(tables), got[0], got[2], got[1],
                     got[3], cu_seqlens=None if decode else dev(cu.astype(np.int32)))
    torch.cuda.synchronize()
    _check(got[0], got[1], want[0], want[1], "K")
    _check(got[2], got[3], want[2], want[3], "V")
    assert pkv.get_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("hkv", [1, 2, 3, 8])
@pytest.mark.parametrize("bs", [256, 512])
def test_store_one_token_per_sequence(hkv, bs):
    ctx = [1, 2, 63, 64, 65, 128, 0, 129, 255, 256, 257, 511, 512, 513, 700, 1]
    _store_case(ctx, [min(1, c) for c in ctx], hkv, bs, 40 + hkv, decode=True)


@pytest.mark.gpu
@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("bs", [256, 768])
def test_store_ragged_chunks(hkv, bs):
    ctx = [1, 64, 65, 300, 130, 0, 600, 1000, 257, 64, 40]
    new = [1, 64, 65, 300, 3, 0, 77, 513, 2, 1, 0]
    _store_case(ctx, new, hkv, bs, 50 + hkv, decode=False)


@pytest.mark.gpu
def test_store_chunk_form_of_a_decode_step_and_one_long_prompt():
    _store_case([5, 65, 300], [1, 1, 1], 2, 256, 60, decode=False, fused=False)
    _store_case([9001], [9001], 2, 256, 61, decode=False)
    _store_case([4133], [4000], 1, 256, 62, decode=False)
    g = w.rng(63)      # many sequences, many of them without a new token
    ctx = g.integers(0, 200, 1500)
    _store_case(ctx, np.minimum(ctx, g.integers(0, 3, 1500)), 1, 256, 63, decode=False)


@pytest.mark.gpu
@pytest.mark.parametrize("decode", [True, False])
def test_store_grows_a_scale_step_by_step(decode):
    """Rows that double in size again and again: every append re-rounds the group's earlier
    rows, and the sequence of calls equals the model's."""
    g = w.rng(70)
    hkv, bs, n = 2, 256, 70
    tables, nb = f8.tables_for([n], bs, g)
    size = np.exp2(g.integers(-30, 30, n).cumsum() / 7.0)[:, None, None]
    t, vals = _bf16(g.standard_normal((n, hkv, D)) * size)
    codes, scale = f8.random_cache(nb, bs, hkv, g)
    kc, ks = f8.device_cache(codes, scale)
    vc, vs = f8.device_cache(codes, scale)
    bt = dev(tables)
    step = 1 if decode else 3
    for p in range(0, n, step):
        m = min(step, n - p)
        cu = None if decode else dev(np.array([0, m], np.int32))
        pkv.kv_store_fp8(t[p:p + m], t[p:p + m], dev(np.array([p + m], np.int32)), bt, kc, vc,
                         ks, vs, cu_seqlens=cu)
        f8.append(vals[p:p + m], codes, scale, tables[0], p)
    _check(kc, ks, codes, scale, "K")
    _check(vc, vs, codes, scale, "V")


@pytest.mark.gpu
@pytest.mark.parametrize("decode", [True, False])
def test_store_special_values(decode):
    """Infinities saturate, NaN stays NaN and neither moves the scale; zeros take the smallest
    scale; the largest and the smallest bf16 values."""
    hkv, bs = 2, 256
    g = w.rng(80)
    x = g.standard_normal((6, hkv, D))
    x[0, 0, 5], x[0, 0, 6], x[0, 1, 7] = np.inf, -np.inf, np.nan
    x[1, 0] = 0.0
    x[2, 1] = 3.0e38
    x[3, 0] = 1e-39
    x[4, 0, ::2] = np.nan
    x[5, 1] = -0.0
    t, vals = _bf16(x)
    ctx = np.arange(1, 7, dtype=np.int32) * 3
    tables, nb = f8.tables_for(ctx, bs, g)
    codes, scale = f8.random_cache(nb, bs, hkv, g)
    kc, ks = f8.device_cache(codes, scale)
    vc, vs = f8.device_cache(codes, scale)
    cu = None if decode else dev(np.arange(7, dtype=np.int32))
    pkv.kv_store_fp8(t, t, dev(ctx), dev(tables), kc, vc, ks, vs, cu_seqlens=cu)
    for b in range(6):
        f8.append(vals[b:b + 1], codes, scale, tables[b], int(ctx[b]) - 1)
    _check(kc, ks, codes, scale, "K")
    _check(vc, vs, codes, scale, "V")


@pytest.mark.gpu
def test_store_skips_bad_data_and_reports_it():
    """A bad length or block id skips that sequence's rows only; every other byte keeps."""
    hkv, bs = 2, 256
    g = w.rng(90)
    tables = np.array([[0, 1], [99, -1], [2, -1], [3, -7], [4, -1]], np.int32)
    codes, scale = f8.random_cache(6, bs, hkv, g)
    t, vals = _bf16(g.standard_normal((5, hkv, D)))
    for decode in (True, False):
        ctx = np.array([513, 5, -3, 257, 9], np.int32)    # past the table, block 99, < 0, -7
        if not decode:
            ctx[2] = 0                                     # fewer positions than new tokens
        c, s = codes.copy(), scale.copy()
        kc, ks = f8.device_cache(c, s)
        vc, vs = f8.device_cache(c, s)
        cu = None if decode else dev(np.arange(6, dtype=np.int32))
        pkv.kv_store_fp8(t, t, dev(ctx), dev(tables), kc, vc, ks, vs, cu_seqlens=cu)
        f8.append(vals[4:5], c, s, tables[4], 8)
        _check(kc, ks, c, s, "K")
        _check(vc, vs, c, s, "V")
        want = pkv.DEVERR_CONTEXT_RANGE | pkv.DEVERR_BLOCK_RANGE
        assert pkv.get_device_errors() == (want if decode else want | pkv.DEVERR_SEQLEN_RANGE)
    # cu_seqlens that go down, below zero and past the rows: nothing but an error bit
    for cu in ([0, 3, 1, 5, 5, 5], [-4, 0, 0, 0, 0, 0], [0, 0, 0, 0, 0, 70]):
        kc, ks = f8.device_cache(codes, scale)
        vc, vs = f8.device_cache(codes, scale)
        tb = np.array([[0, 1], [1, -1], [2, -1], [3, -1], [4, -1]], np.int32)
        pkv.kv_store_fp8(t, t, dev(np.zeros(5, np.int32)), dev(tb), kc, vc, ks, vs,
                         cu_seqlens=dev(np.array(cu, np.int32)))
        assert pkv.get_device_errors() & pkv.DEVERR_SEQLEN_RANGE
        _check(kc, ks, codes, scale, "K")


# ------------------------------------------------------------------------------ the gather
@pytest.mark.gpu
@pytest.mark.parametrize("hkv,bs", [(1, 256), (3, 512), (8, 256)])
def test_gather(hkv, bs):
    g = w.rng(100 + hkv)
    lens = np.array([1, 64, 0, 65, 300, 257, 63, 1025, 0, 2])
    tables, nb = f8.tables_for(lens, bs, g)
    tables[4, 0] = tables[7, 0]      # a shared block
    kc, ks = f8.random_cache(nb, bs, hkv, g)
    vc, vs = f8.random_cache(nb, bs, hkv, g)
    cu = np.concatenate([[3], 3 + np.cumsum(lens)])      # rows 0..2 and the last 5 belong to nobody
    total = int(cu[-1]) + 5
    ko, vo = (torch.full((total, hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    (kd, ksd), (vd, vsd) = f8.device_cache(kc, ks), f8.device_cache(vc, vs)
    got = pkv.kv_gather_fp8(kd, vd, ksd, vsd, dev(tables), dev(cu.astype(np.int32)), total,
                            k_out=ko, v_out=vo)
    assert got[0] is ko and got[1] is vo
    for out, c, s in ((ko, kc, ks), (vo, vc, vs)):
        o = host_f64(out)
        assert (o[:3] == 7).all() and (o[cu[-1]:] == 7).all()
        for b, n in enumerate(lens):
            want = f8.rows(c, s, tables[b], int(n))
            assert np.array_equal(o[cu[b]:cu[b + 1]], want, equal_nan=True), b
    assert pkv.get_device_errors() == 0


@pytest.mark.gpu
def test_gather_bad_data():
    g = w.rng(110)
    kc, ks = f8.random_cache(3, 256, 2, g)
    kd, ksd = f8.device_cache(kc, ks)
    tables = dev(np.array([[0, 55], [1, 2]], np.int32))
    out = pkv.kv_gather_fp8(kd, kd, ksd, ksd, tables, dev(np.array([0, 300, 310], np.int32)), 310)
    o = host_f64(out[0])
    assert np.array_equal(o[:256], f8.rows(kc, ks, [0], 256), equal_nan=True)
    assert (o[256:300] == 0).all()
    assert np.array_equal(o[300:], f8.rows(kc, ks, [1], 10), equal_nan=True)
    assert pkv.get_device_errors() == pkv.DEVERR_BLOCK_RANGE
    for cu in ([0, 700, 700], [0, 5, 3], [0, 5, 400]):   # past the table, down, past the rows
        pkv.kv_gather_fp8(kd, kd, ksd, ksd, tables, dev(np.array(cu, np.int32)), 310)
        assert pkv.get_device_errors() & (pkv.DEVERR_SEQLEN_RANGE | pkv.DEVERR_CONTEXT_RANGE)


# ---------------------------------------------------------------------- refusals (CPU side)
def _cpu_cache(nb=2, bs=256, hkv=2):
    c = torch.zeros((nb, bs, hkv, D), dtype=torch.uint8).view(torch.float8_e4m3fn)
    return c, torch.ones((nb, hkv, bs // 64))


def test_host_tensors_are_refused():
    c, s = _cpu_cache()
    t = torch.zeros((1, 2, D), dtype=torch.bfloat16)
    i = torch.zeros((1, 1), dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.kv_store_fp8(t, t, i[0], i, c, c, s, s)
    with pytest.raises(ValueError):
        pkv.kv_gather_fp8(c, c, s, s, i, torch.zeros(2, dtype=torch.int32), 1)


@pytest.mark.gpu
def test_refusals():
    c, s = (t.cuda() for t in _cpu_cache())
    t = torch.zeros((1, 2, D), dtype=torch.bfloat16, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    bt = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    ok = dict(k=t, v=t, context_lens=one, block_tables=bt, k_cache=c, v_cache=c, k_scale=s,
              v_scale=s)
    bad = [("k", t.float()), ("k", t[:, :1]), ("v", t[:0]), ("k", t.transpose(1, 2)),
           ("context_lens", one.long()), ("block_tables", bt[:, 0]), ("k_cache", c.view(torch.uint8)),
           ("k_scale", s[:, :1]), ("v_scale", s.double()), ("k_cache", c[:, :, :1]),
           ("context_lens", torch.ones(3, dtype=torch.int32, device="cuda"))]
    for name, value in bad:
        with pytest.raises((TypeError, ValueError)):
            pkv.kv_store_fp8(**{**ok, name: value})
    with pytest.raises(ValueError):
        pkv.kv_store_fp8(**ok, cu_seqlens=one)
    with pytest.raises(pkv.PkvError) as e:       # two sequences, one token, no cu_seqlens
        pkv.kv_store_fp8(**{**ok, "context_lens": one.repeat(2), "block_tables": bt.repeat(2, 1)})
    assert e.value.status == pkv.ERR_INVALID_ARG
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    for kw in (dict(k_out=t), dict(v_out=t.float())):
        with pytest.raises((TypeError, ValueError)):
            pkv.kv_gather_fp8(c, c, s, s, bt, cu, 5, **kw)


@pytest.mark.gpu
def test_empty_calls():
    c, s = (t.cuda() for t in _cpu_cache())
    t = torch.zeros((0, 2, D), dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    bt = torch.zeros((0, 1), dtype=torch.int32, device="cuda")
    pkv.kv_store_fp8(t, t, none, bt, c, c, s, s)
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = pkv.kv_gather_fp8(c, c, s, s, bt, cu, 0)
    assert k.shape == v.shape == (0, 2, D)
