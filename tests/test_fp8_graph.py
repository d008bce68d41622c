"""The 8-bit cache's calls captured together in one CUDA graph, as a server replays a step, and
inputs that name the same block or sequence more than once."""
import numpy as np
import pytest
import torch

import fp8_util as f8
import workloads as w
from gpu_util import dev, host_bits
from libbuild import build_and_import

pkv = build_and_import()
D = 128


@pytest.mark.gpu
def test_captured_step_equals_eager_calls():
    """store, decode with weights, gather and evict in one graph over fixed buffers, a batch
    padded with empty rows; every replay against the same calls made eagerly on copies."""
    g = w.rng(900)
    hq, hkv, bs, live, rows, longest, budget = 8, 4, 256, 3, 5, 600, 70
    ctx0 = [63, 300, 511]
    tables, nb = f8.tables_for([longest] * live + [budget] * rows, bs, g)
    src = np.full((rows, 3), -1, np.int32)
    src[:live] = tables[:live, :3]
    src, dst = dev(src), dev(np.ascontiguousarray(tables[live:, :1]))
    start = [t for _ in range(2) for t in f8.device_cache(*f8.random_cache(nb, bs, hkv, g))]
    steps = [[dev(w.host_bf16_normal(g, (rows, n, D))) for n in (hq, hkv, hkv)] for _ in range(3)]
    total = sum(ctx0) + 3 * live

    class State:
        def __init__(self):
            self.kc, self.ks, self.vc, self.vs = (t.clone() for t in start)
            self.q, self.k, self.v = (torch.zeros_like(t) for t in steps[0])
            self.ctx = torch.zeros(rows, dtype=torch.int32, device="cuda")
            self.cu = torch.zeros(rows + 1, dtype=torch.int32, device="cuda")
            self.acc = torch.zeros((rows, hkv, longest), device="cuda")
            self.out = torch.empty_like(self.q)
            self.kg, self.vg = (torch.zeros((total, hkv, D), dtype=torch.bfloat16, device="cuda")
                                for _ in range(2))
            self.space = pkv.decode_fp8_workspace(rows, hq, hkv, D, longest, weights=True)
            self.kept = torch.empty((rows, hkv, budget), dtype=torch.int32, device="cuda")
            self.w_out = torch.empty((rows, hkv, budget), device="cuda")
            self.lens = torch.empty(rows, dtype=torch.int32, device="cuda")

        def load(self, step):
            for mine, t in zip((self.q, self.k, self.v), steps[step]):
                mine.copy_(t)
            ctx = np.zeros(rows, np.int32)
            ctx[:live] = np.array(ctx0) + step + 1
            self.ctx.copy_(dev(ctx))
            self.cu.copy_(dev(np.concatenate([[0], np.cumsum(ctx)]).astype(np.int32)))

        def run(self):
            pools = (self.kc, self.vc, self.ks, self.vs)
            pkv.kv_store_fp8(self.k, self.v, self.ctx, src, *pools)
            pkv.paged_decode_attn_fp8(self.q, *pools, src, self.ctx, longest, D ** -0.5,
                                      weights=self.acc, workspace=self.space, out=self.out)
            pkv.kv_gather_fp8(*pools, src, self.cu, total, self.kg, self.vg)
            pkv.kv_evict(self.acc, self.ctx, longest, src, dst, budget, 16, self.kc, self.vc,
                         self.ks, self.vs, self.kept, self.w_out, self.lens)

        def results(self):
            return [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
                    for t in (self.kc, self.vc, self.ks, self.vs, self.acc, self.out, self.kg,
                              self.vg, self.kept, self.w_out, self.lens)]

    eager, replayed = State(), State()
    replayed.run()                       # (an empty batch, nothing but the warm-up)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed.run()
    for step in range(3):
        for s in (eager, replayed):
            s.load(step)
        eager.run()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(eager.results(), replayed.results())):
            assert torch.equal(a, b), (step, i)
        assert (eager.out[live:] == 0).all() and eager.lens.tolist() == [
            min(budget, n + step + 1) for n in ctx0] + [0] * (rows - live)
    assert pkv.get_device_errors() == 0


@pytest.mark.gpu
def test_shared_blocks_are_read_by_many():
    """One table row for every sequence: gathered and evicted as if each had blocks of its own."""
    g = w.rng(910)
    hkv, bs, n, many, budget = 2, 256, 400, 6, 130
    tables, nb = f8.tables_for([n] + [budget] * many, bs, g)
    pools = [f8.random_cache(nb, bs, hkv, g) for _ in range(2)]
    (kc, ks), (vc, vs) = (f8.device_cache(*p) for p in pools)
    lens = [n - 7 * i for i in range(many)]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    src = dev(np.repeat(tables[:1], many, 0))
    k, v = pkv.kv_gather_fp8(kc, vc, ks, vs, src, dev(cu), int(cu[-1]))
    for (codes, scale), got in zip(pools, (k, v)):
        want = f8.rows(codes, scale, tables[0], n)
        got = w.bf16_bits_to_f32(host_bits(got)).astype(np.float64)
        for i, m in enumerate(lens):
            assert np.array_equal(got[cu[i]:cu[i + 1]], want[:m], equal_nan=True), i
    wts = torch.rand((1, hkv, n), device="cuda").expand(many, hkv, n).contiguous()
    ctx = torch.full((many,), n, dtype=torch.int32, device="cuda")
    dst = np.ascontiguousarray(tables[1:, :1])
    kept, w_out, _ = pkv.kv_evict(wts, ctx, n, src, dev(dst), budget, 20, kc, vc, ks, vs)
    for i in range(1, many):
        assert torch.equal(kept[i], kept[0]) and torch.equal(w_out[i], w_out[0])
        for t in (kc, vc):
            t = t.view(torch.uint8)
            assert torch.equal(t[dst[i, 0], :budget], t[dst[0, 0], :budget])
    # the source blocks are as they were
    for (codes, _), t in zip(pools, (kc, vc)):
        at = tables[0, :2]
        assert np.array_equal(f8.host_codes(t)[at], codes[at])


@pytest.mark.gpu
def test_many_short_sequences():
    """More sequences than one step of the run search tells apart, most of them short or empty."""
    g = w.rng(920)
    hkv, bs, B = 1, 256, 2500
    lens = g.integers(0, 80, B) * (g.random(B) < 0.7)
    tables, nb = f8.tables_for(np.minimum(lens, 1), bs, g)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    codes, scale = f8.random_cache(nb, bs, hkv, g)
    kc, ks = f8.device_cache(codes, scale)
    k, v = pkv.kv_gather_fp8(kc, kc, ks, ks, dev(tables), dev(cu), int(cu[-1]))
    want = np.concatenate([f8.rows(codes, scale, tables[b], int(lens[b])) for b in range(B)])
    for got in (k, v):
        got = w.bf16_bits_to_f32(host_bits(got)).astype(np.float64)
        assert np.array_equal(got, want, equal_nan=True)
    assert pkv.get_device_errors() == 0


@pytest.mark.gpu
def test_out_of_memory_is_torchs_error():
    kc = torch.zeros((1, 256, 8, D), device="cuda").to(torch.float8_e4m3fn)
    ks = torch.ones((1, 8, 4), device="cuda")
    with pytest.raises(torch.OutOfMemoryError):   # 2^31 rows of 2 KiB, more than any device has
        pkv.kv_gather_fp8(kc, kc, ks, ks, torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                          torch.zeros(2, dtype=torch.int32, device="cuda"), 2 ** 31)
