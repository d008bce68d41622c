"""The calls of speculative decoding the way programs make them: several at once, captured graphs that
share a workspace, batches with padding, and what must not spread from one row to another."""
import os
import re

import numpy as np
import pytest
import torch

from libbuild import ROOT, build_and_import
from tree_util import Case, D, assert_close, bf16_weights, ints

pkv = build_and_import()
pytestmark = pytest.mark.gpu
BOTH = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])


def check(c, out):
    assert pkv.get_device_errors(reset=True) == 0
    ref, size = c.reference()
    assert_close(out, ref, size, c.fp8, bf16_weights(c.most, c.hq // c.hkv))


@BOTH
def test_calls_on_two_streams_at_once(fp8):
    cases = [Case([3000, 200, 70], [9, 4, 1], 8, 2, fp8=fp8, seed=1),
             Case([90, 2500, 600, 1], [5, 30, 2, 1], 16, 2, fp8=fp8, seed=2)]
    want = [c.attend(pkv) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[] for _ in cases]
    for _ in range(20):
        for i, (c, s) in enumerate(zip(cases, streams)):
            outs[i].append(c.attend(pkv, stream=s))
    torch.cuda.synchronize()
    for ref, got in zip(want, outs):
        for o in got:
            assert torch.equal(o, ref)
    for c, ref in zip(cases, want):
        check(c, ref)


@BOTH
def test_two_graphs_that_share_a_workspace(fp8):
    cases = [Case([3000, 200, 70], [9, 4, 1], 8, 2, fp8=fp8, seed=3),
             Case([90, 2500, 600], [5, 30, 2], 8, 2, fp8=fp8, seed=4)]
    want = [c.attend(pkv) for c in cases]
    ws = pkv.tree_workspace(3, 30, 8, 2, D, 3000)
    ws.fill_(255)
    graphs, outs = [], []
    torch.cuda.synchronize()
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.attend(pkv, workspace=ws))
        graphs.append(g)
    for turn in (0, 1, 1, 0, 1, 0, 0):
        outs[turn].zero_()
        graphs[turn].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[turn], want[turn])
    for c, ref in zip(cases, want):
        check(c, ref)


@BOTH
@pytest.mark.parametrize("batch", [2, 9, 10, 16, 19, 20, 21, 38, 40])
def test_batches_around_the_number_of_workers(batch, fp8):
    """Whole units to a worker, cuts that move to a unit's end, and cuts that stay."""
    rng = np.random.default_rng(batch)
    for spread in (0, 40, 700):
        ctx = [int(n) for n in 900 - rng.integers(0, spread + 1, batch)]
        c = Case(ctx, [int(n) for n in rng.integers(1, 5, batch)], 16, 8, fp8=fp8, seed=batch)
        check(c, c.attend(pkv))


@BOTH
@pytest.mark.parametrize("batch", [1, 2, 3, 5, 6, 8, 10, 16])
@pytest.mark.parametrize("length", [512, 513, 1024, 1025, 1280, 1281, 1536, 1537])
def test_lengths_up_to_which_nothing_is_cut(batch, length, fp8):
    c = Case([length] * (batch - 1) + [length - 300], [3] * batch, 16, 8, fp8=fp8, seed=length + batch)
    check(c, c.attend(pkv))


@BOTH
def test_any_aligned_workspace_and_output(fp8):
    """16-byte aligned addresses: no more is promised."""
    c = Case([5000, 300], [6, 17], 8, 2, fp8=fp8, seed=5)
    n = pkv.tree_workspace(2, c.most, 8, 2, D, 5000).numel()
    for at in (16, 48):
        ws = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")
        room = torch.zeros((23 * 8 * D + 64,), dtype=torch.bfloat16, device="cuda")
        out = room[at // 2:at // 2 + 23 * 8 * D].view(23, 8, D)
        c.attend(pkv, workspace=ws[at:at + n], out=out)
        check(c, out)
        assert (ws[:at] == 255).all() and (ws[at + n:] == 255).all()
        assert (room[:at // 2] == 0).all() and (room[at // 2 + 23 * 8 * D:] == 0).all()


@BOTH
@pytest.mark.parametrize("scale", [-0.11, 0.0, 1e-30])
def test_other_scales(scale, fp8):
    c = Case([700, 65], [6, 3], 6, 2, fp8=fp8, seed=6)
    c.scale = scale
    check(c, c.attend(pkv))


@BOTH
def test_looser_bounds_and_wider_masks(fp8):
    """A program passes the bounds of its largest batch; bits at n and above do not count."""
    c = Case([700, 65, 1200], [6, 3, 70], 4, 2, fp8=fp8, seed=7)
    want = c.attend(pkv)
    c.mask = torch.cat([c.mask, torch.full((79, 3), -1, dtype=torch.int64, device="cuda")], 1)
    t = 0
    for n in c.nodes:  # every bit behind the tree's last node
        for w in range(2):
            first = min(64, max(0, n - 64 * w))
            keep = (1 << first) - 1
            high = np.array([~keep & (2 ** 64 - 1)], np.uint64).view(np.int64)[0]
            c.mask[t:t + n, w] |= int(high)
        t += n
    c.most = 300
    out = c.attend(pkv)
    check(c, out)
    args = (c.tables, c.lens, 2 ** 31 - 1, c.cu, 70, c.scale)
    if fp8:
        loose = pkv.paged_tree_attn_fp8(c.q, c.k, c.v, *c.scales, *args, c.mask)
    else:
        loose = pkv.paged_tree_attn(c.q, c.k, c.v, *args, c.mask)
    c.most = 70
    check(c, loose)
    check(c, want)


@BOTH
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_a_row_of_q_that_is_not_finite_spoils_itself_only(what, fp8):
    c = Case([700, 300], [6, 20], 6, 2, fp8=fp8, seed=8)
    clean = c.attend(pkv)
    q = c.q.clone()
    q[3, 4, 17] = what
    q[12, 0, 100] = what
    c.q = q
    out = c.attend(pkv)
    hit = torch.zeros((26, 6), dtype=torch.bool, device="cuda")
    hit[3, 4] = hit[12, 0] = True
    assert torch.equal(out[~hit], clean[~hit])
    assert torch.isnan(out[hit]).all()


def append_args():
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    qkv = torch.randn((90, 8 * D), generator=g, device="cuda").to(torch.bfloat16)
    angle = torch.rand((200, D // 2), generator=g, device="cuda") * 6
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1)
    w = torch.ones((D,), dtype=torch.bfloat16, device="cuda")
    return dict(qkv=qkv, positions=torch.arange(90, device="cuda"), cos_sin_cache=cos_sin,
                context_lens=ints([90]), block_tables=ints([[1]]),
                k_cache=torch.zeros((2, 256, 2, D), dtype=torch.float8_e4m3fn, device="cuda"),
                v_cache=torch.zeros((2, 256, 2, D), dtype=torch.float8_e4m3fn, device="cuda"),
                k_scale=torch.full((2, 2, 4), 0.5, device="cuda"),
                v_scale=torch.full((2, 2, 4), 0.5, device="cuda"), num_q_heads=4, q_norm_weight=w,
                k_norm_weight=w, cu_seqlens=ints([0, 90]),
                q_out=torch.full((90, 4, D), 3.0, dtype=torch.bfloat16, device="cuda"))


@BOTH
def test_abort_bit_stops_the_tree_and_the_paths(fp8):
    c = Case([5000, 300], [6, 17], 8, 2, fp8=fp8, seed=10)
    out = torch.full((23, 8, D), 3.0, dtype=torch.bfloat16, device="cuda")
    new = ints([-7, -7])
    k = c.k.view(torch.uint8).clone()
    lists = (ints([[1, 4], [0, 9]]), ints([2, 2]), c.cu, c.lens, c.tables, c.k, c.v, *c.scales)
    pkv.raise_device_errors(pkv.DEVERR_TIMEOUT)
    try:
        c.attend(pkv, out=out)
        pkv.kv_accept(*lists, new_context_lens=new)
        torch.cuda.synchronize()
        assert (out == 3).all() and new.tolist() == [-7, -7]
        assert torch.equal(c.k.view(torch.uint8), k)
    finally:
        assert pkv.get_device_errors() == pkv.DEVERR_TIMEOUT
    c.attend(pkv, out=out)
    check(c, out)
    pkv.kv_accept(*lists, new_context_lens=new)
    assert new.tolist() == [4996, 285] and pkv.get_device_errors() == 0


@pytest.mark.parametrize("step", [False, True])
def test_abort_bit_stops_the_append(step):
    a = append_args()
    if step:
        a.update(cu_seqlens=None, qkv=a["qkv"][:1], positions=a["positions"][:1], q_out=a["q_out"][:1])
    pkv.raise_device_errors(pkv.DEVERR_TIMEOUT)
    try:
        pkv.qk_norm_rope_store_fp8(**a)
        torch.cuda.synchronize()
        assert (a["q_out"] == 3).all() and (a["k_scale"] == 0.5).all()
        assert (a["k_cache"].float() == 0).all() and (a["v_cache"].float() == 0).all()
    finally:
        assert pkv.get_device_errors() == pkv.DEVERR_TIMEOUT
    pkv.qk_norm_rope_store_fp8(**a)
    assert not (a["q_out"] == 3).all() and (a["k_cache"].float() != 0).any()
    assert pkv.get_device_errors() == 0


def test_outputs_that_overlap_inputs_are_refused():
    c = Case([70], [3], 4, 2, seed=11)
    with pytest.raises(pkv.PkvError) as e:
        c.attend(pkv, out=c.q)
    assert e.value.status == pkv.ERR_INVALID_ARG
    a = append_args()
    a["q_out"] = a["qkv"].view(-1)[:90 * 4 * D].view(90, 4, D)
    with pytest.raises(pkv.PkvError) as e:
        pkv.qk_norm_rope_store_fp8(**a)
    assert e.value.status == pkv.ERR_INVALID_ARG


def test_appends_of_many_layers_and_streams():
    """The same call into four layers' caches, two of them on another stream: the same codes."""
    a = append_args()
    s = torch.cuda.Stream()
    pools = []
    torch.cuda.synchronize()
    for i in range(4):
        b = dict(a, k_cache=torch.zeros_like(a["k_cache"]), v_cache=torch.zeros_like(a["v_cache"]),
                 k_scale=a["k_scale"].clone(), v_scale=a["v_scale"].clone(), q_out=None)
        torch.cuda.synchronize()
        q = pkv.qk_norm_rope_store_fp8(**b, stream=s if i & 1 else None)
        pools.append([q.view(torch.uint8), b["k_cache"].view(torch.uint8), b["v_cache"].view(torch.uint8),
                      b["k_scale"], b["v_scale"]])
    torch.cuda.synchronize()
    for other in pools[1:]:
        for x, y in zip(pools[0], other):
            assert torch.equal(x, y)


def test_the_step_of_the_readme():
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    (code,) = [b for b in blocks if "kv_accept" in b]
    c = Case([700, 90, 300], [5, 1, 9], 8, 2, fp8=True, seed=12)
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    angle = torch.rand((800, D // 2), generator=g, device="cuda") * 6
    w = torch.ones((D,), dtype=torch.bfloat16, device="cuda")
    names = dict(pkv=pkv, qkv=torch.randn((15, 12 * D), generator=g, device="cuda").to(torch.bfloat16),
                 positions=torch.arange(15, device="cuda"), num_q_heads=8, q_weight=w, k_weight=w,
                 cos_sin=torch.cat([angle.cos(), angle.sin()], 1), context_lens=c.lens,
                 tables=c.tables, k_cache=c.k, v_cache=c.v, k_scale=c.scales[0], v_scale=c.scales[1],
                 cu_seqlens_q=c.cu, max_context_len=700, max_nodes=9, scale=c.scale,
                 tree_mask=c.mask, accepted=ints([[0, 3], [0, -1], [2, 8]]),
                 num_accepted=ints([2, 1, 2]))
    layer = code.split("# ...")
    exec(compile(layer[0], "README.md", "exec"), names)
    c.q = names["q"]
    check(c, names["out"])
    exec(compile("# ..." + layer[1], "README.md", "exec"), names)
    assert names["new_lens"].tolist() == [697, 90, 293]
    assert pkv.get_device_errors(reset=True) == 0
