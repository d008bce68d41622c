"""Attention of drafted tokens where values are not finite, vanish or lie far apart, and in workspaces of
other calls."""
import numpy as np
import pytest
import torch

from libbuild import build_and_import
from tree_util import Case, D, assert_close, bf16_weights, rows_of

pkv = build_and_import()
pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def put(c, name, b, pos, h, dim, value):
    blk, off = int(c.table_host[b, pos // c.bs]), pos % c.bs
    getattr(c, name)[blk, off, h, dim] = value


# one row tile and several, whole units and cut ones
@pytest.mark.parametrize("ctx,nodes,hq,hkv", [([300, 90], [4, 3], 4, 2), ([17188], [13], 12, 4),
                                              ([700, 300], [40, 3], 32, 4), ([9000, 400], [70, 9], 8, 2)])
def test_an_infinite_value_of_the_context_is_an_infinity(ctx, nodes, hq, hkv):
    """softmax weights are positive: a sum with an infinity is that infinity, with both signs NaN."""
    c = Case(ctx, nodes, hq, hkv, seed=1)
    ref, size = c.reference()
    first = ctx[0] - nodes[0]  # positions of the context below this
    put(c, "v", 0, 37, 0, 5, INF)
    put(c, "v", 0, first - 1, 1, 64, -INF)
    put(c, "v", 0, 3, 1, 9, INF)
    put(c, "v", 0, first - 2, 1, 9, INF)
    put(c, "v", 0, 11, 0, 100, INF)
    put(c, "v", 0, first // 2, 0, 100, -INF)
    put(c, "v", 0, 12, 0, 101, NAN)
    put(c, "v", 0, first // 2, 0, 101, INF)
    pkv.get_device_errors(reset=True)
    out = c.attend(pkv).float()
    assert pkv.get_device_errors(reset=True) == 0
    g, n = hq // hkv, nodes[0]
    assert (out[:n, :g, 5] == INF).all()
    assert (out[:n, g:2 * g, 64] == -INF).all()
    assert (out[:n, g:2 * g, 9] == INF).all()
    assert torch.isnan(out[:n, :g, 100]).all() and torch.isnan(out[:n, :g, 101]).all()
    hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    for h, d in ((0, 5), (1, 64), (1, 9), (0, 100), (0, 101)):
        hit[:n, h * g:(h + 1) * g, d] = True
    assert_close(out[~hit], ref[~hit], size[~hit], False, bf16_weights(c.most, g))


@pytest.mark.parametrize("ctx,nodes,hq,hkv", [([700], [5], 4, 2), ([17188], [13], 12, 4), ([9000], [70], 8, 2)])
def test_an_infinite_value_counts_however_small_its_weight(ctx, nodes, hq, hkv):
    """Scores that spread over hundreds: most weights are below what fp32 holds."""
    c = Case(ctx, nodes, hq, hkv, seed=2)
    c.q = (c.q.float() * 100).to(torch.bfloat16)
    for i in range(0, 60):
        put(c, "v", 0, i * (ctx[0] - nodes[0]) // 60, i % hkv, i, INF if i % 2 else -INF)
    out = c.attend(pkv).float()
    for i in range(60):
        heads = slice(i % hkv * (hq // hkv), (i % hkv + 1) * (hq // hkv))
        assert (out[:, heads, i] == (INF if i % 2 else -INF)).all(), i
        assert torch.isfinite(out[:, heads, 60:]).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("scale", [0.0, 1e-30, -1e-12, 0.09])
def test_a_row_of_zeros_is_the_mean(scale, fp8):
    """Scores of 0, with contexts that end in the first and in the second half of a tile."""
    c = Case([700, 65, 64, 128, 60, 5000], [6, 3, 2, 5, 1, 4], 6, 2, fp8=fp8, seed=3)
    c.scale = scale
    q = c.q.clone()
    q[::2, ::2] = 0
    q[1::2, 1] = 0
    c.q = q
    out = c.attend(pkv)
    ref, size = c.reference()
    assert_close(out, ref, size, fp8)


# whole units and cut ones, one row tile and several
@pytest.mark.parametrize("ctx,n,hq,hkv", [(300, 6, 4, 2), (17188, 13, 12, 4), (9000, 70, 8, 2)])
def test_infinities_of_nodes_leave_what_is_nan_or_infinite_already(ctx, n, hq, hkv):
    c = Case([ctx, 200], [n, 2], hq, hkv, seed=4)
    g, node = hq // hkv, 2
    sees = torch.from_numpy(c.masks[0][:, node]).cuda()
    assert sees[node + 1:].any() and not sees.all()
    at = ctx - n + node
    for dim in (3, 70, 90, 91):
        put(c, "v", 0, at, 0, dim, INF)
    put(c, "v", 0, 40, 0, 70, -INF)
    put(c, "v", 0, ctx - n - 1, 0, 90, NAN)
    put(c, "v", 0, 41, 0, 91, INF)
    q = c.q.clone()
    q[node, 0, 17] = NAN
    c.q = q
    out = c.attend(pkv).float()[:n, :g]
    lost = torch.zeros((n, g), dtype=torch.bool, device="cuda")
    lost[node, 0] = True
    assert torch.isnan(out[lost]).all()
    seen = sees[:, None] & ~lost
    for dim, want in ((3, INF), (70, NAN), (90, NAN), (91, INF)):
        x = out[..., dim]
        assert (torch.isnan(x[seen]) if want != want else x[seen] == want).all(), dim
        x = x[~sees[:, None] & ~lost]
        want = {3: 0.0, 70: -INF, 90: NAN, 91: INF}[dim]
        assert (torch.isnan(x) if want != want else torch.isfinite(x) if want == 0 else x == want).all(), dim


@pytest.mark.parametrize("hq,hkv", [(16, 8), (32, 8), (16, 2), (12, 4), (6, 1), (48, 3), (64, 4), (20, 1)])
def test_a_workspace_is_enough_for_smaller_bounds(hq, hkv):
    seqs = (1, 2, 3, 8, 19, 20, 33, 64, 256, 1000)
    nodes = (1, 2, 7, 8, 9, 16, 17, 32, 33, 48, 64, 65, 96, 97, 128, 129, 200, 256, 257, 400, 1000)
    lens = (1, 64, 65, 128, 500, 4096, 32768, 2 ** 31 - 1)
    size = np.array([[[pkv.lib().pkv_tree_workspace_bytes(b, n, hq, hkv, D, L) for L in lens] for n in nodes]
                     for b in seqs])
    for axis in range(3):
        assert (np.diff(size, axis=axis) >= 0).all(), axis


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("hq,hkv,large", [(32, 8, 65), (16, 2, 33)])
def test_one_workspace_for_trees_of_all_sizes(hq, hkv, large, fp8):
    ws = pkv.tree_workspace(16, large, hq, hkv, D, 4096)
    ws.fill_(255)
    rng = np.random.default_rng(13)
    for n, batch in ((large, 16), (large - 1, 16), (8, 16), (1, 3)):
        ctx = [int(x) for x in rng.integers(3000, 4097, batch)]
        c = Case(ctx, [n] * batch, hq, hkv, fp8=fp8, seed=n)
        out = c.attend(pkv, workspace=ws)
        ref, size = c.reference()
        assert_close(out, ref, size, fp8, bf16_weights(n, hq // hkv))


@pytest.mark.parametrize("ctx,n,hq,hkv", [([700, 190, 64], 5, 4, 2), ([9000], 30, 8, 1), ([2500, 1300], 20, 16, 2)])
def test_scales_of_v_that_lie_far_apart(ctx, n, hq, hkv):
    """A weight with its V scale is an fp16 number, the largest of a row at least 2^6: it is off by 2^-11 of
    itself or by 2^-25, 2^-31 of the largest, times its code. Half of the dims are zeros in the groups
    with large scales, so that what those with small ones add up to is all there is."""
    rng = np.random.default_rng(5)
    c = Case(ctx, [n] * len(ctx), hq, hkv, fp8=True, seed=5)
    scale = c.scales[1]  # [blocks, heads, groups]
    e = torch.from_numpy(rng.choice([-90, -24, -20, -12, -8, 5], scale.shape)).cuda()
    scale.copy_(torch.where(torch.isnan(scale), scale, torch.exp2(e.float())))
    codes = c.v.view(torch.uint8).view(c.nb, c.bs // 64, 64, hkv, D)
    e = e.transpose(1, 2)  # [blocks, groups, heads]
    codes[(e == -90)[:, :, None, :].expand(-1, -1, 64, -1)] = 0
    large = (e >= -8)[:, :, None, :].expand(-1, -1, 64, -1)
    codes[..., 64:][large] = 0
    out = c.attend(pkv).double()
    ref, size = c.reference()
    floor = torch.zeros_like(ref)
    t = 0
    for b, L in enumerate(ctx):
        sees = torch.ones((n, L), dtype=torch.bool)
        sees[:, L - n:] = torch.from_numpy(c.masks[b])
        sees = sees.cuda()[:, None, None, :]
        q = c.q[t:t + n].double().view(n, hkv, hq // hkv, D)
        x = torch.einsum("nhgd,lhd->nhgl", q, c.values("k", b)) * c.scale
        p = torch.softmax(x.masked_fill(~sees, -INF), dim=-1)
        r = torch.from_numpy(rows_of(c.table_host[b], L, c.bs)).cuda()
        s = c.scales[1].transpose(1, 2).reshape(-1, hkv)[r // 64].double()  # [L, heads]
        code = (c.values("v", b) / s[..., None]).abs()
        top = (p * s.T[None, :, None, :]).amax(-1, keepdim=True)
        total = torch.einsum("nl,lhd->nhd", sees[:, 0, 0].double(), code)[:, :, None, :]
        floor[t:t + n] = (2.0 ** -31 * top * total).reshape(n, hq, D)
        t += n
    bound = 2.0 ** -8 * ref.abs() + 2.0 ** -9 * size + floor
    assert ((out - ref).abs() <= bound).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_a_value_that_is_not_finite_in_a_large_tree(fp8):
    """2^18 nodes in a chain, behind 700 positions: what they see of it is found in a bounded time."""
    n, P, bs = 1 << 18, 700, 256
    L = P + n
    nb = -(-L // bs)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    rand = lambda rows, m: m * torch.randn((rows, 1, D), generator=g, device="cuda")
    q = rand(n, 1.0).to(torch.bfloat16)
    k, v = rand(nb * bs, 1.0), rand(nb * bs, 0.3)
    kind, scales = (torch.float8_e4m3fn if fp8 else torch.bfloat16), ()
    k, v = k.to(kind), v.to(kind)
    if fp8:
        scales = tuple(torch.ones((nb, 1, bs // 64), device="cuda") for _ in range(2))
    kd, vd = k.double()[:, 0], v.double()[:, 0]
    v = v.clone()
    raw = v.view(torch.uint8)
    early, late = P + 3, P + 200000
    if fp8:
        raw[early, 0, 7] = raw[late, 0, 9] = 0x7F
    else:
        v[early, 0, 7], v[late, 0, 9] = INF, NAN
    table = torch.arange(nb, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    pools = (k.view(nb, bs, 1, D), v.view(nb, bs, 1, D), *scales)
    pkv.get_device_errors(reset=True)
    call = pkv.paged_tree_attn_fp8 if fp8 else pkv.paged_tree_attn
    out = call(q, *pools, table, lens, L, cu, n, D ** -0.5)
    assert pkv.get_device_errors(reset=True) == 0
    assert torch.isfinite(out[:3]).all()
    x = out[3:, 0, 7].float()
    assert (torch.isnan(x) if fp8 else x == INF).all()
    assert torch.isfinite(out[:200000, 0, 9]).all() and torch.isnan(out[200000:, 0, 9]).all()
    dims = torch.tensor([d for d in range(D) if d not in (7, 9)], device="cuda")
    for i in (0, 2, 3, 63, 64, 127, 128, 70001, 199999, n - 1):
        s = (kd[:P + i + 1] @ q[i, 0].double()) * D ** -0.5
        p = torch.softmax(s, 0)
        ref, size = p @ vd[:P + i + 1], p @ vd[:P + i + 1].abs()
        assert_close(out[i, 0, dims], ref[dims], size[dims], fp8, True)


def test_the_weights_of_small_trees_keep_their_precision_beside_large_ones():
    """Few keys of either sign, so that a weight rounded to bf16 shows."""
    ctx, nodes = [2, 3, 4, 5, 6, 7, 8, 9, 10, 300], [1, 2, 3, 2, 5, 6, 7, 8, 9, 70]
    c = Case(ctx, nodes, 8, 2, seed=7)
    for bound in (70, 300):
        c.most = bound
        mask = torch.nn.functional.pad(c.mask, (0, -(-bound // 64) - c.mask.shape[1]))
        out = c.attend(pkv, tree_mask=mask)
        ref, size = c.reference()
        small = sum(nodes[:-1])
        assert_close(out[:small], ref[:small], size[:small], False, False)
        assert_close(out[small:], ref[small:], size[small:], False, True)
