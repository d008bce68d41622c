"""The operators of speculative decoding over the paged cache whose speed and precision are
followed: the attention of drafted tokens, keeping the accepted ones, and appending to the 8-bit
cache with the norms and the rotation on the way.

Every case has a plain form in elementary torch operations and, where ``own`` is true, the
calls a serving program makes of ``paged_kv_cache_208_gb300``.

  tree     paged_tree_attn / paged_tree_attn_fp8: the drafted tokens of a sequence are the nodes
           of a tree at the end of its context; each attends to the context before them and to
           the nodes that its mask names (a chain's to itself and those before it)
  accept   kv_accept: the rows of the accepted path move up behind the context, in place
  append   qk_norm_rope_store_fp8: norms and rotation of a fused projection's query and key heads,
           queries to bf16, keys and values into the 8-bit cache (e4m3, one power-of-two scale
           per 64 tokens and head)
"""
import random

import numpy as np
import torch

own = False

D = 128      # head dimension of the cache
GROUP = 64   # tokens that share a scale
E4M3_MAX = 448.0
MIN_EXP = -90  # smallest scale exponent
EPS = 1e-6
THETA = 1e6


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a few conversations, four tokens drafted in a row: the step's latency
        dict(name="tree 8x1024, chains of 4", op="tree", cache="bf16", batch=8, lo=1020, hi=1024,
             nlo=4, nhi=4, tree="chain", hq=16, hkv=8, bs=256, lens=1),
        # an ordinary full batch of ragged contexts, each with a small tree
        dict(name="tree 256 ragged, 8 nodes", op="tree", cache="bf16", batch=256, lo=100, hi=2048,
             nlo=5, nhi=8, tree="wide", hq=16, hkv=8, bs=256, lens=2),
        # one conversation over a long document, an odd number of heads in a group
        dict(name="tree 1x17188, 13 nodes 12/4", op="tree", cache="bf16", batch=1, lo=17188,
             hi=17188, nlo=13, nhi=13, tree="wide", hq=12, hkv=4, bs=256, lens=3),
        # long documents, large trees, four query heads to a KV head
        dict(name="tree 16x32768, 64 nodes 32/8", op="tree", cache="bf16", batch=16, lo=30000,
             hi=32768, nlo=48, nhi=64, tree="deep", hq=32, hkv=8, bs=256, lens=4),
        # the 8-bit cache: a few conversations, a tree each
        dict(name="tree fp8 8x1024, 16 nodes", op="tree", cache="fp8", batch=8, lo=900, hi=1024,
             nlo=16, nhi=16, tree="wide", hq=16, hkv=8, bs=256, lens=5),
        # the 8-bit cache: a full batch of ragged contexts
        dict(name="tree fp8 256 ragged, 8 nodes", op="tree", cache="fp8", batch=256, lo=100,
             hi=2048, nlo=5, nhi=8, tree="wide", hq=16, hkv=8, bs=256, lens=6),
        # many query heads on few KV heads, as a tensor-parallel rank of a large model has them
        dict(name="tree fp8 33x4999, 31 nodes 16/2", op="tree", cache="fp8", batch=33, lo=100,
             hi=4999, nlo=9, nhi=31, tree="deep", hq=16, hkv=2, bs=512, lens=7),
        # the accepted path of a few small trees: a call's latency
        dict(name="accept 8", op="accept", cache="bf16", batch=8, lo=200, hi=700, nlo=8, nhi=8,
             tree="wide", hq=16, hkv=8, bs=256, lens=8),
        # the accepted paths of a full batch of large trees
        dict(name="accept 256 of 64 nodes", op="accept", cache="bf16", batch=256, lo=100, hi=700,
             nlo=48, nhi=64, tree="deep", hq=16, hkv=8, bs=256, lens=9),
        # the same on the 8-bit cache, where a row may come to a group with another scale
        dict(name="accept fp8 256 of 64 nodes", op="accept", cache="fp8", batch=256, lo=100,
             hi=700, nlo=48, nhi=64, tree="deep", hq=16, hkv=8, bs=256, lens=10),
        # one decode step of a few conversations
        dict(name="append 8 tokens", op="append", batch=8, lo=200, hi=1024, new=1, norm=True,
             hq=16, hkv=8, bs=256, lens=11),
        # the prompts of a full batch, stored from empty
        dict(name="append 256 prompts", op="append", batch=256, lo=100, hi=1024, new=1024,
             norm=True, hq=16, hkv=8, bs=256, lens=12),
    ]


def _spread(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("tree", "tree", "tree", "accept", "append"))
    c = dict(op=op, batch=_spread(rng, 1, 256), hkv=rng.choice((1, 2, 4, 8)),
             bs=rng.choice((256, 256, 512)), lens=rng.randrange(1 << 20))
    c["hq"] = c["hkv"] * rng.choice((1, 2, 2, 3, 4, 5, 8))
    # at most 2^22 (token, KV head) pairs of the longest length: what 16 x 32768 x 8 heads has
    most = (1 << 22) // (c["batch"] * c["hkv"])
    if op == "append":
        c["norm"] = rng.random() < 0.7
        c["hi"] = _spread(rng, 1, max(1, min(16384, most // 4)))
        c["lo"] = rng.randint(0, c["hi"])
        c["new"] = 1 if rng.random() < 0.4 else _spread(rng, 2, max(2, c["hi"]))
        return c
    c["cache"] = rng.choice(("fp8", "bf16"))
    c["tree"] = rng.choice(("chain", "wide", "deep"))
    c["nhi"] = _spread(rng, 1, 64)
    c["nlo"] = rng.randint(1, c["nhi"])
    if op == "accept":
        most //= 2
    else:
        # and at most 2^30 (context token, node, query head) triples
        most = min(most, (1 << 30) // (c["batch"] * c["nhi"] * c["hq"]))
    c["hi"] = max(c["nhi"], _spread(rng, 1, max(1, min(32768, most))))
    c["lo"] = rng.randint(c["nhi"], c["hi"])
    return c


def _tree(r, kind, n):
    """Parents of n nodes (-1: the root, the token that was sampled last)."""
    if kind == "chain":
        return list(range(-1, n - 1))
    reach = 2 if kind == "deep" else 6
    return [-1] + [r.randint(max(0, i - reach), i - 1) for i in range(1, n)]


def _path(parents, node):
    path = []
    while node >= 0:
        path.append(node)
        node = parents[node]
    return path[::-1]


def _plan(c):
    """Context lengths with the new tokens, new tokens of each sequence, and for the drafts the
    tree and an accepted path of each."""
    r = random.Random(c["lens"])
    ctx = [c["hi"]] + [r.randint(c["lo"], c["hi"]) for _ in range(c["batch"] - 1)]
    if c["op"] == "append":
        if c["new"] == 1:
            return ctx, [min(1, n) for n in ctx], None, None
        return ctx, [min(n, r.randint(max(1, c["new"] // 2), c["new"])) for n in ctx], None, None
    new = [c["nhi"]] + [r.randint(c["nlo"], c["nhi"]) for _ in range(c["batch"] - 1)]
    trees = [_tree(r, c["tree"], n) for n in new]
    paths = [_path(t, r.randrange(len(t))) for t in trees]
    return ctx, new, trees, paths


def _blocks(lens, bs):
    return [-(-n // bs) for n in lens]


# ------------------------------------------------------------------------------ the inputs
def _pow2(e):
    """2^e in float32, built from its bits (e: integers in the normal range)."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _scale_of(amax):
    """The smallest power of two s >= 2^MIN_EXP with amax <= 448 s."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= E4M3_MAX / 512, e - 9, e - 8)
    return _pow2(torch.where(amax > 0, e, MIN_EXP).clamp(min=MIN_EXP))


def _pool8(nb, bs, hkv, mag, gen):
    """An e4m3 pool [nb, bs, hkv, D] with its scales [nb, hkv, bs / GROUP]."""
    codes = torch.empty((nb, bs, hkv, D), dtype=torch.uint8, device="cuda")
    scale = torch.empty((nb, hkv, bs // GROUP), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (bs * hkv * D))
    for i in range(0, nb, step):
        n = min(step, nb - i)
        x = torch.randn((n, bs // GROUP, GROUP, hkv, D), generator=gen, device="cuda") * mag
        # some groups hold larger rows than others
        x *= torch.exp(0.5 * torch.randn((n, bs // GROUP, 1, hkv, 1), generator=gen, device="cuda"))
        s = _scale_of(x.abs().amax(dim=(2, 4)))
        y = (x / s[:, :, None, :, None]).to(torch.float8_e4m3fn)
        codes[i:i + n] = y.view(torch.uint8).reshape(n, bs, hkv, D)
        scale[i:i + n] = s.transpose(1, 2)
    return codes.view(torch.float8_e4m3fn), scale


def _pool16(nb, bs, hkv, mag, gen):
    p = torch.empty((nb, bs, hkv, D), dtype=torch.bfloat16, device="cuda")
    p.normal_(generator=gen)
    return p.mul_(mag.to(torch.bfloat16))


def _tables(counts, ids):
    t = np.full((len(counts), max(counts + [1])), -1, np.int32)
    at = 0
    for i, n in enumerate(counts):
        t[i, :n] = ids[at:at + n]
        at += n
    return torch.from_numpy(t).cuda()


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _mask_words(trees, width):
    """[nodes, width] int64: bit j of a row's word w is set where the node sees node 64 w + j."""
    got = []
    for parents in trees:
        sees = []
        for i, p in enumerate(parents):
            sees.append((sees[p] if p >= 0 else 0) | 1 << i)
        got += [[s >> 64 * w & (1 << 64) - 1 for w in range(width)] for s in sees]
    return torch.from_numpy(np.array(got, np.uint64).view(np.int64)).cuda()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ctx, new, trees, paths = _plan(c)
    B, hq, hkv, bs = c["batch"], c["hq"], c["hkv"], c["bs"]
    counts = _blocks(ctx, bs)
    nb = sum(counts) + 3
    ids = np.random.RandomState(seed & 0x7fffffff).permutation(nb)  # blocks lie anywhere in the pool
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    # channels of unequal size, as projections make them; V smaller than K
    mag = torch.exp(0.5 * randn(2, hkv, D))
    s = dict(case=dict(c), max_ctx=max(ctx), scale=D ** -0.5, tables=_tables(counts, ids),
             ctx=_ints(ctx), cu=_ints([0] + list(np.cumsum(new))))
    if c.get("cache", "fp8") == "fp8":
        s["k"], s["ks"] = _pool8(nb, bs, hkv, mag[0], gen)
        s["v"], s["vs"] = _pool8(nb, bs, hkv, 0.2 * mag[1], gen)
    else:
        s["k"], s["ks"] = _pool16(nb, bs, hkv, mag[0], gen), None
        s["v"], s["vs"] = _pool16(nb, bs, hkv, 0.2 * mag[1], gen), None
    if c["op"] == "append":
        T = B if c["new"] == 1 else sum(new)
        if c["new"] == 1:
            s["cu"] = None
            s["positions"] = _ints([max(0, n - 1) for n in ctx], torch.int64)
        else:
            s["positions"] = _ints(np.concatenate(
                [np.arange(n - m, n) for n, m in zip(ctx, new)]), torch.int64)
        # the fused projection's rows; some are larger than those before them
        qkv = randn(T, (hq + 2 * hkv) * D) * torch.exp(0.3 * randn(T, 1))
        s["qkv"] = qkv.to(torch.bfloat16)
        s["qw"] = s["kw"] = None
        if c["norm"]:
            s["qw"], s["kw"] = torch.exp(0.3 * randn(2, D)).to(torch.bfloat16)
        turn = torch.arange(max(1, s["max_ctx"]), device="cuda").double()[:, None] * \
            THETA ** (-torch.arange(D // 2, device="cuda").double() / (D // 2))
        s["cos_sin"] = torch.cat((turn.cos(), turn.sin()), dim=1).float()
        return s
    s["nmax"] = max(new)
    if c["op"] == "tree":
        s["q"] = (1.5 * randn(sum(new), hq, D)).to(torch.bfloat16)
        s["mask"] = None if c["tree"] == "chain" else _mask_words(trees, -(-s["nmax"] // 64))
    else:
        most = max(len(p) for p in paths)
        s["accepted"] = _ints([p + [-1] * (most - len(p)) for p in paths])
        s["num_accepted"] = _ints([len(p) for p in paths])
    return s


# ------------------------------------------------------------------------- the plain forms
def _rows(tables, pos, bs):
    """Pool rows of positions pos [B, n]."""
    blk = tables.long().gather(1, (pos // bs).clamp(max=tables.shape[1] - 1)).clamp(min=0)
    return blk * bs + pos % bs


def _by_group(scale):
    """The scales [NB, hkv, bs / GROUP] as [NB * bs / GROUP, hkv], a copy."""
    return scale.transpose(1, 2).reshape(-1, scale.shape[1])


def _put_scales(scale, groups):
    nb, hkv, per = scale.shape
    scale.copy_(groups.view(nb, per, hkv).transpose(1, 2))


def _flat(pool):
    wide = torch.uint8 if pool.element_size() == 1 else pool.dtype
    return pool.view(wide).view(-1, pool.shape[2], D)


def _values(pool, scale, rows):
    """float32 values of pool rows: [..., hkv, D]."""
    x = _flat(pool)[rows]
    if scale is None:
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * _by_group(scale)[rows // GROUP][..., None]


def _plain_tree(s):
    c, bs = s["case"], s["case"]["bs"]
    B, hq, hkv, nmax = c["batch"], c["hq"], c["hkv"], s["nmax"]
    g, L, T = hq // hkv, s["max_ctx"], s["q"].shape[0]
    cu, ctx = s["cu"].long(), s["ctx"].long()
    n = cu[1:] - cu[:-1]
    start = ctx - n                                                  # the root's position
    node = torch.arange(nmax, device="cuda")
    live = node < n[:, None]                                         # [B, nmax]
    at = torch.where(live, cu[:-1, None] + node, T)
    # what each node sees of its tree: [B, node, node]
    if s["mask"] is None:
        tree = (node[:, None] >= node).expand(B, nmax, nmax)
    else:
        words = torch.cat((s["mask"], s["mask"][:1]))[at]            # [B, nmax, W]
        tree = (words.gather(2, (node // 64).expand(B, nmax, nmax)) >> node % 64 & 1) != 0
    tree = tree & live[:, None, :]
    pos = torch.arange(L, device="cuda")
    k_node = (pos - start[:, None]).clamp(0, nmax - 1)               # [B, L]
    seen = tree.gather(2, k_node[:, None].expand(B, nmax, L))
    ok = (pos < start[:, None])[:, None] | seen & ((pos >= start[:, None]) & (pos < ctx[:, None]))[:, None]
    valid = pos < ctx[:, None]
    rows = _rows(s["tables"], torch.where(valid, pos, 0), bs)
    q = torch.cat((s["q"], s["q"][:1]))[at].float()                  # [B, nmax, hq, D]
    q = q.view(B, nmax, hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, g * nmax, D)
    k = _values(s["k"], s["ks"], rows).permute(0, 2, 3, 1)           # [B, hkv, D, L]
    x = (torch.matmul(q, k) * s["scale"]).view(B, hkv, g, nmax, L)
    del k
    ok = ok[:, None, None]
    x = torch.where(ok, x, float("-inf"))
    top = x.amax(dim=-1, keepdim=True)
    p = torch.where(ok, torch.exp(x - top), 0.0)
    del x
    total = p.sum(dim=-1, keepdim=True)
    v = _values(s["v"], s["vs"], rows).permute(0, 2, 1, 3)           # [B, hkv, L, D]
    v = torch.where(valid[:, None, :, None], v, 0.0)
    o = torch.matmul(p.view(B, hkv, g * nmax, L), v).view(B, hkv, g, nmax, D)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, nmax, hq, D)
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), n, output_size=T)
    return {"out": o[seq, torch.arange(T, device="cuda") - cu[seq]].to(torch.bfloat16)}


def _plain_accept(s):
    bs = s["case"]["bs"]
    cu, ctx = s["cu"].long(), s["ctx"].long()
    start = ctx - (cu[1:] - cu[:-1])
    got, many = s["accepted"].long(), s["num_accepted"].long()
    place = torch.arange(got.shape[1], device="cuda")
    live = place < many[:, None]
    src = _rows(s["tables"], torch.where(live, start[:, None] + got, 0), bs)
    dst = _rows(s["tables"], torch.where(live, start[:, None] + place, 0), bs)
    new = (start + many).to(torch.int32)
    total = s["k"].shape[0] * bs
    to = torch.where(live, dst, total)
    if s["ks"] is None:
        for name in ("k", "v"):
            flat = _flat(s[name])
            moved = torch.cat((flat, flat[:1]))
            moved[to] = flat[src]
            flat.copy_(moved[:total])
        return {"k": s["k"], "v": s["v"], "context_lens": new}
    head = _rows(s["tables"], start[:, None], bs)[:, 0] // GROUP     # the group of the root
    before = torch.arange(GROUP, device="cuda")
    kept = (before < (start % GROUP)[:, None]) & (many > 0)[:, None]
    r = torch.where(kept, head[:, None] * GROUP + before, total)
    for name in ("k", "v"):
        flat, scale = _flat(s[name]), s[name + "s"]
        old = _by_group(scale)
        mine = old[src // GROUP]                                     # [B, A, hkv]
        now = torch.cat((old, torch.zeros_like(old[:1])))
        spare = total // GROUP
        now.index_reduce_(0, torch.where(live, dst // GROUP, spare).flatten(),
                          mine.flatten(0, 1), "amax")
        now = now[:spare]
        padded = torch.cat((flat, flat[:1]))
        x = padded[r].view(torch.float8_e4m3fn).float() * (old / now)[head][:, None, :, None]
        y = flat[src].view(torch.float8_e4m3fn).float() * (mine / now[dst // GROUP])[..., None]
        padded[r] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        padded[to] = y.to(torch.float8_e4m3fn).view(torch.uint8)
        flat.copy_(padded[:total])
        _put_scales(scale, now)
    return {"k": s["k"], "v": s["v"], "k_scale": s["ks"], "v_scale": s["vs"], "context_lens": new}


def _append_rows(x, pool, scale, rows, start, tables, bs):
    """Append fp32 rows x [T, hkv, D] at pool rows `rows`; the group that a sequence's new tokens
    continue keeps its rows, at the larger of its scale and the new rows' scale."""
    flat = _flat(pool)
    groups = _by_group(scale)
    total = flat.shape[0]
    size = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(dim=2)
    g = rows // GROUP
    amax = torch.zeros_like(groups).index_reduce_(0, g, size, "amax")
    writes = torch.zeros(groups.shape[0], dtype=torch.bool, device=x.device)
    writes[g] = True
    first = _rows(tables, start[:, None], bs)[:, 0] // GROUP
    begun = (start % GROUP != 0) & writes[first]
    old = torch.where(begun[:, None], groups[first], 0.0)
    now = torch.where(writes[:, None], _scale_of(amax), groups)
    now.index_reduce_(0, first, old, "amax")
    # the rows from before, at the new scale
    before = torch.arange(GROUP, device=x.device)
    keep = begun[:, None] & (before < (start % GROUP)[:, None])
    r = torch.where(keep, first[:, None] * GROUP + before, total)
    padded = torch.cat((flat, flat[:1]))
    ratio = torch.where(begun[:, None], old / now[first], 1.0)[:, None, :, None]
    moved = (padded[r].view(torch.float8_e4m3fn).float() * ratio).to(torch.float8_e4m3fn)
    padded[r] = moved.view(torch.uint8)
    y = (x / now[g][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    padded[rows] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    flat.copy_(padded[:total])
    _put_scales(scale, now)


def _plain_append(s):
    c, bs = s["case"], s["case"]["bs"]
    hq, hkv = c["hq"], c["hkv"]
    ctx, cu = s["ctx"].long(), s["cu"]
    T = s["qkv"].shape[0]
    x = s["qkv"].float().view(T, hq + 2 * hkv, D)
    turn = s["cos_sin"][s["positions"]][:, None]
    cos, sin = turn[..., :D // 2], turn[..., D // 2:]

    def rotated(y, weight):
        if weight is not None:
            y = y * torch.rsqrt(y.square().mean(dim=-1, keepdim=True) + EPS) * weight.float()
        a, b = y[..., :D // 2], y[..., D // 2:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)

    q, k = rotated(x[:, :hq], s["qw"]), rotated(x[:, hq:hq + hkv], s["kw"])
    t = torch.arange(T, device="cuda")
    if cu is None:
        start = (ctx - 1).clamp(min=0)
        if c["lo"] == 0:  # a padding row stores nothing
            t = torch.nonzero(ctx > 0)[:, 0]
        seq, pos = t, start[t]
    else:
        cu = cu.long()
        count = cu[1:] - cu[:-1]
        start = ctx - count
        seq = torch.repeat_interleave(torch.arange(len(ctx), device="cuda"), count, output_size=T)
        pos = start[seq] + t - cu[seq]
    rows = _rows(s["tables"][seq], pos[:, None], bs)[:, 0]
    _append_rows(k[t], s["k"], s["ks"], rows, start, s["tables"], bs)
    _append_rows(x[t, hq + hkv:], s["v"], s["vs"], rows, start, s["tables"], bs)
    return {"q": q.to(torch.bfloat16), "k": s["k"], "v": s["v"], "k_scale": s["ks"],
            "v_scale": s["vs"]}


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"tree": _plain_tree, "accept": _plain_accept, "append": _plain_append}[op](s)


def _own(s, op):
    import paged_kv_cache_208_gb300 as pkv
    if op == "append":
        q = pkv.qk_norm_rope_store_fp8(s["qkv"], s["positions"], s["cos_sin"], s["ctx"],
                                       s["tables"], s["k"], s["v"], s["ks"], s["vs"],
                                       s["case"]["hq"], q_norm_weight=s["qw"],
                                       k_norm_weight=s["kw"], eps=EPS, cu_seqlens=s["cu"])
        return {"q": q, "k": s["k"], "v": s["v"], "k_scale": s["ks"], "v_scale": s["vs"]}
    if op == "accept":
        new = pkv.kv_accept(s["accepted"], s["num_accepted"], s["cu"], s["ctx"], s["tables"],
                            s["k"], s["v"], k_scale=s["ks"], v_scale=s["vs"])
        got = {"k": s["k"], "v": s["v"], "context_lens": new}
        return got if s["ks"] is None else got | {"k_scale": s["ks"], "v_scale": s["vs"]}
    if s["ks"] is None:
        return {"out": pkv.paged_tree_attn(s["q"], s["k"], s["v"], s["tables"], s["ctx"],
                                           s["max_ctx"], s["cu"], s["nmax"], s["scale"],
                                           tree_mask=s["mask"])}
    return {"out": pkv.paged_tree_attn_fp8(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["tables"],
                                           s["ctx"], s["max_ctx"], s["cu"], s["nmax"],
                                           s["scale"], tree_mask=s["mask"])}


# ---------------------------------------------------------------------------------- the work
def work(case):
    c = case
    ctx, new, _, paths = _plan(c)
    hq, hkv, bs = c["hq"], c["hkv"], c["bs"]
    lists = 4 * (sum(_blocks(ctx, bs)) + 2 * len(ctx))  # block ids and lengths
    wide = 1 if c.get("cache", "fp8") == "fp8" else 2   # bytes of a cached value
    rows = 2 * hkv * D                                  # values of one token's K and V
    def scales(m):
        return 8 * hkv * (m // GROUP + 1) if wide == 1 else 0
    if c["op"] == "append":
        t = sum(new)
        moved = t * (2 * (hq + 2 * hkv) * D + 2 * hq * D + rows + 4 * D + 8)
        return {"bytes": moved + scales(t) + lists, "flops": t * D * (10 * (hq + hkv) + 2 * hkv)}
    if c["op"] == "accept":
        t = sum(1 for p in paths for j, i in enumerate(p) if i != j)
        listed_nodes = 4 * sum(len(p) for p in paths)
        return {"bytes": 2 * t * rows * wide + scales(t) + lists + listed_nodes,
                "flops": t * rows}
    nodes = sum(new)
    words = 0 if c["tree"] == "chain" else 8 * nodes * -(-max(new) // 64)
    pairs = sum((n - m) * m for n, m in zip(ctx, new))  # (context token, node)
    return {"bytes": sum(ctx) * rows * wide + scales(sum(ctx)) + 4 * nodes * hq * D + words + lists,
            "flops": 4 * pairs * hq * D}


# --------------------------------------------------------------------- exact, in 64 bits
def _two_to(e):
    """2^e in float64, exactly (pow is not, on a GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """float64 values rounded to the nearest e4m3 value, ties to even (|x| <= 448)."""
    _, e = torch.frexp(x)
    step = _two_to(e.clamp(min=-5) - 4)
    return torch.round(x / step) * step


def _sequence(s, name, b, n):
    """float64 rows 0 .. n - 1 of sequence b: [n, hkv, D]."""
    blocks = s["tables"][b, :-(-n // s["case"]["bs"])].long()
    pool, scale = s[name], s[name + "s"]
    if scale is None:
        return pool[blocks].double().flatten(0, 1)[:n]
    codes = pool.view(torch.uint8)[blocks].view(torch.float8_e4m3fn).double()
    per = scale[blocks].double().transpose(1, 2).repeat_interleave(GROUP, 1)
    return (codes * per[..., None]).flatten(0, 1)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "accept": _exact_accept, "append": _exact_append}[case["op"]](
        s, *_plan(case))


def _exact_tree(s, ctx, new, trees, _):
    c = s["case"]
    hkv = c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    t = 0
    for b, (n, m) in enumerate(zip(ctx, new)):
        sees = torch.zeros((m, n), dtype=torch.bool)
        sees[:, :n - m] = True
        for i in range(m):
            sees[i, [n - m + j for j in _path(trees[b], i)]] = True
        q = s["q"][t:t + m].double().view(m, hkv, -1, D)
        x = torch.einsum("mhgd,lhd->hgml", q, _sequence(s, "k", b, n)) * s["scale"]
        p = torch.softmax(x.masked_fill_(~sees.cuda(), float("-inf")), dim=-1)
        o = torch.einsum("hgml,lhd->mhgd", p, _sequence(s, "v", b, n))
        out[t:t + m] = o.reshape(m, -1, D)
        t += m
    return {"out": out}


def _exact_accept(s, ctx, new, _, paths):
    bs = s["case"]["bs"]
    fp8 = s["ks"] is not None
    tables = s["tables"].cpu().numpy()
    got = {"context_lens": None}
    for name in ("k", "v"):
        pool = s[name].view(torch.uint8).view(s[name].dtype).double() if fp8 else s[name].double()
        scale = s[name + "s"].double() if fp8 else None
        for b, (n, m) in enumerate(zip(ctx, new)):
            start, path = n - m, paths[b]
            def at(pos):
                return int(tables[b, pos // bs]), pos % bs
            # the rows that stay and those that move, as they were
            kept = list(range(start // GROUP * GROUP, start)) if fp8 else []
            rows = [(p, p) for p in kept] + [(start + j, start + i) for j, i in enumerate(path)]
            if not fp8:
                was = [pool[at(f)].clone() for _, f in rows]
                for (to, _), x in zip(rows, was):
                    pool[at(to)] = x
                continue
            to = torch.tensor([at(p) for p, _ in rows]).cuda()
            fr = torch.tensor([at(p) for _, p in rows]).cuda()
            was = pool[fr[:, 0], fr[:, 1]]
            mine = scale[fr[:, 0], :, fr[:, 1] // GROUP]              # [rows, hkv]
            base = rows[0][0] // GROUP
            group = torch.tensor([p // GROUP - base for p, _ in rows]).cuda()
            for g in range(int(group[-1]) + 1):
                here = group == g
                blk, off = at(max(start, (base + g) * GROUP))
                top = torch.maximum(scale[blk, :, off // GROUP], mine[here].amax(dim=0))
                pool[to[here, 0], to[here, 1]] = _round_e4m3(
                    was[here] * (mine[here] / top)[..., None])
                scale[blk, :, off // GROUP] = top
        got[name] = pool
        if fp8:
            got[name + "_scale"] = scale
    return got


def _exact_append(s, ctx, new, *_):
    c, bs = s["case"], s["case"]["bs"]
    hq, hkv = c["hq"], c["hkv"]
    T = s["qkv"].shape[0]
    heads = s["qkv"].double().view(T, -1, D)
    angle = torch.complex(*s["cos_sin"].double()[s["positions"]].split(D // 2, dim=1))[:, None]

    def turned(x, w):
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(dim=2, keepdim=True) / D + EPS) * w.double()
        z = torch.complex(x[..., :D // 2].contiguous(), x[..., D // 2:].contiguous()) * angle
        return torch.cat((z.real, z.imag), dim=2)

    got = {"q": turned(heads[:, :hq], s["qw"])}
    sources = {"k": turned(heads[:, hq:hq + hkv], s["kw"]), "v": heads[:, hq + hkv:]}
    tables = s["tables"].cpu().numpy()
    for name, x in sources.items():
        codes = s[name].view(torch.uint8).view(torch.float8_e4m3fn).double()
        scale = s[name + "s"].double()
        t = 0
        for b, (n, m) in enumerate(zip(ctx, new)):
            pos, end = n - m, n
            row = b if c["new"] == 1 else t
            while pos < end:  # one group of GROUP positions at a time
                stop = min(end, (pos // GROUP + 1) * GROUP)
                blk, off = int(tables[b, pos // bs]), pos % bs
                g, base = off // GROUP, off // GROUP * GROUP
                part = x[row:row + stop - pos]
                top = part.abs().amax(dim=(0, 2)).clamp(min=1e-300)
                e = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(min=-1000)
                e = torch.where(top > E4M3_MAX * _two_to(e), e + 1, e)
                e = torch.where(top <= E4M3_MAX * _two_to(e - 1), e - 1, e)
                sc = _two_to(e.clamp(min=MIN_EXP))
                if off > base:
                    sc = torch.maximum(sc, scale[blk, :, g])
                    ratio = (scale[blk, :, g] / sc)[None, :, None]
                    codes[blk, base:off] = _round_e4m3(codes[blk, base:off] * ratio)
                codes[blk, off:off + stop - pos] = _round_e4m3(part / sc[None, :, None])
                scale[blk, :, g] = sc
                row += stop - pos
                pos = stop
            t += m
        got[name], got[name + "_scale"] = codes, scale
    return got
