"""The paged-cache operators whose speed and precision are followed: the 8-bit cache (store,
gather, decode attention) and eviction by accumulated attention weight.

Every case has a plain form in elementary torch operations and, where ``own`` is true, the
calls a serving program makes of ``paged_kv_cache_208_gb300``.

  store    kv_store_fp8: append a batch's new K/V rows to an e4m3 cache that holds one
           power-of-two scale per 64 tokens and head
  decode   paged_decode_attn_fp8: one query token per sequence over that cache
  gather   kv_gather_fp8: cached rows back to packed bf16, as a prefill over a cached prefix
           reads them
  weights  paged_decode_attn_weights / paged_decode_attn_fp8(weights=...): decode attention
           that also adds each cached token's softmax weight to an accumulator
  evict    kv_evict: keep the recent tokens and those with the largest accumulated weight,
           compact their rows into new blocks
"""
import random

import numpy as np
import torch

own = False

D = 128      # head dimension of the cache
GROUP = 64   # tokens that share a scale
E4M3_MAX = 448.0
MIN_EXP = -90  # smallest scale exponent


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a few conversations: eight single rows, a call's latency
        dict(name="store 8 tokens", op="store", batch=8, lo=200, hi=1024, new=1, hq=16, hkv=8,
             bs=256, lens=1),
        # the prompts of a full batch, stored from empty (all of each context is new)
        dict(name="store 256 prompts", op="store", batch=256, lo=100, hi=1024, new=1024, hq=16,
             hkv=8, bs=256, lens=2),
        # a few conversations, the step's latency
        dict(name="decode 8x1024", op="decode", cache="fp8", batch=8, lo=1024, hi=1024, hq=16,
             hkv=8, bs=256, lens=3),
        # an ordinary full batch of ragged contexts
        dict(name="decode 256 ragged", op="decode", cache="fp8", batch=256, lo=100, hi=2048,
             hq=16, hkv=8, bs=256, lens=4),
        # many query heads on few KV heads, as a tensor-parallel rank of a large model has them
        dict(name="decode 33x4999 16/2", op="decode", cache="fp8", batch=33, lo=100, hi=4999,
             hq=16, hkv=2, bs=512, lens=5),
        # long documents
        dict(name="decode 32x32768", op="decode", cache="fp8", batch=32, lo=32768, hi=32768,
             hq=16, hkv=8, bs=256, lens=6),
        # a short cached prefix before a follow-up question
        dict(name="gather 2x300", op="gather", batch=2, lo=250, hi=300, hq=16, hkv=8, bs=256,
             lens=7),
        # the cached prefixes of a batch of prompts
        dict(name="gather 64x2048..2816", op="gather", batch=64, lo=2304, hi=2816, hq=16,
             hkv=8, bs=256, lens=8),
        # heavy-hitter statistics of a small batch on the 8-bit cache
        dict(name="weights fp8 8x1024", op="weights", cache="fp8", batch=8, lo=900, hi=1024,
             hq=16, hkv=8, bs=256, lens=9),
        # heavy-hitter statistics of a full batch on the bf16 cache
        dict(name="weights bf16 256 ragged", op="weights", cache="bf16", batch=256, lo=100,
             hi=2048, hq=16, hkv=8, bs=256, lens=10),
        # one conversation of an 8-bit cache cut down to a quarter
        dict(name="evict fp8 4x4096", op="evict", cache="fp8", batch=4, lo=3000, hi=4096, hq=16,
             hkv=8, bs=256, budget=1024, recent=128, lens=11),
        # long documents cut down to a quarter
        dict(name="evict bf16 16x32768", op="evict", cache="bf16", batch=16, lo=30000, hi=32768,
             hq=16, hkv=8, bs=256, budget=8192, recent=512, lens=12),
    ]


def _spread(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("store", "decode", "gather", "weights", "evict"))
    c = dict(op=op, batch=_spread(rng, 1, 256), hkv=rng.choice((1, 2, 4, 8)),
             bs=rng.choice((256, 256, 512)), lens=rng.randrange(1 << 20))
    c["hq"] = c["hkv"] * rng.choice((1, 2, 2, 3, 4, 5, 8))
    # at most 2^23 (token, head) pairs of the longest length: what 32 x 32768 x 8 heads has,
    # half of it for the operators that move more bytes of each
    most = (1 << 23) // (c["batch"] * c["hkv"])
    most //= {"store": 6, "gather": 2, "evict": 2}.get(op, 1)
    c["hi"] = _spread(rng, 1, max(1, min(32768, most)))
    c["lo"] = rng.randint(0, c["hi"])
    if op == "store":
        c["new"] = 1 if rng.random() < 0.4 else _spread(rng, 2, max(2, c["hi"]))
    if op in ("decode", "weights", "evict"):
        c["cache"] = "fp8" if op == "decode" else rng.choice(("fp8", "bf16"))
    if op == "evict":
        c["budget"] = _spread(rng, 1, max(1, c["hi"] // 2))
        c["recent"] = rng.randint(0, c["budget"])
    return c


def _lengths(c):
    """Context lengths, and new tokens of each sequence (store)."""
    r = random.Random(c["lens"])
    ctx = [c["hi"]] + [r.randint(c["lo"], c["hi"]) for _ in range(c["batch"] - 1)]
    if c["op"] != "store":
        return ctx, None
    if c["new"] == 1:
        return ctx, [min(1, n) for n in ctx]
    return ctx, [min(n, r.randint(max(1, c["new"] // 2), c["new"])) for n in ctx]


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
        s = _scale_of(x.abs().amax(dim=(2, 4)))
        y = (x / s[:, :, None, :, None]).to(torch.float8_e4m3fn)
        codes[i:i + n] = y.view(torch.uint8).reshape(n, bs, hkv, D)
        scale[i:i + n] = s.transpose(1, 2)
    return codes.view(torch.float8_e4m3fn), scale


def _pool16(nb, bs, hkv, mag, gen):
    p = torch.empty((nb, bs, hkv, D), dtype=torch.bfloat16, device="cuda")
    p.normal_(generator=gen)
    return p.mul_(mag.to(torch.bfloat16))


def _tables(counts, width, ids):
    t = np.full((len(counts), width), -1, np.int32)
    at = 0
    for i, n in enumerate(counts):
        t[i, :n] = ids[at:at + n]
        at += n
    return torch.from_numpy(t).cuda()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ctx, new = _lengths(c)
    B, hq, hkv, bs = c["batch"], c["hq"], c["hkv"], c["bs"]
    counts = _blocks(ctx, bs)
    width = max(counts + [1])
    used = sum(counts)
    kept = _blocks([min(n, c["budget"]) for n in ctx], bs) if c["op"] == "evict" else []
    nb = used + sum(kept) + 3
    ids = np.random.RandomState(seed & 0x7fffffff).permutation(nb)  # blocks lie anywhere in the pool
    # channels of unequal size, as projections make them; V smaller than K
    mag = torch.exp(0.5 * torch.randn((2, hkv, D), generator=gen, device="cuda"))
    s = dict(case=dict(c), max_ctx=max(ctx), scale=D ** -0.5,
             tables=_tables(counts, width, ids),
             ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"))
    if c.get("cache", "fp8") == "fp8":
        s["k"], s["ks"] = _pool8(nb, bs, hkv, mag[0], gen)
        s["v"], s["vs"] = _pool8(nb, bs, hkv, 0.2 * mag[1], gen)
    else:
        s["k"], s["ks"] = _pool16(nb, bs, hkv, mag[0], gen), None
        s["v"], s["vs"] = _pool16(nb, bs, hkv, 0.2 * mag[1], gen), None
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    if c["op"] == "store":
        T = B if c["new"] == 1 else sum(new)
        # views into a fused projection's rows; some rows are larger than those before them
        qkv = randn(T, (hq + 2 * hkv) * D) * torch.exp(0.3 * randn(T, 1))
        s["qkv"] = qkv.to(torch.bfloat16)
        s["knew"] = s["qkv"][:, hq * D:(hq + hkv) * D].view(T, hkv, D)
        s["vnew"] = s["qkv"][:, (hq + hkv) * D:].view(T, hkv, D)
        s["cu"] = None
        if c["new"] != 1:
            s["cu"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    if c["op"] in ("decode", "weights"):
        s["q"] = (1.5 * randn(B, hq, D)).to(torch.bfloat16)
        s["workspace"] = None
        if own:
            import paged_kv_cache_208_gb300 as pkv
            sizes = (B, hq, hkv, D, s["max_ctx"])
            s["workspace"] = pkv.decode_weights_workspace(*sizes) if s["ks"] is None else \
                pkv.decode_fp8_workspace(*sizes, weights=c["op"] == "weights")
    if c["op"] == "gather":
        s["total"] = sum(ctx)
        s["cu"] = torch.tensor([0] + list(np.cumsum(ctx)), dtype=torch.int32, device="cuda")
    if c["op"] in ("weights", "evict"):
        shape = (B, hkv, max(1, s["max_ctx"]))
        # what some steps have left there: a heavy tail, and tokens that nothing looked at
        w = torch.exp(2.0 * randn(*shape))
        s["weights"] = torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.05, 0.0, w)
    if c["op"] == "weights":
        s["weights_out"] = torch.zeros(shape, device="cuda")
    if c["op"] == "evict":
        s["dst"] = _tables(kept, max(kept + [1]), ids[used:])
    return s


# ------------------------------------------------------------------------- the plain forms
def _rows(tables, pos, bs):
    """Pool rows of positions pos [B, n] (rows of no block: row 0)."""
    blk = tables.long().gather(1, (pos // bs).clamp(max=tables.shape[1] - 1)).clamp(min=0)
    return blk * bs + pos % bs


def _scales_at(scale, rows, bs):
    """The scale of each pool row and head: [..., hkv]."""
    return scale.transpose(1, 2).reshape(-1, scale.shape[1])[rows // GROUP]


def _values(pool, scale, rows, bs):
    """float32 values of pool rows: [..., hkv, D]."""
    nb, _, hkv, _ = pool.shape
    if scale is None:
        return pool.view(nb * bs, hkv, D)[rows].float()
    x = pool.view(torch.uint8).view(nb * bs, hkv, D)[rows].view(torch.float8_e4m3fn).float()
    return x * _scales_at(scale, rows, bs)[..., None]


def _store_one(x, pool, scale, seq, pos, rows, start, tables, bs):
    """Append rows x [T, hkv, D] at pool rows `rows`; the group that a sequence's new tokens
    continue keeps its rows, at the larger of its scale and the new rows' scale."""
    nb, _, hkv, _ = pool.shape
    flat = pool.view(torch.uint8).view(nb * bs, hkv, D)
    groups = scale.transpose(1, 2).reshape(-1, hkv)          # [nb * bs / GROUP, hkv], a copy
    x = x.float()
    size = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(dim=2)
    g = rows // GROUP
    amax = torch.zeros_like(groups).index_reduce_(0, g, size, "amax")
    # groups with rows from before the call
    first = _rows(tables, start[:, None], bs)[:, 0] // GROUP
    begun = start % GROUP != 0
    writes = torch.zeros(groups.shape[0], dtype=torch.bool, device=x.device)
    writes[g] = True
    begun = begun & writes[first]
    old = torch.where(begun[:, None], groups[first], 0.0)
    need = _scale_of(amax)
    now = torch.where(writes[:, None], need, groups)
    now.index_reduce_(0, first, old, "amax")
    # the rows from before, at the new scale
    r = first[:, None] * GROUP + torch.arange(GROUP, device=x.device)
    keep = begun[:, None] & (torch.arange(GROUP, device=x.device) < (start % GROUP)[:, None])
    before = flat[r]
    ratio = torch.where(begun[:, None], old / now[first], 1.0)[:, None, :, None]
    moved = (before.view(torch.float8_e4m3fn).float() * ratio).to(torch.float8_e4m3fn)
    spare = torch.zeros_like(flat[:1])
    padded = torch.cat((flat, spare))
    padded[torch.where(keep, r, nb * bs)] = moved.view(torch.uint8)
    y = (x / now[g][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    padded[rows] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    flat.copy_(padded[:nb * bs])
    scale.copy_(now.view(nb, bs // GROUP, hkv).transpose(1, 2))


def _plain_store(s):
    bs = s["case"]["bs"]
    ctx, cu = s["ctx"].long(), s["cu"]
    T = s["knew"].shape[0]
    t = torch.arange(T, device="cuda")
    if cu is None:
        count = (ctx > 0).long()
        seq, start = t, ctx - count
        pos = start
        live = count > 0
        if s["case"]["lo"] == 0:  # a padding row stores nothing
            t = torch.nonzero(live)[:, 0]
            seq, pos = t, start[t]
    else:
        cu = cu.long()
        count = cu[1:] - cu[:-1]
        start = ctx - count
        seq = torch.repeat_interleave(torch.arange(len(ctx), device="cuda"), count, output_size=T)
        pos = start[seq] + t - cu[seq]
    rows = _rows(s["tables"][seq], pos[:, None], bs)[:, 0]
    _store_one(s["knew"][t], s["k"], s["ks"], seq, pos, rows, start, s["tables"], bs)
    _store_one(s["vnew"][t], s["v"], s["vs"], seq, pos, rows, start, s["tables"], bs)
    return {"k": s["k"], "v": s["v"], "k_scale": s["ks"], "v_scale": s["vs"]}


def _plain_attend(s):
    """Softmax attention of every query head over its sequence's rows: (out, p [B, hkv, g, L])."""
    c, bs = s["case"], s["case"]["bs"]
    B, hq, hkv = c["batch"], c["hq"], c["hkv"]
    L = max(1, s["max_ctx"])
    pos = torch.arange(L, device="cuda")
    valid = pos < s["ctx"].long()[:, None]                          # [B, L]
    rows = _rows(s["tables"], torch.where(valid, pos, 0), bs)
    q = s["q"].float().view(B, hkv, hq // hkv, D)
    k = _values(s["k"], s["ks"], rows, bs).permute(0, 2, 3, 1)      # [B, hkv, D, L]
    x = torch.matmul(q, k) * s["scale"]
    del k
    ok = valid[:, None, None, :]
    x = torch.where(ok, x, float("-inf"))
    top = x.amax(dim=-1, keepdim=True)
    p = torch.where(ok, torch.exp(x - top), 0.0)
    total = p.sum(dim=-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    v = _values(s["v"], s["vs"], rows, bs).permute(0, 2, 1, 3)      # [B, hkv, L, D]
    v = torch.where(valid[:, None, :, None], v, 0.0)
    return torch.matmul(p, v).reshape(B, hq, D).to(torch.bfloat16), p, valid


def _plain_gather(s):
    bs = s["case"]["bs"]
    cu = s["cu"].long()
    t = torch.arange(s["total"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(cu) - 1, device="cuda"), cu[1:] - cu[:-1],
                                  output_size=s["total"])
    rows = _rows(s["tables"][seq], (t - cu[seq])[:, None], bs)[:, 0]
    return {n: _values(s[n], s[n + "s"], rows, bs).to(torch.bfloat16) for n in ("k", "v")}


def _plain_evict(s):
    c, bs = s["case"], s["case"]["bs"]
    B, hkv, budget = c["batch"], c["hkv"], c["budget"]
    ctx = s["ctx"].long()
    n = ctx.clamp(max=budget)                                        # rows kept of each sequence
    L = max(1, s["max_ctx"])
    pos = torch.arange(L, device="cuda")
    w = s["weights"]
    valid = pos < ctx[:, None]
    recent = valid & (pos >= (ctx - c["recent"])[:, None])
    key = torch.where(recent[:, None], float("inf"), w)
    key = torch.where(valid[:, None], key, float("-inf"))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    place = torch.arange(budget, device="cuda")
    order = order[..., :budget] if L >= budget else torch.nn.functional.pad(order, (0, budget - L))
    live = (place < n[:, None])[:, None].expand(B, hkv, budget)
    kept = torch.where(live, order, 1 << 30).sort(dim=-1).values
    at = torch.where(live, kept, 0)
    kept = torch.where(live, kept, -1).to(torch.int32)
    weights = torch.where(live, w.gather(2, at), 0.0)
    src = _rows(s["tables"], at.reshape(B, -1), bs).view(B, hkv, budget)
    dst = _rows(s["dst"], place.expand(B, budget), bs)[:, None].expand(B, hkv, budget)
    head = torch.arange(hkv, device="cuda")[None, :, None]
    nb = s["k"].shape[0]
    for name in ("k", "v"):
        pool, scale = s[name], s[name + "s"]
        wide = torch.uint8 if scale is not None else torch.bfloat16
        flat = pool.view(wide).view(nb * bs, hkv, D)
        x = flat[src, head]                                          # [B, hkv, budget, D]
        if scale is not None:
            groups = scale.transpose(1, 2).reshape(-1, hkv)
            mine = torch.where(live, groups[src // GROUP, head], 0.0)
            pad = -budget % GROUP
            new = torch.nn.functional.pad(mine, (0, pad)).view(B, hkv, -1, GROUP).amax(dim=-1)
            ratio = torch.where(live, mine / new.repeat_interleave(GROUP, -1)[..., :budget], 0.0)
            x = (x.view(torch.float8_e4m3fn).float() * ratio[..., None]).to(torch.float8_e4m3fn)
            x = x.view(torch.uint8)
            first = dst[:, :, ::GROUP] // GROUP
            groups = torch.cat((groups, groups[:1]))
            groups[torch.where(live[:, :, ::GROUP], first, nb * bs // GROUP), head] = new
            scale.copy_(groups[:-1].view(nb, bs // GROUP, hkv).transpose(1, 2))
        padded = torch.cat((flat, flat[:1]))
        padded[torch.where(live, dst, nb * bs), head] = x
        flat.copy_(padded[:nb * bs])
    return _evicted(s, kept, weights, n.to(torch.int32))


def _evicted(s, kept, weights, n):
    got = {"k": s["k"], "v": s["v"], "kept": kept, "weights": weights, "context_lens": n}
    if s["ks"] is not None:
        got |= {"k_scale": s["ks"], "v_scale": s["vs"]}
    return got


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "store":
        return _plain_store(s)
    if op == "gather":
        return _plain_gather(s)
    if op == "evict":
        return _plain_evict(s)
    out, p, valid = _plain_attend(s)
    if op == "decode":
        return {"out": out}
    s["weights_out"].copy_(torch.where(valid[:, None], s["weights"] + p.sum(dim=2),
                                       s["weights_out"]))
    return {"out": out, "weights": s["weights_out"]}


def _own(s, op):
    import paged_kv_cache_208_gb300 as pkv
    if op == "store":
        pkv.kv_store_fp8(s["knew"], s["vnew"], s["ctx"], s["tables"], s["k"], s["v"], s["ks"],
                         s["vs"], cu_seqlens=s["cu"])
        return {"k": s["k"], "v": s["v"], "k_scale": s["ks"], "v_scale": s["vs"]}
    if op == "gather":
        k, v = pkv.kv_gather_fp8(s["k"], s["v"], s["ks"], s["vs"], s["tables"], s["cu"],
                                 s["total"])
        return {"k": k, "v": v}
    if op == "evict":
        kept, weights, n = pkv.kv_evict(s["weights"], s["ctx"], s["max_ctx"], s["tables"],
                                        s["dst"], s["case"]["budget"], s["case"]["recent"],
                                        s["k"], s["v"], k_scale=s["ks"], v_scale=s["vs"])
        return _evicted(s, kept, weights, n)
    if s["ks"] is not None:
        w = {}
        if op == "weights":
            w = dict(weights=s["weights"], weights_out=s["weights_out"])
        out = pkv.paged_decode_attn_fp8(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["tables"],
                                        s["ctx"], s["max_ctx"], s["scale"],
                                        workspace=s["workspace"], **w)
    else:
        out = pkv.paged_decode_attn_weights(s["q"], s["k"], s["v"], s["tables"], s["ctx"],
                                            s["max_ctx"], s["scale"], s["weights"],
                                            weights_out=s["weights_out"],
                                            workspace=s["workspace"])
    return {"out": out} if op == "decode" else {"out": out, "weights": s["weights_out"]}


# ---------------------------------------------------------------------------------- the work
def work(case):
    c = case
    ctx, new = _lengths(c)
    hq, hkv, bs = c["hq"], c["hkv"], c["bs"]
    n = sum(ctx)
    lists = 4 * (sum(_blocks(ctx, bs)) + len(ctx))      # block ids and lengths
    wide = 1 if c.get("cache", "fp8") == "fp8" else 2   # bytes of a cached value
    def scales(m):
        return 8 * hkv * (m // GROUP + 1) if wide == 1 else 0
    rows = 2 * hkv * D                                  # values of one token's K and V
    if c["op"] == "store":
        t = sum(new)
        return {"bytes": t * rows * 3 + scales(t) + lists, "flops": 2 * t * rows}
    if c["op"] == "gather":
        return {"bytes": n * rows * 3 + scales(n) + lists, "flops": n * rows}
    if c["op"] == "evict":
        m = sum(min(x, c["budget"]) for x in ctx)
        moved = m * rows * wide * 2 + 2 * scales(m)
        return {"bytes": n * hkv * 4 + m * hkv * 8 + moved + lists, "flops": n * hkv}
    attend = n * rows * wide + scales(n) + 4 * c["batch"] * hq * D + lists
    more = 8 * n * hkv if c["op"] == "weights" else 0
    return {"bytes": attend + more, "flops": 4 * n * hq * D}


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
    bs = s["case"]["bs"]
    blocks = s["tables"][b, :-(-n // bs)].long()
    pool, scale = s[name], s[name + "s"]
    if scale is None:
        return pool[blocks].double().flatten(0, 1)[:n]
    codes = pool.view(torch.uint8)[blocks].view(torch.float8_e4m3fn).double()
    per = scale[blocks].double().transpose(1, 2).repeat_interleave(GROUP, 1)
    return (codes * per[..., None]).flatten(0, 1)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    ctx, new = _lengths(case)
    return {"store": _exact_store, "gather": _exact_gather, "decode": _exact_decode,
            "weights": _exact_decode, "evict": _exact_evict}[case["op"]](s, ctx, new)


def _exact_gather(s, ctx, _):
    got = {}
    for name in ("k", "v"):
        rows = [_sequence(s, name, b, n) for b, n in enumerate(ctx) if n]
        got[name] = torch.cat(rows) if rows else torch.zeros((0, s["case"]["hkv"], D)).double()
    return got


def _exact_decode(s, ctx, _):
    c = s["case"]
    out = torch.zeros((c["batch"], c["hq"], D), dtype=torch.float64, device="cuda")
    weights = None
    if c["op"] == "weights":
        weights = s["weights_out"].double()
    for b, n in enumerate(ctx):
        if not n:
            continue
        q = s["q"][b].double().view(c["hkv"], -1, D)
        x = torch.einsum("hgd,lhd->hgl", q, _sequence(s, "k", b, n)) * s["scale"]
        p = torch.softmax(x, dim=-1)
        out[b] = torch.einsum("hgl,lhd->hgd", p, _sequence(s, "v", b, n)).reshape(-1, D)
        if weights is not None:
            weights[b, :, :n] = s["weights"][b, :, :n].double() + p.sum(dim=1)
    return {"out": out} if weights is None else {"out": out, "weights": weights}


def _exact_store(s, ctx, new):
    c, bs = s["case"], s["case"]["bs"]
    got = {}
    tables = s["tables"].cpu().numpy()
    for name in ("k", "v"):
        codes = s[name].view(torch.uint8).view(torch.float8_e4m3fn).double()
        scale = s[name + "s"].double()
        x = s[name + "new"].double()
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


def _exact_evict(s, ctx, _):
    c, bs = s["case"], s["case"]["bs"]
    B, hkv, budget = c["batch"], c["hkv"], c["budget"]
    kept = np.full((B, hkv, budget), -1, np.int64)
    weights = np.zeros((B, hkv, budget))
    w = s["weights"].cpu().numpy().astype(np.float64)
    for b, n in enumerate(ctx):
        last = max(0, n - c["recent"])
        for h in range(hkv):
            if n <= budget:
                at = np.arange(n)
            else:
                best = np.argsort(-w[b, h, :last], kind="stable")[:budget - (n - last)]
                at = np.sort(np.concatenate([best, np.arange(last, n)]))
            kept[b, h, :len(at)] = at
            weights[b, h, :len(at)] = w[b, h, at]
    got = {"kept": None, "context_lens": None, "weights": torch.from_numpy(weights)}
    tables, dst = s["tables"].cpu().numpy(), s["dst"].cpu().numpy()
    for name in ("k", "v"):
        pool, scale = s[name], s[name + "s"]
        codes = pool.view(torch.uint8).view(pool.dtype).double()
        new = None if scale is None else scale.double()
        for b, n in enumerate(ctx):
            m = min(n, budget)
            for h in range(hkv if m else 0):
                at = kept[b, h, :m]
                row = torch.from_numpy(tables[b, at // bs].astype(np.int64) * bs + at % bs).cuda()
                to = np.arange(m)
                to = torch.from_numpy(dst[b, to // bs].astype(np.int64) * bs + to % bs).cuda()
                x = pool.view(torch.uint8).view(pool.dtype)[row // bs, row % bs, h].double() \
                    if scale is None else _codes_at(pool, row, bs, h)
                if scale is not None:
                    mine = scale[row // bs, h, row % bs // GROUP].double()
                    most = torch.stack([p.max() for p in mine.split(GROUP)])
                    x = _round_e4m3(x * (mine / most.repeat_interleave(GROUP)[:m])[:, None])
                    first = to[::GROUP]
                    new[first // bs, h, first % bs // GROUP] = most
                codes[to // bs, to % bs, h] = x
        got[name] = codes
        if new is not None:
            got[name + "_scale"] = new
    return got


def _codes_at(pool, row, bs, h):
    return pool.view(torch.uint8)[row // bs, row % bs, h].view(torch.float8_e4m3fn).double()
