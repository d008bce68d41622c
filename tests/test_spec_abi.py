"""Host-side argument checks of the calls of speculative decoding: the status codes, without a device
and without touching memory."""
import ctypes

from libbuild import build_and_import

pkv = build_and_import()
L = pkv.lib()
FAKE = ctypes.c_void_p(0x1000)    # never dereferenced: every call below fails or returns early
OTHER = ctypes.c_void_p(0x2000)
ODD = ctypes.c_void_p(0x1008)


def _tree(fp8, **kw):
    a = dict(q=FAKE, qs=2048, T=9, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, W=4, cl=FAKE, cu=FAKE,
             B=2, mq=8, maxc=100, m=FAKE, mw=1, hq=16, hkv=8, d=128, bs=256, nb=10, scale=0.088,
             ws=FAKE, wsb=1 << 30, out=FAKE)
    a.update(kw)
    scales = (a["ks"], a["vs"]) if fp8 else ()
    fn = L.pkv_paged_tree_attn_fp8 if fp8 else L.pkv_paged_tree_attn
    return fn(a["q"], a["qs"], a["T"], a["kc"], a["vc"], *scales, a["bt"], a["W"], a["cl"], a["cu"],
              a["B"], a["mq"], a["maxc"], a["m"], a["mw"], a["hq"], a["hkv"], a["d"], a["bs"],
              a["nb"], a["scale"], a["ws"], a["wsb"], a["out"], None)


def test_tree_argument_checks():
    for fp8 in (False, True):
        assert _tree(fp8, B=0) == pkv.OK and _tree(fp8, T=0) == pkv.OK and _tree(fp8, mq=0) == pkv.OK
        for kw in (dict(B=-1), dict(T=-1), dict(mq=-1), dict(maxc=-1), dict(hq=15), dict(hq=0),
                   dict(hkv=0), dict(d=0), dict(bs=0), dict(nb=0), dict(W=0), dict(qs=2040),
                   dict(scale=float("nan")), dict(scale=float("inf")), dict(mq=65), dict(mw=0),
                   dict(mw=-1), dict(q=None), dict(kc=None), dict(vc=None), dict(bt=None),
                   dict(cl=None), dict(cu=None), dict(out=None)):
            assert _tree(fp8, **kw) == pkv.ERR_INVALID_ARG, kw
        for kw in (dict(d=64), dict(bs=64), dict(bs=300), dict(nb=1 << 23), dict(T=1 << 31),
                   dict(qs=2052), dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(out=ODD)):
            assert _tree(fp8, **kw) == pkv.ERR_UNSUPPORTED, kw
    assert _tree(True, ks=None) == _tree(True, vs=None) == pkv.ERR_INVALID_ARG
    assert _tree(True, ks=ODD) == pkv.ERR_UNSUPPORTED
    assert _tree(False, nb=1 << 61) == pkv.ERR_UNSUPPORTED
    assert _tree(False, mq=(1 << 20) + 1, mw=1 << 15) == pkv.ERR_UNSUPPORTED


def test_outputs_that_overlap_inputs():
    at = ctypes.c_void_p
    last = 0x10000 + 2 * (8 * 2048 + 16 * 128)  # behind the last row of q
    for fp8 in (False, True):
        for out in (0x10000, last - 16, 0x10000 - 2 * 9 * 2048 + 16):
            assert _tree(fp8, q=at(0x10000), out=at(out)) == pkv.ERR_INVALID_ARG, hex(out)
        for out in (last, 0x10000 - 2 * 9 * 2048):  # (refused too, for want of a device or a workspace)
            assert _tree(fp8, q=at(0x10000), out=at(out), wsb=0) in (pkv.ERR_CUDA, pkv.ERR_WORKSPACE)
        huge = (1 << 62) - 8
        assert _tree(fp8, q=at(0x10000), out=at(last), qs=huge) == pkv.ERR_INVALID_ARG
    last = 0x10000 + 2 * (8 * 4104 + 4096)
    for out in (0x10000, last - 16):
        assert _append(x=at(0x10000), s=4104, q=at(out)) == pkv.ERR_INVALID_ARG
    for kw in (dict(num=OTHER), dict(cu=OTHER), dict(cl=OTHER), dict(bt=OTHER), dict(acc=OTHER),
               dict(cu=at(0x2000 - 8)), dict(acc=at(0x2000 - 36)), dict(bt=at(0x2000 - 28))):
        assert _accept(**kw) == pkv.ERR_INVALID_ARG, kw


def test_tree_workspace_of_bad_sizes():
    good = [4, 8, 16, 8, 128, 1000]
    for i, bad in ((0, -1), (1, -1), (2, 0), (2, 15), (3, 0), (4, 64), (5, -1)):
        a = list(good)
        a[i] = bad
        assert L.pkv_tree_workspace_bytes(*a) == 0, a


def _accept(**kw):
    a = dict(acc=FAKE, A=5, num=FAKE, cu=FAKE, cl=FAKE, bt=FAKE, W=4, B=2, kc=FAKE, vc=FAKE, ks=None,
             vs=None, hkv=8, d=128, bs=256, nb=10, new=OTHER)
    a.update(kw)
    return L.pkv_kv_accept(a["acc"], a["A"], a["num"], a["cu"], a["cl"], a["bt"], a["W"], a["B"],
                           a["kc"], a["vc"], a["ks"], a["vs"], a["hkv"], a["d"], a["bs"], a["nb"],
                           a["new"], None)


def test_accept_argument_checks():
    assert _accept(B=0) == pkv.OK
    for kw in (dict(B=-1), dict(A=-1), dict(hkv=0), dict(d=0), dict(bs=0), dict(nb=0), dict(W=0),
               dict(acc=None), dict(num=None), dict(cu=None), dict(cl=None), dict(bt=None),
               dict(kc=None), dict(vc=None), dict(new=None), dict(new=FAKE), dict(ks=FAKE),
               dict(vs=FAKE)):
        assert _accept(**kw) == pkv.ERR_INVALID_ARG, kw
    for kw in (dict(d=64), dict(bs=100), dict(bs=64, ks=FAKE, vs=FAKE), dict(kc=ODD), dict(vc=ODD)):
        assert _accept(**kw) == pkv.ERR_UNSUPPORTED, kw


def _append(**kw):
    a = dict(x=FAKE, s=4096, T=9, pos=FAKE, qw=FAKE, kw=FAKE, eps=1e-6, cs=FAKE, mp=100, cu=FAKE,
             cl=FAKE, bt=FAKE, W=4, B=2, q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, hq=16, hkv=8,
             d=128, bs=256, nb=10)
    a.update(kw)
    return L.pkv_qk_norm_rope_store_fp8(
        a["x"], a["s"], a["T"], a["pos"], a["qw"], a["kw"], a["eps"], a["cs"], a["mp"], a["cu"],
        a["cl"], a["bt"], a["W"], a["B"], a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["hq"],
        a["hkv"], a["d"], a["bs"], a["nb"], None)


def test_append_argument_checks():
    assert _append(T=0) == pkv.OK and _append(B=0) == pkv.OK
    for kw in (dict(B=-1), dict(T=-1), dict(hq=0), dict(hkv=0), dict(d=0), dict(bs=0), dict(nb=0),
               dict(W=0), dict(s=4088), dict(mp=0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(cu=None, T=3), dict(qw=None), dict(kw=None), dict(x=None), dict(pos=None),
               dict(cs=None), dict(cl=None), dict(bt=None), dict(q=None), dict(kc=None),
               dict(vc=None), dict(ks=None), dict(vs=None)):
        assert _append(**kw) == pkv.ERR_INVALID_ARG, kw
    for kw in (dict(d=64), dict(bs=64), dict(T=1 << 31), dict(s=4100), dict(x=ODD), dict(qw=ODD),
               dict(kw=ODD), dict(cs=ODD), dict(q=ODD), dict(kc=ODD), dict(ks=ODD)):
        assert _append(**kw) == pkv.ERR_UNSUPPORTED, kw
