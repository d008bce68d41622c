"""Host-side argument checks of the 8-bit cache, attention weight and eviction entry points: the
status codes, without a device and without touching memory."""
import ctypes

from libbuild import build_and_import

pkv = build_and_import()
L = pkv.lib()
FAKE = ctypes.c_void_p(0x1000)    # never dereferenced: every call below fails or returns early
OTHER = ctypes.c_void_p(0x2000)
ODD = ctypes.c_void_p(0x1008)


def _store(**kw):
    a = dict(k=FAKE, ks=1024, v=FAKE, vs=1024, cu=FAKE, ctx=FAKE, bt=FAKE, W=4, B=2, T=9, kc=FAKE,
             vc=FAKE, ksc=FAKE, vsc=FAKE, hkv=8, d=128, bs=256, nb=10)
    a.update(kw)
    return L.pkv_kv_store_fp8(a["k"], a["ks"], a["v"], a["vs"], a["cu"], a["ctx"], a["bt"], a["W"],
                              a["B"], a["T"], a["kc"], a["vc"], a["ksc"], a["vsc"], a["hkv"],
                              a["d"], a["bs"], a["nb"], None)


def test_store_argument_checks():
    assert _store(T=0) == pkv.OK and _store(B=0) == pkv.OK
    assert _store(cu=None, T=0, B=0) == pkv.OK
    for kw in (dict(B=-1), dict(T=-1), dict(hkv=0), dict(d=0), dict(bs=0), dict(nb=0), dict(W=0),
               dict(ks=1016), dict(vs=512), dict(cu=None, T=3), dict(k=None), dict(ctx=None),
               dict(bt=None), dict(kc=None), dict(ksc=None), dict(vsc=None)):
        assert _store(**kw) == pkv.ERR_INVALID_ARG, kw
    for kw in (dict(d=64), dict(bs=64), dict(bs=300), dict(ks=1028), dict(k=ODD), dict(vc=ODD),
               dict(ksc=ODD), dict(T=1 << 31)):
        assert _store(**kw) == pkv.ERR_UNSUPPORTED, kw


def _gather(**kw):
    a = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, W=4, cu=FAKE, N=2, T=9, ko=FAKE, vo=FAKE,
             hkv=8, d=128, bs=256, nb=10)
    a.update(kw)
    return L.pkv_kv_gather_fp8(a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["W"], a["cu"],
                               a["N"], a["T"], a["ko"], a["vo"], a["hkv"], a["d"], a["bs"],
                               a["nb"], None)


def test_gather_argument_checks():
    assert _gather(T=0) == pkv.OK and _gather(N=0) == pkv.OK
    for kw in (dict(N=-1), dict(T=-1), dict(hkv=0), dict(W=0), dict(nb=0), dict(kc=None),
               dict(vs=None), dict(cu=None), dict(ko=None), dict(vo=None)):
        assert _gather(**kw) == pkv.ERR_INVALID_ARG, kw
    for kw in (dict(d=64), dict(bs=128), dict(ko=ODD), dict(kc=ODD), dict(T=1 << 31)):
        assert _gather(**kw) == pkv.ERR_UNSUPPORTED, kw


def _decode8(**kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, W=4, cl=FAKE, B=2, maxc=100,
             hq=16, hkv=8, d=128, bs=256, nb=10, scale=0.088, ns=0, wi=None, wis=0, wo=None, wos=0,
             ws=FAKE, wsb=1 << 30, out=FAKE)
    a.update(kw)
    return L.pkv_paged_decode_attn_fp8(
        a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["W"], a["cl"], a["B"], a["maxc"],
        a["hq"], a["hkv"], a["d"], a["bs"], a["nb"], a["scale"], a["ns"], a["wi"], a["wis"],
        a["wo"], a["wos"], a["ws"], a["wsb"], a["out"], None)


def _decode16(**kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, W=4, cl=FAKE, B=2, maxc=100, hq=16, hkv=8, d=128,
             bs=256, nb=10, scale=0.088, ns=0, wi=FAKE, wis=100, wo=FAKE, wos=100, ws=FAKE,
             wsb=1 << 30, out=FAKE)
    a.update(kw)
    return L.pkv_paged_decode_attn_weights(
        a["q"], a["kc"], a["vc"], a["bt"], a["W"], a["cl"], a["B"], a["maxc"], a["hq"], a["hkv"],
        a["d"], a["bs"], a["nb"], a["scale"], a["ns"], a["wi"], a["wis"], a["wo"], a["wos"],
        a["ws"], a["wsb"], a["out"], None)


def test_decode_argument_checks():
    for call in (_decode8, _decode16):
        assert call(B=0) == pkv.OK
        for kw in (dict(B=-1), dict(maxc=-1), dict(ns=-1), dict(hq=12), dict(hkv=0), dict(W=0),
                   dict(nb=0), dict(scale=float("inf")), dict(q=None), dict(cl=None),
                   dict(out=None), dict(wo=FAKE, wos=99), dict(wo=FAKE, wos=100, wi=FAKE, wis=7)):
            assert call(**kw) == pkv.ERR_INVALID_ARG, (call.__name__, kw)
        for kw in (dict(d=64), dict(bs=128), dict(nb=1 << 24), dict(q=ODD), dict(kc=ODD),
                   dict(out=ODD)):
            assert call(**kw) == pkv.ERR_UNSUPPORTED, (call.__name__, kw)
    assert _decode8(ks=None) == pkv.ERR_INVALID_ARG
    assert _decode8(vs=ODD) == pkv.ERR_UNSUPPORTED
    assert _decode16(wo=None) == pkv.ERR_INVALID_ARG


def test_decode_weights_in_needs_weights_out():
    assert _decode8(wi=FAKE, wis=100, wo=None) == pkv.ERR_INVALID_ARG


def test_workspace_queries():
    for n in (L.pkv_decode_fp8_workspace_bytes(4, 16, 8, 64, 300, 0, 0),
              L.pkv_decode_fp8_workspace_bytes(0, 16, 8, 128, 300, 0, 1),
              L.pkv_decode_weights_workspace_bytes(4, 15, 8, 128, 300, 0),
              L.pkv_decode_weights_workspace_bytes(4, 16, 8, 128, -1, 0)):
        assert n == 0
    plain = L.pkv_decode_fp8_workspace_bytes(4, 16, 8, 128, 300, 0, 0)
    full = L.pkv_decode_fp8_workspace_bytes(4, 16, 8, 128, 300, 0, 1)
    assert plain == full == 0 or full >= plain + 4 * 16 * 300 * 4   # 0 without a device


def _evict(**kw):
    a = dict(w=FAKE, ws=100, cl=FAKE, B=2, maxc=100, budget=10, recent=2, bt=FAKE, W=4, dt=OTHER,
             DW=1, kc=FAKE, vc=FAKE, ks=None, vs=None, hkv=8, d=128, bs=256, nb=10, kept=FAKE,
             wo=OTHER, wos=10, nl=OTHER)
    a.update(kw)
    return L.pkv_kv_evict(a["w"], a["ws"], a["cl"], a["B"], a["maxc"], a["budget"], a["recent"],
                          a["bt"], a["W"], a["dt"], a["DW"], a["kc"], a["vc"], a["ks"], a["vs"],
                          a["hkv"], a["d"], a["bs"], a["nb"], a["kept"], a["wo"], a["wos"],
                          a["nl"], None)


def test_evict_argument_checks():
    assert _evict(B=0) == pkv.OK
    for kw in (dict(B=-1), dict(maxc=-1), dict(budget=0), dict(recent=-1), dict(recent=11),
               dict(W=0), dict(DW=0), dict(hkv=0), dict(nb=0), dict(ws=99), dict(wos=9),
               dict(w=None), dict(cl=None), dict(bt=None), dict(dt=None), dict(kc=None),
               dict(kept=None), dict(nl=None), dict(ks=FAKE), dict(dt=FAKE), dict(nl=FAKE),
               dict(wo=FAKE)):
        assert _evict(**kw) == pkv.ERR_INVALID_ARG, kw
    for kw in (dict(d=64), dict(bs=100), dict(ks=FAKE, vs=FAKE, bs=64), dict(kc=ODD),
               dict(B=1 << 28, hkv=64)):
        assert _evict(**kw) == pkv.ERR_UNSUPPORTED, kw


def test_take_argument_checks():
    assert L.pkv_bm_take(None, 1, FAKE) == pkv.ERR_INVALID_ARG
    bm = pkv.BlockManager(4, 8)
    assert L.pkv_bm_take(bm._h, -1, FAKE) == pkv.ERR_INVALID_ARG
    assert L.pkv_bm_take(bm._h, 1, None) == pkv.ERR_INVALID_ARG
    assert L.pkv_bm_take(bm._h, 0, None) == pkv.OK
