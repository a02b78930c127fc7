"""Argument rules of the attention operators: each answers before any CUDA work. Runs without a GPU."""
import ctypes

import pytest
import torch

import weight_only_quantized_wq4_gb300 as wq4

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(16)]     # aligned stand-ins, never dereferenced
ODD, HALF = ctypes.c_void_p(0x10001), ctypes.c_void_p(0x10008)
REFUSED = (wq4.ERR_INVALID, wq4.ERR_ALIGN, wq4.ERR_UNSUPPORTED, wq4.ERR_WORKSPACE)


@pytest.fixture(scope="module")
def clib():
    wq4.build()
    return wq4.load_library()


def cache(k=P[10], v=P[11], kp=16 * 8 * 64, kt=8 * 64, kh=64, vp=16 * 8 * 64, vt=8 * 64, vh=64, pages=7, page_size=16):
    return wq4.KvCache(getattr(k, "value", k), getattr(v, "value", v), kp, kt, kh, vp, vt, vh, pages, page_size)


def test_append_rules(clib):
    def call(q=P[0], qt=1024, qh=64, k=P[1], kt=1024, kh=64, v=P[2], vt=1024, vh=64, T=5, Hq=16, Hk=8, D=64, dt=0, qw=P[3],
             kw=P[4], eps=1e-6, pos=P[5], freq=P[6], rot=64, inter=0, out=P[7], ot=1024, oh=64, c=None, slots=P[8]):
        return clib.wq4_rope_append(q, qt, qh, k, kt, kh, v, vt, vh, T, Hq, Hk, D, dt, qw, kw, eps, pos, freq, rot, inter, out,
                                    ot, oh, ctypes.byref(c or cache()), slots, None)

    assert call() not in REFUSED and call(dt=1) not in REFUSED and call(inter=1) not in REFUSED
    assert call(rot=0, pos=None, freq=None) not in REFUSED and call(qw=None, kw=None) not in REFUSED
    assert call(q=None, Hq=0, qw=None, out=None) not in REFUSED
    assert call(q=ctypes.c_void_p(0x10002), qt=1025, rot=14) not in REFUSED         # 2-byte rows are allowed
    assert call(T=1, qt=0, kt=0, vt=0, ot=0) not in REFUSED                         # strides that are never used
    assert call(T=0, q=None, k=None, v=None, pos=None, freq=None, out=None, slots=None) == wq4.OK
    for bad in (dict(T=-1), dict(Hq=-1), dict(Hk=0), dict(D=0), dict(dt=2), dict(dt=-1), dict(rot=-2), dict(rot=3), dict(rot=66),
                dict(inter=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(q=None), dict(k=None),
                dict(v=None), dict(qw=None), dict(kw=None), dict(pos=None), dict(freq=None), dict(out=None), dict(slots=None),
                dict(qt=63), dict(qh=63), dict(kt=63), dict(vh=63), dict(ot=0), dict(oh=-64), dict(qt=1 << 41),
                dict(c=cache(k=None)), dict(c=cache(v=None)), dict(c=cache(pages=0)), dict(c=cache(page_size=0)),
                dict(c=cache(kt=63)), dict(c=cache(vp=0))):
        assert call(**bad) == wq4.ERR_INVALID, bad
    for bad in (dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(qw=ODD), dict(kw=ODD), dict(out=ODD), dict(pos=ctypes.c_void_p(0x10004)),
                dict(slots=ctypes.c_void_p(0x10004)), dict(freq=ctypes.c_void_p(0x10002)), dict(c=cache(k=ODD)), dict(c=cache(v=ODD))):
        assert call(**bad) == wq4.ERR_ALIGN, bad
    for bad in (dict(D=1025, qh=2000, kh=2000, vh=2000, oh=2000, qt=9999, kt=9999, vt=9999, ot=9999),
                dict(c=cache(pages=1 << 28))):
        assert call(**bad) == wq4.ERR_UNSUPPORTED, bad


def test_attention_rules(clib):
    def call(q=P[0], qt=1024, qh=64, table=P[1], ld=9, width=9, starts=P[2], ctx=P[3], B=3, T=5, most=4, Hq=16, Hk=8, D=64, dt=0,
             scale=0.1, mask=P[4], words=1, out=P[5], ot=1024, oh=64, lse=P[6], ws=P[7], bytes=1 << 30, c=None):
        return clib.wq4_tree_attention(q, qt, qh, ctypes.byref(c or cache()), table, ld, width, starts, ctx, B, T, most, Hq, Hk, D,
                                       dt, scale, mask, words, out, ot, oh, lse, ws, bytes, None)

    assert call() not in REFUSED and call(dt=1) not in REFUSED and call(mask=None, words=0) not in REFUSED
    assert call(lse=None) not in REFUSED and call(scale=-1.0) not in REFUSED and call(c=cache(page_size=48, kp=1 << 15, vp=1 << 15)) not in REFUSED
    for none in (dict(B=0), dict(T=0)):
        assert call(q=None, table=None, starts=None, ctx=None, out=None, ws=None, bytes=0, **none) == wq4.OK
    for bad in (dict(B=-1), dict(T=-1), dict(most=0), dict(Hq=0), dict(Hk=0), dict(Hq=15), dict(D=0), dict(dt=2), dict(q=None),
                dict(table=None), dict(starts=None), dict(ctx=None), dict(out=None), dict(ld=8), dict(width=0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(words=0), dict(most=65), dict(qt=60), dict(oh=56),
                dict(c=cache(k=None)), dict(c=cache(kh=56))):
        assert call(**bad) == wq4.ERR_INVALID, bad
    for bad in (dict(q=HALF), dict(out=HALF), dict(ws=HALF), dict(qt=1028), dict(oh=68), dict(table=ODD), dict(starts=ODD),
                dict(ctx=ODD), dict(mask=ctypes.c_void_p(0x10004)), dict(lse=ODD), dict(c=cache(k=HALF)), dict(c=cache(vh=68)),
                dict(c=cache(kp=16 * 512 + 4))):
        assert call(**bad) == wq4.ERR_ALIGN, bad
    wide = dict(qt=8192, qh=512, ot=8192, oh=512, c=cache(kp=1 << 17, kt=4096, kh=512, vp=1 << 17, vt=4096, vh=512))
    many = dict(Hq=65536, Hk=1, c=cache(kh=64, vh=64))
    for bad in (dict(most=1 << 15, words=1 << 9, **many), dict(D=63), dict(D=264, **wide), dict(most=(1 << 20) + 1, words=1 << 20), dict(c=cache(page_size=24)),
                dict(c=cache(page_size=8)), dict(c=cache(kp=1 << 39))):
        assert call(**bad) == wq4.ERR_UNSUPPORTED, bad


def test_attention_workspace_rules(clib):
    n = ctypes.c_size_t(0)
    assert clib.wq4_tree_attention_workspace_bytes(3, 4, 16, 8, 64, None) == wq4.ERR_INVALID
    for args, want in (((-1, 4, 16, 8, 64), wq4.ERR_INVALID), ((3, 0, 16, 8, 64), wq4.ERR_INVALID),
                       ((3, 4, 15, 8, 64), wq4.ERR_INVALID), ((3, 4, 16, 8, 100), wq4.ERR_UNSUPPORTED)):
        assert clib.wq4_tree_attention_workspace_bytes(*args, ctypes.byref(n)) == want


def test_verify_rules(clib):
    def call(x=P[0], ld=1000, tok=P[1], par=P[2], starts=P[3], B=3, T=9, most=4, V=1000, dt=2, q=P[4], ldq=1000, heat=P[5], u=P[6],
             uf=P[7], acc=P[8], path=P[9], ldp=3, nxt=P[12]):
        return clib.wq4_verify_drafts(x, ld, tok, par, starts, B, T, most, V, dt, q, ldq, heat, u, uf, acc, path, ldp, nxt, None)

    assert call() not in REFUSED and call(q=None, ldq=0) not in REFUSED and call(heat=None) not in REFUSED
    assert call(x=ctypes.c_void_p(0x10002), dt=0, ld=1001) not in REFUSED and call(most=1, ldp=1) not in REFUSED
    assert call(T=0, x=None, tok=None, par=None, u=None) not in REFUSED
    assert call(B=0, x=None, tok=None, par=None, starts=None, u=None, uf=None, acc=None, path=None, nxt=None) == wq4.OK
    for bad in (dict(B=-1), dict(T=-1), dict(most=0), dict(V=0), dict(dt=3), dict(dt=-1), dict(x=None), dict(tok=None), dict(par=None),
                dict(starts=None), dict(u=None), dict(uf=None), dict(acc=None), dict(path=None), dict(nxt=None), dict(ld=999),
                dict(ldq=999), dict(ldp=2), dict(most=1, ldp=0), dict(ld=1 << 41)):
        assert call(**bad) == wq4.ERR_INVALID, bad
    for bad in (dict(x=ctypes.c_void_p(0x10002)), dict(x=ODD, dt=0), dict(tok=ctypes.c_void_p(0x10004)), dict(par=ODD), dict(starts=ODD),
                dict(q=ODD), dict(heat=ODD), dict(u=ODD), dict(uf=ODD), dict(acc=ODD), dict(path=ODD), dict(nxt=ctypes.c_void_p(0x10004))):
        assert call(**bad) == wq4.ERR_ALIGN, bad
    for bad in (dict(V=400001, ld=400001, ldq=400001), dict(most=(1 << 20) + 1, ldp=1 << 20)):
        assert call(**bad) == wq4.ERR_UNSUPPORTED, bad


def test_binding_refuses_cpu_tensors_and_wrong_types(clib):
    x, c = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 16, 4, 64, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int64)
    i = torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(64, dtype=torch.uint8)
    for call in (lambda: wq4.rope_append(x, x, x, c, c, n), lambda: wq4.rope_append(x, x.float(), x, c, c, n),
                 lambda: wq4.rope_append(x[0], x[0], x[0], c, c, n),
                 lambda: wq4.tree_attention(x, c, c, i[None], i, i, workspace=ws),
                 lambda: wq4.tree_attention(x, c, c, i[None], i, i), lambda: wq4.tree_attention(x.double(), c, c, i[None], i, i, workspace=ws),
                 lambda: wq4.verify_drafts(x[0], n, i, i, x, x, 2), lambda: wq4.verify_drafts(x[0].long(), n, i, i, x, x, 2)):
        with pytest.raises(ValueError):
            call()
